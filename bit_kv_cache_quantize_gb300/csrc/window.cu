// window.cu -- attention within a sliding window whose first tokens stay
// visible: one query per sequence on the packed decode kernel
// (decode_kernel.cuh, WIN), several on the row kernels (rows_kernel.cuh,
// MQ_WINDOW).
//
// A row at position p sees the tokens t <= p with t < n_sinks or
// t > p - window.  Both kernels walk only the closed tiles that hold a token
// some row of the unit sees (win_tiles), so the cost follows the window, not
// the context, and the tiles in between may have been freed.
// Eight query heads per KV head, 8 KV heads, K4/V2: 256 ragged sequences, window
// 4096, 338 us, bound as the whole context's decode is by the warp tensor
// cores and the unpacking (4.7 ns per record); 8 sequences 12 us, latency.
#include "decode_kernel.cuh"
#include "rows_kernel.cuh"

namespace kvarn {

// Raw open tile of (b, h) for a window's single query: len % 128 tokens, 16
// per warp and pass.  With a short window the open tile is on the critical
// path (the whole context's decode hides it behind many packed tiles), so it
// runs on the warp tensor cores like the packed tiles: QK with the queries
// exact in rows 0-7, PV with the probabilities' 16-bit high parts in rows
// 0-7 and low parts in rows 8-15.  The keys go from global memory straight
// into B fragments (the lane's 64 contiguous bytes of its token; the
// contraction order is free), the values through shared memory for the
// transposed load.  Hidden tokens are not loaded, so what they hold (an
// infinity, a NaN) reaches nothing.  A visible infinity would meet weights in
// two parts, one of them 0 or negative, and become NaN: where a warp's sums are
// not finite it takes such values out, repeats the product and adds them by
// their whole weights (the test of the sums costs 64 operations a thread).
template <typename E, int NW>
__device__ void win_tail_chunk(const WindowParams& p, int b, int h, int len, const WinTiles& wt, unsigned char* smem,
                               float* part, int64_t part_stride) {
  const int n = len % T;
  constexpr int NB = 8 / NW;  // 16-token blocks per warp
  const uint32_t sbase = smem_u32(smem);
  smem += ((sbase + 127u) & ~127u) - sbase;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
  const int G = p.G, t0 = len - n;
  const E* kt = static_cast<const E*>(p.tail) + (((int64_t)b * p.num_kv_heads + h) * 2 + 0) * (T * D);
  const E* vt = kt + T * D;
  if (!kcheck(kt, 2 * T * D * sizeof(E), p.tail, (size_t)p.batch * p.num_kv_heads * 2 * T * D * sizeof(E), p.err))
    return;
  auto seen = [&](int t) { return t < n && (t0 + t < p.n_sinks || t0 + t >= wt.lo); };
  unsigned char* vs = smem + warp * (NB * 16 * D * 2);  // this warp's value rows, 256 bytes each
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int r = 2 * q + (lane >> 4), c = lane & 15, t = 16 * (warp + NW * i) + r;
      unsigned char* dst = vs + (16 * i + r) * 256 + ((c ^ (r & 7)) << 4);
      if (seen(t)) cp_async16(dst, vt + t * D + 8 * c);
      else *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
    }
  // k-block kb of QK takes channels 32 j + 4 kb .. + 3 from lane j
  const E* qb = static_cast<const E*>(p.q) + ((int64_t)b * p.num_q_heads + (int64_t)h * G + g) * D + 32 * j;
  uint32_t qa[16];
  {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = g < G ? reinterpret_cast<const uint4*>(qb)[i] : make_uint4(0u, 0u, 0u, 0u);
      qa[4 * i] = v.x; qa[4 * i + 1] = v.y; qa[4 * i + 2] = v.z; qa[4 * i + 3] = v.w;
    }
  }
  const float sl2 = p.scale * LOG2E;
  float sc[2 * NB][2];  // scores of query g, tokens 16 (warp + NW i) + 8 nb + 2 j, + 1
  float m = -INFINITY;
#pragma unroll
  for (int nb = 0; nb < 2 * NB; ++nb) {
    const int tb = 16 * (warp + NW * (nb >> 1)) + 8 * (nb & 1), t = tb + g;
    uint32_t kw[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = seen(t) ? reinterpret_cast<const uint4*>(kt + t * D + 32 * j)[i] : make_uint4(0u, 0u, 0u, 0u);
      kw[4 * i] = v.x; kw[4 * i + 1] = v.y; kw[4 * i + 2] = v.z; kw[4 * i + 3] = v.w;
    }
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < 8; ++kb) {
      const uint32_t a[4] = {qa[2 * kb], 0u, qa[2 * kb + 1], 0u};
      mma16816<E>(c, a, kw[2 * kb], kw[2 * kb + 1]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool in = seen(tb + 2 * j + e);
      sc[nb][e] = in ? c[e] * sl2 : -INFINITY;
      m = fmaxf(m, in ? fmaxf(sc[nb][e], SEEN) : -INFINITY);
    }
  }
  m = quad_max(m);
  const float nm = m == -INFINITY ? 0.f : m;  // a warp that sees nothing keeps zero weights
  float l, acc[16][4];
  uint32_t odd = 0;  // tokens of this warp with values taken out
  cp_async_wait_all();
  __syncwarp();
#pragma unroll 1
  for (bool again = false;; again = true) {
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      uint32_t pa[4];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        const float x = ex2_ftz(sc[2 * i + nb][0] - nm), y = ex2_ftz(sc[2 * i + nb][1] - nm);
        l += x + y;
        uint16_t xh, xl, yh, yl;
        split_hl<E>(x, xh, xl);
        split_hl<E>(y, yh, yl);
        pa[2 * nb] = pack2(xh, yh);
        pa[2 * nb + 1] = pack2(xl, yl);
      }
      const int r = lane & 15;
#pragma unroll
      for (int np = 0; np < 8; ++np) {
        uint32_t v[4];
        ldmatrix_x4_trans(v, vs + (16 * i + r) * 256 + (((2 * np + (lane >> 4)) ^ (r & 7)) << 4));
        mma16816<E>(acc[2 * np], pa, v[0], v[1]);
        mma16816<E>(acc[2 * np + 1], pa, v[2], v[3]);
      }
    }
    float zero = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      zero += (acc[i][0] + acc[i][2]) * 0.f + (acc[i][1] + acc[i][3]) * 0.f;
    if (again || !__any_sync(0xffffffffu, zero != 0.f)) break;
    __syncwarp();  // every lane has read the rows
#pragma unroll 1
    for (int k = 0; k < NB * 8; ++k) {
      const int r = 2 * k + (lane >> 4);
      uint4* x = reinterpret_cast<uint4*>(vs + r * 256 + (((lane & 15) ^ (r & 7)) << 4));
      uint4 y = *x;
      bool bad = false;
      y.x = finite_pair<E>(y.x, bad); y.y = finite_pair<E>(y.y, bad);
      y.z = finite_pair<E>(y.z, bad); y.w = finite_pair<E>(y.w, bad);
      if (bad) {
        *x = y;
        odd |= 1u << r;
      }
    }
    odd = __reduce_or_sync(0xffffffffu, odd);
    if (!odd) break;  // the weights or the sums themselves are not finite
    __syncwarp();
  }
#pragma unroll 1
  for (; odd; odd &= odd - 1) {
    const int k = __ffs(odd) - 1, t = 16 * (warp + NW * (k >> 4)) + (k & 15);
    float s = 0.f;
    if (g < G)
#pragma unroll 1
      for (int c = 0; c < 32; ++c) s = fmaf(to_f(qb[c]), to_f(kt[t * D + 32 * j + c]), s);
    const float w = ex2_ftz(quad_sum(s) * (p.scale * LOG2E) - nm);
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = to_f(vt[t * D + 8 * i + 2 * j + e]);
        if (!isfinite(x)) acc[i][e] += w * x;
      }
  }
  l = quad_sum(l);
  __syncthreads();  // the value rows become the merge area
  DecMerge<NW>& mg = *reinterpret_cast<DecMerge<NW>*>(smem);
  if (j == 0) { mg.m[warp][g] = m; mg.l[warp][g] = l; }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    *reinterpret_cast<float2*>(&mg.acc[warp][g][8 * i + 2 * j]) =
        make_float2(acc[i][0] + acc[i][2], acc[i][1] + acc[i][3]);
  __syncthreads();
  for (int i = tid; i < G * D; i += 32 * NW) {
    const int gg = i / D, c = i % D;
    float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, mg.m[w][gg]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = mg.m[w][gg] == -INFINITY ? 0.f : ex2_ftz(mg.m[w][gg] - M);
      L += f * mg.l[w][gg];
      A += f * mg.acc[w][gg][c];
    }
    float* o = part + gg * part_stride;
    if (c == 0) { o[0] = M; o[1] = L; }
    o[PACC + c] = A;
  }
}

// The open tiles of a WIN_SPLIT call, in front of the packed tiles' kernel: as
// one more CTA of that kernel each would hold half an SM's shared memory for
// its whole latency (39 us of 356 at 256 ragged sequences); here four share an
// SM, and the packed tiles start under them.
template <typename E>
__global__ void __launch_bounds__(128, 4) win_tail_kernel(WindowParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  allow_dependents();
  const int h = blockIdx.x, b = blockIdx.y, len = p.seq_lens[b];
  if (len <= 0 || len > T * p.max_blocks || len % T == 0) return;
  const WinTiles wt = win_tiles(len / T, max(0, len - p.window), p.n_sinks);
  float* o = part_ptr(p, b, h, p.n_chunks, 0);
  if (!kcheck(o, (size_t)p.G * PART * sizeof(float), p.ws, (size_t)p.ws_bytes, p.err)) return;
  win_tail_chunk<E, 4>(p, b, h, len, wt, smem_raw, o, PART);
}

// Shared address of `p` in the CTA of rank `rank` of this cluster, and a load from it.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float cluster_ld(uint32_t a) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(x) : "r"(a) : "memory");
  return x;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t a) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(a)
               : "memory");
  return x;
}
__device__ __forceinline__ void cluster_sync_all() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

// A cluster holds the chunks of one (sequence, KV head), the open tile last.
// One warp per query reads the partials of all of them through distributed
// shared memory and writes the result: no workspace, no second launch (3 us of
// a 12 us call at 8 x 4096 tokens).
template <int NW, typename O>
__device__ void win_cluster_merge(const WindowParams& p, int b, int h, const float* part, O* out) {
  const int n = p.n_chunks, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  cluster_sync_all();
  const int g = blockIdx.x * NW + warp;  // the cluster spans the grid's x: blockIdx.x is the rank
  if (g < p.G) {
    const float* row = part + g * PART;
    float m = lane <= n ? cluster_ld(cluster_addr(row, lane)) : -INFINITY, M = m;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (M != -INFINITY) {
      const float f = m == -INFINITY ? -1.f : exp2f(m - M);  // -1: nothing seen, what the partial holds is not defined
      float L = m == -INFINITY ? 0.f : f * cluster_ld(cluster_addr(row + 1, lane));
#pragma unroll
      for (int s = 16; s >= 1; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
      float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i <= n; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        if (fi < 0.f) continue;  // (a weight of 0 counts: 0 times an infinity is NaN)
        const float4 a = cluster_ld4(cluster_addr(row + PACC + 4 * lane, i));
        float* z = i == n ? y : x;
        z[0] += fi * a.x; z[1] += fi * a.y; z[2] += fi * a.z; z[3] += fi * a.w;
      }
      fwht128(x, lane);
      const float inv = 1.f / L;
      o = make_float4((x[0] * INV_SQRT_D + y[0]) * inv, (x[1] * INV_SQRT_D + y[1]) * inv,
                      (x[2] * INV_SQRT_D + y[2]) * inv, (x[3] * INV_SQRT_D + y[3]) * inv);
    }
    O* dst = out + ((int64_t)b * p.num_q_heads + h * p.G + g) * D + 4 * lane;
    if (kcheck(dst, 4 * sizeof(O), out, (size_t)p.batch * p.num_q_heads * D * sizeof(O), p.err)) store4(dst, o);
  }
  cluster_sync_all();  // the partials stay until every warp has read them
}

namespace {
template <typename E, int KBITS, int VBITS, typename O>
cudaError_t launch_window_cluster_t(const WindowParams& p, int batch, O* out, cudaStream_t s) {
  auto kernel = decode_packed_kernel<E, KBITS, VBITS, 4, WIN_CLUSTER, O>;
  const size_t smem = sizeof(DecSmem<KBITS, VBITS, 4>) + 128;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = smem_attr_once(attr_done, (const void*)kernel, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.n_chunks + 1;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_chunks + 1, p.num_kv_heads, batch);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, out);
}

template <typename E, int KBITS, int VBITS, int NW, typename O>
cudaError_t launch_window_decode_t(const WindowParams& p, int batch, O* out, cudaStream_t s) {
  const size_t smem = sizeof(DecSmem<KBITS, VBITS, NW>) + 128;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = smem_attr_once(attr_done, (const void*)decode_packed_kernel<E, KBITS, VBITS, NW, WIN_SPLIT>, (int)smem);
  if (e != cudaSuccess) return e;
  win_tail_kernel<E><<<dim3(p.num_kv_heads, batch), 128, 8 * 16 * D * 2 + 128, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after_smem(decode_packed_kernel<E, KBITS, VBITS, NW, WIN_SPLIT>, dim3(p.n_chunks, p.num_kv_heads, batch),
                        dim3(32 * NW), smem, s, p, static_cast<float*>(nullptr));
  if (e != cudaSuccess) return e;
  const int64_t warps = (int64_t)batch * p.num_q_heads;
  return launch_after(combine_kernel<true, O>, dim3((unsigned)((warps + 3) / 4)), dim3(128), s, p, 1, batch, out);
}

template <typename E, typename O>
cudaError_t launch_window_decode_p(const WindowParams& p, int batch, O* out, cudaStream_t s) {
  static_assert(sizeof(DecSmem<2, 2, 4>) >= 8 * 16 * D * 2 && sizeof(DecSmem<2, 2, 4>) >= sizeof(DecMerge<4>) &&
                    sizeof(DecSmem<2, 2, 8>) >= sizeof(DecMerge<8>),
                "the open tile's buffers fit");
  if (p.cluster) {
    if (p.k_bits == 2) return launch_window_cluster_t<E, 2, 2>(p, batch, out, s);
    return p.v_bits == 4 ? launch_window_cluster_t<E, 4, 4>(p, batch, out, s)
                         : launch_window_cluster_t<E, 4, 2>(p, batch, out, s);
  }
  if (p.v_bits == 4) return launch_window_decode_t<E, 4, 4, 4>(p, batch, out, s);
  const bool small = p.chunk_tiles <= 8;
  if (p.k_bits == 2)
    return small ? launch_window_decode_t<E, 2, 2, 4>(p, batch, out, s)
                 : launch_window_decode_t<E, 2, 2, 8>(p, batch, out, s);
  return small ? launch_window_decode_t<E, 4, 2, 4>(p, batch, out, s)
               : launch_window_decode_t<E, 4, 2, 8>(p, batch, out, s);
}
}  // namespace

cudaError_t launch_window_decode(const WindowParams& p, int dtype, int batch, void* out, bool out16, cudaStream_t s) {
  if (dtype == KVARN_DTYPE_BF16)
    return out16 ? launch_window_decode_p<__nv_bfloat16>(p, batch, static_cast<__nv_bfloat16*>(out), s)
                 : launch_window_decode_p<__nv_bfloat16>(p, batch, static_cast<float*>(out), s);
  return out16 ? launch_window_decode_p<__half>(p, batch, static_cast<__half*>(out), s)
               : launch_window_decode_p<__half>(p, batch, static_cast<float*>(out), s);
}

cudaError_t launch_window_multiquery(const RowsParams& p, int dtype, int batch, void* out, bool out16, cudaStream_t s) {
  if (dtype == KVARN_DTYPE_BF16)
    return out16 ? launch_rows<MQ_WINDOW, __nv_bfloat16>(p, batch, static_cast<__nv_bfloat16*>(out), s)
                 : launch_rows<MQ_WINDOW, __nv_bfloat16>(p, batch, static_cast<float*>(out), s);
  return out16 ? launch_rows<MQ_WINDOW, __half>(p, batch, static_cast<__half*>(out), s)
               : launch_rows<MQ_WINDOW, __half>(p, batch, static_cast<float*>(out), s);
}

}  // namespace kvarn
