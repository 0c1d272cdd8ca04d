// rows_kernel.cuh -- attention of many query rows over the packed paged cache,
// for window chunks (window.cu) and drafted trees (tree.cu): operands and
// formulas of the causal multi-query kernel (rows_common.cuh), another
// pipeline.
//
// What bounds the causal kernel is the chain of one tile (4.6 K cycles, of
// which the tensor pipe works 2.2 K): its softmax warps find the row maxima,
// write the scores back, exchange the maxima, and only then form the weights.
// Here a tile takes one pass: the weights are taken against the reference m
// the row has so far, a whole number that need not be the maximum (see
// RQ_RAISE).  A warp with a row that has seen nothing yet looks for the maximum
// first.  Eight warps take 16 rows each, in fragments (see the softmax below).
// What bounds it now: the exponentials and their bookkeeping, 3 K of the 4.15 K
// cycles of a tile, on SMs that issue for the unpacking warps at the same
// time (58 % of the issue slots, 78 % of the shared-memory cycles with two
// passes, 53 % with one); for short chunks also the CTA's ends: 9 K cycles from
// its start to the first MMA and 9 K for the result rows, both first touches of
// memory and of code.  32 sequences x 64 drafted nodes behind 16 K tokens:
// 1.84 ms; 32 chunks of 128 tokens, window 2048: 0.79 ms, 0.1 of it raw.
// Tried and left: a thread per row and half tile (8 % slower: every score's
// four scales from shared memory); the scales aK and aV packed in one word (no
// gain); K~ unpacked while the queries still move to tensor memory (no gain);
// two groups of warps on alternate tiles, m handed from tile to tile (4.3 K
// cycles a tile); half tiles as units of QK and PV (6 K: an MMA of 80 columns
// takes as long as one of 128); 16 softmax warps, either layout (2.4 ms: 64
// registers a thread).
// Warps 8-11 unpack K~, 12-14 V~ (their first thread refills the record
// stages), one thread of warp 15 issues the MMAs: sixteen warps keep 128
// registers a thread.  K~, V~ and the scores are double-buffered.
//
// PASSES: 2 = high and low parts of Q' (fp16) and P~ (bf16), products to
// 2^-16 and better: fp32 results and fp16 results.  1 = high parts only, for
// bf16 results, which are rounded by up to 2^-8 of themselves: a weight is off
// by up to 2^-8 of itself (P~; averaged over the tokens) and a channel of Q' by
// up to 2^-11, an eighth of the half step that the query's own bf16 values are
// off; row statistics and accumulators stay fp32.  It halves the tensor work:
// 32 x 128 chunks 790 us against 855 with two passes, 32 x 64 trees 1676
// against 1858, 8 x 27 ragged trees 58.4 against 62.5; error 0.00195 of the
// results' rms against 0.00166.  The zero-points' sum beta and the row sum l then use the rounded weights too
// (through bV / aV and 1 / aV).  With an exact l a weight's error would act on
// its whole value, not on its distance from the result (0.0024 against
// 0.0019 of a result's rms, 0.0017 of it the result's own rounding); with an
// exact beta it would act on the codes alone, which are not centred, and the
// channel that their common part rotates to would collect sqrt(128) times it.
//
// The raw tokens (open tile, drafted nodes) are a kernel of their own in front
// (raw_rows_kernel, two CTAs per SM): its CTAs overlap each other's loads, and
// this kernel starts while they run.  With a single chunk of packed tiles the
// epilogue merges the raw partial, rotates back and writes the result; with
// more, partial rows go to the workspace and mq_combine_kernel finishes.
#pragma once

#include "rows_common.cuh"

namespace kvarn {
namespace {

constexpr int RQ_ST = 256;  // softmax threads (8 warps); then the K~, V~ and issuing warps
constexpr int RQ_KTHREADS = 128, RQ_VTHREADS = 96;
constexpr int RQ_THREADS = RQ_ST + RQ_KTHREADS + RQ_VTHREADS + 32;
constexpr int RQ_WK = RQ_ST / 32, RQ_WV = RQ_WK + 4, RQ_WI = RQ_WV + 3;  // their first warps
constexpr int RQ_WARPS = RQ_THREADS / 32;
constexpr int RQ_REC = 3 * (rec_bytes(4) + rec_bytes(2));  // record stages: 3 (K4/V2, K2/V2) or 2 (K4/V4)
template <int KBITS, int VBITS>
constexpr int rq_stages() { return VBITS == 4 ? 2 : 3; }
static_assert(2 * (rec_bytes(4) + rec_bytes(4)) <= RQ_REC && 3 * head_rec(2, 2) <= RQ_REC, "record stages fit");

struct RQSmem {
  alignas(128) unsigned char qa_lo[QA_BYTES];
  alignas(128) unsigned char kt[2][KT_BYTES];  // also: query staging at the start, result rows at the end
  alignas(128) unsigned char vt[2][VT_BYTES];
  alignas(128) unsigned char rec[RQ_REC];
  alignas(16) float ka[2][T], kb[2][T], va[2][T], vb[2][T], vi[2][T];  // vi: 1 / aV (one pass)
  alignas(16) float row_m[MQ_ROWS], row_l[MQ_ROWS];  // row_m: the rows' largest |Q'| until the tiles are done
  uint32_t qmax, qmin;  // bits of the largest and smallest of the rows' largest |Q'|
  uint64_t rec_full[3], rec_empty[3], kt_full[2], vt_full[2], s_full[2], p_full[2], pv_done[2], fin;
  uint32_t tmem;
  uint32_t rec_ok[3], kt_ok[2];  // the tile in this stage has a block in range
};
// Exponents (log2) of the weights p = 2^(score - reference).  bf16 and fp32
// hold them up to 2^127 and every relative precision is the same at any size,
// so the reference need not be the maximum: it is raised once weights pass
// 2^RQ_RAISE, and at once where they would pass 2^RQ_EMAX (x aV <= 448, x 128
// tokens x 128 tiles of a chunk stay far below 2^127).
constexpr float RQ_RAISE = 30.f, RQ_EMAX = 60.f;
// Largest |Q'| (log2 units per unit of K) a row is scaled for; more is not
// told from infinity.  Ratio of rows' largest from which a block scale is not
// fine enough: 2^12 leaves the smallest row 2^-18 of its own largest.
constexpr float RQ_QMAX = 0x1p100f, RQ_SPREAD = 4096.f;
constexpr int RQ_ROWF = 132;  // floats per staged row
static_assert(MQ_ROWS * RQ_ROWF * 4 <= 2 * KT_BYTES && 16 * 8 * RQ_ROWF * 4 <= 2 * KT_BYTES, "staging fits the K~ buffers");
static_assert(sizeof(RQSmem) + 128 <= 232448, "one CTA per SM");

// 2^-d for a whole number d >= 0, exact (0 past the normal range).
__device__ __forceinline__ float pow2_neg(float d) { return d > 126.f ? 0.f : __int_as_float((127 - (int)d) << 23); }

// Barrier of n threads that also tells all of them whether every one is ok.
__device__ __forceinline__ bool named_and(int id, int n, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// ---- producers: 64 tokens of channel c's V~ row, and its gV entries (the
// fields of unpack_v)
template <int VBITS>
__device__ __forceinline__ void unpack_v_half(const unsigned char* vr, unsigned char* vt, int c, int half) {
  const float gv = e4m3_to_float(vr[c]);
  const __nv_bfloat162 m0 = __float2bfloat162_rn(gv), a0 = __float2bfloat162_rn(-128.f * gv);
  if constexpr (VBITS == 4) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 c4 = *reinterpret_cast<const uint4*>(vr + 512 + 64 * c + 32 * half + 16 * q);
      const uint32_t wv[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t o[4];
#pragma unroll
        for (int s2 = 0; s2 < 4; ++s2) o[s2] = fma_b(lop_magic(wv[e] >> (4 * s2), 0x000F000Fu, MAGIC_BF16), m0, a0);
        *reinterpret_cast<uint4*>(vt + cm_off(c, 64 * half + 8 * (4 * q + e), VT_K / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  } else {
    const __nv_bfloat162 m2 = __float2bfloat162_rn(gv * 0.25f), m4 = __float2bfloat162_rn(gv * 0.0625f);
    const __nv_bfloat162 a2 = __float2bfloat162_rn(-32.f * gv), a4 = __float2bfloat162_rn(-8.f * gv);
    const uint4 c4 = *reinterpret_cast<const uint4*>(vr + 512 + 32 * c + 16 * half);
    const uint32_t wv[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = wv[w], y = x >> 6, z = x >> 12;
      uint32_t o[8];
      o[0] = fma_b(lop_magic(x, 0x00030003u, MAGIC_BF16), m0, a0);
      o[1] = fma_b(lop_magic(x, 0x000C000Cu, MAGIC_BF16), m2, a2);
      o[2] = fma_b(lop_magic(x, 0x00300030u, MAGIC_BF16), m4, a4);
      o[3] = fma_b(lop_magic(y, 0x00030003u, MAGIC_BF16), m0, a0);
      o[4] = fma_b(lop_magic(y, 0x000C000Cu, MAGIC_BF16), m2, a2);
      o[5] = fma_b(lop_magic(y, 0x00300030u, MAGIC_BF16), m4, a4);
      o[6] = fma_b(lop_magic(z, 0x00030003u, MAGIC_BF16), m0, a0);
      o[7] = fma_b(lop_magic(z, 0x000C000Cu, MAGIC_BF16), m2, a2);
      *reinterpret_cast<uint4*>(vt + cm_off(c, 64 * half + 16 * w, VT_K / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(vt + cm_off(c, 64 * half + 16 * w + 8, VT_K / 8)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
  if (half == 0) {
    *reinterpret_cast<uint4*>(vt + cm_off(c, 128, VT_K / 8)) = make_uint4(b2u(m0), 0u, 0u, 0u);  // k 128, 129: beta hi, lo
    *reinterpret_cast<uint4*>(vt + cm_off(c, 136, VT_K / 8)) = make_uint4(0u, 0u, 0u, 0u);
  }
}
__device__ __forceinline__ void zero_v_half(unsigned char* vt, int c, int half) {
#pragma unroll
  for (int k8 = 0; k8 < 8; ++k8)
    *reinterpret_cast<uint4*>(vt + cm_off(c, 64 * half + 8 * k8, VT_K / 8)) = make_uint4(0u, 0u, 0u, 0u);
  if (half == 0) {
    *reinterpret_cast<uint4*>(vt + cm_off(c, 128, VT_K / 8)) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(vt + cm_off(c, 136, VT_K / 8)) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ------------------------------------------------------------------ raw tokens
// The open tile's len % 128 tokens and, for a tree, its nodes (16-bit,
// unrotated, not in the cache) against a row block, on the warp tensor cores:
// q, K and V are exact in their type, the probabilities go in as a high and a
// low part (PASSES as above: 1 takes the high part).  One pass over up to 128 tokens at a time (open tile, then nodes)
// with the running maximum and sum.  Eight warps: ceil(rows / 16) row groups
// (rounded up to 1, 2, 4 or 8), the tokens split over the warps of a row group
// and merged at the end.  Bound by the latency of its loads and its row of
// barriers, hence 96 KB and two CTAs per SM (32 chunks of 128 tokens x 64
// heads, 262144 rows: 0.1 ms for 0.2 GB).
constexpr int RAW_THREADS = 256;
struct RawSmem {
  alignas(128) unsigned char q[MQ_ROWS * D * 2];
  alignas(128) unsigned char k[T * D * 2];  // k and v become the merge area
  alignas(128) unsigned char v[T * D * 2];
  uint64_t mask[MQ_ROWS][2];  // tree: the nodes each row sees
  uint32_t nf[T / 32];        // tokens whose values hold an infinity or a NaN
};
static_assert(8 * 16 * MQ_PART * sizeof(float) <= sizeof(RawSmem::q) + 2 * T * D * 2, "merge area fits");

// Byte offset of the 16-byte chunk c of row r: rows of 256 bytes, chunks
// rotated by the row so that the 8 rows of an ldmatrix phase hit all banks.
__device__ __forceinline__ int raw_off(int r, int c) { return r * 256 + ((c ^ (r & 7)) << 4); }

// The 16-bit pair with its infinities and NaNs set to zero; `bad` notes one.
template <typename E>
__device__ __forceinline__ uint32_t finite_pair(uint32_t x, bool& bad) {
  constexpr uint32_t EXP = std::is_same<E, __half>::value ? 0x7C00u : 0x7F80u;
  if ((x & EXP) == EXP) { x &= 0xFFFF0000u; bad = true; }
  if ((x & (EXP << 16)) == (EXP << 16)) { x &= 0x0000FFFFu; bad = true; }
  return x;
}

// grid (num_kv_heads * n_rowblocks, batch) x 256 threads
template <typename E, int MODE, int PASSES>
__global__ void __launch_bounds__(RAW_THREADS, 2) raw_rows_kernel(RowsParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  allow_dependents();
  const int h = blockIdx.x / p.n_rowblocks, rb = blockIdx.x % p.n_rowblocks, b = blockIdx.y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, j = lane & 3;
  const int len = p.seq_lens[b], nq = mq_queries<MODE>(p, b);
  if (!mq_lengths_ok<MODE>(p, len, nq)) return;  // reported by the packed kernel
  int rows, n_need;
  mq_block_extent<MODE>(p, rb, len, nq, rows, n_need);
  const int n_tail = len % T;
  if (rows <= 0 || (MODE != MQ_TREE && n_tail == 0)) return;
  const uint32_t sbase = smem_u32(smem_raw);
  RawSmem& sm = *reinterpret_cast<RawSmem*>(smem_raw + (((sbase + 127u) & ~127u) - sbase));
  const int t0 = len - n_tail;  // position of open-tile slot 0
  const E* kt = static_cast<const E*>(p.tail) + (((int64_t)b * p.num_kv_heads + h) * 2 + 0) * (T * D);
  const E* vt = kt + T * D;
  if (!kcheck(kt, 2 * T * D * sizeof(E), p.tail, (size_t)gridDim.y * p.num_kv_heads * 2 * T * D * sizeof(E), p.err))
    return;
  const int64_t node0 = ((int64_t)b * p.n_queries * p.num_kv_heads + h) * D, node_stride = (int64_t)p.num_kv_heads * D;

  for (int i = tid; i < MQ_ROWS * 16; i += RAW_THREADS) {
    const int r = i >> 4, c = i & 15, R = rb * MQ_ROWS + r;
    if (r < rows)
      cp_async16(sm.q + raw_off(r, c),
                 static_cast<const E*>(p.q) +
                     (((int64_t)b * p.n_queries + R / p.G) * p.num_q_heads + (int64_t)h * p.G + R % p.G) * D + 8 * c);
    else
      *reinterpret_cast<uint4*>(sm.q + raw_off(r, c)) = make_uint4(0u, 0u, 0u, 0u);
  }
  if constexpr (MODE == MQ_TREE) {
    const int words = (p.n_queries + 63) / 64;
    const int r = tid >> 1, w = tid & 1;
    uint64_t m = 0;
    if (r < rows && w < words) m = p.tree_mask[((int64_t)b * p.n_queries + (rb * MQ_ROWS + r) / p.G) * words + w];
    const int left = nq - 64 * w;  // bits of nodes the sequence does not have are ignored
    if (left < 64) m = left <= 0 ? 0ull : m & ((1ull << left) - 1);
    sm.mask[r][w] = m;
  }
  int nrg = (rows + 15) / 16;
  nrg = nrg <= 2 ? nrg : nrg <= 4 ? 4 : 8;
  const int splits = 8 / nrg, rg = warp % nrg, split = warp / nrg;
  const bool active = 16 * rg < rows;
  const int r0 = 16 * rg + g;
  const float sl2 = p.scale * MQ_LOG2E;
  int pos[2];  // positions of the thread's two rows (window mode)
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = r0 + 8 * e;
    pos[e] = r < rows ? len - p.n_queries + (rb * MQ_ROWS + r) / p.G : -1;
  }
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  float acc[16][4];  // rows 16 rg + g and + 8, channels 8 i + 2 j, + 1
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

#pragma unroll 1
  for (int part = 0; part < (MODE == MQ_TREE ? 2 : 1); ++part) {
    const int n = part == 0 ? n_tail : nq;  // tokens of this part
    if (n == 0) continue;
    auto k_row = [&](int t) { return part == 0 ? kt + t * D : static_cast<const E*>(p.k_draft) + node0 + t * node_stride; };
    auto v_row = [&](int t) { return part == 0 ? vt + t * D : static_cast<const E*>(p.v_draft) + node0 + t * node_stride; };
    const int n_pad = (n + 31) & ~31;
    if (part) __syncthreads();  // the open tile is done with
    for (int i = tid; i < n_pad * 16; i += RAW_THREADS) {
      const int t = i >> 4, c = i & 15;
      if (t < n) {
        cp_async16(sm.k + raw_off(t, c), k_row(t) + 8 * c);
        cp_async16(sm.v + raw_off(t, c), v_row(t) + 8 * c);
      } else {
        *reinterpret_cast<uint4*>(sm.k + raw_off(t, c)) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(sm.v + raw_off(t, c)) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (tid < T / 32) sm.nf[tid] = 0;
    cp_async_wait_all();
    __syncthreads();
    // A token hidden from one row may be seen by another, and 0 x inf is not
    // 0: infinities and NaNs leave the value tile here and are added below,
    // only to the rows that see them.
    for (int i = tid; i < n * 16; i += RAW_THREADS) {
      uint4* x = reinterpret_cast<uint4*>(sm.v + raw_off(i >> 4, i & 15));
      uint4 y = *x;
      bool bad = false;
      y.x = finite_pair<E>(y.x, bad); y.y = finite_pair<E>(y.y, bad);
      y.z = finite_pair<E>(y.z, bad); y.w = finite_pair<E>(y.w, bad);
      if (bad) {
        *x = y;
        atomicOr(&sm.nf[i >> 9], 1u << ((i >> 4) & 31));
      }
    }
    __syncthreads();
    if (!active) continue;
    // whether row e (0, 1) sees token t of this part
    auto sees = [&](int e, int t) -> bool {
      if (t >= n) return false;
      if (MODE == MQ_TREE) return part == 0 || ((sm.mask[r0 + 8 * e][t >> 6] >> (t & 63)) & 1u);
      const int at = t0 + t;
      return at <= pos[e] && (at < p.n_sinks || at > pos[e] - p.window);
    };
    for (int tb = 32 * split; tb < n_pad; tb += 32 * splits) {
      float sc[4][4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) sc[nb][0] = sc[nb][1] = sc[nb][2] = sc[nb][3] = 0.f;
#pragma unroll
      for (int kb = 0; kb < 8; ++kb) {
        uint32_t a[4], k0[4], k1[4];
        ldmatrix_x4(a, sm.q + raw_off(16 * rg + (lane & 15), 2 * kb + (lane >> 4)));
        const int kr = (lane & 7) + ((lane >> 4) << 3), kc = 2 * kb + ((lane >> 3) & 1);
        ldmatrix_x4(k0, sm.k + raw_off(tb + kr, kc));
        ldmatrix_x4(k1, sm.k + raw_off(tb + 16 + kr, kc));
        mma16816<E>(sc[0], a, k0[0], k0[1]);
        mma16816<E>(sc[1], a, k0[2], k0[3]);
        mma16816<E>(sc[2], a, k1[0], k1[1]);
        mma16816<E>(sc[3], a, k1[2], k1[3]);
      }
      float tmax[2] = {-INFINITY, -INFINITY};
      bool all = tb + 32 <= n && (MODE != MQ_TREE || part == 0);
      if (MODE == MQ_WINDOW)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          all = all && (r0 + 8 * e >= rows || (t0 + tb + 31 <= pos[e] &&
                                               (t0 + tb + 31 < p.n_sinks || t0 + tb > pos[e] - p.window)));
      if (__all_sync(0xffffffffu, all)) {
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[nb][e] *= sl2;
            tmax[e >> 1] = fmaxf(tmax[e >> 1], fmaxf(sc[nb][e], SEEN));
          }
      } else {
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool in = sees(e >> 1, tb + 8 * nb + 2 * j + (e & 1));
            sc[nb][e] = in ? sc[nb][e] * sl2 : -INFINITY;
            tmax[e >> 1] = fmaxf(tmax[e >> 1], in ? fmaxf(sc[nb][e], SEEN) : -INFINITY);
          }
      }
      float corr[2], nm[2], psum[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float m_new = fmaxf(m_run[e], quad_max(tmax[e]));
        // a row that has seen nothing yet keeps zero weights (2^-inf), never -inf - -inf
        nm[e] = m_new == -INFINITY ? 0.f : m_new;
        corr[e] = ex2_ftz(m_run[e] - nm[e]);
        m_run[e] = m_new;
      }
      uint32_t ph[2][4], pl[2][4];  // A fragments of the two 16-token halves
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = ex2_ftz(sc[nb][2 * e] - nm[e]), y = ex2_ftz(sc[nb][2 * e + 1] - nm[e]);
          if constexpr (PASSES == 2) {
            uint16_t xh, xl, yh, yl;
            psum[e] += x + y;
            split_hl<E>(x, xh, xl);
            split_hl<E>(y, yh, yl);
            ph[nb >> 1][(nb & 1) * 2 + e] = pack2(xh, yh);
            pl[nb >> 1][(nb & 1) * 2 + e] = pack2(xl, yl);
          } else {
            const uint32_t w = pack2(f2bits<E>(x), f2bits<E>(y));  // the sum takes the weights as rounded
            const float2 r = pair_to_float2<E>(w);
            psum[e] += r.x + r.y;
            ph[nb >> 1][(nb & 1) * 2 + e] = w;
          }
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) l_run[e] = l_run[e] * corr[e] + quad_sum(psum[e]);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        acc[i][0] *= corr[0]; acc[i][1] *= corr[0];
        acc[i][2] *= corr[1]; acc[i][3] *= corr[1];
      }
#pragma unroll
      for (int hb = 0; hb < 2; ++hb)
#pragma unroll
        for (int np = 0; np < 8; ++np) {
          uint32_t vv[4];
          ldmatrix_x4_trans(vv, sm.v + raw_off(tb + 16 * hb + (lane & 15), 2 * np + (lane >> 4)));
          mma16816<E>(acc[2 * np], ph[hb], vv[0], vv[1]);
          mma16816<E>(acc[2 * np + 1], ph[hb], vv[2], vv[3]);
          if constexpr (PASSES == 2) {
            mma16816<E>(acc[2 * np], pl[hb], vv[0], vv[1]);
            mma16816<E>(acc[2 * np + 1], pl[hb], vv[2], vv[3]);
          }
        }
    }
    // the rare infinities and NaNs: weight of the token again, onto the rows that see it
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      if ((t & 31) == 0 && sm.nf[t >> 5] == 0) { t += 31; continue; }
      if (((sm.nf[t >> 5] >> (t & 31)) & 1u) == 0 || (t / 32) % splits != split) continue;
      float s[2] = {0.f, 0.f};
      for (int c = j; c < 16; c += 4) {
        const uint32_t* kw = reinterpret_cast<const uint32_t*>(sm.k + raw_off(t, c));
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 kv = pair_to_float2<E>(kw[w]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 qv =
                pair_to_float2<E>(reinterpret_cast<const uint32_t*>(sm.q + raw_off(r0 + 8 * e, c))[w]);
            s[e] = fmaf(qv.x, kv.x, fmaf(qv.y, kv.y, s[e]));
          }
        }
      }
      const E* vr = v_row(t);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[e] = quad_sum(s[e]) * sl2;
        // (a weight of 0 counts: 0 times an infinity is NaN; a NaN has spoilt the row already)
        const float w = sees(e, t) ? ex2_ftz(s[e] - m_run[e]) : -1.f;
        if (w >= 0.f) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float x = tof(vr[8 * i + 2 * j + u]);
              if (!isfinite(x)) acc[i][2 * e + u] += w * x;
            }
        }
      }
    }
  }
  if (splits == 1) {  // a row group's only warp: nothing to merge
    if (!active) return;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + 8 * e;
      if (r >= rows) continue;
      float* o = mq_part(p, b, h, rb, p.n_chunks, r);
      if (!kcheck(o, MQ_PART * sizeof(float), p.ws, (size_t)p.ws_bytes, p.err)) continue;
      if (j == 0) *reinterpret_cast<float2*>(o) = make_float2(m_run[e], l_run[e]);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float2*>(o + MQ_PACC + 8 * i + 2 * j) = make_float2(acc[i][2 * e], acc[i][2 * e + 1]);
    }
    return;
  }
  __syncthreads();  // every warp is done with the buffers: they become the merge area
  float* merge = reinterpret_cast<float*>(sm.q);
  if (active) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float* o = merge + (warp * 16 + g + 8 * e) * MQ_PART;
      if (j == 0) { o[0] = m_run[e]; o[1] = l_run[e]; }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float2*>(o + MQ_PACC + 8 * i + 2 * j) = make_float2(acc[i][2 * e], acc[i][2 * e + 1]);
    }
  }
  __syncthreads();
  for (int r = warp; r < rows; r += RAW_THREADS / 32) {
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < splits; ++s) M = fmaxf(M, merge[((s * nrg + (r >> 4)) * 16 + (r & 15)) * MQ_PART]);
    for (int s = 0; s < splits; ++s) {
      const float* o = merge + ((s * nrg + (r >> 4)) * 16 + (r & 15)) * MQ_PART;
      if (o[0] == -INFINITY) continue;
      const float f = ex2_ftz(o[0] - M);
      const float4 x = *reinterpret_cast<const float4*>(o + MQ_PACC + 4 * lane);
      L += f * o[1];
      a.x += f * x.x; a.y += f * x.y; a.z += f * x.z; a.w += f * x.w;
    }
    float* o = mq_part(p, b, h, rb, p.n_chunks, r);
    if (!kcheck(o, MQ_PART * sizeof(float), p.ws, (size_t)p.ws_bytes, p.err)) continue;
    if (lane == 0) { o[0] = M; o[1] = L; }
    *reinterpret_cast<float4*>(o + MQ_PACC + 4 * lane) = a;
  }
}

// ------------------------------------------------------------------ packed tiles
// grid (n_chunks, num_kv_heads * n_rowblocks, batch) x 512 threads.  With
// n_chunks == 1 the CTA writes the result rows, else partial rows.
template <typename E, int KBITS, int VBITS, int MODE, int PASSES, typename O>
__global__ void __launch_bounds__(RQ_THREADS, 1) rows_kernel(RowsParams p, O* __restrict__ out) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  allow_dependents();
  const int chunk = blockIdx.x, h = blockIdx.y / p.n_rowblocks, rb = blockIdx.y % p.n_rowblocks, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = p.seq_lens[b], nq = mq_queries<MODE>(p, b);
  const bool fused = p.n_chunks == 1;
  const bool ok_len = mq_lengths_ok<MODE>(p, len, nq);
  if (!ok_len && tid == 0 && chunk == 0 && blockIdx.y == 0) set_error(p.err, KVARN_DEV_ERR_TOKEN_RANGE);
  int rows = 0, n_need = 0, n_tiles = 0;
  if (ok_len) mq_block_extent<MODE>(p, rb, len, nq, rows, n_need);
  WinTiles wt = {};
  if constexpr (MODE == MQ_WINDOW) wt = win_tiles(0, 0, 0);
  const int first = chunk * p.chunk_tiles;
  if (ok_len && rows > 0 && (MODE == MQ_TREE || len > 0)) {
    if constexpr (MODE == MQ_WINDOW) wt = mq_win_tiles(p, rb, len, n_need);
    n_tiles = max(0, min(p.chunk_tiles, (MODE == MQ_WINDOW ? wt.n : n_need) - first));
  }
  auto tile_at = [&](int k) { return MODE == MQ_WINDOW ? wt.at(first + k) : first + k; };
  // rows this CTA writes a result of, beyond those it computes: the zeros of a
  // bad length or an empty slot (a tree: only rows of nodes the sequence has)
  const int out_rows = MODE == MQ_TREE ? (nq >= 0 && nq <= p.n_queries ? nq : 0) * p.G : p.n_queries * p.G;
  const int res_rows = fused ? max(0, min(MQ_ROWS, out_rows - rb * MQ_ROWS)) : 0;
  if (n_tiles == 0 && res_rows == 0) {
    wait_prerequisite();  // the raw kernel is complete when this grid is
    return;
  }
  const uint32_t sbase = smem_u32(smem_raw);
  RQSmem& sm = *reinterpret_cast<RQSmem*>(smem_raw + (((sbase + 127u) & ~127u) - sbase));
  float* rowf = reinterpret_cast<float*>(sm.kt[0]);  // [128][RQ_ROWF] at the end

  if (n_tiles > 0) {
    constexpr int KREC = rec_bytes(KBITS), VREC = rec_bytes(VBITS), NS = rq_stages<KBITS, VBITS>();
    const int32_t* tab = p.block_table + (int64_t)b * p.max_blocks;
    // one bulk copy of the K and V records of tile k, block blk, into its stage (one thread)
    auto issue_rec = [&](int k, int32_t blk) {
      const int s = k % NS;
      const unsigned char* src = p.pool + blk * p.block_bytes + (int64_t)h * (KREC + VREC);
      const bool in = blk >= 0 && blk < p.num_blocks &&
                      kcheck(src, KREC + VREC, p.pool, (size_t)p.num_blocks * p.block_bytes, p.err);
      sm.rec_ok[s] = in;
      if (in) {
        mbar_expect_tx(&sm.rec_full[s], KREC + VREC);
        bulk_g2s(sm.rec + s * (KREC + VREC), src, KREC + VREC, &sm.rec_full[s]);
      } else {
        set_error(p.err, KVARN_DEV_ERR_BLOCK_RANGE);
        mbar_arrive(&sm.rec_full[s]);
      }
    };
    // the query rows are on their way before anything else: warp w takes rows 8 w .. 8 w + 7
    static_assert(RQ_WARPS == 16, "8 rows a warp");
    uint2 raw[8];
#pragma unroll
    for (int rr = 0; rr < 8; ++rr) {
      const int row = 8 * warp + rr, Rr = rb * MQ_ROWS + row;
      raw[rr] = row < rows ? *reinterpret_cast<const uint2*>(
                                 static_cast<const E*>(p.q) +
                                 (((int64_t)b * p.n_queries + Rr / p.G) * p.num_q_heads + (int64_t)h * p.G + Rr % p.G) * D +
                                 4 * lane)
                           : make_uint2(0u, 0u);
    }
    if (warp == RQ_WI) {  // block ids (a lane each), barriers, the first records on their way
      const int32_t blk = lane < min(n_tiles, NS) ? tab[tile_at(lane)] : -1;
      int32_t blks[3];
#pragma unroll
      for (int k = 0; k < NS; ++k) blks[k] = __shfl_sync(0xffffffffu, blk, k);
      if (lane == 0) {
        for (int s = 0; s < NS; ++s) {
          mbar_init(&sm.rec_full[s], 1);
          mbar_init(&sm.rec_empty[s], RQ_KTHREADS + RQ_VTHREADS);
        }
        for (int s = 0; s < 2; ++s) {
          mbar_init(&sm.kt_full[s], RQ_KTHREADS);
          mbar_init(&sm.vt_full[s], RQ_VTHREADS);
          mbar_init(&sm.s_full[s], 1);
          mbar_init(&sm.p_full[s], RQ_ST);
          mbar_init(&sm.pv_done[s], 1);
        }
        mbar_init(&sm.fin, 1);
        fence_mbar_init();
#pragma unroll
        for (int k = 0; k < NS; ++k)
          if (k < n_tiles) issue_rec(k, blks[k]);
      }
      __syncwarp();
      tmem_alloc(&sm.tmem, TM_COLS);
    }
    if (tid == 0) {
      sm.qmax = 0;
      sm.qmin = 0x7F7FFFFFu;
    }
    __syncthreads();
    // ---- query operand: warp w rotates rows 8 w .. 8 w + 7, 4 channels per
    // lane, staged in the K~ buffers, then fp16 core-matrix rows
    float* stage = reinterpret_cast<float*>(sm.kt[0]) + warp * (8 * RQ_ROWF);
    {
      float am[8];
#pragma unroll
      for (int rr = 0; rr < 8; ++rr) {
        const float2 lo = pair_to_float2<E>(raw[rr].x), hi = pair_to_float2<E>(raw[rr].y);
        float x[4] = {lo.x, lo.y, hi.x, hi.y};
        fwht128(x, lane);
        const float f = p.scale * MQ_LOG2E * INV_SQRT_D;
        am[rr] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] *= f;
          am[rr] = fmaxf(am[rr], fabsf(x[i]));
        }
        *reinterpret_cast<float4*>(stage + rr * RQ_ROWF + 4 * lane) = make_float4(x[0], x[1], x[2], x[3]);
      }
#pragma unroll
      for (int m = 16, n = 4; m >= 4; m >>= 1, n >>= 1)  // lane -> largest of row lane / 4
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const bool up = (lane & m) != 0;
          const float other = __shfl_xor_sync(0xffffffffu, up ? am[i] : am[i + n], m);
          am[i] = fmaxf(up ? am[i + n] : am[i], other);
        }
      const float amax = quad_max(am[0]);
      if ((lane & 3) == 0) sm.row_m[8 * warp + (lane >> 2)] = amax;
      const uint32_t u = amax < RQ_QMAX ? __float_as_uint(amax) : 0u;
      const uint32_t hi_u = __reduce_max_sync(0xffffffffu, u), lo_u = __reduce_min_sync(0xffffffffu, u ? u : 0x7F7FFFFFu);
      if (lane == 0) {
        atomicMax(&sm.qmax, hi_u);
        atomicMin(&sm.qmin, lo_u);
      }
    }
    __syncthreads();
    // One power of two for the whole block puts its largest |Q'| in [64, 128):
    // high and low parts keep 2^-24 absolute, 2^-30 of the largest.  Where the
    // rows differ by more than RQ_SPREAD each takes its own (row_ex), and the
    // softmax the general pass, which multiplies by 2^(row_ex - ex).  A row
    // that is not finite spoils its own result alone.
    const float qmax = __uint_as_float(sm.qmax);
    const bool spread = qmax > RQ_SPREAD * __uint_as_float(sm.qmin);
    auto exp_of = [](float m) {
      int e = 0;
      if (m > 0.f) frexpf(m, &e);
      return max(e, -100);
    };
    const int ex = exp_of(qmax);
    auto row_ex = [&](int row) {
      const float m = sm.row_m[row];
      return spread && m > 0.f && m < RQ_QMAX ? exp_of(m) : ex;
    };
    const float cr = ldexpf(1.f, ex - 1);  // score (log2) = cr 2^(row_ex - ex) (aK D_t + bK D_128)
    {
      const int rr = lane & 7, row = 8 * warp + rr;
      const float qs = ldexpf(1.f, 7 - row_ex(row));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int g = (lane >> 3) + 4 * j;  // slot pairs as in the causal kernel
        const int ca = (KBITS == 4) ? 8 * g : 16 * (g >> 1) + 4 * (g & 1), cb = ca + ((KBITS == 4) ? 4 : 8);
        const float4 va = *reinterpret_cast<const float4*>(stage + rr * RQ_ROWF + ca);
        const float4 vb = *reinterpret_cast<const float4*>(stage + rr * RQ_ROWF + cb);
        const float av[4] = {va.x * qs, va.y * qs, va.z * qs, va.w * qs}, bv[4] = {vb.x * qs, vb.y * qs, vb.z * qs, vb.w * qs};
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 hi = __floats2half2_rn(av[i], bv[i]);
          const float2 hf = __half22float2(hi);
          hw[i] = h2u(hi);
          lw[i] = h2u(__floats2half2_rn(av[i] - hf.x, bv[i] - hf.y));
        }
        *reinterpret_cast<uint4*>(sm.vt[0] + cm_off(row, 8 * g, 16)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        if (PASSES == 2)
          *reinterpret_cast<uint4*>(sm.qa_lo + cm_off(row, 8 * g, 16)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    if (warp < 4) {  // Q' hi of row r -> tensor-memory lane r
      const uint32_t lb = tmem + ((uint32_t)(warp * 32) << 16) + TM_QA;
#pragma unroll
      for (int c = 0; c < 64; c += 16) {
        uint32_t w16[16];
#pragma unroll
        for (int g2 = 0; g2 < 4; ++g2) {
          const uint4 v4 = *reinterpret_cast<const uint4*>(sm.vt[0] + cm_off(tid, 2 * c + 8 * g2, 16));
          w16[4 * g2] = v4.x; w16[4 * g2 + 1] = v4.y; w16[4 * g2 + 2] = v4.z; w16[4 * g2 + 3] = v4.w;
        }
        tmem_st16(lb + c, w16);
      }
      tmem_wait_st();
    } else if (warp >= RQ_WK && warp < RQ_WV) {
      for (int i = tid - RQ_ST; i < 2 * 15 * 16; i += 128) {  // K~ rows 129..143 of both buffers
        const int s = i / (15 * 16), rr = 129 + (i / 16) % 15, kg = i % 16;
        *reinterpret_cast<uint4*>(sm.kt[s] + cm_off(rr, 8 * kg, 16)) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp == RQ_WI) {
      // ---------------------------------------------------------- MMA issue (one thread)
      // A thread that issues is held up while the tensor pipe works its queue
      // off (1.1 K cycles for a tile's QK), so it does nothing else.
      if (lane == 0) {
        const uint64_t qa_lo = umma_desc(smem_u32(sm.qa_lo), 128, 2048);
        auto issue_qk = [&](int k) {
          const uint32_t kbase = smem_u32(sm.kt[k & 1]), d = tmem + TM_S + TM_SSTRIDE * (k & 1);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(d, tmem + TM_QA + 8 * kk, umma_desc(kbase + 256 * kk, 128, 2048), IDESC_QK, kk > 0);
          if (PASSES == 2) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ss(d, qa_lo + (uint64_t)(16 * kk), umma_desc(kbase + 256 * kk, 128, 2048), IDESC_QK, 1);
          }
          umma_commit(&sm.s_full[k & 1]);
        };
        auto issue_pv = [&](int k) {
          const uint32_t vb = smem_u32(sm.vt[k & 1]), pa = tmem + TM_S + TM_SSTRIDE * (k & 1);
#pragma unroll
          for (int kk = 0; kk < 9; ++kk)  // hi parts of tokens 16 kk .. 16 kk + 15, then the beta block
            umma_ts(tmem + TM_O, pa + 16 * kk, umma_desc(vb + 256 * kk, 128, VT_K * 16), IDESC_PV,
                    (k > 0 || kk > 0) ? 1u : 0u);
          if (PASSES == 2) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // lo parts
              umma_ts(tmem + TM_O, pa + 16 * kk + 8, umma_desc(vb + 256 * kk, 128, VT_K * 16), IDESC_PV, 1);
          }
          umma_commit(&sm.pv_done[k & 1]);
        };
        bool ok = true;
        for (int k = 0; ok && k < min(n_tiles, 2); ++k) {  // both score buffers start free
          ok = mbar_wait_parked(&sm.kt_full[k], 0, p.err);
          if (!ok) break;
          tc_fence_after();
          issue_qk(k);
        }
        for (int k = 0; ok && k < n_tiles; ++k) {
          const int s = k & 1;
          const uint32_t ph = (k >> 1) & 1;
          ok = mbar_wait_parked(&sm.vt_full[s], ph, p.err) && mbar_wait_parked(&sm.p_full[s], ph, p.err);
          if (!ok) break;
          tc_fence_after();
          issue_pv(k);
          if (k + 2 < n_tiles) {  // the buffer is free once PV(k) has read its P~
            ok = mbar_wait_parked(&sm.kt_full[s], ph ^ 1, p.err) && mbar_wait_parked(&sm.pv_done[s], ph, p.err);
            if (!ok) break;
            tc_fence_after();
            issue_qk(k + 2);
          }
        }
        // every MMA this thread issued has finished before the memory is released
        umma_commit(&sm.fin);
        mbar_wait_parked(&sm.fin, 0, p.err);
      }
      __syncwarp();
    } else if (warp >= RQ_WK && warp < RQ_WV) {
      // ---------------------------------------------------------- K~ and the tokens' scales
      const int pth = tid - RQ_ST;
      bool ok = true;
      for (int k = 0; k < n_tiles; ++k) {
        const int s = k & 1, rs = k % NS;
        const uint32_t ph = (k >> 1) & 1;
        ok = wait_all(&sm.rec_full[rs], (k / NS) & 1, p.err);
        if (ok && k >= 2)  // QK(k - 2) has read this K~, the softmax of k - 2 these scales
          ok = wait_all(&sm.s_full[s], ph ^ 1, p.err) && wait_all(&sm.p_full[s], ph ^ 1, p.err);
        if (!ok) break;
        const unsigned char* kr = sm.rec + rs * (KREC + VREC);
        const unsigned char* vr = kr + KREC;
        const bool in = sm.rec_ok[rs];
        if (pth == 0) sm.kt_ok[s] = in;
        if (in) {
          sm.ka[s][pth] = cr * e4m3_to_float(kr[128 + pth]);  // (a power of two: exact)
          sm.kb[s][pth] = cr * __half2float(*reinterpret_cast<const __half*>(kr + 256 + 2 * pth));
          const float va = e4m3_to_float(vr[128 + pth]);
          const float vb = __half2float(*reinterpret_cast<const __half*>(vr + 256 + 2 * pth));
          sm.va[s][pth] = va;
          const float vi = 1.f / fmaxf(va, 0x1p-9f);  // (steps are 2^-9 or more)
          sm.vb[s][pth] = PASSES == 1 ? vb * vi : vb;
          if (PASSES == 1) sm.vi[s][pth] = vi;
          unpack_k<KBITS>(kr, sm.kt[s], pth);
          if (pth < 16) {  // the g row: K~[128][k] = gK of the slot's channel / 64
            uint32_t o[4];
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
              o[jj] = h2u(__floats2half2_rn(e4m3_to_float(kr[perm_k<KBITS>(8 * pth + 2 * jj)]) * (1.f / 64.f),
                                            e4m3_to_float(kr[perm_k<KBITS>(8 * pth + 2 * jj + 1)]) * (1.f / 64.f)));
            *reinterpret_cast<uint4*>(sm.kt[s] + cm_off(128, 8 * pth, 16)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
          sm.ka[s][pth] = sm.kb[s][pth] = sm.va[s][pth] = sm.vb[s][pth] = sm.vi[s][pth] = 0.f;
          zero_k(sm.kt[s], pth);
          if (pth < 16)
            *reinterpret_cast<uint4*>(sm.kt[s] + cm_off(128, 8 * pth, 16)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
        mbar_arrive(&sm.kt_full[s]);
        mbar_arrive(&sm.rec_empty[rs]);
      }
    } else if (warp >= RQ_WV) {
      // ---------------------------------------------------------- V~ and the records' refill
      const int pth = tid - RQ_ST - RQ_KTHREADS;
      bool ok = true;
      int issued = min(n_tiles, NS);
      int32_t blk = pth == 0 && n_tiles > NS ? tab[tile_at(NS)] : 0;  // of the next tile to fetch
      for (int k = 0; k < n_tiles; ++k) {
        const int s = k & 1, rs = k % NS;
        const uint32_t ph = (k >> 1) & 1;
        ok = wait_all(&sm.rec_full[rs], (k / NS) & 1, p.err);
        if (ok && k >= 2) ok = wait_all(&sm.pv_done[s], ph ^ 1, p.err);  // PV(k - 2) has read this V~
        if (!ok) break;
        // half channels, 32 at a time per warp: 256 over 96 threads
        const bool in = sm.rec_ok[rs];
        for (int i = pth; i < 2 * D; i += RQ_VTHREADS) {
          if (in) unpack_v_half<VBITS>(sm.rec + rs * (KREC + VREC) + KREC, sm.vt[s], i & (D - 1), i >> 7);
          else zero_v_half(sm.vt[s], i & (D - 1), i >> 7);
        }
        fence_proxy_async();
        mbar_arrive(&sm.vt_full[s]);
        mbar_arrive(&sm.rec_empty[rs]);
        if (pth == 0 && k + NS < n_tiles) {  // every producer is done with this stage: refill it
          if (mbar_wait_parked(&sm.rec_empty[rs], (k / NS) & 1, p.err)) {
            issue_rec(k + NS, blk);
            issued = k + NS + 1;
            if (issued < n_tiles) blk = tab[tile_at(issued)];
          }
        }
        __syncwarp();
      }
      if (fused) {  // the raw partials of this CTA's rows: into the L2 while the last tiles finish
        wait_prerequisite();
        const char* raw = reinterpret_cast<const char*>(mq_part(p, b, h, rb, p.n_chunks, 0));
        for (int i = pth * 128; i < rows * MQ_PART * 4; i += RQ_VTHREADS * 128)
          asm volatile("prefetch.global.L2 [%0];\n" ::"l"(raw + i));
      }
      // copies in flight (an early exit) land before the CTA ends: the last of each stage
      if (!ok && pth == 0)
        for (int k = max(0, issued - NS); k < issued; ++k)
          mbar_wait_parked(&sm.rec_full[k % NS], (k / NS) & 1, p.err);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- softmax
      // A warp takes 16 rows.  Scores come in fragments: with
      // lane = 4 g + j the thread holds rows row0 + g and + 8 and of every 8
      // tokens the pair 2 j, 2 j + 1.  A thread per row would need every token's
      // four scales, 16 bytes into each lane for each score: 2 K cycles a tile
      // on the shared-memory pipe, which the MMAs' operands (1.4 K) and the
      // unpacking need too.  Here a pair's scales serve two rows.
      const int g = lane >> 2, j = lane & 3;
      const int row0 = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
      const uint32_t lane_base = tmem + ((uint32_t)row0 << 16);
      auto row_of = [&](int i) { return row0 + g + 8 * i; };
      int pos[2];  // positions of the rows (window mode)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        pos[i] = row_of(i) < rows ? len - p.n_queries + (rb * MQ_ROWS + row_of(i)) / p.G : -1;
      float rs[2];  // the rows' own scale over the block's
#pragma unroll
      for (int i = 0; i < 2; ++i) rs[i] = ldexpf(1.f, row_ex(row_of(i)) - ex);
      float m_own[2];   // reference of the rows
      float2 l_sum[2];  // of this thread's tokens, relative to m_own
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m_own[i] = -INFINITY;
        l_sum[i] = make_float2(0.f, 0.f);
      }
      auto pair_at = [](const float* q, int t) { return *reinterpret_cast<const float2*>(q + t); };
      bool ok = true;
      for (int k = 0; k < n_tiles; ++k) {
        const int s = k & 1;
        const uint32_t ph = (k >> 1) & 1;
        ok = wait_all(&sm.s_full[s], ph, p.err) && wait_all(&sm.kt_full[s], ph, p.err);
        if (!ok) break;
        tc_fence_after();
        const uint32_t ub = lane_base + TM_S + TM_SSTRIDE * s;  // scores, then P~, of the tile
        const float* kap = sm.ka[s] + 2 * j;
        const float* kbp = sm.kb[s] + 2 * j;
        const float* vap = sm.va[s] + 2 * j;
        const float* vbp = sm.vb[s] + 2 * j;
        const float* vip = sm.vi[s] + 2 * j;
        float2 d2[2];  // D_128 of the rows
        {
          uint32_t d[4];
          tmem_ld_16x256b_x1(ub + 128, d);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x = __uint_as_float(__shfl_sync(0xffffffffu, d[2 * i], lane & ~3));
            d2[i] = make_float2(x, x);
          }
        }
        // tokens of the tile row i sees: up to nvis, without hs .. he - 1 (between first tokens and window)
        const int t0 = tile_at(k) * T;
        const bool valid = sm.kt_ok[s];
        const int hs = MODE == MQ_WINDOW ? max(0, p.n_sinks - t0) : 0;
        int nvis[2], he[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          nvis[i] = !valid ? 0 : MODE == MQ_TREE ? T : min(T, pos[i] - t0 + 1);
          he[i] = MODE == MQ_WINDOW ? pos[i] + 1 - p.window - t0 : 0;
        }
        bool all = !spread, dead = false;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (row_of(i) < rows) {
            all = all && nvis[i] >= T && (MODE != MQ_WINDOW || hs >= min(T, he[i]));
            dead = dead || m_own[i] <= SEEN;
          }
        const bool full = __all_sync(0xffffffffu, all);
        // two scores (log2) less the reference of row i, tokens t, t + 1; hidden ones -inf
        auto score2 = [&](auto mask_c, int i, uint32_t x, uint32_t y, float2 a, float2 bz, float2 nm, int t) {
          const float2 dt = make_float2(__uint_as_float(x), __uint_as_float(y));
          float2 e;
          if constexpr (!decltype(mask_c)::value) {
            e = ffma2(a, dt, ffma2(bz, d2[i], nm));
          } else {
            e = ffma2(ffma2(a, dt, fmul2(bz, d2[i])), make_float2(rs[i], rs[i]), nm);
            if (t >= nvis[i] || (MODE == MQ_WINDOW && t >= hs && t < he[i])) e.x = -INFINITY;
            if (t + 1 >= nvis[i] || (MODE == MQ_WINDOW && t + 1 >= hs && t + 1 < he[i])) e.y = -INFINITY;
          }
          return e;
        };
        // the rows' largest scores of tokens c0 .. 127, rounded up (references are whole numbers)
        auto top_from = [&](int c0, float (&top)[2]) {
#pragma unroll
          for (int i = 0; i < 2; ++i) top[i] = -INFINITY;
#pragma unroll 1
          for (int c = c0; c < T; c += 32) {
            uint32_t d[16];
            tmem_ld_16x256b_x4(ub + c, d);
            tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const float2 a = pair_at(kap, c + 8 * n), bz = pair_at(kbp, c + 8 * n);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t* x = d + 4 * n + 2 * i;
                const float2 e = score2(std::true_type{}, i, x[0], x[1], a, bz, make_float2(0.f, 0.f), c + 8 * n + 2 * j);
                top[i] = fmaxf(top[i], fmaxf(e.x, e.y));
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) top[i] = ceilf(quad_max(top[i]));
        };
        // n columns from col on times f per row: P~ words (bf16 pairs; f a power of two, so exact) or O
        auto scale_cols = [&](auto words_c, uint32_t col, int n, const float (&f)[2]) {
          constexpr bool WORDS = decltype(words_c)::value;
          tmem_wait_st();
#pragma unroll 1
          for (int c = 0; c < n; c += 32) {
            uint32_t d[16];
            tmem_ld_16x256b_x4(col + c, d);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float fx = f[(x >> 1) & 1];
              d[x] = WORDS ? b2u(__hmul2(u2b(d[x]), __float2bfloat162_rn(fx)))
                           : __float_as_uint(__uint_as_float(d[x]) * fx);
            }
            tmem_st_16x256b_x4(col + c, d);
          }
        };
        // The reference this tile starts with: the last one seen.  A warp with
        // a row that has no score yet looks for the tile's maximum first.
        float m_use[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) m_use[i] = m_own[i];
        if (__any_sync(0xffffffffu, dead)) {
          float top[2];
          top_from(0, top);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (m_own[i] <= SEEN) {
              const bool sees = nvis[i] > 0 && (hs > 0 || he[i] < nvis[i]);  // some token of this tile
              m_use[i] = fmaxf(fmaxf(m_own[i], top[i]), sees ? SEEN : -INFINITY);
            }
        }
        // P~ = p aV, l += sum p, beta += sum p bV in one pass; p may exceed 1.
        // (l counts from the reference too: m_use differs from m_own only
        // where l is still 0, or NaN.)
        float2 bt[2];
        float emax[2];  // largest exponents of the tile
        auto ref2 = [&](int i) {
          const float m = m_use[i] == -INFINITY ? 0.f : -m_use[i];
          return make_float2(m, m);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          bt[i] = make_float2(0.f, 0.f);
          emax[i] = -INFINITY;
        }
        auto pass = [&](auto mask_c) {
#pragma unroll 1
          for (int c = 0; c < T; c += 32) {
            uint32_t d[16];  // accumulators, then exponents
            tmem_ld_16x256b_x4(ub + c, d);
            tmem_wait_ld();
            float ec[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const float2 a = pair_at(kap, c + 8 * n), bz = pair_at(kbp, c + 8 * n);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t* x = d + 4 * n + 2 * i;
                const float2 e = score2(mask_c, i, x[0], x[1], a, bz, ref2(i), c + 8 * n + 2 * j);
                ec[i] = fmaxf(ec[i], fmaxf(e.x, e.y));
                x[0] = __float_as_uint(e.x);
                x[1] = __float_as_uint(e.y);
              }
            }
            if (__any_sync(0xffffffffu, fmaxf(ec[0], ec[1]) > RQ_EMAX)) {
              // weights about to overflow: raise the reference past the rest
              // of the tile and shrink what there is so far (rare)
              float top[2], f[2];
              top_from(c, top);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float raise = quad_max(ec[i]) > RQ_EMAX ? fmaxf(0.f, top[i] - m_use[i]) : 0.f;
                f[i] = pow2_neg(raise);
                const float2 f2 = make_float2(f[i], f[i]);
                l_sum[i] = fmul2(l_sum[i], f2);
                bt[i] = fmul2(bt[i], f2);
                emax[i] -= raise;
                ec[i] -= raise;
                m_use[i] += raise;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  uint32_t* x = d + 4 * n + 2 * i;
                  x[0] = __float_as_uint(__uint_as_float(x[0]) - raise);
                  x[1] = __float_as_uint(__uint_as_float(x[1]) - raise);
                }
              }
              scale_cols(std::true_type{}, ub, c, f);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) emax[i] = fmaxf(emax[i], ec[i]);
#pragma unroll
            for (int n2 = 0; n2 < 2; ++n2) {  // 16 tokens: hi words to columns 0..7, lo words to 8..15
              uint32_t w[8];
#pragma unroll
              for (int nn = 0; nn < 2; ++nn) {
                const int n = 2 * n2 + nn;
                const float2 av = pair_at(vap, c + 8 * n), bv = pair_at(vbp, c + 8 * n);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t* x = d + 4 * n + 2 * i;
                  const float2 pr = make_float2(ex2_ftz(__uint_as_float(x[0])), ex2_ftz(__uint_as_float(x[1])));
                  const float2 pa = fmul2(pr, av);
                  const __nv_bfloat162 hi = __floats2bfloat162_rn(pa.x, pa.y);
                  w[2 * nn + i] = b2u(hi);
                  if (PASSES == 1) {  // beta and l from the weights as rounded (times bV / aV and 1 / aV)
                    const float2 hf = __bfloat1622float2(hi);
                    l_sum[i] = ffma2(hf, pair_at(vip, c + 8 * n), l_sum[i]);
                    bt[i] = ffma2(hf, bv, bt[i]);
                  } else {
                    l_sum[i] = fadd2(l_sum[i], pr);
                    bt[i] = ffma2(pr, bv, bt[i]);
                    const float2 lo = ffma2(__bfloat1622float2(hi), make_float2(-1.f, -1.f), pa);  // exact product
                    w[4 + 2 * nn + i] = b2u(__floats2bfloat162_rn(lo.x, lo.y));
                  }
                }
              }
              if (PASSES == 2) tmem_st_16x128b_x4(ub + c + 16 * n2, w);
              else tmem_st_16x128b_x2(ub + c + 16 * n2, w);
            }
          }
        };
        // hidden tokens get weight 2^-inf; a row that has seen none yet too (its reference stands in as 0)
        if (full) pass(std::false_type{});
        else pass(std::true_type{});
        // The reference after this tile: raised if the weights have grown
        // large.  For almost every tile there is nothing to do.
        bool change = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) change = change || emax[i] > RQ_RAISE || m_use[i] != m_own[i];
        if (__any_sync(0xffffffffu, change)) {
          float f[2], corr[2];
          bool any_f = false, any_c = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float em = quad_max(emax[i]);
            const float m_new = em > RQ_RAISE ? m_use[i] + ceilf(em) : m_use[i];
            f[i] = m_new == m_use[i] ? 1.f : pow2_neg(m_new - m_use[i]);
            corr[i] = m_new == m_own[i] || m_own[i] <= SEEN ? 1.f : pow2_neg(m_new - m_own[i]);
            any_f = any_f || f[i] != 1.f;
            any_c = any_c || corr[i] != 1.f;
            const float2 f2 = make_float2(f[i], f[i]);
            l_sum[i] = fmul2(l_sum[i], f2);
            bt[i] = fmul2(bt[i], f2);
            m_own[i] = m_new;
          }
          if (__any_sync(0xffffffffu, any_f)) scale_cols(std::true_type{}, ub, T, f);  // this tile's weights
          if (__any_sync(0xffffffffu, any_c)) {  // the accumulator, once PV(k - 1) is done
            ok = wait_all(&sm.pv_done[s ^ 1], ((k - 1) >> 1) & 1, p.err);
            if (!ok) break;
            tc_fence_after();
            scale_cols(std::false_type{}, lane_base + TM_O, D, corr);
          }
        }
        {
          uint32_t w[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float beta = quad_sum(bt[i].x + bt[i].y);
            const __nv_bfloat16 bh = __float2bfloat16_rn(beta);
            const __nv_bfloat16 bl = __float2bfloat16_rn(beta - __bfloat162float(bh));
            w[i] = j == 0 ? (uint32_t)__bfloat16_as_ushort(bh) | ((uint32_t)__bfloat16_as_ushort(bl) << 16) : 0u;
          }
          tmem_st_16x128b_x1(ub + 128, w[0], w[1]);
          tmem_st_16x128b_x1(ub + 132, 0u, 0u);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sm.p_full[s]);
      }
      if (ok) ok = wait_all(&sm.pv_done[(n_tiles - 1) & 1], ((n_tiles - 1) >> 1) & 1, p.err);
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float l = quad_sum(l_sum[i].x + l_sum[i].y);
        if (j == 0) {
          sm.row_m[row_of(i)] = ok ? m_own[i] : -INFINITY;
          sm.row_l[row_of(i)] = ok ? l : 0.f;
        }
      }
      ok = named_and(1, RQ_ST, ok);
      // accumulator out: a thread per row, 64 channels each
      const int r = 32 * (warp & 3) + lane, c0 = 64 * (warp >> 2);
      const bool rv = r < rows;
      float* o = fused ? rowf + r * RQ_ROWF : mq_part(p, b, h, rb, chunk, rv ? r : 0);
      const bool wv = fused || (rv && kcheck(o, MQ_PART * sizeof(float), p.ws, (size_t)p.ws_bytes, p.err));
      float* oa = o + (fused ? 0 : MQ_PACC) + c0;
      if (!fused && wv && c0 == 0) {
        o[0] = sm.row_m[r];
        o[1] = sm.row_l[r];
      }
#pragma unroll 1
      for (int c = 0; c < 64; c += 32) {
        uint32_t d[32];
        tmem_ld32(tmem + ((uint32_t)((warp & 3) * 32) << 16) + TM_O + c0 + c, d);
        tmem_wait_ld();
        if (wv) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(oa + c + i) =
                ok ? make_float4(__uint_as_float(d[i]), __uint_as_float(d[i + 1]), __uint_as_float(d[i + 2]),
                                 __uint_as_float(d[i + 3]))
                   : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == RQ_WI) tmem_dealloc(tmem, TM_COLS);
  }

  wait_prerequisite();  // the raw kernel's partial rows
  if (!fused) return;
  // ---- result rows: a warp takes every sixteenth row, four at a time (their
  // loads in flight together: one by one they took 20 K cycles of a CTA);
  // packed part rotated back, raw part added, normalised
  const bool has_raw = ok_len && (MODE == MQ_TREE ? nq > 0 : len % T != 0);
  constexpr int RU = 4;
#pragma unroll 1
  for (int r0 = warp; r0 < res_rows; r0 += RU * RQ_WARPS) {
    float2 raw_ml[RU];
    float4 raw_a[RU], o[RU];
    int64_t row[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int r = r0 + u * RQ_WARPS, R = rb * MQ_ROWS + r, i = R / p.G;
      row[u] = ((int64_t)b * p.n_queries + i) * p.num_q_heads + (int64_t)h * p.G + (R - i * p.G);
      raw_ml[u] = make_float2(-INFINITY, 0.f);
      raw_a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (has_raw && r < rows) {
        const float* raw = mq_part(p, b, h, rb, p.n_chunks, r);
        raw_ml[u] = *reinterpret_cast<const float2*>(raw);
        raw_a[u] = *reinterpret_cast<const float4*>(raw + MQ_PACC + 4 * lane);
      }
    }
    float x[RU][4], fr[RU], inv[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {  // rows behind `rows` hold nothing that counts
      const int r = min(r0 + u * RQ_WARPS, MQ_ROWS - 1);
      const bool live = ok_len && r < rows;
      const float mp = live && n_tiles > 0 ? sm.row_m[r] : -INFINITY, mr = live ? raw_ml[u].x : -INFINITY;
      const float M = fmaxf(mp, mr), m0 = M == -INFINITY ? 0.f : M;
      const float e = exp2f(mp - m0);
      fr[u] = exp2f(mr - m0);
      float L = fr[u] * raw_ml[u].y;
      x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
      if (mp != -INFINITY) {
        const float4 a = *reinterpret_cast<const float4*>(rowf + r * RQ_ROWF + 4 * lane);
        const float f = e * INV_SQRT_D;
        x[u][0] = f * a.x; x[u][1] = f * a.y; x[u][2] = f * a.z; x[u][3] = f * a.w;
        L += e * sm.row_l[r];
      }
      inv[u] = M == -INFINITY ? 0.f : 1.f / L;  // a row that sees nothing is zeros
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) fwht128(x[u], lane);
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const float f = fr[u], iv = inv[u];
      const float4 a = raw_a[u];
      o[u] = make_float4((x[u][0] + f * a.x) * iv, (x[u][1] + f * a.y) * iv, (x[u][2] + f * a.z) * iv,
                         (x[u][3] + f * a.w) * iv);
      if (r0 + u * RQ_WARPS >= res_rows) break;
      O* dst = out + row[u] * D + 4 * lane;
      if (kcheck(dst, 4 * sizeof(O), out, (size_t)gridDim.z * p.n_queries * p.num_q_heads * D * sizeof(O), p.err))
        store4(dst, o[u]);
    }
  }
}

template <typename E, int KBITS, int VBITS, int MODE, typename O>
cudaError_t launch_rows_t(const RowsParams& p, int batch, O* out, cudaStream_t s) {
  constexpr int PASSES = std::is_same<E, __nv_bfloat16>::value && std::is_same<O, __nv_bfloat16>::value ? 1 : 2;
  const size_t raw_smem = sizeof(RawSmem) + 128, smem = sizeof(RQSmem) + 128;
  static std::atomic<uint64_t> raw_done{0}, attr_done{0};
  cudaError_t e = smem_attr_once(raw_done, (const void*)raw_rows_kernel<E, MODE, PASSES>, (int)raw_smem);
  if (e != cudaSuccess) return e;
  e = smem_attr_once(attr_done, (const void*)rows_kernel<E, KBITS, VBITS, MODE, PASSES, O>, (int)smem);
  if (e != cudaSuccess) return e;
  const int units = p.num_kv_heads * p.n_rowblocks;
  raw_rows_kernel<E, MODE, PASSES><<<dim3(units, batch), RAW_THREADS, raw_smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_after_smem(rows_kernel<E, KBITS, VBITS, MODE, PASSES, O>, dim3(p.n_chunks, units, batch),
                        dim3(RQ_THREADS), smem, s, p, out);
  if (e != cudaSuccess || p.n_chunks == 1) return e;
  const int64_t warps = (int64_t)batch * p.n_queries * p.num_q_heads;
  return launch_after(mq_combine_kernel<MODE, O>, dim3((unsigned)((warps + 3) / 4)), dim3(128), s, p, batch, out);
}

template <int MODE, typename E, typename O>
cudaError_t launch_rows(const RowsParams& p, int batch, O* out, cudaStream_t s) {
  if (p.k_bits == 2) return launch_rows_t<E, 2, 2, MODE>(p, batch, out, s);
  return p.v_bits == 4 ? launch_rows_t<E, 4, 4, MODE>(p, batch, out, s) : launch_rows_t<E, 4, 2, MODE>(p, batch, out, s);
}

}  // namespace
}  // namespace kvarn
