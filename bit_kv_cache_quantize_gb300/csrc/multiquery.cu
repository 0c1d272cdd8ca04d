// multiquery.cu -- causal multi-query attention over the packed paged cache
// (operands and formulas: rows_common.cuh).
//
// Warp roles per CTA (13 warps, one CTA per SM): warps 0-7 run the softmax
// (warp w: rows 32 (w & 3) .. + 31, token half w >> 2), warps 8-11 unpack
// records into the K~ / V~ operands (their first thread refills a record
// stage once all of them are done with it), one thread of warp 12 issues
// the first bulk copies and the MMAs.  Operands that a later tile reuses are
// double-buffered (K~, scores, scales) or guarded by the previous PV (V~).
#include "rows_common.cuh"

namespace kvarn {
namespace {

constexpr int MQ_THREADS = 416;  // warps 0-7 softmax (two per row quarter), 8-11 unpack, 12 issue
constexpr int REC_STAGES = 3;

struct MQSmem {
  alignas(128) unsigned char qa_lo[QA_BYTES];  // Q' lo (the hi half lives in tensor memory)
  alignas(128) unsigned char kt[2][KT_BYTES];
  alignas(128) unsigned char vt[VT_BYTES];
  alignas(128) unsigned char rec[REC_STAGES][HEAD_REC_MAX];  // K record | V record (either widths)
  alignas(16) float ka[2][T], kb[2][T];  // aK, bK per token (per K~ stage)
  alignas(16) float va[2][T], vb[2][T];  // aV, bV per token
  alignas(16) float xmax[2][2][MQ_ROWS];  // tile maximum of each row half (exchanged between halves)
  alignas(16) float xl[2][MQ_ROWS];       // row sums of the two halves at the end
  float qsi[MQ_ROWS];                     // 1 / qs of each row
  uint64_t rec_full[REC_STAGES], rec_empty[REC_STAGES], kt_full[2], qk_done[2], p_full[2], xbar[2];
  uint64_t s_full[2], vt_full, pv_done, fin, lbar;
  uint32_t tmem;
  uint32_t vmask;  // bit k: block id of tile k of this chunk is in range
};
struct MQTailSmem {
  float k[T][D];
  float v[T][D];
};
static_assert(sizeof(MQTailSmem) <= sizeof(MQSmem), "tail buffers fit the packed layout");

// Raw open tile: rows of this row block against its len % 128 tokens, fp32
// on the CUDA cores; two threads per row (64 channels each).
template <typename E>
__device__ void mq_tail(const MQParams& p, int b, int h, int rb, int len, unsigned char* smem) {
  const int n = len % T;
  if (n == 0) return;
  MQTailSmem& sm = *reinterpret_cast<MQTailSmem*>(smem);
  const int tid = threadIdx.x;
  const E* kt = static_cast<const E*>(p.tail) + (((int64_t)b * p.num_kv_heads + h) * 2 + 0) * (T * D);
  const E* vt = kt + T * D;
  for (int i = tid; i < n * D; i += blockDim.x) {
    sm.k[i / D][i % D] = tof(kt[i]);
    sm.v[i / D][i % D] = tof(vt[i]);
  }
  __syncthreads();
  if (tid >= 2 * MQ_ROWS) return;
  const int r = tid >> 1, half = tid & 1;
  int rows, n_need;
  mq_block_extent<MQ_CAUSAL>(p, rb, len, p.n_queries, rows, n_need);
  const int R = rb * MQ_ROWS + r;
  const bool rv = r < rows;
  const int qi = rv ? R / p.G : 0, gq = rv ? R % p.G : 0;
  const int pos = rv ? len - p.n_queries + qi : -1;
  const int t0 = len - n;  // position of slot 0
  const int nv = min(n, pos - t0 + 1);  // tail tokens this row sees (may be <= 0)
  // the query half row stays in its 16-bit pairs (exact); scale after the dot product
  uint32_t q2[32];
  float acc[64];
  {
    const uint4* qr = reinterpret_cast<const uint4*>(
        static_cast<const E*>(p.q) +
        (((int64_t)b * p.n_queries + qi) * p.num_q_heads + (int64_t)h * p.G + gq) * D + 64 * half);
#pragma unroll
    for (int c8 = 0; c8 < 8; ++c8) {
      const uint4 v = rv ? qr[c8] : make_uint4(0u, 0u, 0u, 0u);
      q2[4 * c8] = v.x; q2[4 * c8 + 1] = v.y; q2[4 * c8 + 2] = v.z; q2[4 * c8 + 3] = v.w;
    }
#pragma unroll
    for (int c = 0; c < 64; ++c) acc[c] = 0.f;
  }
  const float fscale = p.scale * MQ_LOG2E;
  float m = -INFINITY, l = 0.f;
  for (int tb = 0; tb < n; tb += 8) {
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = min(tb + i, T - 1);
      float a = 0.f;
      const float4* kk = reinterpret_cast<const float4*>(&sm.k[t][64 * half]);
#pragma unroll
      for (int c4 = 0; c4 < 16; ++c4) {
        const float4 kv = kk[c4];
        const float2 q01 = pair_to_float2<E>(q2[2 * c4]), q23 = pair_to_float2<E>(q2[2 * c4 + 1]);
        a = fmaf(q01.x, kv.x, a);
        a = fmaf(q01.y, kv.y, a);
        a = fmaf(q23.x, kv.z, a);
        a = fmaf(q23.y, kv.w, a);
      }
      a += __shfl_xor_sync(0xffffffffu, a, 1);
      s[i] = (tb + i < nv) ? a * fscale : -INFINITY;
    }
    float bm = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) bm = fmaxf(bm, s[i]);
    if (bm == -INFINITY) continue;
    if (bm > m) {
      const float corr = (m == -INFINITY) ? 0.f : exp2f(m - bm);
      l *= corr;
#pragma unroll
      for (int c = 0; c < 64; ++c) acc[c] *= corr;
      m = bm;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float pr = exp2f(s[i] - m);
      l += pr;
      if (pr != 0.f) {
        const float4* vv = reinterpret_cast<const float4*>(&sm.v[min(tb + i, T - 1)][64 * half]);
#pragma unroll
        for (int c4 = 0; c4 < 16; ++c4) {
          const float4 v4 = vv[c4];
          acc[4 * c4] = fmaf(pr, v4.x, acc[4 * c4]);
          acc[4 * c4 + 1] = fmaf(pr, v4.y, acc[4 * c4 + 1]);
          acc[4 * c4 + 2] = fmaf(pr, v4.z, acc[4 * c4 + 2]);
          acc[4 * c4 + 3] = fmaf(pr, v4.w, acc[4 * c4 + 3]);
        }
      }
    }
  }
  if (!rv) return;
  float* o = mq_part(p, b, h, rb, p.n_chunks, r);
  if (!kcheck(o, MQ_PART * sizeof(float), p.ws, (size_t)p.ws_bytes, p.err)) return;
  if (half == 0) { o[0] = m; o[1] = l; }
#pragma unroll
  for (int c4 = 0; c4 < 16; ++c4)
    *reinterpret_cast<float4*>(o + MQ_PACC + 64 * half + 4 * c4) =
        make_float4(acc[4 * c4], acc[4 * c4 + 1], acc[4 * c4 + 2], acc[4 * c4 + 3]);
}

// grid (n_chunks + 1, num_kv_heads * n_rowblocks, batch) x 416 threads;
// chunk n_chunks handles the raw open tile.
template <typename E, int KBITS, int VBITS>
__global__ void __launch_bounds__(MQ_THREADS, 1) mq_kernel(MQParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  allow_dependents();  // the combine may be scheduled once every CTA has started
  const int chunk = blockIdx.x, h = blockIdx.y / p.n_rowblocks, rb = blockIdx.y % p.n_rowblocks, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int len = p.seq_lens[b];
  if (len < p.n_queries || len > T * p.max_blocks) {
    if (tid == 0 && chunk == 0 && blockIdx.y == 0) set_error(p.err, KVARN_DEV_ERR_TOKEN_RANGE);
    return;
  }
  const uint32_t sbase = smem_u32(smem_raw);
  unsigned char* base = smem_raw + (((sbase + 127u) & ~127u) - sbase);
  if (chunk == p.n_chunks) {
    mq_tail<E>(p, b, h, rb, len, base);
    return;
  }
  int rows, n_need;
  mq_block_extent<MQ_CAUSAL>(p, rb, len, p.n_queries, rows, n_need);
  const int first = chunk * p.chunk_tiles;
  const int n_tiles = min(p.chunk_tiles, n_need - first);
  if (n_tiles <= 0) return;
  constexpr int KREC = rec_bytes(KBITS), VREC = rec_bytes(VBITS);
  MQSmem& sm = *reinterpret_cast<MQSmem*>(base);
  const int32_t* tab = p.block_table + (int64_t)b * p.max_blocks + first;

  uint32_t vmask = 0;  // bit k: block id of tile k of this chunk is in range
  // one bulk copy of the K and V records of tile k into its stage (one thread)
  auto issue_rec = [&](int k) {
    const int s = k % REC_STAGES;
    const unsigned char* src = p.pool + tab[k] * p.block_bytes + (int64_t)h * (KREC + VREC);
    if (((vmask >> k) & 1u) && kcheck(src, KREC + VREC, p.pool, (size_t)p.num_blocks * p.block_bytes, p.err)) {
      mbar_expect_tx(&sm.rec_full[s], KREC + VREC);
      bulk_g2s(sm.rec[s], src, KREC + VREC, &sm.rec_full[s]);
    } else {
      set_error(p.err, KVARN_DEV_ERR_BLOCK_RANGE);
      mbar_arrive(&sm.rec_full[s]);
    }
  };
  if (warp == 12) {
    // block ids (a lane each), barriers, and the first records on their way
    // while the other warps rotate the queries
    const int32_t blk = lane < n_tiles ? tab[lane] : -1;
    vmask = __ballot_sync(0xffffffffu, blk >= 0 && blk < p.num_blocks);
    if (lane == 0) {
      for (int s = 0; s < REC_STAGES; ++s) {
        mbar_init(&sm.rec_full[s], 1);
        mbar_init(&sm.rec_empty[s], 128);
      }
      for (int s = 0; s < 2; ++s) {
        mbar_init(&sm.kt_full[s], 128);
        mbar_init(&sm.qk_done[s], 1);
        mbar_init(&sm.p_full[s], 256);
        mbar_init(&sm.xbar[s], 256);
      }
      mbar_init(&sm.s_full[0], 1);
      mbar_init(&sm.s_full[1], 1);
      mbar_init(&sm.vt_full, 128);
      mbar_init(&sm.pv_done, 1);
      mbar_init(&sm.fin, 1);
      mbar_init(&sm.lbar, 256);
      fence_mbar_init();
      sm.vmask = vmask;
      for (int k = 0; k < min(n_tiles, REC_STAGES); ++k) issue_rec(k);
    }
    __syncwarp();
    tmem_alloc(&sm.tmem, TM_COLS);
  }

  // ---- prologue: query operand (warps 0-3, a thread per row), constant
  // operand regions (producers)
  const int q4 = warp & 3, half = (warp >> 2) & 1;  // softmax warps: row quarter, token half
  const int r = 32 * q4 + lane;
  const int R = rb * MQ_ROWS + r;
  const bool rv = warp < 8 && r < rows;
  const int qi = rv ? R / p.G : 0;
  if (warp < 8) {
    // warp w rotates rows 16 w .. 16 w + 15, 4 channels per lane: x = q H
    // (4-point butterflies in registers, then across lanes), 8 rows at a
    // time staged in shared memory (the second K~ buffer, free until the
    // main loop), then written as fp16 hi / lo core-matrix rows so that the
    // 8 lanes of a store phase write 8 different rows
    float* stage = reinterpret_cast<float*>(sm.kt[1]) + warp * (8 * 132);  // 8 rows of 132 floats per warp
    // All sixteen rows are on their way before the first is needed, into the
    // place of their own lo parts.  Four rows a turn: rotating all sixteen in
    // one straight line is no faster and its code takes 10 us of a small call
    // that finds it in no cache (8 x 4096 tokens, 2 queries, L2 flushed: 72 us
    // against 62; rows loaded one by one 65, and 650 against 615 at 32 x 16 K).
#pragma unroll 4
    for (int rr = 0; rr < 16; ++rr) {
      const int row = 16 * warp + rr, Rr = rb * MQ_ROWS + row;
      unsigned char* dst = sm.qa_lo + row * 256 + 8 * lane;
      if (row < rows)
        cp_async8(dst, static_cast<const E*>(p.q) +
                           (((int64_t)b * p.n_queries + Rr / p.G) * p.num_q_heads + (int64_t)h * p.G + Rr % p.G) * D +
                           4 * lane);
      else
        *reinterpret_cast<uint2*>(dst) = make_uint2(0u, 0u);
    }
    cp_async_wait_all();
    __syncwarp();
#pragma unroll 1
    for (int rg = 0; rg < 2; ++rg) {
#pragma unroll 4
      for (int rr = 0; rr < 8; ++rr) {
        const int row = 16 * warp + 8 * rg + rr;
        float x[4];
        {
          const uint2 raw = *reinterpret_cast<const uint2*>(sm.qa_lo + row * 256 + 8 * lane);  // this lane's own copy
          const float2 lo = pair_to_float2<E>(raw.x), hi = pair_to_float2<E>(raw.y);
          x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
        }
        float u = x[0], v = x[1];
        x[0] = u + v; x[1] = u - v;
        u = x[2]; v = x[3];
        x[2] = u + v; x[3] = u - v;
        u = x[0]; v = x[2];
        x[0] = u + v; x[2] = u - v;
        u = x[1]; v = x[3];
        x[1] = u + v; x[3] = u - v;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const bool upper = (lane & m) != 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, x[i], m);
            x[i] = upper ? (o - x[i]) : (x[i] + o);
          }
        }
        const float f = p.scale * MQ_LOG2E * INV_SQRT_D;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] *= f;
          amax = fmaxf(amax, fabsf(x[i]));
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        int ex = 0;
        if (amax > 0.f) frexpf(amax, &ex);
        const float qs = ldexpf(1.f, 7 - ex);  // max |Q'| in [64, 128)
        if (lane == 0) sm.qsi[row] = ldexpf(1.f, ex - 7);
        *reinterpret_cast<float4*>(stage + rr * 132 + 4 * lane) = make_float4(x[0] * qs, x[1] * qs, x[2] * qs, x[3] * qs);
      }
      __syncwarp();
      // lane: row rr = lane & 7, core-matrix columns g = (lane >> 3) + 4 j
      const int rr = lane & 7, row = 16 * warp + 8 * rg + rr;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int g = (lane >> 3) + 4 * j;
        // slot pairs (2i, 2i + 1) hold channels (ca + i, cb + i): K4 (8g, 8g + 4), K2 (16 (g/2) + 4 (g&1), + 8)
        const int ca = (KBITS == 4) ? 8 * g : 16 * (g >> 1) + 4 * (g & 1), cb = ca + ((KBITS == 4) ? 4 : 8);
        const float4 va = *reinterpret_cast<const float4*>(stage + rr * 132 + ca);
        const float4 vb = *reinterpret_cast<const float4*>(stage + rr * 132 + cb);
        const float av[4] = {va.x, va.y, va.z, va.w}, bv[4] = {vb.x, vb.y, vb.z, vb.w};
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 hi = __floats2half2_rn(av[i], bv[i]);
          const float2 hf = __half22float2(hi);
          hw[i] = h2u(hi);
          lw[i] = h2u(__floats2half2_rn(av[i] - hf.x, bv[i] - hf.y));
        }
        // hi: staged in the V~ buffer (free until the main loop), lo: the shared-memory operand
        *reinterpret_cast<uint4*>(sm.vt + cm_off(row, 8 * g, 16)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(sm.qa_lo + cm_off(row, 8 * g, 16)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
      }
      __syncwarp();
    }
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  vmask = sm.vmask;
  if (warp < 4) {  // Q' hi of row r -> tensor-memory lane r, columns TM_QA .. +63 (the A operand layout)
    const uint32_t lb = tmem + ((uint32_t)(warp * 32) << 16) + TM_QA;
    const int row = tid;
#pragma unroll
    for (int c = 0; c < 64; c += 16) {
      uint32_t w16[16];
#pragma unroll
      for (int g2 = 0; g2 < 4; ++g2) {
        const uint4 v4 = *reinterpret_cast<const uint4*>(sm.vt + cm_off(row, 2 * c + 8 * g2, 16));
        w16[4 * g2] = v4.x; w16[4 * g2 + 1] = v4.y; w16[4 * g2 + 2] = v4.z; w16[4 * g2 + 3] = v4.w;
      }
      tmem_st16(lb + c, w16);
    }
    tmem_wait_st();
  } else if (warp >= 8 && warp < 12) {
    const int pth = tid - 256;
    for (int i = pth; i < 2 * 15 * 16; i += 128) {  // K~ rows 129..143 of both stages
      const int s = i / (15 * 16), rr = 129 + (i / 16) % 15, kg = i % 16;
      *reinterpret_cast<uint4*>(sm.kt[s] + cm_off(rr, 8 * kg, 16)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp == 12) {
    // ------------------------------------------------------------ MMA issue (one thread)
    if (lane == 0) {
      const uint64_t qa_lo = umma_desc(smem_u32(sm.qa_lo), 128, 2048);
      auto issue_qk = [&](int k) {  // S[k & 1] = Q' K~^T over the hi then the lo query halves
        const uint32_t kb = smem_u32(sm.kt[k & 1]), d = tmem + TM_S + TM_SSTRIDE * (k & 1);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ts(d, tmem + TM_QA + 8 * kk, umma_desc(kb + 256 * kk, 128, 2048), IDESC_QK, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ss(d, qa_lo + (uint64_t)(16 * kk), umma_desc(kb + 256 * kk, 128, 2048), IDESC_QK, 1);
        umma_commit(&sm.qk_done[k & 1]);
        umma_commit(&sm.s_full[k & 1]);
      };
      auto issue_pv = [&](int k) {  // D_O += P~ V~^T over the hi (with beta) then the lo halves
        const uint32_t vb = smem_u32(sm.vt), pa = tmem + TM_S + TM_SSTRIDE * (k & 1);
#pragma unroll
        for (int kk = 0; kk < 9; ++kk)  // hi parts of tokens 16 kk .. 16 kk + 15, then the beta block
          umma_ts(tmem + TM_O, pa + 16 * kk, umma_desc(vb + 256 * kk, 128, VT_K * 16), IDESC_PV,
                  (k > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // lo parts
          umma_ts(tmem + TM_O, pa + 16 * kk + 8, umma_desc(vb + 256 * kk, 128, VT_K * 16), IDESC_PV, 1);
        umma_commit(&sm.pv_done);
      };
      bool ok = true;
      for (int k = 0; ok && k < min(n_tiles, 2); ++k) {  // both score buffers start free
        ok = mbar_wait_parked(&sm.kt_full[k], 0, p.err);
        if (!ok) break;
        tc_fence_after();
        issue_qk(k);
      }
      for (int k = 0; ok && k < n_tiles; ++k) {
        ok = mbar_wait_parked(&sm.p_full[k & 1], (k >> 1) & 1, p.err) && mbar_wait_parked(&sm.vt_full, k & 1, p.err);
        if (!ok) break;
        tc_fence_after();
        issue_pv(k);
        if (k + 2 < n_tiles) {  // buffer k & 1 is free once PV(k) has read its P~
          ok = mbar_wait_parked(&sm.kt_full[k & 1], ((k + 2) >> 1) & 1, p.err) &&
               mbar_wait_parked(&sm.pv_done, k & 1, p.err);
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
  } else if (warp >= 8) {
    // ------------------------------------------------------------ producers
    const int pth = tid - 256;
    // V~ columns 136..143 stay zero (the buffer held the query staging until the last barrier)
    *reinterpret_cast<uint4*>(sm.vt + cm_off(pth, 136, VT_K / 8)) = make_uint4(0u, 0u, 0u, 0u);
    bool ok = true;
    for (int k = -1; k < n_tiles; ++k) {
      const int j = k + 1;  // K~ of the next tile first, then V~ of this one
      if (j < n_tiles) {
        const int s = j % REC_STAGES;
        ok = wait_all(&sm.rec_full[s], (j / REC_STAGES) & 1, p.err);
        if (ok && j >= 2)
          ok = wait_all(&sm.qk_done[j & 1], ((j - 2) >> 1) & 1, p.err) &&
               wait_all(&sm.p_full[j & 1], ((j - 2) >> 1) & 1, p.err);
        if (!ok) break;
        const unsigned char* kr = sm.rec[s];
        const unsigned char* vr = kr + KREC;
        if ((vmask >> j) & 1u) {
          sm.ka[j & 1][pth] = e4m3_to_float(kr[128 + pth]);
          sm.kb[j & 1][pth] = __half2float(*reinterpret_cast<const __half*>(kr + 256 + 2 * pth));
          sm.va[j & 1][pth] = e4m3_to_float(vr[128 + pth]);
          sm.vb[j & 1][pth] = __half2float(*reinterpret_cast<const __half*>(vr + 256 + 2 * pth));
          unpack_k<KBITS>(kr, sm.kt[j & 1], pth);
          if (pth < 16) {  // the g row: K~[128][k] = gK of the slot's channel / 64
            uint32_t o[4];
#pragma unroll
            for (int jj = 0; jj < 4; ++jj)
              o[jj] = h2u(__floats2half2_rn(e4m3_to_float(kr[perm_k<KBITS>(8 * pth + 2 * jj)]) * (1.f / 64.f),
                                            e4m3_to_float(kr[perm_k<KBITS>(8 * pth + 2 * jj + 1)]) * (1.f / 64.f)));
            *reinterpret_cast<uint4*>(sm.kt[j & 1] + cm_off(128, 8 * pth, 16)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
        } else {
          sm.ka[j & 1][pth] = sm.kb[j & 1][pth] = sm.va[j & 1][pth] = sm.vb[j & 1][pth] = 0.f;
          zero_k(sm.kt[j & 1], pth);
          if (pth < 16)
            *reinterpret_cast<uint4*>(sm.kt[j & 1] + cm_off(128, 8 * pth, 16)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
        mbar_arrive(&sm.kt_full[j & 1]);
      }
      if (k >= 0) {
        if (k >= 1) ok = wait_all(&sm.pv_done, (k - 1) & 1, p.err);
        if (!ok) break;
        if ((vmask >> k) & 1u) unpack_v<VBITS>(sm.rec[k % REC_STAGES] + KREC, sm.vt, pth);
        else zero_v(sm.vt, pth);
        fence_proxy_async();
        mbar_arrive(&sm.vt_full);
        mbar_arrive(&sm.rec_empty[k % REC_STAGES]);
        if (pth == 0 && k + REC_STAGES < n_tiles) {  // every producer is done with this stage: refill it
          if (mbar_wait_parked(&sm.rec_empty[k % REC_STAGES], (k / REC_STAGES) & 1, p.err)) issue_rec(k + REC_STAGES);
        }
      }
    }
    // copies still in flight (an early exit) land before the CTA ends
    if (!ok && pth == 0) {
      for (int k = 0; k < n_tiles; ++k) mbar_wait_parked(&sm.rec_full[k % REC_STAGES], (k / REC_STAGES) & 1, p.err);
    }
  } else {
    // ------------------------------------------------------------ softmax: row r, tokens 64 half .. +63
    const uint32_t lane_base = tmem + ((uint32_t)(q4 * 32) << 16);
    const int pos = rv ? len - p.n_queries + qi : -1;
    const float cr = 64.f * sm.qsi[r];  // score (log2) = cr (aK D_t + bK D_128)
    const float2 cr2 = make_float2(cr, cr);
    float m_ref = -INFINITY, l_sum = 0.f;
    bool dead = false;
    for (int k = 0; k < n_tiles; ++k) {
      const int s = k & 1;
      const uint32_t sb = lane_base + TM_S + TM_SSTRIDE * s;  // this tile's score / P~ buffer
      if (!wait_all(&sm.s_full[s], (k >> 1) & 1, p.err)) { dead = true; break; }
      tc_fence_after();
      // pass 1: scores s = aK D_t + bK D_128 (units of 1 / cr) of this half's 64
      // tokens, written back in place, and their maximum; masked tokens -> -inf
      float d128;
      {
        uint32_t d1;
        tmem_ld1(sb + 128, d1);
        tmem_wait_ld();
        d128 = __uint_as_float(d1);
      }
      // the scales of this tile (written with its K~; that phase is complete)
      if (!wait_all(&sm.kt_full[s], (k >> 1) & 1, p.err)) { dead = true; break; }
      const int t0 = (first + k) * T + 64 * half;
      const int nvis = ((vmask >> k) & 1u) ? min(64, pos - t0 + 1) : 0;  // tokens of this half the row sees
      const float2 d2 = make_float2(d128, d128);
      float tmax = -INFINITY;
      // the causal mask, in a second copy of the loop that only a tile with
      // hidden tokens takes (padded rows are never written, so they may skip it)
      auto pass1 = [&](auto mask_c) {
        constexpr bool MASK = decltype(mask_c)::value;
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          uint32_t d[16];
          tmem_ld16(sb + 64 * half + c, d);
          const float4* ka4 = reinterpret_cast<const float4*>(sm.ka[s] + 64 * half + c);
          const float4* kb4 = reinterpret_cast<const float4*>(sm.kb[s] + 64 * half + c);
          float4 a4[4], b4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) { a4[j] = ka4[j]; b4[j] = kb4[j]; }
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 s01 = ffma2(make_float2(a4[j].x, a4[j].y),
                               make_float2(__uint_as_float(d[4 * j]), __uint_as_float(d[4 * j + 1])),
                               fmul2(make_float2(b4[j].x, b4[j].y), d2));
            float2 s23 = ffma2(make_float2(a4[j].z, a4[j].w),
                               make_float2(__uint_as_float(d[4 * j + 2]), __uint_as_float(d[4 * j + 3])),
                               fmul2(make_float2(b4[j].z, b4[j].w), d2));
            const int t = c + 4 * j;
            if (MASK && nvis < 64) {
              if (t >= nvis) s01.x = -INFINITY;
              if (t + 1 >= nvis) s01.y = -INFINITY;
              if (t + 2 >= nvis) s23.x = -INFINITY;
              if (t + 3 >= nvis) s23.y = -INFINITY;
            }
            tmax = fmaxf(tmax, fmaxf(fmaxf(s01.x, s01.y), fmaxf(s23.x, s23.y)));
            d[4 * j] = __float_as_uint(s01.x); d[4 * j + 1] = __float_as_uint(s01.y);
            d[4 * j + 2] = __float_as_uint(s23.x); d[4 * j + 3] = __float_as_uint(s23.y);
          }
          tmem_st16(sb + 64 * half + c, d);
        }
      };
      if (__all_sync(0xffffffffu, !rv || nvis >= 64)) pass1(std::false_type{});
      else pass1(std::true_type{});
      tmem_wait_st();
      tc_fence_before();  // both halves read D_128 before either writes beta (ordered by xbar)
      // the row maximum: exchange with the other half through shared memory
      sm.xmax[k & 1][half][r] = tmax;
      mbar_arrive(&sm.xbar[k & 1]);
      if (!wait_all(&sm.xbar[k & 1], (k >> 1) & 1, p.err)) { dead = true; break; }
      tc_fence_after();
      tmax = fmaxf(tmax, sm.xmax[k & 1][half ^ 1][r]) * cr;
      float corr = 1.f;
      bool resc = false;
      if (tmax > m_ref + MQ_TAU) {
        if (m_ref != -INFINITY) {
          corr = ex2_ftz(m_ref - tmax);
          resc = true;
        }
        m_ref = tmax;
        l_sum *= corr;
      }
      const bool live = m_ref != -INFINITY;
      if (__any_sync(0xffffffffu, resc)) {  // rescale the accumulator once the previous PV is done
        if (k > 0 && !wait_all(&sm.pv_done, (k - 1) & 1, p.err)) { dead = true; break; }
        tc_fence_after();
        uint32_t d[16];
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
          tmem_ld16(lane_base + TM_O + 64 * half + c, d);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) d[i] = __float_as_uint(__uint_as_float(d[i]) * corr);
          tmem_st16(lane_base + TM_O + 64 * half + c, d);
        }
      }
      // pass 2: P~ = p aV (bf16 hi, lo) over the scores of each 16-token group,
      // l += sum p, beta += sum p bV
      const float2 nm2 = make_float2(-m_ref, -m_ref);
      float2 lt = make_float2(0.f, 0.f), bt = make_float2(0.f, 0.f);
      // a row that has seen no token yet (reference still -inf) gets p = 0, in
      // a second copy of the loop that only such tiles take
      auto pass2 = [&](auto zero_c) {
        constexpr bool ZERO = decltype(zero_c)::value;
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          uint32_t d[16];
          tmem_ld16(sb + 64 * half + c, d);
          const float4* va4 = reinterpret_cast<const float4*>(sm.va[s] + 64 * half + c);
          const float4* vb4 = reinterpret_cast<const float4*>(sm.vb[s] + 64 * half + c);
          float4 a4[4], b4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) { a4[j] = va4[j]; b4[j] = vb4[j]; }
          tmem_wait_ld();
          uint32_t pw[16];  // hi words 0..7, lo words 8..15
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 e01 = ffma2(cr2, make_float2(__uint_as_float(d[4 * j]), __uint_as_float(d[4 * j + 1])), nm2);
            const float2 e23 = ffma2(cr2, make_float2(__uint_as_float(d[4 * j + 2]), __uint_as_float(d[4 * j + 3])), nm2);
            float2 p01 = make_float2(ex2_ftz(e01.x), ex2_ftz(e01.y)), p23 = make_float2(ex2_ftz(e23.x), ex2_ftz(e23.y));
            if (ZERO && !live) p01 = p23 = make_float2(0.f, 0.f);
            lt = fadd2(lt, fadd2(p01, p23));
            bt = ffma2(p01, make_float2(b4[j].x, b4[j].y), ffma2(p23, make_float2(b4[j].z, b4[j].w), bt));
            const float2 x01 = fmul2(p01, make_float2(a4[j].x, a4[j].y)), x23 = fmul2(p23, make_float2(a4[j].z, a4[j].w));
            const __nv_bfloat162 h01 = __floats2bfloat162_rn(x01.x, x01.y), h23 = __floats2bfloat162_rn(x23.x, x23.y);
            const float2 r01 = ffma2(__bfloat1622float2(h01), make_float2(-1.f, -1.f), x01);  // x - hi, exact product
            const float2 r23 = ffma2(__bfloat1622float2(h23), make_float2(-1.f, -1.f), x23);
            pw[2 * j] = b2u(h01);
            pw[2 * j + 1] = b2u(h23);
            pw[8 + 2 * j] = b2u(__floats2bfloat162_rn(r01.x, r01.y));
            pw[8 + 2 * j + 1] = b2u(__floats2bfloat162_rn(r23.x, r23.y));
          }
          tmem_st16(sb + 64 * half + c, pw);
        }
      };
      if (__all_sync(0xffffffffu, !rv || live)) pass2(std::false_type{});
      else pass2(std::true_type{});
      l_sum += lt.x + lt.y;
      {
        const float beta = bt.x + bt.y;
        const __nv_bfloat16 bh = __float2bfloat16_rn(beta);
        const __nv_bfloat16 bl = __float2bfloat16_rn(beta - __bfloat162float(bh));
        tmem_st1(sb + 128 + half, (uint32_t)__bfloat16_as_ushort(bh) | ((uint32_t)__bfloat16_as_ushort(bl) << 16));
        if (half) {  // k 132..143 of the beta block are zero
          tmem_st2(sb + 130, 0u, 0u);
          tmem_st4(sb + 132, 0u, 0u, 0u, 0u);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.p_full[s]);
    }
    // ---- this CTA's partial of each row: half h writes channels 64 h .. 64 h + 63
    // All products are in (fin, not pv_done: a softmax warp may be here before
    // PV(n_tiles - 2) is done, and a wait on the parity of the last phase would
    // then pass on the one before it).
    bool ok = !dead && wait_all(&sm.fin, 0, p.err);
    sm.xl[half][r] = l_sum;
    mbar_arrive(&sm.lbar);
    ok = wait_all(&sm.lbar, 0, p.err) && ok;
    tc_fence_after();
    float* o = mq_part(p, b, h, rb, chunk, rv ? r : 0);
    const bool wv = rv && kcheck(o, MQ_PART * sizeof(float), p.ws, (size_t)p.ws_bytes, p.err);
    if (wv && half == 0) {
      o[0] = ok ? m_ref : -INFINITY;
      o[1] = ok ? l_sum + sm.xl[1][r] : 0.f;
    }
#pragma unroll
    for (int c = 0; c < 64; c += 16) {
      uint32_t d[16];
      tmem_ld16(lane_base + TM_O + 64 * half + c, d);
      tmem_wait_ld();
      if (wv) {
        float* oa = o + MQ_PACC + 64 * half + c;
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(oa + i) = ok ? make_float4(__uint_as_float(d[i]), __uint_as_float(d[i + 1]),
                                                                __uint_as_float(d[i + 2]), __uint_as_float(d[i + 3]))
                                                  : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, TM_COLS);
}

template <typename E, int KBITS, int VBITS>
cudaError_t launch_mq_t(const MQParams& p, int batch, float* out, cudaStream_t s) {
  const size_t smem = sizeof(MQSmem) + 128;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = smem_attr_once(attr_done, (const void*)mq_kernel<E, KBITS, VBITS>, (int)smem);
  if (e != cudaSuccess) return e;
  mq_kernel<E, KBITS, VBITS><<<dim3(p.n_chunks + 1, p.num_kv_heads * p.n_rowblocks, batch), MQ_THREADS, smem, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int warps = batch * p.n_queries * p.num_q_heads;
  return launch_after(mq_combine_kernel<MQ_CAUSAL, float>, dim3((warps + 3) / 4), dim3(128), s, p, batch, out);
}

}  // namespace

cudaError_t launch_multiquery(const MQParams& p, int dtype, int batch, float* out, cudaStream_t s) {
  if (p.k_bits == 2)
    return dtype == KVARN_DTYPE_BF16 ? launch_mq_t<__nv_bfloat16, 2, 2>(p, batch, out, s)
                                     : launch_mq_t<__half, 2, 2>(p, batch, out, s);
  if (p.v_bits == 4)
    return dtype == KVARN_DTYPE_BF16 ? launch_mq_t<__nv_bfloat16, 4, 4>(p, batch, out, s)
                                     : launch_mq_t<__half, 4, 4>(p, batch, out, s);
  return dtype == KVARN_DTYPE_BF16 ? launch_mq_t<__nv_bfloat16, 4, 2>(p, batch, out, s)
                                   : launch_mq_t<__half, 4, 2>(p, batch, out, s);
}

size_t multiquery_ws_bytes(int batch, int num_kv_heads, int n_rowblocks, int max_blocks, int chunk_tiles) {
  const size_t n_chunks = (size_t)(max_blocks + chunk_tiles - 1) / chunk_tiles;
  return (size_t)batch * num_kv_heads * n_rowblocks * (n_chunks + 1) * MQ_ROWS * MQ_PART * sizeof(float);
}

}  // namespace kvarn
