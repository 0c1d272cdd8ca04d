// rows_common.cuh -- what the multi-query kernels over the packed paged cache
// share: the causal one (multiquery.cu) and those of rows_kernel.cuh, causal
// within a sliding window with visible first tokens (window.cu) and of a
// drafted token tree (tree.cu).  Operand layouts, the unpacking of records into
// them, the partial rows and their combine.
//
// Several new query tokens per sequence (a chunk of prefill, or the draft
// tokens a speculative step verifies) attend to the cache the way one decode
// query does: the closed tiles are read as packed records and dequantised
// inside the attention loop, the open tile is read raw ("Huawei's KVarN puts
// KV-cache quantization inside vLLM's backend", section "The four-stage
// pipeline": dequantisation at read time inside attention).  Query i of a
// sequence of length L sits at position L - n_queries + i and sees the
// tokens at positions <= its own.
//
// With the GQA group folded in, one KV head carries n_queries * G query rows;
// 128 of them form a row block, which makes both contractions full
// 128-row tensor-core tiles.  Per packed tile (128 tokens, one KV head):
//
//   QK (tcgen05, fp16, M = 128 rows, N = 144, K = 128 channels):
//     A = Q' (rotated, scaled query rows; fp16 hi and lo halves, two passes),
//     B = K~ with K~[t][c] = gK_c code_tc / 64 (exact in fp16) for the 128
//     tokens and K~[128][c] = gK_c / 64, so that
//       score_t = (64 / qs) (aK_t D[t] + bK_t D[128]).
//   softmax (two threads per row, one per 64-token half, scores from tensor
//     memory; the halves exchange their maxima through shared memory):
//     running reference m per row, moved only when a tile maximum exceeds it
//     by more than 8 (log2 units), which rescales the accumulator.
//   PV (tcgen05, bf16, M = 128 rows, N = 128 channels, K = 144):
//     A = P~ with P~[t] = p_t aV_t (bf16 hi and lo, two passes) and
//     P~[128], P~[129] = hi and lo of beta = sum_t p_t bV_t; B = V~ with
//     V~[c][t] = gV_c codeV_tc and V~[c][128] = V~[c][129] = gV_c (exact in
//     bf16), so the accumulator collects sum_t p_t gV_c (aV_t code + bV_t).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "tcgen05.cuh"

namespace kvarn {
namespace {

// Which tokens a query row sees: every cached token up to its own position;
// of those the first n_sinks and the last `window`; or, for a node of a
// drafted tree, every cached token and the nodes its mask row names.
constexpr int MQ_CAUSAL = 0, MQ_WINDOW = 1, MQ_TREE = 2;
template <int MODE>
using ModeParams = std::conditional_t<MODE == MQ_CAUSAL, MQParams, RowsParams>;

constexpr float MQ_LOG2E = 1.4426950408889634f;
constexpr uint32_t MAGIC_F16 = 0x64006400u;  // 1024.0 in both fp16 halves
constexpr uint32_t MAGIC_BF16 = 0x43004300u; // 128.0 in both bf16 halves
constexpr int MQ_ROWS = 128;
constexpr int MQ_PART = D + 4;  // floats per split-K partial row: m, l, 2 pad, acc[128]
constexpr int MQ_PACC = 4;
constexpr int KT_ROWS = 144;                 // 128 tokens, the g row, 15 zero rows
constexpr int KT_BYTES = KT_ROWS * D * 2;    // K~, fp16, K-major core matrices
constexpr int VT_K = 144;                    // 128 tokens, beta hi / lo, 14 zero columns
constexpr int VT_BYTES = D * VT_K * 2;       // V~, bf16, K-major core matrices
constexpr int QA_BYTES = MQ_ROWS * D * 2;
// tensor-memory columns: accumulator O, then two score buffers S (144 each).
// The softmax overwrites a tile's scores in place, first with the scaled
// scores, then with the P~ operand: for tokens 16 j .. 16 j + 15 the bf16 hi
// parts go to columns 16 j .. 16 j + 7 and the lo parts to 16 j + 8 .. 16 j + 15
// (exactly the columns those tokens' scores occupied); columns 128..135 take
// the beta entries (k 128..143).
constexpr uint32_t TM_O = 0, TM_S = 128, TM_SSTRIDE = 144, TM_COLS = 512;
constexpr uint32_t TM_QA = 416;  // Q' hi (the A operand of the first QK pass), 64 columns
constexpr uint32_t IDESC_QK = umma_idesc(128, KT_ROWS, 0);
constexpr uint32_t IDESC_PV = umma_idesc(128, D, 1);
constexpr float MQ_TAU = 8.f;  // log2 headroom before the row reference moves

template <typename E>
__device__ __forceinline__ float tof(E x) {
  if constexpr (std::is_same<E, __half>::value) return __half2float(x);
  else return __bfloat162float(x);
}
// Two 16-bit values of E (low half first) -> exact floats.
template <typename E>
__device__ __forceinline__ float2 pair_to_float2(uint32_t u) {
  if constexpr (std::is_same<E, __half>::value) return __half22float2(*reinterpret_cast<__half2*>(&u));
  else return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t b2u(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __nv_bfloat162 u2b(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }

// Byte offset of element (row r, k) of a K-major operand made of 8-row x
// 16-byte core matrices, `kb` core matrices per row group along K.
__host__ __device__ constexpr int cm_off(int r, int k, int kb) {
  return ((r >> 3) * kb + (k >> 3)) * 128 + (r & 7) * 16 + (k & 7) * 2;
}

// Channel held by contraction slot k of the QK operands.  A key word of
// 4-bit codes yields channel pairs (c, c + 4) per masked field, a word of
// 2-bit codes pairs (c, c + 8), and a pair fills two adjacent slots.
template <int KBITS>
__host__ __device__ constexpr int perm_k(int k) {
  if constexpr (KBITS == 4) {
    const int j = k & 7;
    return (k & ~7) + (j >> 1) + 4 * (j & 1);
  } else {
    const int j = k & 15;
    return (k & ~15) + (j >> 1) + 8 * (j & 1);
  }
}

// (x & mask) | magic as one three-input logic op, then y * m + a (one
// rounding; exact whenever the result is representable).
__device__ __forceinline__ uint32_t lop_magic(uint32_t x, uint32_t mask, uint32_t magic) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;\n" : "=r"(y) : "r"(x), "r"(mask), "r"(magic));
  return y;
}
__device__ __forceinline__ uint32_t fma_h(uint32_t y, __half2 m, __half2 a) { return h2u(__hfma2(u2h(y), m, a)); }
__device__ __forceinline__ uint32_t fma_b(uint32_t y, __nv_bfloat162 m, __nv_bfloat162 a) {
  return b2u(__hfma2(u2b(y), m, a));
}

__device__ __forceinline__ float* mq_part(const MQParams& p, int b, int h, int rb, int chunk, int r) {
  return p.ws + (((((int64_t)b * p.num_kv_heads + h) * p.n_rowblocks + rb) * (p.n_chunks + 1) + chunk) * MQ_ROWS + r) *
                    MQ_PART;
}

// Query tokens of sequence b (a tree may have fewer nodes than the array).
template <int MODE>
__device__ __forceinline__ int mq_queries(const ModeParams<MODE>& p, int b) {
  if constexpr (MODE == MQ_TREE)
    if (p.node_counts) return p.node_counts[b];
  return p.n_queries;
}

// Rows of row block rb and the number of closed tiles it reads, up to the
// last position any of its rows sees.
template <int MODE>
__device__ __forceinline__ void mq_block_extent(const MQParams& p, int rb, int len, int nq, int& rows, int& n_need) {
  rows = min(MQ_ROWS, nq * p.G - rb * MQ_ROWS);
  if (MODE == MQ_TREE) {
    n_need = len / T;
    return;
  }
  const int pos_hi = len - p.n_queries + (rb * MQ_ROWS + rows - 1) / p.G;
  n_need = min(len / T, pos_hi / T + 1);
}
// The closed tiles row block rb visits (MQ_WINDOW): from its first row's window on.
__device__ __forceinline__ WinTiles mq_win_tiles(const RowsParams& p, int rb, int len, int n_need) {
  return win_tiles(n_need, max(0, len - p.n_queries + (rb * MQ_ROWS) / p.G + 1 - p.window), p.n_sinks);
}

// Lengths a unit can work with; 0 marks an empty slot of a window call.
template <int MODE>
__device__ __forceinline__ bool mq_lengths_ok(const MQParams& p, int len, int nq) {
  if (len < 0 || len > T * p.max_blocks) return false;
  if (MODE == MQ_TREE) return nq >= 0 && nq <= p.n_queries;
  return len >= p.n_queries || (MODE == MQ_WINDOW && len == 0);
}

// Warp-uniform bounded wait: every lane waits, all report failure together.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, int32_t* err) {
  const bool ok = mbar_wait_parked(bar, parity, err);
  return __all_sync(0xffffffffu, ok);
}

// ---- producers: K~ rows of 8 tokens x 16 channels per thread
// Thread pth takes channels 16 cg .. 16 cg + 15 of tokens 8 (tq + 2 i) + tl,
// i = 0..7, so the 8 lanes of a store phase write 8 rows of one core matrix.
__device__ __forceinline__ int k_token(int pth, int i) { return 8 * ((pth >> 6) + 2 * i) + (pth & 7); }

template <int KBITS>
__device__ __forceinline__ void unpack_k(const unsigned char* kr, unsigned char* kt, int pth) {
  const int cg = (pth >> 3) & 7;
  const uint4 g16 = *reinterpret_cast<const uint4*>(kr + 16 * cg);
  const uint32_t gw[4] = {g16.x, g16.y, g16.z, g16.w};
  auto gval = [&](int c) { return e4m3_to_float((uint8_t)(gw[c >> 2] >> (8 * (c & 3)))); };
  if constexpr (KBITS == 4) {
    // word w (channels 8w' .. 8w'+7 of this group) -> pairs (0,4),(1,5) at bits 0 / 4, (2,6),(3,7) after >> 8
    __half2 mul[2][4], add[2][4];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int c0 = 8 * w + f, c1 = c0 + 4;
        const float sh = (f & 1) ? 1.f / 1024.f : 1.f / 64.f;   // field at bit 4 (f odd) or bit 0
        const float ad = (f & 1) ? -1.f : -16.f;
        mul[w][f] = __floats2half2_rn(gval(c0) * sh, gval(c1) * sh);
        add[w][f] = __floats2half2_rn(gval(c0) * ad, gval(c1) * ad);
      }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = k_token(pth, i);
      const uint2 cw = *reinterpret_cast<const uint2*>(kr + 512 + 64 * t + 8 * cg);
      const uint32_t wv[2] = {cw.x, cw.y};
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t x = wv[w], x8 = x >> 8;
        uint4 o;
        o.x = fma_h(lop_magic(x, 0x000F000Fu, MAGIC_F16), mul[w][0], add[w][0]);
        o.y = fma_h(lop_magic(x, 0x00F000F0u, MAGIC_F16), mul[w][1], add[w][1]);
        o.z = fma_h(lop_magic(x8, 0x000F000Fu, MAGIC_F16), mul[w][2], add[w][2]);
        o.w = fma_h(lop_magic(x8, 0x00F000F0u, MAGIC_F16), mul[w][3], add[w][3]);
        *reinterpret_cast<uint4*>(kt + cm_off(t, 16 * cg + 8 * w, 16)) = o;
      }
    }
  } else {
    // one word per token: channel pairs (j, j+8) at crumb j (j < 4) or, after >> 8, crumb j - 4
    __half2 mul[8], add[8];
#pragma unroll
    for (int f = 0; f < 8; ++f) {
      const int c0 = f, c1 = f + 8;
      const int pos = 2 * (f & 3);  // bit position of the field
      const float sh = 1.f / (64.f * (float)(1 << pos)), ad = -16.f / (float)(1 << pos);
      mul[f] = __floats2half2_rn(gval(c0) * sh, gval(c1) * sh);
      add[f] = __floats2half2_rn(gval(c0) * ad, gval(c1) * ad);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = k_token(pth, i);
      const uint32_t x = *reinterpret_cast<const uint32_t*>(kr + 512 + 32 * t + 4 * cg), x8 = x >> 8;
      uint32_t o[8];
#pragma unroll
      for (int f = 0; f < 8; ++f)
        o[f] = fma_h(lop_magic(f < 4 ? x : x8, 0x00030003u << (2 * (f & 3)), MAGIC_F16), mul[f], add[f]);
      *reinterpret_cast<uint4*>(kt + cm_off(t, 16 * cg, 16)) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(kt + cm_off(t, 16 * cg + 8, 16)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// ---- producers: zero operands for a tile whose block id is out of range
// (its record buffer holds no data; the rows mask every token of it)
__device__ __forceinline__ void zero_k(unsigned char* kt, int pth) {
  const int cg = (pth >> 3) & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    *reinterpret_cast<uint4*>(kt + cm_off(k_token(pth, i), 16 * cg, 16)) = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(kt + cm_off(k_token(pth, i), 16 * cg + 8, 16)) = make_uint4(0u, 0u, 0u, 0u);
  }
}
__device__ __forceinline__ void zero_v(unsigned char* vt, int c) {
#pragma unroll
  for (int k8 = 0; k8 < 17; ++k8) *reinterpret_cast<uint4*>(vt + cm_off(c, 8 * k8, VT_K / 8)) = make_uint4(0u, 0u, 0u, 0u);
}

// ---- producers: V~ row of channel c (128 tokens) plus its gV entries
template <int VBITS>
__device__ __forceinline__ void unpack_v(const unsigned char* vr, unsigned char* vt, int c) {
  if constexpr (VBITS == 4) {
    // 16 words of 8 tokens; token pair (2s, 2s + 1) of word w at bits 4s, 16 + 4s:
    // shifted to bits 0 and 16, each field reads 128 + code in bf16
    const float gv = e4m3_to_float(vr[c]);
    const __nv_bfloat162 m0 = __float2bfloat162_rn(gv), a0 = __float2bfloat162_rn(-128.f * gv);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 c4 = *reinterpret_cast<const uint4*>(vr + 512 + 64 * c + 16 * q);
      const uint32_t wv[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t x = wv[e];
        uint32_t o[4];
#pragma unroll
        for (int s2 = 0; s2 < 4; ++s2) o[s2] = fma_b(lop_magic(x >> (4 * s2), 0x000F000Fu, MAGIC_BF16), m0, a0);
        *reinterpret_cast<uint4*>(vt + cm_off(c, 8 * (4 * q + e), VT_K / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    const uint32_t g2 = b2u(m0);  // k 128..131: beta hi, lo of the two row halves
    *reinterpret_cast<uint4*>(vt + cm_off(c, 128, VT_K / 8)) = make_uint4(g2, g2, 0u, 0u);
    return;
  }
  // a field at bit q reads 128 + 2^q code: times gV / 2^q, minus 128 gV / 2^q
  const float gv = e4m3_to_float(vr[c]);
  const __nv_bfloat162 m0 = __float2bfloat162_rn(gv), m2 = __float2bfloat162_rn(gv * 0.25f),
                       m4 = __float2bfloat162_rn(gv * 0.0625f);
  const __nv_bfloat162 a0 = __float2bfloat162_rn(-128.f * gv), a2 = __float2bfloat162_rn(-32.f * gv),
                       a4 = __float2bfloat162_rn(-8.f * gv);
  const uint4 c0 = *reinterpret_cast<const uint4*>(vr + 512 + 32 * c);
  const uint4 c1 = *reinterpret_cast<const uint4*>(vr + 512 + 32 * c + 16);
  const uint32_t wv[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    // tokens 16w + (2s, 2s+1) sit at bits 2s of the low / high half-word
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
    *reinterpret_cast<uint4*>(vt + cm_off(c, 16 * w, VT_K / 8)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(vt + cm_off(c, 16 * w + 8, VT_K / 8)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
  const uint32_t g2 = b2u(m0);  // k 128..131: beta hi, lo of the two row halves
  *reinterpret_cast<uint4*>(vt + cm_off(c, 128, VT_K / 8)) = make_uint4(g2, g2, 0u, 0u);
}

// One warp per output row (sequence, query, query head): merge the split-K
// partials, rotate the packed part back, add the raw part, normalise.
// O: float, or a 16-bit type (one rounding of the fp32 result).
template <int MODE, typename O>
__global__ void __launch_bounds__(128) mq_combine_kernel(ModeParams<MODE> p, int batch, O* __restrict__ out) {
  wait_prerequisite();  // the split-K kernel's partial rows
  const int wid = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int per_seq = p.n_queries * p.num_q_heads;
  if (wid >= batch * per_seq) return;
  const int b = wid / per_seq, qi = (wid % per_seq) / p.num_q_heads, hq = wid % p.num_q_heads;
  const int h = hq / p.G, gq = hq % p.G;
  const int R = qi * p.G + gq, rb = R / MQ_ROWS, r = R % MQ_ROWS;
  const int len = p.seq_lens[b], nq = mq_queries<MODE>(p, b);
  if (MODE == MQ_TREE && (nq > p.n_queries || qi >= nq)) return;  // rows behind a sequence's tree stay as they are
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const float* plo = mq_part(p, b, h, rb, 0, r);
  const size_t pspan = (size_t)(mq_part(p, b, h, rb, p.n_chunks, r) + MQ_PART - plo) * sizeof(float);
  if (mq_lengths_ok<MODE>(p, len, nq) && (MODE == MQ_TREE || len > 0) &&
      kcheck(plo, pspan, p.ws, (size_t)p.ws_bytes, p.err)) {
    int rows, n_need;
    mq_block_extent<MODE>(p, rb, len, nq, rows, n_need);
    if constexpr (MODE == MQ_WINDOW) n_need = mq_win_tiles(p, rb, len, n_need).n;
    const int n_c = (n_need + p.chunk_tiles - 1) / p.chunk_tiles;
    const bool has_tail = MODE == MQ_TREE || (len % T) != 0;  // a tree's raw part holds its nodes
    // lane i holds the header of chunk i, so every load of a group of 32
    // chunks is in flight at once; the sums run in chunk order
    const float* tail = mq_part(p, b, h, rb, p.n_chunks, r);
    float M = has_tail ? tail[0] : -INFINITY;
    for (int i = lane; i < n_c; i += 32) M = fmaxf(M, mq_part(p, b, h, rb, i, r)[0]);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, m));
    float Lsum = 0.f;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    if (M != -INFINITY) {
      for (int i0 = 0; i0 < n_c; i0 += 32) {
        float fl = 0.f, ll = 0.f;
        if (i0 + lane < n_c) {
          const float2 ml = *reinterpret_cast<const float2*>(mq_part(p, b, h, rb, i0 + lane, r));
          fl = (ml.x == -INFINITY) ? 0.f : exp2f(ml.x - M);
          ll = ml.y;
        }
#pragma unroll 4
        for (int i = i0; i < min(n_c, i0 + 32); ++i) {
          const float f = __shfl_sync(0xffffffffu, fl, i - i0), l = __shfl_sync(0xffffffffu, ll, i - i0);
          const float4 a = *reinterpret_cast<const float4*>(mq_part(p, b, h, rb, i, r) + MQ_PACC + 4 * lane);
          Lsum += f * l;
          x[0] += f * a.x; x[1] += f * a.y; x[2] += f * a.z; x[3] += f * a.w;
        }
      }
    }
    // x = x H / sqrt(128) over the 128 channels held 4 per lane
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
      for (int e = 0; e < 4; ++e) {
        const float other = __shfl_xor_sync(0xffffffffu, x[e], m);
        x[e] = upper ? (other - x[e]) : (x[e] + other);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= INV_SQRT_D;
    if (has_tail && M != -INFINITY) {
      const float* pp = mq_part(p, b, h, rb, p.n_chunks, r);
      const float f = (pp[0] == -INFINITY) ? 0.f : exp2f(pp[0] - M);
      Lsum += f * pp[1];
      const float4 a = *reinterpret_cast<const float4*>(pp + MQ_PACC + 4 * lane);
      x[0] += f * a.x; x[1] += f * a.y; x[2] += f * a.z; x[3] += f * a.w;
    }
    const float inv = (MODE != MQ_CAUSAL || Lsum > 0.f) ? 1.f / Lsum : 0.f;
    if (MODE == MQ_CAUSAL || M != -INFINITY) o = make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
  }
  O* dst = out + (((int64_t)b * p.n_queries + qi) * p.num_q_heads + hq) * D + 4 * lane;
  if (kcheck(dst, 4 * sizeof(O), out, (size_t)batch * p.n_queries * p.num_q_heads * D * sizeof(O), p.err))
    store4(dst, o);
}

}  // namespace
}  // namespace kvarn
