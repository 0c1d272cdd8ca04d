// kvarn_abi.cu -- the extern "C" entry points declared in include/kvarn.h:
// host-side validation, launch configuration and status codes.  No
// allocation, no global state, no exceptions across the boundary.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/kvarn.h"

#include "params.h"

namespace kvarn {
constexpr int kChunkTiles = 16;  // packed tiles per split-K CTA of an ordinary call (sizes the workspace)
constexpr int kSmallChunkTiles = 8;  // of a small call: two tiles per warp of its 4-warp CTAs
// A call whose table spans fewer (sequence, KV head, tile) units than this
// is small: 16-tile chunks would give it under three waves of two 8-warp
// CTAs per SM on 152 SMs (3 x 304 x 16), so it takes 8-tile chunks, twice
// the CTAs.  The rule depends only on the call's shape, so the workspace
// size does too.
constexpr long long kSmallCallUnits = 3LL * 304 * 16;

static bool small_call(int batch, int num_kv_heads, int max_blocks) {
  return (long long)batch * num_kv_heads * max_blocks < kSmallCallUnits;
}

// Fewest packed tiles per split-K CTA a call of this shape may use.
static int min_chunk_tiles(int batch, int num_kv_heads, int max_blocks) {
  return small_call(batch, num_kv_heads, max_blocks) ? kSmallChunkTiles : kChunkTiles;
}

// Packed tiles per split-K CTA for one call: 8 for a small call; else the
// longest of 64 and 32 (longer CTAs amortise the per-CTA query set-up and
// merge) that still gives at least three waves of CTAs at two per SM, else 16.
// The K4/V4 preset, whose CTAs have 4 warps, stops at 32 (8 tiles a warp).
static int choose_chunk_tiles(const kvarn_config* cfg, int batch, int num_kv_heads, int max_blocks) {
  if (small_call(batch, num_kv_heads, max_blocks)) return kSmallChunkTiles;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return kChunkTiles;
  const long long units = (long long)batch * num_kv_heads;
  for (int chunk : {64, 32})
    if ((chunk == 32 || cfg->v_bits != 4) && units * ((max_blocks + chunk - 1) / chunk) >= 6LL * sms) return chunk;
  return kChunkTiles;
}
constexpr int kF16ChunkTiles = 16;
constexpr int kMaxTableBlocks = (1 << 24) - 1;  // 128 x the columns stays an int32 (window, tree, pages)

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Shape checks shared by every entry point.
static kvarn_status check_config(const kvarn_config* c) {
  if (!c) return KVARN_ERR_INVALID;
  if (c->num_kv_heads < 1 || c->num_q_heads < 1 || c->num_blocks < 0 || c->sinkhorn_iters < 0 ||
      c->sinkhorn_iters > 64 || c->head_dim < 1 || c->tile_tokens < 1)
    return KVARN_ERR_INVALID;
  if (c->num_q_heads % c->num_kv_heads) return KVARN_ERR_INVALID;
  if (c->dtype != KVARN_DTYPE_F16 && c->dtype != KVARN_DTYPE_BF16) return KVARN_ERR_INVALID;
  // presets: kvarn_k4v2 (4-bit keys, 2-bit values), K2/V2 and K4/V4
  const bool preset = (c->k_bits == 4 && c->v_bits == 2) || (c->k_bits == 2 && c->v_bits == 2) ||
                      (c->k_bits == 4 && c->v_bits == 4);
  if (c->head_dim != 128 || c->tile_tokens != 128 || !preset) return KVARN_ERR_UNSUPPORTED;
  if (c->num_q_heads / c->num_kv_heads > 8) return KVARN_ERR_UNSUPPORTED;
  return KVARN_OK;
}

static kvarn_status cuda_status(cudaError_t e) { return e == cudaSuccess ? KVARN_OK : KVARN_ERR_CUDA; }
}  // namespace kvarn

using namespace kvarn;

extern "C" {

size_t kvarn_block_bytes(const kvarn_config* cfg) {
  if (check_config(cfg) != KVARN_OK) return 0;
  return static_cast<size_t>(cfg->num_kv_heads) * head_rec(cfg->k_bits, cfg->v_bits);
}

size_t kvarn_tail_bytes(const kvarn_config* cfg, int32_t batch) {
  if (check_config(cfg) != KVARN_OK || batch < 0) return 0;
  return static_cast<size_t>(batch) * cfg->num_kv_heads * 2 * 128 * 128 * 2;
}

size_t kvarn_fp16_block_bytes(const kvarn_config* cfg) {
  if (check_config(cfg) != KVARN_OK) return 0;
  return static_cast<size_t>(cfg->num_kv_heads) * 2 * 128 * 128 * 2;
}

size_t kvarn_decode_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t max_blocks) {
  if (check_config(cfg) != KVARN_OK || batch < 0 || max_blocks < 1) return 0;
  const int G = cfg->num_q_heads / cfg->num_kv_heads;
  const size_t a = decode_ws_bytes(batch, cfg->num_kv_heads, G, max_blocks,
                                   min_chunk_tiles(batch, cfg->num_kv_heads, max_blocks));
  const size_t b = decode_ws_bytes(batch, cfg->num_kv_heads, G, max_blocks, kF16ChunkTiles);
  return a > b ? a : b;
}

kvarn_status kvarn_quantize_tiles(const kvarn_config* cfg, const void* k, const void* v, int64_t token_stride_elems,
                                  int64_t n_tokens, const int64_t* tile_first_token, const int32_t* tile_dst_block,
                                  int32_t n_tiles, void* block_pool, int32_t* dev_err, void* stream) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (n_tiles < 0 || n_tokens < 0) return KVARN_ERR_INVALID;
  if (n_tiles == 0) return KVARN_OK;
  if (!k || !v || !tile_first_token || !tile_dst_block || (!block_pool && cfg->num_blocks > 0)) return KVARN_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(block_pool)) return KVARN_ERR_INVALID;
  if (token_stride_elems % 8 || token_stride_elems < static_cast<int64_t>(cfg->num_kv_heads) * 128)
    return KVARN_ERR_INVALID;
  if (static_cast<int64_t>(n_tiles) * cfg->num_kv_heads * 2 > 0x7fffffffLL) return KVARN_ERR_INVALID;
  QuantizeParams p{k, v, token_stride_elems, n_tokens, tile_first_token, tile_dst_block,
                   static_cast<unsigned char*>(block_pool), static_cast<int64_t>(kvarn_block_bytes(cfg)),
                   cfg->num_kv_heads, cfg->num_blocks, cfg->sinkhorn_iters, cfg->k_bits, cfg->v_bits, dev_err};
  return cuda_status(launch_quantize(p, cfg->dtype, n_tiles, static_cast<cudaStream_t>(stream)));
}

size_t kvarn_token_errors_scratch_bytes(const kvarn_config* cfg, int32_t n_tiles, int32_t is_v) {
  if (check_config(cfg) != KVARN_OK || n_tiles < 0) return 0;
  return static_cast<size_t>(n_tiles) * cfg->num_kv_heads *
         static_cast<size_t>(is_v ? rec_bytes(cfg->v_bits) : rec_bytes(cfg->k_bits));
}

kvarn_status kvarn_token_errors(const kvarn_config* cfg, const void* x, int64_t token_stride_elems, int64_t n_tokens,
                                const int64_t* tile_first_token, int32_t n_tiles, int32_t is_v, int32_t rotate,
                                int32_t sinkhorn_iters, void* scratch, size_t scratch_bytes, float* out,
                                int32_t* dev_err, void* stream) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (n_tiles < 0 || n_tokens < 0 || (is_v != 0 && is_v != 1) || (rotate != 0 && rotate != 1) ||
      sinkhorn_iters < 0 || sinkhorn_iters > 64)
    return KVARN_ERR_INVALID;
  if (n_tiles == 0) return KVARN_OK;
  if (!x || !tile_first_token || !scratch || !out) return KVARN_ERR_INVALID;
  if (!aligned16(x) || !aligned16(scratch) || !aligned16(out)) return KVARN_ERR_INVALID;
  if (token_stride_elems % 8 || token_stride_elems < static_cast<int64_t>(cfg->num_kv_heads) * 128)
    return KVARN_ERR_INVALID;
  if (static_cast<int64_t>(n_tiles) * cfg->num_kv_heads > 0x7fffffffLL) return KVARN_ERR_INVALID;
  if (scratch_bytes < kvarn_token_errors_scratch_bytes(cfg, n_tiles, is_v)) return KVARN_ERR_INVALID;
  ErrParams p{x, token_stride_elems, n_tokens, tile_first_token, static_cast<unsigned char*>(scratch), out,
              cfg->num_kv_heads, sinkhorn_iters, cfg->k_bits, cfg->v_bits, is_v, rotate, dev_err};
  return cuda_status(launch_token_errors(p, cfg->dtype, n_tiles, static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_append_tokens(const kvarn_config* cfg, const void* k_new, const void* v_new, const int32_t* pos,
                                 const int32_t* block_table, int32_t max_blocks, int32_t batch, void* tail_pool,
                                 void* block_pool, int32_t* dev_err, void* stream) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || max_blocks < 1) return KVARN_ERR_INVALID;
  if (batch == 0) return KVARN_OK;
  if (static_cast<int64_t>(batch) * cfg->num_kv_heads * 2 > 0x7fffffffLL) return KVARN_ERR_INVALID;
  if (!k_new || !v_new || !pos || !block_table || !tail_pool || (!block_pool && cfg->num_blocks > 0)) return KVARN_ERR_INVALID;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(tail_pool) || !aligned16(block_pool))
    return KVARN_ERR_INVALID;
  AppendParams p{k_new, v_new, pos, block_table, max_blocks, cfg->num_kv_heads, cfg->num_blocks, cfg->sinkhorn_iters,
                 tail_pool, static_cast<unsigned char*>(block_pool), static_cast<int64_t>(kvarn_block_bytes(cfg)),
                 cfg->k_bits, cfg->v_bits, dev_err};
  return cuda_status(launch_append(p, cfg->dtype, batch, static_cast<cudaStream_t>(stream)));
}

static kvarn_status check_decode(const kvarn_config* cfg, const void* q, const int32_t* block_table,
                                 int32_t max_blocks, const int32_t* seq_lens, int32_t batch, const void* pool,
                                 float* out, void* workspace, size_t workspace_bytes) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || max_blocks < 1 || batch > 65535) return KVARN_ERR_INVALID;
  if (batch == 0) return KVARN_OK;
  if (!q || !block_table || !seq_lens || (!pool && cfg->num_blocks > 0) || !out || !workspace) return KVARN_ERR_INVALID;
  if (!aligned16(q) || !aligned16(pool) || !aligned16(out) || !aligned16(workspace)) return KVARN_ERR_INVALID;
  if (workspace_bytes < kvarn_decode_workspace_bytes(cfg, batch, max_blocks)) return KVARN_ERR_INVALID;
  return KVARN_OK;
}

static kvarn_status decode_call(const kvarn_config* cfg, const void* q, const int32_t* block_table,
                                int32_t max_blocks, const int32_t* seq_lens, int32_t batch, const void* block_pool,
                                const void* tail_pool, float softmax_scale, float* out, void* workspace,
                                size_t workspace_bytes, int32_t* dev_err, void* stream, int32_t wait_polls,
                                int32_t skip_first_copy) {
  kvarn_status st = check_decode(cfg, q, block_table, max_blocks, seq_lens, batch, block_pool, out, workspace,
                                 workspace_bytes);
  if (st != KVARN_OK || batch == 0) return st;
  if (!tail_pool || !aligned16(tail_pool)) return KVARN_ERR_INVALID;
  const int chunk = choose_chunk_tiles(cfg, batch, cfg->num_kv_heads, max_blocks);
  const int n_chunks = (max_blocks + chunk - 1) / chunk;
  DecodeParams p{q, block_table, seq_lens, static_cast<const unsigned char*>(block_pool), tail_pool,
                 static_cast<float*>(workspace), dev_err, static_cast<int64_t>(kvarn_block_bytes(cfg)), softmax_scale,
                 max_blocks, cfg->num_kv_heads, cfg->num_q_heads, cfg->num_q_heads / cfg->num_kv_heads,
                 cfg->num_blocks, chunk, n_chunks, cfg->k_bits, cfg->v_bits, wait_polls, skip_first_copy,
                 static_cast<int64_t>(workspace_bytes)};
  return cuda_status(launch_decode(p, cfg->dtype, batch, out, static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_decode_attention(const kvarn_config* cfg, const void* q, const int32_t* block_table,
                                    int32_t max_blocks, const int32_t* seq_lens, int32_t batch, const void* block_pool,
                                    const void* tail_pool, float softmax_scale, float* out, void* workspace,
                                    size_t workspace_bytes, int32_t* dev_err, void* stream) {
  return decode_call(cfg, q, block_table, max_blocks, seq_lens, batch, block_pool, tail_pool, softmax_scale, out,
                     workspace, workspace_bytes, dev_err, stream, 0, 0);
}

kvarn_status kvarn_test_decode_wait_expiry(const kvarn_config* cfg, const void* q, const int32_t* block_table,
                                           int32_t max_blocks, const int32_t* seq_lens, int32_t batch,
                                           const void* block_pool, const void* tail_pool, float softmax_scale,
                                           float* out, void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                           int32_t wait_polls, void* stream) {
  if (wait_polls < 1) return KVARN_ERR_INVALID;
  return decode_call(cfg, q, block_table, max_blocks, seq_lens, batch, block_pool, tail_pool, softmax_scale, out,
                     workspace, workspace_bytes, dev_err, stream, wait_polls, 1);
}

// Packed tiles per split-K CTA of the multi-query kernel (one CTA per SM):
// 32 while that leaves at least three waves, else 16 (sizes the workspace).
static int choose_mq_chunk(int units, int max_blocks) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return kChunkTiles;
  const long long ctas = (long long)units * ((max_blocks + 31) / 32);
  return ctas >= 3LL * sms ? 32 : kChunkTiles;
}

static int mq_rowblocks(const kvarn_config* cfg, int n_queries) {
  const int G = cfg->num_q_heads / cfg->num_kv_heads;
  return (n_queries * G + 127) / 128;
}

size_t kvarn_multiquery_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t max_blocks,
                                        int32_t n_queries) {
  if (check_config(cfg) != KVARN_OK || batch < 0 || max_blocks < 1 || n_queries < 1 || n_queries > 4096) return 0;
  return multiquery_ws_bytes(batch, cfg->num_kv_heads, mq_rowblocks(cfg, n_queries), max_blocks, kChunkTiles);
}

kvarn_status kvarn_multiquery_attention(const kvarn_config* cfg, const void* q, int32_t n_queries,
                                        const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                                        int32_t batch, const void* block_pool, const void* tail_pool,
                                        float softmax_scale, float* out, void* workspace, size_t workspace_bytes,
                                        int32_t* dev_err, void* stream) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || max_blocks < 1 || batch > 65535 || n_queries < 1 || n_queries > 4096) return KVARN_ERR_INVALID;
  if (batch == 0) return KVARN_OK;
  if (!q || !block_table || !seq_lens || (!block_pool && cfg->num_blocks > 0) || !tail_pool || !out || !workspace)
    return KVARN_ERR_INVALID;
  if (!aligned16(q) || !aligned16(block_pool) || !aligned16(tail_pool) || !aligned16(out) || !aligned16(workspace))
    return KVARN_ERR_INVALID;
  if (workspace_bytes < kvarn_multiquery_workspace_bytes(cfg, batch, max_blocks, n_queries)) return KVARN_ERR_INVALID;
  const int n_rb = mq_rowblocks(cfg, n_queries);
  if ((long long)cfg->num_kv_heads * n_rb > 65535) return KVARN_ERR_UNSUPPORTED;
  const int chunk = choose_mq_chunk(batch * cfg->num_kv_heads * n_rb, max_blocks);
  const int n_chunks = (max_blocks + chunk - 1) / chunk;
  MQParams p{q, block_table, seq_lens, static_cast<const unsigned char*>(block_pool), tail_pool,
             static_cast<float*>(workspace), dev_err, static_cast<int64_t>(kvarn_block_bytes(cfg)), softmax_scale,
             max_blocks, cfg->num_kv_heads, cfg->num_q_heads, cfg->num_q_heads / cfg->num_kv_heads, cfg->num_blocks,
             n_queries, n_rb, chunk, n_chunks, cfg->k_bits, cfg->v_bits, static_cast<int64_t>(workspace_bytes)};
  return cuda_status(launch_multiquery(p, cfg->dtype, batch, out, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ window, tree
// Shapes of the window and tree calls, and with them the split and the
// workspace, follow from the arguments alone: 152 SMs.
static constexpr int kSMs = 152;

// A window's single query whose sequences visit at most n_vis closed tiles.
// A small call runs as one cluster per (sequence, KV head): up to seven CTAs
// of 4 tiles (one per warp) or 8 and one for the open tile, if they are all
// resident at once (two per SM); no workspace.  Otherwise the longest chunk of
// 64 and 32 tiles that leaves three waves of CTAs, else 16 (as the full
// decode), or 8 where that gives too few CTAs.
constexpr int kClusterMax = 8;
static int window_chunk(const kvarn_config* cfg, int64_t units, int n_vis, int* cluster) {
  for (int chunk : {4, 8}) {
    const int64_t ctas = (n_vis + chunk - 1) / chunk + 1;
    if (ctas <= kClusterMax && units * ctas <= 2 * kSMs) {
      *cluster = 1;
      return chunk;
    }
  }
  *cluster = 0;
  if (units * n_vis < kSmallCallUnits) return kSmallChunkTiles;
  for (int chunk : {64, 32})
    if ((chunk == 32 || cfg->v_bits != 4) && units * ((n_vis + chunk - 1) / chunk) >= 6LL * kSMs) return chunk;
  return kChunkTiles;
}

// Packed tiles per split-K CTA (one per SM) of a multi-query window or tree
// call: the split whose waves of CTAs take the least time, each CTA costing
// its tiles plus a set-up of about kMqSetup tiles' time.  Beyond 32 tiles only
// where six waves of CTAs remain, which even out sequences of different length;
// up to 128, which bounds what one long sequence adds.  (32 sequences x 64
// drafted nodes x 16 K tokens: one chunk of 128 tiles instead of four of 32
// spares the partial rows and their combine.)
static constexpr int kMqSetup = 3;
static int short_mq_chunk(int64_t units, int n_vis) {
  int best = 1;
  int64_t least = INT64_MAX;
  for (int c = 1; c <= 128 && c <= n_vis; ++c) {
    const int64_t ctas = units * ((n_vis + c - 1) / c), waves = (ctas + kSMs - 1) / kSMs, cost = waves * (c + kMqSetup);
    if (c > 32 && ctas < 6 * kSMs) break;
    if (cost <= least) { least = cost; best = c; }
  }
  return best;
}

struct WindowShape {
  int window, n_sinks;  // clipped to the table
  int n_vis;            // closed tiles a unit visits, at most
  int n_rb;             // row blocks per KV head (several queries)
  int chunk, n_chunks;
  int cluster;
  size_t ws_bytes;
};

static kvarn_status window_shape(const kvarn_config* cfg, int32_t batch, int32_t max_blocks, int32_t n_queries,
                                 int32_t window, int32_t n_sinks, WindowShape* w) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || batch > 65535 || max_blocks < 1 || max_blocks > kMaxTableBlocks || n_queries < 1 ||
      n_queries > 4096 || window < 1 || n_sinks < 0)
    return KVARN_ERR_INVALID;
  const int G = cfg->num_q_heads / cfg->num_kv_heads, tokens = 128 * max_blocks;
  if ((int64_t)batch * n_queries * cfg->num_q_heads > 0x7fffffffLL) return KVARN_ERR_UNSUPPORTED;
  w->window = window < tokens ? window : tokens;
  w->n_sinks = n_sinks < tokens ? n_sinks : tokens;
  // the rows of a unit span `span` positions, so their windows reach over
  // window + span - 1 tokens: at most that many tiles, plus a partial one at
  // each end (a single query's end is the open tile)
  const int span = n_queries == 1 ? 1 : (n_queries < 128 / G + 2 ? n_queries : 128 / G + 2);
  const int64_t tiles = (w->n_sinks + 127) / 128 +
                        (n_queries == 1 ? ((int64_t)w->window + 127) / 128 : ((int64_t)w->window + span - 2) / 128 + 2);
  w->n_vis = tiles < max_blocks ? (int)tiles : max_blocks;
  if (n_queries == 1) {
    const int64_t units = (int64_t)batch * cfg->num_kv_heads;
    w->n_rb = 0;
    w->chunk = window_chunk(cfg, units, w->n_vis, &w->cluster);
    w->ws_bytes = w->cluster ? 16 : decode_ws_bytes(batch, cfg->num_kv_heads, G, w->n_vis, w->chunk);
  } else {
    w->n_rb = mq_rowblocks(cfg, n_queries);
    if ((long long)cfg->num_kv_heads * w->n_rb > 65535) return KVARN_ERR_UNSUPPORTED;
    w->chunk = short_mq_chunk((int64_t)batch * cfg->num_kv_heads * w->n_rb, w->n_vis);
    w->ws_bytes = multiquery_ws_bytes(batch, cfg->num_kv_heads, w->n_rb, w->n_vis, w->chunk);
  }
  w->n_chunks = (w->n_vis + w->chunk - 1) / w->chunk;
  return KVARN_OK;
}

size_t kvarn_window_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t max_blocks, int32_t n_queries,
                                    int32_t window, int32_t n_sinks) {
  WindowShape w;
  return window_shape(cfg, batch, max_blocks, n_queries, window, n_sinks, &w) == KVARN_OK ? w.ws_bytes : 0;
}

kvarn_status kvarn_window_attention(const kvarn_config* cfg, const void* q, int32_t n_queries,
                                    const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                                    int32_t batch, int32_t window, int32_t n_sinks, const void* block_pool,
                                    const void* tail_pool, float softmax_scale, void* out, int32_t out_dtype,
                                    void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  WindowShape w;
  kvarn_status st = window_shape(cfg, batch, max_blocks, n_queries, window, n_sinks, &w);
  if (st != KVARN_OK) return st;
  if (out_dtype != KVARN_OUT_F32 && out_dtype != KVARN_OUT_16) return KVARN_ERR_INVALID;
  if (batch == 0) return KVARN_OK;
  if (!q || !block_table || !seq_lens || (!block_pool && cfg->num_blocks > 0) || !tail_pool || !out || !workspace)
    return KVARN_ERR_INVALID;
  if (!aligned16(q) || !aligned16(block_pool) || !aligned16(tail_pool) || !aligned16(out) || !aligned16(workspace))
    return KVARN_ERR_INVALID;
  if (workspace_bytes < w.ws_bytes) return KVARN_ERR_INVALID;
  const int G = cfg->num_q_heads / cfg->num_kv_heads;
  const auto pool = static_cast<const unsigned char*>(block_pool);
  const bool out16 = out_dtype == KVARN_OUT_16;
  if (n_queries == 1) {
    WindowParams p{{q, block_table, seq_lens, pool, tail_pool, static_cast<float*>(workspace), dev_err,
                   static_cast<int64_t>(kvarn_block_bytes(cfg)), softmax_scale, max_blocks, cfg->num_kv_heads,
                   cfg->num_q_heads, G, cfg->num_blocks, w.chunk, w.n_chunks, cfg->k_bits, cfg->v_bits, 0, 0,
                   static_cast<int64_t>(workspace_bytes)}, w.window, w.n_sinks, batch, w.cluster};
    return cuda_status(launch_window_decode(p, cfg->dtype, batch, out, out16, static_cast<cudaStream_t>(stream)));
  }
  RowsParams p{{q, block_table, seq_lens, pool, tail_pool, static_cast<float*>(workspace), dev_err,
             static_cast<int64_t>(kvarn_block_bytes(cfg)), softmax_scale, max_blocks, cfg->num_kv_heads,
             cfg->num_q_heads, G, cfg->num_blocks, n_queries, w.n_rb, w.chunk, w.n_chunks, cfg->k_bits, cfg->v_bits,
             static_cast<int64_t>(workspace_bytes)}, w.window, w.n_sinks};
  return cuda_status(launch_window_multiquery(p, cfg->dtype, batch, out, out16, static_cast<cudaStream_t>(stream)));
}

struct TreeShape {
  int n_rb, chunk, n_chunks;
  size_t ws_bytes;
};

static kvarn_status tree_shape(const kvarn_config* cfg, int32_t batch, int32_t max_blocks, int32_t n_nodes,
                               TreeShape* t) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || batch > 65535 || max_blocks < 1 || max_blocks > kMaxTableBlocks || n_nodes < 1)
    return KVARN_ERR_INVALID;
  if (n_nodes > KVARN_TREE_MAX_NODES) return KVARN_ERR_UNSUPPORTED;
  if ((int64_t)batch * n_nodes * cfg->num_q_heads > 0x7fffffffLL) return KVARN_ERR_UNSUPPORTED;
  t->n_rb = mq_rowblocks(cfg, n_nodes);
  if ((long long)cfg->num_kv_heads * t->n_rb > 65535) return KVARN_ERR_UNSUPPORTED;
  t->chunk = short_mq_chunk((int64_t)batch * cfg->num_kv_heads * t->n_rb, max_blocks);
  t->n_chunks = (max_blocks + t->chunk - 1) / t->chunk;
  t->ws_bytes = multiquery_ws_bytes(batch, cfg->num_kv_heads, t->n_rb, max_blocks, t->chunk);
  return KVARN_OK;
}

size_t kvarn_tree_workspace_bytes(const kvarn_config* cfg, int32_t batch, int32_t max_blocks, int32_t n_nodes) {
  TreeShape t;
  return tree_shape(cfg, batch, max_blocks, n_nodes, &t) == KVARN_OK ? t.ws_bytes : 0;
}

kvarn_status kvarn_tree_attention(const kvarn_config* cfg, const void* q, const void* k_draft, const void* v_draft,
                                  const uint64_t* tree_mask, int32_t n_nodes, const int32_t* node_counts,
                                  const int32_t* block_table, int32_t max_blocks, const int32_t* seq_lens,
                                  int32_t batch, const void* block_pool, const void* tail_pool, float softmax_scale,
                                  void* out, int32_t out_dtype, void* workspace, size_t workspace_bytes,
                                  int32_t* dev_err, void* stream) {
  TreeShape t;
  kvarn_status st = tree_shape(cfg, batch, max_blocks, n_nodes, &t);
  if (st != KVARN_OK) return st;
  if (out_dtype != KVARN_OUT_F32 && out_dtype != KVARN_OUT_16) return KVARN_ERR_INVALID;
  if (batch == 0) return KVARN_OK;
  if (!q || !k_draft || !v_draft || !tree_mask || !block_table || !seq_lens ||
      (!block_pool && cfg->num_blocks > 0) || !tail_pool || !out || !workspace)
    return KVARN_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_draft) || !aligned16(v_draft) || !aligned16(block_pool) || !aligned16(tail_pool) ||
      !aligned16(out) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return KVARN_ERR_INVALID;
  if (workspace_bytes < t.ws_bytes) return KVARN_ERR_INVALID;
  RowsParams p{{q, block_table, seq_lens, static_cast<const unsigned char*>(block_pool), tail_pool,
             static_cast<float*>(workspace), dev_err, static_cast<int64_t>(kvarn_block_bytes(cfg)), softmax_scale,
             max_blocks, cfg->num_kv_heads, cfg->num_q_heads, cfg->num_q_heads / cfg->num_kv_heads, cfg->num_blocks,
             n_nodes, t.n_rb, t.chunk, t.n_chunks, cfg->k_bits, cfg->v_bits, static_cast<int64_t>(workspace_bytes)},
             0, 0, k_draft, v_draft, tree_mask, node_counts};
  return cuda_status(launch_tree(p, cfg->dtype, batch, out, out_dtype == KVARN_OUT_16,
                                 static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_commit_tokens(const kvarn_config* cfg, const void* k_draft, const void* v_draft, int32_t n_nodes,
                                 const int32_t* path, int32_t max_path, const int32_t* path_lens, const int32_t* pos,
                                 const int32_t* block_table, int32_t max_blocks, int32_t batch, void* tail_pool,
                                 void* block_pool, int32_t* dev_err, void* stream) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || max_blocks < 1 || max_blocks > kMaxTableBlocks || n_nodes < 1 || max_path < 1 ||
      (!path && max_path > n_nodes))
    return KVARN_ERR_INVALID;
  if (max_path > 128) return KVARN_ERR_UNSUPPORTED;
  if (batch == 0) return KVARN_OK;
  if (static_cast<int64_t>(batch) * cfg->num_kv_heads * 2 > 0x7fffffffLL) return KVARN_ERR_INVALID;
  if (!k_draft || !v_draft || !path_lens || !pos || !block_table || !tail_pool || (!block_pool && cfg->num_blocks > 0))
    return KVARN_ERR_INVALID;
  if (!aligned16(k_draft) || !aligned16(v_draft) || !aligned16(tail_pool) || !aligned16(block_pool))
    return KVARN_ERR_INVALID;
  CommitParams p{k_draft, v_draft, path, path_lens, n_nodes, max_path,
                 AppendParams{nullptr, nullptr, pos, block_table, max_blocks, cfg->num_kv_heads, cfg->num_blocks,
                              cfg->sinkhorn_iters, tail_pool, static_cast<unsigned char*>(block_pool),
                              static_cast<int64_t>(kvarn_block_bytes(cfg)), cfg->k_bits, cfg->v_bits, dev_err}};
  return cuda_status(launch_commit(p, cfg->dtype, batch, static_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------------------ pages
static kvarn_status check_pages(const kvarn_config* cfg, const void* table, int32_t max_blocks, int32_t batch,
                                const void* refs) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || max_blocks < 1 || max_blocks > kMaxTableBlocks || (int64_t)batch * max_blocks > 0x7fffffffLL)
    return KVARN_ERR_INVALID;
  if (batch == 0) return KVARN_OK;
  if (!table || (!refs && cfg->num_blocks > 0) || !aligned16(refs)) return KVARN_ERR_INVALID;
  return KVARN_OK;
}

size_t kvarn_pages_workspace_bytes(const kvarn_config* cfg, int32_t batch) {
  if (check_config(cfg) != KVARN_OK || batch < 0) return 0;
  return pages_ws_bytes(cfg->num_blocks);
}

static PageParams page_params(const kvarn_config* cfg, int32_t* table, int32_t max_blocks, int32_t batch, int32_t* refs,
                              int32_t* dev_err) {
  PageParams p = {};
  p.table = table;
  p.refs = refs;
  p.err = dev_err;
  p.max_blocks = max_blocks;
  p.batch = batch;
  p.num_blocks = cfg->num_blocks;
  return p;
}

kvarn_status kvarn_alloc_blocks(const kvarn_config* cfg, int32_t* block_table, int32_t max_blocks, int32_t batch,
                                const int32_t* tile_begin, const int32_t* tile_end, int32_t* refs, void* workspace,
                                size_t workspace_bytes, int32_t* dev_err, void* stream) {
  kvarn_status st = check_pages(cfg, block_table, max_blocks, batch, refs);
  if (st != KVARN_OK || batch == 0) return st;
  if (!tile_begin || !tile_end || !workspace || !aligned16(workspace) ||
      workspace_bytes < pages_ws_bytes(cfg->num_blocks))
    return KVARN_ERR_INVALID;
  PageParams p = page_params(cfg, block_table, max_blocks, batch, refs, dev_err);
  p.tile_begin = tile_begin;
  p.tile_end = tile_end;
  p.ws = static_cast<int32_t*>(workspace);
  return cuda_status(launch_alloc(p, static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_free_blocks(const kvarn_config* cfg, int32_t* block_table, int32_t max_blocks, int32_t batch,
                               const int32_t* tile_begin, const int32_t* tile_end, int32_t* refs, int32_t* dev_err,
                               void* stream) {
  kvarn_status st = check_pages(cfg, block_table, max_blocks, batch, refs);
  if (st != KVARN_OK || batch == 0) return st;
  if (!tile_begin || !tile_end) return KVARN_ERR_INVALID;
  PageParams p = page_params(cfg, block_table, max_blocks, batch, refs, dev_err);
  p.tile_begin = tile_begin;
  p.tile_end = tile_end;
  return cuda_status(launch_free(p, static_cast<cudaStream_t>(stream)));
}

static kvarn_status check_fork(const kvarn_config* cfg, const int32_t* parent, int32_t group, int32_t batch,
                               const int32_t* seq_lens, int32_t max_blocks) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || max_blocks < 1 || max_blocks > kMaxTableBlocks || group < 1) return KVARN_ERR_INVALID;
  if (batch == 0) return KVARN_OK;
  if (!parent || !seq_lens) return KVARN_ERR_INVALID;
  if (group > KVARN_FORK_MAX_GROUP || (batch + group - 1LL) / group > 65535) return KVARN_ERR_UNSUPPORTED;
  return KVARN_OK;
}

kvarn_status kvarn_fork_tails(const kvarn_config* cfg, const int32_t* parent, int32_t group, int32_t batch,
                              const int32_t* seq_lens, int32_t max_blocks, void* tail_pool, int32_t* dev_err,
                              void* stream) {
  kvarn_status st = check_fork(cfg, parent, group, batch, seq_lens, max_blocks);
  if (st != KVARN_OK || batch == 0) return st;
  if (!tail_pool || !aligned16(tail_pool)) return KVARN_ERR_INVALID;
  if (cfg->num_kv_heads > 32767) return KVARN_ERR_UNSUPPORTED;
  ForkParams p{parent, const_cast<int32_t*>(seq_lens), nullptr, nullptr, tail_pool, dev_err, group, batch, max_blocks,
               cfg->num_blocks, cfg->num_kv_heads};
  return cuda_status(launch_fork_tails(p, static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_fork_sequences(const kvarn_config* cfg, const int32_t* parent, int32_t group, int32_t batch,
                                  int32_t* block_table, int32_t max_blocks, int32_t* seq_lens, int32_t* refs,
                                  int32_t* dev_err, void* stream) {
  kvarn_status st = check_fork(cfg, parent, group, batch, seq_lens, max_blocks);
  if (st != KVARN_OK) return st;
  st = check_pages(cfg, block_table, max_blocks, batch, refs);
  if (st != KVARN_OK || batch == 0) return st;
  ForkParams p{parent, seq_lens, block_table, refs, nullptr, dev_err, group, batch, max_blocks, cfg->num_blocks,
               cfg->num_kv_heads};
  return cuda_status(launch_fork_sequences(p, static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_compact_blocks(const kvarn_config* cfg, int32_t* block_table, int32_t max_blocks, int32_t batch,
                                  int32_t* refs, int32_t* move_src, int32_t* move_dst, int32_t* counts,
                                  void* workspace, size_t workspace_bytes, int32_t* dev_err, void* stream) {
  kvarn_status st = check_pages(cfg, block_table, max_blocks, batch, refs);
  if (st != KVARN_OK) return st;
  if ((!refs && cfg->num_blocks > 0) || !aligned16(refs) || (cfg->num_blocks > 0 && (!move_src || !move_dst)) ||
      !counts || !workspace || !aligned16(workspace) || workspace_bytes < pages_ws_bytes(cfg->num_blocks))
    return KVARN_ERR_INVALID;
  PageParams p = page_params(cfg, block_table, max_blocks, batch, refs, dev_err);
  p.move_src = move_src;
  p.move_dst = move_dst;
  p.counts = counts;
  p.ws = static_cast<int32_t*>(workspace);
  return cuda_status(launch_compact(p, static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_copy_blocks(const kvarn_config* cfg, const void* src_pool, int32_t src_blocks,
                               const int32_t* src_ids, void* dst_pool, const int32_t* dst_ids, int32_t n,
                               const int32_t* n_dev, int32_t* dev_err, void* stream) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (n < 0 || src_blocks < 0) return KVARN_ERR_INVALID;
  if (n == 0) return KVARN_OK;
  if ((!src_pool && src_blocks > 0) || (!dst_pool && cfg->num_blocks > 0) || !src_ids || !dst_ids ||
      !aligned16(src_pool) || !aligned16(dst_pool))
    return KVARN_ERR_INVALID;
  CopyParams p{static_cast<const unsigned char*>(src_pool), static_cast<unsigned char*>(dst_pool), src_ids, dst_ids,
               n_dev, n, src_blocks, cfg->num_blocks, cfg->num_kv_heads, head_rec(cfg->k_bits, cfg->v_bits), dev_err};
  return cuda_status(launch_copy_blocks(p, static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_decode_attention_noalloc(const kvarn_config* cfg, const void* q, const int32_t* block_table,
                                            int32_t max_blocks, const int32_t* seq_lens, int32_t batch,
                                            const void* block_pool, const void* tail_pool, float softmax_scale,
                                            float* out, int32_t* dev_err, void* stream) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (batch < 0 || max_blocks < 1 || batch > 65535) return KVARN_ERR_INVALID;
  if (batch == 0) return KVARN_OK;
  if (!q || !block_table || !seq_lens || (!block_pool && cfg->num_blocks > 0) || !tail_pool || !out) return KVARN_ERR_INVALID;
  if (!aligned16(q) || !aligned16(block_pool) || !aligned16(tail_pool) || !aligned16(out)) return KVARN_ERR_INVALID;
  const int G = cfg->num_q_heads / cfg->num_kv_heads;
  if (decode_ws_bytes(batch, cfg->num_kv_heads, G, max_blocks, kChunkTiles) > KVARN_NOALLOC_SCRATCH_BYTES)
    return KVARN_ERR_UNSUPPORTED;  // larger than the fixed scratch: use kvarn_decode_attention
  int chunk = choose_chunk_tiles(cfg, batch, cfg->num_kv_heads, max_blocks);
  if (decode_ws_bytes(batch, cfg->num_kv_heads, G, max_blocks, chunk) > KVARN_NOALLOC_SCRATCH_BYTES)
    chunk = kChunkTiles;  // a small call's finer split does not fit: the ordinary split does
  const int n_chunks = (max_blocks + chunk - 1) / chunk;
  DecodeParams p{q, block_table, seq_lens, static_cast<const unsigned char*>(block_pool), tail_pool, nullptr, dev_err,
                 static_cast<int64_t>(kvarn_block_bytes(cfg)), softmax_scale, max_blocks, cfg->num_kv_heads,
                 cfg->num_q_heads, G, cfg->num_blocks, chunk, n_chunks, cfg->k_bits, cfg->v_bits};
  return cuda_status(launch_decode_noalloc(p, cfg->dtype, batch, out, static_cast<cudaStream_t>(stream)));
}

kvarn_status kvarn_fp16_decode_attention(const kvarn_config* cfg, const void* q, const int32_t* block_table,
                                         int32_t max_blocks, const int32_t* seq_lens, int32_t batch,
                                         const void* fp16_pool, float softmax_scale, float* out, void* workspace,
                                         size_t workspace_bytes, int32_t* dev_err, void* stream) {
  kvarn_status st = check_decode(cfg, q, block_table, max_blocks, seq_lens, batch, fp16_pool, out, workspace,
                                 workspace_bytes);
  if (st != KVARN_OK || batch == 0) return st;
  if (cfg->num_blocks < 1) return KVARN_ERR_INVALID;
  const int n_chunks = (max_blocks + kF16ChunkTiles - 1) / kF16ChunkTiles;
  DecodeParams p{q, block_table, seq_lens, nullptr, nullptr, static_cast<float*>(workspace), dev_err, 0,
                 softmax_scale, max_blocks, cfg->num_kv_heads, cfg->num_q_heads,
                 cfg->num_q_heads / cfg->num_kv_heads, cfg->num_blocks, kF16ChunkTiles, n_chunks, 16, 16, 0, 0,
                 static_cast<int64_t>(workspace_bytes)};
  cudaError_t e = launch_decode_f16(p, fp16_pool, cfg->dtype, batch, out, static_cast<cudaStream_t>(stream));
  if (e == cudaErrorInvalidValue) return KVARN_ERR_INVALID;
  if (e == cudaErrorNotSupported) return KVARN_ERR_UNSUPPORTED;
  return cuda_status(e);
}

kvarn_status kvarn_dequantize(const kvarn_config* cfg, const void* block_pool, const int32_t* blocks, int32_t n,
                              float* out, int32_t* dev_err, void* stream) {
  kvarn_status st = check_config(cfg);
  if (st != KVARN_OK) return st;
  if (n < 0) return KVARN_ERR_INVALID;
  if (n == 0) return KVARN_OK;
  if ((!block_pool && cfg->num_blocks > 0) || !blocks || !out || !aligned16(block_pool) || !aligned16(out))
    return KVARN_ERR_INVALID;
  if (cfg->num_kv_heads > 65535) return KVARN_ERR_INVALID;
  return cuda_status(launch_dequantize(static_cast<const unsigned char*>(block_pool),
                                       static_cast<int64_t>(kvarn_block_bytes(cfg)), blocks, n, cfg->num_blocks,
                                       cfg->num_kv_heads, cfg->k_bits, cfg->v_bits, out, dev_err,
                                       static_cast<cudaStream_t>(stream)));
}

const char* kvarn_status_string(kvarn_status s) {
  switch (s) {
    case KVARN_OK: return "ok";
    case KVARN_ERR_INVALID: return "invalid argument";
    case KVARN_ERR_UNSUPPORTED: return "unsupported configuration";
    case KVARN_ERR_CUDA: return "CUDA launch or runtime error";
  }
  return "unknown status";
}

}  // extern "C"
