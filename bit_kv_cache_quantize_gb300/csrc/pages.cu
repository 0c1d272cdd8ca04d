// pages.cu -- the pages of the cache as state on the device: blocks handed
// out, released, shared by forked sequences, moved together and copied.  All
// of it is driven by device arrays (block table, reference counts, parents),
// so a serving step with branches captures into a graph and never waits for
// the host.
//
// The calls come in chains (fork the tails, then the rows, then allocate), so
// every kernel here is launched as a programmatic dependent: it is set up while
// the one before still runs and waits for it before it touches anything.
//
// A closed tile never changes, so two sequences that share a context share
// its blocks (refs[block] = table entries that name it; 0 = free); only the
// raw open tile is copied at a fork.
#include <algorithm>

#include "common.cuh"

namespace kvarn {
namespace {

constexpr int PG_THREADS = 1024;

// Exclusive prefix sum of one int per thread over the block (a multiple of
// 32 threads); `total` gets the block's sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int v = x;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, m);
    if (lane >= m) v += o;
  }
  __syncthreads();  // the previous use of warp_sums is over
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < nw; ++w) {
    const int s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  total = all;
  return before + v - x;
}

// Tile range of sequence s clipped to the table; an impossible one is empty.
__device__ __forceinline__ bool tile_range(const PageParams& p, int s, int& t0, int& t1) {
  t0 = p.tile_begin[s];
  t1 = p.tile_end[s];
  if (t0 < 0 || t1 > p.max_blocks) return false;
  t1 = max(t0, t1);
  return true;
}

// One CTA: list the open entries of all ranges in (sequence, tile) order,
// then hand them the free ids as a scan over refs finds them.  Latency is
// what bounds a step's call (a tile per sequence, ids in the first slab), so
// the entries are spread over the threads by a prefix sum of the ranges (a
// warp per sequence took eight dependent rounds at 256 sequences: 15 us
// against the 7 of this form), the first slab of counts is loaded before
// anything else, and a thread that finds a free id writes the entry itself.
constexpr int AL_IDS = 8;  // ids per thread and slab
__device__ __forceinline__ uint32_t free_bits(const PageParams& p, int64_t b) {  // of ids b .. b + 7
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < AL_IDS; i += 4) {
    if (b + i + 4 <= p.num_blocks) {
      const int4 v = *reinterpret_cast<const int4*>(p.refs + b + i);
      m |= (uint32_t)(v.x == 0) << i | (uint32_t)(v.y == 0) << (i + 1) | (uint32_t)(v.z == 0) << (i + 2) |
           (uint32_t)(v.w == 0) << (i + 3);
    } else {
      for (int k = i; k < i + 4; ++k) m |= (uint32_t)(b + k < p.num_blocks && p.refs[b + k] == 0) << k;
    }
  }
  return m;
}

__global__ void __launch_bounds__(PG_THREADS) alloc_kernel(PageParams p) {
  allow_dependents();
  wait_prerequisite();
  __shared__ int sums[PG_THREADS / 32];
  __shared__ int first[PG_THREADS];  // entries before each sequence of the slab
  __shared__ int begin[PG_THREADS];
  const int tid = threadIdx.x;
  constexpr int64_t SLAB = PG_THREADS * AL_IDS;
  uint32_t next = free_bits(p, (int64_t)tid * AL_IDS);
  int32_t* open = p.ws;  // [need] the open entries, as offsets into the table
  int need = 0;
  // (counters up to 2^31 - 1 in steps of the block: unsigned, the last step passes it)
  for (uint32_t s0 = 0; s0 < (uint32_t)p.batch; s0 += PG_THREADS) {
    const uint32_t s = s0 + tid;
    int t0 = 0, t1 = 0;
    if (s < (uint32_t)p.batch && !tile_range(p, (int)s, t0, t1)) {
      set_error(p.err, KVARN_DEV_ERR_TOKEN_RANGE);
      t0 = t1 = 0;
    }
    int total;
    const int before = block_scan(t1 - t0, sums, total);
    first[tid] = before;
    begin[tid] = t0;
    __syncthreads();
    for (uint32_t e0 = 0; e0 < (uint32_t)total; e0 += PG_THREADS) {
      const uint32_t e = e0 + tid;
      int at = -1;
      if (e < (uint32_t)total) {
        int lo = 0;  // the last sequence that starts at or before e (an empty range shares its start with the next)
#pragma unroll
        for (int step = PG_THREADS / 2; step > 0; step >>= 1)
          if (first[lo + step] <= (int)e) lo += step;
        const int off = (int)(s0 + lo) * p.max_blocks + begin[lo] + (int)e - first[lo];
        if (p.table[off] < 0) at = off;
      }
      int all;
      const int rank = need + block_scan(at >= 0, sums, all);
      if (at >= 0 && rank < p.num_blocks) open[rank] = at;  // no more than the pool could serve
      need += all;
    }
    __syncthreads();  // first and begin are rewritten
  }
  __syncthreads();  // the list is complete
  int found = 0;
  for (int64_t b0 = 0; b0 < p.num_blocks && found < need; b0 += SLAB) {
    uint32_t m = next;
    if (b0 + SLAB < p.num_blocks) next = free_bits(p, b0 + SLAB + (int64_t)tid * AL_IDS);
    int all, rank = found + block_scan(__popc(m), sums, all);
    for (; m && rank < need; m &= m - 1, ++rank) {
      const int32_t id = (int32_t)(b0 + (int64_t)tid * AL_IDS + __ffs(m) - 1);
      p.table[open[rank]] = id;
      p.refs[id] = 1;
    }
    found += all;
  }
  if (found < need && tid == 0) set_error(p.err, KVARN_DEV_ERR_POOL_FULL);
}

// One reference less for each of N blocks (-1: none); a count that is not
// positive is an error and stays.  All the decrements are in flight before
// the first answer is looked at.
template <int N>
__device__ __forceinline__ void drop_refs(int32_t* refs, int num_blocks, int32_t* err, const int32_t (&id)[N]) {
  int32_t was[N];
#pragma unroll
  for (int k = 0; k < N; ++k) was[k] = id[k] >= 0 && id[k] < num_blocks ? atomicSub(refs + id[k], 1) : 1;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (id[k] >= num_blocks) set_error(err, KVARN_DEV_ERR_BLOCK_RANGE);
    if (was[k] <= 0) {
      atomicAdd(refs + id[k], 1);
      set_error(err, KVARN_DEV_ERR_REF_COUNT);
    }
  }
}

// A thread per table entry.
__global__ void __launch_bounds__(128) free_kernel(PageParams p) {
  allow_dependents();
  wait_prerequisite();
  const int64_t segs = (p.max_blocks + 127) / 128;
  const int s = (int)(blockIdx.x / segs), t = (int)(blockIdx.x % segs) * 128 + threadIdx.x;
  int t0, t1;
  if (!tile_range(p, s, t0, t1)) {
    if (t == 0) set_error(p.err, KVARN_DEV_ERR_TOKEN_RANGE);
    return;
  }
  if (t < t0 || t >= t1) return;
  int32_t* e = p.table + (int64_t)s * p.max_blocks + t;
  const int32_t id[1] = {*e};
  if (id[0] < 0) return;
  *e = -1;
  drop_refs(p.refs, p.num_blocks, p.err, id);
}

// The parent of slot s and the length it brings, or s itself where either is
// impossible (the error is stored and the slot stays as it is).
__device__ __forceinline__ int fork_parent(const ForkParams& p, int s, int g0, int group, bool report, int& len) {
  const int parent = p.parent[s];
  len = 0;
  if (parent == -1) return -1;
  if (parent < g0 || parent >= g0 + group) {
    if (report) set_error(p.err, KVARN_DEV_ERR_SLOT_RANGE);
    return s;
  }
  len = p.seq_lens[parent];
  if (len < 0 || len > T * p.max_blocks) {
    if (report) set_error(p.err, KVARN_DEV_ERR_TOKEN_RANGE);
    return s;
  }
  return parent;
}

// Open tiles of a group of slots, in place: slot s takes the live tokens of
// its parent's open tile.  A CTA owns some 16-byte columns of the tile for
// ALL slots of the group, so it can load every value it will store, meet at
// a barrier, and store: any map of parents (a parent overwritten itself, a
// cycle, one parent for all) needs no second copy of the tiles.
// 2048 values per CTA (8 per thread in flight).  Bound by latency: launch,
// parents, one round trip of loads.
constexpr int FT_THREADS = 256, FT_PIECES = 8;
constexpr int FT_GROUP = KVARN_FORK_MAX_GROUP;  // two columns per CTA
static_assert(FT_THREADS * FT_PIECES >= FT_GROUP && PG_THREADS * 8 >= FT_GROUP, "a column of a group fits a CTA");
__global__ void __launch_bounds__(FT_THREADS) fork_tails_kernel(ForkParams p) {
  allow_dependents();
  wait_prerequisite();
  __shared__ int16_t parent[FT_GROUP];  // offset in the group, -1: nothing to copy
  __shared__ uint8_t live[FT_GROUP];    // tokens the parent's open tile holds
  __shared__ int most;
  const int tid = threadIdx.x, g0 = blockIdx.z * p.group, group = min(p.group, p.batch - g0);
  const int cols = FT_THREADS * FT_PIECES / p.group, c0 = blockIdx.x * cols;
  if (tid == 0) most = 0;
  __syncthreads();
  for (int i = tid; i < group; i += FT_THREADS) {
    int len;
    const int s = g0 + i, par = fork_parent(p, s, g0, group, blockIdx.x == 0 && blockIdx.y == 0, len);
    const bool moves = par >= 0 && par != s;
    parent[i] = moves ? par - g0 : -1;
    live[i] = moves ? len % T : 0;
    if (moves) atomicMax(&most, len % T);
  }
  __syncthreads();
  if ((c0 >> 4) >= most) return;  // uniform: no slot has a token in these columns
  uint4* tail = static_cast<uint4*>(p.tail);
  const int64_t unit = (int64_t)T * D * 2 / 16;                     // 16-byte values of one tile
  const int64_t stride = unit * 2 * p.num_kv_heads;                 // of one slot
  uint4* base = tail + g0 * stride + blockIdx.y * unit;
  uint4 v[FT_PIECES];
  int64_t dst[FT_PIECES];
#pragma unroll
  for (int k = 0; k < FT_PIECES; ++k) {
    const int e = tid + k * FT_THREADS, slot = e / cols, col = c0 + e % cols;
    dst[k] = -1;
    if (slot < group && col < unit && parent[slot] >= 0 && (col >> 4) < live[slot]) {
      dst[k] = slot * stride + col;
      v[k] = base[parent[slot] * stride + col];
    }
  }
  __syncthreads();  // every value of these columns is in registers
#pragma unroll
  for (int k = 0; k < FT_PIECES; ++k)
    if (dst[k] >= 0 && kcheck(base + dst[k], 16, tail, (size_t)p.batch * stride * 16, p.err)) base[dst[k]] = v[k];
}

// Rows of the block table, reference counts and lengths of a group of slots,
// in place, one CTA per group: the same load, barrier, store over the table's
// columns.  Entries past the closed tiles are not inherited: the block a tile
// will close into belongs to one sequence.
constexpr int FS_PIECES = 8;
__global__ void __launch_bounds__(PG_THREADS) fork_sequences_kernel(ForkParams p) {
  allow_dependents();
  wait_prerequisite();
  __shared__ int32_t parent[FT_GROUP], len[FT_GROUP];
  const int tid = threadIdx.x, g0 = blockIdx.x * p.group, group = min(p.group, p.batch - g0);
  for (int i = tid; i < group; i += PG_THREADS) parent[i] = fork_parent(p, g0 + i, g0, group, true, len[i]);
  __syncthreads();
  const int cols = PG_THREADS * FS_PIECES / group;
  int32_t* rows = p.table + (int64_t)g0 * p.max_blocks;
  for (int c0 = 0; c0 < p.max_blocks; c0 += cols) {
    int32_t was[FS_PIECES], now[FS_PIECES];
#pragma unroll
    for (int k = 0; k < FS_PIECES; ++k) {
      const int e = tid + k * PG_THREADS, slot = e / cols, t = c0 + e % cols;
      was[k] = now[k] = -1;
      if (slot < group && t < p.max_blocks && parent[slot] != g0 + slot) {
        was[k] = rows[(int64_t)slot * p.max_blocks + t];
        if (parent[slot] >= 0 && t < len[slot] / T) now[k] = p.table[(int64_t)parent[slot] * p.max_blocks + t];
      }
    }
    __syncthreads();  // these columns are in registers
#pragma unroll
    for (int k = 0; k < FS_PIECES; ++k) {
      const int e = tid + k * PG_THREADS, slot = e / cols, t = c0 + e % cols;
      if (now[k] == was[k]) {
        was[k] = -1;
        continue;
      }
      rows[(int64_t)slot * p.max_blocks + t] = now[k];
      if (now[k] >= p.num_blocks) set_error(p.err, KVARN_DEV_ERR_BLOCK_RANGE);
      else if (now[k] >= 0) atomicAdd(p.refs + now[k], 1);
    }
    drop_refs(p.refs, p.num_blocks, p.err, was);
  }
  __syncthreads();
  for (int i = tid; i < group; i += PG_THREADS)
    if (parent[i] != g0 + i) p.seq_lens[g0 + i] = len[i];
}

// ---- compaction.  With L live blocks, those with ids >= L (movers) take the
// free ids below L (holes); there are as many of one as of the other.  Both
// ranks come from live_before(id), the live blocks with smaller ids: a hole's
// is id - live_before(id), and counting movers from the top, a mover's is
// L - 1 - live_before(id).  So one prefix sum pairs them, without a sort and
// without a second pass: three short launches whatever the pool's size.
constexpr int CP_THREADS = 256, CP_IDS = 16, CP_CHUNK = CP_THREADS * CP_IDS;

__device__ __forceinline__ uint32_t live_bits(const PageParams& p, int64_t b) {  // of ids b .. b + 15
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CP_IDS; i += 4) {
    if (b + i + 4 <= p.num_blocks) {
      const int4 v = *reinterpret_cast<const int4*>(p.refs + b + i);
      m |= (uint32_t)(v.x > 0) << i | (uint32_t)(v.y > 0) << (i + 1) | (uint32_t)(v.z > 0) << (i + 2) |
           (uint32_t)(v.w > 0) << (i + 3);
    } else {
      for (int k = i; k < i + 4; ++k) m |= (uint32_t)(b + k < p.num_blocks && p.refs[b + k] > 0) << k;
    }
  }
  return m;
}

__global__ void __launch_bounds__(CP_THREADS) compact_count_kernel(PageParams p) {
  wait_prerequisite();
  allow_dependents();  // only now: the plan reads refs before it waits for the counts
  __shared__ int sums[CP_THREADS / 32];
  int all;
  block_scan(__popc(live_bits(p, (int64_t)blockIdx.x * CP_CHUNK + threadIdx.x * CP_IDS)), sums, all);
  if (threadIdx.x == 0) p.ws[blockIdx.x] = all;
}

__global__ void __launch_bounds__(CP_THREADS) compact_plan_kernel(PageParams p, int n_chunks) {
  allow_dependents();
  __shared__ int sums[CP_THREADS / 32];
  const int tid = threadIdx.x;
  const int64_t b0 = (int64_t)blockIdx.x * CP_CHUNK + tid * CP_IDS;
  const uint32_t m = live_bits(p, b0);  // the counting kernel only reads refs: no need to wait for it
  wait_prerequisite();                  // the chunks' counts
  int before = 0, total = 0;
  for (int c = tid; c < n_chunks; c += CP_THREADS) {
    const int n = p.ws[c];
    total += n;
    if (c < (int)blockIdx.x) before += n;
  }
  int L, base;
  block_scan(total, sums, L);
  block_scan(before, sums, base);
  int all, at = base + block_scan(__popc(m), sums, all);
  int32_t* rank = p.ws + n_chunks;  // of each id: its move (id >= L) or 0, or -1 where no count holds it
#pragma unroll
  for (int i = 0; i < CP_IDS; ++i) {
    const int64_t id = b0 + i;
    if (id >= p.num_blocks) break;
    const bool used = (m >> i) & 1u;
    rank[id] = !used ? -1 : id >= L ? L - 1 - at : 0;
    if (id >= L) {
      if (used) p.move_src[L - 1 - at] = (int32_t)id;
    } else if (!used) {
      p.move_dst[id - at] = (int32_t)id;
    }
    at += used;
    if (id == L - 1) p.counts[1] = L - at;  // holes below L = moves
  }
  if (blockIdx.x == 0 && tid == 0) {
    p.counts[0] = L;
    if (L == 0) p.counts[1] = 0;
  }
}

__global__ void __launch_bounds__(CP_THREADS) compact_apply_kernel(PageParams p, int n_chunks) {
  allow_dependents();
  wait_prerequisite();  // the plan
  const int L = p.counts[0], moves = p.counts[1];
  const int32_t* rank = p.ws + n_chunks;
  const int64_t step = (int64_t)gridDim.x * CP_THREADS, i0 = (int64_t)blockIdx.x * CP_THREADS + threadIdx.x;
  for (int64_t i = i0; i < moves; i += step) {
    const int32_t a = p.move_src[i], b = p.move_dst[i];
    p.refs[b] = p.refs[a];
    p.refs[a] = 0;
  }
  for (int64_t i = i0; i < (int64_t)p.batch * p.max_blocks; i += step) {
    const int32_t id = p.table[i];
    if (id < 0) continue;
    if (id >= p.num_blocks) {
      set_error(p.err, KVARN_DEV_ERR_BLOCK_RANGE);
    } else if (rank[id] < 0) {
      set_error(p.err, KVARN_DEV_ERR_REF_COUNT);  // the table names a block that no count holds
    } else if (id >= L) {
      p.table[i] = p.move_dst[rank[id]];
    }
  }
}

// Records from one pool to another (or within one), one (block, KV head) at a
// time through a ring of shared-memory stages: bulk copies in, bulk copies
// out, one thread per CTA.  Bound by memory alone.
constexpr int CB_STAGES = 6, CB_CTAS = 2;
struct CopySmem {
  alignas(128) unsigned char buf[CB_STAGES][HEAD_REC_MAX];
  uint64_t bar[CB_STAGES];
};
__device__ __forceinline__ void bulk_s2g(void* gmem, const void* smem, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(gmem), "r"(smem_u32(smem)),
               "r"(bytes)
               : "memory");
}
__global__ void __launch_bounds__(32) copy_blocks_kernel(CopyParams p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  allow_dependents();
  if (threadIdx.x != 0) return;
  const uint32_t sbase = smem_u32(smem_raw);
  CopySmem& sm = *reinterpret_cast<CopySmem*>(smem_raw + (((sbase + 127u) & ~127u) - sbase));
  for (int s = 0; s < CB_STAGES; ++s) mbar_init(&sm.bar[s], 1);
  fence_mbar_init();
  wait_prerequisite();
  int n = p.n;
  if (p.n_dev) n = min(n, max(0, *p.n_dev));
  const int64_t items = (int64_t)n * p.num_kv_heads;
  const uint32_t bytes = p.head_bytes;
  const int64_t mine = items > blockIdx.x ? (items - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  // item k of this CTA: start its copy in; false where an id is out of range
  auto start = [&](int64_t k) -> bool {
    const int64_t item = blockIdx.x + k * gridDim.x;
    const int i = (int)(item / p.num_kv_heads), h = (int)(item % p.num_kv_heads);
    const int32_t a = p.src_ids[i], b = p.dst_ids[i];
    const int s = (int)(k % CB_STAGES);
    if (a < 0 || a >= p.src_blocks || b < 0 || b >= p.dst_blocks) {
      set_error(p.err, KVARN_DEV_ERR_BLOCK_RANGE);
      mbar_arrive(&sm.bar[s]);
      return false;
    }
    mbar_expect_tx(&sm.bar[s], bytes);
    bulk_g2s_stream(sm.buf[s], p.src + (a * (int64_t)p.num_kv_heads + h) * bytes, bytes, &sm.bar[s]);
    return true;
  };
  uint32_t ok = 0;  // stages whose item copies
  const int64_t ahead = CB_STAGES / 2;  // copies in flight inwards; the other stages drain outwards
  for (int64_t k = 0; k < min(mine, ahead); ++k) ok |= start(k) ? 1u << (k % CB_STAGES) : 0u;
  bool here = true;
  for (int64_t k = 0; k < mine; ++k) {
    const int s = (int)(k % CB_STAGES);
    here = mbar_wait_parked(&sm.bar[s], (k / CB_STAGES) & 1, p.err);
    if (!here) {  // error word set; the copies still in flight land (bounded) before the memory goes
      for (int64_t i = k; i < min(mine, k + ahead); ++i)
        mbar_wait_parked(&sm.bar[i % CB_STAGES], (i / CB_STAGES) & 1, p.err);
      break;
    }
    if ((ok >> s) & 1u) {
      const int64_t item = blockIdx.x + k * gridDim.x;
      unsigned char* dst = p.dst + (p.dst_ids[item / p.num_kv_heads] * (int64_t)p.num_kv_heads + item % p.num_kv_heads) *
                                       bytes;
      if (kcheck(dst, bytes, p.dst, (size_t)p.dst_blocks * p.num_kv_heads * bytes, p.err)) bulk_s2g(dst, sm.buf[s], bytes);
    }
    asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");  // one group per item, an empty one for a bad id
    if (k + ahead < mine) {
      // item k + ahead takes the stage of item k + ahead - CB_STAGES; only the
      // CB_STAGES - ahead newer copies out may still be reading theirs
      asm volatile("cp.async.bulk.wait_group.read %0;\n" ::"n"(CB_STAGES / 2) : "memory");
      const int s2 = (int)((k + ahead) % CB_STAGES);
      ok = (ok & ~(1u << s2)) | (start(k + ahead) ? 1u << s2 : 0u);
    }
  }
  // the copies out have read their stages and are complete before the CTA ends
  asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
}

}  // namespace

cudaError_t launch_alloc(const PageParams& p, cudaStream_t s) {
  return launch_after(alloc_kernel, dim3(1), dim3(PG_THREADS), s, p);
}

cudaError_t launch_free(const PageParams& p, cudaStream_t s) {
  const int64_t segs = (p.max_blocks + 127) / 128;
  return launch_after(free_kernel, dim3((unsigned)(p.batch * segs)), dim3(128), s, p);
}

cudaError_t launch_fork_tails(const ForkParams& p, cudaStream_t s) {
  const int cols = FT_THREADS * FT_PIECES / p.group, unit = T * D * 2 / 16;
  const dim3 grid((unit + cols - 1) / cols, p.num_kv_heads * 2, (p.batch + p.group - 1) / p.group);
  return launch_after(fork_tails_kernel, grid, dim3(FT_THREADS), s, p);
}

cudaError_t launch_fork_sequences(const ForkParams& p, cudaStream_t s) {
  return launch_after(fork_sequences_kernel, dim3((p.batch + p.group - 1) / p.group), dim3(PG_THREADS), s, p);
}

size_t pages_ws_bytes(int64_t num_blocks) {
  // ranks, and the counts of the chunks: an empty pool has one too
  const int64_t chunks = std::max<int64_t>((num_blocks + CP_CHUNK - 1) / CP_CHUNK, 1);
  return (size_t)((num_blocks + chunks + 3) / 4 * 16);
}

cudaError_t launch_compact(const PageParams& p, cudaStream_t s) {
  const int chunks = (int)std::max<int64_t>(((int64_t)p.num_blocks + CP_CHUNK - 1) / CP_CHUNK, 1);
  cudaError_t e = launch_after(compact_count_kernel, dim3(chunks), dim3(CP_THREADS), s, p);
  if (e != cudaSuccess) return e;
  e = launch_after(compact_plan_kernel, dim3(chunks), dim3(CP_THREADS), s, p, chunks);
  if (e != cudaSuccess) return e;
  const int64_t work = std::max<int64_t>((int64_t)p.batch * p.max_blocks, p.num_blocks);
  const unsigned grid = (unsigned)std::min<int64_t>(std::max<int64_t>((work + CP_THREADS - 1) / CP_THREADS, 1), 152 * 8);
  return launch_after(compact_apply_kernel, dim3(grid), dim3(CP_THREADS), s, p, chunks);
}

cudaError_t launch_copy_blocks(const CopyParams& p, cudaStream_t s) {
  const size_t smem = sizeof(CopySmem) + 128;
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = smem_attr_once(attr_done, (const void*)copy_blocks_kernel, (int)smem);
  if (e != cudaSuccess) return e;
  const int64_t items = (int64_t)p.n * p.num_kv_heads;
  return launch_after_smem(copy_blocks_kernel, dim3((unsigned)std::min<int64_t>(items, 152 * CB_CTAS)), dim3(32), smem, s, p);
}

}  // namespace kvarn
