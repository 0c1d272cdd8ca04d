// tree.cu -- attention of a drafted token tree over the packed paged cache
// (rows_kernel.cuh, MQ_TREE): every node sees the whole cached context
// and the nodes its mask row names; the nodes' own keys and values are 16-bit
// arrays beside the cache, because a tile that has closed cannot give a
// rejected token back.
//
// The packed tiles need no mask: nodes x group rows in 128-row blocks on the
// 5th-generation tensor cores (rows_kernel).  The open tile and the nodes are
// one raw part on the warp tensor cores in front (raw_rows_kernel).
// fp16, 8 query heads per KV head, 8 KV heads: 32 sequences x 64 nodes behind
// 16 K tokens 1.84 ms (0.52 PFLOP/s of useful products; 1.89 measured for a
// library product), 8 ragged sequences x 27 nodes 56 us; bf16, one sequence x 8
// nodes 16 us, three launches' latency.
#include "rows_kernel.cuh"

namespace kvarn {

cudaError_t launch_tree(const RowsParams& p, int dtype, int batch, void* out, bool out16, cudaStream_t s) {
  if (dtype == KVARN_DTYPE_BF16)
    return out16 ? launch_rows<MQ_TREE, __nv_bfloat16>(p, batch, static_cast<__nv_bfloat16*>(out), s)
                 : launch_rows<MQ_TREE, __nv_bfloat16>(p, batch, static_cast<float*>(out), s);
  return out16 ? launch_rows<MQ_TREE, __half>(p, batch, static_cast<__half*>(out), s)
               : launch_rows<MQ_TREE, __half>(p, batch, static_cast<float*>(out), s);
}

}  // namespace kvarn
