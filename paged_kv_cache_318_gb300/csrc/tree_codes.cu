// Attention of a tree of drafted tokens over caches of codes: E4M3, and E2M1
// with block scales (the kernel: tree_attn.cuh).
#include "tree_attn.cuh"

namespace pkv {
namespace tree {

cudaError_t launch_codes(const Params& p, int D, bool bf16, int kv,
                         const CUtensorMap& mk, const CUtensorMap& mv,
                         const CUtensorMap& mq, int grid,
                         const cudaLaunchAttribute* attr,
                         cudaStream_t stream) {
  if (kv == kE4m3)
    return bf16 ? launch_d<__nv_bfloat16, kE4m3>(p, D, mk, mv, mq, grid, attr,
                                                 stream)
                : launch_d<__half, kE4m3>(p, D, mk, mv, mq, grid, attr,
                                          stream);
  return bf16 ? launch_d<__nv_bfloat16, kE2m1>(p, D, mk, mv, mq, grid, attr,
                                               stream)
              : launch_d<__half, kE2m1>(p, D, mk, mv, mq, grid, attr, stream);
}

}  // namespace tree
}  // namespace pkv
