// tree_bf16.cu — attention of drafted token trees over bf16 pools (tree_attn.cuh).
#include "tree_attn.cuh"

namespace pkv {

cudaError_t launch_tree_bf16(const tree::Params& P, int mode) { return tree::launch_mode<16, 16>(P, mode); }

}  // namespace pkv
