// tree_k4v4.cu — attention of drafted token trees over k4v4 pools (tree_attn.cuh).
#include "tree_attn.cuh"

namespace pkv {

cudaError_t launch_tree_k4v4(const tree::Params& P, int mode) { return tree::launch_mode<4, 4>(P, mode); }

}  // namespace pkv
