// tree_k8v8.cu — attention of drafted token trees over k8v8 pools (tree_attn.cuh).
#include "tree_attn.cuh"

namespace pkv {

cudaError_t launch_tree_k8v8(const tree::Params& P, int mode) { return tree::launch_mode<8, 8>(P, mode); }

}  // namespace pkv
