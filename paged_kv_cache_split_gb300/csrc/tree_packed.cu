// tree_packed.cu — attention of drafted token trees over packed pools (tree_attn.cuh).
#include "tree_attn.cuh"

namespace pkv {

cudaError_t launch_tree_packed(const tree::Params& P, int mode) { return tree::launch_mode<true>(P, mode); }

}  // namespace pkv
