// tree_e4m3.cu -- FP8 E4M3-cache instantiations of the tree attention (tree.cuh), in a unit of their
// own so that the kernels compile in parallel.
#include "tree.cuh"

namespace pkv {

bool select_tree_e4m3(int D, int BS, TreeKernelInfo* info) {
  return select_tree_code<CODE_E4M3>(D, BS, info);
}

}  // namespace pkv
