// tree_e5m2.cu -- FP8 E5M2-cache instantiations of the tree attention (tree.cuh), in a unit of their
// own so that the kernels compile in parallel.
#include "tree.cuh"

namespace pkv {

bool select_tree_e5m2(int D, int BS, TreeKernelInfo* info) {
  return select_tree_code<CODE_E5M2>(D, BS, info);
}

}  // namespace pkv
