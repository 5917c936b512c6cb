// tree_int8.cu -- INT8-cache instantiations of the tree attention (tree.cuh), in a unit of their
// own so that the kernels compile in parallel.
#include "tree.cuh"

namespace pkv {

bool select_tree_int8(int D, int BS, TreeKernelInfo* info) {
  return select_tree_code<CODE_I8>(D, BS, info);
}

}  // namespace pkv
