// tree_bf16.cu -- bf16-cache instantiations of the tree attention (tree.cuh) and the kernel table
// over every KV dtype.
#include "tree.cuh"

namespace pkv {

bool select_tree(int D, int BS, int kvt, TreeKernelInfo* info) {
  switch (kvt) {
    case PKV_KV_BF16: return select_tree_code<-1>(D, BS, info);
    case PKV_KV_INT8: return select_tree_int8(D, BS, info);
    case PKV_KV_FP8_E4M3: return select_tree_e4m3(D, BS, info);
    case PKV_KV_FP8_E5M2: return select_tree_e5m2(D, BS, info);
    default: return false;
  }
}

}  // namespace pkv
