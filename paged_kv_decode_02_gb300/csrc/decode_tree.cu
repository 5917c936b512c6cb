// decode_tree.cu -- bf16-cache instantiations of the tcgen05 decode kernel (decode_tc.cuh) for a
// tree of new tokens, and the kernel table over every KV dtype.
#include "decode_tc.cuh"

namespace pkv {

bool select_decode_tree(int D, int BS, bool split, int kvt, DecodeKernelInfo* info) {
  switch (kvt) {
    case PKV_KV_BF16: return select_tc_code<-1, true>(D, BS, false, split, info);
    case PKV_KV_INT8: return select_decode_tree_int8(D, BS, split, info);
    case PKV_KV_FP8_E4M3: return select_decode_tree_e4m3(D, BS, split, info);
    case PKV_KV_FP8_E5M2: return select_decode_tree_e5m2(D, BS, split, info);
    default: return false;
  }
}

}  // namespace pkv
