// decode_tree_e5m2.cu -- E5M2-cache instantiations of the tcgen05 decode kernel (decode_tc.cuh) for a
// tree of new tokens.
#include "decode_tc.cuh"

namespace pkv {

bool select_decode_tree_e5m2(int D, int BS, bool split, DecodeKernelInfo* info) {
  return select_tc_code<CODE_E5M2, true>(D, BS, false, split, info);
}

}  // namespace pkv
