// decode_tree_e4m3.cu -- E4M3-cache instantiations of the tcgen05 decode kernel (decode_tc.cuh) for a
// tree of new tokens.
#include "decode_tc.cuh"

namespace pkv {

bool select_decode_tree_e4m3(int D, int BS, bool split, DecodeKernelInfo* info) {
  return select_tc_code<CODE_E4M3, true>(D, BS, false, split, info);
}

}  // namespace pkv
