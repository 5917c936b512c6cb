// decode_tree_int8.cu -- INT8-cache instantiations of the tcgen05 decode kernel (decode_tc.cuh) for a
// tree of new tokens.
#include "decode_tc.cuh"

namespace pkv {

bool select_decode_tree_int8(int D, int BS, bool split, DecodeKernelInfo* info) {
  return select_tc_code<CODE_I8, true>(D, BS, false, split, info);
}

}  // namespace pkv
