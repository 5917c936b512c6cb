// tree_int8.cu -- INT8-cache instantiations of the tree decode kernel (decode_tc.cuh), in a unit
// of their own so that the kernels compile in parallel.
#include "decode_tc.cuh"

namespace pkv {

bool select_tree_int8(int D, int BS, bool row_tiles, bool split, DecodeKernelInfo* info) {
  return select_tc_code<CODE_I8, true>(D, BS, row_tiles, split, info);
}

}  // namespace pkv
