// tree_e4m3.cu -- FP8 E4M3-cache instantiations of the tree decode kernel (decode_tc.cuh), in a unit
// of their own so that the kernels compile in parallel.
#include "decode_tc.cuh"

namespace pkv {

bool select_tree_e4m3(int D, int BS, bool row_tiles, bool split, DecodeKernelInfo* info) {
  return select_tc_code<CODE_E4M3, true>(D, BS, row_tiles, split, info);
}

}  // namespace pkv
