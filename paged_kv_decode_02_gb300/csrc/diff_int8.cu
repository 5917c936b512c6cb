// diff_int8.cu -- differential decode over INT8 caches.
#include "decode_diff.cuh"

namespace pkv {

bool select_diff_int8(int D, int BS, int pairs, DiffKernelInfo* info) {
  return select_diff_q8<CODE_I8>(D, BS, pairs, info);
}

}  // namespace pkv
