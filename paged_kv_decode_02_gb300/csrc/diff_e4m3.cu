// diff_e4m3.cu -- differential decode over E4M3 caches.
#include "decode_diff.cuh"

namespace pkv {

bool select_diff_e4m3(int D, int BS, int pairs, DiffKernelInfo* info) {
  return select_diff_q8<CODE_E4M3>(D, BS, pairs, info);
}

}  // namespace pkv
