// diff_e5m2.cu -- differential decode over E5M2 caches.
#include "decode_diff.cuh"

namespace pkv {

bool select_diff_e5m2(int D, int BS, int pairs, DiffKernelInfo* info) {
  return select_diff_q8<CODE_E5M2>(D, BS, pairs, info);
}

}  // namespace pkv
