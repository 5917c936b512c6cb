// diff_bf16.cu -- differential decode over bf16 caches.
#include "decode_diff.cuh"

namespace pkv {

bool select_diff_bf16(int D, int BS, int pairs, DiffKernelInfo* info) {
  // items of 16 KiB (K and V): 16 tokens at head_dim 128 (half a 32-token block), 32 at 64
  if (D == 128) *info = diff_shape<128, DiffPathBf16<128, 16, 1>, 1, 2>(pairs);
  else if (D == 64 && BS == 16) *info = diff_shape<64, DiffPathBf16<64, 16, 2>, 1, 2>(pairs);
  else if (D == 64 && BS == 32) *info = diff_shape<64, DiffPathBf16<64, 32, 1>, 1, 2>(pairs);
  else return false;
  return true;
}

}  // namespace pkv
