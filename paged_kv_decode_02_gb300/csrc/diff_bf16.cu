// diff_bf16.cu -- differential decode over bf16 caches.
#include "decode_diff.cuh"

namespace pkv {

bool select_diff_bf16(int D, int BS, DiffKernelInfo* info) {
  // items of 16 KiB (K and V): 16 tokens at head_dim 128 (half a 32-token block), 32 at 64
  if (D == 128) *info = make_diff_info<128, -1, 16, 1>();
  else if (D == 64 && BS == 16) *info = make_diff_info<64, -1, 16, 2>();
  else if (D == 64 && BS == 32) *info = make_diff_info<64, -1, 32, 1>();
  else return false;
  return true;
}

}  // namespace pkv
