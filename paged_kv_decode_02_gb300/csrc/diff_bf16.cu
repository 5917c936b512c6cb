// diff_bf16.cu -- differential decode over bf16 caches.
#include "decode_diff.cuh"

namespace pkv {

namespace {
// Units of up to 4 query pairs: a warp per stream; up to 8: the warp takes both groups of 4
// (two warps per stream, reading the same tiles, on GB300: 64 x 2048 tokens, 64 / 8 heads
// of 128: 97.7 us against 95.2; one sequence of 131072: 96.0 against 91.5); up to 12: three
// warps of 4, whose registers leave room for 12 warps per SM (96 / 8 heads: 104 us, 115 with
// two of 8; over one-byte caches, where each warp widens all codes, it loses: INT8 117.6 us
// against 114.2); up to 16: two warps of 8 (128 / 8: 119 us; four of 4 137).
template <int D, int BOX, int SUB>
DiffKernelInfo diff_shape_bf16(int pairs) {
  if (pairs <= 4) return make_diff_info<D, DiffPathBf16<D, BOX, SUB, 1>, 4, 1, 1, 3>();
  if (pairs <= 8) return make_diff_info<D, DiffPathBf16<D, BOX, SUB, 2>, 4, 1, 1, 2>();
  if (pairs <= 12) return make_diff_info<D, DiffPathBf16<D, BOX, SUB, 1>, 2, 3, 2, 2>();
  return make_diff_info<D, DiffPathBf16<D, BOX, SUB, 2>, 2, 2, 2, 2>();
}
}  // namespace

bool select_diff_bf16(int D, int BS, int pairs, DiffKernelInfo* info) {
  // items of 16 KiB (K and V): 16 tokens at head_dim 128 (half a 32-token block), 32 at 64
  if (D == 128) *info = diff_shape_bf16<128, 16, 1>(pairs);
  else if (D == 64 && BS == 16) *info = diff_shape_bf16<64, 16, 2>(pairs);
  else if (D == 64 && BS == 32) *info = diff_shape_bf16<64, 32, 1>(pairs);
  else return false;
  return true;
}

}  // namespace pkv
