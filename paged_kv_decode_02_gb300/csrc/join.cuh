// join.cuh -- records of an item that was cut between CTAs' stretches (prompt.cuh, tree.cuh),
// joined by the kernels that follow.
//
// A record is (o, m, l) of 256 rows: outputs that are not normalised yet, the maximum they refer
// to (log2 units), the sum of their weights. The item that CTA c's stretch begins and does not end
// has its first record in that CTA's cut, and its others are the first records of the CTAs after
// it, up to the one that ends it; they meet at the largest maximum:
//   M = max m_i;  L = sum l_i 2^(m_i - M);  O = sum o_i 2^(m_i - M);  out = O / L.
// The records are some MB that were just written, so the time is that of the loads' chain: all of
// a thread's rows are loaded at once, and a warp reads 32 CTAs' cuts to see which continue.
// Measured on GB300, whole calls, rows and cuts one after the other -> at once (us): a tree of 33
// nodes over 131071 tokens, E4M3 (19 parts) 207 -> 179; prompts of 1024 tokens, 32 / 32 heads,
// 37.9 -> 35.5, of 600, 8 / 8, 27.7 -> 21.4, 16 x 1024, 64 / 8, 349 -> 345. Two parts at once: 176
// for the tree, 1 to 4 % more for the others (registers). 16 rows a CTA: within 1 %, three short
// prompts 14.5 -> 16.0.
#pragma once

#include "common.cuh"
#include "decode.cuh"
#include "internal.h"

namespace pkv {

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;  // rows per CTA

// Rows row[0 .. R-1], columns 4 dq .. of each: O and L. By whole warps.
template <int D, int R, typename Cut>
__device__ __forceinline__ void join_parts(const Cut* cuts, const float* part_ml,
                                           const float* part_o, int c, int G, int slot,
                                           const int (&row)[R], int dq, float4 (&o)[R],
                                           float (&L)[R]) {
  float M[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    M[i] = -INFINITY;
    L[i] = 0.f;
    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto add = [&](int record) {
    float2 ml[R];
    float4 v[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const size_t rec = size_t(record) * 256 + row[i];
      ml[i] = reinterpret_cast<const float2*>(part_ml)[rec];
      v[i] = reinterpret_cast<const float4*>(part_o)[rec * (D / 4) + dq];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      // a part that saw nothing has no output; a NaN sum goes on
      if (!(ml[i].x > -INFINITY) && ml[i].y == 0.f) continue;
      const float m = fmaxf(M[i], ml[i].x);
      const float a = M[i] > -INFINITY ? fast_exp2(M[i] - m) : 0.f;
      const float b = ml[i].x > -INFINITY ? fast_exp2(ml[i].x - m) : 1.f;
      L[i] = L[i] * a + ml[i].y * b;
      o[i] = make_float4(o[i].x * a + v[i].x * b, o[i].y * a + v[i].y * b,
                         o[i].z * a + v[i].z * b, o[i].w * a + v[i].w * b);
      M[i] = m;
    }
  };
  add(slot);
  const int lane = threadIdx.x & 31;
  for (int c0 = c + 1; c0 < G; c0 += 32) {
    const int state = c0 + lane < G ? cuts[c0 + lane].state : 0;
    const bool empty = state & kPromptEmpty, on = !empty && (state & kPromptContinues);
    const uint32_t stops =
        __ballot_sync(0xffffffffu, !empty && (!on || (state & kPromptEnds) != 0));
    uint32_t parts = __ballot_sync(0xffffffffu, on);
    if (stops) parts &= 0xffffffffu >> (32 - __ffs(stops));  // up to the one that ends it
    for (; parts; parts &= parts - 1) add(2 * (c0 + __ffs(parts) - 1));
    if (stops) break;
  }
}

}  // namespace pkv
