// diff_merge.cu -- folds the records of units cut between CTAs of the differential decode.
//
// One warp per (sequence, unit, query pair): both maps' parts fold with the online-softmax
// rescaling (fold.cuh), a lane holding D / 64 output quads of each map; then the
// difference, the optional norm (a warp reduction) and the bf16 row, as in
// decode_diff.cuh. It also writes zeros for empty sequences and, when a status word is
// given, checks the sequence's context length and block ids (a sequence that fails gets
// zeros). Units that one CTA covered leave at once.
#include "common.cuh"
#include "fold.cuh"
#include "internal.h"

namespace pkv {

constexpr int kDiffMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kDiffMergeWarps * 32) paged_diff_merge_kernel(const DiffParams p) {
  constexpr int Q = D / 2, PER = Q / 32;  // quads of a 2 D row, per lane
  pdl_wait_prior_grid();
  const int lane = threadIdx.x & 31;
  const int U = p.P * p.nsg;
  const long long item = (long long)blockIdx.x * kDiffMergeWarps + (threadIdx.x >> 5);
  if (item >= (long long)p.B * U * p.gs) return;
  const int r = int(item % p.gs);
  const int u = int(item / p.gs % U), s = int(item / p.gs / U);
  const int row = (u % p.nsg) * p.gs + r;  // query pair within the KV pair
  const bool active = row < p.g;
  const int qp = u / p.nsg * p.g + row;
  const int n = p.prefix[s + 1] - p.prefix[s];
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                        (size_t(s) * p.P * p.g + qp) * (2 * D));
  bool zero = n == 0;
  if (p.status != nullptr) {
    int flags = 0;
    const int L = p.context_lens[s];
    if (lane == 0 && (L < 0 || L > p.MBS * p.BS)) flags = PKV_DEV_BAD_CONTEXT_LEN;
    const int nblk = L <= 0 ? 0 : min((L + p.BS - 1) / p.BS, p.MBS);
    for (int j = lane; j < nblk; j += 32) {
      const int id = p.block_tables[size_t(s) * p.MBS + j];
      if (id < 0 || id >= p.NB) flags |= PKV_DEV_BAD_BLOCK_ID;
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags) {
      if (lane == 0 && u == 0 && r == 0) atomicOr(p.status, flags);
      zero = true;
    }
  }
  if (!active) return;
  if (zero) {
#pragma unroll
    for (int k = 0; k < PER; ++k) out[k * 32 + lane] = make_uint2(0u, 0u);
    return;
  }
  const long long T = (long long)U * p.prefix[p.B];
  const long long A = (long long)U * p.prefix[s] + (long long)u * n;
  const int G = p.G;
  auto owner = [&](long long x) { return int(((x + 1) * G + T - 1) / T) - 1; };
  const int w0 = owner(A), w1 = owner(A + n - 1);
  if (w0 == w1) return;
  const bool dense = T >= G;  // else ranges hold one item at most: part i is item A + i's
  const int nparts = dense ? w1 - w0 + 1 : n;
  const bool first_cut = T * w0 / G < A;  // CTA w0 had another unit before this one
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  float4 v[2][PER];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      Fold f = fold_empty();
      fold_parts<8>(f, 0, 1, nparts, [&](int i, const float2*& pm, const float4*& po) {
        const size_t slot = dense ? size_t(2 * (w0 + i) + (i == 0 && first_cut ? 1 : 0))
                                  : size_t(2) * owner(A + i);
        const size_t rr = (slot * 2 + m) * p.gs + r;
        pm = ml + rr;
        po = reinterpret_cast<const float4*>(p.part_o + rr * (2 * D)) + k * 32 + lane;
      });
      const float inv = (f.l > 0.f ? 1.f / f.l : 0.f) * (m == 0 ? 1.f : -p.lam[qp]);
      v[m][k] = make_float4(f.o.x * inv, f.o.y * inv, f.o.z * inv, f.o.w * inv);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    v[0][k].x += v[1][k].x;
    v[0][k].y += v[1][k].y;
    v[0][k].z += v[1][k].z;
    v[0][k].w += v[1][k].w;
    const float4 a = v[0][k];
    ss += a.x * a.x + a.y * a.y + a.z * a.z + a.w * a.w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const uint2* w = static_cast<const uint2*>(p.norm_w);
  const float f = w ? rsqrtf(ss * (1.f / (2 * D)) + p.eps) * p.out_scale : p.out_scale;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    float4 g = make_float4(f, f, f, f);
    if (w) {
      const uint2 u2 = w[k * 32 + lane];
      const float2 a = unpack_bf16x2(u2.x), b = unpack_bf16x2(u2.y);
      g = make_float4(f * a.x, f * a.y, f * b.x, f * b.y);
    }
    const float4 a = v[0][k];
    out[k * 32 + lane] =
        make_uint2(pack_bf16x2(a.x * g.x, a.y * g.y), pack_bf16x2(a.z * g.z, a.w * g.w));
  }
}

void launch_diff_merge(const DiffParams& p, cudaStream_t stream) {
  const long long items = (long long)p.B * p.P * p.nsg * p.gs;
  if (items <= 0) return;
  DiffParams copy = p;
  void* args[] = {&copy};
  const void* fn = p.D == 128 ? reinterpret_cast<const void*>(&paged_diff_merge_kernel<128>)
                              : reinterpret_cast<const void*>(&paged_diff_merge_kernel<64>);
  launch_pdl(fn, dim3(unsigned((items + kDiffMergeWarps - 1) / kDiffMergeWarps)),
             dim3(kDiffMergeWarps * 32), args, 0, stream);
}

}  // namespace pkv
