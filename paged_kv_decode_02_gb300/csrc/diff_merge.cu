// diff_merge.cu -- folds the records of units cut between CTAs of the differential decode.
//
// One CTA part per (sequence, unit, query pair): both maps' records fold with the
// online-softmax rescaling (fold.cuh), one output quad of one map per lane, so D / 32 warps
// hold both rows of 2 D columns and every record of a chunk is requested at once; kGroups
// such sets share the records of a pair when few pairs leave the GPU idle otherwise. Then
// the difference, the optional norm and the bf16 row, as in decode_diff.cuh. It also
// writes zeros for empty sequences and, when a status word is given, checks the sequence's
// context length and block ids (a sequence that fails gets zeros). Units that one CTA
// covered leave at once.
#include "common.cuh"
#include "fold.cuh"
#include "internal.h"

namespace pkv {

namespace {
constexpr int kDiffMergeThreads = 256;
}

// kGroups == 1: a CTA takes several pairs; else one pair and kGroups sets of warps.
template <int D, int kGroups>
__global__ void __launch_bounds__(kGroups == 1 ? kDiffMergeThreads : kGroups * D,
                                  kGroups == 1 ? 5 : 1)
    paged_diff_merge_kernel(const DiffParams p) {
  constexpr int Q = D / 2;          // quads of a 2 D row
  constexpr int kSet = 2 * Q;       // threads of a set: quads of both maps
  constexpr int kSets = kGroups == 1 ? kDiffMergeThreads / kSet : kGroups;
  __shared__ float4 s_o[kSets][kSet];
  __shared__ float2 s_ml[kSets][kSet];
  __shared__ float s_sum[kSets][Q / 32 + 1];
  pdl_wait_prior_grid();
  const int set = threadIdx.x / kSet, t = threadIdx.x % kSet;
  const int map = t / Q, quad = t % Q, lane = threadIdx.x & 31;
  const int group = kGroups == 1 ? 0 : set;
  const int U = p.P * p.nsg;
  const unsigned item = kGroups == 1 ? blockIdx.x * kSets + set : blockIdx.x;
  const unsigned unit = item / unsigned(p.gs);
  const bool valid = unit < unsigned(p.B * U);
  const int r = int(item % unsigned(p.gs));
  const int s = valid ? int(unit / unsigned(U)) : 0, u = int(unit % unsigned(U));
  const int row = (u % p.nsg) * p.gs + r;  // query pair within the KV pair
  const int qp = u / p.nsg * p.g + row;
  const int L = p.context_lens[s];
  const int2 part = valid ? reinterpret_cast<const int2*>(p.parts)[unit] : make_int2(-1, 0);
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                        (size_t(s) * p.P * p.g + qp) * (2 * D));
  bool active = valid && row < p.g;
  bool zero = L <= 0;
  if (p.status != nullptr) {
    int flags = 0;
    if (L < 0 || L > p.MBS * p.BS) flags = PKV_DEV_BAD_CONTEXT_LEN;
    const int nblk = L <= 0 ? 0 : (min(L, p.MBS * p.BS) - 1) / p.BS + 1;
    for (int j = lane; j < nblk; j += 32) {  // every warp for itself
      const int id = p.block_tables[size_t(s) * p.MBS + j];
      if (id < 0 || id >= p.NB) flags |= PKV_DEV_BAD_BLOCK_ID;
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags) {
      if (valid && t == 0 && group == 0 && u == 0 && r == 0) atomicOr(p.status, flags);
      zero = true;
    }
  }
  if (active && zero && map == 0 && group == 0) out[quad] = make_uint2(0u, 0u);
  active = active && !zero && part.x >= 0;  // (an empty sequence has no entry)

  Fold f = fold_empty();
  if (active) {
    const int w0 = part.x >> 1, nparts = part.y - w0 + 1;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    auto part_of = [&](int i, const float2*& pm, const float4*& po) {
      const size_t slot = i == 0 ? part.x : 2 * (w0 + i);
      const size_t rr = (slot * 2 + map) * p.gs + r;
      pm = ml + rr;
      po = reinterpret_cast<const float4*>(p.part_o + rr * (2 * D)) + quad;
    };
    fold_parts<kGroups == 1 ? 4 : 8>(f, group, kGroups, nparts, part_of);
  }
  if constexpr (kGroups > 1) {
    s_o[set][t] = f.o;
    s_ml[set][t] = make_float2(f.m, f.l);
    __syncthreads();
    if (group == 0) {
#pragma unroll 1
      for (int k = 1; k < kGroups; ++k)
        fold_merge(f, Fold{s_ml[k][t].x, s_ml[k][t].y, s_o[k][t]});
    }
    __syncthreads();
  }
  // (a map without a score above -inf is 0 / 0, NaN, like a unit that is not cut)
  const float inv = 1.f / f.l;
  float4 v = make_float4(f.o.x * inv, f.o.y * inv, f.o.z * inv, f.o.w * inv);
  if (map == 1 && group == 0) s_o[set][quad] = v;
  __syncthreads();
  if (map == 0 && group == 0) {
    const float lam = active ? p.lam[qp] : 0.f;
    const float4 y = s_o[set][quad];
    v = make_float4(v.x - lam * y.x, v.y - lam * y.y, v.z - lam * y.z, v.w - lam * y.w);
    float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) s_sum[set][quad / 32] = ss;
  }
  __syncthreads();
  if (map == 0 && group == 0 && active) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < Q / 32; ++k) ss += s_sum[set][k];
    const uint2* w = static_cast<const uint2*>(p.norm_w);
    const float g = w ? rsqrtf(ss * (1.f / (2 * D)) + p.eps) * p.out_scale : p.out_scale;
    float4 m = make_float4(g, g, g, g);
    if (w) {
      const uint2 u2 = w[quad];
      const float2 a = unpack_bf16x2(u2.x), b = unpack_bf16x2(u2.y);
      m = make_float4(g * a.x, g * a.y, g * b.x, g * b.y);
    }
    out[quad] = make_uint2(pack_bf16x2(v.x * m.x, v.y * m.y), pack_bf16x2(v.z * m.z, v.w * m.w));
  }
}

void launch_diff_merge(const DiffParams& p, cudaStream_t stream) {
  const long long items = (long long)p.B * p.P * p.nsg * p.gs;  // below 2^31: api.cu
  if (items <= 0) return;
  DiffParams copy = p;
  void* args[] = {&copy};
  // few pairs may be cut into many records each: 8 sets of warps per pair
  constexpr int kG = 8;
  const bool few = items * kG * p.D <= 152 * 2048;
  const int per = few ? 1 : kDiffMergeThreads / p.D;
  const dim3 grid(unsigned((items + per - 1) / per)), block(few ? kG * p.D : kDiffMergeThreads);
  const void* fn =
      p.D == 128 ? (few ? reinterpret_cast<const void*>(&paged_diff_merge_kernel<128, kG>)
                        : reinterpret_cast<const void*>(&paged_diff_merge_kernel<128, 1>))
                 : (few ? reinterpret_cast<const void*>(&paged_diff_merge_kernel<64, kG>)
                        : reinterpret_cast<const void*>(&paged_diff_merge_kernel<64, 1>));
  launch_pdl(fn, grid, block, args, 0, stream);
}

}  // namespace pkv
