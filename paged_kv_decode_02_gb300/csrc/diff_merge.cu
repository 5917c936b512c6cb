// diff_merge.cu -- folds the records of units cut between CTAs of the differential decode.
//
// Both maps' records of a (sequence, unit, query pair) fold with the online-softmax
// rescaling (fold.cuh), one output quad of one map per lane; then the difference, the
// optional norm and the bf16 row, as in decode_diff.cuh. It also writes zeros for empty
// sequences and, when a status word is given, checks the sequence's context length and
// block ids (a sequence that fails gets zeros). Units that one CTA covered leave at once, and
// are not visited at all where units are many.
//
// Bound by latency (records are 2 KiB per CTA of the decode and query pair, mostly in L2), so
// the work of a pair spreads as far as the GPU has room: with many pairs D lanes fold a pair's
// few records one chunk after another; with few pairs, whose records may be hundreds, a
// cluster of CTAs shares the columns and sets of lanes share the records.
#include "common.cuh"
#include "fold.cuh"
#include "internal.h"

namespace pkv {

namespace {
constexpr int kDiffMergeThreads = 256;

// Quad `quad` of an output row: v, normed (its mean square: ms) and scaled.
__device__ __forceinline__ void store_row(const DiffParams& p, uint2* out, int quad, float4 v,
                                          float ms) {
  const uint2* w = static_cast<const uint2*>(p.norm_w);
  const float g = w ? rsqrtf(ms + p.eps) * p.out_scale : p.out_scale;
  float4 m = make_float4(g, g, g, g);
  if (w) {
    const uint2 u2 = w[quad];
    const float2 a = unpack_bf16x2(u2.x), b = unpack_bf16x2(u2.y);
    m = make_float4(g * a.x, g * a.y, g * b.x, g * b.y);
  }
  out[quad] = make_uint2(pack_bf16x2(v.x * m.x, v.y * m.y), pack_bf16x2(v.z * m.z, v.w * m.w));
}
}

// Whether sequence s fails the status word's checks, by a warp: the flags (0: it passes).
__device__ __forceinline__ int seq_flags(const DiffParams& p, int s, int L, int lane) {
  int flags = 0;
  if (L < 0 || L > p.MBS * p.BS) flags = PKV_DEV_BAD_CONTEXT_LEN;
  const int nblk = L <= 0 ? 0 : (min(L, p.MBS * p.BS) - 1) / p.BS + 1;
  for (int j = lane; j < nblk; j += 32) {
    const int id = p.block_tables[size_t(s) * p.MBS + j];
    if (id < 0 || id >= p.NB) flags |= PKV_DEV_BAD_BLOCK_ID;
  }
  return __reduce_or_sync(0xffffffffu, flags);
}

// kByCta: the cut units go by the CTAs that began them (more units than CTAs: most are whole);
// behind them a warp per sequence checks it and writes the zeros. Else a set per (sequence,
// unit, query pair) does it all.
template <int D, bool kByCta>
__global__ void __launch_bounds__(kDiffMergeThreads, 5) paged_diff_merge_kernel(const DiffParams p) {
  constexpr int Q = D / 2;          // quads of a 2 D row
  constexpr int kSet = 2 * Q;       // threads of a set: quads of both maps
  constexpr int kSets = kDiffMergeThreads / kSet;
  __shared__ float4 s_o[kSets][Q];
  __shared__ float s_sum[kSets][Q / 32 + 1];
  pdl_wait_prior_grid();
  const int set = threadIdx.x / kSet, t = threadIdx.x % kSet;
  const int map = t / Q, quad = t % Q, lane = threadIdx.x & 31;
  const int U = p.P * p.nsg;
  const unsigned item = blockIdx.x * kSets + set;
  const unsigned owner = item / unsigned(p.gs);  // unit, or CTA
  const int r = int(item % unsigned(p.gs));
  unsigned unit = owner;
  int cut = 0;
  bool valid;
  if constexpr (kByCta) {
    const unsigned merging = (unsigned(p.G * p.gs) + kSets - 1) / kSets;  // CTAs
    if (blockIdx.x >= merging) {
      const int s = int(blockIdx.x - merging) * (kDiffMergeThreads / 32) + threadIdx.x / 32;
      if (s >= p.B) return;
      const int L = p.context_lens[s];
      const int flags = p.status != nullptr ? seq_flags(p, s, L, lane) : 0;
      if (flags && lane == 0) atomicOr(p.status, flags);
      if (L > 0 && !flags) return;
      const size_t n = size_t(p.P) * p.g * (2 * D / 8);  // 16-byte words of the sequence
      uint4* o = static_cast<uint4*>(p.out) + s * n;
      for (size_t i = lane; i < n; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
      return;
    }
    cut = owner < unsigned(p.G) ? p.cuts[owner] : -1;
    valid = cut >= 0;
    unit = valid ? unsigned(cut) >> 1 : 0u;
  } else {
    valid = unit < unsigned(p.B * U);
  }
  const int s = valid ? int(unit / unsigned(U)) : 0, u = int(unit % unsigned(U));
  const int row = (u % p.nsg) * p.gs + r;  // query pair within the KV pair
  const int qp = u / p.nsg * p.g + row;
  const int L = p.context_lens[s];
  int2 part = valid ? reinterpret_cast<const int2*>(p.parts)[unit] : make_int2(-1, 0);
  if constexpr (kByCta) part.x = valid ? int(2 * owner) + (cut & 1) : -1;
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                        (size_t(s) * p.P * p.g + qp) * (2 * D));
  bool active = valid && row < p.g;
  bool zero = L <= 0;
  if (p.status != nullptr) {
    const int flags = seq_flags(p, s, L, lane);
    if (flags) {
      if (!kByCta && valid && t == 0 && u == 0 && r == 0) atomicOr(p.status, flags);
      zero = true;
    }
  }
  if (!kByCta && active && zero && map == 0) out[quad] = make_uint2(0u, 0u);
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
    fold_parts<4>(f, 0, 1, nparts, part_of);
  }
  // (a map without a score above -inf is 0 / 0, NaN, like a unit that is not cut)
  const float inv = 1.f / f.l;
  float4 v = make_float4(f.o.x * inv, f.o.y * inv, f.o.z * inv, f.o.w * inv);
  if (map == 1) s_o[set][quad] = v;
  __syncthreads();
  if (map == 0) {
    const float lam = active ? p.lam[qp] : 0.f;
    const float4 y = s_o[set][quad];
    v = make_float4(v.x - lam * y.x, v.y - lam * y.y, v.z - lam * y.z, v.w - lam * y.w);
    float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) s_sum[set][quad / 32] = ss;
  }
  __syncthreads();
  if (map == 0 && active) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < Q / 32; ++k) ss += s_sum[set][k];
    store_row(p, out, quad, v, ss * (1.f / (2 * D)));
  }
}

// The merge of few pairs, whose records may be many: a cluster of kSlices CTAs per pair, each
// 2 D / kSlices columns of both maps. A set of kSet lanes holds a quad per lane; kThreads /
// kSet sets share the records and fold by shuffles, within a warp and then, through shared
// memory, over the warps. The norm's sum of squares meets in every CTA of the cluster.
template <int D, int kSlices, int kThreads>
__global__ void __cluster_dims__(kSlices, 1, 1) __launch_bounds__(kThreads, kThreads == 64 ? 12 : 3)
    paged_diff_merge_wide_kernel(const DiffParams p) {
  constexpr int kQuads = 2 * D / 4 / kSlices;  // of a row, per CTA
  constexpr int kSet = 2 * kQuads, kWarps = kThreads / 32;
  static_assert(kSet <= 32 && kSet * kWarps <= kThreads, "a set fits a warp, its folds the CTA");
  __shared__ float4 s_o[kSet][kWarps];
  __shared__ float2 s_ml[kSet][kWarps];
  __shared__ float4 s_v[kSet];
  __shared__ float s_sum[kSlices];
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // every CTA runs
  pdl_wait_prior_grid();
  const int tid = threadIdx.x, lane = tid & 31;
  const int slice = blockIdx.x % kSlices;
  const unsigned item = blockIdx.x / kSlices;
  const int U = p.P * p.nsg;
  const unsigned unit = item / unsigned(p.gs);
  const int r = int(item % unsigned(p.gs));
  const int s = int(unit / unsigned(U)), u = int(unit % unsigned(U));
  const int row = (u % p.nsg) * p.gs + r;  // query pair within the KV pair
  const int qp = u / p.nsg * p.g + row;
  const int L = p.context_lens[s];
  const int2 part = reinterpret_cast<const int2*>(p.parts)[unit];
  uint2* out = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                        (size_t(s) * p.P * p.g + qp) * (2 * D));
  bool zero = L <= 0;
  if (p.status != nullptr) {
    int flags = L < 0 || L > p.MBS * p.BS ? PKV_DEV_BAD_CONTEXT_LEN : 0;
    const int nblk = L <= 0 ? 0 : (min(L, p.MBS * p.BS) - 1) / p.BS + 1;
    bool bad = false;
    for (int j = tid; j < nblk; j += kThreads) {
      const int id = p.block_tables[size_t(s) * p.MBS + j];
      bad |= id < 0 || id >= p.NB;
    }
    if (__syncthreads_or(bad)) flags |= PKV_DEV_BAD_BLOCK_ID;
    if (flags) {
      if (tid == 0 && slice == 0 && u == 0 && r == 0) atomicOr(p.status, flags);
      zero = true;
    }
  }
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  // the same in every CTA of the cluster
  if (row >= p.g) return;
  if (zero) {
    if (tid < kQuads) out[slice * kQuads + tid] = make_uint2(0u, 0u);
    return;
  }
  if (part.x < 0) return;

  Fold f = fold_empty();
  {
    const int set = tid / kSet, map = tid % kSet / kQuads, quad = slice * kQuads + tid % kQuads;
    const int w0 = part.x >> 1, nparts = part.y - w0 + 1;
    const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
    auto part_of = [&](int i, const float2*& pm, const float4*& po) {
      const size_t slot = i == 0 ? part.x : 2 * (w0 + i);
      const size_t rr = (slot * 2 + map) * p.gs + r;
      pm = ml + rr;
      po = reinterpret_cast<const float4*>(p.part_o + rr * (2 * D)) + quad;
    };
    fold_parts<8>(f, set, kThreads / kSet, nparts, part_of);
  }
  auto fold_lanes = [&](int first, int end) {
#pragma unroll
    for (int k = first; k < end; k <<= 1) {
      Fold o;
      o.m = __shfl_xor_sync(0xffffffffu, f.m, k);
      o.l = __shfl_xor_sync(0xffffffffu, f.l, k);
      o.o.x = __shfl_xor_sync(0xffffffffu, f.o.x, k);
      o.o.y = __shfl_xor_sync(0xffffffffu, f.o.y, k);
      o.o.z = __shfl_xor_sync(0xffffffffu, f.o.z, k);
      o.o.w = __shfl_xor_sync(0xffffffffu, f.o.w, k);
      fold_merge(f, o);
    }
  };
  fold_lanes(kSet, 32);
  if (lane < kSet) {
    s_o[lane][tid / 32] = f.o;
    s_ml[lane][tid / 32] = make_float2(f.m, f.l);
  }
  __syncthreads();
  if (tid / 32 < (kSet * kWarps + 31) / 32) {  // lane groups of kWarps: one of the set's lanes each
    const int c = tid / kWarps, e = tid % kWarps;
    f = fold_empty();
    if (c < kSet) f = Fold{s_ml[c][e].x, s_ml[c][e].y, s_o[c][e]};
    fold_lanes(1, kWarps);
    // (a map without a score above -inf is 0 / 0, NaN, like a unit that is not cut)
    const float inv = 1.f / f.l;
    if (c < kSet && e == 0)
      s_v[c] = make_float4(f.o.x * inv, f.o.y * inv, f.o.z * inv, f.o.w * inv);
  }
  __syncthreads();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (tid < 32) {
    if (lane < kQuads) {
      const float lam = p.lam[qp];
      const float4 x = s_v[lane], y = s_v[kQuads + lane];
      v = make_float4(x.x - lam * y.x, x.y - lam * y.y, x.z - lam * y.z, x.w - lam * y.w);
    }
    float ss = v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
    if (lane < kSlices)  // into CTA lane's s_sum[slice]
      asm volatile(
          "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
          "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(smem_u32(&s_sum[slice])),
          "r"(lane), "f"(ss)
          : "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < kQuads) {
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < kSlices; ++k) ss += s_sum[k];
    store_row(p, out, slice * kQuads + tid, v, ss * (1.f / (2 * D)));
  }
}

void launch_diff_merge(const DiffParams& p, cudaStream_t stream) {
  const long long items = (long long)p.B * p.P * p.nsg * p.gs;  // below 2^31: api.cu
  if (items <= 0) return;
  DiffParams copy = p;
  void* args[] = {&copy};
  // Threads per pair, by the pairs that share the GPU (whole calls on GB300, head_dim 128):
  //   1 pair, 304 records (bf16, 131072 tokens): one CTA for all columns 96 us, 4 x 64
  //   threads 41, 4 x 128 37, 8 x 256 29.5, 8 x 512 28.3;
  //   16 pairs, 114 records (bf16, 8192 tokens): 29.6, 15.8, 14.8, 13.4, 16.3;
  //   64 pairs (4 x 8192 tokens): 31.9, 27.9, 27.5, 30.7, 39.2;
  //   256 pairs (E4M3, 16 x ~1024): 22.5, 17.3, 19.1, 29.7, 62;
  //   384 pairs (bf16, 24 x ~2048): 46.7, 46.6, 47.7; 512 (32 x ~2048): 57.6, 59.1, 61.9.
  const int pick = items <= 32 ? 0 : items <= 384 ? 1 : 2;
  constexpr int kCtas[] = {8, 4, 1}, kThr[] = {256, 64, kDiffMergeThreads};
  const void* fns[2][3] = {
      {reinterpret_cast<const void*>(&paged_diff_merge_wide_kernel<64, 8, 256>),
       reinterpret_cast<const void*>(&paged_diff_merge_wide_kernel<64, 4, 64>),
       reinterpret_cast<const void*>(&paged_diff_merge_kernel<64, false>)},
      {reinterpret_cast<const void*>(&paged_diff_merge_wide_kernel<128, 8, 256>),
       reinterpret_cast<const void*>(&paged_diff_merge_wide_kernel<128, 4, 64>),
       reinterpret_cast<const void*>(&paged_diff_merge_kernel<128, false>)}};
  const int per = kDiffMergeThreads / p.D;  // pairs per CTA of the last
  unsigned grid = unsigned(pick < 2 ? items * kCtas[pick] : (items + per - 1) / per);
  const void* fn = fns[p.D == 128][pick];
  // at most one cut unit per CTA of the decode begins there: where units are more than CTAs
  // (256 sequences of ~46 tokens, 64/8 heads, bf16: 1024 units, 37.1 us -> 32.8; of ~300
  // tokens, 32/8 heads: 61.2 -> 59.7; of one token: 12.5 -> 10.8)
  if (pick == 2 && (long long)p.B * p.P * p.nsg > p.G) {
    constexpr int kWarps = kDiffMergeThreads / 32;
    grid = unsigned((p.G * p.gs + per - 1) / per) + unsigned((p.B + kWarps - 1) / kWarps);
    fn = p.D == 128 ? reinterpret_cast<const void*>(&paged_diff_merge_kernel<128, true>)
                    : reinterpret_cast<const void*>(&paged_diff_merge_kernel<64, true>);
  }
  launch_pdl(fn, dim3(grid), dim3(kThr[pick]), args, 0, stream);
}

}  // namespace pkv
