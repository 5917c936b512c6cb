// gather.cu -- cached rows read back: the tokens of each sequence, in order, as dense bf16
// rows (one-byte codes times their row's scale, rounded once).
//
// Row out_offsets[s] + i of the output is token starts[s] + i of sequence s, reached
// through the block table ("分页注意力", chenk.top page). A copy, bound by memory: K and V of
// 65536 tokens, 32 heads of 128, bf16: 2148 MB in 309 us (6950 GB/s); 110943 tokens of 8
// heads, E5M2: 689 MB in 104 us (6600 GB/s). A CTA takes 2^tile_log2 consecutive output
// tokens: a warp finds the sequence of the first of up to 32 of them (a 32-way search of the
// offsets by its lanes, two dependent loads for a thousand sequences where a bisection has
// ten), each lane its own token's and the cache row through the table, then all threads move
// rows, 8 elements each (a 16-byte store), with several loads in flight. Rows of one head and
// consecutive tokens are neighbours in the cache, rows of one token neighbours in the output,
// so both sides move whole rows of D elements.
#include "common.cuh"
#include "decode.cuh"
#include "internal.h"

namespace pkv {

namespace {
constexpr int kGatherThreads = 128;
constexpr int kUnroll = 4;         // loads in flight per thread
constexpr int kGatherMaxLog2 = 7;  // at most 128 tokens per CTA
}  // namespace

// The last of the sequences 0 .. B - 1 whose offset is at most n (0 if none is), by the
// whole warp.
__device__ __forceinline__ int gather_sequence_of(const int32_t* offsets, int B, long long n,
                                                  int lane) {
  int lo = 0, len = B;  // the answer is in [lo, lo + len)
  while (len > 1) {
    const int step = (len + 31) / 32, at = lo + lane * step;
    const bool ok = at < lo + len && (lane == 0 || __ldg(offsets + at) <= n);
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, ok));  // offsets never fall
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

template <int D, int CODE>
__global__ void __launch_bounds__(kGatherThreads) paged_kv_gather_kernel(const GatherParams p) {
  constexpr int CPR = D / 8;                   // 8-element chunks per row
  constexpr int RPS = kGatherThreads / CPR;    // rows per step of the CTA
  __shared__ int s_row[1 << kGatherMaxLog2];  // cache row of head 0; -1: zeros, -2: none
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int tid = threadIdx.x, lane = tid & 31;
  const int tokens = 1 << p.tile_log2;
  const long long n0 = (long long)blockIdx.x << p.tile_log2;
  // A warp finds the sequence of the first of up to 32 tokens; a lane's own is the same one,
  // or some way on (bisected for).
  for (int i0 = tid & ~31; i0 < tokens; i0 += kGatherThreads) {
    const int i = i0 + lane;
    const long long n = n0 + i;
    int s = gather_sequence_of(p.offsets, p.B, n0 + i0, lane);
    int row = -2;
    if (i < tokens && n < p.N) {
      int o0 = __ldg(p.offsets + s), o1 = __ldg(p.offsets + s + 1);
      if (o1 <= n) {
        int end = p.B;  // the answer is in [s, end)
        while (end - s > 1) {
          const int mid = s + (end - s) / 2;
          if (__ldg(p.offsets + mid) <= n) s = mid;
          else end = mid;
        }
        o0 = __ldg(p.offsets + s);
        o1 = __ldg(p.offsets + s + 1);
      }
      if (o0 <= n && n < o1) {
        const long long tok = (p.starts ? (long long)__ldg(p.starts + s) : 0ll) + (n - o0);
        int flag = 0;
        row = -1;
        if (tok < 0 || tok >= (long long)p.MBS << p.bs_log2) {
          flag = PKV_DEV_BAD_CONTEXT_LEN;
        } else {
          const int id = __ldg(p.block_tables + size_t(s) * p.MBS + (tok >> p.bs_log2));
          if (id < 0 || id >= p.NB) flag = PKV_DEV_BAD_BLOCK_ID;
          else
            row = ((id * p.Hkv) << p.bs_log2) + int(tok & ((1 << p.bs_log2) - 1));
        }
        if (flag && p.status) atomicOr(p.status, flag);
      }
    }
    if (i < tokens) s_row[i] = row;
  }
  // the offsets themselves: 0 <= offsets[0], never falling, at most N
  if (p.status && blockIdx.x == 0 && blockIdx.y == 0) {
    for (int s = tid; s < p.B; s += kGatherThreads) {
      const int o0 = __ldg(p.offsets + s), o1 = __ldg(p.offsets + s + 1);
      if (o0 < 0 || o1 < o0 || o1 > p.N) atomicOr(p.status, PKV_DEV_BAD_CONTEXT_LEN);
    }
  }
  __syncthreads();
  for (int side = blockIdx.y; side < 2; side += gridDim.y) {  // K, V
    const bool isv = side != 0;
    const uint8_t* cache = isv ? p.vc : p.kc;
    const float* scale = isv ? p.vs : p.ks;
    uint4* out = static_cast<uint4*>(isv ? p.ov : p.ok);
    const int c = tid % CPR;
    const int rows = p.Hkv << p.tile_log2;  // row i: head i >> tile_log2, token i & (tokens - 1)
    for (int i0 = tid / CPR; i0 < rows; i0 += RPS * kUnroll) {
      uint4 raw[kUnroll];
      float sc[kUnroll];
      int src[kUnroll];  // (fewer than 2^31 rows: api.cu)
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        const int i = i0 + k * RPS;
        const int r = i < rows ? s_row[i & (tokens - 1)] : -2;
        src[k] = r < 0 ? r : r + ((i >> p.tile_log2) << p.bs_log2);
        raw[k] = make_uint4(0u, 0u, 0u, 0u);
        sc[k] = 0.f;
        if (src[k] >= 0) {
          if constexpr (CODE < 0) {
            raw[k] = __ldg(reinterpret_cast<const uint4*>(cache) + size_t(src[k]) * CPR + c);
          } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(cache) + size_t(src[k]) * CPR + c);
            raw[k].x = v.x;
            raw[k].y = v.y;
            sc[k] = __ldg(scale + src[k]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kUnroll; ++k) {
        if (src[k] == -2) continue;
        const int i = i0 + k * RPS;
        uint4 v = raw[k];
        if constexpr (CODE >= 0) {
          using Codec = Code8<CODE>;
          const uint32_t w[2] = {Codec::pre(raw[k].x), Codec::pre(raw[k].y)};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 a = unpack_f16x2(Codec::lo(w[e])), b = unpack_f16x2(Codec::hi(w[e]));
            o[2 * e] = pack_bf16x2(a.x * sc[k], a.y * sc[k]);
            o[2 * e + 1] = pack_bf16x2(b.x * sc[k], b.y * sc[k]);
          }
          v = src[k] < 0 ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(o[0], o[1], o[2], o[3]);
        }
        const long long n = n0 + (i & (tokens - 1));
        out[(n * p.Hkv + (i >> p.tile_log2)) * CPR + c] = v;
      }
    }
  }
}

cudaError_t launch_gather(int code, int D, const GatherParams& p, cudaStream_t stream) {
  if (p.N <= 0) return cudaSuccess;
  const void* fn = nullptr;
#define PKV_GATHER(DD, CC) \
  if (D == DD && code == CC) fn = reinterpret_cast<const void*>(&paged_kv_gather_kernel<DD, CC>);
  PKV_GATHER(128, -1)
  PKV_GATHER(64, -1)
  PKV_GATHER(128, CODE_I8)
  PKV_GATHER(64, CODE_I8)
  PKV_GATHER(128, CODE_E4M3)
  PKV_GATHER(64, CODE_E4M3)
  PKV_GATHER(128, CODE_E5M2)
  PKV_GATHER(64, CODE_E5M2)
#undef PKV_GATHER
  if (!fn) return cudaErrorInvalidValue;
  GatherParams copy = p;
  // A CTA moves K and V of as many tokens as give a thread 8 chunks. On GB300 with 4, 8, 12
  // and 16 chunks (CTAs of 256 threads): INT8, ~30000 tokens of 8 heads of 128, 49.0, 38.4,
  // 38.6, 38.6 us; bf16, 65536 tokens of 32 heads, 332, 308, 310, 310. With 8, CTAs of 256,
  // 128 and 64 threads: 38.4, 37.7, 37.9 us; 16 sequences of ~100 tokens 4.4, 3.9, 3.9. A
  // warp per token's search, where lanes now have a token each: 40.9, and one head of 64
  // (640000 tokens) 173 us for 49. Where the tiles leave SMs idle, K and V apart and fewer
  // tokens, down to one chunk per thread (47 tokens of 8 heads of 64: 3.6 -> 2.1 us).
  const int per_token = p.Hkv * (D / 8);  // chunks of K
  auto tiles = [&] { return ((long long)p.N + (1 << copy.tile_log2) - 1) >> copy.tile_log2; };
  copy.tile_log2 = 0;
  while (copy.tile_log2 < kGatherMaxLog2 && (2 * per_token << copy.tile_log2) < 8 * kGatherThreads)
    ++copy.tile_log2;
  const int sides = tiles() < 304 ? 2 : 1;
  while (sides == 2 && copy.tile_log2 > 0 && tiles() * sides < 304 &&
         (per_token << copy.tile_log2) > kGatherThreads)
    --copy.tile_log2;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(unsigned(tiles()), sides), dim3(kGatherThreads), args, 0, stream);
}

}  // namespace pkv
