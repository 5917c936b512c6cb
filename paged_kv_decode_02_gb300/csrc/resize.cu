// resize.cu -- sequences grow and shrink: block tables, slots and positions from lengths.
//
// Sequence s holds the first ceil(len / bs) entries of its table row. Growing from len to
// target takes ceil(target / bs) - ceil(len / bs) blocks off a list of free ones and gives
// each new token its position and slot; shrinking gives blocks back ("块管理器：分页如何运作",
// chenk.top page: a request appends blocks as it grows and frees them when it ends).
//
// The list is a stack. All blocks given back are pushed, the last of the last sequence first,
// so that the first one ends on top; then the growing sequences pop theirs in order. Nothing
// is moved twice: with F blocks given back and N taken, taken block i is given-back block i
// where i < F, else entry count - 1 - (i - F) of the list, and the given-back blocks i >= N
// go to entries count + F - 1 - i. So every item's source follows from three exclusive sums
// over the sequences (tokens, blocks taken, blocks given back), and a growth that is undone
// by the next call leaves the list as it was.
// Table rows are read where sequences shrink and written where they grow, the list is read
// (N > F) or written (F > N): no item waits for another, but lengths and the list's count are
// written only once every reader is done.
//
// The sums are a scan over the batch by a CTA's threads, kept in its shared memory; a warp finds
// the sequence of the first of 32 tokens by a 32-way search there, a lane its own from it on.
// Few tokens: one CTA does it all, and hands back what comes back in the same call, however many
// blocks. Many, or none: CTAs on every SM write tables, list and rows, each with its own scan of the
// batch, and a second launch of one CTA then writes lengths, count and offsets (no CTA may change
// what another still reads); it computes its sums beside the first.
// Bound by the chain of length, scan, search, table entry (1.8 MB of rows take 0.3 us). Measured
// on GB300, GPU time of two calls, in and out: 256 prompts of 1 .. 900 tokens 9.4 us (all by one
// CTA some 470; sums of warps added up by each thread 14.3; the commit's sums after the rows
// 22.0); 4096 of 1 .. 200 tokens 23.9; 64 sequences that grow by a token 6.4. Of one call in which 256
// sequences grow by a token 3.5; with one of 2000 tokens that leaves meanwhile 4.2, with 56 of 8000
// (28000 blocks, by the one CTA) 65: such a step is better two calls, the leaving ones first.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace pkv {

namespace {
constexpr int kResizeThreads = 1024;
constexpr int kResizeSmall = 256;       // threads where batch and tokens are no more
constexpr int kResizeOneCta = 4096;     // tokens (or blocks) up to which one CTA does it all
enum : int { kAll = 0, kRows = 1, kCommit = 2 };

// The last of the sequences lo .. hi - 1 whose exclusive sum is at most x (lo if none is).
__device__ __forceinline__ int owner_of(const int* sums, int lo, int hi, int x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}
// The same of 0 .. n - 1, by a whole warp.
__device__ __forceinline__ int owner_by_warp(const int* sums, int n, int x, int lane) {
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 31) / 32, at = lo + lane * step;
    const bool ok = at < lo + len && (lane == 0 || sums[at] <= x);
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, ok));  // sums never fall
    lo += k * step;
    len = min(step, len - k * step);
  }
  return lo;
}

__device__ __forceinline__ int clamp_i32(long long x) {
  return int(x < 0x7fffffffll ? x : 0x7fffffffll);
}
}  // namespace

// What a sequence asks for (nothing if a length does not fit its table row).
struct ResizeWant {
  int len, target, tokens, take, give;
  bool bad;
};

__device__ __forceinline__ ResizeWant resize_want(const ResizeParams& p, int s) {
  ResizeWant w;
  w.len = p.lens[s];
  w.target = p.targets[s];
  const long long room = (long long)p.MBS << p.bs_log2;
  w.bad = w.len < 0 || w.target < 0 || w.len > room || w.target > room;
  if (w.bad) w.target = w.len;
  const int up = (1 << p.bs_log2) - 1;
  // (lengths stay below 2^31 - 2^5: api.cu)
  const int d = w.bad ? 0 : ((w.target + up) >> p.bs_log2) - ((w.len + up) >> p.bs_log2);
  w.tokens = max(0, w.target - w.len);
  w.take = max(0, d);
  w.give = max(0, -d);
  return w;
}

template <int PART>
__global__ void __launch_bounds__(kResizeThreads) paged_kv_resize_kernel(const ResizeParams p) {
  extern __shared__ int s_sums[];  // exclusive sums: tokens, blocks taken, blocks given back
  const int B = p.B;
  int* s_tok = s_sums;
  int* s_take = s_tok + B + 1;
  int* s_give = s_take + B + 1;
  __shared__ long long s_warp[3][kResizeThreads / 32];
  __shared__ int s_taken;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  const int at = blockIdx.x * threads + tid, step = gridDim.x * threads;
  const int up = (1 << p.bs_log2) - 1;
  // kCommit computes its sums while kRows runs, which started after all before it had ended, and
  // changes nothing that the sums read
  if constexpr (PART != kCommit) {
    pdl_wait_prior_grid();
    pdl_allow_next_grid();
  }
  if (tid == 0) s_taken = 0;
  int flags = 0;
  int count = *p.free_count;
  if (count < 0 || count > p.F) {
    count = max(0, min(count, p.F));
    flags |= PKV_DEV_NO_BLOCKS;
  }
  // ---- the three sums, 64 bits wide until they are stored (wishes may exceed any list) ----
  const int per = (B + threads - 1) / threads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long sum[3] = {0, 0, 0};
  ResizeWant mine = {};  // the first of the thread's sequences
  for (int s = b0; s < b1; ++s) {
    const ResizeWant w = resize_want(p, s);
    if (s == b0) mine = w;
    if (w.bad) flags |= PKV_DEV_BAD_CONTEXT_LEN;
    sum[0] += w.tokens;
    sum[1] += w.take;
    sum[2] += w.give;
  }
  long long incl[3] = {sum[0], sum[1], sum[2]};
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long y = __shfl_up_sync(0xffffffffu, incl[i], off);
      if (lane >= off) incl[i] += y;
    }
  }
  if (lane == 31)
    for (int i = 0; i < 3; ++i) s_warp[i][warp] = incl[i];
  __syncthreads();
  const int warps = threads / 32;
  if (warp < 3) {  // warp i: the warps' sums i, inclusive
    long long x = lane < warps ? s_warp[warp][lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    s_warp[warp][lane] = x;
  }
  __syncthreads();
  long long run[3], total[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    run[i] = incl[i] - sum[i] + (warp > 0 ? s_warp[i][warp - 1] : 0);
    total[i] = s_warp[i][warps - 1];
  }
  // (B times the table row's length is below 2^30: block sums fit 32 bits)
  const int given = int(total[2]);
  const long long avail = (long long)count + given;
  // A sequence grows if its tokens have rows and its blocks are there. Once one in order
  // lacks either, so does every later one that asks for the same: the blocks taken are the
  // first ones.
  auto fits = [&](long long tok0, int tokens, int take0, int take) {
    return tok0 + tokens <= p.T && (take == 0 || (long long)take0 + take <= avail);
  };
  for (int s = b0; s < b1; ++s) {
    const ResizeWant w = s == b0 ? mine : resize_want(p, s);
    s_tok[s] = clamp_i32(run[0]);
    s_take[s] = int(run[1]);
    s_give[s] = int(run[2]);
    if (w.tokens > 0) {
      if (!fits(run[0], w.tokens, int(run[1]), w.take)) flags |= PKV_DEV_NO_BLOCKS;
      else if (w.take > 0) atomicMax(&s_taken, int(run[1]) + w.take);
    }
    run[0] += w.tokens;
    run[1] += w.take;
    run[2] += w.give;
  }
  if (tid == 0) {
    s_tok[B] = clamp_i32(total[0]);
    s_take[B] = int(total[1]);
    s_give[B] = given;
  }
  __syncthreads();
  const int taken = s_taken;
  if constexpr (PART != kCommit) {
    // given-back block i: the entries that shrinking sequences no longer hold
    auto given_block = [&](int i) {
      const int s = owner_of(s_give, 0, B, i);
      const int col = ((p.targets[s] + up) >> p.bs_log2) + (i - s_give[s]);
      return p.tables[size_t(s) * p.MBS + col];
    };
    auto taken_block = [&](int i) {
      return i < given ? given_block(i) : p.free_list[count - 1 - (i - given)];
    };
    int full = 0;
    for (int i = at; i < taken; i += step) {
      const int s = owner_of(s_take, 0, B, i);
      const int col = ((p.lens[s] + up) >> p.bs_log2) + (i - s_take[s]);
      p.tables[size_t(s) * p.MBS + col] = taken_block(i);
    }
    for (int i = taken + at; i < given; i += step) {
      const long long to = (long long)count + given - 1 - i;
      if (to < p.F) p.free_list[to] = given_block(i);
      else full = PKV_DEV_NO_BLOCKS;  // more blocks than the list holds: lost
    }
    if (PART == kRows && full && p.status) atomicOr(p.status, full);
    flags |= full;
    // ---- the new tokens ----
    const int all = s_tok[B];
    for (long long t0 = at - lane; t0 < p.T; t0 += step) {
      const long long t = t0 + lane;
      int s = owner_by_warp(s_tok, B, int(t0), lane);
      if (t >= p.T) continue;
      long long slot = -1, pos = 0;
      if (t < all) {
        if (s_tok[s + 1] <= t) s = owner_of(s_tok, s, B, int(t));
        const int tok0 = s_tok[s], take0 = s_take[s];
        if (fits(tok0, s_tok[s + 1] - tok0, take0, s_take[s + 1] - take0)) {
          const int len = p.lens[s];
          const int n = len + int(t - tok0), col = n >> p.bs_log2;
          const int held = (len + up) >> p.bs_log2;
          const int id = col < held ? p.tables[size_t(s) * p.MBS + col]
                                    : taken_block(take0 + col - held);
          slot = ((long long)id << p.bs_log2) + (n & up);
          pos = n;
        }
      }
      p.slots[t] = slot;
      p.positions[t] = pos;
    }
  }
  if constexpr (PART == kCommit) {
    pdl_wait_prior_grid();
    pdl_allow_next_grid();
  }
  if constexpr (PART != kRows) {
    for (int s = tid; s <= B; s += threads) p.offsets[s] = s_tok[s];
    __syncthreads();  // every read of the lengths and the count is done
    for (int s = b0; s < b1; ++s) {
      const ResizeWant w = s == b0 ? mine : resize_want(p, s);
      if (!w.bad && (w.tokens == 0 || fits(s_tok[s], w.tokens, s_take[s], w.take)))
        p.lens[s] = w.target;
    }
    if (tid == 0) *p.free_count = int(min((long long)p.F, avail - taken));
    if (flags && p.status) atomicOr(p.status, flags);
  }
}

cudaError_t launch_resize(const ResizeParams& p, cudaStream_t stream) {
  const size_t smem = size_t(12) * (p.B + 1);
  ResizeParams copy = p;
  void* args[] = {&copy};
  auto go = [&](const void* fn, int grid, int threads) {
    // (a CTA has 48 KB without asking, static arrays among them: some 800 bytes here)
    if (smem > 40 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 12 * (kResizeMaxSeqs + 1));
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(fn, dim3(grid), dim3(threads), args, smem, stream);
  };
  // (a call without tokens gives blocks back, as many as the tables hold at most)
  const long long work = p.T > 0 ? p.T : (long long)p.B * p.MBS;
  if (work <= kResizeOneCta)
    return go(reinterpret_cast<const void*>(&paged_kv_resize_kernel<kAll>), 1,
              p.B <= kResizeSmall && p.T <= kResizeSmall ? kResizeSmall : kResizeThreads);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int rows = int(std::min(work, 1ll << 30) - 1) / kResizeThreads + 1;  // CTAs with one per thread
  e = go(reinterpret_cast<const void*>(&paged_kv_resize_kernel<kRows>), rows < sms ? rows : sms,
         kResizeThreads);
  if (e != cudaSuccess) return e;
  return go(reinterpret_cast<const void*>(&paged_kv_resize_kernel<kCommit>), 1,
            p.B <= kResizeSmall ? kResizeSmall : kResizeThreads);
}

}  // namespace pkv
