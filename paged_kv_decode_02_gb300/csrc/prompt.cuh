// prompt.cuh -- causal attention of whole prompts on the fifth-generation tensor cores:
// packed sequences of different lengths, grouped heads, dense bf16 rows (instantiated in
// prompt.cu).
//
// Sequence s has nq query rows (tokens) and nk >= or < nq key rows, the queries being its
// last tokens: query i sees keys j <= nk - nq + i ("两个特性截然不同的阶段", chenk.top page: the
// prefill computes attention over the whole prompt at once; nk > nq is a chunk of chunked
// prefill over keys that are already cached).
//   out[i, h] = softmax(scale * K q[i, h]) V over the keys it sees (zeros if none).
//
// Work. The g query heads of a KV head share its keys, so a tile of 128 MMA rows is
// tpt = 128 / g tokens times g heads (row = token * g + head; the last 128 % g rows are
// unused), and K and V are read once for all of them. An item is two such tiles, X = 0 and 1,
// of one KV head: 2 tpt consecutive tokens; its keys are walked in tiles of kKeys. The items of
// all sequences and heads lie on one line on which an item takes as many positions as its
// last token sees keys, plus a constant for its end, and each CTA takes an equal stretch of it:
// stretches are cut between key tiles, an item that is cut leaves unnormalised records
// (o, m, l), at most two per CTA, that a second kernel joins. So one long prompt and many
// short ones fill the SMs alike, without host knowledge of the lengths, and no order of
// atomics touches a result.
//
// A CTA (704 threads, 80 registers):
//   warp 0      TMA: Q of both tiles, K and V tiles through one ring of stages;
//   warps 1, 2  one thread each issues S_X = Q_X K_j^T into the score columns of tile 0, tile 1;
//   warps 3, 20 one thread each issues O_X += P_X V_j with P_X (bf16) read from TMEM, after the
//               warp has zeroed V rows past the sequence's end (they may hold anything). Four
//               issuers, since a thread spends 500 to 700 cycles on the waits and commits around
//               its MMAs, with nearly none queued behind them, and 300 to 450 on the MMAs: one
//               thread for all of them took 4900 cycles a step, two (one per tile) 2300;
//   warp 21     walks the CTA's stretch and tells the others its segments, through a queue;
//   warps 4..11 softmax of tile 0, warps 12..19 of tile 1: two threads per query row, each
//               with half of the tile's columns (and of O's), so that four warps per SM
//               sub-partition hide each other's latencies.
// Scores, P and O of both tiles have TMEM columns of their own, so the scores of key tile j + 1
// are computed while the exponentials of tile j run (as soon as its scores have been read), and
// a softmax never waits for P.V: the tensor cores are what the loop should wait for. For D = 128
// that fits 512 columns with key tiles of 80 (2 x (80 + 40 + 128)). Measured on GB300, cycles
// of the MMAs of one 128-row tile per key tile, of the ideal rate's: N = 64 648 (79 %), 80 717
// (89 %), 96 813 (94 %), 128 1025 (100 %; Q and K come from shared memory, whose bandwidth bounds
// small N); with 128 keys, P over the scores it came from and so every step of a tile in
// sequence, a step took 3500 cycles for two tiles, where the MMAs take 2050.
// GPU time on GB300, calls of a graph: 32768 tokens, 32 / 8 heads, 6.1 ms (1440 TFLOP/s; 6.3 to 6.7
// where inputs change from call to call, by the power the part is given); 8192 tokens 427 us (1290);
// 16 x 1024, 64 / 8 heads, 333 us (820); chunks of 256 over 1500, 184 us (1000). What is left is the end of an item, some 7000 cycles of a tile's
// softmax warps where a step of 80 keys takes 2050: the last P.V, O through shared memory to its
// rows, the next segment; and the softmax does not fit its registers (80 a thread: 60 to 64 bytes of
// spill stores, 72 to 80 of loads). Tried, and slower: the end put off behind the next item's first softmax
// (340 -> 413 us at 16 x 1024: longer live ranges in the loop), the next segment taken before it
// (377), both P.V by one thread and the walk by the TMA thread (393, with 91 registers in place of
// 80), rows stored as whole lines, half a warp's at a time (430), segments read again at their end
// (fewer spills: 339), waits by try_wait (8192 tokens: 437 -> 503).
// The softmax keeps a reference maximum per row that moves only when a tile's maximum exceeds
// it by more than 8 (log2 units; weights then reach 2^8 and keep their relative precision), so
// O is rescaled in TMEM a few times per item at most. Scores, maxima and sums are fp32; a
// weight is rounded once to bf16 as the MMA's operand, the sum takes it before that: results are
// within 0.0018 to 0.0022 (relative, all elements) of those in 64 bits, of which the rounding of the
// output alone makes 0.0016. Weights as two bf16 terms, whose second P.V adds the rest, leave only
// that rounding, and cost 25 % (16 x 1024, 64 / 8 heads: 333 -> 418 us) to 44 % (32768 tokens): P of
// both terms leaves TMEM columns for 64 keys a tile, and P.V doubles. One term, as in the multi-query
// decode of the same rows.
// Every wait is bounded: on a timeout the CTA sets a status bit, lets its copies and MMAs
// complete, frees its TMEM and leaves.
#pragma once

#include "decode.cuh"
#include "tcgen05.cuh"

namespace pkv {

template <int D>
struct PromptCfg {
  static constexpr int kRows = 128;              // MMA rows of a tile
  static constexpr int kKeys = 80;               // keys per tile
  static constexpr int kSlabs = D / 64;          // 128-byte column slabs of a row
  static constexpr int kSlabQ = kRows * 128;     // bytes of one slab of a Q tile
  static constexpr int kTileQ = kSlabs * kSlabQ;
  static constexpr int kSlab = kKeys * 128;      // bytes of one slab of a K or V tile
  static constexpr int kTile = kSlabs * kSlab;
  static constexpr int kStages = 6;
  static constexpr int kOffQ = 0;                // both tiles' queries
  static constexpr int kOffKV = 2 * kTileQ;      // the ring: K, V, K, V, ...
  static constexpr int kOffOut = kOffKV + kStages * kTile;  // 32 rows of 64 bytes per softmax warp
  static constexpr int kQueue = 4;               // segments told ahead
  static constexpr int kOffQueue = kOffOut + 16 * 2048;  // 64 bytes each
  static constexpr int kOffBar = kOffQueue + kQueue * 64;
  // full[stages] empty[stages] qfull[2] qempty[2] sfull[2] sread[2] pfull[2] pdone[2] ofree[2]
  // mdone[4] told[queue] heard[queue]
  static constexpr int kNumBars = 2 * kStages + 18 + 2 * kQueue;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmemSlot + 4;
  static constexpr int kOffScan = (kOffAbort + 4 + 15) / 16 * 16;  // warps' sums, both ends
  static constexpr int kSmem = kOffScan + 256 + 1024;              // + alignment of the base
  static constexpr int kThreads = 704;
  // TMEM columns of tile 0 and tile 1: scores (fp32), P (bf16 pairs), O (fp32)
  static constexpr int kColS = 0, kColP = 2 * kKeys, kColO = 3 * kKeys;
  static_assert(kColO + 2 * D <= 512, "TMEM columns");
  static_assert(kKeys % 16 == 0 && kSlab % 1024 == 0 && kOffOut % 1024 == 0, "swizzle atoms");
  static_assert(kStages % 2 == 0, "K tiles on even stages");
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// One sequence's rows, and its items of `per` tokens.
struct PromptSeq {
  int q0, nq, k0, nk;
  __device__ __forceinline__ void load(const PromptParams& p, int s) {
    q0 = __ldg(p.q_offsets + s);
    k0 = __ldg(p.kv_offsets + s);
    const int q1 = __ldg(p.q_offsets + s + 1), k1 = __ldg(p.kv_offsets + s + 1);
    const bool bad = q0 < 0 || q1 < q0 || q1 > p.Tq || k0 < 0 || k1 < k0 || k1 > p.Tk;
    nq = bad ? 0 : q1 - q0;
    nk = bad ? 0 : k1 - k0;
  }
  __device__ __forceinline__ bool bad(const PromptParams& p, int s) const {
    const int a = __ldg(p.q_offsets + s), b = __ldg(p.q_offsets + s + 1);
    const int c = __ldg(p.kv_offsets + s), d = __ldg(p.kv_offsets + s + 1);
    return a < 0 || b < a || b > p.Tq || c < 0 || d < c || d > p.Tk;
  }
  __device__ __forceinline__ int items(int per) const { return (nq + per - 1) / per; }
  // keys that the first `end` tokens see
  __device__ __forceinline__ int seen(int end) const { return max(0, nk - nq + end); }
  // positions of a head's first i items (i <= items): each takes the keys its last token
  // sees, and `cost`
  __device__ __forceinline__ long long before(int i, int per, int cost) const {
    const int all = items(per);
    const long long f = i < all ? i : all - 1;  // full items: the last one ends at nq
    if (all == 0) return 0;
    const long long e = (long long)nk - nq;
    const long long i0 = e < 0 ? (-e) / per : 0;  // items before it see nothing
    long long sum = i * (long long)cost;
    if (f > i0) sum += (f - i0) * e + per * ((f * (f + 1) - i0 * (i0 + 1)) / 2);
    if (i == all) sum += nk;
    return sum;
  }
  __device__ __forceinline__ int key_tiles(int end, int keys) const {
    return max(1, (seen(end) + keys - 1) / keys);
  }
};

// A place on the line: key tile j of item i of KV head h of sequence s.
struct PromptPlace {
  int s, h, i, j;
};

// What a CTA does of one item: key tiles [ja, jb) of n; tile X takes those below nx[X].
struct alignas(16) PromptSeg {
  PromptSeq q;
  int s, h, i, ja, jb, n;
  int nx0, nx1;
  int some;  // 0: there is none, the stretch is over
  int pad[3];
  __device__ __forceinline__ int nx(int X) const { return X ? nx1 : nx0; }
  // tile X has key tiles [ja, end(X)) here
  __device__ __forceinline__ int end(int X) const { return min(jb, nx(X)); }
  __device__ __forceinline__ bool has(int X) const { return nx(X) > ja; }
};

static_assert(sizeof(PromptSeg) == 64, "a place in the queue");

// Walks a CTA's stretch, one segment after the other.
struct PromptWalk {
  PromptPlace at, stop;
  PromptSeq q;
  bool loaded;
  __device__ __forceinline__ void begin(const PromptPlace& a, const PromptPlace& b) {
    at = a;
    stop = b;
    loaded = false;
  }
  // the next segment, if there is one
  __device__ __forceinline__ bool next(const PromptParams& p, PromptSeg& g) {
    const int per = 2 * p.tpt;
    for (;;) {
      if (at.s >= p.B || at.s > stop.s) return false;
      if (!loaded) {
        q.load(p, at.s);
        loaded = true;
      }
      if (at.i >= q.items(per)) {
        at.i = at.j = 0;
        if (q.nq == 0 || ++at.h >= p.Hkv) {
          at.h = 0;
          ++at.s;
          loaded = false;
        }
        continue;
      }
      const bool last = at.s == stop.s && at.h == stop.h && at.i == stop.i;
      if (at.s == stop.s && (at.h > stop.h || (at.h == stop.h && at.i > stop.i))) return false;
      const int t0 = at.i * per, t1 = min(q.nq, t0 + per);
      g.q = q;
      g.s = at.s;
      g.h = at.h;
      g.i = at.i;
      g.n = q.key_tiles(t1, p.keys);
      g.ja = at.j;
      g.jb = last ? min(stop.j, g.n) : g.n;
      g.nx0 = q.key_tiles(min(q.nq, t0 + p.tpt), p.keys);
      g.nx1 = t0 + p.tpt < q.nq ? g.n : 0;
      if (g.nx1 == 0) g.nx0 = g.n;
      at.j = 0;
      ++at.i;
      if (last && g.jb <= g.ja) return false;
      if (g.jb > g.ja) return true;
    }
  }
};

// The place of position x of sequence s's part of the line (0 <= x < its length).
__device__ __forceinline__ PromptPlace prompt_locate(const PromptParams& p, const PromptSeq& q,
                                                     int s, long long x) {
  const int per = 2 * p.tpt, all = q.items(per);
  const long long head = q.before(all, per, p.item_cost);
  PromptPlace c;
  c.s = s;
  c.h = int(x / head);
  x -= c.h * head;
  int lo = 0, hi = all;  // before(lo) <= x < before(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q.before(mid, per, p.item_cost) <= x) lo = mid;
    else hi = mid;
  }
  c.i = lo;
  x -= q.before(lo, per, p.item_cost);
  const int n = q.key_tiles(min(q.nq, (lo + 1) * per), p.keys);
  c.j = int(min((long long)n, (x + p.keys - 1) / p.keys));
  return c;
}

// A row's softmax state: the reference of its weights and of O (log2 units; the same in both
// threads), and the sum of this thread's weights.
struct PromptRow {
  float m, l;
};

// A warp's place in its tile's pipeline: TMEM columns of scores, P and O; barriers; the step.
struct PromptStep {
  uint32_t ts, tp, to, sread, pdone, pfull, step;
  int lane;
  bool begun;  // O holds key tiles before this one
};

// Half a row (a thread) of a score tile: the scores become weights 2^(scale s - m), bf16 pairs in
// P's columns. kWhole: the row sees all of the tile's columns, else the first `vis` of this half;
// kNeg: the scale is negative. Returns false on a timeout.
template <int D, bool kWhole, bool kNeg, typename Wait>
__device__ __forceinline__ bool prompt_softmax(const PromptStep& at, float sl, int vis,
                                               tc::RowPair& pair, PromptRow& row, bool& gone,
                                               const Wait& wait) {
  constexpr int N = PromptCfg<D>::kKeys / 2;
  uint32_t s[N];
  tc::tmem_ld(at.ts, s);
  tc::fence_before_sync();
  __syncwarp();
  if (at.lane == 0) mbar_arrive(at.sread);  // the next scores may come
  if constexpr (!kWhole) {
#pragma unroll
    for (int t = 0; t < N; ++t)
      if (t >= vis) s[t] = kNeg ? 0x7f800000u : 0xff800000u;  // the scaled score: -inf
  }
  auto most = [](float x, float y, float z) {
    return kNeg ? fminf(x, fminf(y, z)) : fmax3(x, y, z);
  };
  float mx[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) mx[t] = __uint_as_float(s[t]);
#pragma unroll
  for (int t = 0; t < (N - 8) / 2; ++t)
    mx[t & 7] = most(mx[t & 7], __uint_as_float(s[8 + 2 * t]), __uint_as_float(s[9 + 2 * t]));
  const float mine = sl * most(most(mx[0], mx[1], mx[2]), most(mx[3], mx[4], mx[5]),
                               most(mx[6], mx[7], mx[7]));
  const float top = fmaxf(mine, pair.swap(mine, gone));
  if (gone) return false;
  float alpha = 1.f;
  const bool up = top > row.m + 8.f;
  if (up) {
    alpha = fast_exp2(row.m - top);  // 0 while the row has seen nothing
    row.m = top;
    row.l *= alpha;
  }
  // (scores of -inf alone: weights 0, not 2^(-inf + inf))
  const float m = row.m > -INFINITY ? row.m : 0.f;
  const float2 sl2 = make_float2(sl, sl), nm2 = make_float2(-m, -m);
  float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  uint32_t pk[N / 2];
#pragma unroll
  for (int t = 0; t < N; t += 2) {
    const float2 x =
        __ffma2_rn(make_float2(__uint_as_float(s[t]), __uint_as_float(s[t + 1])), sl2, nm2);
    float2 w = make_float2(fast_exp2(x.x), fast_exp2(x.y));
    if constexpr (!kWhole) {
      w.x = t < vis ? w.x : 0.f;
      w.y = t + 1 < vis ? w.y : 0.f;
    }
    ls[(t >> 1) & 1] = __fadd2_rn(ls[(t >> 1) & 1], w);
    pk[t / 2] = pack_bf16x2(w.x, w.y);
  }
  const float2 l2 = __fadd2_rn(ls[0], ls[1]);
  row.l += l2.x + l2.y;
  // P.V of the tile before has completed: P's columns are free, O holds what came before
  if (at.step > 0 && !wait(at.pdone, at.step - 1)) return false;
  tc::fence_after_sync();
  if (at.begun && __any_sync(0xffffffffu, up)) {
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 16) {
      uint32_t o[16];
      tc::tmem_ld16(at.to + c, o);
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
      tc::tmem_st16(at.to + c, o);
    }
  }
  tc::tmem_st(at.tp, pk);
  tc::fence_before_sync();
  __syncwarp();
  if (at.lane == 0) mbar_arrive(at.pfull);
  return true;
}

template <int D>
__global__ void __launch_bounds__(PromptCfg<D>::kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tmq,
                            const __grid_constant__ CUtensorMap tmk,
                            const __grid_constant__ CUtensorMap tmv, const PromptParams p) {
  using K = PromptCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + K::kOffAbort);
  long long* s_scan = reinterpret_cast<long long*>(gbase + K::kOffScan);  // [22] warps' sums
  PromptPlace* s_place = reinterpret_cast<PromptPlace*>(s_scan + 22);     // [2]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return base + K::kOffBar + 8 * i; };
  auto full = [&](int st) { return bar(st); };
  auto empty = [&](int st) { return bar(K::kStages + st); };
  constexpr int kB = 2 * K::kStages;
  auto qfull = [&](int X) { return bar(kB + X); };
  auto qempty = [&](int X) { return bar(kB + 2 + X); };
  auto sfull = [&](int X) { return bar(kB + 4 + X); };
  auto sread = [&](int X) { return bar(kB + 6 + X); };
  auto pfull = [&](int X) { return bar(kB + 8 + X); };
  auto pdone = [&](int X) { return bar(kB + 10 + X); };
  auto ofree = [&](int X) { return bar(kB + 12 + X); };
  auto mdone = [&](int i) { return bar(kB + 14 + i); };
  auto told = [&](int i) { return bar(kB + 18 + i); };
  auto heard = [&](int i) { return bar(kB + 18 + K::kQueue + i); };
  const uint32_t tmem_slot = base + K::kOffTmemSlot;

  if (tid == 0) {
    for (int i = 0; i < K::kNumBars; ++i) {
      const int k = (i - kB) >> 1;
      // sread, pfull, ofree: one arrival per softmax warp; empty: one per tile
      const bool soft = i >= kB && (k == 3 || k == 4 || k == 6);
      // heard: one per warp that listens
      mbar_init(bar(i), soft                            ? 8
                        : i >= K::kStages && i < kB     ? 2
                        : i >= kB + 18 + K::kQueue      ? 21
                                                        : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tc::tmem_alloc(tmem_slot, 512);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmq);
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  pdl_wait_prior_grid();

  // ---- the line: each thread sums some sequences, the block scans, and the threads that
  //      hold the two ends of this CTA's stretch locate them ----
  const int per = 2 * p.tpt;
  const int chunk = (p.B + K::kThreads - 1) / K::kThreads;
  const int b0 = min(p.B, tid * chunk), b1 = min(p.B, b0 + chunk);
  long long sum = 0;
  int bad = 0;
  for (int s = b0; s < b1; ++s) {
    PromptSeq q;
    q.load(p, s);
    if (p.status && q.bad(p, s)) bad = PKV_DEV_BAD_CONTEXT_LEN;
    sum += p.Hkv * q.before(q.items(per), per, p.item_cost);
  }
  if (bad && blockIdx.x == 0) atomicOr(p.status, bad);
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (tid < 2) s_place[tid] = PromptPlace{p.B, 0, 0, 0};
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  long long run = incl - sum, total = 0;
  for (int w = 0; w < K::kThreads / 32; ++w) {
    if (w < warp) run += s_scan[w];
    total += s_scan[w];
  }
  // stretches of at least min_range positions; CTAs past the last one do nothing
  const int G = int(min((long long)gridDim.x, max(1ll, total / p.min_range)));
  const int c = blockIdx.x;
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + K::kOffTmemSlot);
  if (c < G) {
    for (int e = 0; e < 2; ++e) {
      const long long x = total / G * (c + e) + total % G * (c + e) / G;
      if (x < run || x >= run + sum) continue;  // (x = total: the place past the end)
      long long r = run;
      for (int s = b0; s < b1; ++s) {
        PromptSeq q;
        q.load(p, s);
        const long long len = p.Hkv * q.before(q.items(per), per, p.item_cost);
        if (x < r + len) {
          s_place[e] = prompt_locate(p, q, s, x - r);
          break;
        }
        r += len;
      }
    }
  }
  __syncthreads();
  const bool active = c < G;
  // the join's CTAs come early and wait (16 x 1024, 64 / 8 heads: 345 -> 341 us)
  pdl_allow_next_grid();
  const PromptPlace first = s_place[0], stop = s_place[1];
  PromptWalk walk;
  walk.begin(first, stop);
  // the next segment told, to one lane or to a whole warp; false: the stretch is over
  uint32_t heard_of = 0;
  auto take = [&](PromptSeg& g, bool whole_warp) {
    const uint32_t slot = heard_of % K::kQueue;
    bool ok = tc::poll_or_abort(told(slot), (heard_of / K::kQueue) & 1u, p.timeout_ns, abort_flag);
    if (whole_warp) ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    if (!ok) return false;
    ++heard_of;
    const uint32_t from = base + K::kOffQueue + slot * 64;
    uint4* to = reinterpret_cast<uint4*>(&g);
#pragma unroll
    for (int k = 0; k < 4; ++k) to[k] = lds128(from + 16 * k);
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(heard(slot));
    return g.some != 0;
  };
  if (warp == 21) {
    // ---------------- the walk ----------------
    if (lane == 0) {
      // for the kernel that joins the records: how the first segment and the last one are cut
      PromptCut cut = {-1, 0, 0, 0, active ? kPromptEmpty : 0};
      PromptSeg g;
      bool ok = active;
      for (uint32_t n = 0; ok; ++n) {
        const uint32_t slot = n % K::kQueue;
        g.some = walk.next(p, g) ? 1 : 0;
        if (n >= K::kQueue)
          ok = tc::wait_or_abort(heard(slot), (n / K::kQueue - 1) & 1u, p.timeout_ns, abort_flag);
        if (!ok) break;
        const uint4* from = reinterpret_cast<const uint4*>(&g);
#pragma unroll
        for (int k = 0; k < 4; ++k) tc::sts128(base + K::kOffQueue + slot * 64 + 16 * k, from[k]);
        mbar_arrive(told(slot));
        if (!g.some) break;
        if (n == 0)
          cut.state = (g.ja > 0 ? kPromptContinues : 0) |
                      (g.ja > 0 && g.jb == g.n ? kPromptEnds : 0);
        if (g.ja == 0 && g.jb < g.n) {  // (the last segment)
          cut.state |= kPromptBegins;
          cut.slot = 2 * c + (n > 0 ? 1 : 0);
          cut.s = g.s;
          cut.h = g.h;
          cut.i = g.i;
        }
      }
      p.cuts[c] = cut;
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 20) {
    if (active) {
      // ---------------- softmax: one query row per thread ----------------
      const int X = warp >= 12 ? 1 : 0, quarter = warp & 3, hp = (warp >> 2 & 1) ^ 1;
      const int r = quarter * 32 + lane;
      const uint32_t trow = tmem + (uint32_t(quarter * 32) << 16);
      // this thread's half of the scores, of P and of O
      const uint32_t ts = trow + K::kColS + X * K::kKeys + hp * (K::kKeys / 2);
      const uint32_t tp = trow + K::kColP + X * (K::kKeys / 2) + hp * (K::kKeys / 4);
      const uint32_t to = trow + K::kColO + X * D + hp * (D / 2);
      const uint32_t stage = base + K::kOffOut + uint32_t(warp - 4) * 2048;
      tc::RowPair pair = {stage + lane * 8, stage + lane * 8 + (hp ? -4 : 4) * 2048,
                          1 + X * 4 + quarter};
      bool gone = false;
      const float sl = p.scale_log2;
      const int rt = r / p.g, rh = r % p.g;  // token of the tile, head of the group
      uint32_t step = 0;
      auto wait = [&](uint32_t b, uint32_t phase) {
        return __all_sync(0xffffffffu,
                          tc::poll_or_abort(b, phase & 1u, p.timeout_ns, abort_flag)) != 0;
      };
      bool ok = true, first_seg = true;
      PromptSeg g;
      while (ok && take(g, true)) {
        const int tok = g.i * per + X * p.tpt + rt;
        const bool row_ok = rt < p.tpt && tok < g.q.nq;
        // keys the row sees; rows that are not stored see what the warp's last one does, so that
        // it runs one path
        const int own = g.q.nk - g.q.nq + tok + 1;
        const bool idle = !__any_sync(0xffffffffu, row_ok);
        const int most = __reduce_max_sync(0xffffffffu, row_ok ? own : -0x7fffffff);
        const int sees = row_ok ? own : most;
        const int least = __reduce_min_sync(0xffffffffu, sees);
        PromptRow row = {-INFINITY, 0.f};
        const int je = g.end(X);
        for (int j = g.ja; j < je; ++j, ++step) {
          ok = wait(sfull(X), step);
          if (!ok) break;
          tc::fence_after_sync();
          const int vis = sees - j * K::kKeys - hp * (K::kKeys / 2);  // columns of the half seen
          const bool whole = least >= (j + 1) * K::kKeys;
          const PromptStep at = {ts, tp, to, sread(X), pdone(X), pfull(X), step, lane, j > g.ja};
          if (idle) {  // no row of this warp is stored
            ok = step == 0 || wait(pdone(X), step - 1);
            if (ok && lane == 0) {
              mbar_arrive(sread(X));
              mbar_arrive(pfull(X));
            }
          } else if (whole) {
            ok = sl < 0.f ? prompt_softmax<D, true, true>(at, sl, vis, pair, row, gone, wait)
                          : prompt_softmax<D, true, false>(at, sl, vis, pair, row, gone, wait);
          } else {
            ok = sl < 0.f ? prompt_softmax<D, false, true>(at, sl, vis, pair, row, gone, wait)
                          : prompt_softmax<D, false, false>(at, sl, vis, pair, row, gone, wait);
          }
          if (!ok) break;
        }
        if (!ok) break;
        const bool cut = g.ja > 0 || g.jb < g.n;
        const size_t rec = (size_t(2 * c + (first_seg ? 0 : 1)) * 2 + X) * K::kRows + r;
        first_seg = false;
        const float l = row.l + pair.swap(row.l, gone);
        if (gone) break;
        pair.meet();  // the places are about to hold output
        if (cut && hp == 0) reinterpret_cast<float2*>(p.part_ml)[rec] = make_float2(row.m, l);
        if (je <= g.ja) continue;  // nothing of this tile here
        // ---- the segment's end: the output, or a record ----
        ok = wait(pdone(X), step - 1);
        if (!ok) break;
        tc::fence_after_sync();
        const float inv = l > 0.f ? 1.f / l : 0.f;
        // Through shared memory, 64 bytes of each of the warp's rows at a time (chunks swizzled
        // by the row), so that four lanes store a row's 64 bytes.
        uint8_t* row_out = cut ? reinterpret_cast<uint8_t*>(p.part_o + rec * D + hp * (D / 2))
                               : reinterpret_cast<uint8_t*>(
                                     reinterpret_cast<__nv_bfloat16*>(p.out) +
                                     (long long)(g.q.q0 + tok) * p.out_stride +
                                     (long long)(g.h * p.g + rh) * D + hp * (D / 2));
        if (!row_ok) row_out = nullptr;
        int ln;  // (the lane, read anew: what is made from it holds no registers in the loop above)
        asm volatile("mov.u32 %0, %%laneid;" : "=r"(ln));
        auto put = [&](int ch, const uint4& v) {
          tc::sts128(stage + ln * 64 + ((ch ^ (ln >> 1 & 3)) << 4), v);
        };
        auto flush = [&](int at) {  // the staged bytes are bytes `at` .. `at` + 63 of the rows
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int from = 8 * k + (ln >> 2), ch = ln & 3;
            uint8_t* dst = reinterpret_cast<uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row_out), from));
            const uint4 v = lds128(stage + from * 64 + ((ch ^ (from >> 1 & 3)) << 4));
            if (dst) *reinterpret_cast<uint4*>(dst + at + ch * 16) = v;
          }
          __syncwarp();
        };
        if (!idle) {
#pragma unroll 1
          for (int c1 = 0; c1 < D / 2; c1 += 32) {
            uint32_t o[32];
            tc::tmem_ld32(to + c1, o);
            if (cut) {
#pragma unroll
              for (int half = 0; half < 2; ++half) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  put(e, make_uint4(o[16 * half + 4 * e], o[16 * half + 4 * e + 1],
                                    o[16 * half + 4 * e + 2], o[16 * half + 4 * e + 3]));
                flush((c1 + 16 * half) * 4);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  w[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * inv,
                                     __uint_as_float(o[8 * e + 2 * k + 1]) * inv);
                put(e, make_uint4(w[0], w[1], w[2], w[3]));
              }
              flush(c1 * 2);
            }
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofree(X));
      }
      if (!gone) pair.leave();
      tc::fence_before_sync();
    }
  } else {
    if (active && warp == 0) {
      // ---------------- TMA ----------------
      if (lane == 0) {
        int u = 0, qn[2] = {0, 0};
        bool ok = true;
        PromptSeg g;
        auto load_tile = [&](const CUtensorMap* map, int h, int row) {
          const int st = u % K::kStages, n = u / K::kStages;
          if (n > 0)
            ok = ok && tc::wait_or_abort(empty(st), uint32_t(n - 1) & 1u, p.timeout_ns, abort_flag);
          if (!ok) return;
          mbar_arrive_expect_tx(full(st), K::kTile);
#pragma unroll
          for (int sl = 0; sl < K::kSlabs; ++sl)
            tma_load_3d(base + K::kOffKV + st * K::kTile + sl * K::kSlab, map, full(st), sl * 64,
                        h, row);
          ++u;
        };
        while (ok && take(g, false)) {
          load_tile(&tmk, g.h, g.q.k0 + g.ja * K::kKeys);
          for (int X = 0; ok && X < 2; ++X) {
            if (!g.has(X)) continue;
            if (qn[X] > 0)
              ok = tc::wait_or_abort(qempty(X), uint32_t(qn[X] - 1) & 1u, p.timeout_ns, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(qfull(X), uint32_t(p.tpt * p.g) * D * 2);
#pragma unroll
            for (int sl = 0; sl < K::kSlabs; ++sl)
              tma_load_3d(base + K::kOffQ + X * K::kTileQ + sl * K::kSlabQ, &tmq, qfull(X), sl * 64,
                          g.h * p.g, g.q.q0 + g.i * per + X * p.tpt);
            ++qn[X];
          }
          for (int j = g.ja; ok && j < g.jb; ++j) {
            if (j > g.ja) load_tile(&tmk, g.h, g.q.k0 + j * K::kKeys);
            if (ok) load_tile(&tmv, g.h, g.q.k0 + j * K::kKeys);
          }
        }
        // every copy issued must have landed before the CTA may exit
        for (int v = max(0, u - K::kStages); v < u; ++v)
          mbar_wait_bounded(full(v % K::kStages), uint32_t(v / K::kStages) & 1u, p.timeout_ns);
        for (int X = 0; X < 2; ++X)
          if (qn[X] > 0) mbar_wait_bounded(qfull(X), uint32_t(qn[X] - 1) & 1u, p.timeout_ns);
      }
      __syncwarp();
    } else if (active && warp <= 2) {
      // ---------------- scores of tile X ----------------
      if (lane == 0) {
        const int X = warp - 1;
        constexpr uint32_t kId = tc::idesc_bf16<128, K::kKeys, false>();
        const uint64_t desc_q = tc::sdesc_sw128(base + K::kOffQ + X * K::kTileQ, 16, 1024);
        const uint64_t desc_k = tc::sdesc_sw128(base + K::kOffKV, 16, 1024);
        const uint32_t ts = tmem + K::kColS + X * K::kKeys;
        bool ok = true;
        auto wait = [&](uint32_t b, uint32_t phase) {
          ok = ok && tc::poll_or_abort(b, phase & 1u, p.timeout_ns, abort_flag);
        };
        int st = 0;  // the ring's even stages hold K tiles
        uint32_t turn = 0, n = 0, segs = 0;
        PromptSeg g;
        while (ok && take(g, false)) {
          const int je = g.end(X);
          if (g.ja < je) wait(qfull(X), segs++);
          for (int j = g.ja; ok && j < g.jb; ++j) {
            wait(full(st), turn);
            if (j < je) {
              if (n++ > 0) wait(sread(X), n - 2);  // the scores before have been read
              if (!ok) break;
              tc::fence_after_sync();
              const uint64_t kd = desc_k + uint64_t(st) * (K::kTile >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_bf16(ts, desc_q + (kk >> 2) * (K::kSlabQ >> 4) + (kk & 3) * 2,
                             kd + (kk >> 2) * (K::kSlab >> 4) + (kk & 3) * 2, kId,
                             kk > 0 ? 1u : 0u);
              tc::commit(sfull(X));
              tc::commit(empty(st));
              if (j == je - 1) tc::commit(qempty(X));
            } else if (ok) {  // not used (and not let go before it is there)
              mbar_arrive(empty(st));
            }
            if ((st += 2) == K::kStages) {
              st = 0;
              turn ^= 1u;
            }
          }
        }
        tc::commit(mdone(warp - 1));  // every MMA issued must have completed before TMEM is freed
        mbar_wait_bounded(mdone(warp - 1), 0u, p.timeout_ns);
      }
      __syncwarp();
    } else if (active) {
      // ---------------- P.V of tile X ----------------
      const int X = warp == 3 ? 0 : 1;
      constexpr uint32_t kId = tc::idesc_bf16<128, D, true>();
      const uint64_t desc_v = tc::sdesc_sw128(base + K::kOffKV, K::kSlab, 1024);
      const uint32_t tp = tmem + K::kColP + X * (K::kKeys / 2);
      const uint32_t to = tmem + K::kColO + X * D;
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t phase) {  // by the first lane, for the warp
        ok = ok && (lane != 0 || tc::poll_or_abort(b, phase & 1u, p.timeout_ns, abort_flag));
        ok = __shfl_sync(0xffffffffu, int(ok), 0) != 0;
      };
      int st = 1;  // the ring's odd stages hold V tiles
      uint32_t turn = 0, n = 0, segs = 0;
      PromptSeg g;
      while (ok && take(g, true)) {
        const int je = g.end(X);
        for (int j = g.ja; ok && j < g.jb; ++j) {
          wait(full(st), turn);
          if (!ok) break;
          if (j < je) {
            const int r0 = g.q.nk - j * K::kKeys;  // rows of the sequence
            if (r0 < K::kKeys) {
              const uint32_t vb = base + K::kOffKV + st * K::kTile + r0 * 128;
              for (int k = lane; k < (K::kKeys - r0) * 8; k += 32)  // whole rows, swizzled or not
#pragma unroll
                for (int sl = 0; sl < K::kSlabs; ++sl)
                  tc::sts128(vb + sl * K::kSlab + k * 16, make_uint4(0u, 0u, 0u, 0u));
              fence_proxy_async_smem();  // before the MMAs read them
              __syncwarp();
            }
            if (j == g.ja && segs++ > 0) wait(ofree(X), segs - 2);
            wait(pfull(X), n++);
            if (!ok) break;
            if (lane == 0) {
              tc::fence_after_sync();
              const uint64_t vd = desc_v + uint64_t(st) * (K::kTile >> 4);
#pragma unroll
              for (int kk = 0; kk < K::kKeys / 16; ++kk)
                tc::mma_bf16_tmem_a(to, tp + kk * 8, vd + kk * 128, kId,
                                    (j > g.ja || kk > 0) ? 1u : 0u);
              tc::commit(pdone(X));
              tc::commit(empty(st));
            }
            __syncwarp();
          } else if (lane == 0) {
            mbar_arrive(empty(st));
          }
          if ((st += 2) > K::kStages) {
            st = 1;
            turn ^= 1u;
          }
        }
      }
      if (lane == 0) {
        tc::commit(mdone(2 + X));
        mbar_wait_bounded(mdone(2 + X), 0u, p.timeout_ns);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (*abort_flag && tid == 0 && p.status) atomicOr(p.status, PKV_DEV_TIMEOUT);
  if (warp == 1) {
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

}  // namespace pkv
