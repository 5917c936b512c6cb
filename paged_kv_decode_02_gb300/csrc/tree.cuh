// tree.cuh -- attention of a tree of drafted tokens over the paged cache, on the
// fifth-generation tensor cores (instantiated per KV dtype in tree_bf16.cu, tree_int8.cu,
// tree_e4m3.cu and tree_e5m2.cu).
//
// The last t cached tokens of a sequence are the nodes of a tree ("推测解码", chenk.top page, with
// several candidates per position); node i sees every token before them and the nodes whose
// bits its mask has set:
//   out[i, h] = softmax(scale * K q[i, h]) V over those tokens, reached through the block table.
// The context's bytes, which every row of a head shares, are the floor; more than 128 rows per
// head, and more than 64 over one-byte caches (fewer: decode_tc.cuh, chosen in api.cu), are bound
// by what is done with a tile on chip.
//
// Work. A query row is (node, head of the group); tpt = 128 / g nodes make a tile of 128 MMA
// rows (g > 128: the group is cut into equal parts first). The context is walked in key tiles of
// 64 tokens, by two pipelines X = 0 and 1. An item is one KV head with either two row tiles, one
// per pipeline, that share each key tile, or, where only one is left, that row tile in both
// pipelines, which take the even and the odd key tiles; their states meet at its end. (One
// pipeline alone waits for itself: scores, softmax, P.V in turn.) Items lie on a line, each as
// long as its context plus a constant, and every CTA takes an equal stretch of it; an item cut
// between stretches leaves records (o, m, l) that a second kernel joins, as in the prompt
// attention (prompt.cuh), whose pipelines these are:
//   warp 0       TMA: the blocks of K and V tiles (lane b block b), ids read a tile ahead, and the
//                query rows;
//   warps 1, 2   S_X = Q_X K_j^T; warps 3, 20: O_X += P_X V_j (bf16 caches: after zeroing V rows
//                past the context, which may hold anything);
//   warps 4..11, 12..19  softmax of pipeline 0, 1 and the end of each segment: two threads per
//                query row, each with half of a key tile's columns, and of O's;
//   warp 21      walks the stretch and tells the others its segments;
//   warps 22..27 (one-byte caches) widen codes in shared memory, three warps a tile, one trio the
//                K tiles, one the V tiles (so that one's waits pass while the other works).
// One-byte caches: codes land in a ring of their own and become fp16 exactly, K and V; K's scale
// multiplies the fp32 score, V's scale the weight (tcgen05.cuh: kLift16). Q is fp16 too: a row's bf16
// values times the power of two that takes its largest to [2^14, 2^15), which loses nothing of a value
// within 2^-28 of the largest and 2^-39 of the largest below; the row's scale takes the power back.
// Weights are rounded once, to bf16 (fp16 over one-byte caches), scores, maxima and sums are fp32; the
// reference maximum moves when a tile's exceeds it by more than 8 (log2 units). Results are within
// 0.0020 to 0.0024 (bf16) and 0.0017 (one-byte) of those in 64 bits, of which the rounding of the
// output makes 0.0017; bf16 weights as two terms, with a second P.V, would leave only that and cost 10
// to 15 % (64 x 1733, trees of 60: 151 -> 169 us), so they are one, as in the multi-query decode.
// Measured on GB300, whole calls: 64 x 1733 tokens, 60 nodes, 32 / 8 heads, bf16 151 us (2400 to
// 2900 cycles per key tile of two row tiles, of which the MMAs take 1300: scores, softmax and P.V
// of a tile wait for each other, and an item's end takes some 8000; 36 to 60 bytes of registers are
// spilled), INT8 209; 16 x 8192, INT8 204 (3500 cycles: the widening and 16 softmax warps share the
// issue slots; with fp16 values of code x scale, which V rows of some sizes do not survive, 195, and
// without widening 170); 1 x 131071, 33 nodes, E4M3 184. The roles' loops are kept small: with the
// widening unrolled the kernel waited for instructions (4 of 12 warps per issue: 248 for 215), and with
// a second way to the reference for tiles whose V scales are alike it took 208 for 204. Slower: four V
// and two K warps (INT8 205 -> 221), converters on low warps (207 -> 221), lighter polling (205 -> 212:
// the barriers' unit is shared), both pipelines at a split item's end (bf16 129 -> 135).
// Every wait is bounded: on a timeout the CTA sets a status bit, lets its copies and MMAs
// complete, frees its TMEM and leaves.
#pragma once

#include "decode.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace pkv {

template <int D, int BS, int CODE>
struct TreeCfg {
  static constexpr bool kQ8 = CODE >= 0;
  static constexpr int kKeys = 64;
  static constexpr int kBlocks = kKeys / BS;     // blocks per key tile
  static constexpr int kSlabs = D / 64;          // 128-byte column slabs of a 16-bit row
  static constexpr int kSlabQ = 128 * 128;
  static constexpr int kTileQ = kSlabs * kSlabQ;
  static constexpr int kSlab = kKeys * 128;
  static constexpr int kTile = kSlabs * kSlab;   // a K or V tile, 16 bits
  static constexpr int kStages = kQ8 ? 4 : 6;    // of the ring K, V, K, V, ...
  static constexpr int kCodes = kKeys * D;       // a tile of codes
  static constexpr int kCodeStages = kQ8 ? 6 : 0;
  // key tile n: slot n % 16, K scales, V scales and V scales' exponents (value_log)
  static constexpr int kScaleSlots = kQ8 ? 16 : 0;
  static constexpr int kSlot = 3 * kKeys * 4;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileQ;
  static constexpr int kOffCodes = kOffKV + kStages * kTile;
  static constexpr int kOffOut = kOffCodes + kCodeStages * kCodes;  // 32 rows of 64 bytes a warp
  static constexpr int kOffScales = kOffOut + 16 * 2048;
  // (m, l) of pipeline 1's rows of a split item, for pipeline 0: [128]
  static constexpr int kOffState = kOffScales + kScaleSlots * kSlot;
  static constexpr int kQueue = 4;
  static constexpr int kOffQueue = kOffState + 128 * 8;
  static constexpr int kOffBar = kOffQueue + kQueue * 64;
  // full[stages] empty[stages] cfull[codes] cempty[codes] qfull[2] qempty[2] sfull[2] sread[2]
  // pfull[2] pdone[2] ofree[2] mdone[4] qland[2] told[queue] heard[queue] sgiven
  static constexpr int kNumBars = 2 * kStages + 2 * kCodeStages + 21 + 2 * kQueue;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmemSlot + 4;
  static constexpr int kOffScan = (kOffAbort + 4 + 15) / 16 * 16;
  static constexpr int kSmem = kOffScan + 272 + 1024;
  static constexpr int kConvWarps = kQ8 ? 6 : 0;
  static constexpr int kThreads = (22 + kConvWarps) * 32;
  static constexpr int kListeners = 21 + kConvWarps;  // warps that hear of segments
  static constexpr int kColS = 0, kColP = 2 * kKeys, kColO = 3 * kKeys;
  static_assert(kColO + 2 * D <= 512, "TMEM columns");
  static_assert(kStages % 2 == 0 && kCodeStages % 2 == 0, "K tiles on even stages");
  static_assert(kOffCodes % 1024 == 0 && kOffOut % 1024 == 0, "swizzle atoms");
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// A sequence: its context, its tree, and its items.
struct TreeSeq {
  int len, nodes, tiles;  // row tiles
  __device__ __forceinline__ void load(const TreeParams& p, int s) {
    len = min(max(__ldg(p.context_lens + s), 0), p.MBS * p.BS);
    nodes = p.tree_lens ? min(max(__ldg(p.tree_lens + s), 0), p.q_len) : p.q_len;
    nodes = min(nodes, len);
    tiles = (nodes + p.tpt - 1) / p.tpt;
  }
  __device__ __forceinline__ int items(const TreeParams& p) const {
    return p.HV * ((tiles + 1) >> 1);  // (none: no nodes, the rows are zeros)
  }
  __device__ __forceinline__ long long length(const TreeParams& p) const {
    return (long long)items(p) * (len + p.item_cost);
  }
};

// What a CTA does of one item: key tiles [ja, jb) of n.
struct alignas(16) TreeSeg {
  int s, hv, row0, ja;   // row0: first node of tile 0
  int jb, n, len, nodes;
  int split;             // 1: one row tile, pipeline X takes the key tiles of parity X
  int some;              // 0: there is none, the stretch is over
  int pad[6];
  __device__ __forceinline__ bool uses(int X, int j) const { return !split || (j & 1) == X; }
  // key tiles of pipeline X in the segment
  __device__ __forceinline__ int count(int X) const {
    return split ? (jb + 1 - X) / 2 - (ja + 1 - X) / 2 : jb - ja;
  }
  __device__ __forceinline__ int first(int X) const {
    return split ? ja + ((ja ^ X) & 1) : ja;
  }
};
static_assert(sizeof(TreeSeg) == 64, "a place in the queue");

struct TreePlace {
  int s, u, j;  // sequence, item of the sequence, key tile
};

// Unnormalised state of a row in one pipeline.
struct TreeRow {
  float m, l;
};

struct TreeStep {
  uint32_t ts, tp, to, sread, pdone, pfull, step;
  int lane;
  bool begun;
};

// Half a row (a thread) of a score tile: 32 scores become weights 2^(scale s - m) (one-byte caches:
// times 2^kLift16 and V scales; `scales`: this half's in the tile's slot), 16-bit pairs in P's columns.
// kWhole: the row sees all columns, else those whose bits are set in `seen`;
// sl >= 0 (the scores' MMA has changed sign for a negative scale).
template <int D, int CODE, bool kWhole, typename Wait>
__device__ __forceinline__ bool tree_softmax(const TreeStep& at, float sl, uint32_t scales,
                                             uint32_t seen, tc::RowPair& pair, TreeRow& row,
                                             bool& gone, const Wait& wait) {
  constexpr bool kQ8 = CODE >= 0;
  constexpr uint32_t kV = TreeCfg<D, 16, CODE>::kKeys * 4;  // bytes from K scales to V scales
  auto pair_of = [](uint32_t a, uint32_t b) {
    return make_float2(__uint_as_float(a), __uint_as_float(b));
  };
  const float2 sl2 = make_float2(sl, sl);
  uint32_t s[32];
  tc::tmem_ld32(at.ts, s);
  tc::fence_before_sync();
  __syncwarp();
  if (at.lane == 0) mbar_arrive(at.sread);  // the next scores may come
  if constexpr (kQ8) {  // each column times its K scale
#pragma unroll
    for (int t = 0; t < 32; t += 4) {
      const uint4 k4 = lds128(scales + 4 * t);
      const float2 a = __fmul2_rn(pair_of(s[t], s[t + 1]), pair_of(k4.x, k4.y));
      const float2 b = __fmul2_rn(pair_of(s[t + 2], s[t + 3]), pair_of(k4.z, k4.w));
      s[t] = __float_as_uint(a.x);
      s[t + 1] = __float_as_uint(a.y);
      s[t + 2] = __float_as_uint(b.x);
      s[t + 3] = __float_as_uint(b.y);
    }
  }
  if constexpr (!kWhole) {
#pragma unroll
    for (int t = 0; t < 32; ++t)
      if (!(seen >> t & 1u)) s[t] = 0xff800000u;  // -inf
  }
  float mx[4], mine;
  if constexpr (kQ8) {  // the largest scaled score plus exponent of the V scale
#pragma unroll
    for (int t = 0; t < 32; t += 4) {
      const uint4 g4 = lds128(scales + 2 * kV + 4 * t);
      const float2 a = __ffma2_rn(pair_of(s[t], s[t + 1]), sl2, pair_of(g4.x, g4.y));
      const float2 b = __ffma2_rn(pair_of(s[t + 2], s[t + 3]), sl2, pair_of(g4.z, g4.w));
      const int i = t >> 1 & 2;
      mx[i] = t < 8 ? fmaxf(a.x, a.y) : fmax3(mx[i], a.x, a.y);
      mx[i + 1] = t < 8 ? fmaxf(b.x, b.y) : fmax3(mx[i + 1], b.x, b.y);
    }
    mine = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
  } else {
#pragma unroll
    for (int t = 0; t < 4; ++t) mx[t] = __uint_as_float(s[t]);
#pragma unroll
    for (int t = 0; t < 14; ++t)
      mx[t & 3] = fmax3(mx[t & 3], __uint_as_float(s[4 + 2 * t]), __uint_as_float(s[5 + 2 * t]));
    mine = sl * fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
  }
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
  const float nm = (kQ8 ? tc::kLift16 : 0.f) - m;
  const float2 nm2 = make_float2(nm, nm);
  float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  uint32_t pk[16];
#pragma unroll
  for (int t = 0; t < 32; t += 4) {
    uint4 v4;
    if constexpr (kQ8) v4 = lds128(scales + kV + 4 * t);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int u = t + 2 * i;
      const float2 x = __ffma2_rn(pair_of(s[u], s[u + 1]), sl2, nm2);
      float2 w = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      if constexpr (!kWhole) {
        w.x = seen >> u & 1u ? w.x : 0.f;
        w.y = seen >> (u + 1) & 1u ? w.y : 0.f;
      }
      ls[i] = __fadd2_rn(ls[i], w);
      if constexpr (kQ8) {
        const float2 pv = __fmul2_rn(w, i ? pair_of(v4.z, v4.w) : pair_of(v4.x, v4.y));
        pk[u / 2] = pack_f16x2(pv.x, pv.y);
      } else {
        pk[u / 2] = pack_bf16x2(w.x, w.y);
      }
    }
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
  tc::tmem_st16(at.tp, pk);
  tc::fence_before_sync();
  __syncwarp();
  if (at.lane == 0) mbar_arrive(at.pfull);
  return true;
}

// Sixteen codes -> two 16-byte chunks of fp16, exact.
template <int CODE>
__device__ __forceinline__ void widen16(const uint4& raw, uint4& a, uint4& b) {
  using Codec = Code8<CODE>;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t o[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t x = Codec::pre(w[e]);
    o[2 * e] = Codec::lo(x);
    o[2 * e + 1] = Codec::hi(x);
  }
  a = make_uint4(o[0], o[1], o[2], o[3]);
  b = make_uint4(o[4], o[5], o[6], o[7]);
}

template <int D, int BS, int CODE>
__global__ void __launch_bounds__(TreeCfg<D, BS, CODE>::kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tmq,
                          const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv, const TreeParams p) {
  using K = TreeCfg<D, BS, CODE>;
  constexpr bool kQ8 = K::kQ8;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + K::kOffAbort);
  long long* s_scan = reinterpret_cast<long long*>(gbase + K::kOffScan);  // [28] warps' sums
  TreePlace* s_place = reinterpret_cast<TreePlace*>(s_scan + 28);         // [2]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return base + K::kOffBar + 8 * i; };
  auto full = [&](int st) { return bar(st); };
  auto empty = [&](int st) { return bar(K::kStages + st); };
  auto cfull = [&](int st) { return bar(2 * K::kStages + st); };
  auto cempty = [&](int st) { return bar(2 * K::kStages + K::kCodeStages + st); };
  constexpr int kB = 2 * K::kStages + 2 * K::kCodeStages;
  auto qfull = [&](int X) { return bar(kB + X); };
  auto qempty = [&](int X) { return bar(kB + 2 + X); };
  auto sfull = [&](int X) { return bar(kB + 4 + X); };
  auto sread = [&](int X) { return bar(kB + 6 + X); };
  auto pfull = [&](int X) { return bar(kB + 8 + X); };
  auto pdone = [&](int X) { return bar(kB + 10 + X); };
  auto ofree = [&](int X) { return bar(kB + 12 + X); };
  auto mdone = [&](int i) { return bar(kB + 14 + i); };
  auto qland = [&](int X) { return bar(kB + 18 + X); };  // one-byte caches: bf16 rows are there
  auto told = [&](int i) { return bar(kB + 20 + i); };
  auto heard = [&](int i) { return bar(kB + 20 + K::kQueue + i); };
  const uint32_t sgiven = bar(kB + 20 + 2 * K::kQueue);  // pipeline 1's state is there
  const uint32_t tmem_slot = base + K::kOffTmemSlot;

  if (tid == 0) {
    for (int i = 0; i < K::kNumBars; ++i) {
      int n = 1;
      if (i < K::kStages) n = kQ8 ? 3 : 1;                   // full: a copy, or three converters
      else if (i < 2 * K::kStages) n = 2;                    // empty: both pipelines
      else if (i >= 2 * K::kStages + K::kCodeStages && i < kB) n = 3;  // cempty: three converters
      const int k = (i - kB) >> 1;
      // one per softmax warp; qfull over bf16 caches: a copy
      if (i >= kB && (k == 3 || k == 4 || k == 6 || (kQ8 && k == 0))) n = 8;
      if (i >= kB + 20 + K::kQueue) n = K::kListeners;
      if (i == kB + 20 + 2 * K::kQueue) n = 4;
      mbar_init(bar(i), n);
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
  const int chunk = (p.B + K::kThreads - 1) / K::kThreads;
  const int b0 = min(p.B, tid * chunk), b1 = min(p.B, b0 + chunk);
  long long sum = 0;
  for (int s = b0; s < b1; ++s) {
    TreeSeq q;
    q.load(p, s);
    sum += q.length(p);
  }
  long long incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  if (tid < 2) s_place[tid] = TreePlace{p.B, 0, 0};
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  long long run = incl - sum, total = 0;
  for (int w = 0; w < K::kThreads / 32; ++w) {
    if (w < warp) run += s_scan[w];
    total += s_scan[w];
  }
  const int G = int(min((long long)gridDim.x, max(1ll, total / p.min_range)));
  const int c = blockIdx.x;
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + K::kOffTmemSlot);
  if (c < G) {
    for (int e = 0; e < 2; ++e) {
      const long long x = total / G * (c + e) + total % G * (c + e) / G;
      if (x < run || x >= run + sum) continue;  // (x = total: the place past the end)
      long long r = run;
      for (int s = b0; s < b1; ++s) {
        TreeSeq q;
        q.load(p, s);
        const long long len = q.length(p);
        if (x < r + len) {
          const long long one = q.len + p.item_cost, o = (x - r) % one;
          const int n = (q.len + K::kKeys - 1) / K::kKeys;
          s_place[e] = TreePlace{s, int((x - r) / one),
                                 int(min((long long)n, (o + K::kKeys - 1) / K::kKeys))};
          break;
        }
        r += len;
      }
    }
  }
  __syncthreads();
  const bool active = c < G;
  // the next segment told, to one lane or to a whole warp; false: the stretch is over
  uint32_t heard_of = 0;
  auto take = [&](TreeSeg& g, bool whole_warp) {
    const uint32_t slot = heard_of % K::kQueue;
    bool ok = tc::poll_or_abort<true>(told(slot), (heard_of / K::kQueue) & 1u, p.timeout_ns,
                                      abort_flag);
    if (whole_warp) ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    if (!ok) return false;
    ++heard_of;
    const uint32_t from = base + K::kOffQueue + slot * 64;
    uint4* to = reinterpret_cast<uint4*>(&g);
#pragma unroll
    for (int k = 0; k < 3; ++k) to[k] = lds128(from + 16 * k);
    if (whole_warp) __syncwarp();
    if (!whole_warp || lane == 0) mbar_arrive(heard(slot));
    return g.some != 0;
  };

  if (warp == 21) {
    // ---------------- the walk ----------------
    if (lane == 0) {
      const TreePlace first = s_place[0], stop = s_place[1];
      // for the kernel that joins the records: how the first segment and the last one are cut
      TreeCut cut = {-1, 0, 0, active ? kPromptEmpty : 0};
      TreePlace at = first;
      TreeSeq q = {0, 0, 0};
      bool loaded = false, ok = active;
      for (uint32_t n = 0; ok; ++n) {
        TreeSeg g;
        g.some = 0;
        while (at.s < p.B && at.s <= stop.s) {
          if (!loaded) {
            q.load(p, at.s);
            loaded = true;
          }
          if (at.u >= q.items(p)) {
            ++at.s;
            at.u = at.j = 0;
            loaded = false;
            continue;
          }
          const bool last = at.s == stop.s && at.u == stop.u;
          if (at.s == stop.s && at.u > stop.u) break;
          const int pairs = (q.tiles + 1) >> 1;
          const int pr = at.u % pairs;
          g.s = at.s;
          g.hv = at.u / pairs;
          g.row0 = 2 * pr * p.tpt;
          g.n = (q.len + K::kKeys - 1) / K::kKeys;
          g.ja = at.j;
          g.jb = last ? min(stop.j, g.n) : g.n;
          g.len = q.len;
          g.nodes = q.nodes;
          g.split = 2 * pr + 1 >= q.tiles ? 1 : 0;
          at.j = 0;
          ++at.u;
          if (g.jb > g.ja) {
            g.some = 1;
            break;
          }
          if (last) break;
        }
        const uint32_t slot = n % K::kQueue;
        if (n >= K::kQueue)
          ok = tc::wait_or_abort(heard(slot), (n / K::kQueue - 1) & 1u, p.timeout_ns, abort_flag);
        if (!ok) break;
        const uint4* from = reinterpret_cast<const uint4*>(&g);
#pragma unroll
        for (int k = 0; k < 3; ++k) tc::sts128(base + K::kOffQueue + slot * 64 + 16 * k, from[k]);
        mbar_arrive(told(slot));
        if (!g.some) break;
        if (n == 0)
          cut.state = (g.ja > 0 ? kPromptContinues : 0) |
                      (g.ja > 0 && g.jb == g.n ? kPromptEnds : 0);
        if (g.ja == 0 && g.jb < g.n) {  // (the last segment)
          cut.state |= kPromptBegins;
          cut.slot = 2 * c + (n > 0 ? 1 : 0);
          cut.s = g.s;
          cut.u = at.u - 1;
        }
      }
      p.cuts[c] = cut;
    }
    __syncwarp();
  } else if (active && warp >= 4 && warp < 20) {
    // ---------------- softmax: two threads per query row ----------------
    const int X = warp >= 12 ? 1 : 0, quarter = warp & 3, hp = (warp >> 2 & 1) ^ 1;
    const int r = quarter * 32 + lane;
    const uint32_t trow = tmem + (uint32_t(quarter * 32) << 16);
    // this thread's half of the scores, of P and of O
    const uint32_t ts = trow + K::kColS + X * K::kKeys + hp * 32;
    const uint32_t tp = trow + K::kColP + X * (K::kKeys / 2) + hp * 16;
    const uint32_t to0 = trow + K::kColO + hp * (D / 2), to = to0 + X * D;
    const uint32_t stage = base + K::kOffOut + uint32_t(warp - 4) * 2048;
    tc::RowPair pair = {stage + lane * 8, stage + lane * 8 + (hp ? -4 : 4) * 2048,
                        1 + X * 4 + quarter};
    bool gone = false;
    const int rt = r / p.g, rh = r % p.g;  // node of the tile, head of the (part of the) group
    auto wait = [&](uint32_t b, uint32_t phase) {
      return __all_sync(0xffffffffu, tc::poll_or_abort<true>(b, phase & 1u, p.timeout_ns,
                                                             abort_flag)) != 0;
    };
    uint32_t step = 0, uses = 0, given = 0, tile_no = 0;
    const float scale = fabsf(p.scale_log2);
    float row_sl = scale;  // of the segment whose queries were taken last
    // One-byte caches: the segment's query rows, which have landed in this pipeline's Q buffer,
    // from bf16 to fp16 in place, each times a power of two.
    auto take_q = [&](const TreeSeg& g) -> bool {
      if (!kQ8 || g.count(X) == 0) return true;
      if (!wait(qland(X), uses++)) return false;
      int ln;
      asm volatile("mov.u32 %0, %%laneid;" : "=r"(ln));
      const int r = quarter * 32 + ln;
      const uint32_t qa = base + K::kOffQ + X * K::kTileQ + r * 128;
      constexpr int kChunks = D / 16;  // of this thread's half of the row
      auto at = [&](int k) {
        const int ch = hp * kChunks + k;
        return qa + (ch >> 3) * K::kSlabQ + (((ch & 7) ^ (r & 7)) << 4);
      };
      uint4 v[kChunks];
      uint32_t top = 0;  // the largest magnitude, as bf16 bits
#pragma unroll
      for (int k = 0; k < kChunks; ++k) v[k] = lds128(at(k));
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, w[e] >> 16 & 0x7fffu));
      }
      top = max(top, pair.swap(top, gone));
      if (gone) return false;
      // times 2^(141 - exponent field): the largest comes to [2^14, 2^15). A factor that fp32
      // holds: none for rows without a finite value above 2^-112.
      const int field = int(top >> 7);
      const bool fit = field > 15 && field < 255;
      const float f = fit ? __uint_as_float(uint32_t(268 - field) << 23) : 1.f;
      row_sl = fit ? scale * __uint_as_float(uint32_t(field - 14) << 23) : scale;
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = unpack_bf16x2(w[e]);
          o[e] = pack_f16x2(x.x * f, x.y * f);
        }
        tc::sts128(at(k), make_uint4(o[0], o[1], o[2], o[3]));
      }
      fence_proxy_async_smem();  // before the MMAs read them
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull(X));
      return true;
    };
    TreeSeg g;
    bool first_seg = true, ok = true;
    while (ok && take(g, true)) {
      ok = take_q(g);
      if (!ok) break;
      const int node = g.row0 + (g.split ? 0 : X) * p.tpt + rt;
      const bool stored = rt < p.tpt && node < p.q_len;  // a row of the output
      const bool sees = stored && node < g.nodes;
      const bool idle = !__any_sync(0xffffffffu, sees);
      const int before = g.len - g.nodes;  // tokens before the first node
      const uint32_t* mask =
          p.tree_mask + (size_t(g.s) * p.q_len + (stored ? node : 0)) * p.tree_words;
      const float sl = row_sl;
      // which of the 32 tokens from pos on this row sees
      auto bits_at = [&](int pos) -> uint32_t {
        if (!sees) return 0u;
        const int off = pos - before;  // first token as a node
        if (off <= -32) return 0xffffffffu;
        auto word = [&](int i) { return i >= 0 && i < p.tree_words ? __ldg(mask + i) : 0u; };
        const int w = off >> 5;  // (off >= -31: word -1 holds the tokens before the nodes)
        uint32_t bits = __funnelshift_r(w < 0 ? 0xffffffffu : word(w), word(w + 1), off & 31);
        const int left = g.nodes - off;  // bits past the last node are nobody's
        if (left < 32) bits &= left <= 0 ? 0u : (1u << left) - 1u;
        return bits;
      };
      TreeRow row = {-INFINITY, 0.f};
      const int j0 = g.first(X), dj = g.split ? 2 : 1;
      for (int j = j0; j < g.jb; j += dj, ++step) {
        ok = wait(sfull(X), step);
        if (!ok) break;
        tc::fence_after_sync();
        const TreeStep at = {ts, tp, to, sread(X), pdone(X), pfull(X), step, lane, j > j0};
        const uint32_t scales =
            base + K::kOffScales + ((tile_no + uint32_t(j - g.ja)) % 16u) * K::kSlot + hp * 128;
        if (idle) {  // no row of this warp sees anything
          ok = step == 0 || wait(pdone(X), step - 1);
          if (ok && lane == 0) {
            mbar_arrive(sread(X));
            mbar_arrive(pfull(X));
          }
        } else if ((j + 1) * K::kKeys <= before) {
          ok = tree_softmax<D, CODE, true>(at, sl, scales, 0u, pair, row, gone, wait);
        } else {
          const uint32_t seen = bits_at(j * K::kKeys + 32 * hp);
          ok = tree_softmax<D, CODE, false>(at, sl, scales, seen, pair, row, gone, wait);
        }
        if (!ok) break;
      }
      if (!ok) break;
      tile_no += uint32_t(g.jb - g.ja);
      row.l += pair.swap(row.l, gone);
      if (gone) break;
      pair.meet();  // the places are about to hold output
      const int mine = g.count(X), other = g.split ? g.count(1) : 0;
      if (mine > 0) ok = wait(pdone(X), step - 1);
      if (!ok) break;
      if (!sees) row = TreeRow{-INFINITY, 0.f};
      const bool cut = g.ja > 0 || g.jb < g.n;
      const size_t rec = (size_t(2 * c + (first_seg ? 0 : 1)) * 2 + (g.split ? 0 : X)) * 128 + r;
      first_seg = false;
      // ---- the segment's end: the output, or a record; of a split item by pipeline 0, once
      //      pipeline 1's state is there ----
      const uint32_t state = base + K::kOffState + r * 8;
      float f0 = 1.f, f1 = 0.f;
      if (g.split) {
        // (pipeline 1's state and O stay until pipeline 0 has read them: ofree)
        if (X == 1 && mine > 0 && hp == 0) {
          tc::sts32(state, __float_as_uint(row.m));
          tc::sts32(state + 4, __float_as_uint(row.l));
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(sgiven);
        }
        if (X == 0 && other > 0) {
          ok = wait(sgiven, given++);
          if (!ok) break;
          const TreeRow theirs = {__uint_as_float(lds32(state)), __uint_as_float(lds32(state + 4))};
          const float m = fmaxf(row.m, theirs.m);
          // (a pipeline without a tile or a sight has m = -inf and l = 0)
          f0 = row.m > -INFINITY ? fast_exp2(row.m - m) : 1.f;
          f1 = theirs.m > -INFINITY ? fast_exp2(theirs.m - m) : 1.f;
          row.l = row.l * f0 + theirs.l * f1;
          row.m = m;
        }
      }
      tc::fence_after_sync();
      if (!g.split || X == 0) {
        if (cut && hp == 0) reinterpret_cast<float2*>(p.part_ml)[rec] = make_float2(row.m, row.l);
        const float inv = row.l > 0.f ? 1.f / row.l : row.l == 0.f ? 0.f : row.l;  // (NaN stays)
        if (!cut) {
          f0 *= inv;
          f1 *= inv;
        }
        // Through shared memory, 64 bytes of each of the warp's rows at a time (chunks swizzled by
        // the row), so that four lanes store a row's 64 bytes.
        uint8_t* row_out = nullptr;
        if (stored)
          row_out = cut ? reinterpret_cast<uint8_t*>(p.part_o + rec * D + hp * (D / 2))
                        : reinterpret_cast<uint8_t*>(
                              reinterpret_cast<__nv_bfloat16*>(p.out) +
                              ((size_t(g.s) * p.q_len + node) * p.Hq + g.hv * p.g + rh) * D +
                              hp * (D / 2));
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
        if (__any_sync(0xffffffffu, stored)) {
#pragma unroll 1
          for (int c1 = 0; c1 < D / 2; c1 += 16) {
            uint32_t o[16];
            if (mine > 0) {
              tc::tmem_ld16(to + c1, o);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = sees ? __float_as_uint(__uint_as_float(o[e]) * f0) : 0u;
            if (other > 0) {
              uint32_t o1[16];
              tc::tmem_ld16(to0 + D + c1, o1);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (sees)
                  o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e])));
            }
            if (cut) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                put(e, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
              flush(c1 * 4);
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  w[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]),
                                     __uint_as_float(o[8 * e + 2 * k + 1]));
                put((c1 & 16) / 8 + e, make_uint4(w[0], w[1], w[2], w[3]));
              }
              if (c1 & 16) flush(c1 / 32 * 64);
            }
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (mine > 0 && (!g.split || X == 0)) mbar_arrive(ofree(X));
        if (other > 0 && X == 0) mbar_arrive(ofree(1));  // (read here)
      }
    }
    if (!gone) pair.leave();
    tc::fence_before_sync();
  } else if (active && warp == 0) {
    // ---------------- TMA ----------------
    const int rows_total = p.NB * p.Hkv * BS;  // a box at this row is all zero fill
    constexpr int kRing = kQ8 ? K::kCodeStages : K::kStages;
    int st = 0, u = 0;
    uint32_t turn = 0, tile_no = 0;
    uint32_t qn[2] = {0, 0};
    int q_left = 0;  // bit X: pipeline X's query rows of the segment are still to be sent for
    bool ok = true;
    TreeSeg g;
    // the query rows, as soon as the scores of the segment before have been computed (each lane's
    // look at the barrier is its own: the warp goes by all of them, or its lanes could part here)
    auto send_queries = [&] {
#pragma unroll
      for (int X = 0; X < 2; ++X) {
        if (!(q_left >> X & 1)) continue;
        if (qn[X] > 0 &&
            !__all_sync(0xffffffffu, mbar_test_wait(qempty(X), (qn[X] - 1) & 1u)))
          continue;
        const uint32_t b = kQ8 ? qland(X) : qfull(X);
        if (lane == 0) {
          mbar_arrive_expect_tx(b, uint32_t(p.tpt * p.g) * D * 2);
#pragma unroll
          for (int sl = 0; sl < K::kSlabs; ++sl)
            tma_load_3d(base + K::kOffQ + X * K::kTileQ + sl * K::kSlabQ, &tmq, b, sl * 64,
                        g.hv * p.g, g.s * p.q_len + g.row0 + (g.split ? 0 : X) * p.tpt);
        }
        __syncwarp();
        ++qn[X];
        q_left &= ~(1 << X);
      }
    };
    // waits for a barrier, or for the queries to have been sent for (bar 0), sending meanwhile
    auto wait = [&](uint32_t b, uint32_t phase) {
      uint64_t t0 = 0;
      for (uint32_t it = 1; ok; ++it) {
        if (__all_sync(0xffffffffu, b ? mbar_test_wait(b, phase & 1u) : q_left == 0)) break;
        if (q_left) send_queries();
        if ((it & 127u) == 0u) {
          const uint64_t now = global_timer_ns();
          if (t0 == 0) t0 = now;
          if (now - t0 > p.timeout_ns) *abort_flag = 1;
          ok = !__any_sync(0xffffffffu, *abort_flag != 0);
        }
      }
    };
    while (ok && take(g, true)) {
      const int h = g.hv / p.parts;
      q_left = (g.count(0) > 0 ? 1 : 0) | (g.count(1) > 0 ? 2 : 0);
      // lane b: cache row of block b of key tile j (rows_total: none)
      auto block_row = [&](int j) -> int {
        const int blk = j * K::kBlocks + lane;
        if (lane >= K::kBlocks || j >= g.jb || blk * BS >= g.len) return rows_total;
        int phys = __ldg(p.block_tables + size_t(g.s) * p.MBS + blk);
        phys = (phys < 0 || phys >= p.NB) ? 0 : phys;  // never copy outside the pool
        return (phys * p.Hkv + h) * BS;
      };
      int row = block_row(g.ja);
      for (int j = g.ja; ok && j < g.jb; ++j) {
        const int row_next = block_row(j + 1);
        const int row0 = __shfl_sync(0xffffffffu, row, 0);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t fb = kQ8 ? cfull(st) : full(st);
          if (u >= kRing) wait(kQ8 ? cempty(st) : empty(st), turn ^ 1u);
          if (!ok) break;
          const CUtensorMap* map = kv ? &tmv : &tmk;
          if constexpr (kQ8) {
            // (with the K tile the scales of both)
            if (lane == 0) mbar_arrive_expect_tx(fb, K::kCodes + (kv ? 0 : 2 * K::kKeys * 4));
            __syncwarp();
            if (lane < K::kBlocks) {
              tma_load_2d(base + K::kOffCodes + st * K::kCodes + lane * BS * D, map, fb, 0, row);
              if (kv == 0) {  // (a block past the context: zero codes, and another block's scales)
                const uint32_t sc = base + K::kOffScales + (tile_no % 16u) * K::kSlot;
                const size_t at = size_t(row == rows_total ? row0 : row);
                bulk_load(sc + lane * BS * 4, p.k_scale + at, BS * 4, fb);
                bulk_load(sc + K::kKeys * 4 + lane * BS * 4, p.v_scale + at, BS * 4, fb);
              }
            }
          } else {
            if (lane == 0) mbar_arrive_expect_tx(fb, K::kTile);
            __syncwarp();
            if (lane < K::kBlocks)
#pragma unroll
              for (int sl = 0; sl < K::kSlabs; ++sl)
                tma_load_2d(base + K::kOffKV + st * K::kTile + sl * K::kSlab + lane * BS * 128, map,
                            fb, sl * 64, row);
          }
          ++u;
          if (++st == kRing) {
            st = 0;
            turn ^= 1u;
          }
          if (q_left) send_queries();
        }
        ++tile_no;
        row = row_next;
      }
      if (q_left) wait(0u, 0u);
    }
    if (lane == 0) {  // every copy issued must have landed before the CTA may exit
      for (int v = max(0, u - kRing); v < u; ++v)
        mbar_wait_bounded(kQ8 ? cfull(v % kRing) : full(v % kRing), uint32_t(v / kRing) & 1u,
                          p.timeout_ns);
      for (int X = 0; X < 2; ++X)
        if (qn[X] > 0)
          mbar_wait_bounded(kQ8 ? qland(X) : qfull(X), (qn[X] - 1) & 1u, p.timeout_ns);
    }
    __syncwarp();
  } else if (active && (warp == 1 || warp == 2)) {
    // ---------------- scores of pipeline X ----------------
    if (lane == 0) {
      const int X = warp - 1;
      const uint32_t kId =
          (kQ8 ? tc::idesc_f16<128, K::kKeys, false>() : tc::idesc_bf16<128, K::kKeys, false>()) |
          (p.scale_log2 < 0.f ? tc::kIdescNegA : 0u);
      const uint64_t desc_q = tc::sdesc_sw128(base + K::kOffQ + X * K::kTileQ, 16, 1024);
      const uint64_t desc_k = tc::sdesc_sw128(base + K::kOffKV, 16, 1024);
      const uint32_t ts = tmem + K::kColS + X * K::kKeys;
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t phase) {
        ok = ok && tc::poll_or_abort<true>(b, phase & 1u, p.timeout_ns, abort_flag);
      };
      int st = 0;  // the ring's even stages hold K tiles
      uint32_t turn = 0, n = 0, segs = 0;
      TreeSeg g;
      while (ok && take(g, false)) {
        int left = g.count(X);
        if (left > 0) wait(qfull(X), segs++);
        for (int j = g.ja; ok && j < g.jb; ++j) {
          wait(full(st), turn);
          if (g.uses(X, j)) {
            if (n++ > 0) wait(sread(X), n - 2);  // the scores before have been read
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t kd = desc_k + uint64_t(st) * (K::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              tc::mma_bf16(ts, desc_q + (kk >> 2) * (K::kSlabQ >> 4) + (kk & 3) * 2,
                           kd + (kk >> 2) * (K::kSlab >> 4) + (kk & 3) * 2, kId, kk > 0 ? 1u : 0u);
            tc::commit(sfull(X));
            tc::commit(empty(st));
            if (--left == 0) tc::commit(qempty(X));
          } else if (ok) {  // the other pipeline's (not let go before it is there)
            mbar_arrive(empty(st));
          }
          if ((st += 2) == K::kStages) {
            st = 0;
            turn ^= 1u;
          }
        }
      }
      tc::commit(mdone(X));  // every MMA issued must have completed before TMEM is freed
      mbar_wait_bounded(mdone(X), 0u, p.timeout_ns);
    }
    __syncwarp();
  } else if (active && (warp == 3 || warp == 20)) {
    // ---------------- P.V of pipeline X ----------------
    const int X = warp == 3 ? 0 : 1;
    constexpr uint32_t kId = kQ8 ? tc::idesc_f16<128, D, true>() : tc::idesc_bf16<128, D, true>();
    const uint64_t desc_v = tc::sdesc_sw128(base + K::kOffKV, K::kSlab, 1024);
    const uint32_t tp = tmem + K::kColP + X * (K::kKeys / 2), to = tmem + K::kColO + X * D;
    bool ok = true;
    auto wait = [&](uint32_t b, uint32_t phase) {
      ok = ok && __all_sync(0xffffffffu,
                            tc::poll_or_abort<true>(b, phase & 1u, p.timeout_ns, abort_flag)) != 0;
    };
    int st = 1;  // the ring's odd stages hold V tiles
    uint32_t turn = 0, n = 0, segs = 0;
    TreeSeg g;
    while (ok && take(g, true)) {
      const int j0 = g.first(X);
      for (int j = g.ja; ok && j < g.jb; ++j) {
        wait(full(st), turn);
        if (!ok) break;
        if (g.uses(X, j)) {
          const int r0 = g.len - j * K::kKeys;  // rows of the context
          if (!kQ8 && r0 < K::kKeys) {
            const uint32_t vb = base + K::kOffKV + st * K::kTile + r0 * 128;
            for (int k = lane; k < (K::kKeys - r0) * 8; k += 32)  // whole rows, swizzled or not
#pragma unroll
              for (int sl = 0; sl < K::kSlabs; ++sl)
                tc::sts128(vb + sl * K::kSlab + k * 16, make_uint4(0u, 0u, 0u, 0u));
            fence_proxy_async_smem();  // before the MMAs read them
            __syncwarp();
          }
          if (j == j0 && segs++ > 0) wait(ofree(X), segs - 2);
          wait(pfull(X), n++);
          if (!ok) break;
          if (lane == 0) {
            tc::fence_after_sync();
            const uint64_t vd = desc_v + uint64_t(st) * (K::kTile >> 4);
#pragma unroll
            for (int kk = 0; kk < K::kKeys / 16; ++kk)
              tc::mma_bf16_tmem_a(to, tp + kk * 8, vd + kk * 128, kId,
                                  (j > j0 || kk > 0) ? 1u : 0u);
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
  } else if (kQ8 && active && warp >= 22) {
    // ---------------- converters: codes -> fp16 in the MMA's layout ----------------
    const bool kv = warp >= 25;  // V tiles
    const int ct = tid - (kv ? 25 : 22) * 32;
    constexpr int kSeg = D >= 128 ? 128 : 64;      // swizzle span of a row of codes
    constexpr int kChunks = K::kKeys * (D / 16);   // of 16 codes
    int st = kv ? 1 : 0, cst = st;  // K tiles on the rings' even stages, V tiles on the odd ones
    uint32_t turn = 0, cturn = 0, tile_no = 0;
    bool ok = true, begun = false;
    auto wait = [&](uint32_t b, uint32_t phase) {
      ok = ok && __all_sync(0xffffffffu,
                            tc::poll_or_abort<true>(b, phase & 1u, p.timeout_ns, abort_flag)) != 0;
    };
    TreeSeg g;
    while (ok && take(g, true)) {
      for (int j = g.ja; ok && j < g.jb; ++j, ++tile_no) {
        const int valid = g.len - j * K::kKeys;  // rows of the context
        wait(cfull(cst), cturn);
        if (begun) wait(empty(st), turn ^ 1u);
        if (!ok) break;
        const uint32_t codes = base + K::kOffCodes + cst * K::kCodes;
        const uint32_t tile = base + K::kOffKV + st * K::kTile;
        if (!kv && ct < K::kKeys) {  // the V scales' exponents, for the softmax
          const uint32_t vs =
              base + K::kOffScales + (tile_no % 16u) * K::kSlot + (K::kKeys + ct) * 4;
          if (ct >= valid) tc::sts32(vs, 0u);  // (past the context a scale may be anything)
          tc::sts32(vs + K::kKeys * 4,
                    __float_as_uint(value_log(ct < valid ? lds32(vs) : 0u)));
        }
        // chunk idx: columns 16 (4 slab + c) .. of row t; eight lanes take two rows' halves (D =
        // 128: different ones), which fall on different banks, codes and 16-bit chunks alike.
        // (Not unrolled: the kernel's roles run side by side, and their loops are to stay in the
        // SM's instruction caches.)
#pragma unroll 1
        for (int idx = ct; idx < kChunks; idx += 96) {
          const int cc = idx & 3, t = idx >> 2 & 63, slab = (idx >> 8) ^ (t & (K::kSlabs - 1));
          uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
          if (!kv || t < valid)  // (past the context a V row may be anything, its weights are 0)
            widen16<kQ8 ? CODE : 0>(
                lds128(codes + swz<kSeg>(uint32_t(t * D + (4 * slab + cc) * 16))), a, b);
          const uint32_t out = tile + slab * K::kSlab + t * 128;
          tc::sts128(out + (((2 * cc) ^ (t & 7)) << 4), a);
          tc::sts128(out + (((2 * cc + 1) ^ (t & 7)) << 4), b);
        }
        fence_proxy_async_smem();  // the 16-bit values, for the MMAs
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full(st));
          mbar_arrive(cempty(cst));
        }
        if ((st += 2) >= K::kStages) {
          st -= K::kStages;
          turn ^= 1u;
          begun = true;
        }
        if ((cst += 2) >= K::kCodeStages) {
          cst -= K::kCodeStages;
          cturn ^= 1u;
        }
      }
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

template <int CODE>
bool select_tree_code(int D, int BS, TreeKernelInfo* info) {
#define PKV_TREE(DD, BB)                                                                    \
  if (D == DD && BS == BB) {                                                                \
    info->fn = reinterpret_cast<const void*>(&tree_attention_kernel<DD, BB, CODE>);         \
    info->threads = TreeCfg<DD, BB, CODE>::kThreads;                                        \
    info->smem = TreeCfg<DD, BB, CODE>::kSmem;                                              \
    return true;                                                                            \
  }
  PKV_TREE(128, 16)
  PKV_TREE(128, 32)
  PKV_TREE(64, 16)
  PKV_TREE(64, 32)
#undef PKV_TREE
  return false;
}

}  // namespace pkv
