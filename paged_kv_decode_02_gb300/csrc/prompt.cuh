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
// of one KV head: 2 tpt consecutive tokens; its keys are walked in tiles of 128. The items of
// all sequences and heads lie on one line on which an item takes as many positions as its
// last token sees keys, plus a constant for its end, and each CTA takes an equal stretch of it:
// stretches are cut between key tiles, an item that is cut leaves unnormalised records
// (o, m, l), at most two per CTA, that a second kernel joins. So one long prompt and many
// short ones fill the SMs alike, without host knowledge of the lengths, and no order of
// atomics touches a result.
//
// A CTA (384 threads) runs two score tiles against each other, so that the tensor cores work
// on one while the exponentials of the other run:
//   warp 0      TMA: Q of both tiles, K and V tiles through one ring of stages;
//   warp 1      TMEM, and one thread issues every MMA: S_X = Q_X K^T into the tile's score
//               columns, then O_X += P_X V with P_X (bf16) read from TMEM, where it lies over
//               the scores it came from;
//   warp 2      zeroes V rows past the sequence's end (they may hold anything);
//   warps 4..7  softmax of tile 0, warps 8..11 of tile 1: one query row per thread.
// Per pair of 128 x 128 tiles and D = 128 the MMAs take 4 x 512 cycles and the exponentials
// 128 per thread on four SM sub-partitions.
// The softmax keeps a reference maximum per row that moves only when a tile's maximum exceeds
// it by more than 8 (log2 units; weights then reach 2^8 and keep their relative precision), so
// O is rescaled in TMEM a few times per item at most. Scores, maxima and sums are fp32; a
// weight is rounded once to bf16 as the MMA's operand, the sum takes it before that.
// Every wait is bounded: on a timeout the CTA sets a status bit, lets its copies and MMAs
// complete, frees its TMEM and leaves.
#pragma once

#include "internal.h"
#include "tcgen05.cuh"

namespace pkv {

template <int D>
struct PromptCfg {
  static constexpr int kRows = 128;              // MMA rows of a tile
  static constexpr int kKeys = 128;              // keys per tile
  static constexpr int kSlabs = D / 64;          // 128-byte column slabs of a row
  static constexpr int kSlab = kKeys * 128;      // bytes of one slab of a tile
  static constexpr int kTile = kSlabs * kSlab;   // a Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr int kOffQ = 0;                // both tiles' queries
  static constexpr int kOffKV = 2 * kTile;       // the ring: K, V, K, V, ...
  static constexpr int kOffBar = kOffKV + kStages * kTile;
  // full[stages] empty[stages] qfull[2] qempty[2] sfull[2] pfull[2] ofull[2] ofree[2] vfix vseen
  // mdone
  static constexpr int kNumBars = 2 * kStages + 15;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffAbort = kOffTmemSlot + 4;
  static constexpr int kOffSent = kOffAbort + 4;  // copies into the ring sent for so far
  static constexpr int kOffScan = (kOffSent + 4 + 15) / 16 * 16;  // warps' sums, both ends
  static constexpr int kSmem = kOffScan + 256 + 1024;              // + alignment of the base
  static constexpr int kThreads = 384;
  static constexpr int kColS = 0, kColO = 256;   // S_X (P_X over it) and O_X, 128 columns each
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
  __device__ __forceinline__ int key_tiles(int end) const {
    return max(1, (seen(end) + 127) / 128);
  }
};

// A place on the line: key tile j of item i of KV head h of sequence s.
struct PromptPlace {
  int s, h, i, j;
};

// What a CTA does of one item: key tiles [ja, jb) of n; tile X takes those below nx[X].
struct PromptSeg {
  PromptSeq q;
  int s, h, i, ja, jb, n;
  int nx0, nx1;
  __device__ __forceinline__ int nx(int X) const { return X ? nx1 : nx0; }
  // tile X has key tiles [ja, end(X)) here
  __device__ __forceinline__ int end(int X) const { return min(jb, nx(X)); }
  __device__ __forceinline__ bool has(int X) const { return nx(X) > ja; }
};

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
      g.n = q.key_tiles(t1);
      g.ja = at.j;
      g.jb = last ? min(stop.j, g.n) : g.n;
      g.nx0 = q.key_tiles(min(q.nq, t0 + p.tpt));
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
  const int n = q.key_tiles(min(q.nq, (lo + 1) * per));
  c.j = int(min((long long)n, (x + 127) / 128));
  return c;
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
  volatile int* sent = reinterpret_cast<volatile int*>(gbase + K::kOffSent);
  long long* s_scan = reinterpret_cast<long long*>(gbase + K::kOffScan);  // [12] warps' sums
  PromptPlace* s_place = reinterpret_cast<PromptPlace*>(s_scan + 12);     // [2]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return base + K::kOffBar + 8 * i; };
  auto full = [&](int st) { return bar(st); };
  auto empty = [&](int st) { return bar(K::kStages + st); };
  constexpr int kB = 2 * K::kStages;
  auto qfull = [&](int X) { return bar(kB + X); };
  auto qempty = [&](int X) { return bar(kB + 2 + X); };
  auto sfull = [&](int X) { return bar(kB + 4 + X); };
  auto pfull = [&](int X) { return bar(kB + 6 + X); };
  auto ofull = [&](int X) { return bar(kB + 8 + X); };
  auto ofree = [&](int X) { return bar(kB + 10 + X); };
  const uint32_t vfix = bar(kB + 12), vseen = bar(kB + 13), mdone = bar(kB + 14);
  const uint32_t tmem_slot = base + K::kOffTmemSlot;

  if (tid == 0) {
    for (int i = 0; i < K::kNumBars; ++i) {
      const bool soft = i >= kB + 6 && i < kB + 8, epi = i >= kB + 10 && i < kB + 12;
      mbar_init(bar(i), soft || epi ? 4 : 1);  // pfull, ofree: one arrival per softmax warp
    }
    *abort_flag = 0;
    *sent = 0;
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
  const PromptPlace first = s_place[0], stop = s_place[1];
  PromptWalk walk;
  walk.begin(first, stop);
  if (tid == 0) {  // for the kernel that joins the records
    PromptCut cut = {-1, 0, 0, 0, 0};
    if (active) {
      PromptWalk w2 = walk;
      PromptSeg g;
      if (!w2.next(p, g)) {
        cut.state = kPromptEmpty;
      } else {
        // the first segment, and the last one (the item that holds `stop`)
        cut.state = (g.ja > 0 ? kPromptContinues : 0) | (g.ja > 0 && g.jb == g.n ? kPromptEnds : 0);
        if (g.ja == 0 && g.jb < g.n) {
          cut.state |= kPromptBegins;
          cut.slot = 2 * c;
          cut.s = g.s, cut.h = g.h, cut.i = g.i;
        } else if (stop.j > 0 && stop.s < p.B && !(g.s == stop.s && g.h == stop.h && g.i == stop.i)) {
          PromptSeq q;
          q.load(p, stop.s);
          if (stop.j < q.key_tiles(min(q.nq, (stop.i + 1) * per))) {
            cut.state |= kPromptBegins;
            cut.slot = 2 * c + 1;
            cut.s = stop.s, cut.h = stop.h, cut.i = stop.i;
          }
        }
      }
    }
    p.cuts[c] = cut;
  }

  // the softmax warps take registers over from the first warpgroup: 128 x 72 + 256 x 216 =
  // 384 x 168, what the block is launched with
  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    if (active) {
      // ---------------- softmax: one query row per thread ----------------
      const int X = warp >= 8 ? 1 : 0, quarter = warp & 3;
      const int r = quarter * 32 + lane;
      const uint32_t trow = tmem + (uint32_t(quarter * 32) << 16);
      const uint32_t ts = trow + K::kColS + X * 128, to = trow + K::kColO + X * 128;
      const float sl = p.scale_log2, asl = fabsf(sl);
      const int rt = r / p.g, rh = r % p.g;  // token of the tile, head of the group
      int step = 0;
      bool ok = true, first_seg = true;
      PromptSeg g;
      while (ok && walk.next(p, g)) {
        const int tok = g.i * per + X * p.tpt + rt;
        const bool row_ok = rt < p.tpt && tok < g.q.nq;
        const int sees = g.q.nk - g.q.nq + tok + 1;  // keys the row sees (if any)
        float m = -INFINITY, l = 0.f;
        const int je = g.end(X);
        for (int j = g.ja; j < je; ++j, ++step) {
          if (!__all_sync(0xffffffffu, tc::wait_or_abort(sfull(X), uint32_t(step) & 1u, p.timeout_ns,
                                                         abort_flag))) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          // columns this row may see in the tile; rows that are not stored follow the warp's
          // largest count, so that it runs one path
          const int vis_row = row_ok ? min(K::kKeys, sees - j * K::kKeys) : -1;
          const int vis_w = __reduce_max_sync(0xffffffffu, vis_row);
          const int vis = row_ok ? vis_row : vis_w;
          uint32_t s[K::kKeys];
          tc::tmem_ld128(ts, s);
          if (sl < 0.f) {  // a negative scale is carried by the scores' signs
  #pragma unroll
            for (int t = 0; t < K::kKeys; ++t) s[t] ^= 0x80000000u;
          }
          const bool whole = __all_sync(0xffffffffu, vis >= K::kKeys);
          if (!whole) {
  #pragma unroll
            for (int t = 0; t < K::kKeys; ++t)
              if (t >= vis) s[t] = 0xff800000u;  // -inf
          }
          float mx[8];
  #pragma unroll
          for (int t = 0; t < 8; ++t) mx[t] = __uint_as_float(s[t]);
  #pragma unroll
          for (int t = 0; t < (K::kKeys - 8) / 2; ++t)
            mx[t & 7] = fmax3(mx[t & 7], __uint_as_float(s[8 + 2 * t]), __uint_as_float(s[9 + 2 * t]));
          const float mt = asl * fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]),
                                       fmaxf(mx[6], mx[7]));
          float alpha = 1.f;
          bool rescale = false;
          if (vis > 0 && mt > m + 8.f) {
            alpha = fast_exp2(m - mt);  // 0 while the row has seen nothing
            m = mt;
            l *= alpha;
            rescale = j > g.ja;
          }
          if (__any_sync(0xffffffffu, rescale)) {  // O holds the tiles before this one
            if (!__all_sync(0xffffffffu, tc::wait_or_abort(ofull(X), uint32_t(step - 1) & 1u,
                                                           p.timeout_ns, abort_flag))) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
  #pragma unroll
            for (int c1 = 0; c1 < D; c1 += 32) {
              uint32_t o[32];
              tc::tmem_ld32(to + c1, o);
  #pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tc::tmem_st32(to + c1, o);
            }
          }
          const float2 asl2 = make_float2(asl, asl), nm2 = make_float2(-m, -m);
          float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};
  #pragma unroll
          for (int c1 = 0; c1 < K::kKeys; c1 += 64) {
            uint32_t pk[32];
  #pragma unroll
            for (int t = 0; t < 64; t += 2) {
              const int a = c1 + t;
              const float2 x = __ffma2_rn(
                  make_float2(__uint_as_float(s[a]), __uint_as_float(s[a + 1])), asl2, nm2);
              float2 w = make_float2(fast_exp2(x.x), fast_exp2(x.y));
              if (!whole) {
                w.x = a < vis ? w.x : 0.f;
                w.y = a + 1 < vis ? w.y : 0.f;
              }
              ls[(t >> 1) & 3] = __fadd2_rn(ls[(t >> 1) & 3], w);
              pk[t / 2] = pack_bf16x2(w.x, w.y);
            }
            tc::tmem_st32(ts + c1 / 2, pk);
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(pfull(X));
          const float2 l2 = __fadd2_rn(__fadd2_rn(ls[0], ls[1]), __fadd2_rn(ls[2], ls[3]));
          l += l2.x + l2.y;
        }
        if (!ok) break;
        const bool cut = g.ja > 0 || g.jb < g.n;
        const size_t rec = (size_t(2 * c + (first_seg ? 0 : 1)) * 2 + X) * K::kRows + r;
        first_seg = false;
        if (cut) reinterpret_cast<float2*>(p.part_ml)[rec] = make_float2(m, l);
        if (je <= g.ja) continue;  // nothing of this tile here
        // ---- the segment's end: the output, or a record ----
        if (!__all_sync(0xffffffffu, tc::wait_or_abort(ofull(X), uint32_t(step - 1) & 1u, p.timeout_ns,
                                                       abort_flag))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const float inv = l > 0.f ? 1.f / l : 0.f;
        __nv_bfloat16* orow = reinterpret_cast<__nv_bfloat16*>(p.out) +
                              (long long)(g.q.q0 + tok) * p.out_stride +
                              (long long)(g.h * p.g + rh) * D;
  #pragma unroll
        for (int c1 = 0; c1 < D; c1 += 32) {
          uint32_t o[32];
          __syncwarp();
          tc::tmem_ld32(to + c1, o);
          if (!row_ok) {
          } else if (cut) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + rec * D + c1);
  #pragma unroll
            for (int e = 0; e < 32; e += 4)
              dst[e / 4] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                       __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
          } else {
            uint4* dst = reinterpret_cast<uint4*>(orow + c1);
  #pragma unroll
            for (int e = 0; e < 32; e += 8)
              dst[e / 8] = make_uint4(
                  pack_bf16x2(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv),
                  pack_bf16x2(__uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv),
                  pack_bf16x2(__uint_as_float(o[e + 4]) * inv, __uint_as_float(o[e + 5]) * inv),
                  pack_bf16x2(__uint_as_float(o[e + 6]) * inv, __uint_as_float(o[e + 7]) * inv));
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(ofree(X));
      }
      tc::fence_before_sync();
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (active && warp == 0) {
      // ---------------- TMA ----------------
      if (lane == 0) {
        int u = 0, qn[2] = {0, 0};
        bool ok = true;
        PromptSeg g;
        auto load_tile = [&](const CUtensorMap* map, int h, int row) {
          const int st = u % K::kStages, n = u / K::kStages;
          if (n > 0) ok = ok && tc::wait_or_abort(empty(st), uint32_t(n - 1) & 1u, p.timeout_ns, abort_flag);
          if (!ok) return;
          mbar_arrive_expect_tx(full(st), K::kTile);
  #pragma unroll
          for (int sl = 0; sl < K::kSlabs; ++sl)
            tma_load_3d(base + K::kOffKV + st * K::kTile + sl * K::kSlab, map, full(st), sl * 64, h, row);
          ++u;
        };
        while (ok && walk.next(p, g)) {
          load_tile(&tmk, g.h, g.q.k0 + g.ja * K::kKeys);
          for (int X = 0; ok && X < 2; ++X) {
            if (!g.has(X)) continue;
            if (qn[X] > 0)
              ok = tc::wait_or_abort(qempty(X), uint32_t(qn[X] - 1) & 1u, p.timeout_ns, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(qfull(X), uint32_t(p.tpt * p.g) * D * 2);
  #pragma unroll
            for (int sl = 0; sl < K::kSlabs; ++sl)
              tma_load_3d(base + K::kOffQ + X * K::kTile + sl * K::kSlab, &tmq, qfull(X), sl * 64,
                          g.h * p.g, g.q.q0 + g.i * per + X * p.tpt);
            ++qn[X];
          }
          for (int j = g.ja; ok && j < g.jb; ++j) {
            if (j > g.ja) load_tile(&tmk, g.h, g.q.k0 + j * K::kKeys);
            if (ok) load_tile(&tmv, g.h, g.q.k0 + j * K::kKeys);
          *sent = u;
          }
        }
        // every copy issued must have landed before the CTA may exit
        for (int v = max(0, u - K::kStages); v < u; ++v)
          mbar_wait_bounded(full(v % K::kStages), uint32_t(v / K::kStages) & 1u, p.timeout_ns);
        for (int X = 0; X < 2; ++X)
          if (qn[X] > 0) mbar_wait_bounded(qfull(X), uint32_t(qn[X] - 1) & 1u, p.timeout_ns);
      }
      __syncwarp();
    } else if (active && warp == 1) {
      // ---------------- MMA issuer ----------------
      if (lane == 0) {
        constexpr uint32_t kIdS = tc::idesc_bf16<128, K::kKeys, false>();
        constexpr uint32_t kIdO = tc::idesc_bf16<128, D, true>();
        constexpr uint32_t kTileDesc = K::kTile >> 4, kSlabDesc = K::kSlab >> 4;
        const uint64_t desc_q = tc::sdesc_sw128(base + K::kOffQ, 16, 1024);
        const uint64_t desc_k = tc::sdesc_sw128(base + K::kOffKV, 16, 1024);
        const uint64_t desc_v = tc::sdesc_sw128(base + K::kOffKV, K::kSlab, 1024);
        int steps[2] = {0, 0};   // P.V issued per tile
        int uses[2] = {0, 0};    // segments begun per tile (queries loaded)
        int opened[2] = {0, 0};  // segments whose first P.V was issued
        int fixes = 0;           // V tiles with zeroed rows so far
        bool ok = true;
        auto wait = [&](uint32_t b, int phase) {
          ok = ok && tc::wait_or_abort(b, uint32_t(phase) & 1u, p.timeout_ns, abort_flag);
        };
        // S_X of key tile j of segment g, whose K is ring load u
        auto issue_s = [&](int X, const PromptSeg& g, int j, int u, bool last_user) {
          const int st = u % K::kStages;
          if (j == g.ja) wait(qfull(X), uses[X]++);
          wait(full(st), u / K::kStages);
          if (!ok) return;
          tc::fence_after_sync();
          const uint64_t qd = desc_q + X * kTileDesc, kd = desc_k + uint64_t(st) * kTileDesc;
  #pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t ko = (kk >> 2) * kSlabDesc + (kk & 3) * 2;
            tc::mma_bf16(tmem + K::kColS + X * 128, qd + ko, kd + ko, kIdS, kk > 0 ? 1u : 0u);
          }
          tc::commit(sfull(X));
          if (j == g.end(X) - 1) tc::commit(qempty(X));
          if (last_user) tc::commit(empty(st));
        };
        auto issue_pv = [&](int X, const PromptSeg& g, int j, int u, bool last_user) {
          const int st = u % K::kStages;
          wait(full(st), u / K::kStages);
          if ((j + 1) * K::kKeys > g.q.nk) {
            wait(vfix, fixes);
            if (ok && last_user) mbar_arrive(vseen);
          }
          wait(pfull(X), steps[X]);
          if (j == g.ja && opened[X]++ > 0) wait(ofree(X), opened[X] - 2);
          if (!ok) return;
          tc::fence_after_sync();
          const uint64_t vd = desc_v + uint64_t(st) * kTileDesc;
  #pragma unroll
          for (int kk = 0; kk < K::kKeys / 16; ++kk)
            tc::mma_bf16_tmem_a(tmem + K::kColO + X * 128, tmem + K::kColS + X * 128 + kk * 8,
                                vd + kk * 128, kIdO, (j > g.ja || kk > 0) ? 1u : 0u);
          tc::commit(ofull(X));
          if (last_user) tc::commit(empty(st));
          ++steps[X];
        };
        PromptSeg g, nx;
        int u = 0;  // ring load of the segment's first K
        bool have = walk.next(p, g);
        if (have)
          for (int X = 0; ok && X < 2; ++X)
            if (g.has(X)) issue_s(X, g, g.ja, 0, X == (g.nx1 > 0 ? 1 : 0));
        while (ok && have) {
          const bool more = walk.next(p, nx);
          const int next_u = u + 2 * (g.jb - g.ja);
          const int lastX = g.nx1 > 0 ? 1 : 0;
          for (int j = g.ja; ok && j < g.jb; ++j) {
            for (int X = 0; ok && X < 2; ++X) {
              if (j < g.nx(X)) issue_pv(X, g, j, u + 2 * (j - g.ja) + 1, X == lastX);
              if (!ok) break;
              if (j + 1 < g.end(X)) issue_s(X, g, j + 1, u + 2 * (j + 1 - g.ja), X == lastX);
              else if (j == g.jb - 1 && more && nx.has(X))
                issue_s(X, nx, nx.ja, next_u, X == (nx.nx1 > 0 ? 1 : 0));
            }
            if ((j + 1) * K::kKeys > g.q.nk) ++fixes;
          }
          g = nx;
          u = next_u;
          have = more;
        }
        tc::commit(mdone);  // every MMA issued must have completed before TMEM is freed
        mbar_wait_bounded(mdone, 0u, p.timeout_ns);
      }
      __syncwarp();
    } else if (active && warp == 2) {
      // ---------------- V rows past the sequence's end ----------------
      PromptSeg g;
      int u = 0, fixes = 0;
      bool ok = true;
      while (ok && walk.next(p, g)) {
        // only the last key tile of the sequence can reach past nk
        const int j = max(0, (g.q.nk + K::kKeys - 1) / K::kKeys - 1);
        if (j >= g.ja && j < g.jb && (j + 1) * K::kKeys > g.q.nk) {
          const int v = u + 2 * (j - g.ja) + 1, st = v % K::kStages;
          // Waits on a parity must not be two phases off. The stage's copy is under way (so
          // `full` is in its phase, and stays there until the MMAs have had the tile), and the
          // MMA thread has seen the last tile zeroed.
          uint64_t since = global_timer_ns();
          for (int n = *sent, last = n; n <= v && !*abort_flag; n = *sent) {
            __nanosleep(100);
            const uint64_t now = global_timer_ns();
            if (n != last) {  // the walk goes on
              last = n;
              since = now;
            } else if (now - since > p.timeout_ns) {
              *abort_flag = 1;
            }
          }
          __syncwarp();
          if (__any_sync(0xffffffffu, *abort_flag)) break;
          ok = fixes == 0 ||
               __all_sync(0xffffffffu, tc::wait_or_abort(vseen, uint32_t(fixes - 1) & 1u,
                                                         p.timeout_ns, abort_flag));
          ok = ok && __all_sync(0xffffffffu,
                                tc::wait_or_abort(full(st), uint32_t(v / K::kStages) & 1u,
                                                  p.timeout_ns, abort_flag));
          if (!ok) break;
          ++fixes;
          const uint32_t vb = base + K::kOffKV + st * K::kTile;
          const int r0 = g.q.nk - j * K::kKeys;
          for (int k = lane; k < (K::kKeys - r0) * 8; k += 32)  // whole rows: no need to unswizzle
  #pragma unroll
            for (int sl = 0; sl < K::kSlabs; ++sl)
              tc::sts128(vb + sl * K::kSlab + r0 * 128 + k * 16, make_uint4(0u, 0u, 0u, 0u));
          fence_proxy_async_smem();  // before the MMAs read them
          __syncwarp();
          if (lane == 0) mbar_arrive(vfix);
        }
        u += 2 * (g.jb - g.ja);
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

}  // namespace pkv
