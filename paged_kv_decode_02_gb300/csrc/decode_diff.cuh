// decode_diff.cuh -- single-token differential attention over the paged KV cache.
//
// Heads go in pairs (2j, 2j + 1), each pair one differential head. Query pair j reads KV
// pair p = j / g (g = Hq / Hkv); with V' = [V_2p | V_2p+1] the pair's two value rows side
// by side (2 D wide),
//   A_m = softmax(scale * K_{2p+m} q_{2j+m}),  m = 0, 1
//   o   = A_0 V' - lambda_j A_1 V',
//   out = out_scale * (o * rsqrt(mean(o^2) + eps) * w)     (or out_scale * o, no weight),
// over the sequence's cached tokens ("分页注意力", chenk.top page). As in decode.cuh every
// cached byte is read once per step and HBM bandwidth is the bound, at the same bytes as
// the plain decode.
//
// * Transposed contractions: tokens (scores) or value columns (P.V) on the M = 16 side of
//   an m16n8k16 MMA, query rows on N = 8: row 2i is the first map of the warp's query pair
//   i, row 2i + 1 the second. Four pairs fill the 8 columns, where rows on M would leave
//   half of 16 empty and double the accumulators (128 registers a lane for 2 D = 256
//   columns; here 64). More pairs are more groups of 8 columns on the same K and V operands,
//   two to a warp at most. S^T = K q^T runs per K head over all 8 columns; the columns of the
//   other map are not read. The weights turn from S^T's accumulators into P^T's operand
//   by a movmatrix per 8 tokens. A pair's two maps are neighbouring columns of one lane:
//   the difference is local, the norm one reduction over 8 lanes. (Rows on M measured 499 us
//   for 355 on 128 x 8192 tokens, INT8, 32/8 heads.)
// * Work split: (sequence, unit, item) triples in one flat order, an item `kItem` tokens of
//   one KV pair, cut into G equal ranges, one per CTA. A unit is up to 16 query pairs of a
//   KV pair. The CTA's warps form streams of kRows warps (of up to 8 pairs each, reading
//   the same tiles); stream i takes items i, i + N, ... of the range with its own
//   online-softmax state and ring; at the end of a unit the streams' states fold through
//   shared memory (a unit of one item: no fold). A CTA rather than a warp owns a range
//   because a cut unit's record is 2 rows of 2 D floats per query pair: fewer, larger
//   ranges leave fewer records. A unit inside one range is finished there; a cut one
//   leaves a record per CTA, which the merge kernel (diff_merge.cu) folds.
// * Data movement: a TMA tensor copy brings 16 (or 32) tokens of both heads of a pair at
//   once (4-D map: swizzle span, token in block, block and head, half of the row). K and V
//   of an item have a barrier each: the ring's next K is requested as soon as the scores
//   are done with this one's, its V when P.V is (by the last of the stream's warps).
// * One-byte caches as in decode.cuh: codes widened exactly to fp16, the K scale on the
//   fp32 score, the V scale folded into the fp16 weight, there under a power of two that
//   follows the V scales (DiffPathQ8).
// * Measured on GB300, head_dim 128, whole calls: INT8, 128 x 8192 tokens, 32/8 heads 346 us
//   (2217 MB, 6400 GB/s); bf16, 64 ragged contexts (110943 tokens), 64/8 heads 77.5 us (457 MB,
//   5890 GB/s: some 3 us before the first tile, 7 us of merge, and the ends of units); E4M3,
//   one context of 131071, 32/8 heads 47.7 to 50 us (277 MB, 5800 to 5540 GB/s). With more than
//   4 query pairs per KV pair a one-byte cache is bound by the warps' own instructions (8 warps
//   of 255 registers per SM): 64 x 2048, 64/8 heads, blocks of 16 and 32 tokens, INT8 72.0 and
//   68.4 us (279 MB, 3870 and 4080 GB/s), E4M3 66.5 and 63.6.
#pragma once

#include "common.cuh"
#include "decode.cuh"
#include "fold.cuh"
#include "internal.h"

namespace pkv {

// L2 policy of lines that are read once: the first to go. Cached rows stream through and
// leave the L2 to the queries, records and outputs (ragged batch of 64, bf16: 83.5 -> 80.4
// us; INT8, 128 x 8192: 350.7 -> 344.0; a batch of 256 that shares 2048 of 2312 tokens, whose
// shared blocks do come from L2: 150.7 -> 152.3).
__device__ __forceinline__ uint64_t l2_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// 4-D tiled tensor copy global -> shared; completes its bytes on the mbarrier.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
      : "memory");
}

// Transposes an 8x8 matrix of 16-bit values held by the warp (lane: row lane / 4, columns
// 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// A box: kBox tokens of both heads of a pair, as the TMA lands it: [half][head][token] rows
// of kSeg bytes, swizzled. An item is kSub boxes.
template <int D, int CODE, int BOX, int SUB>
struct DiffGeom {
  static constexpr bool kQ8 = CODE >= 0;
  static constexpr int kBox = BOX, kSub = SUB, kItem = BOX * SUB;
  static constexpr int kElt = kQ8 ? 1 : 2;
  static constexpr int kRowBytes = D * kElt;
  static constexpr int kSeg = kRowBytes >= 128 ? 128 : 64;
  static constexpr int kHalves = kRowBytes / kSeg;
  static constexpr int kChunksPerSeg = kSeg / 16;
  static constexpr int kChunksPerRow = kRowBytes / 16;
  static constexpr int kBoxBytes = 2 * BOX * kRowBytes;
  static constexpr int kTile = kBoxBytes * SUB;          // K (or V) of an item
  static constexpr int kScaleBox = kQ8 ? 2 * BOX * 4 : 0;
  static constexpr int kScales = kScaleBox * SUB;
  // half a warp's state in the fold: half of o as 16-byte words per lane, and m and l
  static constexpr int kState = (D / 16 + 1) * 512;
  static_assert(kBoxBytes % 1024 == 0, "boxes must keep 1024-byte alignment");

  // The swizzle repeats every 8 rows, so the offset of a chunk is that of its row's place in
  // 8 (a lane's own, in a register) plus a constant for the rest.
  __device__ static __forceinline__ uint32_t lane_off(int row, int ci) {
    return swz<kSeg>(uint32_t(row * kSeg + ci * 16));
  }
  // t: a multiple of 8
  __device__ static constexpr uint32_t rest_off(int hd, int t, int half) {
    return uint32_t((t / BOX) * kBoxBytes + ((half * 2 + hd) * BOX + t % BOX) * kSeg);
  }
  // Swizzled byte offset of 16-byte chunk cc of token t (of the item) of pair head hd.
  __device__ static __forceinline__ uint32_t off(int hd, int t, int cc) {
    const int b = t / BOX, tb = t % BOX;
    const int half = cc / kChunksPerSeg, ci = cc % kChunksPerSeg;
    return uint32_t(b * kBoxBytes) +
           swz<kSeg>(uint32_t(((half * 2 + hd) * BOX + tb) * kSeg + ci * 16));
  }
  // Byte offset of the scale of token t of pair head hd.
  __device__ static __forceinline__ uint32_t scale_off(int hd, int t) {
    return uint32_t((t / BOX) * kScaleBox + hd * BOX * 4 + (t % BOX) * 4);
  }
};

// State of one warp. Lane (gid, cq) = (lane / 4, lane % 4) holds both maps (columns 2 cq
// and 2 cq + 1) of query pair cq: o[mt][0..1] of one value column of m-tile mt,
// o[mt][2..3] of another; m and l of the pair's maps (l summed over this lane's tokens
// only, until close()).
template <int D>
struct DiffState {
  static constexpr int kMT = 2 * D / 16;
  float o[kMT][4];
  float m0, m1, l0, l1;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kMT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  }
  __device__ __forceinline__ void scale(float a0, float a1) {
    l0 *= a0;
    l1 *= a1;
    times(0, kMT, make_float2(a0, a1));
  }
  // Tiles [t0, t1) of o times f, by map.
  __device__ __forceinline__ void times(int t0, int t1, float2 f) {
#pragma unroll
    for (int i = t0; i < t1; ++i) {
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        const float2 v = __fmul2_rn(make_float2(o[i][c], o[i][c + 1]), f);
        o[i][c] = v.x;
        o[i][c + 1] = v.y;
      }
    }
  }
  // New maxima over an item (mx: this lane's tokens): rescales the state, returns what the
  // item's scores subtract. A map without a score above -inf yet subtracts 0.
  __device__ __forceinline__ void raise(float mx0, float mx1, float& mn0, float& mn1) {
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, k));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, k));
    }
    const float p0 = m0, p1 = m1;
    m0 = fmaxf(m0, mx0);
    m1 = fmaxf(m1, mx1);
    mn0 = m0 == -INFINITY ? 0.f : m0;
    mn1 = m1 == -INFINITY ? 0.f : m1;
    // most items raise no maximum: then every factor is 1 (or the state is still 0)
    if (__any_sync(0xffffffffu, m0 != p0 || m1 != p1))
      scale(fast_exp2(p0 - mn0), fast_exp2(p1 - mn1));
  }
  __device__ __forceinline__ void close() {
#pragma unroll
    for (int k = 4; k < 32; k <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, k);
      l1 += __shfl_xor_sync(0xffffffffu, l1, k);
    }
  }
  // Half h of the state into buf, for another warp to fold in.
  __device__ __forceinline__ void put(uint8_t* buf, int h, int lane) const {
    float4* b = reinterpret_cast<float4*>(buf) + lane;
#pragma unroll
    for (int i = 0; i < kMT / 2; ++i) {
      const float* v = h ? o[kMT / 2 + i] : o[i];
      b[i * 32] = make_float4(v[0], v[1], v[2], v[3]);
    }
    if (h == 0) b[kMT / 2 * 32] = make_float4(m0, m1, l0, l1);
  }
  // Folds another warp's half h in; f: the factors of its maps, set with half 0.
  __device__ __forceinline__ void fold(const uint8_t* buf, int h, int lane, float2& f) {
    const float4* b = reinterpret_cast<const float4*>(buf) + lane;
    if (h == 0) {
      const float4 s = b[kMT / 2 * 32];
      const float n0 = fmaxf(m0, s.x), n1 = fmaxf(m1, s.y);
      const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
      f = make_float2(fast_exp2(s.x - z0), fast_exp2(s.y - z1));
      scale(fast_exp2(m0 - z0), fast_exp2(m1 - z1));
      m0 = n0;
      m1 = n1;
      l0 = fmaf(s.z, f.x, l0);
      l1 = fmaf(s.w, f.y, l1);
    }
#pragma unroll
    for (int i = 0; i < kMT / 2; ++i) {
      const float4 v = b[i * 32];
      float* d = h ? o[kMT / 2 + i] : o[i];
      const float2 lo = __ffma2_rn(make_float2(v.x, v.y), f, make_float2(d[0], d[1]));
      const float2 hi = __ffma2_rn(make_float2(v.z, v.w), f, make_float2(d[2], d[3]));
      d[0] = lo.x;
      d[1] = lo.y;
      d[2] = hi.x;
      d[3] = hi.y;
    }
  }
};

// bf16 cache. The difference of the two maps loses what they have in common, and with it
// whatever was rounded in that part; so a softmax weight enters P.V as two bf16 terms, the
// weight rounded and the rest rounded (2^-17 of it in all), on the same V operand.
template <int D, int BOX, int SUB, int NT>
struct DiffPathBf16 {
  using Geo = DiffGeom<D, -1, BOX, SUB>;
  static constexpr int kNT = NT;  // groups of 4 query pairs of the warp
  static constexpr int kKS = D / 16, kT = Geo::kItem / 16;
  static constexpr int kPer = Geo::kChunksPerSeg / 2;  // 32-byte steps of a row segment
  uint32_t qb[NT][kKS][2];
  uint32_t ko[kPer], vo[kPer];  // the lane's places in K and V tiles
  DiffState<D> st[NT];

  __device__ __forceinline__ void init(int lane) {
    const int r8 = lane & 7, mi = lane >> 3;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      ko[i] = Geo::lane_off(r8, 2 * i + (mi >> 1)) + (mi & 1) * 8 * Geo::kSeg;
      vo[i] = Geo::lane_off(r8, 2 * i + (mi & 1)) + (mi >> 1) * 8 * Geo::kSeg;
    }
  }

  // A lane's columns of a 2 D row: kRun neighbouring ones from column(k, gid), in
  // o[at(k, e)][half(k, e) * 2 + map].
  static constexpr int kRun = 1, kRuns = 2 * D / 8;
  __device__ static __forceinline__ int column(int k, int gid) { return 8 * k + gid; }
  __device__ static __forceinline__ float at(const float (&o)[2 * D / 16][4], int k, int,
                                             int map) {
    return o[k / 2][2 * (k % 2) + map];
  }
  __device__ static __forceinline__ void times(float (&d)[1], const __nv_bfloat16* w) {
    const unsigned short u = __ldg(reinterpret_cast<const unsigned short*>(w));
    d[0] *= __uint_as_float(uint32_t(u) << 16);
  }

  // q: row gid (pair gid / 2's map gid % 2) of the query rows of group g, when live.
  __device__ __forceinline__ void begin(int g, const __nv_bfloat16* q, bool live, int lane,
                                        float) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(q) + (lane & 3);
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
      qb[g][ks][0] = live ? __ldg(w + 8 * ks) : 0u;
      qb[g][ks][1] = live ? __ldg(w + 8 * ks + 4) : 0u;
    }
    st[g].clear();
  }
  __device__ __forceinline__ void close(int g) { st[g].close(); }

  // Scores of tokens 16 t + gid (x[g][t][0..1], by map) and 16 t + 8 + gid (x[g][t][2..3]) in
  // log2 units; tokens from nvalid on are -inf.
  __device__ __forceinline__ void scores(float (&x)[NT][kT][4], uint32_t sK, uint32_t,
                                         int nvalid, int lane, float scale_log2) {
    const int gid = lane >> 2;
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float a[NT][4] = {}, b[NT][4] = {};
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        uint32_t k0[4], k1[4];
        ldmatrix_x4(k0, sK + ko[ks % kPer] + Geo::rest_off(0, 16 * t, ks / kPer));
        ldmatrix_x4(k1, sK + ko[ks % kPer] + Geo::rest_off(1, 16 * t, ks / kPer));
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          mma_bf16_16816(a[g], k0, qb[g][ks][0], qb[g][ks][1]);
          mma_bf16_16816(b[g], k1, qb[g][ks][0], qb[g][ks][1]);
        }
      }
      const bool lo = 16 * t + gid < nvalid, hi = 16 * t + 8 + gid < nvalid;
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        x[g][t][0] = lo ? a[g][0] * scale_log2 : -INFINITY;
        x[g][t][1] = lo ? b[g][1] * scale_log2 : -INFINITY;
        x[g][t][2] = hi ? a[g][2] * scale_log2 : -INFINITY;
        x[g][t][3] = hi ? b[g][3] * scale_log2 : -INFINITY;
      }
    }
  }

  // mn: what the scores of each map of each group subtract.
  __device__ __forceinline__ void values(float (&x)[NT][kT][4], uint32_t sV, uint32_t, int,
                                         const float2 (&mn)[NT], int) {
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
      for (int g = 0; g < NT; ++g) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float w0 = fast_exp2(x[g][t][2 * h] - mn[g].x);
          const float w1 = fast_exp2(x[g][t][2 * h + 1] - mn[g].y);
          st[g].l0 += w0;
          st[g].l1 += w1;
          const uint32_t w = pack_bf16x2(w0, w1);
          const float2 f = unpack_bf16x2(w);
          pb[g][h] = transpose_8x8(w);
          pl[g][h] = transpose_8x8(pack_bf16x2(w0 - f.x, w1 - f.y));
        }
      }
#pragma unroll
      for (int mt = 0; mt < 2 * D / 16; ++mt) {
        uint32_t v[4];
        constexpr int kMt = D / 16;  // m-tiles of a head
        ldmatrix_x4_trans(v, sV + vo[mt % kPer] +
                                 Geo::rest_off(mt / kMt, 16 * t, mt % kMt / kPer));
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          mma_bf16_16816(st[g].o[mt], v, pb[g][0], pb[g][1]);
          mma_bf16_16816(st[g].o[mt], v, pl[g][0], pl[g][1]);
        }
      }
    }
  }
};

// One-byte codes (fp16 MMAs on exactly widened codes). A softmax weight times its token's V
// scale is rounded to fp16 (2^-11 of it; the row sums are of the unrounded weights). The
// product also carries a power of two per value head, which takes the largest V scale of the
// stream's tokens so far to 2^14 to 2^15; a larger one rescales the state, as a larger score
// does, and the unit's end undoes it. So rows of any size stay in fp16's normal numbers for
// weights down to 2^-28 of the largest, and a smaller weight is off by 2^-39 of that scale at
// most (131072 of them: by 2^-22 of the largest row). With a constant in its place (2^6, 2^8,
// 2^15) 32766 tokens 8 to 10 nats below four others lost 23 to 88 % of the output on V rows of
// absmax 1e-3 and 1e-4, and rows above 1e5 overflowed. The price, on GB300 (64 x 2048 tokens of
// head_dim 128): 64/8 heads INT8 70.7 -> 72.1 us, E4M3 66.0 -> 66.7, E5M2 61.5 -> 64.1; 128/8
// INT8 118.5 -> 122.2; 0.3 % with up to 4 query pairs, where memory is the bound.
// One fp16 term per weight, where a bf16 cache has two bf16 ones: a second term takes 64/8
// heads INT8 from 72.5 to 80.4 us and 128/8 from 123 to 138 (nothing with up to 4 query pairs
// over long contexts). What it mends, maps that cancel to 3 % of themselves, whose normed
// difference is off by 0.9 to 1.2 % (0.17 % with two terms, the output's own rounding), is
// less than what the codes have cost such a difference: 1.2 % (INT8), 4 % (E4M3), 8 % (E5M2)
// where both maps read the same K rows, 27 % and more where they do not.
template <int D, int CODE, int BOX, int SUB, int NT>
struct DiffPathQ8 {
  using Geo = DiffGeom<D, CODE, BOX, SUB>;
  static constexpr int kNT = NT;  // groups of 4 query pairs: they share each widened code
  using Codec = Code8<CODE>;
  static constexpr int kKS = D / 16, kT = Geo::kItem / 16;
  static constexpr int kQB = D / 4, kQC = kQB / 16;  // bytes of a K row each lane reads
  static constexpr int kVK = D / 32;  // 32-column steps of a head's V row
  uint32_t qb[NT][kKS][2];
  uint32_t ko[kQC], vo[kVK];  // the lane's places in K and V tiles
  float rs0[NT], rs1[NT], off0[NT], off1[NT];
  float up[2];  // each value head's power of two
  DiffState<D> st[NT];

  __device__ __forceinline__ void init(int lane) {
    const int gid = lane >> 2, cq = lane & 3;
#pragma unroll
    for (int i = 0; i < kQC; ++i) ko[i] = Geo::lane_off(gid, kQC * cq + i);
#pragma unroll
    for (int i = 0; i < kVK; ++i)
      vo[i] = Geo::lane_off(2 * cq, 2 * i + (gid >> 2)) + 4 * (gid & 3);
  }
  // the same place one row on (from an even row)
  __device__ static __forceinline__ uint32_t next_row(uint32_t at) {
    return Geo::kSeg == 128 ? (at ^ 16u) + 128u : at + 64u;
  }

  // m-tiles 2 k and 2 k + 1 (k counts over both heads): rows gid and gid + 8 hold elements
  // 32 k + 4 gid + 0..1 and + 2..3 of the 2 D row: a lane's run k is 4 neighbours.
  static constexpr int kRun = 4, kRuns = 2 * D / 32;
  __device__ static __forceinline__ int column(int k, int gid) { return 32 * k + 4 * gid; }
  __device__ static __forceinline__ float at(const float (&o)[2 * D / 16][4], int k, int e,
                                             int map) {
    return o[2 * k + e / 2][2 * (e % 2) + map];
  }
  __device__ static __forceinline__ void times(float (&d)[4], const __nv_bfloat16* w) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(w));
    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
    d[0] *= a.x;
    d[1] *= a.y;
    d[2] *= b.x;
    d[3] *= b.y;
  }

  // A larger V scale than the powers of two were made for: takes the item's largest (mx: this
  // lane's token's, by head) to 2^14 to 2^15, and the states to the new units. (At first 2^126,
  // whose inverse is a normal number too.)
  __device__ __forceinline__ void raise_v(const float (&mx)[2]) {
#pragma unroll
    for (int hd = 0; hd < 2; ++hd) {
      // (as integers: positive floats keep their order)
      const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(mx[hd]))) >> 23;
      const uint32_t old = __float_as_uint(up[hd]) >> 23, now = min(268u - e, old);
      const float f = old - now < 127u ? __uint_as_float((127u - (old - now)) << 23) : 0.f;
      up[hd] = __uint_as_float(now << 23);
#pragma unroll
      for (int g = 0; g < NT; ++g)
        st[g].times(hd * (D / 16), (hd + 1) * (D / 16), make_float2(f, f));
    }
  }
  __device__ __forceinline__ void close(int g) {
    st[g].close();
#pragma unroll
    for (int hd = 0; hd < 2; ++hd) {
      const float f = __uint_as_float((254u << 23) - __float_as_uint(up[hd]));  // 1 / up
      st[g].times(hd * (D / 16), (hd + 1) * (D / 16), make_float2(f, f));
    }
  }

  // The row is scaled by a power of two to near 2^14 (then exact in fp16 for entries above
  // 2^-28 of the largest), rs the score scale that undoes it; INT8 codes enter the score
  // MMA as code + 1152, whose 1152 * sum(q) comes off the score.
  __device__ __forceinline__ void begin(int g, const __nv_bfloat16* q, bool live, int lane,
                                        float scale_log2) {
    const int cq = lane & 3;
    const uint2* qd = reinterpret_cast<const uint2*>(q);
    float f[kKS][4], mx = 0.f;
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
      const uint2 a = live ? __ldg(qd + (kQB / 4) * cq + ks) : make_uint2(0u, 0u);
      const float2 lo = unpack_bf16x2(a.x), hi = unpack_bf16x2(a.y);
      f[ks][0] = lo.x; f[ks][1] = lo.y; f[ks][2] = hi.x; f[ks][3] = hi.y;
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(f[ks][e]));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // 2^(14 - e) for mx in [2^(e-1), 2^e), by its exponent field (at most 2^126, whose
    // inverse is a normal number too)
    const uint32_t field = min(267u - (__float_as_uint(mx) >> 23), 253u);
    const float sc = __uint_as_float(field << 23);
    const float rs = scale_log2 * __uint_as_float((254u - field) << 23);
    float t = 0.f;
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
      qb[g][ks][0] = pack_f16x2(f[ks][0] * sc, f[ks][1] * sc);
      qb[g][ks][1] = pack_f16x2(f[ks][2] * sc, f[ks][3] * sc);
      const float2 a = unpack_f16x2(qb[g][ks][0]), b = unpack_f16x2(qb[g][ks][1]);
      t += (a.x + a.y) + (b.x + b.y);
    }
    float qs = 0.f;
    if constexpr (CODE == CODE_I8) {
      t += __shfl_xor_sync(0xffffffffu, t, 1);
      t += __shfl_xor_sync(0xffffffffu, t, 2);
      qs = 1152.f * t;
    }
    // of this lane's columns: query rows 2 cq and 2 cq + 1
    rs0[g] = __shfl_sync(0xffffffffu, rs, 8 * cq);
    rs1[g] = __shfl_sync(0xffffffffu, rs, 8 * cq + 4);
    off0[g] = __shfl_sync(0xffffffffu, qs, 8 * cq);
    off1[g] = __shfl_sync(0xffffffffu, qs, 8 * cq + 4);
    up[0] = up[1] = 0x1p126f;
    st[g].clear();
  }

  __device__ __forceinline__ void scores(float (&x)[NT][kT][4], uint32_t sK, uint32_t sKs,
                                         int nvalid, int lane, float) {
    const int gid = lane >> 2;
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      float acc[NT][2][4] = {};
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
#pragma unroll
        for (int ch = 0; ch < kQC; ++ch) {
          const uint4 r0 = lds128(sK + ko[ch] + Geo::rest_off(hd, 16 * t, 0));
          const uint4 r1 = lds128(sK + ko[ch] + Geo::rest_off(hd, 16 * t + 8, 0));
          const uint32_t w0[4] = {Codec::pre(r0.x), Codec::pre(r0.y), Codec::pre(r0.z),
                                  Codec::pre(r0.w)};
          const uint32_t w1[4] = {Codec::pre(r1.x), Codec::pre(r1.y), Codec::pre(r1.z),
                                  Codec::pre(r1.w)};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int ks = 4 * ch + k;
            uint32_t a[4];
            if constexpr (CODE == CODE_I8) {
              a[0] = prmt(w0[k], 0x64646464u, 0x4140u);
              a[1] = prmt(w1[k], 0x64646464u, 0x4140u);
              a[2] = prmt(w0[k], 0x64646464u, 0x4342u);
              a[3] = prmt(w1[k], 0x64646464u, 0x4342u);
            } else {
              a[0] = Codec::lo(w0[k]);
              a[1] = Codec::lo(w1[k]);
              a[2] = Codec::hi(w0[k]);
              a[3] = Codec::hi(w1[k]);
            }
#pragma unroll
            for (int g = 0; g < NT; ++g)
              mma_f16_16816(acc[g][hd], a, qb[g][ks][0], qb[g][ks][1]);
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = 16 * t + 8 * h + gid;
        const bool ok = tok < nvalid;
        const float k0 = lds_f32(sKs + Geo::scale_off(0, tok));
        const float k1 = lds_f32(sKs + Geo::scale_off(1, tok));
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          x[g][t][2 * h] = ok ? (acc[g][0][2 * h] - off0[g]) * k0 * rs0[g] : -INFINITY;
          x[g][t][2 * h + 1] = ok ? (acc[g][1][2 * h + 1] - off1[g]) * k1 * rs1[g] : -INFINITY;
        }
      }
    }
  }

  __device__ __forceinline__ void values(float (&x)[NT][kT][4], uint32_t sV, uint32_t sVs,
                                         int nvalid, const float2 (&mn)[NT], int lane) {
    const int gid = lane >> 2;
    // V scales (past the context: 0), a token per lane, of which most items raise none
    static_assert(Geo::kItem == 32, "a token per lane");
    float mx[2];
#pragma unroll
    for (int hd = 0; hd < 2; ++hd)
      mx[hd] = lane < nvalid ? lds_f32(sVs + Geo::scale_off(hd, lane)) : 0.f;
    const bool above = fmaxf(fabsf(mx[0]) * up[0], fabsf(mx[1]) * up[1]) >= 0x1p15f;
    if (__builtin_expect(__any_sync(0xffffffffu, above), 0)) raise_v(mx);
#pragma unroll
    for (int t = 0; t < kT; ++t) {
      uint32_t pb[NT][2][2];  // each value head has its own scales
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = 16 * t + 8 * h + gid;
        const float v0 = tok < nvalid ? lds_f32(sVs + Geo::scale_off(0, tok)) * up[0] : 0.f;
        const float v1 = tok < nvalid ? lds_f32(sVs + Geo::scale_off(1, tok)) * up[1] : 0.f;
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          const float w0 = fast_exp2(x[g][t][2 * h] - mn[g].x);
          const float w1 = fast_exp2(x[g][t][2 * h + 1] - mn[g].y);
          st[g].l0 += w0;
          st[g].l1 += w1;
          pb[g][0][h] = transpose_8x8(pack_f16x2(w0 * v0, w1 * v0));
          pb[g][1][h] = transpose_8x8(pack_f16x2(w0 * v1, w1 * v1));
        }
      }
#pragma unroll
      for (int k = 0; k < 2 * kVK; ++k) {
        const int hd = k / kVK;  // tokens 16 t + 2 cq, the next, and both 8 on
        const uint32_t at = sV + vo[k % kVK], at1 = next_row(at);
        const uint32_t w0 = Codec::pre(lds32(at + Geo::rest_off(hd, 16 * t, 0)));
        const uint32_t w1 = Codec::pre(lds32(at1 + Geo::rest_off(hd, 16 * t, 0)));
        const uint32_t w2 = Codec::pre(lds32(at + Geo::rest_off(hd, 16 * t + 8, 0)));
        const uint32_t w3 = Codec::pre(lds32(at1 + Geo::rest_off(hd, 16 * t + 8, 0)));
        const uint32_t x01 = prmt(w0, w1, 0x5140u), x23 = prmt(w0, w1, 0x7362u);
        const uint32_t y01 = prmt(w2, w3, 0x5140u), y23 = prmt(w2, w3, 0x7362u);
        const uint32_t a[4] = {Codec::lo(x01), Codec::hi(x01), Codec::lo(y01), Codec::hi(y01)};
        const uint32_t b[4] = {Codec::lo(x23), Codec::hi(x23), Codec::lo(y23), Codec::hi(y23)};
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          mma_f16_16816(st[g].o[2 * k], a, pb[g][hd][0], pb[g][hd][1]);
          mma_f16_16816(st[g].o[2 * k + 1], b, pb[g][hd][0], pb[g][hd][1]);
        }
      }
    }
  }
};

// Items of sequence i: its cached tokens, clamped to its table, in runs of `item`.
__device__ __forceinline__ int diff_items(const DiffParams& p, int i, int item) {
  const int L = __ldg(p.context_lens + i);
  return (max(0, min(L, p.MBS * p.BS)) + item - 1) / item;
}

// Start of range w of G equal ranges of T positions (G <= T): floor(T w / G), with T / G
// given as q and the rest r.
__device__ __forceinline__ long long diff_start(long long q, unsigned r, unsigned w, unsigned G) {
  return q * w + r * w / G;  // r, w <= G: within 32 bits
}

// Shared memory of a CTA: the streams' rings, the fold's states, barriers and counters,
// the items' prefix.
template <class Geo, int NT, int kStreams, int kRows, int kStages>
struct DiffSmem {
  // Folds go pairwise, whole states at once, where two groups of 4 query pairs per warp leave
  // two CTAs to the SM and so the room for N / 2 states; else one after the other, a half
  // state at a time.
  static constexpr bool kTree = NT > 1 && kStreams > 2;
  static constexpr int kFold = kStreams == 1 ? 0 : kTree ? kStreams / 2 * 2 * NT : 1;  // halves
  static constexpr int kSlot = 2 * Geo::kTile;                    // K and V of an item
  static constexpr int kRing = kStages * kSlot;
  static constexpr int kOffScale = kStreams * kRing;
  static constexpr int kOffState = kOffScale + kStreams * kStages * 2 * Geo::kScales;
  static constexpr int kOffBar = kOffState + kRows * kFold * Geo::kState;
  static constexpr int kOffCnt = kOffBar + kStreams * kStages * 16;
  static constexpr int kOffPrefix = (kOffCnt + kStreams * kStages * 8 + 15) / 16 * 16;
};

template <int D, class Path, int kStreams, int kRows, int kStages, int kCtas>
__global__ void __launch_bounds__(kStreams * kRows * 32, kCtas)
    paged_diff_decode_kernel(const __grid_constant__ CUtensorMap tmk,
                             const __grid_constant__ CUtensorMap tmv, const DiffParams p) {
  using Geo = typename Path::Geo;
  using S = DiffSmem<Geo, Path::kNT, kStreams, kRows, kStages>;
  constexpr int N = kStreams, kWarps = kStreams * kRows, kThreads = kWarps * 32;
  constexpr int NT = Path::kNT;
  const int B = p.B;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (base - smem_u32(smem_raw));
  int* prefix = reinterpret_cast<int*>(gen + S::kOffPrefix);  // items before sequence s
  __shared__ int2 warp_tot[kWarps];
  __shared__ int4 bound[2];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int stream = warp / kRows, tile = warp % kRows;
  const int gid = lane >> 2, cq = lane & 3;
  auto sK = [&](int st) { return base + stream * S::kRing + st * S::kSlot; };
  auto sV = [&](int st) { return sK(st) + Geo::kTile; };
  auto sKs = [&](int st) {
    return base + S::kOffScale + (stream * kStages + st) * 2 * Geo::kScales;
  };
  auto sVs = [&](int st) { return sKs(st) + Geo::kScales; };
  auto barK = [&](int st) { return base + S::kOffBar + (stream * kStages + st) * 16; };
  auto barV = [&](int st) { return barK(st) + 8; };
  if (lane == 0 && tile == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(barK(st), 1);
      mbar_init(barV(st), 1);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  if constexpr (kRows > 1) {
    if (tid < kStreams * kStages * 2) reinterpret_cast<int*>(gen + S::kOffCnt)[tid] = 0;
  }
  pdl_wait_prior_grid();
  if (tid == 0) p.cuts[blockIdx.x] = -1;  // no unit is left to others, so far
  if (p.norm_w && tid < D / 32)  // read at the end of a unit
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p.norm_w) + tid * 128));
  if (tid < (p.P * p.g + 31) / 32)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.lam + tid * 32));

  // ---- this CTA's range and the items per sequence (every CTA computes them) ----
  // The ranges are G equal cuts of a weighted order, in which a unit takes its items and
  // then unit_cost positions that hold none: what ending it costs the CTA.
  const int U = p.P * p.nsg;  // units per sequence
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  auto weight_of = [&](int m) { return m > 0 ? m + p.unit_cost : 0; };
  int2 run = make_int2(0, 0);  // items and weight before sequence b0
  bool all_short = true;       // no unit has more items than the CTA has streams
  for (int i = b0; i < b1; ++i) {
    const int m = diff_items(p, i, Geo::kItem);
    all_short &= m <= N;
    run.x += m;
    run.y += weight_of(m);
  }
  {
    int2 incl = run;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl.x, off);
      const int y = __shfl_up_sync(0xffffffffu, incl.y, off);
      if (lane >= off) {
        incl.x += x;
        incl.y += y;
      }
    }
    if (lane == 31) warp_tot[warp] = incl;
    run = make_int2(incl.x - run.x, incl.y - run.y);
  }
  all_short = __syncthreads_and(all_short);
  int2 total = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) {
      run.x += total.x;
      run.y += total.y;
    }
    total.x += warp_tot[w].x;
    total.y += warp_tot[w].y;
  }
  const long long T = (long long)U * total.y;
  const int G = int(min((long long)gridDim.x, (T + p.min_range - 1) / p.min_range));
  if (int(blockIdx.x) >= G) return;
  const long long q0 = T < (1ll << 32) ? (long long)(unsigned(T) / unsigned(G)) : T / G;
  const unsigned rest = unsigned(T - q0 * G);
  const long long at[2] = {diff_start(q0, rest, blockIdx.x, G),
                           diff_start(q0, rest, blockIdx.x + 1, G)};
  if (tid == 0) prefix[0] = 0;
  for (int i = b0; i < b1; ++i) {
    const int m = diff_items(p, i, Geo::kItem), w = weight_of(m);
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // the thread whose sequence holds an end of the range
      const long long rem = at[e] - (long long)U * run.y;
      if (rem >= 0 && rem < (long long)U * w) bound[e] = make_int4(i, run.x, run.y, m);
    }
    run.x += m;
    run.y += w;
    prefix[i + 1] = run.x;
  }
  __syncthreads();
  // the first unit and item at or after an end, and the items before it
  auto locate = [&](int e, Cursor& c) {
    const int4 f = bound[e];
    const int w = weight_of(f.w);
    const long long rem = at[e] - (long long)U * f.z;
    c.s = f.x;
    c.n = f.w;
    c.u = rem < (1ll << 32) ? int(unsigned(rem) / unsigned(w)) : int(rem / w);
    c.j = min(c.n, int(rem - (long long)c.u * w));
    // where the streams take every unit at once, none is cut: its first item decides (4
    // sequences of ~30 tokens, head_dim 64: 8.2 -> 6.7 us; 200 of ~20: 8.8 -> 7.6)
    if (c.j > 0 && all_short) c.j = c.n;
    const long long before = (long long)U * f.y + (long long)c.u * c.n + c.j;
    if (c.j == c.n) {  // among a unit's empty positions: the next unit
      c.j = 0;
      if (++c.u == U) {
        c.u = 0;
        do { ++c.s; } while (c.s < B && prefix[c.s + 1] == prefix[c.s]);
        c.n = c.s < B ? prefix[c.s + 1] - prefix[c.s] : 0;
      }
    }
    return before;
  };
  Cursor cur;  // the segment: unit cur.u of sequence cur.s from its item cur.j on
  const long long end =
      int(blockIdx.x) + 1 == G ? (long long)U * total.x : locate(1, cur);
  const int n = int(end - locate(0, cur));
  if (n == 0) return;

  // the producer's item: number pi of the CTA's range, every N-th one is this stream's.
  // Each of the stream's warps keeps it; the last one to leave a tile requests the next.
  Cursor pc = cur;
  int pi = 0, pid[Geo::kSub], pL = 0, pLs = -1;
  auto advance = [&](int k) {
    pi += k;
    if (pi >= n) return;
    pc.j += k;
    while (pc.j >= pc.n) {
      pc.j -= pc.n;
      if (++pc.u == U) {
        pc.u = 0;
        do { ++pc.s; } while (prefix[pc.s + 1] == prefix[pc.s]);
        pc.n = prefix[pc.s + 1] - prefix[pc.s];
      }
    }
  };
  // lane 0: the physical blocks of the producer's item, read ahead of their copies
  auto fetch = [&]() {
    if (lane != 0 || pi >= n) return;
    if (pc.s != pLs) {
      pL = min(__ldg(p.context_lens + pc.s), p.MBS * p.BS);
      pLs = pc.s;
    }
#pragma unroll
    for (int k = 0; k < Geo::kSub; ++k) {
      const int t = (pc.j * Geo::kSub + k) * Geo::kBox;
      pid[k] = __ldg(p.block_tables + size_t(pc.s) * p.MBS + min(t / p.BS, p.MBS - 1));
    }
  };
  const uint64_t policy = l2_evict_first();
  // lane 0: requests K (or V) of the producer's item; boxes past the context are left out
  auto request = [&](const CUtensorMap* map, uint32_t dst, uint32_t scales, const float* scale,
                     uint32_t bar) {
    const int t0 = pc.j * Geo::kItem;
    const int boxes = min(Geo::kSub, (pL - t0 + Geo::kBox - 1) / Geo::kBox);
    mbar_arrive_expect_tx(bar, uint32_t(boxes) * (Geo::kBoxBytes + Geo::kScaleBox));
    const int head = 2 * (pc.u / p.nsg);
#pragma unroll
    for (int k = 0; k < Geo::kSub; ++k) {
      if (k >= boxes) break;
      const int in = (t0 + k * Geo::kBox) % p.BS;
      const int id = pid[k] < 0 || pid[k] >= p.NB ? 0 : pid[k];  // stay in the pool
      const int row = id * 2 * p.P + head;
      tma_load_4d(dst + k * Geo::kBoxBytes, map, bar, 0, in, row, 0, policy);
      if constexpr (Geo::kQ8)  // a box is a whole block: both heads' scales are neighbours
        bulk_load(scales + k * Geo::kScaleBox, scale + size_t(row) * Geo::kBox, Geo::kScaleBox,
                  bar);
    }
  };
  // Brings a unit's query rows near ahead of its first item: loads queue behind the copies
  // (3.5 us for the first unit's, asked for after the first copies).
  auto prefetch_q = [&](int s0, int u0) {
    const int r0 = (u0 % p.nsg) * p.gs;
    const int lines = min(p.gs, p.g - r0) * (D / 32);  // of 128 bytes: 2 rows of D a pair
    const char* rows = static_cast<const char*>(p.q) +
                       (size_t(s0) * 2 * p.P * p.g + 2 * (u0 / p.nsg * p.g + r0)) * (D * 2);
    for (int k = lane; k < lines; k += 32)
      asm volatile("prefetch.global.L1 [%0];" ::"l"(rows + k * 128));
  };
  // the warp has read its share of a tile (which: 0 K, 1 V): whether lane 0 is to refill it
  auto released = [&](int st, int which) {
    fence_proxy_async_smem();  // this lane's reads before the refill
    __syncwarp();
    if (lane != 0 || pi >= n) return false;
    if constexpr (kRows > 1) {
      int* c = reinterpret_cast<int*>(gen + S::kOffCnt) + (stream * kStages + st) * 2 + which;
      __threadfence_block();
      if ((atomicAdd(c, 1) + 1) % kRows != 0) return false;
      __threadfence_block();
    }
    return true;
  };

  if (warp == 0) prefetch_q(cur.s, cur.u);
  advance(stream);
#pragma unroll
  for (int st = 0; st < kStages; ++st) {
    fetch();
    if (tile == 0 && lane == 0 && pi < n) {
      request(&tmk, sK(st), sKs(st), p.k_scale, barK(st));
      request(&tmv, sV(st), sVs(st), p.v_scale, barV(st));
    }
    advance(N);
  }
  fetch();

  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
  const int Hq = 2 * p.P * p.g;
  Path path;
  path.init(lane);
  int st = 0;
  uint32_t par = 0;
  bool dead = false, first = true;
  for (int i = 0; i < n;) {
    const int len = min(n - i, cur.n - cur.j);
    const int pair0 = cur.u / p.nsg * p.g;                       // of the KV pair
    const int r0 = (cur.u % p.nsg) * p.gs, rows = min(p.gs, p.g - r0);  // of the unit
    // streams with items here fold into the one that takes the first item
    const int rank = (stream - i % N + N) % N, active = min(len, N);
    if (rank < active) {
#pragma unroll
      for (int g = 0; g < NT; ++g) {
        const int row = 4 * (tile * NT + g) + (gid >> 1);  // of this lane's query row
        const bool live = row < rows;
        path.begin(g, q + (size_t(cur.s) * Hq +
                           (live ? 2 * (pair0 + r0 + row) + (gid & 1) : 0)) * D,
                   live, lane, p.scale_log2);
      }
      const int L = min(__ldg(p.context_lens + cur.s), p.MBS * p.BS);
      for (int k = i + rank; k < i + len && !dead; k += N) {
        const int nvalid = L - (cur.j + k - i) * Geo::kItem;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(barK(st), par, p.timeout_ns))) {
          dead = true;
          break;
        }
        float x[NT][Path::kT][4];
        path.scores(x, sK(st), sKs(st), nvalid, lane, p.scale_log2);
        if (released(st, 0)) request(&tmk, sK(st), sKs(st), p.k_scale, barK(st));
        float2 mn[NT];
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
          for (int t = 0; t < Path::kT; ++t) {
            mx0 = fmax3(mx0, x[g][t][0], x[g][t][2]);
            mx1 = fmax3(mx1, x[g][t][1], x[g][t][3]);
          }
          path.st[g].raise(mx0, mx1, mn[g].x, mn[g].y);
        }
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(barV(st), par, p.timeout_ns))) {
          dead = true;
          break;
        }
        // rows past the context may hold anything (even NaN): zero them before P.V (every
        // warp of the stream does, before its own reads: the same zeros)
        if (nvalid < Geo::kItem) {
          for (int c = lane; c < (Geo::kItem - nvalid) * 2 * Geo::kChunksPerRow; c += 32) {
            const int t = nvalid + c / (2 * Geo::kChunksPerRow);
            const int cc = c % (2 * Geo::kChunksPerRow);
            sts128_zero(sV(st) + Geo::off(cc / Geo::kChunksPerRow, t, cc % Geo::kChunksPerRow));
          }
          __syncwarp();
        }
        path.values(x, sV(st), sVs(st), nvalid, mn, lane);
        if (released(st, 1)) request(&tmv, sV(st), sVs(st), p.v_scale, barV(st));
        const int s0 = pc.s, u0 = pc.u;
        advance(N);
        fetch();
        if (pi < n && (pc.s != s0 || pc.u != u0)) prefetch_q(pc.s, pc.u);
        if (++st == kStages) {
          st = 0;
          par ^= 1u;
        }
      }
#pragma unroll
      for (int g = 0; g < NT; ++g) path.close(g);
    }

    // ---- fold the streams' states into rank 0's ----
    uint8_t* buf = gen + S::kOffState + tile * S::kFold * Geo::kState;
    if constexpr (S::kTree) {
#pragma unroll
      for (int far = N / 2; far > 0; far >>= 1) {
        if (active <= far) continue;  // (the same for all threads, like every branch round a sync)
#pragma unroll
        for (int g = 0; g < 2 * NT; ++g)
          if (rank >= far && rank < min(2 * far, active))
            path.st[g / 2].put(buf + ((rank - far) * 2 * NT + g) * Geo::kState, g % 2, lane);
        __syncthreads();
        float2 f = make_float2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < 2 * NT; ++g)
          if (rank + far < min(2 * far, active))
            path.st[g / 2].fold(buf + (rank * 2 * NT + g) * Geo::kState, g % 2, lane, f);
        __syncthreads();  // before the next states are put there
      }
    } else if constexpr (kStreams > 1) {
      for (int r = 1; r < active; ++r) {
#pragma unroll
        for (int g = 0; g < NT; ++g) {
          float2 f = make_float2(0.f, 0.f);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (rank == r) path.st[g].put(buf, h, lane);
            __syncthreads();
            if (rank == 0) path.st[g].fold(buf, h, lane, f);
            __syncthreads();  // before the next half, or unit, is put there
          }
        }
      }
    }
    const bool whole = cur.j == 0 && len == cur.n;
    // where the merge finds the unit's records: the first's slot (-1: none, it is done
    // here) and the last's CTA; the others are the first segments of the CTAs between
    if (rank == 0 && tile == 0 && lane == 0) {
      int* part = p.parts + 2 * (size_t(cur.s) * U + cur.u);
      if (cur.j == 0) part[0] = whole ? -1 : 2 * int(blockIdx.x) + (first ? 0 : 1);
      if (cur.j == 0 && !whole)  // at most one: the range's last segment
        p.cuts[blockIdx.x] = 2 * (cur.s * U + cur.u) + (first ? 0 : 1);
      if (cur.j + len == cur.n) part[1] = int(blockIdx.x);
    }
#pragma unroll
    for (int g = 0; g < NT; ++g) {
      const int pr = 4 * (tile * NT + g) + cq;  // this lane's query pair within the unit
      if (rank != 0 || pr >= rows) continue;
      DiffState<D>& state = path.st[g];
      if (!whole) {
        const size_t slot = size_t(2) * blockIdx.x + (first ? 0 : 1);
        const size_t r = slot * 2 * p.gs + pr;
        float* o0 = p.part_o + r * (2 * D);
        float* o1 = o0 + size_t(p.gs) * (2 * D);
#pragma unroll
        for (int k = 0; k < Path::kRuns; ++k) {
          const int c = Path::column(k, gid);
          if constexpr (Path::kRun == 4) {
            float v[2][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[0][e] = Path::at(state.o, k, e, 0);
              v[1][e] = Path::at(state.o, k, e, 1);
            }
            *reinterpret_cast<float4*>(o0 + c) = make_float4(v[0][0], v[0][1], v[0][2], v[0][3]);
            *reinterpret_cast<float4*>(o1 + c) = make_float4(v[1][0], v[1][1], v[1][2], v[1][3]);
          } else {
            o0[c] = Path::at(state.o, k, 0, 0);
            o1[c] = Path::at(state.o, k, 0, 1);
          }
        }
        if (gid == 0) {
          float2* ml = reinterpret_cast<float2*>(p.part_ml);
          // NaN scores alone leave m at -inf, which the merge takes for no token: m = 0
          // keeps such a record in
          ml[r] = make_float2(isnan(state.l0) ? 0.f : state.m0, state.l0);
          ml[r + p.gs] = make_float2(isnan(state.l1) ? 0.f : state.m1, state.l1);
        }
      } else {
        const int qp = pair0 + r0 + pr;
        const float i0 = 1.f / state.l0;
        const float i1 = 1.f / state.l1 * __ldg(p.lam + qp);
        const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.norm_w);
        float ss = 0.f, d[Path::kRuns][Path::kRun];
#pragma unroll
        for (int k = 0; k < Path::kRuns; ++k) {
#pragma unroll
          for (int e = 0; e < Path::kRun; ++e) {
            d[k][e] = Path::at(state.o, k, e, 0) * i0 - Path::at(state.o, k, e, 1) * i1;
            ss = fmaf(d[k][e], d[k][e], ss);
          }
        }
        // over the 8 lanes of the pair (they branch alike)
        const uint32_t lanes = 0x11111111u << cq;
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) ss += __shfl_xor_sync(lanes, ss, k);
        float f = p.out_scale;
        if (w) {  // every weight is asked for before the first store
          f *= rsqrtf(ss * (1.f / (2 * D)) + p.eps);
#pragma unroll
          for (int k = 0; k < Path::kRuns; ++k) Path::times(d[k], w + Path::column(k, gid));
        }
        __nv_bfloat16* out =
            static_cast<__nv_bfloat16*>(p.out) + (size_t(cur.s) * (Hq / 2) + qp) * (2 * D);
#pragma unroll
        for (int k = 0; k < Path::kRuns; ++k) {
          const int c = Path::column(k, gid);
          if constexpr (Path::kRun == 4)
            *reinterpret_cast<uint2*>(out + c) = make_uint2(pack_bf16x2(d[k][0] * f, d[k][1] * f),
                                                            pack_bf16x2(d[k][2] * f, d[k][3] * f));
          else
            out[c] = __float2bfloat16(d[k][0] * f);
        }
      }
    }
    first = false;
    i += len;
    cur.j = 0;
    if (++cur.u == U) {
      cur.u = 0;
      if (i < n) {
        do { ++cur.s; } while (prefix[cur.s + 1] == prefix[cur.s]);
        cur.n = prefix[cur.s + 1] - prefix[cur.s];
      }
    }
  }
  if (dead) {
    if (lane == 0 && p.status) atomicOr(p.status, PKV_DEV_TIMEOUT);
    // let copies in flight land before the CTA's shared memory goes: at most the current
    // phase of each barrier is open (with nothing requested the wait runs out)
    for (int k = 0; k < kStages; ++k) {
      for (uint32_t p2 = 0; p2 < 2; ++p2) {
        mbar_wait_bounded(barK(k), p2, p.timeout_ns);
        mbar_wait_bounded(barV(k), p2, p.timeout_ns);
      }
    }
  }
}

template <int D, class Path, int kStreams, int kRows, int kStages, int kCtas>
DiffKernelInfo make_diff_info() {
  using S = DiffSmem<typename Path::Geo, Path::kNT, kStreams, kRows, kStages>;
  static_assert(Path::Geo::kItem >= kDiffLeastItem, "more items than the host counts with");
  DiffKernelInfo info{};
  info.fn = reinterpret_cast<const void*>(
      &paged_diff_decode_kernel<D, Path, kStreams, kRows, kStages, kCtas>);
  info.threads = kStreams * kRows * 32;
  info.smem = 1024 + S::kOffPrefix;
  // the sequences that every instance takes (pagedkv.h), 2 KiB left to static variables
  static_assert(1024 + S::kOffPrefix + 4 * (30000 + 4) + 2048 <= 227 * 1024, "batch table");
  info.box = Path::Geo::kBox;
  return info;
}

// One-byte caches, units of up to 4 query pairs: a warp per stream; up to 8: the warp takes
// both groups of 4, so that a code is widened once for both; up to 16: two such warps.
template <int D, int CODE, int BOX, int SUB>
DiffKernelInfo diff_shape_q8(int pairs) {
  constexpr int kS = D == 128 ? 1 : 2;  // items of 16 or 8 KiB
  if (pairs <= 4) return make_diff_info<D, DiffPathQ8<D, CODE, BOX, SUB, 1>, 4, 1, kS, 3>();
  if (pairs <= 8) return make_diff_info<D, DiffPathQ8<D, CODE, BOX, SUB, 2>, 4, 1, kS, 2>();
  return make_diff_info<D, DiffPathQ8<D, CODE, BOX, SUB, 2>, 2, 2, 2 * kS, 2>();
}

template <int CODE>
bool select_diff_q8(int D, int BS, int pairs, DiffKernelInfo* info) {
  // items of 32 tokens (K and V: 16 KiB at head_dim 128); a box is a block
  if (D == 128 && BS == 16) *info = diff_shape_q8<128, CODE, 16, 2>(pairs);
  else if (D == 128 && BS == 32) *info = diff_shape_q8<128, CODE, 32, 1>(pairs);
  else if (D == 64 && BS == 16) *info = diff_shape_q8<64, CODE, 16, 2>(pairs);
  else if (D == 64 && BS == 32) *info = diff_shape_q8<64, CODE, 32, 1>(pairs);
  else return false;
  return true;
}

}  // namespace pkv
