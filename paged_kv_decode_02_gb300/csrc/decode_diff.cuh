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
// * One contraction for both maps: the M = 16 rows of an m16n8k16 MMA are up to 8 query
//   pairs' first maps (rows 0-7) and second maps (rows 8-15). Scores are
//   [Q_0; 0] K_2p^T + [0; Q_1] K_2p+1^T, the two heads accumulating apart; P [16 x tokens]
//   then multiplies V' once for both maps, so a V tile is read from shared memory once.
//   Rows r and r + 8 of an MMA's accumulator are in the same lane: the difference, and the
//   norm up to one 4-lane reduction, are local.
// * Work split: (sequence, unit, item) triples in one flat order, an item `kItem` tokens of
//   one KV pair, cut into G equal ranges, one per CTA (two CTAs per SM). Warp w of a CTA
//   takes items w, w + N, ... of its range with its own online-softmax state and its own
//   one-item ring; at the end of a unit the N states fold pairwise through shared memory
//   (fold.cuh's rescaling). A CTA rather than a warp owns a range because a cut unit's
//   record is 16 rows of 2 D floats: N times fewer records than with a range per warp.
//   A unit inside one CTA's range is finished there; a cut one leaves a record per CTA,
//   which the merge kernel (diff_merge.cu) folds.
// * Data movement: a TMA tensor copy brings 16 (or 32) tokens of both heads of a pair at
//   once (4-D map: swizzle span, token in block, block and head, half of the row). K and V
//   of an item have a barrier each: the next item's K is requested as soon as the scores
//   are done with this one's, its V when P.V is.
// * One-byte caches as in decode.cuh: codes widened exactly to fp16, the K scale on the
//   fp32 score, the V scale folded into the fp16 weight.
#pragma once

#include "common.cuh"
#include "decode.cuh"
#include "fold.cuh"
#include "internal.h"

namespace pkv {

constexpr int kDiffWarps = 4;

// 4-D tiled tensor copy global -> shared; completes its bytes on the mbarrier.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
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
  // a warp's ring: K, V, K scales, V scales, two barriers
  static constexpr int kOffV = kTile, kOffKs = 2 * kTile, kOffVs = kOffKs + kScales;
  static constexpr int kOffBar = kOffVs + kScales;
  static constexpr int kRing = (kOffBar + 16 + 1023) / 1024 * 1024;
  // one warp's state in the pairwise fold: o as 16-byte words per lane, (m, l) x 2 rows
  static constexpr int kStateWords = 2 * D / 8;
  static constexpr int kState = kStateWords * 512 + 512;
  static_assert(kBoxBytes % 1024 == 0, "boxes must keep 1024-byte alignment");

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

// State of one warp: rows gid (first map of the unit's query pair gid) and gid + 8 (second
// map) of the 16-row MMA; o[nd][0..1] belong to the first, o[nd][2..3] to the second.
template <int D>
struct DiffState {
  static constexpr int kND = 2 * D / 8;
  float o[kND][4];
  float m0, m1, l0, l1;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nd = 0; nd < kND; ++nd) o[nd][0] = o[nd][1] = o[nd][2] = o[nd][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  }
  // New row maxima over an item: rescales the state, returns what the item's scores
  // subtract. Every token of an item that a warp takes is of the context, so the maxima
  // are of at least one score; -inf (a score of -inf) subtracts 0.
  __device__ __forceinline__ void raise(float mx0, float mx1, float& mn0, float& mn1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    const float p0 = m0, p1 = m1;
    m0 = fmaxf(m0, mx0);
    m1 = fmaxf(m1, mx1);
    mn0 = m0 == -INFINITY ? 0.f : m0;
    mn1 = m1 == -INFINITY ? 0.f : m1;
    const float a0 = fast_exp2(p0 - mn0), a1 = fast_exp2(p1 - mn1);
    l0 *= a0;
    l1 *= a1;
#pragma unroll
    for (int nd = 0; nd < kND; ++nd) {
      o[nd][0] *= a0;
      o[nd][1] *= a0;
      o[nd][2] *= a1;
      o[nd][3] *= a1;
    }
  }
  __device__ __forceinline__ void put(uint8_t* buf, int lane) const {
    float4* b = reinterpret_cast<float4*>(buf);
#pragma unroll
    for (int nd = 0; nd < kND; ++nd)
      b[nd * 32 + lane] = make_float4(o[nd][0], o[nd][1], o[nd][2], o[nd][3]);
    b[kND * 32 + lane] = make_float4(m0, m1, l0, l1);
  }
  __device__ __forceinline__ void fold(const uint8_t* buf, int lane) {
    const float4* b = reinterpret_cast<const float4*>(buf);
    const float4 s = b[kND * 32 + lane];
    const float n0 = fmaxf(m0, s.x), n1 = fmaxf(m1, s.y);
    const float z0 = n0 == -INFINITY ? 0.f : n0, z1 = n1 == -INFINITY ? 0.f : n1;
    const float a0 = fast_exp2(m0 - z0), a1 = fast_exp2(m1 - z1);
    const float b0 = fast_exp2(s.x - z0), b1 = fast_exp2(s.y - z1);
    m0 = n0;
    m1 = n1;
    l0 = l0 * a0 + s.z * b0;
    l1 = l1 * a1 + s.w * b1;
#pragma unroll
    for (int nd = 0; nd < kND; ++nd) {
      const float4 v = b[nd * 32 + lane];
      o[nd][0] = o[nd][0] * a0 + v.x * b0;
      o[nd][1] = o[nd][1] * a0 + v.y * b0;
      o[nd][2] = o[nd][2] * a1 + v.z * b1;
      o[nd][3] = o[nd][3] * a1 + v.w * b1;
    }
  }
};

// Tensor-core path over a bf16 cache. The softmax weights enter P.V as bf16 (half a step
// of 2^-9 each, averaging out over tokens) and the row sums are of the rounded weights.
template <int D, int BOX, int SUB>
struct DiffPathBf16 {
  using Geo = DiffGeom<D, -1, BOX, SUB>;
  static constexpr int kKS = D / 16, kNT = Geo::kItem / 8, kKK = Geo::kItem / 16;
  static constexpr float kOutScale = 1.f;
  uint32_t qa[kKS][4];
  DiffState<D> st;

  // A 2 D row from the lanes' columns: run k holds 2 neighbouring ones, from column(k, cq).
  static constexpr int kRun = 2, kRuns = 2 * D / 8;
  __device__ static __forceinline__ int column(int k, int cq) { return k * 8 + 2 * cq; }
  __device__ static __forceinline__ float at(const float (&o)[kRuns][4], int k, int e, int row) {
    return o[k][2 * row + e];
  }

  // q0, q1: the two maps' query rows of query pair gid (D elements), when live.
  __device__ __forceinline__ void begin(const __nv_bfloat16* q0, const __nv_bfloat16* q1,
                                        bool live, int cq, float) {
    const uint32_t* w0 = reinterpret_cast<const uint32_t*>(q0);
    const uint32_t* w1 = reinterpret_cast<const uint32_t*>(q1);
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
      const int w = 8 * ks + cq;
      qa[ks][0] = live ? __ldg(w0 + w) : 0u;
      qa[ks][1] = live ? __ldg(w1 + w) : 0u;
      qa[ks][2] = live ? __ldg(w0 + w + 4) : 0u;
      qa[ks][3] = live ? __ldg(w1 + w + 4) : 0u;
    }
    st.clear();
  }

  // Scores of the item's tokens, in log2 units; tokens from nvalid on are -inf.
  __device__ __forceinline__ void scores(float (&x)[kNT][4], uint32_t sK, uint32_t, int nvalid,
                                         int lane, float scale_log2) {
    const int r8 = lane & 7, mi = lane >> 3, cq = lane & 3;
#pragma unroll
    for (int np = 0; np < kNT / 2; ++np) {
      float a[2][4] = {}, b[2][4] = {};  // first and second heads' scores apart
#pragma unroll
      for (int ks = 0; ks < kKS; ++ks) {
        uint32_t k0[4], k1[4];
        const int t = np * 16 + ((mi >> 1) << 3) + r8, cc = 2 * ks + (mi & 1);
        ldmatrix_x4(k0, sK + Geo::off(0, t, cc));
        ldmatrix_x4(k1, sK + Geo::off(1, t, cc));
        const uint32_t q0[4] = {qa[ks][0], 0u, qa[ks][2], 0u};
        const uint32_t q1[4] = {0u, qa[ks][1], 0u, qa[ks][3]};
        mma_bf16_16816(a[0], q0, k0[0], k0[1]);
        mma_bf16_16816(a[1], q0, k0[2], k0[3]);
        mma_bf16_16816(b[0], q1, k1[0], k1[1]);
        mma_bf16_16816(b[1], q1, k1[2], k1[3]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool ok = np * 16 + h * 8 + 2 * cq + e < nvalid;
          x[2 * np + h][e] = ok ? a[h][e] * scale_log2 : -INFINITY;
          x[2 * np + h][e + 2] = ok ? b[h][e + 2] * scale_log2 : -INFINITY;
        }
      }
    }
  }

  __device__ __forceinline__ void values(float (&x)[kNT][4], uint32_t sV, uint32_t, int,
                                         float mn0, float mn1, int lane) {
    const int r8 = lane & 7, mi = lane >> 3;
#pragma unroll
    for (int kk = 0; kk < kKK; ++kk) {
      uint32_t pa[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* s = x[2 * kk + h];
        pa[2 * h] = pack_bf16x2(fast_exp2(s[0] - mn0), fast_exp2(s[1] - mn0));
        pa[2 * h + 1] = pack_bf16x2(fast_exp2(s[2] - mn1), fast_exp2(s[3] - mn1));
        const float2 f0 = unpack_bf16x2(pa[2 * h]), f1 = unpack_bf16x2(pa[2 * h + 1]);
        st.l0 += f0.x + f0.y;
        st.l1 += f1.x + f1.y;
      }
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
#pragma unroll
        for (int n2 = 0; n2 < D / 16; ++n2) {
          uint32_t b[4];
          ldmatrix_x4_trans(
              b, sV + Geo::off(hd, 16 * kk + ((mi & 1) << 3) + r8, 2 * n2 + (mi >> 1)));
          mma_bf16_16816(st.o[hd * (D / 8) + 2 * n2], pa, b[0], b[1]);
          mma_bf16_16816(st.o[hd * (D / 8) + 2 * n2 + 1], pa, b[2], b[3]);
        }
      }
    }
  }
};

// Tensor-core path over one-byte codes (fp16 MMAs on exactly widened codes; kVUp as in
// MmaPathInt8 keeps the weight times the V scale out of fp16's subnormal range).
template <int D, int CODE, int BOX, int SUB>
struct DiffPathQ8 {
  using Geo = DiffGeom<D, CODE, BOX, SUB>;
  using Codec = Code8<CODE>;
  static constexpr float kVUp = CODE == CODE_E5M2 ? 32768.f : CODE == CODE_E4M3 ? 256.f : 1.f;
  static constexpr float kOutScale = 1.f / kVUp;
  static constexpr int kKS = D / 16, kNT = Geo::kItem / 8, kKK = Geo::kItem / 16;
  static constexpr int kQB = D / 4, kQC = kQB / 16;  // bytes of a K row each lane reads
  uint32_t qa[kKS][4];
  float rs0, rs1, qb0, qb1;
  DiffState<D> st;

  // n-tile 4 k + i (k counts over both heads), column n holds element 32 k + 4 n + i of the
  // 2 D row: a lane's run k is the 8 elements from 32 k + 8 cq.
  static constexpr int kRun = 8, kRuns = 2 * D / 32;
  __device__ static __forceinline__ int column(int k, int cq) { return 32 * k + 8 * cq; }
  __device__ static __forceinline__ float at(const float (&o)[2 * D / 8][4], int k, int e,
                                             int row) {
    return o[4 * k + e % 4][2 * row + e / 4];
  }

  // One map's row: scaled by a power of two to near 2^14 (then exact in fp16 for entries
  // above 2^-28 of the largest), rs the score scale that undoes it; INT8 codes enter the
  // score MMA as code + 1152, whose 1152 * sum(q) comes off the score.
  __device__ __forceinline__ void load_row(const __nv_bfloat16* q, bool live, int cq, int slot,
                                           float scale_log2, float& rs, float& qb) {
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
    int ex = 0;
    if (mx > 0.f) { frexpf(mx, &ex); ex = 14 - ex; }
    const float sc = ldexpf(1.f, ex);
    rs = scale_log2 * ldexpf(1.f, -ex);
    float t = 0.f;
#pragma unroll
    for (int ks = 0; ks < kKS; ++ks) {
      qa[ks][slot] = pack_f16x2(f[ks][0] * sc, f[ks][1] * sc);
      qa[ks][slot + 2] = pack_f16x2(f[ks][2] * sc, f[ks][3] * sc);
      const float2 a = unpack_f16x2(qa[ks][slot]), b = unpack_f16x2(qa[ks][slot + 2]);
      t += (a.x + a.y) + (b.x + b.y);
    }
    qb = 0.f;
    if constexpr (CODE == CODE_I8) {
      t += __shfl_xor_sync(0xffffffffu, t, 1);
      t += __shfl_xor_sync(0xffffffffu, t, 2);
      qb = 1152.f * t;
    }
  }

  __device__ __forceinline__ void begin(const __nv_bfloat16* q0, const __nv_bfloat16* q1,
                                        bool live, int cq, float scale_log2) {
    load_row(q0, live, cq, 0, scale_log2, rs0, qb0);
    load_row(q1, live, cq, 1, scale_log2, rs1, qb1);
    st.clear();
  }

  __device__ __forceinline__ void scores(float (&x)[kNT][4], uint32_t sK, uint32_t sKs,
                                         int nvalid, int lane, float) {
    const int gid = lane >> 2, cq = lane & 3;
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      float a[2][4] = {};
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
#pragma unroll
        for (int ch = 0; ch < kQC; ++ch) {
          const uint4 raw = lds128(sK + Geo::off(hd, nt * 8 + gid, kQC * cq + ch));
          const uint32_t w[4] = {Codec::pre(raw.x), Codec::pre(raw.y), Codec::pre(raw.z),
                                 Codec::pre(raw.w)};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int ks = 4 * ch + k;
            const uint32_t q[4] = {hd ? 0u : qa[ks][0], hd ? qa[ks][1] : 0u,
                                   hd ? 0u : qa[ks][2], hd ? qa[ks][3] : 0u};
            if constexpr (CODE == CODE_I8)
              mma_f16_16816(a[hd], q, prmt(w[k], 0x64646464u, 0x4140u),
                            prmt(w[k], 0x64646464u, 0x4342u));
            else
              mma_f16_16816(a[hd], q, Codec::lo(w[k]), Codec::hi(w[k]));
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = nt * 8 + 2 * cq + e;
        const bool ok = tok < nvalid;
        x[nt][e] = ok ? (a[0][e] - qb0) * lds_f32(sKs + Geo::scale_off(0, tok)) * rs0 : -INFINITY;
        x[nt][e + 2] =
            ok ? (a[1][e + 2] - qb1) * lds_f32(sKs + Geo::scale_off(1, tok)) * rs1 : -INFINITY;
      }
    }
  }

  __device__ __forceinline__ void values(float (&x)[kNT][4], uint32_t sV, uint32_t sVs,
                                         int nvalid, float mn0, float mn1, int lane) {
    const int gid = lane >> 2, cq = lane & 3;
#pragma unroll
    for (int kk = 0; kk < kKK; ++kk) {
      float w[2][4];  // weights of tokens 16 kk + 8 h + 2 cq (+ 1)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float* s = x[2 * kk + h];
        w[h][0] = fast_exp2(s[0] - mn0);
        w[h][1] = fast_exp2(s[1] - mn0);
        w[h][2] = fast_exp2(s[2] - mn1);
        w[h][3] = fast_exp2(s[3] - mn1);
        st.l0 += w[h][0] + w[h][1];
        st.l1 += w[h][2] + w[h][3];
      }
      const int ta = 16 * kk + 2 * cq;
#pragma unroll
      for (int hd = 0; hd < 2; ++hd) {
        uint32_t pa[4];  // each value head has its own scales
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float vs[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = ta + 8 * h + e;
            vs[e] = tok < nvalid ? lds_f32(sVs + Geo::scale_off(hd, tok)) * kVUp : 0.f;
          }
          pa[2 * h] = pack_f16x2(w[h][0] * vs[0], w[h][1] * vs[1]);
          pa[2 * h + 1] = pack_f16x2(w[h][2] * vs[0], w[h][3] * vs[1]);
        }
#pragma unroll
        for (int qg = 0; qg < D / 32; ++qg) {
          const int bo = 32 * qg + 4 * gid, ch = bo >> 4, wi = bo & 15;
          const uint32_t w0 = Codec::pre(lds32(sV + Geo::off(hd, ta, ch) + wi));
          const uint32_t w1 = Codec::pre(lds32(sV + Geo::off(hd, ta + 1, ch) + wi));
          const uint32_t w2 = Codec::pre(lds32(sV + Geo::off(hd, ta + 8, ch) + wi));
          const uint32_t w3 = Codec::pre(lds32(sV + Geo::off(hd, ta + 9, ch) + wi));
          const uint32_t x01 = prmt(w0, w1, 0x5140u), x23 = prmt(w0, w1, 0x7362u);
          const uint32_t y01 = prmt(w2, w3, 0x5140u), y23 = prmt(w2, w3, 0x7362u);
          float (*o)[4] = &st.o[hd * (D / 8) + 4 * qg];
          mma_f16_16816(o[0], pa, Codec::lo(x01), Codec::lo(y01));
          mma_f16_16816(o[1], pa, Codec::hi(x01), Codec::hi(y01));
          mma_f16_16816(o[2], pa, Codec::lo(x23), Codec::lo(y23));
          mma_f16_16816(o[3], pa, Codec::hi(x23), Codec::hi(y23));
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

template <int D, class Path>
__global__ void __launch_bounds__(kDiffWarps * 32, 2)
    paged_diff_decode_kernel(const __grid_constant__ CUtensorMap tmk,
                             const __grid_constant__ CUtensorMap tmv, const DiffParams p) {
  using Geo = typename Path::Geo;
  constexpr int N = kDiffWarps, kThreads = N * 32, kND = 2 * D / 8;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gen = smem_raw + (base - smem_u32(smem_raw));
  uint8_t* states = gen + N * Geo::kRing;                       // [N / 2] folded states
  int* prefix = reinterpret_cast<int*>(states + (N / 2) * Geo::kState);
  __shared__ int warp_tot[N];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, cq = lane & 3;
  const int B = p.B;
  const uint32_t ring = base + warp * Geo::kRing;
  const uint32_t sK = ring, sV = ring + Geo::kOffV;
  const uint32_t sKs = ring + Geo::kOffKs, sVs = ring + Geo::kOffVs;
  const uint32_t barK = ring + Geo::kOffBar, barV = barK + 8;
  if (lane == 0) {
    mbar_init(barK, 1);
    mbar_init(barV, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmk);
    tma_prefetch_desc(&tmv);
  }
  pdl_wait_prior_grid();

  // ---- items per sequence and their exclusive prefix (every CTA computes it) ----
  {
    const int per = (B + kThreads - 1) / kThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int sum = 0;
    for (int i = b0; i < b1; ++i) sum += diff_items(p, i, Geo::kItem);
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < warp; ++w) run += warp_tot[w];
    if (tid == 0) prefix[0] = 0;
    for (int i = b0; i < b1; ++i) {
      run += diff_items(p, i, Geo::kItem);
      prefix[i + 1] = run;
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = tid; i <= B; i += kThreads) p.prefix[i] = prefix[i];
  }

  const int U = p.P * p.nsg;  // units per sequence
  const long long T = (long long)U * prefix[B];
  const long long a = T * blockIdx.x / gridDim.x, b = T * (blockIdx.x + 1) / gridDim.x;
  const int n = int(b - a);
  if (n == 0) return;

  Cursor cur;  // the segment: unit cur.u of sequence cur.s from its item cur.j on
  cursor_locate(cur, a, prefix, B, U);
  // the producer's item: number pi of the CTA's range, every N-th one is this warp's
  Cursor pc = cur;
  int pi = 0, pid[Geo::kSub], pL = 0;
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
    pL = min(__ldg(p.context_lens + pc.s), p.MBS * p.BS);
#pragma unroll
    for (int k = 0; k < Geo::kSub; ++k) {
      const int t = (pc.j * Geo::kSub + k) * Geo::kBox;
      pid[k] = 0;
      if (t < pL) {
        const int id = __ldg(p.block_tables + size_t(pc.s) * p.MBS + t / p.BS);
        pid[k] = id < 0 || id >= p.NB ? 0 : id;  // stay in the pool
      }
    }
  };
  // lane 0: requests K (or V) of the producer's item; boxes past the context are left out
  auto issue = [&](const CUtensorMap* map, uint32_t tile, uint32_t scales, const float* scale,
                   uint32_t bar) {
    if (lane != 0 || pi >= n) return;
    const int t0 = pc.j * Geo::kItem;
    const int boxes = min(Geo::kSub, (pL - t0 + Geo::kBox - 1) / Geo::kBox);
    mbar_arrive_expect_tx(bar, uint32_t(boxes) * (Geo::kBoxBytes + Geo::kScaleBox));
    const int head = 2 * (pc.u / p.nsg);
#pragma unroll
    for (int k = 0; k < Geo::kSub; ++k) {
      if (k >= boxes) break;
      const int in = (t0 + k * Geo::kBox) % p.BS;
      const int row = pid[k] * 2 * p.P + head;
      tma_load_4d(tile + k * Geo::kBoxBytes, map, bar, 0, in, row, 0);
      if constexpr (Geo::kQ8)  // a box is a whole block: both heads' scales are neighbours
        bulk_load(scales + k * Geo::kScaleBox, scale + size_t(row) * Geo::kBox, Geo::kScaleBox,
                  bar);
    }
  };
  advance(warp);
  fetch();
  issue(&tmk, sK, sKs, p.k_scale, barK);
  issue(&tmv, sV, sVs, p.v_scale, barV);

  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q);
  Path path;
  uint32_t par = 0;
  bool dead = false, first = true;
  for (int i = 0; i < n;) {
    const int len = min(n - i, cur.n - cur.j);
    const int pair = cur.u / p.nsg, r0 = (cur.u % p.nsg) * p.gs;
    const bool live = gid < p.gs && r0 + gid < p.g;
    const int qp = pair * p.g + r0 + gid;  // this lane's query pair of the sequence
    const int Hq = 2 * p.P * p.g;
    const __nv_bfloat16* qr = q + (size_t(cur.s) * Hq + (live ? 2 * qp : 0)) * D;
    path.begin(qr, qr + D, live, cq, p.scale_log2);
    const int L = min(__ldg(p.context_lens + cur.s), p.MBS * p.BS);

    int k = i + (warp - i % N + N) % N;
    for (; k < i + len && !dead; k += N) {
      const int nvalid = L - (cur.j + k - i) * Geo::kItem;
      advance(N);  // pc: the item after this one
      fetch();
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(barK, par, p.timeout_ns))) {
        dead = true;  // let what is in flight land before the warp goes on
        mbar_wait_bounded(barK, par, p.timeout_ns);
        mbar_wait_bounded(barV, par, p.timeout_ns);
        break;
      }
      float x[Path::kNT][4];
      path.scores(x, sK, sKs, nvalid, lane, p.scale_log2);
      fence_proxy_async_smem();  // this lane's reads of K before its refill
      __syncwarp();
      issue(&tmk, sK, sKs, p.k_scale, barK);
      float mx0 = -INFINITY, mx1 = -INFINITY, mn0, mn1;
#pragma unroll
      for (int t = 0; t < Path::kNT; ++t) {
        mx0 = fmax3(mx0, x[t][0], x[t][1]);
        mx1 = fmax3(mx1, x[t][2], x[t][3]);
      }
      path.st.raise(mx0, mx1, mn0, mn1);
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(barV, par, p.timeout_ns))) {
        dead = true;
        mbar_wait_bounded(barV, par, p.timeout_ns);
        if (pi < n) mbar_wait_bounded(barK, par ^ 1u, p.timeout_ns);  // the K just requested
        break;
      }
      // rows past the context may hold anything (even NaN): zero them before P.V
      if (nvalid < Geo::kItem) {
        for (int c = lane; c < (Geo::kItem - nvalid) * 2 * Geo::kChunksPerRow; c += 32) {
          const int t = nvalid + c / (2 * Geo::kChunksPerRow), cc = c % (2 * Geo::kChunksPerRow);
          sts128_zero(sV + Geo::off(cc / Geo::kChunksPerRow, t, cc % Geo::kChunksPerRow));
        }
        __syncwarp();
      }
      path.values(x, sV, sVs, nvalid, mn0, mn1, lane);
      fence_proxy_async_smem();
      __syncwarp();
      issue(&tmv, sV, sVs, p.v_scale, barV);
      par ^= 1u;
    }
    if (dead && lane == 0 && p.status) atomicOr(p.status, PKV_DEV_TIMEOUT);

    // ---- fold the warps' states into warp 0's ----
    DiffState<D>& st = path.st;
    st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, 1);
    st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, 2);
    st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, 1);
    st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, 2);
#pragma unroll
    for (int half = N / 2; half > 0; half >>= 1) {
      if (warp >= half && warp < 2 * half) st.put(states + (warp - half) * Geo::kState, lane);
      __syncthreads();
      if (warp < half) st.fold(states + warp * Geo::kState, lane);
      __syncthreads();  // before the next level, or the next unit, writes there again
    }
    if (warp == 0) {
      const bool complete = cur.j == 0 && len == cur.n;
      if (!complete) {
        const size_t slot = size_t(2) * blockIdx.x + (first ? 0 : 1);
        const size_t r = slot * 2 * p.gs + gid;
        if (gid < p.gs) {
          float* o0 = p.part_o + r * (2 * D);
          float* o1 = o0 + size_t(p.gs) * (2 * D);
#pragma unroll
          for (int k2 = 0; k2 < Path::kRuns; ++k2) {
            const int c = Path::column(k2, cq);
#pragma unroll
            for (int e = 0; e < Path::kRun; e += 2) {
              *reinterpret_cast<float2*>(o0 + c + e) =
                  make_float2(Path::at(st.o, k2, e, 0) * Path::kOutScale,
                              Path::at(st.o, k2, e + 1, 0) * Path::kOutScale);
              *reinterpret_cast<float2*>(o1 + c + e) =
                  make_float2(Path::at(st.o, k2, e, 1) * Path::kOutScale,
                              Path::at(st.o, k2, e + 1, 1) * Path::kOutScale);
            }
          }
          if (cq == 0) {
            float2* ml = reinterpret_cast<float2*>(p.part_ml);
            ml[r] = make_float2(st.m0, st.l0);
            ml[r + p.gs] = make_float2(st.m1, st.l1);
          }
        }
      } else {
        const float i0 = Path::kOutScale / st.l0;
        const float i1 = Path::kOutScale / st.l1 * (live ? __ldg(p.lam + qp) : 0.f);
        float ss = 0.f;
#pragma unroll
        for (int nd = 0; nd < kND; ++nd) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float d = st.o[nd][e] * i0 - st.o[nd][e + 2] * i1;
            st.o[nd][e] = d;
            ss = fmaf(d, d, ss);
          }
        }
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += __shfl_xor_sync(0xffffffffu, ss, 2);
        const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.norm_w);
        const float f = w ? rsqrtf(ss * (1.f / (2 * D)) + p.eps) * p.out_scale : p.out_scale;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) +
                             (size_t(cur.s) * (Hq / 2) + (live ? qp : 0)) * (2 * D);
        if (live) {
#pragma unroll
          for (int k2 = 0; k2 < Path::kRuns; ++k2) {
            const int c = Path::column(k2, cq);
#pragma unroll
            for (int e = 0; e < Path::kRun; e += 2) {
              float2 g = make_float2(f, f);
              if (w) {
                g = unpack_bf16x2(__ldg(reinterpret_cast<const uint32_t*>(w + c + e)));
                g = make_float2(f * g.x, f * g.y);
              }
              *reinterpret_cast<uint32_t*>(out + c + e) =
                  pack_bf16x2(Path::at(st.o, k2, e, 0) * g.x, Path::at(st.o, k2, e + 1, 0) * g.y);
            }
          }
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
}

template <int D, int CODE, int BOX, int SUB>
DiffKernelInfo make_diff_info() {
  using Geo = DiffGeom<D, CODE, BOX, SUB>;
  DiffKernelInfo info{};
  if constexpr (CODE < 0)
    info.fn = reinterpret_cast<const void*>(&paged_diff_decode_kernel<D, DiffPathBf16<D, BOX, SUB>>);
  else
    info.fn = reinterpret_cast<const void*>(
        &paged_diff_decode_kernel<D, DiffPathQ8<D, CODE, BOX, SUB>>);
  info.threads = kDiffWarps * 32;
  info.smem = 1024 + kDiffWarps * Geo::kRing + kDiffWarps / 2 * Geo::kState;
  info.box = BOX;
  info.item = Geo::kItem;
  return info;
}

template <int CODE>
bool select_diff_q8(int D, int BS, DiffKernelInfo* info) {
  // items of 32 tokens (K and V: 16 KiB at head_dim 128); a box is a block
  if (D == 128 && BS == 16) *info = make_diff_info<128, CODE, 16, 2>();
  else if (D == 128 && BS == 32) *info = make_diff_info<128, CODE, 32, 1>();
  else if (D == 64 && BS == 16) *info = make_diff_info<64, CODE, 16, 2>();
  else if (D == 64 && BS == 32) *info = make_diff_info<64, CODE, 32, 1>();
  else return false;
  return true;
}

}  // namespace pkv
