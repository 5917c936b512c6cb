// rotate.cu -- per-head norms and position rotation of new queries and keys, written with
// the values into the paged cache in one pass.
//
// For every new token t and head row x [D] of its q and k (fp32 arithmetic):
//   y = x * rsqrt(mean(x^2) + eps) * w        (w: the q or k norm weight; no weight: y = x)
//   (y_a, y_b) <- (y_a c_i - y_b s_i, y_b c_i + y_a s_i)   for i < R/2,
// where c_i, s_i are row positions[t] of the caller's table and (a, b) = (i, i + R/2), or
// (2i, 2i + 1) interleaved; elements from R on stay y. A rotated q row leaves as bf16; a
// rotated k row goes to its slot as bf16 or, in a one-byte cache, through the absmax
// quantiser of the append kernels, applied to the fp32 row (one rounding instead of two);
// v rows are copied or quantised as the append kernels do. ("块管理器：分页如何运作" and
// "KV 缓存量化", chenk.top page, say where the rows go; the norm and rotation are those of
// the models that such caches serve.)
//
// Bound by memory: a row is read and written once. Measured on GB300: 8192 tokens of 32/32
// heads of 128, half rotated, interleaved, bf16 cache 60 us (405 MB, 6740 GB/s); of 32/8
// heads, normed, 32 us (206 MB, 6420 GB/s); into INT8 37.1 us (189 MB, 5110 GB/s: there the
// quantiser's instructions count, half the issue slots), E4M3 and E5M2 36.2. D / 16 lanes
// share a row; a lane holds the two 16-byte chunks that its rotation pairs (chunks j and
// j + R/16, or 2j and 2j + 1 interleaved; R is a multiple of 16), so both elements of every
// pair are in one lane and only the norm's and the quantiser's row reductions cross lanes.
// With many rows a lane group takes kU rows of one token: their loads are in flight together
// and share the token's position, slot and table row.
#include "common.cuh"
#include "encode.cuh"
#include "internal.h"

namespace pkv {

namespace {
// Small CTAs: a CTA loads, then computes, then stores, and many small ones overlap these. On
// GB300, 8192 tokens of 32/32 heads of 128 (bf16 cache, 4 rows per lane group): 512 threads
// 80.5 us, 256 63.3, 128 61.5, 64 61.0. Rows per lane group and CTAs per SM (8192 tokens of
// 32/8 heads, normed, bf16 and INT8 caches; 65536 tokens of 2/2 heads, INT8): 1 and 16 51.4,
// 51.8, 53.9 us; 2 and 16 32.7, 38.2, 47.9; 3 and 12 32.1, 37.3, 40.4; 4 and 10 33.2, 38.8,
// 45.1. CTAs that stay and load ahead of their computing have fewer registers for rows and
// lose (2 and 10: 34.8, 37.7, 50.2).
constexpr int kRotThreads = 64;
constexpr int kRotCtas = 12;       // per SM
constexpr int kMany = 3;           // rows per lane group

__device__ __forceinline__ void unpack8(const uint4& u, float2* f) {
  f[0] = unpack_bf16x2(u.x);
  f[1] = unpack_bf16x2(u.y);
  f[2] = unpack_bf16x2(u.z);
  f[3] = unpack_bf16x2(u.w);
}
__device__ __forceinline__ uint4 pack8(const float2* f) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                    pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}
__device__ __forceinline__ void load8(const float* p, float2* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = make_float2(a.x, a.y);
  f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y);
  f[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
}  // namespace

// CODE: CODE_I8 / CODE_E4M3 / CODE_E5M2, or -1 for a bf16 cache.
template <int D, int CODE, int kU>
__global__ void __launch_bounds__(kRotThreads, kRotCtas)
    paged_kv_rotate_append_kernel(const RotateParams p) {
  constexpr int LPR = D / 16;  // lanes per row
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int rows = p.Hq + 2 * p.Hkv;  // rows per token: q, then k, then v heads
  const unsigned sets = unsigned(rows + kU - 1) / kU;  // of a token; set i: rows i + k sets
  const unsigned item = blockIdx.x * (kRotThreads / LPR) + threadIdx.x / LPR;
  const int j = threadIdx.x % LPR;
  // the row's lanes: they branch alike
  const uint32_t group = ((1u << LPR) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
  // the lane's two chunks of a row: a rotation pair's, or two of the rest
  const int nrot = p.R / 16;
  const bool turns = j < nrot;
  int ca = 2 * j, cb = 2 * j + 1;
  if (!p.interleaved && turns) {
    ca = j;
    cb = j + nrot;
  }
  const uint4* qw = static_cast<const uint4*>(p.q_norm);
  const uint4* kw = static_cast<const uint4*>(p.k_norm);
  if (item >= unsigned(p.T) * sets) return;
  const long long t = item / sets;
  const int first = int(item - unsigned(t) * sets);
  // the token's q, k and v rows
  const __nv_bfloat16* qrow = static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride;
  const __nv_bfloat16* krow =
      static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride - p.Hq * D;
  const __nv_bfloat16* vrow =
      static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride - (p.Hq + p.Hkv) * D;
  // (a row read here may be the one written below: out may be q)
  uint4 raw[kU][2];
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const int r = first + k * int(sets);
    if (r < rows) {
      const uint4* src = reinterpret_cast<const uint4*>(
          (r < p.Hq ? qrow : r < p.Hq + p.Hkv ? krow : vrow) + r * D);
      raw[k][0] = src[ca];
      raw[k][1] = src[cb];
    }
  }
  const long long pos = p.positions[t];
  const long long slot = p.slots[t];
  // (a lambda: as the rest of the kernel it compiles to more address arithmetic; 8192 tokens
  // of 32/8 heads, bf16: 33.0 us, so 32.0)
  const auto finish = [&](const uint4 (&raw)[kU][2]) {
    const bool bad = pos < 0 || pos >= p.P;
    if (bad && first == 0 && j == 0 && p.status) atomicOr(p.status, PKV_DEV_BAD_POSITION);
    float2 c[4], s[4];
    if (turns && !bad) {
      const float* cs = p.cos_sin + pos * p.R + 8 * j;
      load8(cs, c);
      load8(cs + p.R / 2, s);
    }
    const bool skip = bad || slot < 0 || slot >= (long long)p.NB << p.bs_log2;
    // cache row of KV head 0: (block * Hkv + head) * BS + offset
    const long long drow0 = (((slot >> p.bs_log2) * p.Hkv) << p.bs_log2) +
                            (slot & ((1 << p.bs_log2) - 1));

#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int r = first + k * int(sets);
      if (r >= rows) break;
      const bool isq = r < p.Hq, isv = r >= p.Hq + p.Hkv;
      float2 x[8];  // chunk ca, then chunk cb
      unpack8(raw[k][0], x);
      unpack8(raw[k][1], x + 4);
      const uint4* w = isq ? qw : kw;
      if (!isv && w != nullptr) {
        float2 s2 = both(0.f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s2 = __ffma2_rn(x[e], x[e], s2);
        float ss = s2.x + s2.y;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
        const float2 rstd = both(rsqrtf(ss * (1.f / D) + p.eps));
        float2 f[4];
        unpack8(__ldg(w + ca), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __fmul2_rn(__fmul2_rn(x[e], rstd), f[e]);
        unpack8(__ldg(w + cb), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 + e] = __fmul2_rn(__fmul2_rn(x[4 + e], rstd), f[e]);
      }
      if (turns && !bad && !isv) {
        if (p.interleaved) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float ci = i % 2 ? c[i / 2].y : c[i / 2].x, si = i % 2 ? s[i / 2].y : s[i / 2].x;
            x[i] = make_float2(x[i].x * ci - x[i].y * si, x[i].y * ci + x[i].x * si);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = x[i], b = x[4 + i];
            x[i] = __ffma2_rn(a, c[i], __fmul2_rn(b, make_float2(-s[i].x, -s[i].y)));
            x[4 + i] = __ffma2_rn(b, c[i], __fmul2_rn(a, s[i]));
          }
        }
      }
      if (isq) {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                              t * p.out_stride + r * D);
        dst[ca] = bad ? make_uint4(0u, 0u, 0u, 0u) : pack8(x);
        dst[cb] = bad ? make_uint4(0u, 0u, 0u, 0u) : pack8(x + 4);
        continue;
      }
      const int h = isv ? r - p.Hq - p.Hkv : r - p.Hq;
      const long long drow = drow0 + (h << p.bs_log2);
      if constexpr (CODE < 0) {
        if (skip) continue;
        uint4* dst = reinterpret_cast<uint4*>(isv ? p.vc : p.kc) + drow * (D / 8);
        dst[ca] = pack8(x);
        dst[cb] = pack8(x + 4);
      } else {
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmax3(amax, fabsf(x[e].x), fabsf(x[e].y));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, o));
        if (skip) continue;
        const float sc = __fdiv_rn(amax, Encode8<CODE>::kMax);
        uint32_t u[4] = {0u, 0u, 0u, 0u};
        if (sc > 0.f) {
          const RowEncoder<CODE> enc(sc);
#pragma unroll
          for (int e = 0; e < 4; ++e) u[e] = enc.four(x + 2 * e);
        }
        uint2* dst = reinterpret_cast<uint2*>(isv ? p.vc : p.kc) + drow * (D / 8);
        dst[ca] = make_uint2(u[0], u[1]);
        dst[cb] = make_uint2(u[2], u[3]);
        if (j == 0) (isv ? p.vs : p.ks)[drow] = sc;
      }
    }
  };
  finish(raw);
}

template <int D, int CODE>
cudaError_t launch_rotate(const RotateParams& p, cudaStream_t stream) {
  // few rows: a row per lane group, as many of them as there are; rows enough for every
  // SM's threads twice over: kMany rows each
  const long long rows = p.Hq + 2 * p.Hkv;
  if (p.T * rows >= (1ll << 31)) return cudaErrorInvalidValue;
  const bool many = p.T * rows * (D / 16) >= 2ll * 152 * 2048;
  const long long items = p.T * (many ? (rows + kMany - 1) / kMany : rows);
  constexpr int per = kRotThreads / (D / 16);
  RotateParams copy = p;
  void* args[] = {&copy};
  const void* fn =
      many ? reinterpret_cast<const void*>(&paged_kv_rotate_append_kernel<D, CODE, kMany>)
           : reinterpret_cast<const void*>(&paged_kv_rotate_append_kernel<D, CODE, 1>);
  return launch_pdl(fn, dim3(unsigned((items + per - 1) / per)), dim3(kRotThreads), args, 0,
                    stream);
}

cudaError_t launch_rotate_append(int code, int D, const RotateParams& p, cudaStream_t stream) {
  if (p.T <= 0) return cudaSuccess;
  switch (code) {
    case -1: return D == 128 ? launch_rotate<128, -1>(p, stream) : launch_rotate<64, -1>(p, stream);
    case CODE_I8:
      return D == 128 ? launch_rotate<128, CODE_I8>(p, stream)
                      : launch_rotate<64, CODE_I8>(p, stream);
    case CODE_E4M3:
      return D == 128 ? launch_rotate<128, CODE_E4M3>(p, stream)
                      : launch_rotate<64, CODE_E4M3>(p, stream);
    case CODE_E5M2:
      return D == 128 ? launch_rotate<128, CODE_E5M2>(p, stream)
                      : launch_rotate<64, CODE_E5M2>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace pkv
