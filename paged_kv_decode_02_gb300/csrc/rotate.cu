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
// Bound by memory: a row is read and written once. D / 16 lanes share a row; a lane holds
// the two 16-byte chunks that its rotation pairs (chunks j and j + R/16, or 2j and 2j + 1
// interleaved; R is a multiple of 16), so both elements of every pair are in one lane and
// only the norm's and the quantiser's row reductions cross lanes. With many rows a lane
// group takes kU rows of one token: their loads are in flight together and share the
// token's position, slot and table row.
#include "common.cuh"
#include "encode.cuh"
#include "internal.h"

namespace pkv {

namespace {
// Small CTAs: a CTA loads, then computes, then stores, and many small ones overlap these.
// With kMany rows per lane group on GB300, 8192 tokens of 32/32 heads of 128 (bf16 cache):
// 512 threads 80.5 us, 256 63.3, 128 61.5, 64 61.0; 4096 tokens of 64/8 heads, normed, INT8:
// 38 us at 256, 34 at 64. Rows per lane group (256 threads): 1 84.9 us, 2 67.7, 4 63.3.
constexpr int kRotThreads = 64;
constexpr int kRotCtas = 12;       // per SM: 80 registers a thread
constexpr int kMany = 4;

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 p = unpack_bf16x2(w[e]);
    f[2 * e] = p.x;
    f[2 * e + 1] = p.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void load8(const float* p, float* f) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
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
  const long long t = item / sets;
  if (t >= p.T) return;
  const int first = int(item - unsigned(t) * sets);

  // the lane's two chunks of a row: a rotation pair's, or two of the rest
  const int nrot = p.R / 16;
  const bool turns = j < nrot;
  int ca = 2 * j, cb = 2 * j + 1;
  if (!p.interleaved && turns) {
    ca = j;
    cb = j + nrot;
  }
  // the token's q, k and v rows
  const __nv_bfloat16* rows_of[3] = {
      static_cast<const __nv_bfloat16*>(p.q) + t * p.q_stride,
      static_cast<const __nv_bfloat16*>(p.k) + t * p.k_stride - p.Hq * D,
      static_cast<const __nv_bfloat16*>(p.v) + t * p.v_stride - (p.Hq + p.Hkv) * D};
  // (a row read here may be the one written below: out may be q)
  uint4 raw[kU][2];
#pragma unroll
  for (int k = 0; k < kU; ++k) {
    const int r = first + k * int(sets);
    if (r < rows) {
      const uint4* src = reinterpret_cast<const uint4*>(
          rows_of[r < p.Hq ? 0 : r < p.Hq + p.Hkv ? 1 : 2] + r * D);
      raw[k][0] = src[ca];
      raw[k][1] = src[cb];
    }
  }
  const long long pos = p.positions[t];
  const long long slot = p.slots[t];
  const bool bad = pos < 0 || pos >= p.P;
  if (bad && first == 0 && j == 0 && p.status) atomicOr(p.status, PKV_DEV_BAD_POSITION);
  float c[8], s[8];
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
    float x[16];
    unpack8(raw[k][0], x);
    unpack8(raw[k][1], x + 8);
    const uint4* w = static_cast<const uint4*>(isq ? p.q_norm : p.k_norm);
    if (!isv && w != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
      const float rstd = rsqrtf(ss * (1.f / D) + p.eps);
      float f[16];
      unpack8(__ldg(w + ca), f);
      unpack8(__ldg(w + cb), f + 8);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = x[e] * rstd * f[e];
    }
    if (turns && !bad && !isv) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = a * c[i] - b * s[i];
          x[2 * i + 1] = b * c[i] + a * s[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = x[i], b = x[8 + i];
          x[i] = a * c[i] - b * s[i];
          x[8 + i] = b * c[i] + a * s[i];
        }
      }
    }
    if (isq) {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                            t * p.out_stride + r * D);
      dst[ca] = bad ? make_uint4(0u, 0u, 0u, 0u) : pack8(x);
      dst[cb] = bad ? make_uint4(0u, 0u, 0u, 0u) : pack8(x + 8);
      continue;
    }
    const int h = isv ? r - p.Hq - p.Hkv : r - p.Hq;
    const long long drow = drow0 + (h << p.bs_log2);
    if constexpr (CODE < 0) {
      if (skip) continue;
      uint4* dst = reinterpret_cast<uint4*>(isv ? p.vc : p.kc) + drow * (D / 8);
      dst[ca] = pack8(x);
      dst[cb] = pack8(x + 8);
    } else {
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 16; e += 2) amax = fmax3(amax, fabsf(x[e]), fabsf(x[e + 1]));
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(group, amax, o));
      if (skip) continue;
      const float sc = __fdiv_rn(amax, Encode8<CODE>::kMax);
      uint32_t u[4] = {0u, 0u, 0u, 0u};
      if (sc > 0.f) {
        const RowEncoder<CODE> enc(sc);
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = enc.four(x + 4 * e);
      }
      uint2* dst = reinterpret_cast<uint2*>(isv ? p.vc : p.kc) + drow * (D / 8);
      dst[ca] = make_uint2(u[0], u[1]);
      dst[cb] = make_uint2(u[2], u[3]);
      if (j == 0) (isv ? p.vs : p.ks)[drow] = sc;
    }
  }
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
