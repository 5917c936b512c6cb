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
// only the norm's and the quantiser's row reductions cross lanes.
#include "common.cuh"
#include "encode.cuh"
#include "internal.h"

namespace pkv {

namespace {
constexpr int kRotThreads = 256;

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
template <int D, int CODE>
__global__ void __launch_bounds__(kRotThreads)
    paged_kv_rotate_append_kernel(const RotateParams p) {
  constexpr int LPR = D / 16;  // lanes per row
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int rows = p.Hq + 2 * p.Hkv;  // rows per token: q, then k, then v heads
  const long long row = ((long long)blockIdx.x * kRotThreads + threadIdx.x) / LPR;
  const int j = threadIdx.x % LPR;
  // the row's lanes: they branch alike
  const uint32_t group = ((1u << LPR) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
  const bool live = row < (long long)p.T * rows;
  const int t = live ? int(row / rows) : 0;
  const int r = live ? int(row % rows) : 0;
  const bool isq = r < p.Hq, isv = r >= p.Hq + p.Hkv;
  const int h = isq ? r : isv ? r - p.Hq - p.Hkv : r - p.Hq;

  // the lane's two chunks of the row: a rotation pair's, or two of the rest
  const int nrot = p.R / 16;
  const bool turns = j < nrot && !isv;
  int ca = 2 * j, cb = 2 * j + 1;
  if (!p.interleaved && j < nrot) {
    ca = j;
    cb = j + nrot;
  }
  const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(isq ? p.q : isv ? p.v : p.k) +
                             (long long)t * (isq ? p.q_stride : isv ? p.v_stride : p.k_stride) +
                             h * D;
  float x[16];
  // (a row read here may be the one written below: out may be q)
  unpack8(reinterpret_cast<const uint4*>(src)[ca], x);
  unpack8(reinterpret_cast<const uint4*>(src)[cb], x + 8);
  const long long pos = p.positions[t];
  const long long slot = isq ? 0 : p.slots[t];
  const bool bad = pos < 0 || pos >= p.P;
  if (bad && live && r == 0 && j == 0 && p.status) atomicOr(p.status, PKV_DEV_BAD_POSITION);

  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(isq ? p.q_norm : p.k_norm);
  if (!isv && w != nullptr) {
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
    const float rstd = rsqrtf(ss * (1.f / D) + p.eps);
    float f[16];
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + ca), f);
    unpack8(__ldg(reinterpret_cast<const uint4*>(w) + cb), f + 8);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = x[e] * rstd * f[e];
  }
  if (turns && !bad) {
    const float* cs = p.cos_sin + pos * p.R + 8 * j;
    float c[8], s[8];
    load8(cs, c);
    load8(cs + p.R / 2, s);
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
    if (!live) return;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) +
                                          (long long)t * p.out_stride + h * D);
    dst[ca] = bad ? make_uint4(0u, 0u, 0u, 0u) : pack8(x);
    dst[cb] = bad ? make_uint4(0u, 0u, 0u, 0u) : pack8(x + 8);
    return;
  }
  const bool skip = !live || bad || slot < 0 || slot >= (long long)p.NB * p.BS;
  const long long drow = (slot / p.BS * p.Hkv + h) * p.BS + slot % p.BS;
  if constexpr (CODE < 0) {
    if (skip) return;
    uint4* dst = reinterpret_cast<uint4*>(isv ? p.vc : p.kc) + drow * (D / 8);
    dst[ca] = pack8(x);
    dst[cb] = pack8(x + 8);
  } else {
    using Enc = Encode8<CODE>;
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[e]));
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
      amax = fmaxf(amax, __shfl_xor_sync(group, amax, o));
    if (skip) return;
    const float s = __fdiv_rn(amax, Enc::kMax);
    uint32_t u[4] = {0u, 0u, 0u, 0u};
    if (s > 0.f) {
#pragma unroll
      for (int e = 0; e < 16; ++e) u[e / 4] |= uint32_t(Enc::code(x[e], s)) << (8 * (e % 4));
    }
    uint2* dst = reinterpret_cast<uint2*>(isv ? p.vc : p.kc) + drow * (D / 8);
    dst[ca] = make_uint2(u[0], u[1]);
    dst[cb] = make_uint2(u[2], u[3]);
    if (j == 0) (isv ? p.vs : p.ks)[drow] = s;
  }
}

cudaError_t launch_rotate_append(int code, int D, const RotateParams& p, cudaStream_t stream) {
  if (p.T <= 0) return cudaSuccess;
  const long long threads = (long long)p.T * (p.Hq + 2 * p.Hkv) * (D / 16);
  const long long grid = (threads + kRotThreads - 1) / kRotThreads;
  if (grid >= (1ll << 31)) return cudaErrorInvalidValue;
  const void* fn = nullptr;
#define PKV_ROTATE(DD, CC) \
  if (D == DD && code == CC) \
    fn = reinterpret_cast<const void*>(&paged_kv_rotate_append_kernel<DD, CC>);
  PKV_ROTATE(128, -1)
  PKV_ROTATE(64, -1)
  PKV_ROTATE(128, CODE_I8)
  PKV_ROTATE(64, CODE_I8)
  PKV_ROTATE(128, CODE_E4M3)
  PKV_ROTATE(64, CODE_E4M3)
  PKV_ROTATE(128, CODE_E5M2)
  PKV_ROTATE(64, CODE_E5M2)
#undef PKV_ROTATE
  if (!fn) return cudaErrorInvalidValue;
  RotateParams copy = p;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(unsigned(grid)), dim3(kRotThreads), args, 0, stream);
}

}  // namespace pkv
