// keep.cu -- the accepted tokens of a verified draft move up in the cache: cached row
// base + path[i] of a sequence becomes row base + i, for K and V (and scales) of every KV
// head ("推测解码", chenk.top page: the accepted prefix of the draft stays; of a tree of
// drafted tokens one path does, whose rows lie scattered among the others').
//
// path rises, so path[i] >= i: a row's new place is never a later row's old one, and rows can
// move in place, a group at a time in order, once a whole group has been read. Bound by
// memory and, at a draft's size, by the latency of length, path, table and row in a chain.
// A CTA moves one head of one sequence, K and V together, up to four 16-byte words per thread
// and group. Measured on GB300 (calls back to back): 64 sequences, up to 4 tokens of 4 drafts, 8
// heads of 128 in bf16, 7.7 us; 256 sequences, up to 21 tokens, INT8, 9.3 us for 8 MB.
#include "common.cuh"
#include "internal.h"

namespace pkv {

namespace {
constexpr int kKeepThreads = 128;
constexpr int kKeepWords = 4;  // words per thread and group
}  // namespace

template <int ROW16>  // 16-byte words of a cached row
__global__ void __launch_bounds__(kKeepThreads) paged_kv_keep_kernel(const KeepParams p) {
  constexpr int kRows = kKeepThreads * kKeepWords / (2 * ROW16);  // rows (K and V) per group
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int s = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv, tid = threadIdx.x;
  const int base = __ldg(p.base + s);
  const int n = p.kept ? __ldg(p.kept + s) : p.width;
  const int32_t* path = p.path + size_t(s) * p.width;
  const long long room = (long long)p.MBS << p.bs_log2;
  int flags = (base < 0 || n < 0 || n > p.width) ? PKV_DEV_BAD_CONTEXT_LEN : 0;
  // cache row (of head 0) of token t; a bad one is flagged
  auto row_of = [&](long long t) -> long long {
    if (t < 0 || t >= room) {
      flags |= PKV_DEV_BAD_CONTEXT_LEN;
      return 0;
    }
    const int id = __ldg(p.tables + size_t(s) * p.MBS + (t >> p.bs_log2));
    if (id < 0 || id >= p.NB) {
      flags |= PKV_DEV_BAD_BLOCK_ID;
      return 0;
    }
    return ((long long)(id * p.Hkv + h) << p.bs_log2) + (t & ((1 << p.bs_log2) - 1));
  };
  if (!flags)  // the whole path first: a sequence with any fault stays as it was
    for (int i = tid; i < n; i += kKeepThreads) {
      const int at = __ldg(path + i);
      if (at < 0 || (i > 0 && at <= __ldg(path + i - 1))) flags |= PKV_DEV_BAD_CONTEXT_LEN;
      row_of((long long)base + at);
      row_of((long long)base + i);
    }
  if (__syncthreads_or(flags)) {
    if (flags && p.status) atomicOr(p.status, flags);
    return;
  }
  for (int i0 = 0; i0 < n; i0 += kRows) {
    uint4 v[kKeepWords];
    uint4* dst[kKeepWords];
#pragma unroll
    for (int k = 0; k < kKeepWords; ++k) {
      const int w = tid + k * kKeepThreads;
      const int side = w / (kRows * ROW16), i = i0 + w / ROW16 % kRows;
      dst[k] = nullptr;
      if (i >= n) continue;
      const int at = __ldg(path + i);
      if (at == i) continue;
      uint4* cache = reinterpret_cast<uint4*>(side ? p.vc : p.kc) + w % ROW16;
      dst[k] = cache + row_of((long long)base + i) * ROW16;
      v[k] = __ldcg(cache + row_of((long long)base + at) * ROW16);
    }
    float sc = 0.f;
    float* sdst = nullptr;
    if (p.ks && tid < 2 * kRows) {  // one scale per row
      const int i = i0 + tid % kRows;
      if (i < n) {
        float* scale = tid < kRows ? p.ks : p.vs;
        const int at = __ldg(path + i);
        if (at != i) {
          sdst = scale + row_of((long long)base + i);
          sc = __ldcg(scale + row_of((long long)base + at));
        }
      }
    }
    __syncthreads();  // the group is read
#pragma unroll
    for (int k = 0; k < kKeepWords; ++k)
      if (dst[k]) *dst[k] = v[k];
    if (sdst) *sdst = sc;
    // the next group's rows lie past this one's new places: no further barrier
  }
}

cudaError_t launch_keep(int row_bytes, const KeepParams& p, cudaStream_t stream) {
  const void* fn =
      row_bytes == 256   ? reinterpret_cast<const void*>(&paged_kv_keep_kernel<16>)
      : row_bytes == 128 ? reinterpret_cast<const void*>(&paged_kv_keep_kernel<8>)
                         : reinterpret_cast<const void*>(&paged_kv_keep_kernel<4>);
  KeepParams copy = p;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(unsigned(p.B) * unsigned(p.Hkv)), dim3(kKeepThreads), args, 0, stream);
}

}  // namespace pkv
