// tree_join.cu -- what follows the tree attention (tree.cuh): records of items cut between two
// CTAs' stretches are joined, rows past each tree's tiles become zeros, and, with a status word,
// every sequence is checked.
#include "tree.cuh"

namespace pkv {

namespace {
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;   // rows per CTA
constexpr int kZeroCtas = 152;  // CTAs that zero rows, sequence after sequence
}  // namespace

// Zeroes rows [first, q_len) of sequence s's output, by a CTA (part y of n).
__device__ __forceinline__ void zero_rows(const TreeParams& p, int s, int first, int y, int n) {
  const long long chunks = (long long)(p.q_len - first) * p.Hq * (p.D / 8);
  uint4* o = reinterpret_cast<uint4*>(p.out) + ((long long)s * p.q_len + first) * p.Hq * (p.D / 8);
  for (long long k = (long long)y * blockDim.x + threadIdx.x; k < chunks;
       k += (long long)n * blockDim.x)
    o[k] = make_uint4(0u, 0u, 0u, 0u);
}

// CTA (c, y), c < G: rows 32 y .. of the item that CTA c's stretch begins and does not end. Its
// parts are that record and the first records of the CTAs after it, up to the one that ends the
// item; they meet at the largest of their maxima. A row takes D / 4 lanes, a quad of columns each.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeParams p, int G) {
  constexpr int Q = D / 4;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  if (int(blockIdx.x) >= G) {
    for (int s = blockIdx.x - G; s < p.B; s += gridDim.x - G) {
      TreeSeq q;
      q.load(p, s);
      if (q.tiles * p.tpt < p.q_len) zero_rows(p, s, q.tiles * p.tpt, blockIdx.y, gridDim.y);
    }
    return;
  }
  const TreeCut cut = p.cuts[blockIdx.x];
  if (!(cut.state & kPromptBegins)) return;
  TreeSeq q;
  q.load(p, cut.s);
  const int pairs = (q.tiles + 1) >> 1, pr = cut.u % pairs, hv = cut.u / pairs;
  const int rows = 2 * pr + 1 >= q.tiles ? 128 : 256;
  const int dq = threadIdx.x % Q;
  for (int r0 = threadIdx.x / Q; r0 < kJoinRows; r0 += kJoinThreads / Q) {
    const int row = blockIdx.y * kJoinRows + r0, X = row >> 7, r = row & 127;
    const int rt = r / p.g, node = (2 * pr + X) * p.tpt + rt;
    if (row >= rows || rt >= p.tpt || node >= p.q_len) continue;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int slot) {
      const size_t rec = size_t(slot) * 256 + row;
      const float2 ml = reinterpret_cast<const float2*>(p.part_ml)[rec];
      // a part that saw nothing has no output; a NaN sum goes on
      if (!(ml.x > -INFINITY) && ml.y == 0.f) return;
      const float4 v = reinterpret_cast<const float4*>(p.part_o)[rec * Q + dq];
      const float m = fmaxf(M, ml.x);
      const float a = M > -INFINITY ? fast_exp2(M - m) : 0.f;
      const float b = ml.x > -INFINITY ? fast_exp2(ml.x - m) : 1.f;
      L = L * a + ml.y * b;
      o = make_float4(o.x * a + v.x * b, o.y * a + v.y * b, o.z * a + v.z * b, o.w * a + v.w * b);
      M = m;
    };
    add(cut.slot);
    for (int c = blockIdx.x + 1; c < G; ++c) {
      const int state = p.cuts[c].state;
      if (state & kPromptEmpty) continue;
      if (!(state & kPromptContinues)) break;
      add(2 * c);
      if (state & kPromptEnds) break;
    }
    const float inv = L > 0.f ? 1.f / L : L == 0.f ? 0.f : L;  // (NaN stays)
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) +
                         ((size_t(cut.s) * p.q_len + node) * p.Hq + hv * p.g + r % p.g) * D;
    reinterpret_cast<uint2*>(out)[dq] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

// Lengths and the block ids that they need, a CTA per sequence at a time: flags, and zeros for a
// sequence that fails.
__global__ void __launch_bounds__(kJoinThreads) tree_check_kernel(const TreeParams p) {
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  for (int s = blockIdx.x; s < p.B; s += gridDim.x) {
    const int len = __ldg(p.context_lens + s);
    const int nodes = p.tree_lens ? __ldg(p.tree_lens + s) : p.q_len;
    int flags = 0;
    if (len < 0 || len > p.MBS * p.BS || nodes < 0 || nodes > p.q_len || (len > 0 && len < nodes))
      flags |= PKV_DEV_BAD_CONTEXT_LEN;
    const int blocks = (min(max(len, 0), p.MBS * p.BS) + p.BS - 1) / p.BS;
    for (int j = threadIdx.x; j < blocks; j += kJoinThreads) {
      const int id = __ldg(p.block_tables + size_t(s) * p.MBS + j);
      if (id < 0 || id >= p.NB) flags |= PKV_DEV_BAD_BLOCK_ID;
    }
    if (__syncthreads_or(flags)) {
      if (flags) atomicOr(p.status, flags);
      zero_rows(p, s, 0, 0, 1);
    }
  }
}

cudaError_t launch_tree_join(const TreeParams& p, int grid, cudaStream_t stream) {
  const void* fn = p.D == 128 ? reinterpret_cast<const void*>(&tree_join_kernel<128>)
                              : reinterpret_cast<const void*>(&tree_join_kernel<64>);
  TreeParams copy = p;
  int G = grid;
  void* args[] = {&copy, &G};
  const int zeros = p.B < kZeroCtas ? p.B : kZeroCtas;
  cudaError_t e = launch_pdl(fn, dim3(unsigned(grid + zeros), 256 / kJoinRows),
                             dim3(kJoinThreads), args, 0, stream);
  if (e != cudaSuccess || !p.status) return e;
  void* check_args[] = {&copy};
  return launch_pdl(reinterpret_cast<const void*>(&tree_check_kernel),
                    dim3(unsigned(p.B < 4 * kZeroCtas ? p.B : 4 * kZeroCtas)), dim3(kJoinThreads),
                    check_args, 0, stream);
}

}  // namespace pkv
