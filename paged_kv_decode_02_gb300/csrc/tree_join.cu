// tree_join.cu -- what follows the tree attention (tree.cuh): records of items cut between two
// CTAs' stretches are joined, rows past each tree's tiles become zeros, and, with a status word,
// every sequence is checked.
#include "join.cuh"
#include "tree.cuh"

namespace pkv {

namespace {
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

// CTA (c, y), c < G: rows 32 y .. of the item that CTA c's stretch begins and does not end. A row
// takes D / 4 lanes, a quad of columns each. The CTAs after those zero what no tile covers.
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
  constexpr int R = kJoinRows * Q / kJoinThreads;  // rows of a thread
  const int dq = threadIdx.x % Q;
  int row[R];
  float4 o[R];
  float L[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    row[i] = blockIdx.y * kJoinRows + threadIdx.x / Q + i * (kJoinThreads / Q);
  join_parts<D>(p.cuts, p.part_ml, p.part_o, blockIdx.x, G, cut.slot, row, dq, o, L);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int X = row[i] >> 7, r = row[i] & 127;
    const int rt = r / p.g, node = (2 * pr + X) * p.tpt + rt;
    if (row[i] >= rows || rt >= p.tpt || node >= p.q_len) continue;
    const float inv = L[i] > 0.f ? 1.f / L[i] : L[i] == 0.f ? 0.f : L[i];  // (NaN stays)
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) +
                         ((size_t(cut.s) * p.q_len + node) * p.Hq + hv * p.g + r % p.g) * D;
    reinterpret_cast<uint2*>(out)[dq] =
        make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv),
                   pack_bf16x2(o[i].z * inv, o[i].w * inv));
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
