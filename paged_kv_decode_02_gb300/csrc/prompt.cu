// prompt.cu -- instantiations of the prompt attention (prompt.cuh) and the kernel that joins
// the records of items cut between two CTAs' stretches.
#include "join.cuh"
#include "prompt.cuh"

namespace pkv {

// CTA (c, y): rows 32 y .. of the item that CTA c's stretch begins and does not end. A row takes
// D / 4 lanes, a quad of columns each.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const PromptParams p, int G) {
  constexpr int Q = D / 4;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const PromptCut cut = p.cuts[blockIdx.x];
  if (!(cut.state & kPromptBegins)) return;
  PromptSeq q;
  q.load(p, cut.s);
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
    const int rt = r / p.g, tok = (2 * cut.i + X) * p.tpt + rt;
    if (rt >= p.tpt || tok >= q.nq) continue;
    const float inv = L[i] > 0.f ? 1.f / L[i] : L[i] == 0.f ? 0.f : L[i];  // (NaN stays)
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) +
                         (long long)(q.q0 + tok) * p.out_stride +
                         (long long)(cut.h * p.g + r % p.g) * D;
    reinterpret_cast<uint2*>(out)[dq] =
        make_uint2(pack_bf16x2(o[i].x * inv, o[i].y * inv),
                   pack_bf16x2(o[i].z * inv, o[i].w * inv));
  }
}

cudaError_t launch_prompt_merge(const PromptParams& p, int grid, cudaStream_t stream) {
  const void* fn = p.D == 128 ? reinterpret_cast<const void*>(&prompt_join_kernel<128>)
                              : reinterpret_cast<const void*>(&prompt_join_kernel<64>);
  PromptParams copy = p;
  int G = grid;
  void* args[] = {&copy, &G};
  return launch_pdl(fn, dim3(unsigned(grid), 256 / kJoinRows), dim3(kJoinThreads), args, 0, stream);
}

bool select_prompt(int D, PromptKernelInfo* info) {
  if (D != 64 && D != 128) return false;
  info->fn = D == 128 ? reinterpret_cast<const void*>(&prompt_attention_kernel<128>)
                      : reinterpret_cast<const void*>(&prompt_attention_kernel<64>);
  info->threads = PromptCfg<128>::kThreads;
  info->keys = D == 128 ? PromptCfg<128>::kKeys : PromptCfg<64>::kKeys;
  info->smem = D == 128 ? PromptCfg<128>::kSmem : PromptCfg<64>::kSmem;
  return true;
}

}  // namespace pkv
