// prompt.cu -- instantiations of the prompt attention (prompt.cuh) and the kernel that joins
// the records of items cut between two CTAs' stretches.
#include "prompt.cuh"

namespace pkv {

namespace {
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;  // rows per CTA
}  // namespace

// CTA (c, y): rows 32 y .. of the item that CTA c's stretch begins and does not end. Its parts
// are that record and the first records of the CTAs after it, up to the one that ends the item;
// they meet at the largest of their maxima. A row takes D / 4 lanes, a quad of columns each.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const PromptParams p, int G) {
  constexpr int Q = D / 4;
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const PromptCut cut = p.cuts[blockIdx.x];
  if (!(cut.state & kPromptBegins)) return;
  PromptSeq q;
  q.load(p, cut.s);
  const int dq = threadIdx.x % Q;
  for (int r0 = threadIdx.x / Q; r0 < kJoinRows; r0 += kJoinThreads / Q) {
    const int row = blockIdx.y * kJoinRows + r0, X = row >> 7, r = row & 127;
    const int rt = r / p.g, tok = (2 * cut.i + X) * p.tpt + rt;
    if (rt >= p.tpt || tok >= q.nq) continue;
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
                         (long long)(q.q0 + tok) * p.out_stride +
                         (long long)(cut.h * p.g + r % p.g) * D;
    reinterpret_cast<uint2*>(out)[dq] =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
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
