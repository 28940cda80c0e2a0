// prefill_window.cu -- paged prefill over a sliding window and a few first tokens,
// and over the block-scaled 8-bit cache: the prefill kernel's run-time-windowed
// instances (group size at run time too).
//
// New token at position p attends keys t <= p with t > p - window or t < sinks. A
// unit's 128 / G tokens walk the 128-key tiles that hold a key some of them
// attends: the first tokens' tiles, then those from its first token's window on.
// Blocks of those tiles that no row attends are not loaded (nor is their table
// entry read), a row's mask is one bit per key of a 32-key chunk.
#include "prefill_fa.cuh"

namespace pa {

namespace {

template <bool K8, bool V8, bool BSC>
int launch_x(const FaArgs& a, int dtype, const CUtensorMap& q, const CUtensorMap& k,
             const CUtensorMap& v, cudaStream_t stream) {
  if (dtype == PA_BF16)
    return a.bs == 16 ? launch_fa_t<1, 16, 0, K8, V8, true, BSC>(a, q, k, v, stream)
                      : launch_fa_t<1, 32, 0, K8, V8, true, BSC>(a, q, k, v, stream);
  return a.bs == 16 ? launch_fa_t<0, 16, 0, K8, V8, true, BSC>(a, q, k, v, stream)
                    : launch_fa_t<0, 32, 0, K8, V8, true, BSC>(a, q, k, v, stream);
}

}  // namespace

int launch_prefill_window(const PrefillLaunch& p, cudaStream_t stream) {
  const int G = p.Hq / p.Hkv;
  const bool k8 = p.k_dtype == PA_FP8_E4M3, v8 = p.v_dtype == PA_FP8_E4M3;
  CUtensorMap q, k, v;
  if (!make_fa_maps(p, G, k8, v8, &q, &k, &v)) return PA_ERR_CUDA;
  FaArgs a{};
  a.out = p.out;
  a.out_dtype = p.out_dtype;
  a.block_tables = p.block_tables;
  a.max_blocks = p.max_blocks;
  a.context_lens = p.context_lens;
  a.query_start = p.query_start;
  a.B = p.B; a.Hq = p.Hq; a.Hkv = p.Hkv; a.bs = p.bs; a.num_blocks = p.num_blocks;
  const int tpu = kM / G;
  a.chunks = p.max_query_len / tpu + (p.max_query_len % tpu != 0);
  a.scale_log2 = p.scale_log2;
  a.v_scale = v8 ? p.v_scale : 1.f;
  a.max_context_len = p.max_context_len;
  a.err_flag = p.err_flag;
  a.window = p.window; a.sinks = p.sinks;
  a.k_scales = p.k_scales; a.v_scales = p.v_scales;
  if (p.k_scales) return launch_x<true, true, true>(a, p.dtype, q, k, v, stream);
  if (k8 && v8) return launch_x<true, true, false>(a, p.dtype, q, k, v, stream);
  if (k8) return launch_x<true, false, false>(a, p.dtype, q, k, v, stream);
  if (v8) return launch_x<false, true, false>(a, p.dtype, q, k, v, stream);
  return launch_x<false, false, false>(a, p.dtype, q, k, v, stream);
}

}  // namespace pa
