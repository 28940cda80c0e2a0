// pa_api_window.cu -- the extern "C" boundary of the rotary append, the windowed
// attention and the block-scaled 8-bit cache: argument checks, workspace
// carve-up, launches.
#include <climits>

#include "pa_internal.h"

using namespace pa;

namespace {

// Shared body of pa_rope_and_cache_kv and pa_rope_and_cache_blk8 (blk8: the
// pools hold codes with a scale per block and KV head, and the rotation may be
// left out).
int rope_impl(RopeArgs a, int src_dtype, bool blk8, void* stream) {
  if (src_dtype < PA_F32 || src_dtype > PA_BF16) return PA_ERR_DTYPE;
  if (a.T < 0 || a.Hq < 0 || a.Hkv <= 0 || a.D <= 0 || a.bs <= 0 || a.num_blocks < 0 || a.max_pos < 0)
    return PA_ERR_SHAPE;
  if (!supported_shape(a.Hkv, a.Hkv, a.D, a.bs)) return PA_ERR_UNSUPPORTED;
  const bool turn = a.cos_sin != nullptr;
  if (turn && (a.rot <= 0 || a.rot > a.D || a.rot % 16)) return PA_ERR_SHAPE;
  if (!blk8 && ((a.k_fp8 && !scale_ok(a.k_scale)) || (a.v_fp8 && !scale_ok(a.v_scale))))
    return PA_ERR_SHAPE;
  if (a.Hq > 65535 || a.Hkv > 65535) return PA_ERR_UNSUPPORTED;
  // token strides: a token's heads are dense, tokens do not overlap, rows start
  // on 16 bytes
  const long long es = esize_of(src_dtype);
  auto stride_ok = [&](long long s, int heads) {
    return s >= (long long)heads * a.D && s <= LLONG_MAX / (8LL * (a.T > 0 ? a.T : 1)) && s * es % 16 == 0;
  };
  if (!stride_ok(a.k_stride, a.Hkv) || !stride_ok(a.v_stride, a.Hkv)) return PA_ERR_SHAPE;
  if (a.Hq > 0 && (!stride_ok(a.q_stride, a.Hq) || !stride_ok(a.qo_stride, a.Hq))) return PA_ERR_SHAPE;
  // in place means row by row: with two strides one token's result would land on another's input
  if (a.Hq > 0 && a.T > 1 && a.query && a.query == a.query_out && a.q_stride != a.qo_stride) return PA_ERR_SHAPE;
  if (a.T == 0) return PA_OK;
  if (!a.key || !a.value || !a.key_cache || !a.value_cache || !a.slot_mapping) return PA_ERR_NULL;
  if (a.Hq > 0 && (!a.query || !a.query_out)) return PA_ERR_NULL;
  if (blk8 && (!a.k_scales || !a.v_scales)) return PA_ERR_NULL;
  if (turn != (a.positions != nullptr)) return PA_ERR_NULL;
  if (!turn && (!blk8 || a.Hq > 0)) return PA_ERR_NULL;    // nothing to do to a query without a rotation
  if (!aligned16(a.key) || !aligned16(a.value) || !aligned16(a.key_cache) ||
      !aligned16(a.value_cache) || !aligned16(a.cos_sin) ||
      (a.Hq > 0 && (!aligned16(a.query) || !aligned16(a.query_out))))
    return PA_ERR_ALIGN;
  if (!turn) a.rot = 0;
  return launch_rope_and_cache(a, src_dtype, blk8, static_cast<cudaStream_t>(stream));
}

// Shared body of the windowed and block-scaled decodes (k_scales NULL: per-pool
// element types and scales).
int decode_window_impl(void* out, int out_dtype, const void* query, int q_dtype,
                       const void* key_cache, int k_dtype, float k_scale, const void* value_cache,
                       int v_dtype, float v_scale, bool blk8, const float* k_scales,
                       const float* v_scales, const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* context_lens, int B, int Hq, int Hkv, int D, int block_size,
                       int num_blocks, float scale, int window, int num_sinks, int max_context_len,
                       void* workspace, size_t workspace_bytes, uint32_t* err_flag, void* stream) {
  if (q_dtype < PA_F32 || q_dtype > PA_BF16) return PA_ERR_DTYPE;
  if (!pool_types_ok(q_dtype, k_dtype, v_dtype)) return PA_ERR_DTYPE;
  if (out_dtype != PA_F32 && out_dtype != q_dtype) return PA_ERR_DTYPE;
  if (B < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || block_size <= 0 || num_blocks < 0 ||
      max_blocks_per_seq <= 0 || max_context_len < 0 || window < (blk8 ? 0 : 1) || num_sinks < 0)
    return PA_ERR_SHAPE;
  if (!supported_shape(Hq, Hkv, D, block_size)) return PA_ERR_UNSUPPORTED;
  const bool k8 = !blk8 && k_dtype == PA_FP8_E4M3, v8 = !blk8 && v_dtype == PA_FP8_E4M3;
  if (!std::isfinite(scale) || (k8 && !scale_ok(k_scale)) || (v8 && !scale_ok(v_scale)))
    return PA_ERR_SHAPE;
  if (B > 65535 || Hq > 65535) return PA_ERR_UNSUPPORTED;
  if (B == 0) return PA_OK;
  if (num_blocks == 0) return PA_ERR_SHAPE;
  if (!out || !query || !key_cache || !value_cache || !block_tables || !context_lens)
    return PA_ERR_NULL;
  if (blk8 && (!k_scales || !v_scales)) return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache))
    return PA_ERR_ALIGN;
  WinArgs a{};
  a.out = out; a.out_dtype = out_dtype; a.q = query; a.q_dtype = q_dtype;
  a.k_cache = key_cache; a.v_cache = value_cache; a.k_dtype = k_dtype; a.v_dtype = v_dtype;
  a.k_scales = blk8 ? k_scales : nullptr;
  a.v_scales = blk8 ? v_scales : nullptr;
  a.block_tables = block_tables; a.max_blocks = max_blocks_per_seq; a.context_lens = context_lens;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.bs = block_size; a.num_blocks = num_blocks;
  a.scale_log2 = scale * kLog2e * (k8 ? k_scale : 1.f);
  a.v_scale = v8 ? v_scale : 1.f;
  a.window = window; a.sinks = num_sinks; a.max_context_len = max_context_len;
  a.err_flag = err_flag;
  plan_window(a);
  const size_t need = window_scratch_bytes(a);
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PA_ERR_WORKSPACE;
  carve_window(a, static_cast<char*>(workspace));
  a.wait_ns = tc_wait_ns();
  a.test_withhold = tc_test_withhold_q();
  return launch_decode_window(a, static_cast<cudaStream_t>(stream));
}

// Shared body of the windowed and block-scaled prefills.
int prefill_window_impl(void* out, int out_dtype, const void* query, int q_dtype,
                        const void* key_cache, int k_dtype, float k_scale, const void* value_cache,
                        int v_dtype, float v_scale, bool blk8, const float* k_scales,
                        const float* v_scales, const int32_t* block_tables, int max_blocks_per_seq,
                        const int32_t* context_lens, const int32_t* query_start, int B, int T,
                        int max_query_len, int Hq, int Hkv, int D, int block_size, int num_blocks,
                        float scale, int window, int num_sinks, int max_context_len,
                        uint32_t* err_flag, void* stream) {
  if (q_dtype < PA_F32 || q_dtype > PA_BF16) return PA_ERR_DTYPE;
  if (out_dtype != PA_F32 && out_dtype != q_dtype) return PA_ERR_DTYPE;
  const bool k8 = k_dtype == PA_FP8_E4M3, v8 = v_dtype == PA_FP8_E4M3;
  if ((!k8 && k_dtype != q_dtype) || (!v8 && v_dtype != q_dtype)) return PA_ERR_DTYPE;
  if (B < 0 || T < 0 || max_query_len < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || block_size <= 0 ||
      num_blocks < 0 || max_blocks_per_seq <= 0 || max_context_len < 0 ||
      window < (blk8 ? 0 : 1) || num_sinks < 0)
    return PA_ERR_SHAPE;
  if (!supported_shape(Hq, Hkv, D, block_size) ||
      !prefill_fa_supported(q_dtype, Hq, Hkv, D, block_size))
    return PA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale)) return PA_ERR_SHAPE;
  if (!blk8 && ((k8 && !scale_ok(k_scale)) || (v8 && !scale_ok(v_scale)))) return PA_ERR_SHAPE;
  if (B == 0 || T == 0 || max_query_len == 0) return PA_OK;
  if (num_blocks == 0) return PA_ERR_SHAPE;
  if (!out || !query || !key_cache || !value_cache || !block_tables || !context_lens || !query_start)
    return PA_ERR_NULL;
  if (blk8 && (!k_scales || !v_scales)) return PA_ERR_NULL;
  if (!aligned16(out) || !aligned16(query) || !aligned16(key_cache) || !aligned16(value_cache))
    return PA_ERR_ALIGN;
  PrefillLaunch p{};
  p.out = out; p.out_dtype = out_dtype; p.q = query;
  p.k_cache = key_cache; p.v_cache = value_cache; p.dtype = q_dtype;
  p.k_dtype = k_dtype; p.v_dtype = v_dtype;
  p.v_scale = v8 && !blk8 ? v_scale : 1.f;
  p.block_tables = block_tables; p.max_blocks = max_blocks_per_seq;
  p.context_lens = context_lens; p.query_start = query_start;
  // (a bound past all the tokens would only add chunks that hold none, each walked by every CTA)
  p.B = B; p.T = T; p.max_query_len = max_query_len < T ? max_query_len : T; p.Hq = Hq; p.Hkv = Hkv; p.bs = block_size;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * kLog2e * (k8 && !blk8 ? k_scale : 1.f);
  p.max_context_len = max_context_len;
  p.err_flag = err_flag;
  p.window = window; p.sinks = num_sinks;
  p.k_scales = blk8 ? k_scales : nullptr;
  p.v_scales = blk8 ? v_scales : nullptr;
  return launch_prefill_window(p, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int pa_rope_and_cache_kv(void* query_out, int64_t query_out_stride, const void* query,
                         int64_t query_stride, const void* key, int64_t key_stride,
                         const void* value, int64_t value_stride, int src_dtype,
                         const int64_t* positions, const float* cos_sin, int max_positions,
                         int rot_dim, int interleaved, void* key_cache, int k_dtype, float k_scale,
                         void* value_cache, int v_dtype, float v_scale,
                         const int64_t* slot_mapping, int T, int Hq, int Hkv, int D,
                         int block_size, int num_blocks, uint32_t* err_flag, void* stream) {
  const bool kf = k_dtype == PA_FP8_E4M3, vf = v_dtype == PA_FP8_E4M3;
  if ((!kf && k_dtype != src_dtype) || (!vf && v_dtype != src_dtype)) return PA_ERR_DTYPE;
  RopeArgs a{};
  a.query_out = query_out; a.query = query; a.key = key; a.value = value;
  a.qo_stride = query_out_stride; a.q_stride = query_stride; a.k_stride = key_stride;
  a.v_stride = value_stride;
  a.positions = positions; a.cos_sin = cos_sin; a.max_pos = max_positions; a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.key_cache = key_cache; a.value_cache = value_cache;
  a.k_fp8 = kf; a.v_fp8 = vf; a.k_scale = k_scale; a.v_scale = v_scale;
  a.slot_mapping = slot_mapping;
  a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.bs = block_size; a.num_blocks = num_blocks;
  a.err_flag = err_flag;
  return rope_impl(a, src_dtype, false, stream);
}

int pa_rope_and_cache_blk8(void* query_out, int64_t query_out_stride, const void* query,
                           int64_t query_stride, const void* key, int64_t key_stride,
                           const void* value, int64_t value_stride, int src_dtype,
                           const int64_t* positions, const float* cos_sin, int max_positions,
                           int rot_dim, int interleaved, void* key_cache, void* value_cache,
                           float* k_scales, float* v_scales, const int64_t* slot_mapping, int T,
                           int Hq, int Hkv, int D, int block_size, int num_blocks,
                           uint32_t* err_flag, void* stream) {
  RopeArgs a{};
  a.query_out = query_out; a.query = query; a.key = key; a.value = value;
  a.qo_stride = query_out_stride; a.q_stride = query_stride; a.k_stride = key_stride;
  a.v_stride = value_stride;
  a.positions = positions; a.cos_sin = cos_sin; a.max_pos = max_positions; a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.key_cache = key_cache; a.value_cache = value_cache;
  a.k_scales = k_scales; a.v_scales = v_scales;
  a.slot_mapping = slot_mapping;
  a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.bs = block_size; a.num_blocks = num_blocks;
  a.err_flag = err_flag;
  return rope_impl(a, src_dtype, true, stream);
}

int pa_copy_scales(float* dst_k_scales, float* dst_v_scales, const float* src_k_scales,
                   const float* src_v_scales, const int64_t* block_mapping, int num_pairs, int Hkv,
                   int src_blocks, int dst_blocks, uint32_t* err_flag, void* stream) {
  if (num_pairs < 0 || Hkv <= 0 || src_blocks < 0 || dst_blocks < 0) return PA_ERR_SHAPE;
  if (Hkv > 65535) return PA_ERR_UNSUPPORTED;
  if (num_pairs == 0) return PA_OK;
  if (!dst_k_scales || !dst_v_scales || !src_k_scales || !src_v_scales || !block_mapping)
    return PA_ERR_NULL;
  return launch_copy_scales(dst_k_scales, dst_v_scales, src_k_scales, src_v_scales, block_mapping,
                            num_pairs, Hkv, src_blocks, dst_blocks, err_flag,
                            static_cast<cudaStream_t>(stream));
}

size_t pa_window_workspace_size(int B, int Hq, int Hkv, int D, int max_context_len, int window,
                                int num_sinks) {
  if (B <= 0 || max_context_len < 0 || window < 0 || num_sinks < 0 || B > 65535 || Hq > 65535 ||
      !supported_shape(Hq, Hkv, D, 16))
    return 0;
  WinArgs a{};
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.D = D; a.max_context_len = max_context_len;
  a.window = window; a.sinks = num_sinks;
  // enough for any pool type
  a.k_dtype = PA_F32;
  plan_window(a);
  const size_t f32 = window_scratch_bytes(a);
  a.k_dtype = PA_F16;
  plan_window(a);
  const size_t other = window_scratch_bytes(a);
  return f32 > other ? f32 : other;
}

int pa_decode_window_kv(void* out, int out_dtype, const void* query, int q_dtype,
                        const void* key_cache, int k_dtype, float k_scale, const void* value_cache,
                        int v_dtype, float v_scale, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* context_lens, int B, int Hq, int Hkv,
                        int D, int block_size, int num_blocks, float scale, int window,
                        int num_sinks, int max_context_len, void* workspace,
                        size_t workspace_bytes, uint32_t* err_flag, void* stream) {
  return decode_window_impl(out, out_dtype, query, q_dtype, key_cache, k_dtype, k_scale,
                            value_cache, v_dtype, v_scale, false, nullptr, nullptr, block_tables,
                            max_blocks_per_seq, context_lens, B, Hq, Hkv, D, block_size,
                            num_blocks, scale, window, num_sinks, max_context_len, workspace,
                            workspace_bytes, err_flag, stream);
}

int pa_decode_blk8(void* out, int out_dtype, const void* query, int q_dtype, const void* key_cache,
                   const void* value_cache, const float* k_scales, const float* v_scales,
                   const int32_t* block_tables, int max_blocks_per_seq,
                   const int32_t* context_lens, int B, int Hq, int Hkv, int D, int block_size,
                   int num_blocks, float scale, int window, int num_sinks, int max_context_len,
                   void* workspace, size_t workspace_bytes, uint32_t* err_flag, void* stream) {
  return decode_window_impl(out, out_dtype, query, q_dtype, key_cache, PA_FP8_E4M3, 1.f,
                            value_cache, PA_FP8_E4M3, 1.f, true, k_scales, v_scales, block_tables,
                            max_blocks_per_seq, context_lens, B, Hq, Hkv, D, block_size,
                            num_blocks, scale, window, num_sinks, max_context_len, workspace,
                            workspace_bytes, err_flag, stream);
}

int pa_prefill_window_kv(void* out, int out_dtype, const void* query, int q_dtype,
                         const void* key_cache, int k_dtype, float k_scale, const void* value_cache,
                         int v_dtype, float v_scale, const int32_t* block_tables,
                         int max_blocks_per_seq, const int32_t* context_lens,
                         const int32_t* query_start, int B, int T, int max_query_len, int Hq,
                         int Hkv, int D, int block_size, int num_blocks, float scale, int window,
                         int num_sinks, int max_context_len, uint32_t* err_flag, void* stream) {
  return prefill_window_impl(out, out_dtype, query, q_dtype, key_cache, k_dtype, k_scale,
                             value_cache, v_dtype, v_scale, false, nullptr, nullptr, block_tables,
                             max_blocks_per_seq, context_lens, query_start, B, T, max_query_len, Hq,
                             Hkv, D, block_size, num_blocks, scale, window, num_sinks,
                             max_context_len, err_flag, stream);
}

int pa_prefill_blk8(void* out, int out_dtype, const void* query, int q_dtype, const void* key_cache,
                    const void* value_cache, const float* k_scales, const float* v_scales,
                    const int32_t* block_tables, int max_blocks_per_seq,
                    const int32_t* context_lens, const int32_t* query_start, int B, int T,
                    int max_query_len, int Hq, int Hkv, int D, int block_size, int num_blocks,
                    float scale, int window, int num_sinks, int max_context_len,
                    uint32_t* err_flag, void* stream) {
  return prefill_window_impl(out, out_dtype, query, q_dtype, key_cache, PA_FP8_E4M3, 1.f,
                             value_cache, PA_FP8_E4M3, 1.f, true, k_scales, v_scales, block_tables,
                             max_blocks_per_seq, context_lens, query_start, B, T, max_query_len, Hq,
                             Hkv, D, block_size, num_blocks, scale, window, num_sinks,
                             max_context_len, err_flag, stream);
}

}  // extern "C"
