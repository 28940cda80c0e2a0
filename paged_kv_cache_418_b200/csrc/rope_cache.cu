// rope_cache.cu -- append a step's K and V rows to the paged cache with the
// rotary position embedding applied on the way.
//
// Rotation of one head of one token at position p, over pairs (x_a, x_b) of its
// first rot elements (a = i, b = i + rot / 2, or a = 2i, b = 2i + 1):
//   x_a' = x_a cos[p][i] - x_b sin[p][i],   x_b' = x_b cos[p][i] + x_a sin[p][i]
// in fp32 with every product and sum rounded (no fused multiply-add): the result
// is then a fixed sequence of roundings, which decides an 8-bit code the same
// way for every caller and checker. Query heads are rotated to query_out, key
// heads on their way into the pool, value heads only move.
//
// Both kernels move each element once: (Hq + 2 Hkv) D elements read and written
// per token, a row of cosines and sines, and no second pass over q or k.
#include <cfloat>

#include "pa_internal.h"

namespace pa {

namespace {

// 8 consecutive elements of T, widened to fp32.
template <typename T> __device__ __forceinline__ void load8(const T* p, float* f) {
#pragma unroll
  for (int c = 0; c < 8 / Vec<T>::N; ++c)
    widen16<T>(*reinterpret_cast<const uint4*>(p + c * Vec<T>::N), f + c * Vec<T>::N);
}

__device__ __forceinline__ uint32_t pack2(float a, float b, const __half*) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 fp32 values rounded to T and stored to 8 consecutive elements.
template <typename T> __device__ __forceinline__ void store8(T* p, const float* f) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1], p), pack2(f[2], f[3], p),
                                              pack2(f[4], f[5], p), pack2(f[6], f[7], p));
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// 8 fp32 values over the pool's scale as E4M3 codes.
__device__ __forceinline__ void store8_codes(uint8_t* p, const float* f, float scale) {
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    w[k] = e4m3x2(__fdiv_rn(f[4 * k], scale), __fdiv_rn(f[4 * k + 1], scale)) |
           (e4m3x2(__fdiv_rn(f[4 * k + 2], scale), __fdiv_rn(f[4 * k + 3], scale)) << 16);
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float ra = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  const float rb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = ra;
  b = rb;
}

}  // namespace

// One item is 16 elements of one head: 8 pairs of the rotated part, or 16
// elements behind it. blockIdx.x = token; the CTA's threads stride the token's
// items (query heads, key heads, value heads), and as the stride is a multiple
// of a head's items a thread keeps its place in the head: its 8 cosines and
// sines are loaded once for all its heads. blockIdx.y splits the heads when
// there are few tokens.
template <typename TS, bool IL>
__global__ void __launch_bounds__(256)
rope_and_cache_kernel(const RopeArgs a) {
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x;
  const int64_t slot = a.slot_mapping[t];
  if (slot < 0) return;                                   // padding token
  const int64_t pos = a.positions[t];
  const bool bad_slot = slot >= (int64_t)a.num_blocks * a.bs;
  if (bad_slot || pos < 0 || pos >= a.max_pos) {
    if (threadIdx.x == 0 && blockIdx.y == 0)
      flag_error(a.err_flag, bad_slot ? PA_DEV_BAD_SLOT : PA_DEV_BAD_POS);
    return;
  }
  const int per_head = a.D / 16;                          // 4 or 8
  const int c = threadIdx.x % per_head;
  const int half = a.rot / 2;
  const bool turned = c < half / 8;
  float cs[8], sn[8];
  if (turned) {
    const float* row = a.cos_sin + (size_t)pos * a.rot + 8 * c;
    load8<float>(row, cs);
    load8<float>(row + half, sn);
  }
  // the item's two runs of 8 elements
  const int e0 = turned && !IL ? 8 * c : 16 * c;
  const int e1 = turned && !IL ? half + 8 * c : 16 * c + 8;
  const int heads = a.Hq + 2 * a.Hkv;
  const int step = blockDim.x / per_head;
  for (int h = threadIdx.x / per_head + blockIdx.y * step; h < heads; h += step * gridDim.y) {
    const bool isq = h < a.Hq, isv = h >= a.Hq + a.Hkv;
    const int hh = isq ? h : isv ? h - a.Hq - a.Hkv : h - a.Hq;
    const TS* src = isq ? static_cast<const TS*>(a.query) + (size_t)t * a.q_stride
                  : isv ? static_cast<const TS*>(a.value) + (size_t)t * a.v_stride
                        : static_cast<const TS*>(a.key) + (size_t)t * a.k_stride;
    src += (size_t)hh * a.D;
    float f[16];
    load8<TS>(src + e0, f);
    load8<TS>(src + e1, f + 8);
    if (turned && !isv) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (IL) rotate(f[2 * i], f[2 * i + 1], cs[i], sn[i]);
        else rotate(f[i], f[8 + i], cs[i], sn[i]);
      }
    }
    if (isq) {
      TS* dst = static_cast<TS*>(a.query_out) + (size_t)t * a.qo_stride + (size_t)hh * a.D;
      store8<TS>(dst + e0, f);
      store8<TS>(dst + e1, f + 8);
    } else {
      const size_t row = ((size_t)slot * a.Hkv + hh) * a.D;
      void* pool = isv ? a.value_cache : a.key_cache;
      if (isv ? a.v_fp8 : a.k_fp8) {
        const float scale = isv ? a.v_scale : a.k_scale;
        store8_codes(static_cast<uint8_t*>(pool) + row + e0, f, scale);
        store8_codes(static_cast<uint8_t*>(pool) + row + e1, f + 8, scale);
      } else {
        store8<TS>(static_cast<TS*>(pool) + row + e0, f);
        store8<TS>(static_cast<TS*>(pool) + row + e1, f + 8);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Append to the block-scaled 8-bit cache.
//
// A physical block holds, per KV head, E4M3 codes times one power of two
// s = 2^e. Rows enter with the smallest s that holds their largest finite
// magnitude (amax / s <= 448): a power of two makes x / s exact, so a code is
// one rounding of the value, and moving a block to a larger scale only rounds
// what falls under the E4M3 grid. A block whose offset 0 is written starts anew
// (its former tenant's scale is dropped); any other block's scale only grows,
// and when it does the rows that this call does not write are rounded to it.
//
// A run is the consecutive tokens that share a physical block (at most one
// block's rows); its first token's CTAs own the block: one warp per (KV head,
// K or V) reads the run's rows twice (the largest magnitude, then the codes;
// the second read hits L1), so scales and codes need no second launch and no
// atomics. Every CTA also rotates its share of its token's query heads.

namespace {

// A lane's 4 elements of a row of D: pair slots j = 2 l and 2 l + 1 of the
// head's D / 2 pairs (l = lane within the row's D / 4 lanes).
struct PairSlot {
  int e0, e1;          // first of two adjacent elements of each run
  bool turned;
};
template <bool IL>
__device__ __forceinline__ PairSlot pair_slot(int l, int rot) {
  const int j = 2 * l, half = rot / 2;
  PairSlot s;
  s.turned = j < half;
  if (s.turned && !IL) { s.e0 = j; s.e1 = half + j; }
  else { s.e0 = 2 * j; s.e1 = 2 * j + 2; }     // interleaved, or behind the rotated part
  return s;
}

template <typename TS> __device__ __forceinline__ void load2(const TS* p, float* f) {
  if constexpr (sizeof(TS) == 4) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x; f[1] = v.y;
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    if constexpr (sizeof(TS) == 2) {
      if (std::is_same<TS, __half>::value) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w));
        f[0] = v.x; f[1] = v.y;
      } else {
        f[0] = __uint_as_float(w << 16);
        f[1] = __uint_as_float(w & 0xffff0000u);
      }
    }
  }
}

// This lane's 4 values of token tok's row (rotated for a key head).
template <typename TS, bool IL>
__device__ __forceinline__ void row4(const RopeArgs& a, const TS* src, const PairSlot& s, bool rot,
                                     int64_t pos, int l, float* f) {
  load2<TS>(src + s.e0, f);
  load2<TS>(src + s.e1, f + 2);
  if (rot && s.turned) {
    const float* cs = a.cos_sin + (size_t)pos * a.rot + 2 * l;
    const float2 c = *reinterpret_cast<const float2*>(cs);
    const float2 n = *reinterpret_cast<const float2*>(cs + a.rot / 2);
    if (IL) {
      rotate(f[0], f[1], c.x, n.x);
      rotate(f[2], f[3], c.y, n.y);
    } else {
      rotate(f[0], f[2], c.x, n.x);
      rotate(f[1], f[3], c.y, n.y);
    }
  }
}

}  // namespace

template <typename TS, bool IL>
__global__ void __launch_bounds__(256)
rope_and_cache_blk8_kernel(const RopeArgs a) {
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t slots = (int64_t)a.num_blocks * a.bs;
  const int64_t slot = a.slot_mapping[t];
  if (slot < 0) return;                                   // padding token
  if (slot >= slots) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(a.err_flag, PA_DEV_BAD_SLOT);
    return;
  }
  const bool turn = a.cos_sin != nullptr;
  auto pos_ok = [&](int64_t p) { return !turn || (p >= 0 && p < a.max_pos); };

  // ---- this token's query heads, split over blockIdx.y
  const int64_t pos = turn ? a.positions[t] : 0;
  if (!pos_ok(pos)) {
    if (threadIdx.x == 0 && blockIdx.y == 0) flag_error(a.err_flag, PA_DEV_BAD_POS);
  } else if (turn) {
    const int per_head = a.D / 16;
    const int c = threadIdx.x % per_head;
    const int half = a.rot / 2;
    const bool turned = c < half / 8;
    const int e0 = turned && !IL ? 8 * c : 16 * c;
    const int e1 = turned && !IL ? half + 8 * c : 16 * c + 8;
    const int step = blockDim.x / per_head;
    // blockIdx.y takes a contiguous share of the heads
    const int share = (a.Hq + gridDim.y - 1) / gridDim.y;
    const int h1 = min(a.Hq, ((int)blockIdx.y + 1) * share);
    for (int h = blockIdx.y * share + threadIdx.x / per_head; h < h1; h += step) {
      const TS* src = static_cast<const TS*>(a.query) + (size_t)t * a.q_stride + (size_t)h * a.D;
      float f[16], cs[8], sn[8];
      load8<TS>(src + e0, f);
      load8<TS>(src + e1, f + 8);
      if (turned) {
        const float* row = a.cos_sin + (size_t)pos * a.rot + 8 * c;
        load8<float>(row, cs);
        load8<float>(row + half, sn);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (IL) rotate(f[2 * i], f[2 * i + 1], cs[i], sn[i]);
          else rotate(f[i], f[8 + i], cs[i], sn[i]);
        }
      }
      TS* dst = static_cast<TS*>(a.query_out) + (size_t)t * a.qo_stride + (size_t)h * a.D;
      store8<TS>(dst + e0, f);
      store8<TS>(dst + e1, f + 8);
    }
  }

  // ---- the block of the run that starts at this token
  const int64_t block = slot / a.bs;
  if (t > 0) {
    const int64_t before = a.slot_mapping[t - 1];
    if (before >= 0 && before < slots && before / a.bs == block) return;
  }
  // lane i: token t + i of the run (off < 0: not of the run, or its position is bad)
  int off = -1;
  bool same = false;
  int64_t lpos = 0;
  if (lane < a.bs && t + lane < a.T) {
    const int64_t s = a.slot_mapping[t + lane];
    same = s >= 0 && s < slots && s / a.bs == block;
    if (same) {
      off = (int)(s - block * a.bs);
      if (turn) lpos = a.positions[t + lane];
      if (!pos_ok(lpos)) off = -1;
    }
  }
  const uint32_t run = __ballot_sync(0xffffffffu, same);
  const int n = run == 0xffffffffu ? 32 : __ffs(~run) - 1;      // tokens of the run
  if (lane >= n) off = -1;
  const uint32_t written = __reduce_or_sync(0xffffffffu, off >= 0 ? 1u << off : 0u);
  if (!written) return;

  const int lpr = a.D / 4;                     // lanes per row: 16 or 32
  const int rpw = 32 / lpr;                    // rows a warp takes at once
  const int l = lane % lpr, sub = lane / lpr;
  const PairSlot ps = pair_slot<IL>(l, a.rot);
  for (int u = blockIdx.y * 8 + warp; u < 2 * a.Hkv; u += 8 * gridDim.y) {
    const bool isv = u >= a.Hkv;
    const int h = isv ? u - a.Hkv : u;
    const int64_t stride = isv ? a.v_stride : a.k_stride;
    const TS* src = static_cast<const TS*>(isv ? a.value : a.key) + (size_t)t * stride + (size_t)h * a.D;
    float* scales = isv ? a.v_scales : a.k_scales;
    const size_t si = (size_t)block * a.Hkv + h;
    const bool fresh = written & 1u;
    const float old = fresh ? 0.f : scales[si];
    // the largest finite magnitude of the run's rows
    float top = 0.f;
    for (int i0 = 0; i0 < n; i0 += 4 * rpw) {
      float f[4][4];
      bool on[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * rpw + sub;
        on[k] = __shfl_sync(0xffffffffu, off, i & 31) >= 0 && i < n;
        const int64_t p = __shfl_sync(0xffffffffu, lpos, i & 31);
        if (on[k]) row4<TS, IL>(a, src + (size_t)i * stride, ps, turn && !isv, p, l, f[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (!on[k]) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float m = fabsf(f[k][e]);
          top = m <= FLT_MAX ? fmaxf(top, m) : top;
        }
      }
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    float scale = block_scale_for(top);
    if (!fresh) {
      if (!block_scale_ok(old)) {
        if (lane == 0) flag_error(a.err_flag, PA_DEV_BAD_SCALE);
        continue;
      }
      scale = fmaxf(scale, old);
    }
    const float inv = __fdiv_rn(1.f, scale);     // a power of two: exact
    uint8_t* pool = static_cast<uint8_t*>(isv ? a.value_cache : a.key_cache) +
                    ((size_t)block * a.bs * a.Hkv + h) * a.D;
    const size_t pitch = (size_t)a.Hkv * a.D;
    for (int i0 = 0; i0 < n; i0 += 4 * rpw) {
      float f[4][4];
      int o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * rpw + sub;
        o[k] = __shfl_sync(0xffffffffu, off, i & 31);
        if (i >= n) o[k] = -1;
        const int64_t p = __shfl_sync(0xffffffffu, lpos, i & 31);
        if (o[k] >= 0) row4<TS, IL>(a, src + (size_t)i * stride, ps, turn && !isv, p, l, f[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (o[k] < 0) continue;
        uint8_t* row = pool + o[k] * pitch;
        const uint32_t c0 = e4m3x2(__fmul_rn(f[k][0], inv), __fmul_rn(f[k][1], inv));
        const uint32_t c1 = e4m3x2(__fmul_rn(f[k][2], inv), __fmul_rn(f[k][3], inv));
        *reinterpret_cast<uint16_t*>(row + ps.e0) = (uint16_t)c0;
        *reinterpret_cast<uint16_t*>(row + ps.e1) = (uint16_t)c1;
      }
    }
    if (!fresh && scale > old) {
      // the block's other rows, rounded to the larger scale
      const float ratio = __fdiv_rn(old, scale);
      for (int r = sub; r < a.bs; r += rpw) {
        if ((written >> r) & 1u) continue;
        uint32_t* p = reinterpret_cast<uint32_t*>(pool + r * pitch) + l;
        const uint32_t w = *p;
        uint32_t out = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
              static_cast<__nv_fp8x2_storage_t>((w >> (16 * k)) & 0xffffu), __NV_E4M3);
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hr));
          out |= e4m3x2(__fmul_rn(v.x, ratio), __fmul_rn(v.y, ratio)) << (16 * k);
        }
        *p = out;
      }
    }
    if (lane == 0) scales[si] = scale;
  }
}

// Scales of whole blocks, beside pa_copy_blocks / pa_swap_blocks: one thread per
// (pair, KV head).
__global__ void copy_scales_kernel(float* __restrict__ dst_k, float* __restrict__ dst_v,
                                   const float* __restrict__ src_k, const float* __restrict__ src_v,
                                   const int64_t* __restrict__ block_mapping, long long n, int Hkv,
                                   int src_blocks, int dst_blocks, uint32_t* err_flag) {
  pdl_trigger();
  pdl_wait();
  const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  if (i >= n) return;
  const long long p = i / Hkv;
  const int h = (int)(i - p * Hkv);
  const int64_t src = block_mapping[2 * p], dst = block_mapping[2 * p + 1];
  if (src < 0 || src >= src_blocks || dst < 0 || dst >= dst_blocks) {
    if (h == 0) flag_error(err_flag, PA_DEV_BAD_PAIR);
    return;
  }
  dst_k[(size_t)dst * Hkv + h] = src_k[(size_t)src * Hkv + h];
  dst_v[(size_t)dst * Hkv + h] = src_v[(size_t)src * Hkv + h];
}

int launch_copy_scales(float* dst_k, float* dst_v, const float* src_k, const float* src_v,
                       const int64_t* block_mapping, int num_pairs, int Hkv, int src_blocks,
                       int dst_blocks, uint32_t* err_flag, cudaStream_t stream) {
  const long long n = (long long)num_pairs * Hkv;
  const cudaError_t e =
      launch_k(copy_scales_kernel, dim3((unsigned)((n + 127) / 128)), dim3(128), 0, stream, dst_k,
               dst_v, src_k, src_v, block_mapping, n, Hkv, src_blocks, dst_blocks, err_flag);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

namespace {

template <typename TS>
int launch_rope_t(const RopeArgs& a, bool blk8, cudaStream_t stream) {
  // blk8: one warp per (KV head, K or V). Else: split the heads only while the
  // tokens leave SMs empty.
  int y;
  if (blk8) {
    y = (2 * a.Hkv + 7) / 8;
  } else {
    const int items = (a.Hq + 2 * a.Hkv) * (a.D / 16);
    y = (items + 255) / 256;
    while (y > 1 && (long long)a.T * y > 8 * kSMs) --y;
  }
  const dim3 grid((unsigned)a.T, (unsigned)y), block(256);
  cudaError_t e;
  if (blk8)
    e = a.interleaved ? launch_k(rope_and_cache_blk8_kernel<TS, true>, grid, block, 0, stream, a)
                      : launch_k(rope_and_cache_blk8_kernel<TS, false>, grid, block, 0, stream, a);
  else
    e = a.interleaved ? launch_k(rope_and_cache_kernel<TS, true>, grid, block, 0, stream, a)
                      : launch_k(rope_and_cache_kernel<TS, false>, grid, block, 0, stream, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

int launch_rope_and_cache(const RopeArgs& a, int src_dtype, bool blk8, cudaStream_t stream) {
  switch (src_dtype) {
    case PA_F32: return launch_rope_t<float>(a, blk8, stream);
    case PA_F16: return launch_rope_t<__half>(a, blk8, stream);
    case PA_BF16: return launch_rope_t<__nv_bfloat16>(a, blk8, stream);
  }
  return PA_ERR_DTYPE;
}

}  // namespace pa
