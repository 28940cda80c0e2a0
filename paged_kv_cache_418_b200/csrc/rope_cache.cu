// rope_cache.cu -- append a step's K and V rows to the paged cache with the
// rotary position embedding applied on the way.
//
// Rotation of one head of one token at position p, over pairs (x_a, x_b) of its
// first rot elements (a = i, b = i + rot / 2, or a = 2i, b = 2i + 1):
//   x_a' = x_a cos[p][i] - x_b sin[p][i],   x_b' = x_b cos[p][i] + x_a sin[p][i]
// in fp32 with every product and sum rounded (no fused multiply-add): the result
// is then a fixed sequence of roundings, which decides an 8-bit code the same
// way for every caller and reader of it. Query heads are rotated to query_out, key
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

// 8 fp32 values rounded to T and stored to 8 consecutive elements, marked to leave
// L2 first: a chunk's rows (84 MB written at 8 x 512 tokens of 64 + 8 heads) would
// push out each other's lines half-written otherwise (33.7 -> 29.9 us there).
template <typename T> __device__ __forceinline__ void store8(T* p, const float* f) {
  if constexpr (sizeof(T) == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
  } else {
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack2(f[0], f[1], p), pack2(f[2], f[3], p),
                                                   pack2(f[4], f[5], p), pack2(f[6], f[7], p)));
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

// One item is 16 elements of one head: 8 pairs of the rotated part (elements e0 ..
// and e1 ..), or 16 elements behind it. A thread keeps its place c in the head (its
// stride over the heads is a multiple of a head's items), so it loads its 8 cosines
// and sines once per token.
struct Place {
  int e0, e1;          // first elements of the item's two runs of 8
  bool turned;
};
template <bool IL> __device__ __forceinline__ Place place_of(int c, int rot) {
  const int half = rot / 2;
  Place p;
  p.turned = c < half / 8;
  p.e0 = p.turned && !IL ? 8 * c : 16 * c;
  p.e1 = p.turned && !IL ? half + 8 * c : 16 * c + 8;
  return p;
}
// (Past L1: read once. Not through the read-only path: a query may be rotated in
// place.)
__device__ __forceinline__ uint4 ld_row16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

// The item's bytes, as loaded.
template <typename T> struct Item {
  static constexpr int N = 8 * sizeof(T) / 16;
  uint4 v[2 * N];
  __device__ __forceinline__ void load(const T* src, const Place& p) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      v[k] = ld_row16(src + p.e0 + k * Vec<T>::N);
      v[N + k] = ld_row16(src + p.e1 + k * Vec<T>::N);
    }
  }
  __device__ __forceinline__ void widen(float* f) const {
#pragma unroll
    for (int k = 0; k < 2 * N; ++k) widen16<T>(v[k], f + k * Vec<T>::N);
  }
};
template <bool IL> __device__ __forceinline__ void turn(float* f, const float* cs, const float* sn) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (IL) rotate(f[2 * i], f[2 * i + 1], cs[i], sn[i]);
    else rotate(f[i], f[8 + i], cs[i], sn[i]);
  }
}

// Heads [h0, heads) in steps of one token's query | key | value heads, place c in
// each: the loads of U heads are in flight before the first is rotated and stored.
template <typename TS, bool IL, int U>
__device__ __forceinline__ void rope_heads(const RopeArgs& a, int t, int c, int h0, int step, int heads) {
  const Place pl = place_of<IL>(c, a.rot);
  auto source = [&](int h) -> const TS* {
    if (h < a.Hq) return static_cast<const TS*>(a.query) + (size_t)t * a.q_stride + (size_t)h * a.D;
    if (h < a.Hq + a.Hkv)
      return static_cast<const TS*>(a.key) + (size_t)t * a.k_stride + (size_t)(h - a.Hq) * a.D;
    return static_cast<const TS*>(a.value) + (size_t)t * a.v_stride + (size_t)(h - a.Hq - a.Hkv) * a.D;
  };
  Item<TS> it[U];
#pragma unroll
  for (int k = 0; k < U; ++k)
    if (h0 + k * step < heads) it[k].load(source(h0 + k * step), pl);
  const int64_t slot = a.slot_mapping[t], pos = a.positions[t];
  if (slot < 0) return;                                   // padding token
  const bool bad_slot = slot >= (int64_t)a.num_blocks * a.bs;
  if (bad_slot || pos < 0 || pos >= a.max_pos) {
    if (h0 == 0 && c == 0) flag_error(a.err_flag, bad_slot ? PA_DEV_BAD_SLOT : PA_DEV_BAD_POS);
    return;
  }
  float cs[8], sn[8];
  if (pl.turned) {
    const float* row = a.cos_sin + (size_t)pos * a.rot + 8 * c;
    load8<float>(row, cs);
    load8<float>(row + a.rot / 2, sn);
  }
  for (int hb = h0; hb < heads; hb += U * step) {
    if (hb != h0) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (hb + k * step < heads) it[k].load(source(hb + k * step), pl);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = hb + k * step;
      if (h >= heads) break;
      float f[16];
      it[k].widen(f);
      const bool isv = h >= a.Hq + a.Hkv;
      if (pl.turned && !isv) turn<IL>(f, cs, sn);
      if (h < a.Hq) {
        TS* dst = static_cast<TS*>(a.query_out) + (size_t)t * a.qo_stride + (size_t)h * a.D;
        store8<TS>(dst + pl.e0, f);
        store8<TS>(dst + pl.e1, f + 8);
        continue;
      }
      const size_t row = ((size_t)slot * a.Hkv + (isv ? h - a.Hq - a.Hkv : h - a.Hq)) * a.D;
      void* pool = isv ? a.value_cache : a.key_cache;
      if (isv ? a.v_fp8 : a.k_fp8) {
        const float scale = isv ? a.v_scale : a.k_scale;
        store8_codes(static_cast<uint8_t*>(pool) + row + pl.e0, f, scale);
        store8_codes(static_cast<uint8_t*>(pool) + row + pl.e1, f + 8, scale);
      } else {
        store8<TS>(static_cast<TS*>(pool) + row + pl.e0, f);
        store8<TS>(static_cast<TS*>(pool) + row + pl.e1, f + 8);
      }
    }
  }
}

}  // namespace

// blockIdx.x = token; its items (query heads, key heads, value heads) over the
// CTA's 128 threads, and over blockIdx.y when there are few tokens. Five heads of a
// thread in flight: one round for 64 + 8 + 8 heads of 128. (At 8 x 512 such bf16
// tokens, 170 MB: 256 threads and two heads 34.1 us, 128 and five 29.9 us, 5.7 TB/s,
// 87% of a plain copy. The same bytes with other numbers of heads, 2 / 3 / 5 / 8 in flight,
// with a cold L2: 128 + 8 + 8 43 / 43 / 41 / 39 us, 32 + 32 + 32 41 with each, 32 + 8 + 8
// 45 / 43 / 47 / 49, 16 + 2 + 2 61 / 61 / 74 / 76.)
template <typename TS, bool IL>
__global__ void __launch_bounds__(128, 4)
rope_and_cache_kernel(const RopeArgs a) {
  pdl_trigger();
  pdl_wait();
  const int per_head = a.D / 16, step = 128 / per_head;
  rope_heads<TS, IL, sizeof(TS) == 4 ? 2 : 5>(a, blockIdx.x, threadIdx.x % per_head,
                                              threadIdx.x / per_head + blockIdx.y * step, step * gridDim.y,
                                              a.Hq + 2 * a.Hkv);
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
// block's rows). One warp takes a run's rows of one KV head of K or V: 16
// elements per lane and row, up to four rows of every lane in registers at once, so
// a run of 16 tokens (32 at D = 64) is read once: the largest magnitude over the warp,
// the scale, the codes. No second launch, no atomics. (A run of 32 at D = 128 is
// read twice, the second time from L1 or L2.)
//
// Bound by the chain of a run (slots, rows, maximum, codes), which the query's copies
// beside it hide in part: ragged chunks of fp16 MHA (63 MB) 23 us, 2.7 TB/s; a decode step
// of 128 sequences 5.8 us. A CTA per (run, head) that reads its rows twice took 124 us,
// cosines and sines staged in shared memory 25.7.

namespace {

template <typename TS, bool IL>
__device__ __forceinline__ void append_run(const RopeArgs& a, int t, int n, int64_t block, uint32_t written,
                                           int off, int lpos, int u, int lane) {
  constexpr int U = 4;                         // rows of a lane at once
  const bool isv = u >= a.Hkv;
  const int h = isv ? u - a.Hkv : u;
  const int lpt = a.D / 16, tps = 32 / lpt;    // lanes per row, rows per step
  const int c = lane % lpt, sub = lane / lpt;
  Place pl = place_of<IL>(c, a.rot);
  pl.turned = pl.turned && !isv;               // (a value row's runs are merely read in that order)
  const int64_t stride = isv ? a.v_stride : a.k_stride;
  const TS* src = static_cast<const TS*>(isv ? a.value : a.key) + (size_t)t * stride + (size_t)h * a.D;
  float* scales = (isv ? a.v_scales : a.k_scales) + (size_t)block * a.Hkv + h;
  const bool fresh = written & 1u;
  const float old = fresh ? 0.f : *scales;
  Item<TS> it[U];
  int o[U], p[U];
  // rows i0 + k * tps + sub as loaded; o[k] < 0: not a row of the run
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + k * tps + sub;
      o[k] = __shfl_sync(0xffffffffu, off, i & 31);
      p[k] = __shfl_sync(0xffffffffu, lpos, i & 31);
      if (i >= n) o[k] = -1;
      if (o[k] >= 0) it[k].load(src + (size_t)i * stride, pl);
    }
  };
  // row k rotated (the second time its cosines and sines come from L1; keeping the
  // rotated rows instead of the loaded ones would take twice the registers)
  auto rotated = [&](int k, float* f) {
    it[k].widen(f);
    if (pl.turned) {
      float cs[8], sn[8];
      const float* row = a.cos_sin + (size_t)p[k] * a.rot + 8 * c;
      load8<float>(row, cs);
      load8<float>(row + a.rot / 2, sn);
      turn<IL>(f, cs, sn);
    }
  };
  // the largest finite magnitude of the run's rows (the maximum drops NaN; infinities
  // are left out in a second look, if there are any)
  float top = 0.f;
  for (int i0 = 0; i0 < n; i0 += U * tps) {
    load(i0);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (o[k] < 0) continue;
      float f[16];
      rotated(k, f);
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) most = fmaxf(most, fabsf(f[e]));
      if (most > FLT_MAX) {
        most = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) most = fabsf(f[e]) <= FLT_MAX ? fmaxf(most, fabsf(f[e])) : most;
      }
      top = fmaxf(top, most);
    }
  }
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  float scale = block_scale_for(top);
  if (!fresh) {
    if (!block_scale_ok(old)) {
      if (lane == 0) flag_error(a.err_flag, PA_DEV_BAD_SCALE);
      return;
    }
    scale = fmaxf(scale, old);
  }
  const float inv = __fdiv_rn(1.f, scale);     // a power of two: exact
  uint8_t* pool = static_cast<uint8_t*>(isv ? a.value_cache : a.key_cache) +
                  ((size_t)block * a.bs * a.Hkv + h) * a.D;
  const size_t pitch = (size_t)a.Hkv * a.D;
  const bool again = n > U * tps;              // the registers hold the last rows only
  for (int i0 = 0; i0 < n; i0 += U * tps) {
    if (again) load(i0);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (o[k] < 0) continue;
      float f[16];
      rotated(k, f);
      uint32_t w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        w[x] = e4m3x2(__fmul_rn(f[4 * x], inv), __fmul_rn(f[4 * x + 1], inv)) |
               (e4m3x2(__fmul_rn(f[4 * x + 2], inv), __fmul_rn(f[4 * x + 3], inv)) << 16);
      uint8_t* row = pool + o[k] * pitch;
      *reinterpret_cast<uint2*>(row + pl.e0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + pl.e1) = make_uint2(w[2], w[3]);
    }
  }
  if (!fresh && scale > old) {
    // the block's other rows, rounded to the larger scale
    const float ratio = __fdiv_rn(old, scale);
    for (int r = sub; r < a.bs; r += tps) {
      if ((written >> r) & 1u) continue;
      uint4* p = reinterpret_cast<uint4*>(pool + r * pitch) + c;
      const uint4 v = *p;
      float x[16];
      widen16<__nv_fp8_e4m3>(v, x);
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = e4m3x2(__fmul_rn(x[4 * k], ratio), __fmul_rn(x[4 * k + 1], ratio)) |
               (e4m3x2(__fmul_rn(x[4 * k + 2], ratio), __fmul_rn(x[4 * k + 3], ratio)) << 16);
      *p = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (lane == 0) *scales = scale;
}

}  // namespace

// kv of the grid's CTAs, spread evenly over it, take the pools (latency-bound, beside
// the query's copies, which are not): CTA (tokens [x tb, (x + 1) tb), 8 of the 2 Hkv
// (KV head, K or V) pairs), a warp per (run that starts there, pair). The others
// rotate the query heads of two tokens each.
template <typename TS, bool IL>
__global__ void __launch_bounds__(256, sizeof(TS) == 4 ? 2 : 3)
rope_and_cache_blk8_kernel(const RopeArgs a, int kv, int tb) {
  pdl_trigger();
  pdl_wait();
  const long long grid = gridDim.x, id = blockIdx.x;
  const int kv_id = (int)(id * kv / grid);               // kv CTAs before this one
  if ((int)((id + 1) * kv / grid) == kv_id) {
    const int t = 2 * (int)(id - kv_id) + (threadIdx.x >> 7), per_head = a.D / 16;
    if (t < a.T)
      rope_heads<TS, IL, 2>(a, t, threadIdx.x % per_head, (threadIdx.x & 127) / per_head, 128 / per_head, a.Hq);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ys = (2 * a.Hkv + 7) / 8;
  const int y = kv_id % ys, t0 = kv_id / ys * tb;
  const int pairs = min(8, 2 * a.Hkv - 8 * y);
  const int64_t slots = (int64_t)a.num_blocks * a.bs;
  const bool turn = a.cos_sin != nullptr;
  const int sh = a.bs == 32 ? 5 : 4;
  // slots and positions of tokens t0 + lane and t0 + 32 + lane (a run may go on past
  // the CTA's tokens), and the slot before them
  auto slot_of = [&](int t) -> int64_t { return t < a.T ? a.slot_mapping[t] : -1; };
  const int64_t s0 = slot_of(t0 + lane), s1 = tb > 1 ? slot_of(t0 + 32 + lane) : -1;
  const int64_t before = t0 > 0 ? a.slot_mapping[t0 - 1] : -1;
  // position, -1 if it is bad
  auto pos_of = [&](int t) -> int {
    if (!turn || t >= a.T) return 0;
    const int64_t p = a.positions[t];
    return p >= 0 && p < a.max_pos ? (int)p : -1;
  };
  const int p0 = pos_of(t0 + lane), p1 = tb > 1 ? pos_of(t0 + 32 + lane) : 0;
  auto in_pool = [&](int64_t s) { return s >= 0 && s < slots; };
  const int b0 = in_pool(s0) ? (int)(s0 >> sh) : -1;      // block of the lane's token, -1: none
  int prev = __shfl_up_sync(0xffffffffu, b0, 1);
  if (lane == 0) prev = in_pool(before) ? (int)(before >> sh) : -1;
  if (lane < tb && y == 0 && warp == 0) {
    if (s0 >= slots) flag_error(a.err_flag, PA_DEV_BAD_SLOT);
    else if (s0 >= 0 && p0 < 0) flag_error(a.err_flag, PA_DEV_BAD_POS);
  }
  const uint32_t heads = __ballot_sync(0xffffffffu, lane < tb && b0 >= 0 && b0 != prev);   // runs start
  const int work = __popc(heads) * pairs;
  int block = -1, lpos = 0, run = -1, n = 0, off = -1, first = 0;
  uint32_t written = 0;
  for (int x = warp; x < work; x += 8) {
    if (x / pairs != run) {
      run = x / pairs;
      uint32_t rest = heads;                   // its first token: the run-th set bit
      for (int k = 0; k < run; ++k) rest &= rest - 1;
      first = __ffs(rest) - 1;
      block = __shfl_sync(0xffffffffu, b0, first);
      // lane i: token first + i of the run (off < 0: not of the run, or its position is bad)
      const int at = first + lane;
      const int64_t sa = __shfl_sync(0xffffffffu, s0, at & 31), sb = __shfl_sync(0xffffffffu, s1, at & 31);
      const int pa_ = __shfl_sync(0xffffffffu, p0, at & 31), pb = __shfl_sync(0xffffffffu, p1, at & 31);
      const int64_t s = at < 32 ? sa : sb;
      lpos = at < 32 ? pa_ : pb;
      const bool same = lane < a.bs && in_pool(s) && (int)(s >> sh) == block;
      const uint32_t in = __ballot_sync(0xffffffffu, same);
      n = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
      off = lane < n && lpos >= 0 ? (int)(s & (a.bs - 1)) : -1;
      written = __reduce_or_sync(0xffffffffu, off >= 0 ? 1u << off : 0u);
    }
    if (written)
      append_run<TS, IL>(a, t0 + first, n, block, written, off, lpos, 8 * y + x % pairs, lane);
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
  cudaError_t e;
  if (blk8) {
    // Tokens per CTA: one while that leaves a warp per (token, head, K or V) in two
    // waves of the GPU (a decode step: every token is a run of its own); else 16, of
    // which a chunk's runs leave about one per CTA. With one / 16, 64 + 8 + 8 heads: a step of
    // 128 tokens 12 / 51 us, of 296 16 / 55, of 512 23 / 55, of 2048 61 / 78; a chunk of 512
    // 18 / 14 us, of 2048 41 / 29 (32 + 32 + 32 heads: 80 / 37). The host cannot see which of
    // the two a call is: past the limit a step pays for the chunks.
    const int ys = (2 * a.Hkv + 7) / 8;
    const int tb = (long long)a.T * ys <= 4 * kSMs ? 1 : 16;
    const long long kv = ((long long)a.T + tb - 1) / tb * ys;
    const long long grid = kv + (a.Hq > 0 ? (a.T + 1) / 2 : 0);
    if (grid > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    e = a.interleaved ? launch_k(rope_and_cache_blk8_kernel<TS, true>, dim3((unsigned)grid), dim3(256), 0,
                                 stream, a, (int)kv, tb)
                      : launch_k(rope_and_cache_blk8_kernel<TS, false>, dim3((unsigned)grid), dim3(256), 0,
                                 stream, a, (int)kv, tb);
  } else {
    // split a token's heads only while the tokens leave SMs empty
    const int items = (a.Hq + 2 * a.Hkv) * (a.D / 16);
    int y = (items + 127) / 128;
    while (y > 1 && (long long)a.T * y > 8 * kSMs) --y;
    const dim3 grid((unsigned)a.T, (unsigned)y);
    e = a.interleaved ? launch_k(rope_and_cache_kernel<TS, true>, grid, dim3(128), 0, stream, a)
                      : launch_k(rope_and_cache_kernel<TS, false>, grid, dim3(128), 0, stream, a);
  }
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
