// window_common.cuh -- what the windowed decode kernels share: which tokens a
// sequence's query attends, the split of the work over the CTAs, and the
// warp-level products.
#pragma once

#include <math_constants.h>

#include <cfloat>

#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kTok = 16;                        // tokens per tile
// Work split: cost of a step of a unit, of a unit's start and end (about a step: its query,
// and its output or piece), and the least share worth a CTA (a unit's start and two steps:
// below that the merge costs more than the CTA saves).
constexpr int kTileCost = 16;
constexpr int kUnitCost = 16;
constexpr int kMinShare = kUnitCost + 2 * kTileCost;

// The tokens a sequence's query attends, by tile.
struct Span {
  int lo, sk, ctx;    // visible: t < ctx and (t >= lo or t < sk)
  int n0, w0, n;      // virtual tile v < n: tile v (v < n0) or v - n0 + w0
  __device__ __forceinline__ int tile(int v) const { return v < n0 ? v : v - n0 + w0; }
  __device__ __forceinline__ bool sees(int t) const { return t < ctx && (t >= lo || t < sk); }
  // every token of the tile that starts at t0
  __device__ __forceinline__ bool whole(int t0) const {
    return t0 + kTok <= ctx && (t0 >= lo || t0 + kTok <= sk);
  }
};

__device__ __forceinline__ bool bad_context(const WinArgs& a, int ctx) {
  return ctx < 0 || ctx > (long long)a.max_blocks * a.bs || ctx > a.max_context_len;
}

// A bad length attends nothing (n = 0), as does an empty sequence.
__device__ __forceinline__ Span span_of(const WinArgs& a, int ctx) {
  Span s;
  s.ctx = bad_context(a, ctx) ? 0 : ctx;
  s.lo = a.window > 0 ? max(0, s.ctx - a.window) : 0;
  s.sk = min(a.sinks, s.lo);
  s.w0 = s.lo / kTok;
  s.n0 = min((s.sk + kTok - 1) / kTok, s.w0);
  s.n = s.n0 + (s.ctx + kTok - 1) / kTok - s.w0;
  return s;
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

template <bool BF>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x0, x1 as packed 16-bit values and what their rounding lost (times up), the same way.
template <bool BF>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo, float up = 1.f) {
  if (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn((x0 - f.x) * up, (x1 - f.y) * up);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn((x0 - f.x) * up, (x1 - f.y) * up);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&r);
  }
}

// Four E4M3 codes as two pairs of packed f16, exactly.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

constexpr int esize(int dt) { return dt == PA_FP8_E4M3 ? 1 : 2; }

// Work split. A unit is (sequence, y) with y < ny the KV heads or groups of them and
// the chunks of their query heads; it has ceil(n / step) steps of `step` tiles and
// costs kTileCost each plus kUnitCost. The units' costs laid end to end are cut
// into equal shares, one per CTA; step j of a unit that starts at position s sits at
// s + kUnitCost + kTileCost j.
struct Share {
  long long lo, hi, total;
  int shares;                // CTAs with a share (those past it have nothing to do)
  long long base0;           // where the first unit of the share starts
  int p0;                    // that unit
};

__device__ __forceinline__ int steps_of(const Span& s, int step) { return (s.n + step - 1) / step; }

// a / b for non-negative numbers, in 32 bits where they fit (a 64-bit division is a
// call of some hundred instructions, and a share starts with several).
__device__ __forceinline__ long long quot(long long a, long long b) {
  if ((unsigned long long)(a | b) >> 32) return a / b;
  return (long long)((uint32_t)a / (uint32_t)b);
}

// The CTA whose share holds position pos: share c is [c C / n, (c + 1) C / n).
__device__ __forceinline__ int share_of(long long pos, const Share& w) {
  return (int)quot((pos + 1) * w.shares - 1, w.total);
}

// The share of CTA cta; every thread of the CTA calls it (two barriers).
template <int THREADS>
__device__ __forceinline__ Share find_share(const WinArgs& a, int ny, int step, int cta, int ctas) {
  __shared__ long long sm_scan[THREADS / 32];
  __shared__ long long sm_base;
  __shared__ int sm_first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto cost_of = [&](int b) -> long long {
    const Span s = span_of(a, __ldg(a.context_lens + b));
    return (long long)ny * ((long long)kTileCost * steps_of(s, step) + kUnitCost);
  };
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += cost_of(b);
  long long incl = sum;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, x);
    if (lane >= x) incl += y;
  }
  if (lane == 31) sm_scan[warp] = incl;
  __syncthreads();
  Share w;
  long long before = incl - sum;
  w.total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) {
    if (i < warp) before += sm_scan[i];
    w.total += sm_scan[i];
  }
  w.shares = (int)min((long long)ctas, max(1ll, w.total / kMinShare));
  w.lo = quot(cta * w.total, w.shares);
  w.hi = quot((cta + 1) * w.total, w.shares);
  if (w.lo >= before && w.lo < before + sum) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const long long cb = cost_of(b);
      if (w.lo < at + cb) {
        const long long one = quot(cb, ny);
        const int y = (int)quot(w.lo - at, one);
        sm_first = b * ny + y;
        sm_base = at + y * one;
        break;
      }
      at += cb;
    }
  }
  __syncthreads();
  w.p0 = cta < w.shares ? sm_first : 0;
  w.base0 = cta < w.shares ? sm_base : w.total;
  return w;
}

// 32 units of a share from w.p0 on, one per lane, and the share moved past them.
struct Batch {
  int b, y, ctx;             // sequence, y, context length (as stored)
  int s0, s1;                // the share's steps of the unit
  int first, last;           // CTAs that hold the unit's first and last step
  bool starts;               // the unit starts in this share
  int n;                     // steps of the unit (0: nothing to attend)
  int count;                 // units of the batch (the same in every lane)
};
__device__ __forceinline__ Batch next_batch(const WinArgs& a, Share& w, int ny, int step, int cta, int lane) {
  const int units = a.B * ny, p = w.p0 + lane;
  Batch u = {0, 0, 0, 0, 0, cta, cta, false, 0, 0};
  long long cost = 0;
  if (p < units) {
    u.b = p / ny;
    u.y = p - u.b * ny;
    u.ctx = __ldg(a.context_lens + u.b);
    u.n = steps_of(span_of(a, u.ctx), step);
    cost = (long long)kTileCost * u.n + kUnitCost;
  }
  long long end = cost;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, end, x);
    if (lane >= x) end += y;
  }
  end += w.base0;
  const long long start = end - cost;
  if (p < units) {
    const long long t = start + kUnitCost;
    u.s0 = (int)min((long long)u.n, max(0ll, (w.lo - t + kTileCost - 1) / kTileCost));
    u.s1 = (int)min((long long)u.n, max(0ll, (w.hi - t + kTileCost - 1) / kTileCost));
    u.starts = start >= w.lo && start < w.hi;
    if (u.n > 0) {
      u.first = share_of(t, w);
      u.last = share_of(t + (long long)kTileCost * (u.n - 1), w);
    }
  }
  u.count = __popc(__ballot_sync(0xffffffffu, p < units && start < w.hi));
  w.base0 = __shfl_sync(0xffffffffu, end, 31);
  w.p0 += 32;
  return u;
}

}  // namespace

}  // namespace pa
