// decode_window.cu -- decode attention over part of a sequence's tokens (a
// sliding window and a few first tokens) and over the block-scaled 8-bit cache.
//
// A sequence of ctx tokens whose last one is the query's attends the tokens
//   t < ctx  with  t >= ctx - window  or  t < sinks     (window 0: every t < ctx).
// Its tokens are walked in tiles of 16 (half a block or a whole one); the tiles
// that hold a visible token are the first n0 (sinks) and those from w0 on (the
// window), so virtual tile v is tile v or v - n0 + w0 and nothing between is
// read, its block-table entries included.
//
// The work per visible (token, KV head) is 2 D bytes-per-element of K and V
// against 4 D flops per query head: with up to 16 query heads per KV head it is
// bound by HBM, so the kernel is built around bytes in flight. Every warp owns a
// ring of tiles in shared memory that it fills with 16-byte asynchronous copies
// (no registers held, no barrier with the other warps) and takes its tiles from
// it. The products are warp-level m16n8k16 MMAs whose operands the warp reads
// from its tile in the order the instruction wants:
//   S[16 x 8 keys]  = Q . K^T : A = the query heads in rows 0-7, what their
//     rounding to 16 bits lost in rows 8-15 (an 8-bit pool meets queries of any
//     type at ~22 bits), B = K rows as they lie, the dims permuted alike on both
//     sides so a lane's operands are one 16-byte run of a row;
//   O[16 x 8 dims] += P . V : rows 0-7 the weights, rows 8-15 what their rounding
//     to 16 bits lost, so the MMA rows that 8 heads leave empty carry the second
//     half of the precision and the two halves are added at the end.
// 8-bit codes are widened to f16 (exactly) between shared memory and the MMA.
//
// Block-scaled pools: K's power of two multiplies the scores of its block's
// tokens. V's would have to multiply the weights before they are rounded to
// 16 bits, where a small scale would push them under f16's range; instead the
// running maximum is taken over log2 of the whole contribution, s' = s + log2(vs)
// (an exact integer): weights w = 2^(s' - m') are normalised to the largest
// contribution, and the exp-sum counts w 2^-log2(vs).
#include <math_constants.h>

#include <cfloat>

#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kTok = 16;                        // tokens per tile
constexpr int kHeads = 8;                       // query heads per CTA
constexpr float kMove = 8.f;                    // the reference maximum moves when passed by 2^8:
                                                // weights stay under 2^8, far inside f16

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

__device__ __forceinline__ Span span_of(int ctx, int window, int sinks) {
  Span s;
  s.ctx = ctx;
  s.lo = window > 0 ? max(0, ctx - window) : 0;
  s.sk = min(sinks, s.lo);
  s.w0 = s.lo / kTok;
  s.n0 = min((s.sk + kTok - 1) / kTok, s.w0);
  s.n = s.n0 + (ctx + kTok - 1) / kTok - s.w0;
  return s;
}

__device__ __forceinline__ bool bad_context(const WinArgs& a, int ctx) {
  return ctx < 0 || ctx > (long long)a.max_blocks * a.bs || ctx > a.max_context_len;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes from global to shared memory, zeros when !take (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// x0, x1 as packed 16-bit values and what their rounding lost, the same way.
template <bool BF>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  if (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(x0 - f.x, x1 - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(x0 - f.x, x1 - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&r);
  }
}

// Two E4M3 codes (the low 16 bits) as packed f16, exactly.
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

__device__ __forceinline__ float load_q1(const void* q, size_t i, int dtype) {
  if (dtype == PA_F32) return static_cast<const float*>(q)[i];
  if (dtype == PA_F16) return __half2float(static_cast<const __half*>(q)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i]);
}

constexpr int esize(int dt) { return dt == PA_F32 ? 4 : dt == PA_FP8_E4M3 ? 1 : 2; }

// The tile's shared-memory layout: K rows then V rows, 16-byte chunks swizzled
// within a row so that the reads below touch every bank once per eight lanes
// (K: lanes read 4 adjacent chunks of 2 rows; V: 2 adjacent chunks of 4 rows
// two apart; fp32: one chunk of 8 rows).
template <int DT, int D> struct Rows {
  static constexpr int ROWB = D * esize(DT);
  static constexpr int CPR = ROWB / 16;         // chunks per row
  static constexpr int BYTES = kTok * ROWB;
  static __device__ __forceinline__ uint32_t k_at(int row, int c) {
    const int sw = DT == PA_F32 ? (row & 7) : CPR >= 8 ? ((row & 1) << 2) : 0;
    return (uint32_t)(row * ROWB + ((c ^ sw) << 4));
  }
  static __device__ __forceinline__ uint32_t v_at(int row, int c) {
    const int sw = CPR >= 8 ? (row & 7) : ((row >> 1) & 3);
    return (uint32_t)(row * ROWB + ((c ^ sw) << 4));
  }
};

// Tiles a warp keeps in its ring: 24 KB of bytes in flight per warp (two CTAs of
// four warps per SM), at least two.
constexpr int stages_for(int tile_bytes) {
  const int n = 24 * 1024 / tile_bytes;
  return n < 2 ? 2 : n > 8 ? 8 : n;
}

// Copies of one tile of one KV head into a ring stage.
template <int KT, int VT, int D>
__device__ __forceinline__ void issue_tile(const WinArgs& a, uint32_t stage, const Span& sp, int t0,
                                           int id, int in_block, int h, int lane) {
  using RK = Rows<KT, D>;
  using RV = Rows<VT, D>;
  const bool ok = id >= 0;
  const size_t row0 = ((size_t)(ok ? id : 0) * a.bs + in_block) * a.Hkv + h;
  const char* kp = static_cast<const char*>(a.k_cache) + (ok ? row0 * RK::ROWB : 0);
  const char* vp = static_cast<const char*>(a.v_cache) + (ok ? row0 * RV::ROWB : 0);
#pragma unroll
  for (int i = 0; i < RK::CPR / 2; ++i) {
    const int x = i * 32 + lane, row = x / RK::CPR, c = x % RK::CPR;
    const bool take = ok && sp.sees(t0 + row);
    copy16(stage + RK::k_at(row, c), take ? kp + (size_t)row * a.Hkv * RK::ROWB + c * 16 : kp, take);
  }
#pragma unroll
  for (int i = 0; i < RV::CPR / 2; ++i) {
    const int x = i * 32 + lane, row = x / RV::CPR, c = x % RV::CPR;
    const bool take = ok && sp.sees(t0 + row);
    copy16(stage + RK::BYTES + RV::v_at(row, c), take ? vp + (size_t)row * a.Hkv * RV::ROWB + c * 16 : vp,
           take);
  }
}

// What a warp knows of its next 32 tiles, one per lane: the block (-1: bad) and,
// for block-scaled pools, its scales.
struct Ahead {
  int id;
  float ks;        // K scale
  int lvs;         // log2 of the V scale
};
template <bool BSC>
__device__ __forceinline__ Ahead look_up(const WinArgs& a, const int32_t* table, const Span& sp, int v,
                                         int v_end, int h) {
  Ahead x{-1, 1.f, 0};
  if (v < v_end) {
    x.id = __ldg(table + sp.tile(v) * kTok / a.bs);
    if (x.id < 0 || x.id >= a.num_blocks) {
      flag_error(a.err_flag, PA_DEV_BAD_BLOCK_ID);
      x.id = -1;
    } else if (BSC) {
      const float ks = __ldg(a.k_scales + (size_t)x.id * a.Hkv + h);
      const float vs = __ldg(a.v_scales + (size_t)x.id * a.Hkv + h);
      if (!block_scale_ok(ks) || !block_scale_ok(vs)) {
        flag_error(a.err_flag, PA_DEV_BAD_SCALE);
        x.id = -1;
      } else {
        x.ks = ks;
        x.lvs = block_scale_log2(vs);
      }
    }
  }
  return x;
}

// The CTA's warps' (m, l, acc) for gc heads joined and written: the output, or a
// part for the merge.
template <int D, int HEADS>
__device__ __forceinline__ void finish(const WinArgs& a, const float* sm_acc, const float* sm_m,
                                       const float* sm_l, int gc, int b, int hq0, int part, bool last) {
  for (int i = threadIdx.x; i < gc * D; i += kWarps * 32) {
    const int g = i / D, d = i - g * D;
    float M = -FLT_MAX, L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w * HEADS + g]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float c = ex2(sm_m[w * HEADS + g] - M);
      L = fmaf(sm_l[w * HEADS + g], c, L);
      O = fmaf(sm_acc[(w * HEADS + g) * D + d], c, O);
    }
    if (last) {
      store_out(a.out, ((size_t)b * a.Hq + hq0 + g) * D + d, L == 0.f ? 0.f : O / L * a.v_scale,
                a.out_dtype);
    } else {
      const size_t slot = ((size_t)b * a.P + part) * a.Hq + hq0 + g;
      a.ws_acc[slot * D + d] = O;
      if (d == 0) { a.ws_m[slot] = M; a.ws_l[slot] = L; }
    }
  }
}

// Zero rows of a sequence with nothing to attend or a bad length (part 0 writes them).
template <int D>
__device__ __forceinline__ void zero_rows(const WinArgs& a, int gc, int b, int hq0) {
  for (int i = threadIdx.x; i < gc * D; i += kWarps * 32)
    store_out(a.out, ((size_t)b * a.Hq + hq0) * D + i, 0.f, a.out_dtype);
}

}  // namespace

// KT, VT: pool element types. BSC: both pools hold codes with one scale per
// block and KV head. CTA = (part, KV head and chunk of 8 query heads, sequence),
// four warps that take the part's tiles in turn.
template <int KT, int VT, int D, bool BSC>
__global__ void __launch_bounds__(kWarps * 32)
decode_window_kernel(const WinArgs a) {
  using RK = Rows<KT, D>;
  using RV = Rows<VT, D>;
  constexpr bool KBF = KT == PA_BF16, VBF = VT == PA_BF16;
  constexpr bool K8 = KT == PA_FP8_E4M3, V8 = VT == PA_FP8_E4M3;
  constexpr int STAGE = RK::BYTES + RV::BYTES;
  constexpr int NST = stages_for(STAGE);
  constexpr int KS = D / 16;                    // k-steps of the score product
  constexpr int NT = D / 8;                     // 8-wide dim tiles of the output product
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_q[kHeads * D];
  __shared__ float sm_f[kHeads];                // score factor of each head
  __shared__ float sm_m[kWarps * kHeads], sm_l[kWarps * kHeads];
  static_assert(kWarps * kHeads * D * 4 <= kWarps * NST * STAGE, "the joined sums reuse the rings");
  pdl_trigger();
  pdl_wait();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = a.Hq / a.Hkv;
  const int chunks = (G + kHeads - 1) / kHeads;
  const int h = blockIdx.y / chunks, chunk = blockIdx.y - h * chunks;
  const int b = blockIdx.z, part = blockIdx.x;
  const int hq0 = h * G + chunk * kHeads, gc = min(kHeads, G - chunk * kHeads);

  const int ctx = a.context_lens[b];
  if (bad_context(a, ctx) || ctx == 0) {
    if (part == 0) {
      if (ctx != 0 && threadIdx.x == 0 && blockIdx.y == 0) flag_error(a.err_flag, PA_DEV_BAD_CTX);
      zero_rows<D>(a, gc, b, hq0);
    }
    return;
  }
  const Span sp = span_of(ctx, a.window, a.sinks);
  const int v0 = part * a.ptiles;
  if (v0 >= sp.n) return;
  const int v1 = min(sp.n, v0 + a.ptiles);

  const int32_t* table = a.block_tables + (size_t)b * a.max_blocks;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (NST * STAGE);
  const int mine = (v1 - v0 - warp + kWarps - 1) / kWarps;     // tiles of this warp (<= 0: none)
  Ahead now = look_up<BSC>(a, table, sp, v0 + warp + kWarps * lane, v1, h);
  Ahead next = now;
  // stage k % NST <- the warp's tile k (tiles 0-31 of the current batch are in
  // `now`, those of the next one in `next`)
  auto issue = [&](int k, const Ahead& from) {
    const int id = __shfl_sync(0xffffffffu, from.id, k & 31);
    const int t0 = sp.tile(v0 + warp + kWarps * k) * kTok;
    issue_tile<KT, VT, D>(a, ring + (k % NST) * STAGE, sp, t0, id, t0 & (a.bs - 1), h, lane);
  };
#pragma unroll
  for (int k = 0; k < NST - 1; ++k) {
    if (k < mine) issue(k, now);
    copy_commit();
  }

  // the query heads in fp32; an 8-bit K pool takes them scaled by a power of two
  // that puts the head's largest element into [2^14, 2^15)
  for (int r = warp; r < kHeads; r += kWarps) {
    float x[D / 32];
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      x[e] = r < gc ? load_q1(a.q, ((size_t)b * a.Hq + hq0 + r) * D + e * 32 + lane, a.q_dtype) : 0.f;
      top = fmaxf(top, fabsf(x[e]));
    }
    float factor = a.scale_log2;
    if (K8) {
      const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
      const int e = (int)(bits >> 23) - 127;                // exponent of the largest element
      if (e >= -100 && e < 127) {
        const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);   // 2^(14 - e)
#pragma unroll
        for (int i = 0; i < D / 32; ++i) x[i] *= up;
        factor = a.scale_log2 * __uint_as_float((uint32_t)(e - 14 + 127) << 23);
      }
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) sm_q[r * D + e * 32 + lane] = x[e];
    if (lane == 0) sm_f[r] = factor;
  }
  __syncthreads();
  // A operand of the score product: k-step 2 i + j (16-bit K) or 4 i + j (codes)
  // takes 4 elements of the 8 or 16 of a lane's run
  uint32_t qa[KS][4];
  constexpr int RUN = K8 ? 16 : 8;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int i = ks / (RUN / 4), j = ks % (RUN / 4);
    const float* x = sm_q + g * D + i * 4 * RUN + t * RUN + 4 * j;
    split2<KBF>(x[0], x[1], qa[ks][0], qa[ks][1]);
    split2<KBF>(x[2], x[3], qa[ks][2], qa[ks][3]);
  }
  const float factor = sm_f[g];

  float m = -FLT_MAX, l = 0.f;
  float o[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

  for (int k = 0; k < mine; ++k) {
    // batches of 32 tiles: the next one's blocks are looked up before its first
    // tile is issued, NST - 1 tiles ahead
    const int ki = k + NST - 1;
    if ((ki & 31) == 0 || k == 0) {
      const int base = (ki & ~31);
      next = base == 0 ? now : look_up<BSC>(a, table, sp, v0 + warp + kWarps * (base + lane), v1, h);
    }
    __syncwarp();                               // every lane has read the stage's last tile
    if (ki < mine) issue(ki, next);
    copy_commit();
    copy_wait<NST - 1>();
    __syncwarp();
    if ((k & 31) == 0 && k > 0) now = next;
    const int id = __shfl_sync(0xffffffffu, now.id, k & 31);
    const float ks_b = BSC ? __shfl_sync(0xffffffffu, now.ks, k & 31) : 1.f;
    const int lvs = BSC ? __shfl_sync(0xffffffffu, now.lvs, k & 31) : 0;
    if (id < 0) continue;
    const int t0 = sp.tile(v0 + warp + kWarps * k) * kTok;
    const uint32_t kst = ring + (k % NST) * STAGE, vst = kst + RK::BYTES;

    // ---- scores: two 8-key products
    float c[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
    for (int i = 0; i < D / (4 * RUN); ++i) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint4 w = lds16(kst + RK::k_at(8 * nt + g, 4 * i + t));
        if (K8) {
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma<false>(c[nt], qa[4 * i + j], widen2(ww[j]), widen2(ww[j] >> 16));
        } else {
          mma<KBF>(c[nt], qa[2 * i], w.x, w.y);
          mma<KBF>(c[nt], qa[2 * i + 1], w.z, w.w);
        }
      }
    }
    // ---- online softmax of head g over keys 8 nt + 2 t + {0, 1}
    const float f = BSC ? factor * ks_b : factor;
    float s[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[nt][e] = (c[nt][e] + c[nt][e + 2]) * f;
        if (BSC) s[nt][e] += (float)lvs;
      }
    if (!sp.whole(t0)) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!sp.sees(t0 + 8 * nt + 2 * t + e)) s[nt][e] = -CUDART_INF_F;
    }
    float mx = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (__any_sync(0xffffffffu, mx > m + kMove)) {
      const float mn = mx > m + kMove ? mx : m;
      const float alpha = ex2(m - mn);
      m = mn;
      l *= alpha;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j][0] *= alpha; o[j][1] *= alpha; o[j][2] *= alpha; o[j][3] *= alpha;
      }
    }
    float p[2][2], sum = 0.f;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        p[nt][e] = ex2(s[nt][e] - m);
        sum += p[nt][e];
      }
    if (BSC) l = fmaf(sum, __uint_as_float((uint32_t)(127 - lvs) << 23), l);
    else l += sum;
    uint32_t pa_[4];
    split2<VBF>(p[0][0], p[0][1], pa_[0], pa_[1]);
    split2<VBF>(p[1][0], p[1][1], pa_[2], pa_[3]);

    // ---- O += P . V: the lane's tokens are 2 t, 2 t + 1, 2 t + 8, 2 t + 9
    if constexpr (V8 && D == 64) {
      uint2 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 2 * t + (i & 1) + 8 * (i >> 1);
        w[i] = lds8(vst + RV::v_at(row, g >> 1) + 8 * (g & 1));
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t r0 = q ? w[0].y : w[0].x, r1 = q ? w[1].y : w[1].x;
        const uint32_t r2 = q ? w[2].y : w[2].x, r3 = q ? w[3].y : w[3].x;
        const uint32_t x0 = __byte_perm(r0, r1, 0x5140), x1 = __byte_perm(r0, r1, 0x7362);
        const uint32_t y0 = __byte_perm(r2, r3, 0x5140), y1 = __byte_perm(r2, r3, 0x7362);
        mma<false>(o[4 * q], pa_, widen2(x0), widen2(y0));
        mma<false>(o[4 * q + 1], pa_, widen2(x0 >> 16), widen2(y0 >> 16));
        mma<false>(o[4 * q + 2], pa_, widen2(x1), widen2(y1));
        mma<false>(o[4 * q + 3], pa_, widen2(x1 >> 16), widen2(y1 >> 16));
      }
    } else {
#pragma unroll
      for (int cg = 0; cg < RV::CPR / 8; ++cg) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 2 * t + (i & 1) + 8 * (i >> 1);
          w[i] = lds16(vst + RV::v_at(row, 8 * cg + g));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t r0 = (&w[0].x)[q], r1 = (&w[1].x)[q], r2 = (&w[2].x)[q], r3 = (&w[3].x)[q];
          if (V8) {
            const uint32_t x0 = __byte_perm(r0, r1, 0x5140), x1 = __byte_perm(r0, r1, 0x7362);
            const uint32_t y0 = __byte_perm(r2, r3, 0x5140), y1 = __byte_perm(r2, r3, 0x7362);
            mma<false>(o[4 * q], pa_, widen2(x0), widen2(y0));
            mma<false>(o[4 * q + 1], pa_, widen2(x0 >> 16), widen2(y0 >> 16));
            mma<false>(o[4 * q + 2], pa_, widen2(x1), widen2(y1));
            mma<false>(o[4 * q + 3], pa_, widen2(x1 >> 16), widen2(y1 >> 16));
          } else {
            mma<VBF>(o[8 * cg + 2 * q], pa_, __byte_perm(r0, r1, 0x5410), __byte_perm(r2, r3, 0x5410));
            mma<VBF>(o[8 * cg + 2 * q + 1], pa_, __byte_perm(r0, r1, 0x7632),
                     __byte_perm(r2, r3, 0x7632));
          }
        }
      }
    }
  }
  copy_wait<0>();
  __syncthreads();                              // the rings are free

  // ---- join the warps
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (t == 0) { sm_m[warp * kHeads + g] = m; sm_l[warp * kHeads + g] = l; }
  float* sm_acc = reinterpret_cast<float*>(smem);
  constexpr int EPV = V8 && D == 128 ? 16 : 8;  // dims of a lane's run of a V row
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int d = (j / EPV) * (8 * EPV) + 2 * t * EPV + j % EPV;
    sm_acc[(warp * kHeads + g) * D + d] = o[j][0] + o[j][2];
    sm_acc[(warp * kHeads + g) * D + d + EPV] = o[j][1] + o[j][3];
  }
  __syncthreads();
  finish<D, kHeads>(a, sm_acc, sm_m, sm_l, gc, b, hq0, part, sp.n <= a.ptiles);
}

// fp32 pools: the same walk and ring, products on the CUDA cores (4 query heads
// per CTA). Scores: lane = (token, half of the dims); output: a lane owns D / 32
// dims of every head.
template <int D>
__global__ void __launch_bounds__(kWarps * 32)
decode_window_f32_kernel(const WinArgs a) {
  using R = Rows<PA_F32, D>;
  constexpr int HC = 4;
  constexpr int STAGE = 2 * R::BYTES;
  constexpr int NST = stages_for(STAGE);
  constexpr int PER = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float sm_q[HC * D];
  __shared__ float sm_m[kWarps * HC], sm_l[kWarps * HC];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv;
  const int chunks = (G + HC - 1) / HC;
  const int h = blockIdx.y / chunks, chunk = blockIdx.y - h * chunks;
  const int b = blockIdx.z, part = blockIdx.x;
  const int hq0 = h * G + chunk * HC, gc = min(HC, G - chunk * HC);
  const int ctx = a.context_lens[b];
  if (bad_context(a, ctx) || ctx == 0) {
    if (part == 0) {
      if (ctx != 0 && threadIdx.x == 0 && blockIdx.y == 0) flag_error(a.err_flag, PA_DEV_BAD_CTX);
      zero_rows<D>(a, gc, b, hq0);
    }
    return;
  }
  const Span sp = span_of(ctx, a.window, a.sinks);
  const int v0 = part * a.ptiles;
  if (v0 >= sp.n) return;
  const int v1 = min(sp.n, v0 + a.ptiles);
  const int32_t* table = a.block_tables + (size_t)b * a.max_blocks;
  uint8_t* ring_p = smem + warp * (NST * STAGE);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(ring_p);
  const int mine = (v1 - v0 - warp + kWarps - 1) / kWarps;
  auto block_of = [&](int k) {
    return look_up<false>(a, table, sp, v0 + warp + kWarps * k, v1, h).id;
  };
  auto issue = [&](int k, int id) {
    const int t0 = sp.tile(v0 + warp + kWarps * k) * kTok;
    issue_tile<PA_F32, PA_F32, D>(a, ring + (k % NST) * STAGE, sp, t0, id, t0 & (a.bs - 1), h, lane);
  };
  int ids[NST];                                 // blocks of the tiles in the ring
#pragma unroll
  for (int k = 0; k < NST - 1; ++k) {
    ids[k] = block_of(k);
    if (k < mine) issue(k, ids[k]);
    copy_commit();
  }
  for (int i = threadIdx.x; i < HC * D; i += kWarps * 32)
    sm_q[i] = i < gc * D ? static_cast<const float*>(a.q)[((size_t)b * a.Hq + hq0) * D + i] * a.scale_log2
                         : 0.f;
  __syncthreads();

  float m[HC], l[HC], o[HC][PER];
#pragma unroll
  for (int g = 0; g < HC; ++g) {
    m[g] = -FLT_MAX;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[g][e] = 0.f;
  }
  const int row = lane & 15, hf = lane >> 4;
  for (int k0 = 0; k0 < mine; k0 += NST) {
#pragma unroll
    for (int u = 0; u < NST; ++u) {             // stage = u, so ids[] stays in registers
      const int k = k0 + u;
      if (k >= mine) break;
      const int ki = k + NST - 1;
      const int nid = block_of(ki);
      __syncwarp();
      if (ki < mine) issue(ki, nid);
      ids[(u + NST - 1) % NST] = nid;
      copy_commit();
      copy_wait<NST - 1>();
      __syncwarp();
      if (ids[u] < 0) continue;
      const int t0 = sp.tile(v0 + warp + kWarps * k) * kTok;
      const uint8_t* kst = ring_p + u * STAGE;
      const uint8_t* vst = kst + R::BYTES;
      float s[HC];
#pragma unroll
      for (int g = 0; g < HC; ++g) s[g] = 0.f;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const int cc = hf * (D / 8) + c;
        const float4 kv = *reinterpret_cast<const float4*>(kst + R::k_at(row, cc));
#pragma unroll
        for (int g = 0; g < HC; ++g) {
          const float4 q = *reinterpret_cast<const float4*>(sm_q + g * D + 4 * cc);
          s[g] = fmaf(q.x, kv.x, fmaf(q.y, kv.y, fmaf(q.z, kv.z, fmaf(q.w, kv.w, s[g]))));
        }
      }
      const bool sees = sp.sees(t0 + row);
      float p[HC];
#pragma unroll
      for (int g = 0; g < HC; ++g) {
        s[g] += __shfl_xor_sync(0xffffffffu, s[g], 16);
        if (!sees) s[g] = -CUDART_INF_F;
        float mx = s[g];
#pragma unroll
        for (int x = 8; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
        const float mn = fmaxf(m[g], mx);
        const float alpha = exp2f(m[g] - mn);
        m[g] = mn;
        p[g] = exp2f(s[g] - mn);
        l[g] = l[g] * alpha + p[g];             // lanes 0-15 and 16-31 hold the same tokens
#pragma unroll
        for (int e = 0; e < PER; ++e) o[g][e] *= alpha;
      }
#pragma unroll 4
      for (int r = 0; r < kTok; ++r) {
        float v[PER];
        const int d0 = lane * PER;
        const uint8_t* vr = vst + R::v_at(r, d0 / 4) + (d0 % 4) * 4;
        if constexpr (PER == 4) {
          const float4 w = *reinterpret_cast<const float4*>(vr);
          v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
        } else {
          const float2 w = *reinterpret_cast<const float2*>(vr);
          v[0] = w.x; v[1] = w.y;
        }
#pragma unroll
        for (int g = 0; g < HC; ++g) {
          const float pr = __shfl_sync(0xffffffffu, p[g], r);
#pragma unroll
          for (int e = 0; e < PER; ++e) o[g][e] = fmaf(pr, v[e], o[g][e]);
        }
      }
    }
  }
  copy_wait<0>();
  __syncthreads();
  float* sm_acc = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int g = 0; g < HC; ++g) {
#pragma unroll
    for (int x = 8; x >= 1; x >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], x);
    if (lane == 0) { sm_m[warp * HC + g] = m[g]; sm_l[warp * HC + g] = l[g]; }
#pragma unroll
    for (int e = 0; e < PER; ++e) sm_acc[(warp * HC + g) * D + lane * PER + e] = o[g][e];
  }
  __syncthreads();
  finish<D, HC>(a, sm_acc, sm_m, sm_l, gc, b, hq0, part, sp.n <= a.ptiles);
}

// Sequences cut into parts: one warp per (sequence, query head) joins them.
template <int D>
__global__ void __launch_bounds__(128) decode_window_merge_kernel(const WinArgs a) {
  constexpr int PER = D / 32;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x * 4ll + warp;
  if (row >= (long long)a.B * a.Hq) return;
  const int b = (int)(row / a.Hq), hq = (int)(row - (long long)b * a.Hq);
  const int ctx = a.context_lens[b];
  if (bad_context(a, ctx) || ctx == 0) return;
  const Span sp = span_of(ctx, a.window, a.sinks);
  const int parts = (sp.n + a.ptiles - 1) / a.ptiles;
  if (parts <= 1) return;
  const size_t base = (size_t)b * a.P * a.Hq + hq;
  float M = -FLT_MAX;
  for (int j = lane; j < parts; j += 32) M = fmaxf(M, a.ws_m[base + (size_t)j * a.Hq]);
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  float L = 0.f, O[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) O[e] = 0.f;
#pragma unroll 4
  for (int j = 0; j < parts; ++j) {
    const size_t slot = base + (size_t)j * a.Hq;
    const float c = ex2(a.ws_m[slot] - M);
    L = fmaf(a.ws_l[slot], c, L);
#pragma unroll
    for (int e = 0; e < PER; ++e) O[e] = fmaf(a.ws_acc[slot * D + e * 32 + lane], c, O[e]);
  }
  const float inv = L == 0.f ? 0.f : a.v_scale / L;
#pragma unroll
  for (int e = 0; e < PER; ++e)
    store_out(a.out, (size_t)row * D + e * 32 + lane, O[e] * inv, a.out_dtype);
}

namespace {

// Dynamic shared memory above 48 KB needs the attribute, per device.
template <typename K>
cudaError_t allow_smem(K kern, int bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <int KT, int VT, int D, bool BSC>
int launch_window_t(const WinArgs& a, cudaStream_t stream) {
  constexpr int STAGE = Rows<KT, D>::BYTES + Rows<VT, D>::BYTES;
  constexpr int SMEM = kWarps * stages_for(STAGE) * STAGE;
  const int G = a.Hq / a.Hkv, chunks = (G + kHeads - 1) / kHeads;
  auto kern = decode_window_kernel<KT, VT, D, BSC>;
  if (allow_smem(kern, SMEM) != cudaSuccess) return PA_ERR_CUDA;
  const dim3 grid((unsigned)a.P, (unsigned)(a.Hkv * chunks), (unsigned)a.B);
  return launch_k(kern, grid, dim3(kWarps * 32), SMEM, stream, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D>
int launch_window_f32(const WinArgs& a, cudaStream_t stream) {
  constexpr int STAGE = 2 * Rows<PA_F32, D>::BYTES;
  constexpr int SMEM = kWarps * stages_for(STAGE) * STAGE;
  const int G = a.Hq / a.Hkv, chunks = (G + 3) / 4;
  auto kern = decode_window_f32_kernel<D>;
  if (allow_smem(kern, SMEM) != cudaSuccess) return PA_ERR_CUDA;
  const dim3 grid((unsigned)a.P, (unsigned)(a.Hkv * chunks), (unsigned)a.B);
  return launch_k(kern, grid, dim3(kWarps * 32), SMEM, stream, a) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int D>
int launch_window_d(const WinArgs& a, cudaStream_t stream) {
  constexpr int F8 = PA_FP8_E4M3;
  if (a.k_scales) return launch_window_t<F8, F8, D, true>(a, stream);
  const int k = a.k_dtype, v = a.v_dtype;
  if (k == PA_F32 && v == PA_F32) return launch_window_f32<D>(a, stream);
  if (k == F8 && v == F8) return launch_window_t<F8, F8, D, false>(a, stream);
  if (k == PA_F16 && v == PA_F16) return launch_window_t<PA_F16, PA_F16, D, false>(a, stream);
  if (k == PA_BF16 && v == PA_BF16) return launch_window_t<PA_BF16, PA_BF16, D, false>(a, stream);
  if (k == F8 && v == PA_F16) return launch_window_t<F8, PA_F16, D, false>(a, stream);
  if (k == F8 && v == PA_BF16) return launch_window_t<F8, PA_BF16, D, false>(a, stream);
  if (k == PA_F16 && v == F8) return launch_window_t<PA_F16, F8, D, false>(a, stream);
  if (k == PA_BF16 && v == F8) return launch_window_t<PA_BF16, F8, D, false>(a, stream);
  return PA_ERR_DTYPE;
}

}  // namespace

// Parts: enough CTAs for every SM several times over, at least two tiles per
// warp in each.
void plan_window(WinArgs& a) {
  const int G = a.Hq / a.Hkv;
  const int mc = a.max_context_len > 0 ? a.max_context_len : 1;
  long long tiles = (mc + (long long)kTok - 1) / kTok;
  if (a.window > 0) {
    const long long w = ((long long)a.window + kTok - 1) / kTok + 1 +
                        ((long long)a.sinks + kTok - 1) / kTok;
    if (w < tiles) tiles = w;
  }
  const long long units = (long long)a.B * a.Hkv * ((G + kHeads - 1) / kHeads);
  long long P = (8LL * kSMs + units - 1) / units;
  const long long most = (tiles + 2 * kWarps - 1) / (2 * kWarps);
  if (P > most) P = most;
  if (P < 1) P = 1;
  a.ptiles = (int)((tiles + P - 1) / P);
  a.P = (int)((tiles + a.ptiles - 1) / a.ptiles);
}

size_t window_scratch_bytes(int B, int Hq, int D, int P) { return workspace_bytes_for(B, Hq, D, P); }

int launch_decode_window(const WinArgs& a, cudaStream_t stream) {
  int rc = a.D == 64 ? launch_window_d<64>(a, stream) : launch_window_d<128>(a, stream);
  if (rc == PA_OK && a.P > 1) {
    const dim3 grid((unsigned)(((long long)a.B * a.Hq + 3) / 4));
    const cudaError_t e = a.D == 64
        ? launch_k(decode_window_merge_kernel<64>, grid, dim3(128), 0, stream, a)
        : launch_k(decode_window_merge_kernel<128>, grid, dim3(128), 0, stream, a);
    rc = e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  }
  return rc;
}

}  // namespace pa
