// decode_window.cu -- decode attention over part of a sequence's tokens (a
// sliding window and a few first tokens) and over the block-scaled 8-bit cache,
// 16- and 8-bit pools.
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
// bound by HBM, so the kernel is built around bytes in flight. One CTA per SM:
// a producer warp and eight consumer warps around a ring of 192 KB. A step of the
// ring holds, for a group of HG = 8, 4, 2 or 1 neighbouring KV heads, 8 / HG
// sub-tiles of 16 or 32 tokens, so that every consumer warp has one (head,
// sub-tile): TMA brings 16 tokens of all the group's heads in one box (4-32 KB;
// boxes of one head are bound by TMA issue), 128-byte swizzled. With HG = 8
// each warp owns a head's whole softmax and never meets the others.
//
// Work split. A unit is (sequence, group of HG KV heads, chunk of up to 8 query
// heads); the CTAs take equal shares of the units' costs (window_common.cuh). A
// unit inside one share is written to the output; a cut one leaves one piece per
// CTA (slot 2c + 1 where the unit starts, 2c in the CTAs after it) that the merge
// kernel joins in the order of the CTAs. No CTA waits for another.
//
// The products are warp-level m16n8k16 MMAs whose operands the warp reads from
// its tile in the order the instruction wants:
//   S[16 x 8 keys]  = Q . K^T : A = the query heads in rows 0-7, what their
//     rounding to 16 bits lost in rows 8-15 (an 8-bit pool meets queries of any
//     type at ~22 bits), B = K rows as they lie, the dims permuted alike on both
//     sides so a lane's operands are one 16-byte run of a row;
//   O[16 x 8 dims] += P . V : rows 0-7 the weights, rows 8-15 what their rounding
//     to 16 bits lost, so the MMA rows that 8 heads leave empty carry the second
//     half of the precision and the two halves are added at the end.
// Over f16 and 8-bit V the weights are f16, whose grid ends at 2^-24. One key that takes most of
// the weight (the first tokens that a window keeps are there for that) would leave every other
// weight on that grid's last steps, and their second parts with them. So the reference lies 2^7
// under the maximum, which puts the largest weight into [2^7, 2^15], and the second parts are
// stored 2^11 times larger (rows 8-15 have sums of their own): a weight is held to 2^-22 of itself
// and 2^-43 of the row's largest. bf16 has fp32's range and needs neither.
// 8-bit codes are widened to f16 (exactly) between shared memory and the MMA. The
// 8 keys of a score product are tokens 0 4 2 6 5 1 7 3 of their tile: in that order
// both the K reads (4 chunks of 2 rows) and the V reads (2 chunks of 4 rows) of
// eight lanes fall on different banks under the 128-byte swizzle.
// (Warp-level MMAs rather than tcgen05: at 4-16 flops per byte the tensor work is a
// few percent of either pipe, and they take the weights from the registers the
// softmax leaves them in, while a tcgen05 tile pays a round trip of scores and
// weights through tensor memory and, for 8-bit V, a widened copy of the tile in
// shared memory.)
//
// Measured (one B200, copy rate 6.55 TB/s; calls back to back): 64 fp16 MHA sequences under a
// window of 1000 (846 MB) 143-147 us, 5.8 TB/s; 8 long bf16 GQA sequences under a window of 4096
// (137 MB) 39 us, 3.5 TB/s; block-scaled GQA (550 MB) 118-124 us (through a graph 115), 4.5 TB/s,
// and one long sequence (205 MB) 53 us, 3.9 TB/s. In steady state a CTA runs at ~95% of its part
// of the copy rate; ~2 us go by before a CTA knows its share, as much again until its first tile
// is there, ~5 with the merge kernel, and the SMs' speeds differ by 7% either way. When those
// figures were 142, 38, 109 and 50, a ring of cp.async copies per warp instead took 323, 43, 251
// and 86 us, and eight consumer warps without the register split (whose producer then spills)
// 144, 41, 122 and 51.
//
// Block-scaled pools: K's power of two multiplies the scores of its block's
// tokens. V's would have to multiply the weights before they are rounded to
// 16 bits, where a small scale would push them under f16's range; instead the
// running maximum is taken over log2 of the whole contribution, s' = s + log2(vs)
// (an exact integer): weights w = 2^(s' - m) are normalised to the largest
// contribution. The exp-sum has a reference r of its own, over the scores alone,
// l = sum 2^(s - r): a block of tiny V counts in it although its contribution is nothing
// (w 2^-log2(vs) would lose it once w is under fp32's range). The row is O / l 2^(m - r); both
// references are whole numbers, so that factor is exact. The second exponential per score
// is 4 of a lane and box, beside the widening of 128 codes.
//
// Every pipeline wait is bounded (wait_ns, 1 s): one that gives up sets PA_DEV_TIMEOUT,
// raises the CTA's abort flag, and the producer waits for its copies in flight.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "tc_ptx.cuh"
#include "window_common.cuh"

namespace pa {

namespace {

using namespace tc;

constexpr int kCons = 8;                        // consumer warps
constexpr int kThreads = (kCons + 4) * 32;      // two warpgroups of consumers, one with the producer
constexpr int kRing = 192 * 1024;
constexpr int kHeads = 8;                       // query heads of a KV head per unit
constexpr int kMaxSub = 16;                     // (box, head) pairs of a step

// Token of key n of an 8-key score product.
__device__ __forceinline__ int tok_of(int n) { return (int)((0x37156240u >> (4 * n)) & 7u); }

// What the consumers of a step need of it: per box its first token (-1: not there),
// per (box, head) the scales.
struct Meta {
  int t0[kMaxSub];
  float ks[kMaxSub];
  int lvs[kMaxSub];                             // log2 of the V scale; kNoScale: skip the box
};
constexpr int kNoScale = 1 << 20;

template <int KT, int VT, int D, bool BSC>
struct Core {
  static constexpr bool KBF = KT == PA_BF16, VBF = VT == PA_BF16;
  static constexpr bool K8 = KT == PA_FP8_E4M3, V8 = VT == PA_FP8_E4M3;
  static constexpr int EK = esize(KT), EV = esize(VT);
  static constexpr int TW = D * (EK + EV) <= 256 ? 2 : 1;       // 16-token boxes of a warp per step
  static constexpr int LBK = D * EK < 128 ? D * EK : 128;       // bytes of a line of a K row
  static constexpr int LBV = D * EV < 128 ? D * EV : 128;
  static constexpr int KBYTES = kCons * TW * kTok * D * EK, VBYTES = kCons * TW * kTok * D * EV;
  static constexpr int STAGE = KBYTES + VBYTES;
  static constexpr int NST = kRing / STAGE;
  static constexpr int KS = D / 16;             // k-steps of the score product
  static constexpr int NT = D / 8;              // 8-wide dim tiles of the output product
  static constexpr int RUN = K8 ? 16 : 8;       // dims of a lane's run of a K row
  static constexpr int EPV = V8 && D == 128 ? 16 : 8;   // dims of a lane's run of a V row
  static constexpr int NS = 2 * NT;             // output values per lane: slot e * NT + j
  // The reference is set 2^kLow under a maximum and moves when passed by 2^kMove: f16
  // weights reach 2^15, and the second part of one, at most 2^4, times kUp too.
  static constexpr float kLow = VBF ? 0.f : 7.f, kMove = VBF ? 8.f : 15.f;
  static constexpr float kUp = VBF ? 1.f : 2048.f;
  static_assert(NST >= 3 && kRing % STAGE == 0, "ring");

  static constexpr float kSumMove = 40.f;       // r moves when passed by 2^40: l < 2^40 tokens

  uint32_t qa[KS][4];
  float factor, m, l;
  float r;                                      // BSC: the exp-sum's reference
  float o[NT][4];
  // offsets of this lane's operands in a head's box
  uint32_t kx;                                  // K: key tok_of(g), chunk t (chunk 4 + t: ^ 64)
  uint32_t vx[2];                               // V: tokens of keys 2 t and 2 t + 1, run g

  static __device__ __forceinline__ int dim_of(int s, int lane) {
    const int e = s / NT, j = s % NT;
    return (j / EPV) * (8 * EPV) + (2 * (lane & 3) + e) * EPV + j % EPV;
  }
  // 16-byte chunk c of token row r within a line of LB bytes, as TMA swizzles it
  template <int LB> static __device__ __forceinline__ uint32_t at(int r, int c) {
    return (uint32_t)(r * LB + ((LB == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4));
  }
  __device__ __forceinline__ void init(int lane) {
    const int g = lane >> 2, t = lane & 3;
    kx = at<LBK>(tok_of(g), t);
    for (int i = 0; i < 2; ++i)
      vx[i] = LBV == 128 ? at<LBV>(tok_of(2 * t + i), g) : at<LBV>(tok_of(2 * t + i), g >> 1) + 8 * (g & 1);
  }

  // the unit's query heads [gc][D]; an 8-bit K pool takes each scaled by a power
  // of two that puts its largest element into [2^14, 2^15)
  __device__ __forceinline__ void start(const WinArgs& a, size_t q0, int gc, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float x[D / 4];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < D / (4 * RUN); ++i) {
#pragma unroll
      for (int c = 0; c < RUN / 8; ++c) {
        float* f = x + i * RUN + c * 8;
        if (g < gc) {
          const size_t p = q0 + (size_t)g * D + i * 4 * RUN + t * RUN + c * 8;
          if (a.q_dtype == PA_F32) {
            widen16<float>(*reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + p), f);
            widen16<float>(*reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + p + 4), f + 4);
          } else if (a.q_dtype == PA_F16) {
            widen16<__half>(*reinterpret_cast<const uint4*>(static_cast<const __half*>(a.q) + p), f);
          } else {
            widen16<__nv_bfloat16>(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + p), f);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = 0.f;
        }
      }
    }
    factor = a.scale_log2;
    if (K8) {
#pragma unroll
      for (int k = 0; k < D / 4; ++k) top = fmaxf(top, fabsf(x[k]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = (int)(__float_as_uint(top) >> 23) - 127;    // exponent of the largest element
      if (e >= -100 && e < 127) {
        const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);   // 2^(14 - e)
#pragma unroll
        for (int k = 0; k < D / 4; ++k) x[k] *= up;
        factor = a.scale_log2 * __uint_as_float((uint32_t)(e - 14 + 127) << 23);
      }
    }
    // k-step 2 i + j (16-bit K) or 4 i + j (codes): 4 elements of the lane's run i
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      split2<KBF>(x[4 * ks], x[4 * ks + 1], qa[ks][0], qa[ks][1]);
      split2<KBF>(x[4 * ks + 2], x[4 * ks + 3], qa[ks][2], qa[ks][3]);
    }
    m = r = -FLT_MAX;
    l = 0.f;
#pragma unroll
    for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  }

  // TW boxes of the warp's head. kb, vb: the head's part of box 0 in the stage,
  // kbox, vbox: from box to box, khalf, vhalf: from a row's first line to its second.
  __device__ __forceinline__ void step(uint32_t kb, uint32_t vb, uint32_t kbox, uint32_t vbox,
                                       uint32_t khalf, uint32_t vhalf, const Span& sp, const int* t0,
                                       const float* ks, const int* lvs, int lane) {
    const int t = lane & 3;
    // ---- scores: two 8-key products per box
    float s[TW][2][2];
#pragma unroll
    for (int w = 0; w < TW; ++w) {
      float c[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < D / (4 * RUN); ++i) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint4 v = lds16(kb + w * kbox + (LBK == 128 ? (i >> 1) * khalf : 0) + 8 * nt * LBK +
                                ((i & 1) ? kx ^ 64u : kx));
          if (K8) {
            const uint32_t ww[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t b0, b1;
              widen4(ww[j], b0, b1);
              mma<false>(c[nt], qa[(4 * i + j) % KS], b0, b1);
            }
          } else {
            mma<KBF>(c[nt], qa[(2 * i) % KS], v.x, v.y);
            mma<KBF>(c[nt], qa[(2 * i + 1) % KS], v.z, v.w);
          }
        }
      }
      // head g over the tokens of keys 8 nt + 2 t + {0, 1}
      const float f = BSC ? factor * ks[w] : factor;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s[w][nt][e] = (c[nt][e] + c[nt][e + 2]) * f;
          if (BSC) s[w][nt][e] += (float)lvs[w];      // s'
        }
    }
    bool whole[TW];
#pragma unroll
    for (int w = 0; w < TW; ++w) {
      whole[w] = t0[w] >= 0 && sp.whole(t0[w]);
      if (!whole[w]) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (t0[w] < 0 || !sp.sees(t0[w] + 8 * nt + tok_of(2 * t + e))) s[w][nt][e] = -CUDART_INF_F;
      }
    }
    // ---- online softmax
    float mx = -CUDART_INF_F, mr = -CUDART_INF_F;
#pragma unroll
    for (int w = 0; w < TW; ++w) {
      const float most = fmaxf(fmaxf(s[w][0][0], s[w][0][1]), fmaxf(s[w][1][0], s[w][1][1]));
      mx = fmaxf(mx, most);
      if (BSC) mr = fmaxf(mr, most - (float)lvs[w]);
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    if (__any_sync(0xffffffffu, mx - m > kMove || (BSC && mr > r + kSumMove))) {
      const float mn = mx - m > kMove ? floorf(mx) - kLow : m;
      const float alpha = ex2(m - mn);
      m = mn;
      if (!BSC) l *= alpha;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        o[j][0] *= alpha; o[j][1] *= alpha; o[j][2] *= alpha; o[j][3] *= alpha;
      }
      if (BSC) {
        mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, 1));
        mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, 2));
        const float rn = mr > r + kSumMove ? floorf(mr) : r;
        l *= ex2(r - rn);
        r = rn;
      }
    }
#pragma unroll
    for (int w = 0; w < TW; ++w) {
      float p[2][2], sum = 0.f;
      const float back = (float)lvs[w] + r;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[nt][e] = ex2(s[w][nt][e] - m);
          sum += BSC ? ex2(s[w][nt][e] - back) : p[nt][e];
        }
      l += sum;
      uint32_t pw[4];
      split2<VBF>(p[0][0], p[0][1], pw[0], pw[1], kUp);
      split2<VBF>(p[1][0], p[1][1], pw[2], pw[3], kUp);
      // ---- O += P . V: the lane's tokens are those of keys 2 t, 2 t + 1 and 8 + them
      if (t0[w] < 0) continue;                  // what lies in the stage may be anything
      uint32_t keep = 15u;                      // which of the four to take: V rows that are not
      if (!whole[w]) {                          // visible may hold NaN, their weights are 0
        keep = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          keep |= sp.sees(t0[w] + 8 * (i >> 1) + tok_of(2 * t + (i & 1))) ? 1u << i : 0u;
      }
      const uint32_t base = vb + w * vbox;
      if constexpr (V8 && D == 64) {
        uint2 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = lds8(base + 8 * (i >> 1) * LBV + vx[i & 1]);
          if (!((keep >> i) & 1u)) v[i] = make_uint2(0, 0);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
          codes(q, pw, q ? v[0].y : v[0].x, q ? v[1].y : v[1].x, q ? v[2].y : v[2].x, q ? v[3].y : v[3].x);
      } else {
#pragma unroll
        for (int cg = 0; cg < D * EV / LBV; ++cg) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = lds16(base + cg * vhalf + 8 * (i >> 1) * LBV + vx[i & 1]);
            if (!((keep >> i) & 1u)) v[i] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t r0 = (&v[0].x)[q], r1 = (&v[1].x)[q], r2 = (&v[2].x)[q], r3 = (&v[3].x)[q];
            if (V8) {
              codes(q, pw, r0, r1, r2, r3);
            } else {
              mma<VBF>(o[(8 * cg + 2 * q) % NT], pw, __byte_perm(r0, r1, 0x5410), __byte_perm(r2, r3, 0x5410));
              mma<VBF>(o[(8 * cg + 2 * q + 1) % NT], pw, __byte_perm(r0, r1, 0x7632),
                       __byte_perm(r2, r3, 0x7632));
            }
          }
        }
      }
    }
  }
  // four dims' products from four codes of each of the lane's tokens
  __device__ __forceinline__ void codes(int q, const uint32_t* pw, uint32_t r0, uint32_t r1, uint32_t r2,
                                        uint32_t r3) {
    const uint32_t x0 = __byte_perm(r0, r1, 0x5140), x1 = __byte_perm(r0, r1, 0x7362);
    const uint32_t y0 = __byte_perm(r2, r3, 0x5140), y1 = __byte_perm(r2, r3, 0x7362);
    uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
    widen4(x0, a0, a1);
    widen4(x1, a2, a3);
    widen4(y0, b0, b1);
    widen4(y1, b2, b3);
    mma<false>(o[(4 * q) % NT], pw, a0, b0);
    mma<false>(o[(4 * q + 1) % NT], pw, a1, b1);
    mma<false>(o[(4 * q + 2) % NT], pw, a2, b2);
    mma<false>(o[(4 * q + 3) % NT], pw, a3, b3);
  }
  __device__ __forceinline__ float value(int s) const {
    const int e = s / NT, j = s % NT;
    return fmaf(o[j][e + 2], 1.f / kUp, o[j][e]);
  }
};

// A piece of a cut unit holds normalised rows, and of each the exp-sum as l * 2^ref with l in
// [1, 2) (0: nothing attended; scores in the 10^5s: l as it is).
__device__ __forceinline__ void put_sum(float* ws_m, float* ws_l, size_t i, float ref, float l) {
  const uint32_t b = __float_as_uint(l);
  if (l > 0.f && l <= FLT_MAX && fabsf(ref) < 65536.f) {    // (ref + exponent is exact there)
    ref += (float)((int)(b >> 23) - 127);
    l = __uint_as_float((b & 0x7fffffu) | 0x3f800000u);
  }
  ws_m[i] = ref;
  ws_l[i] = l;
}

// n consecutive values to out[i ..]: 8 to a 16-bit output or 4 to an fp32 one at once.
__device__ __forceinline__ void store8_out(void* out, size_t i, const float* f, int dt) {
  if (dt == PA_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + i);
    p[0] = make_float4(f[0], f[1], f[2], f[3]);
    p[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (dt == PA_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

constexpr int kMaxStages = 6;
// ring | metadata, barriers | sums to join (groups of fewer than 8 heads only)
template <class C> constexpr int meta_bytes() { return C::NST * (int)sizeof(Meta) + 2 * kMaxStages * 8; }
template <class C> constexpr int smem_bytes(int hg) {
  return 1024 + kRing + meta_bytes<C>() + (hg < kCons ? kCons * C::NS * 32 * 4 : 0);
}

}  // namespace

template <int KT, int VT, int D, bool BSC>
__global__ void __launch_bounds__(kThreads, 1)
decode_window_kernel(const WinArgs a, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV) {
  using C = Core<KT, VT, D, BSC>;
  constexpr int NST = C::NST, TW = C::TW;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  Meta* meta = reinterpret_cast<Meta*>(smem + kRing);
  float* sm_join = reinterpret_cast<float*>(smem + kRing + meta_bytes<C>());
  const uint32_t sring = smem_addr(smem);
  const uint32_t bars = smem_addr(meta + NST);
  auto full = [&](int s) { return bars + 16u * (uint32_t)s; };
  auto empty = [&](int s) { return bars + 16u * (uint32_t)s + 8u; };
  __shared__ uint32_t sm_abort;
  __shared__ float sm_m[kCons][kHeads], sm_l[kCons][kHeads], sm_r[BSC ? kCons : 1][kHeads];
  volatile uint32_t* abort_flag = &sm_abort;
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == kCons * 32) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmV)) : "memory");
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kCons);
    }
    sm_abort = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();

  const int G = a.Hq / a.Hkv;
  const int hg = a.hg, nsub = kCons / hg, nbox = nsub * TW;
  const int chunks = (G + kHeads - 1) / kHeads;
  const int ny = a.Hkv / hg * chunks;
  const int cta = blockIdx.x;
  Share w = find_share<kThreads>(a, ny, nbox, cta, gridDim.x);    // (its barriers publish the inits)
  if (cta >= w.shares) return;
  const int units = a.B * ny;
  const uint32_t kboxb = (uint32_t)(hg * kTok * D * C::EK), vboxb = (uint32_t)(hg * kTok * D * C::EV);

  // 384 threads are launched with 168 registers each; the producer's warpgroup gives
  // half of its own to the consumers: 128 * 88 + 256 * 208 = 64,512 = 384 * 168
  if (warp >= kCons) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp > kCons) return;
    // ------------------------------------------------------------ producer
    int seq = 0;
    bool stop = false;
    while (!stop && w.p0 < units && w.base0 < w.hi) {
      const Batch u = next_batch(a, w, ny, nbox, cta, lane);
      for (int i = 0; i < u.count && !stop; ++i) {
        const int s0 = __shfl_sync(0xffffffffu, u.s0, i), s1 = __shfl_sync(0xffffffffu, u.s1, i);
        if (s0 >= s1) continue;
        const int b = __shfl_sync(0xffffffffu, u.b, i);
        const int h0 = __shfl_sync(0xffffffffu, u.y, i) / chunks * hg;
        const Span sp = span_of(a, __shfl_sync(0xffffffffu, u.ctx, i));
        const int32_t* table = a.block_tables + (size_t)b * a.max_blocks;
        // this lane's box of step k: its id, two steps ahead; then its scales (lane =
        // (box, head)), one ahead
        auto fetch = [&](int k) {
          const int v = k * nbox + lane;
          return lane < nbox && k < s1 && v < sp.n ? __ldg(table + sp.tile(v) * kTok / a.bs) : -1;
        };
        float ks_n = 1.f, vs_n = 1.f;
        auto fetch_scales = [&](int id) {
          if (BSC) {
            const int bid = __shfl_sync(0xffffffffu, id, lane / hg);
            if (lane < nbox * hg && bid >= 0 && bid < a.num_blocks) {
              ks_n = __ldg(a.k_scales + (size_t)bid * a.Hkv + h0 + lane % hg);
              vs_n = __ldg(a.v_scales + (size_t)bid * a.Hkv + h0 + lane % hg);
            }
          }
        };
        int id1 = fetch(s0), id2 = fetch(s0 + 1);
        fetch_scales(id1);
        for (int k = s0; k < s1; ++k, ++seq) {
          const int id = id1;
          const float ks = ks_n, vs = vs_n;
          id1 = id2;
          id2 = fetch(k + 2);
          fetch_scales(id1);
          const int v = k * nbox + lane;
          const bool want = lane < nbox && v < sp.n;
          const int t0 = want ? sp.tile(v) * kTok : -1;
          const bool ok = want && id >= 0 && id < a.num_blocks;
          if (want && !ok) flag_error(a.err_flag, PA_DEV_BAD_BLOCK_ID);
          const uint32_t have = __ballot_sync(0xffffffffu, ok);
          const int st = seq % NST;
          bool room = true;
          if (lane == 0) room = mbar_wait(empty(st), ((seq / NST) & 1) ^ 1, abort_flag, a.wait_ns);
          if (!__shfl_sync(0xffffffffu, room, 0)) { stop = true; break; }
          if (a.test_withhold && seq == 0) continue;
          // the copies first: the step's barrier cannot complete before lane 0 arrives
          // with the expected bytes, once the scales are here and written
          if (ok) {
            const uint32_t dst = sring + st * C::STAGE;
            const int off = t0 & (a.bs - 1);
            tma_load_5d(dst + lane * kboxb, &tmK, 0, off, h0, 0, id, full(st));
            tma_load_5d(dst + C::KBYTES + lane * vboxb, &tmV, 0, off, h0, 0, id, full(st));
          }
          if (lane < kMaxSub) {
            meta[st].t0[lane] = ok ? t0 : -1;
            if (BSC) {
              const bool there = lane < nbox * hg && ((have >> (lane / hg)) & 1u);
              const bool good = block_scale_ok(ks) && block_scale_ok(vs);
              if (there && !good) flag_error(a.err_flag, PA_DEV_BAD_SCALE);
              meta[st].ks[lane] = there && good ? ks : 1.f;
              meta[st].lvs[lane] = !there || good ? (there ? block_scale_log2(vs) : 0) : kNoScale;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(full(st), (uint32_t)__popc(have) * (kboxb + vboxb));
        }
      }
    }
    if (lane == 0) {
      if (stop) {
        *abort_flag = 1u;
        flag_error(a.err_flag, PA_DEV_TIMEOUT);
      }
      // never leave with copies in flight
      for (int q = max(a.test_withhold ? 1 : 0, seq - NST); q < seq; ++q) {
        const uint64_t b0 = globaltimer();
        while (!mbar_try(full(q % NST), (q / NST) & 1) && globaltimer() - b0 < kWaitNs) {}
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
  const int hd = warp % hg, sub = warp / hg;    // the warp's head of the group and its sub-tile
  const uint32_t khead = (uint32_t)(hd * kTok * C::LBK), vhead = (uint32_t)(hd * kTok * C::LBV);
  const uint32_t khalf = (uint32_t)(hg * kTok * C::LBK), vhalf = (uint32_t)(hg * kTok * C::LBV);
  auto cons_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kCons * 32) : "memory"); };
  C core;
  core.init(lane);
  bool failed = false;
  int seq = 0;
  while (w.p0 < units && w.base0 < w.hi) {
    const int p0 = w.p0;
    const Batch u = next_batch(a, w, ny, nbox, cta, lane);
#pragma unroll 1
    for (int i = 0; i < u.count; ++i) {
      const int b = __shfl_sync(0xffffffffu, u.b, i), y = __shfl_sync(0xffffffffu, u.y, i);
      const int s0 = __shfl_sync(0xffffffffu, u.s0, i), s1 = __shfl_sync(0xffffffffu, u.s1, i);
      const int ctx = __shfl_sync(0xffffffffu, u.ctx, i), n = __shfl_sync(0xffffffffu, u.n, i);
      const int first = __shfl_sync(0xffffffffu, u.first, i), last = __shfl_sync(0xffffffffu, u.last, i);
      const bool starts = __shfl_sync(0xffffffffu, (int)u.starts, i);
      const int h = y / chunks * hg + hd, chunk = y % chunks;
      const int gc = min(kHeads, G - chunk * kHeads);
      const size_t row0 = (size_t)b * a.Hq + h * G + chunk * kHeads;   // of this warp's head
      if (starts && threadIdx.x == 0) a.cuts[p0 + i] = make_int2(first, last);
      if (n == 0) {
        // an empty sequence's (or one of a bad length) rows are zeros
        if (starts && sub == 0) {
          if (y == 0 && threadIdx.x == 0 && ctx != 0) flag_error(a.err_flag, PA_DEV_BAD_CTX);
          for (int x = lane; x < gc * D; x += 32) store_out(a.out, row0 * D + x, 0.f, a.out_dtype);
        }
        continue;
      }
      if (s0 >= s1) continue;
      const Span sp = span_of(a, ctx);
      core.start(a, row0 * D, gc, lane);
#pragma unroll 1
      for (int k = s0; k < s1; ++k, ++seq) {
        const int st = seq % NST;
        // the warp gives up as one: what follows takes all of its lanes
        if (!failed && __any_sync(0xffffffffu, !mbar_wait(full(st), (seq / NST) & 1, abort_flag, a.wait_ns))) {
          failed = true;
          *abort_flag = 1u;
          if (lane == 0) flag_error(a.err_flag, PA_DEV_TIMEOUT);
        }
        if (failed) continue;
        int t0[TW], lvs[TW];
        float ks[TW];
        bool any = false;
#pragma unroll
        for (int x = 0; x < TW; ++x) {
          const int box = sub * TW + x;
          t0[x] = meta[st].t0[box];
          ks[x] = 1.f;
          lvs[x] = 0;
          if (BSC) {
            ks[x] = meta[st].ks[box * hg + hd];
            lvs[x] = meta[st].lvs[box * hg + hd];
            if (lvs[x] == kNoScale) { t0[x] = -1; lvs[x] = 0; }
          }
          any |= t0[x] >= 0;
        }
        if (any)
          core.step(sring + st * C::STAGE + sub * TW * kboxb + khead,
                    sring + st * C::STAGE + C::KBYTES + sub * TW * vboxb + vhead, kboxb, vboxb, khalf,
                    vhalf, sp, t0, ks, lvs, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(st));
      }
      // ---- the unit's end: this warp's sums to the output or to a piece
      core.l += __shfl_xor_sync(0xffffffffu, core.l, 1);
      core.l += __shfl_xor_sync(0xffffffffu, core.l, 2);
      const bool whole = first == last;
      const int g = lane >> 2;
      const size_t slot = 2 * (size_t)cta + (cta == first ? 1 : 0);
      const size_t prow = slot * (hg * kHeads) + hd * kHeads;          // of the pieces
      if (nsub == 1) {
        const Norm<BSC> norm = norm_of<BSC>(core.m - core.r, core.l, a.v_scale);
#pragma unroll
        for (int s = 0; s < C::NS; s += 8) {
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = norm(core.value(s + k));
          const int d = C::dim_of(s, lane);
          if (whole) {
            if (g < gc) store8_out(a.out, (row0 + g) * D + d, f, a.out_dtype);
          } else {
            store8_out(a.ws_acc, (prow + g) * D + d, f, PA_F32);
          }
        }
        if (!whole && (lane & 3) == 0)
          put_sum(a.ws_m, a.ws_l, prow + g, BSC ? core.r : core.m, core.l);
      } else {
        // the sub-tiles' warps of a head join their sums, each a part of the values
        cons_sync();                            // the last unit's sums have been read
        if ((lane & 3) == 0) {
          sm_m[warp][g] = core.m;
          sm_l[warp][g] = core.l;
          if (BSC) sm_r[warp][g] = core.r;
        }
#pragma unroll
        for (int s = 0; s < C::NS; ++s) sm_join[(warp * C::NS + s) * 32 + lane] = core.value(s);
        cons_sync();
        float M = -FLT_MAX, R = -FLT_MAX, L = 0.f;
        for (int x = 0; x < nsub; ++x) {
          M = fmaxf(M, sm_m[x * hg + hd][g]);
          if (BSC) R = fmaxf(R, sm_r[x * hg + hd][g]);
        }
        float cf[kCons];
#pragma unroll
        for (int x = 0; x < kCons; ++x) {
          cf[x] = x < nsub ? ex2(sm_m[x * hg + hd][g] - M) : 0.f;
          if (x < nsub) L = fmaf(sm_l[x * hg + hd][g], BSC ? ex2(sm_r[x * hg + hd][g] - R) : cf[x], L);
        }
        const Norm<BSC> norm = norm_of<BSC>(M - R, L, a.v_scale);
        for (int s = sub * (C::NS / nsub); s < (sub + 1) * (C::NS / nsub); ++s) {
          float O = 0.f;
#pragma unroll
          for (int x = 0; x < kCons; ++x)
            if (x < nsub) O = fmaf(sm_join[((x * hg + hd) * C::NS + s) * 32 + lane], cf[x], O);
          const int d = C::dim_of(s, lane);
          if (whole) {
            if (g < gc) store_out(a.out, (row0 + g) * D + d, norm(O), a.out_dtype);
          } else {
            a.ws_acc[(prow + g) * D + d] = norm(O);
          }
        }
        if (!whole && sub == 0 && (lane & 3) == 0)
          put_sum(a.ws_m, a.ws_l, prow + g, BSC ? R : M, L);
      }
    }
  }
}

// Units cut between CTAs: NW warps per (sequence, query head) join its pieces,
// every NW-th each, four pieces' loads in flight at a time. A piece is a normalised row and its
// exp-sum l 2^m: the row is the pieces' mean by those. (The weights are kept under 2^-8, so that the
// largest values do not leave fp32 before the division.)
template <int D, int NW>
__global__ void __launch_bounds__(NW < 4 ? 128 : NW * 32) decode_window_merge_kernel(const WinArgs a) {
  constexpr int PER = D / 32, RPB = NW < 4 ? 4 / NW : 1;         // rows per block
  __shared__ float sm_m[NW], sm_l[NW], sm_o[NW][D];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = blockIdx.x * (long long)RPB + warp / NW;
  const int part = warp % NW;
  // (for NW >= 4 the block is one row and takes every branch together)
  if (row >= (long long)a.B * a.Hq) return;
  const int b = (int)(row / a.Hq), hq = (int)(row - (long long)b * a.Hq);
  const int G = a.Hq / a.Hkv, h = hq / G, g = hq - h * G;
  const int chunks = (G + a.heads - 1) / a.heads;
  const int y = h / a.hg * chunks + g / a.heads;
  const int2 cut = a.cuts[(size_t)b * (a.Hkv / a.hg * chunks) + y];
  if (cut.x == cut.y) return;                  // whole, or empty
  // (a launch whose waits gave up may have left no cuts)
  if (cut.x < 0 || cut.y < cut.x || cut.y >= a.grid) return;
  const int rows = a.hg * a.heads, r = h % a.hg * a.heads + g % a.heads;
  float M = -FLT_MAX, L = 0.f, O[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) O[e] = 0.f;
  for (int c0 = cut.x + part; c0 <= cut.y; c0 += 4 * NW) {
    float m[4], l[4], v[4][PER];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = min(c0 + k * NW, cut.y);
      const size_t s = (2 * (size_t)c + (c == cut.x ? 1 : 0)) * rows + r;
      m[k] = a.ws_m[s];
      l[k] = a.ws_l[s];
      const float* p = a.ws_acc + s * D + lane * PER;
      if constexpr (PER == 4) {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[k][0] = x.x; v[k][1] = x.y;
      }
    }
    float mn = M;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + k * NW <= cut.y) mn = fmaxf(mn, m[k]);
    const float cs = ex2(M - mn);
    M = mn;
    L *= cs;
#pragma unroll
    for (int e = 0; e < PER; ++e) O[e] *= cs;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (c0 + k * NW > cut.y) continue;
      const float f = l[k] * ex2(m[k] - M - 9.f);
      L += f;
#pragma unroll
      for (int e = 0; e < PER; ++e) O[e] = fmaf(v[k][e], f, O[e]);
    }
  }
  if (NW >= 4) {
    if (lane == 0) { sm_m[warp] = M; sm_l[warp] = L; }
#pragma unroll
    for (int e = 0; e < PER; ++e) sm_o[warp][lane * PER + e] = O[e];
    __syncthreads();
    if (part != 0) return;
    M = -FLT_MAX;
    L = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) O[e] = 0.f;
#pragma unroll
    for (int x = 0; x < NW; ++x) M = fmaxf(M, sm_m[x]);
#pragma unroll
    for (int x = 0; x < NW; ++x) {
      const float f = ex2(sm_m[x] - M);
      L = fmaf(sm_l[x], f, L);
#pragma unroll
      for (int e = 0; e < PER; ++e) O[e] = fmaf(sm_o[x][lane * PER + e], f, O[e]);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int e = 0; e < PER; ++e)
    store_out(a.out, (size_t)row * D + lane * PER + e, O[e] * inv, a.out_dtype);
}

namespace {

// Pool [NB][bs][Hkv][D] seen as [NB][lines of a row][Hkv][bs][line]: a box of 16
// tokens of hg heads, every line of their rows.
bool make_map(const WinArgs& a, const void* pool, int dt, CUtensorMap* m) {
  auto enc = encode_fn();
  if (!enc || a.num_blocks <= 0) return false;
  const int es = dt == PA_FP8_E4M3 ? 1 : 2;
  const int lb = a.D * es < 128 ? a.D * es : 128, lines = a.D * es / lb;
  const cuuint64_t row = (cuuint64_t)a.D * es, tok = row * a.Hkv;
  const cuuint64_t dims[5] = {(cuuint64_t)(lb / es), (cuuint64_t)a.bs, (cuuint64_t)a.Hkv,
                              (cuuint64_t)lines, (cuuint64_t)a.num_blocks};
  const cuuint64_t strides[4] = {tok, row, (cuuint64_t)lb, tok * a.bs};
  const cuuint32_t box[5] = {(cuuint32_t)(lb / es), (cuuint32_t)kTok, (cuuint32_t)a.hg, (cuuint32_t)lines, 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc(m, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                        : dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
             5, const_cast<void*>(pool), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             lb == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KT, int VT, int D, bool BSC>
int launch_window_t(const WinArgs& a, cudaStream_t stream) {
  using C = Core<KT, VT, D, BSC>;
  static_assert(smem_bytes<C>(1) + 1024 <= 227 * 1024, "shared memory per CTA");
  const int smem = smem_bytes<C>(a.hg);
  auto kern = decode_window_kernel<KT, VT, D, BSC>;
  // dynamic shared memory above 48 KB needs the attribute, on the current device: always the most
  // any call of the kernel takes, as another thread's call may set it before this one's launch
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<C>(1)) != cudaSuccess)
    return PA_ERR_CUDA;
  CUtensorMap k, v;
  if (!make_map(a, a.k_cache, KT, &k) || !make_map(a, a.v_cache, VT, &v)) return PA_ERR_CUDA;
  return launch_k(kern, dim3((unsigned)a.grid), dim3(kThreads), smem, stream, a, k, v) == cudaSuccess
             ? PA_OK : PA_ERR_CUDA;
}

template <int D>
int launch_window_d(const WinArgs& a, cudaStream_t stream) {
  constexpr int F8 = PA_FP8_E4M3;
  if (a.k_scales) return launch_window_t<F8, F8, D, true>(a, stream);
  const int k = a.k_dtype, v = a.v_dtype;
  if (k == F8 && v == F8) return launch_window_t<F8, F8, D, false>(a, stream);
  if (k == PA_F16 && v == PA_F16) return launch_window_t<PA_F16, PA_F16, D, false>(a, stream);
  if (k == PA_BF16 && v == PA_BF16) return launch_window_t<PA_BF16, PA_BF16, D, false>(a, stream);
  if (k == F8 && v == PA_F16) return launch_window_t<F8, PA_F16, D, false>(a, stream);
  if (k == F8 && v == PA_BF16) return launch_window_t<F8, PA_BF16, D, false>(a, stream);
  if (k == PA_F16 && v == F8) return launch_window_t<PA_F16, F8, D, false>(a, stream);
  if (k == PA_BF16 && v == F8) return launch_window_t<PA_BF16, F8, D, false>(a, stream);
  return PA_ERR_DTYPE;
}

template <int D>
int launch_merge_d(const WinArgs& a, cudaStream_t stream) {
  const long long rows = (long long)a.B * a.Hq;
  // warps per row by the pieces to expect: with few units most CTAs hold a part of
  // one, with many a unit is rarely cut in more than two or three. The whole decode of 200,000
  // block-scaled tokens, 64 heads over 8, with 16 / 4 / 1 warps per row: 1 sequence 100 / 111 /
  // 145 us, 8 102 / 100 / 104, 20 107 / 100 / 101, 70 129 / 104 / 100, 128 157 / 111 / 102;
  // 8 heads over 1: 1 sequence 37 / 43 / 59, 16 33 / 34 / 37, 70 37 / 35 / 35.
  const long long units = rows / (a.hg * a.heads) + 1;
  cudaError_t e;
  if (units <= a.grid / 8)
    e = launch_k(decode_window_merge_kernel<D, 16>, dim3((unsigned)rows), dim3(512), 0, stream, a);
  else if (units <= a.grid / 2)
    e = launch_k(decode_window_merge_kernel<D, 4>, dim3((unsigned)rows), dim3(128), 0, stream, a);
  else
    e = launch_k(decode_window_merge_kernel<D, 1>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, stream, a);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// The unit of work, and one CTA per SM (fewer when there cannot be that many shares).
void plan_window(WinArgs& a) {
  const int G = a.Hq / a.Hkv;
  if (a.k_dtype == PA_F32) {
    a.hg = 1;
    a.heads = 4;
  } else {
    a.hg = a.Hkv % 8 == 0 ? 8 : a.Hkv % 4 == 0 ? 4 : a.Hkv % 2 == 0 ? 2 : 1;
    a.heads = kHeads;
  }
  const int mc = a.max_context_len > 0 ? a.max_context_len : 1;
  long long tiles = (mc + (long long)kTok - 1) / kTok;
  if (a.window > 0) {
    const long long w = ((long long)a.window + kTok - 1) / kTok + 1 +
                        ((long long)a.sinks + kTok - 1) / kTok;
    if (w < tiles) tiles = w;
  }
  const double units = (double)a.B * (a.Hkv / a.hg) * ((G + a.heads - 1) / a.heads);
  const double most = units * ((double)tiles * kTileCost + kUnitCost) / kMinShare;
  const int sms = sm_count_cached();
  a.grid = most >= sms ? sms : most < 1 ? 1 : (int)most;
}

// Two piece slots per CTA, then where each unit is cut.
size_t window_scratch_bytes(const WinArgs& a) {
  const size_t rows = 2 * (size_t)a.grid * a.hg * a.heads;
  const int G = a.Hq / a.Hkv;
  return up256(rows * a.D * 4) + 2 * up256(rows * 4) +
         up256((size_t)a.B * (a.Hkv / a.hg) * ((G + a.heads - 1) / a.heads) * sizeof(int2));
}
void carve_window(WinArgs& a, char* w) {
  const size_t rows = 2 * (size_t)a.grid * a.hg * a.heads;
  a.ws_acc = reinterpret_cast<float*>(w);
  w += up256(rows * a.D * 4);
  a.ws_m = reinterpret_cast<float*>(w);
  w += up256(rows * 4);
  a.ws_l = reinterpret_cast<float*>(w);
  w += up256(rows * 4);
  a.cuts = reinterpret_cast<int2*>(w);
}

int launch_decode_window(const WinArgs& a, cudaStream_t stream) {
  int rc = a.k_dtype == PA_F32 ? launch_decode_window_f32(a, stream)
           : a.D == 64 ? launch_window_d<64>(a, stream) : launch_window_d<128>(a, stream);
  // one CTA holds every unit whole
  if (rc == PA_OK && a.grid > 1)
    rc = a.D == 64 ? launch_merge_d<64>(a, stream) : launch_merge_d<128>(a, stream);
  return rc;
}

}  // namespace pa
