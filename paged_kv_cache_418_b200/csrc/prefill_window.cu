// prefill_window.cu -- paged prefill over a sliding window and a few first tokens,
// and over the block-scaled 8-bit cache, on the 5th-generation tensor cores.
//
// The new token at position p of its sequence attends the keys
//   t <= p  with  t > p - window  or  t < sinks      (window 0: every t <= p).
// Work unit = (sequence, chunk of 256 / G new tokens, KV head): two query tiles of 128
// rows (token, head of the group), each the M of its MMAs. Its key tiles are the 128-key
// tiles with a key some row attends: the first n0 (sinks) and those from w0 on (the window
// of its first token); a query tile skips those it attends nothing of. Blocks that no row
// attends are not loaded, nor are their table entries read. Per query tile and key tile
//   S[128 x 128] = Q . K^T, in two halves of 64 keys,
//   O[128 x 128] += P . V, P written over S in tensor memory,
// which fills tensor memory: 2 x (S 128 + O 128) columns. The two query tiles share every
// K and V tile (one copy, one widening), and one's products run while the other's softmax
// does; the scores of a half are issued as soon as the output product of the last tile's
// same half has read the weights under them, half a tile ahead of the softmax.
// A query tile has four softmax warps, a row per thread, 64 scores in registers at a time,
// and its own issuing warp. The reference maximum of a row moves only when a half passes it
// by far, and is floored at -FLT_MAX, so masked scores (-inf) need no guard. A tile that
// every row sees whole skips the masks.
//
// 16-bit pools: the products take the query's type, and the weights two 16-bit parts
// (hi + lo, ~16 bits).
// f16 weights (f16 and 8-bit V) end at 2^-24. One key that takes most of the weight (the first
// tokens that a window keeps are there for that) would leave every other weight on the last
// steps of that grid, so their reference lies 2^10 under the maximum: the largest weight of a row
// is in [2^10, 2^15.5], and half a step of the grid is 2^-35 of that. (Lower moves the reference
// more often, as the scores of a random prompt rise by 2^2 to 2^5 after the first keys: windowed
// f16 chunks 269 us at 2^9 and 2^10, 287 at 2^11, 304 at 2^12.)
// 8-bit pools: four converter warps widen each tile's codes to f16 (exactly, in place:
// TMA leaves a row's 128 codes in the line of its second half) ahead of the tensor
// cores; a bf16 query is rescaled by a power of two per row and becomes f16 too, exactly
// (an element 2^-39 of its row's largest is rounded), once per unit. Weights over 8-bit V
// are two f16 parts for fp32 and f16 outputs. For bf16 outputs, whose own half step is 2^-8 of a
// value, they are one, each off by up to 2^-11 of itself (8192-token prompt over the block-scaled
// cache: 661 us with one part, 792 with two).
//
// Where a unit has one query tile only, both groups take every other key tile of it, and
// the first joins the two parts (small ragged chunks: 17.9 -> 16.2 us; with two weight parts and
// the row sum's own reference 18.7).
//
// Measured (8192-token prompt, 32 query heads over 8, 550 GFLOP; calls back to back):
// block-scaled cache with bf16 output 681 us, 807 TFLOP/s, with f16 output (two weight parts)
// 810-860; 8-bit pools without block scales 613-669; bf16 pools 736-800. Windowed chunks (8 x
// 512) 274 us in bf16, 261-272 in f16. (The ranges are of several boxes and of the power limit,
// which the longer ones reach.) Units of one query tile whose rows two threads share took 763 us
// on the prompt and 298 on the bf16 chunks when this layout took 629 and 270, and with the codes
// widened by the softmax warps 2110. A pair of tiles took ~5000 cycles at 629 us: a softmax warp
// ~2100 for each half (some 1100 of them its 64 exponentials, beside the other query
// tile's) without ever waiting for scores; the tensor cores are busy for 2048 of them,
// shared memory for ~3000 (the operand of S that is the query is read once per 64 keys),
// the special-function units for 2048. What mattered besides the layout: elect.sync for the
// issuing threads (a product's issue took 110 cycles without it, 25 with it), an issuing
// warp per query tile (a step of the issue, waits and commits included, is ~1100 cycles),
// packed fp32 operations, and reading the block scales before the scores (shared-memory
// loads are slow beside the MMAs').
//
// Block-scaled pools: K's power of two multiplies its keys' scores; V's enters as its
// log2, s' = s + log2(vs), so the running maximum is that of the whole contribution and
// the weights 2^(s' - m) are normalised to the largest one. The row sum has a reference r of
// its own, over the scores alone, l = sum 2^(s - r): a block of tiny V counts in it although
// its contribution is nothing. 16 keys of one block share the factor 2^(m - log2(vs) - r)
// between the two; only where their contributions are all under 2^-96 of the reference (and
// fp32 is about to lose them) but a score over 2^-45 of r's are their exponentials taken a
// second time. A tile can hold such keys only if its least log2(vs) is under m - r - 51.
// The row is O / l 2^(m - r), exactly, as m - r is a whole number. (8192-token prompt: 650 us
// with the row sum taken from the weights, 677 so; all of this in the loop over the scores,
// unrolled, 778.) m itself is no whole number: 2^kLow under the maximum, not under its floor,
// the weight of a key that outweighs the rest is a power of two, which loses nothing to f16. The producer leaves a tile's scales and the mask of its missing
// blocks in a ring of shared-memory slots.
//
// CTA, persistent over rounds of units in alternating directions: warps 0-7 softmax,
// then (8-bit pools) 8-11 converters, then the TMA producer and the two MMA issuers. Every
// pipeline wait is bounded (wait_ns, 1 s); one that gives up sets PA_DEV_TIMEOUT, raises the
// CTA's abort flag, and every role drains its asynchronous work, frees tensor memory
// and returns.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <cfloat>

#include "pa_internal.h"
#include "tc_ptx.cuh"

namespace pa {

namespace {

using namespace tc;

constexpr int kD = 128;
constexpr int kM = 128;                         // rows of a query tile, two of which make a unit
constexpr int kTile = 128;                      // keys per tile
constexpr int kHalf = 128 * 128;                // one 64-wide d-half of a 128-row operand
constexpr int kOp = 2 * kHalf;                  // one 128 x 128 16-bit operand: 32 KB
constexpr int kNST = 4;                         // ring stages: K in the even ones, V in the odd ones
constexpr int kNQ = 3;                          // query tiles in shared memory
constexpr int kTmemCols = 512;                  // S/P x2, O x2 (by query tile of the unit)
constexpr int kSlots = 4;                       // tiles of scales and masks (see the producer)

constexpr int OFF_Q = 0;                        // [kNQ][32 KB]
constexpr int OFF_KV = kNQ * kOp;               // [kNST][32 KB]
constexpr int OFF_BAR = OFF_KV + kNST * kOp;
enum { B_FULL = 0, B_EMPTY = kNST, B_CONV = 2 * kNST, B_QFULL = 3 * kNST, B_QEMPTY = B_QFULL + kNQ,
       B_QCONV = B_QEMPTY + kNQ, B_SFULL = B_QCONV + kNQ, B_PREADY = B_SFULL + 4, B_OSTEP = B_PREADY + 4,
       B_OFULL = B_OSTEP + 2, B_ODONE = B_OFULL + 2, B_DONE = B_ODONE + 2, B_XCH = B_DONE + 2, B_COUNT = B_XCH + 1 };
constexpr int OFF_MISC = OFF_BAR + 8 * B_COUNT;
constexpr int OFF_SLOT = (OFF_MISC + 12 + 15) / 16 * 16;  // (tensor memory, abort flag, wait limit)
struct Slot {                                   // of a tile: what the producer knows of its blocks
  float ks[8], lvs[8];                          // K scale, log2 of the V scale
  uint32_t missing;                             // blocks that were not loaded
  float lvmin;                                  // the least of lvs
  uint32_t pad[2];
};
constexpr int OFF_ROWE = OFF_SLOT + kSlots * (int)sizeof(Slot);  // [kNQ][128] exponents of rescaled rows
constexpr int OFF_XCH = OFF_ROWE + kNQ * 128;                    // [2][128] maxima and sums of a second part
constexpr int kSmem = OFF_XCH + 2 * 128 * 4 + 1024;              // + alignment slack
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");

struct Args {
  void* out;
  int out_dtype;
  const int32_t* block_tables;
  int max_blocks;
  const int32_t* context_lens;
  const int32_t* query_start;
  int B, T, Hq, Hkv, num_blocks, chunks;
  float scale_log2;
  float v_scale;        // value of one V unit (FP8 V pool; 1 otherwise)
  int max_context_len;
  uint32_t* err_flag;
  int window, sinks;
  const float* k_scales;
  const float* v_scales;
  uint32_t wait_ns;             // limit of every pipeline wait
  int test_withhold;            // tests: leave the CTA's first query tile out
};

// Some rows attend keys t < t1 with t >= lo or t < sk.
struct Reach {
  int t1, lo, sk;
  // some of the n keys from t on are attended
  __device__ __forceinline__ bool needs(int t, int n) const { return t < t1 && (t + n > lo || t < sk); }
};
// ntok new tokens from position pos on
__device__ __forceinline__ Reach reach_of(const Args& a, int pos, int ntok) {
  Reach x;
  x.t1 = ntok > 0 ? pos + ntok : 0;
  x.lo = a.window > 0 && ntok > 0 ? max(0, pos - a.window + 1) : 0;
  x.sk = min(a.sinks, x.lo);
  return x;
}

struct Unit {
  int b, c, h;
  int qrow0;            // first query row (token) of the chunk in [T]
  int ntok;             // new tokens of the chunk (0: nothing to do)
  int pos0;             // position of the chunk's first token
  int tpt;              // tokens of a query tile
  Reach all;            // of the chunk; its tiles are the first n0 and those from w0 on
  int n0, w0, ntiles;
  bool bad;             // the sequence's lengths are inconsistent
  __device__ __forceinline__ int tile0(int k) const { return (k < n0 ? k : k - n0 + w0) * kTile; }
  __device__ __forceinline__ int tokens(int g) const { return min(tpt, ntok - g * tpt); }   // of query tile g
  __device__ __forceinline__ int pos(int g) const { return pos0 + g * tpt; }
  __device__ __forceinline__ bool two() const { return ntok > tpt; }
};

// What the g-th issuer and softmax warps do of a unit: query tile g and the key tiles it
// attends something of, or, where there is only one query tile, every other key tile of
// it (the two parts are joined at the end).
struct Part {
  Reach reach;
  int sinks, from, last;  // its key tiles: k < sinks, from <= k <= last (split: every other one)
  bool on, split;
  __device__ __forceinline__ bool takes(int g, int k) const {
    return split ? (k & 1) == g : k < sinks || (k >= from && k <= last);
  }
  // its first key tile, and the one behind k
  __device__ __forceinline__ int first(int g) const { return split ? g : sinks > 0 ? 0 : from; }
  __device__ __forceinline__ int next(int k) const {
    k += split ? 2 : 1;
    return k >= sinks && k < from ? from : k;
  }
};
__device__ __forceinline__ Part part_of(const Args& a, const Unit& x, int g) {
  Part p;
  p.split = !x.two() && x.ntiles > 1;
  p.on = g == 0 || x.two() || p.split;
  p.reach = x.two() ? reach_of(a, x.pos(g), x.tokens(g)) : x.all;
  p.last = x.two() ? (p.reach.t1 - 1) / kTile - x.w0 + x.n0 : x.ntiles - 1 - (p.split && ((x.ntiles - 1 - g) & 1));
  p.sinks = (p.reach.sk + kTile - 1) / kTile;
  if (p.sinks > x.n0) p.sinks = x.n0 + max(0, p.sinks - x.w0);
  p.from = p.reach.lo / kTile - x.w0 + x.n0;
  if (!p.on) p.sinks = 0, p.last = -1;
  if (p.split) p.from = 0;
  return p;
}

__device__ __forceinline__ Unit unit_of(const Args& a, int G, int bs, long long u) {
  Unit x;
  x.tpt = kM / G;
  x.h = (int)(u % a.Hkv);
  const long long t = u / a.Hkv;
  x.b = (int)(t % a.B);
  x.c = a.chunks - 1 - (int)(t / a.B);          // late chunks first: they attend the most keys
  const int qs = __ldg(a.query_start + x.b), qe = __ldg(a.query_start + x.b + 1);
  const int n = qe - qs, ctx = __ldg(a.context_lens + x.b);
  x.bad = qs < 0 || n < 0 || qe > a.T || ctx < n || ctx > (long long)a.max_blocks * bs || ctx > a.max_context_len;
  const long long done = (long long)x.c * 2 * x.tpt;    // the sequence's new tokens before the chunk
  x.ntok = x.bad ? 0 : (int)max(0ll, min(2ll * x.tpt, n - done));
  x.qrow0 = (int)(qs + done);
  x.pos0 = (int)(ctx - n + done);
  x.all = reach_of(a, x.pos0, x.ntok);
  x.w0 = x.all.lo / kTile;
  x.n0 = min((x.all.sk + kTile - 1) / kTile, x.w0);
  x.ntiles = x.n0 + (x.all.t1 + kTile - 1) / kTile - x.w0;
  return x;
}

// The k-th unit of CTA cta: rounds of grid units in alternating directions.
__device__ __forceinline__ long long unit_index(long long k, int cta, int grid) {
  return k * grid + ((k & 1) ? grid - 1 - cta : cta);
}

// Bounded wait for the phase with the given parity; false = gave up. The limit lies beside the
// abort flag: as a kernel argument it took registers of every role (windowed bf16 chunks
// 279 -> 295 us).
__device__ __forceinline__ bool pipe_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  if (mbar_try(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try(bar, parity)) return true;
    if (abort_flag[0] || globaltimer() - t0 > abort_flag[1]) return false;
  }
}

// One lane of the (converged) warp. Not lane == 0: only elect.sync tells the compiler
// that a single thread goes on, so that the operands of the tensor instructions need no
// loop over the lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mov.b64 c, {%6, %7};"
      " fma.rn.f32x2 d, a, b, c; mov.b64 {%0, %1}, d; }"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{ .reg .b64 a, b, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5};"
      " add.rn.f32x2 d, a, b; mov.b64 {%0, %1}, d; }"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Two fp32 weights (not negative) as packed 16-bit values, and (LO) what their rounding lost.
// f16 parts: hi is the weight cut to ten fraction bits, which takes no conversion back.
template <bool BF, bool LO>
__device__ __forceinline__ void pack2(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  if (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    if (LO) {
      const float2 f = __bfloat1622float2(h);
      const __nv_bfloat162 l = __floats2bfloat162_rn(p0 - f.x, p1 - f.y);
      lo = *reinterpret_cast<const uint32_t*>(&l);
    }
  } else {
    const float h0 = LO ? __uint_as_float(__float_as_uint(p0) & 0xffffe000u) : p0;
    const float h1 = LO ? __uint_as_float(__float_as_uint(p1) & 0xffffe000u) : p1;
    const __half2 h = __floats2half2_rn(h0, h1);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    if (LO) {
      const float2 f = fma2(make_float2(h0, h1), make_float2(-1.f, -1.f), make_float2(p0, p1));
      const __half2 l = __floats2half2_rn(f.x, f.y);
      lo = *reinterpret_cast<const uint32_t*>(&l);
    }
  }
}

// 16 packed columns of this thread's TMEM lane, without waiting.
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// 2^n of a whole number n, 0 under 2^-126 (n <= 127): without the special-function unit.
__device__ __forceinline__ float pow2_of(float n) {
  return __uint_as_float(__float_as_uint(fmaxf(n + 8388735.f, 8388608.f)) << 23);    // (2^23 + 127)
}

// One column of this thread's TMEM lane.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r) : "r"(taddr) : "memory");
  return __uint_as_float(r);
}

// Widen row `row` of a stage's codes (its line of the second half) to f16, in place;
// zero: zeros instead.
__device__ __forceinline__ void widen_row(uint8_t* stage, int row, bool zero) {
  const int sw = row & 7;
  const uint8_t* src = stage + kHalf + row * 128;
  uint4 c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    c[j] = zero ? make_uint4(0, 0, 0, 0) : *reinterpret_cast<const uint4*>(src + ((j ^ sw) << 4));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // codes 16 j .. 16 j + 15: d-half j / 4, 16-byte chunks 2 (j % 4) and the next
    const uint32_t w[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
          : "=r"(o[2 * k]), "=r"(o[2 * k + 1]) : "r"(w[k]));
    uint8_t* dst = stage + (j >> 2) * kHalf + row * 128;
    const int c0 = 2 * (j & 3);
    *reinterpret_cast<uint4*>(dst + ((c0 ^ sw) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(dst + (((c0 + 1) ^ sw) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

// Row `row` of a bf16 query operand as f16, in place, times the power of two that
// puts its largest element into [2^14, 2^15); returns that power's exponent.
__device__ __forceinline__ int rescale_row(uint8_t* op, int row) {
  // (the second look at the row is cheaper than 64 registers)
  auto chunk = [&](int j) {
    return reinterpret_cast<uint4*>(op + (j >> 3) * kHalf + row * 128 + (((j & 7) ^ (row & 7)) << 4));
  };
  float top = 0.f;
#pragma unroll 4
  for (int j = 0; j < 16; ++j) {
    float f[8];
    widen16<__nv_bfloat16>(*chunk(j), f);
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(f[k]));
  }
  int e = 14 - ((int)(__float_as_uint(top) >> 23) - 127);
  if (e < -113 || e > 114) e = 0;               // infinite, or too small to matter
  const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll 4
  for (int j = 0; j < 16; ++j) {
    float f[8];
    widen16<__nv_bfloat16>(*chunk(j), f);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 h = __floats2half2_rn(f[2 * k] * up, f[2 * k + 1] * up);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *chunk(j) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return e;
}

// Wait for this thread's tensor-memory loads, the 64 registers of which are not to be
// used before.
__device__ __forceinline__ void tmem_wait_ld64(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 64; i += 4)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3])::"memory");
}

// The row sum l 2^r of a part in one word, r given as a whole number of powers of two from the
// part's m (kMove, kSumMove and the V scales keep it within +-256 with l's own exponent): nine bits of
// exponent over l's fraction, 0 for no sum, 511 for one that is not finite.
__device__ __forceinline__ float pack_sum(float l, float r) {
  const uint32_t b = __float_as_uint(l);
  uint32_t w = 0;
  if (!(l <= FLT_MAX)) w = 511u << 23;
  else if (l > 0.f)
    w = (uint32_t)max(1, min(510, (int)(b >> 23) - 127 + (int)r + 256)) << 23 | (b & 0x7fffffu);
  return __uint_as_float(w);
}
// Its l, in [1, 2), and reference (r: the part's m).
__device__ __forceinline__ float unpack_sum(float word, float& r) {
  const uint32_t w = __float_as_uint(word);
  if (w == 0) return 0.f;
  if (w >> 23 == 511u) return CUDART_NAN_F;
  r += (float)((int)(w >> 23) - 256);
  return __uint_as_float((w & 0x7fffffu) | 0x3f800000u);
}

// Warps of the CTA and their registers, moved between warpgroups: without converters
// 384 threads are launched with 168 each: 256 * 208 + 128 * 88 = 64,512; with them 512
// with 128: 256 * 184 + 128 * 80 + 128 * 64 = 65,536.
template <bool CONV> struct Roles {
  static constexpr int kConv = 8, kProd = CONV ? 12 : 8, kMma = kProd + 1, kThreads = CONV ? 512 : 384;
};

}  // namespace

// FMT: the query's type (0 f16, 1 bf16). K8 / V8: that pool holds codes. BSC (K8 and
// V8): with scales per block and KV head. LO: weights in two parts.
template <int FMT, int BS, bool K8, bool V8, bool BSC, bool LO>
__global__ void __launch_bounds__((Roles<K8 || V8>::kThreads), 1)
prefill_window_kernel(const Args a, const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  constexpr bool CONV = K8 || V8;               // converter warps
  constexpr bool QC = K8 && FMT == 1;           // the query becomes f16
  constexpr int FS = K8 ? 0 : FMT, FO = V8 ? 0 : FMT;     // operand types of the two products
  // The reference of a row is set 2^kLow under its maximum and moves when a half tile passes it
  // by 2^kMove: rarely, as that waits for the output product in flight. f16 weights stay under
  // 65504, with half a power of two for a score whose maximum was rounded to fp32 before m was
  // subtracted; bf16 ones leave room for 2^60 of values and sums in fp32.
  constexpr float kLow = FO == 1 ? 0.f : 10.f, kMove = FO == 1 ? 64.f : 15.5f;
  constexpr float kSumMove = 8.f;               // BSC: r moves when passed by 2^8
  using R = Roles<CONV>;
  constexpr int NB_T = kTile / BS;              // physical blocks per tile
  constexpr uint32_t kBlkBits = (uint32_t)((1ull << BS) - 1ull);   // one block's keys in a chunk mask
  constexpr uint32_t IDESC_S = make_idesc(FS, 0, 0, kTile / 2, kM);
  constexpr uint32_t IDESC_O = make_idesc(FO, 0, 1, kD, kM);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_addr(smem);
  auto bar = [&](int i) { return sbase + OFF_BAR + 8u * (uint32_t)i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + OFF_MISC + 4);
  Slot* slots = reinterpret_cast<Slot*>(smem + OFF_SLOT);
  int8_t* rowe = reinterpret_cast<int8_t*>(smem + OFF_ROWE);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv;
  const long long U = (long long)a.B * a.chunks * a.Hkv;
  pdl_trigger();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kNST; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 2);
      mbar_init(bar(B_CONV + s), 128);
    }
    for (int i = 0; i < kNQ; ++i) {
      mbar_init(bar(B_QFULL + i), 1);
      // both issuers, and (QC) the softmax threads of both parts, which read the rows'
      // exponents: those of a part alone arrive twice
      mbar_init(bar(B_QEMPTY + i), QC ? 258 : 2);
      mbar_init(bar(B_QCONV + i), 128);
    }
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(bar(B_SFULL + 2 * i + h), 1);
        mbar_init(bar(B_PREADY + 2 * i + h), 128);
      }
      mbar_init(bar(B_OSTEP + i), 1);
      mbar_init(bar(B_DONE + i), 1);
      if (i == 0) mbar_init(bar(B_XCH), 128);
      mbar_init(bar(B_OFULL + i), 1);
      mbar_init(bar(B_ODONE + i), 128);
    }
    abort_flag[0] = 0u;
    abort_flag[1] = a.wait_ns;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == R::kMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_s = tmem;                  // S/P: [0, 128), [128, 256)
  const uint32_t tmem_o = tmem + 2 * kTile;      // O: [256, 384), [384, 512)
  auto give_up = [&]() {
    *abort_flag = 1u;
    flag_error(a.err_flag, PA_DEV_TIMEOUT);
  };
  // a stage holding K (kv = 0) or V (kv = 1) is ready for the tensor cores when TMA
  // filled it (16-bit pool) or when the converters widened it
  auto ready_bar = [&](int kv, int s) { return bar(((kv ? V8 : K8) ? B_CONV : B_FULL) + s); };

  if (warp >= R::kProd) {
    if constexpr (CONV) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == R::kProd) {
      // ---------------------------------------------------------- producer
      // The lanes share a tile's copies: lane q < NB_T has its q-th block, reads its id
      // two tiles ahead and its scales one ahead. It writes a tile's slot once it has the
      // tile's K stage, that is after the scores of the tile two before it and the output
      // products of the one before that: every softmax and converter thread is past the
      // slot of the tile four before, so four slots are enough.
      int tc_ = 0, issued = 0, qn = 0;
      bool stop = false;
      for (long long kk = 0; !stop; ++kk) {
        const long long u = unit_index(kk, blockIdx.x, gridDim.x);
        if (u >= U) break;
        const Unit x = unit_of(a, G, BS, u);
        if (lane == 0 && x.bad && x.c == 0 && x.h == 0) flag_error(a.err_flag, PA_DEV_BAD_CTX);
        if (x.ntok <= 0) continue;
        // query tile g: the first one ahead of the unit's tiles, the second behind the first
        // of them (its buffer is that of the last unit's first query tile)
        auto load_q = [&](int g) -> bool {
          const int qi = qn % kNQ;
          bool ok = true;
          if (lane == 0) {
            ok = pipe_wait(bar(B_QEMPTY + qi), ((qn / kNQ) & 1) ^ 1, abort_flag);
            if (ok && !(a.test_withhold && qn == 0)) {
              mbar_expect_tx(bar(B_QFULL + qi), (uint32_t)kOp);
              for (int hh = 0; hh < 2; ++hh)
                tma_load_4d(sbase + OFF_Q + qi * kOp + hh * kHalf, &tmQ, 0, hh, x.h * G, x.qrow0 + g * x.tpt,
                            bar(B_QFULL + qi));
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (ok) ++qn;
          return ok;
        };
        if (!load_q(0)) { stop = true; break; }
        const int32_t* table = a.block_tables + (size_t)x.b * a.max_blocks;
        // this lane's block of tile k is one some row attends; its id (-1: none)
        auto wants = [&](int k) { return lane < NB_T && x.all.needs(x.tile0(k) + lane * BS, BS); };
        auto fetch = [&](int k) -> int {
          return k < x.ntiles && wants(k) ? __ldg(table + x.tile0(k) / BS + lane) : -1;
        };
        float ks_n = 1.f, vs_n = 1.f;
        auto fetch_scales = [&](int id) {
          if (BSC && id >= 0 && id < a.num_blocks) {
            ks_n = __ldg(a.k_scales + (size_t)id * a.Hkv + x.h);
            vs_n = __ldg(a.v_scales + (size_t)id * a.Hkv + x.h);
          }
        };
        int id1 = fetch(0), id2 = fetch(1);
        fetch_scales(id1);
        for (int k = 0; k < x.ntiles && !stop; ++k, ++tc_) {
          int phys = id1;
          const float ks = ks_n, vs = vs_n;
          id1 = id2;
          id2 = fetch(k + 2);
          fetch_scales(id1);
          const bool want = wants(k);
          if (want && (phys < 0 || phys >= a.num_blocks)) {
            flag_error(a.err_flag, PA_DEV_BAD_BLOCK_ID);
            phys = -1;
          }
          if (BSC && want && phys >= 0 && !(block_scale_ok(ks) && block_scale_ok(vs))) {
            flag_error(a.err_flag, PA_DEV_BAD_SCALE);
            phys = -1;
          }
          const uint32_t here = __ballot_sync(0xffffffffu, phys >= 0);
          const int lvmin = BSC ? __reduce_min_sync(0xffffffffu, phys >= 0 ? block_scale_log2(vs) : 0x7fffffff) : 0;
          // per 128-byte line of rows of the blocks that are loaded
          const uint32_t bytes = (uint32_t)__popc(here) * (BS * 128u);
          for (int kv = 0; kv < 2; ++kv) {
            const int seq = 2 * tc_ + kv, s = seq % kNST;
            const bool codes = kv ? V8 : K8;
            bool room = true;
            if (lane == 0) room = pipe_wait(bar(B_EMPTY + s), ((seq / kNST) & 1) ^ 1, abort_flag);
            if (!__shfl_sync(0xffffffffu, room, 0)) { stop = true; break; }
            if (kv == 0) {
              Slot& slot = slots[tc_ % kSlots];
              if (BSC && lane < NB_T) {
                slot.ks[lane] = phys >= 0 ? ks : 1.f;
                slot.lvs[lane] = phys >= 0 ? (float)block_scale_log2(vs) : 0.f;
              }
              if (lane == 0) {
                slot.missing = ~here;
                if (BSC) slot.lvmin = (float)lvmin;
              }
              __syncwarp();
            }
            if (lane == 0) mbar_expect_tx(bar(B_FULL + s), codes ? bytes : 2u * bytes);
            __syncwarp();
            const uint32_t dst = sbase + OFF_KV + s * kOp;
            if (phys >= 0) {
              if (codes) {
                tma_load_4d(dst + kHalf + lane * (BS * 128), kv ? &tmV : &tmK, 0, 0, x.h, phys,
                            bar(B_FULL + s));
              } else {
                for (int hh = 0; hh < 2; ++hh)
                  tma_load_5d(dst + hh * kHalf + lane * (BS * 128), kv ? &tmV : &tmK, 0, 0, x.h, hh, phys,
                              bar(B_FULL + s));
              }
            }
            ++issued;
          }
          if (k == 0 && !stop && x.two() && !load_q(1)) stop = true;
        }
      }
      if (lane == 0) {
        if (stop) give_up();
        // never leave with copies in flight: the last loads of every stage and query buffer
        for (int seq = max(0, issued - kNST); seq < issued; ++seq) {
          const uint64_t t0 = globaltimer();
          while (!mbar_try(bar(B_FULL + seq % kNST), (seq / kNST) & 1) && globaltimer() - t0 < kWaitNs) {}
        }
        for (int q = max(a.test_withhold ? 1 : 0, qn - kNQ); q < qn; ++q) {
          const uint64_t t0 = globaltimer();
          while (!mbar_try(bar(B_QFULL + q % kNQ), (q / kNQ) & 1) && globaltimer() - t0 < kWaitNs) {}
        }
      }
    } else if (warp <= R::kMma + 1 && elect_one()) {
      // ---------------------------------------------------------- MMA issuers
      // One warp per query tile: a step of the issue (three waits, 12 or 16 products, two
      // commits) takes ~1100 cycles, so one warp for both would set the pace. Per key tile
      // and half of its keys: the output product of that half of the last key tile, then
      // this one's scores (over the weights that product has read: the tensor pipe is in
      // order), so that scores are ready half a tile ahead of the softmax. Stages and query
      // tiles are empty when both issuers are past them, and each issuer waits for every one
      // in turn, its own or not: a parity wait is only exact within one phase.
      const int g = warp - R::kMma;
      int tc_ = 0, qn = 0;                       // key tiles, query tiles of the CTA so far
      int tiles = 0, units = 0;                  // of this query tile
      bool ok = true;
      for (long long kk = 0; ok; ++kk) {
        const long long u = unit_index(kk, blockIdx.x, gridDim.x);
        if (u >= U) break;
        const Unit x = unit_of(a, G, BS, u);
        if (x.ntok <= 0) continue;
        const Part mine = part_of(a, x, g);
        const int qt = qn + (mine.split ? 0 : g), qi = qt % kNQ;
        const uint32_t qst = sbase + OFF_Q + qi * kOp;
        // the other part's query tile
        auto pass_q = [&](int q) -> bool {
          if (!pipe_wait(bar((QC ? B_QCONV : B_QFULL) + q % kNQ), (q / kNQ) & 1, abort_flag)) return false;
          mbar_arrive(bar(B_QEMPTY + q % kNQ));
          return true;
        };
        if (g == 1 && !mine.split && !pass_q(qn)) { ok = false; break; }
        int done = 0;                            // tiles whose scores were issued, of this unit
        bool pend = false;
        for (int k = 0; k <= x.ntiles && ok; ++k) {
          const bool was = pend, more = k < x.ntiles;
          const int seq = 2 * (tc_ + k), s = seq % kNST, sv = (seq - 1) % kNST;
          pend = more && mine.takes(g, k);
          const uint32_t kst = sbase + OFF_KV + s * kOp, vst = sbase + OFF_KV + sv * kOp;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // ---- the last tile: n-th of the query tile, the unit's first if first
            if (was) {
              const int n = tiles - 1 - (h == 1 && pend);
              const bool first = h == 0 && done == 1;
              ok = pipe_wait(bar(B_PREADY + 2 * g + h), n & 1, abort_flag);
              // O is that of the last unit until its epilogue has read it
              if (ok && first && units > 0) ok = pipe_wait(bar(B_ODONE + g), (units - 1) & 1, abort_flag);
              if (ok && h == 0) ok = pipe_wait(ready_bar(1, sv), ((seq - 1) / kNST) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int part = 0; part < (LO ? 2 : 1); ++part) {
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk) {
                  const uint64_t bd = sw128_desc(vst + h * (kTile / 2) * 128 + kk * 16 * 128, kHalf, 1024);
                  mma_f16_ta(tmem_o + g * kD,
                             tmem_s + g * kTile + h * (kTile / 2) + (kk >> 1) * 32 + part * 16 + (kk & 1) * 8,
                             bd, IDESC_O, (first && part == 0 && kk == 0) ? 0u : 1u);
                }
              }
              if (h == 0) mma_commit(bar(B_OSTEP + g));
              if (h == 1 && k - 1 == mine.last) {
                mma_commit(bar(B_OFULL + g));
                ++units;
              }
            } else if (k > 0 && h == 0 && !pipe_wait(ready_bar(1, sv), ((seq - 1) / kNST) & 1, abort_flag)) {
              ok = false;
              break;
            }
            if (k > 0 && h == 1) mma_commit(bar(B_EMPTY + sv));
            // ---- this one
            if (more && h == 0) {
              if (pend && done == 0)
                ok = pipe_wait(bar((QC ? B_QCONV : B_QFULL) + qi), (qt / kNQ) & 1, abort_flag);
              ok = ok && pipe_wait(ready_bar(0, s), (seq / kNST) & 1, abort_flag);
              if (!ok) break;
              done += pend;
              tiles += pend;
            }
            if (pend) {
              tc_fence_after();
#pragma unroll
              for (int ks = 0; ks < kD / 16; ++ks) {
                const uint64_t ad = sw128_desc(qst + (ks >> 2) * kHalf + (ks & 3) * 32, 16, 1024);
                const uint64_t bd = sw128_desc(kst + (ks >> 2) * kHalf + h * (kTile / 2) * 128 + (ks & 3) * 32, 16, 1024);
                mma_f16(tmem_s + g * kTile + h * (kTile / 2), ad, bd, IDESC_S, ks > 0 ? 1u : 0u);
              }
              mma_commit(bar(B_SFULL + 2 * g + h));
              if (h == 1 && k == mine.last) mma_commit(bar(B_QEMPTY + qi));
            }
            if (more && h == 1) mma_commit(bar(B_EMPTY + s));
          }
        }
        if (ok && g == 0 && x.two()) ok = pass_q(qn + 1);
        tc_ += x.ntiles;
        qn += x.two() ? 2 : 1;
      }
      if (!ok) give_up();
      mma_commit(bar(B_DONE + g));               // every issued MMA done before TMEM is freed
      const uint64_t t0 = globaltimer();
      while (!mbar_try(bar(B_DONE + g), 0) && globaltimer() - t0 < kWaitNs) {}
    }
  } else if (CONV && warp >= R::kConv) {
    // ------------------------------------------------------------ converters
    if constexpr (CONV) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      const int r = threadIdx.x - R::kConv * 32;   // this thread's row of every operand
      int tc_ = 0, qn = 0;
      bool ok = true;
      auto convert_q = [&]() -> bool {
        const int qi = qn % kNQ;
        if (!pipe_wait(bar(B_QFULL + qi), (qn / kNQ) & 1, abort_flag)) return false;
        rowe[qi * 128 + r] = (int8_t)rescale_row(smem + OFF_Q + qi * kOp, r);
        fence_proxy_async();
        mbar_arrive(bar(B_QCONV + qi));
        ++qn;
        return true;
      };
      for (long long kk = 0; ok; ++kk) {
        const long long u = unit_index(kk, blockIdx.x, gridDim.x);
        if (u >= U) break;
        const Unit x = unit_of(a, G, BS, u);
        if (x.ntok <= 0) continue;
        if (QC && !convert_q()) { ok = false; break; }
        for (int k = 0; k < x.ntiles && ok; ++k, ++tc_) {
          for (int kv = 0; kv < 2; ++kv) {
            if (!(kv ? V8 : K8)) continue;
            const int seq = 2 * tc_ + kv, s = seq % kNST;
            if (!pipe_wait(bar(B_FULL + s), (seq / kNST) & 1, abort_flag)) { ok = false; break; }
            const int t = x.tile0(k) + r;
            // a V row no row of the unit attends meets only zero weights: it must be finite
            const bool zero = kv && (!x.all.needs(t, 1) || ((slots[tc_ % kSlots].missing >> (r / BS)) & 1u));
            widen_row(smem + OFF_KV + s * kOp, r, zero);
            fence_proxy_async();
            mbar_arrive(bar(B_CONV + s));
          }
          if (QC && k == 0 && ok && x.two() && !convert_q()) ok = false;
        }
      }
      if (!ok) give_up();
    }
  } else {
    // ------------------------------------------------------------ softmax / epilogue
    if constexpr (CONV) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int r = threadIdx.x & 127;             // query row = TMEM lane
    const int qt = threadIdx.x >> 7;             // query tile of the unit
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t srow = tmem_s + lane_off + qt * kTile, orow_t = tmem_o + lane_off + qt * kD;
    const int tl = r / G, hg = r - (r / G) * G;  // token of the query tile, head of the group
    bool failed = false;
    int tc_ = 0, qn = 0;                         // key tiles and query tiles of the CTA so far
    int tiles = 0, units = 0, splits = 0;        // of this part; units in two parts
    float* xch = reinterpret_cast<float*>(smem + OFF_XCH);
    for (long long kk = 0; !failed; ++kk) {
      const long long u = unit_index(kk, blockIdx.x, gridDim.x);
      if (u >= U) break;
      const Unit x = unit_of(a, G, BS, u);
      if (x.ntok <= 0) continue;
      const Part part = part_of(a, x, qt);
      const int base = tc_, qs = part.split ? 0 : qt, q = qn + qs;     // its query tile: qs
      tc_ += x.ntiles;
      qn += x.two() ? 2 : 1;
      if (!part.on) continue;
      const int ntok = x.tokens(qs), pos0 = x.pos(qs);
      const bool row_ok = tl < ntok;
      const int pos = pos0 + tl;                 // this row attends keys t <= pos with
      const int wlo = a.window > 0 ? max(0, pos - a.window + 1) : 0;   // t >= wlo or t < sinks
      // the window of the query tile's last token starts at last_lo
      const int last_lo = a.window > 0 ? max(0, part.reach.t1 - a.window) : 0;
      const int32_t* table = a.block_tables + (size_t)x.b * a.max_blocks;
      float m = -FLT_MAX, l = 0.f;
      float back_m = 0.f;                        // BSC: the row sum's reference r as m - r
      float f0 = a.scale_log2;                   // score factor of the row
      if constexpr (QC) {
        // (The first scores say that the query tile was converted. To wait for that itself
        // would not do: a part that sat out units may be phases ahead of it.)
        if (!pipe_wait(bar(B_SFULL + 2 * qt), tiles & 1, abort_flag)) failed = true;
        f0 *= __uint_as_float((uint32_t)(127 - rowe[q % kNQ * 128 + r]) << 23);
        mbar_arrive(bar(B_QEMPTY + q % kNQ));
        if (!part.split) mbar_arrive(bar(B_QEMPTY + q % kNQ));
      }
      bool first = true;
      for (int k = part.first(qt); k <= part.last; k = part.next(k)) {
        const int ts = x.tile0(k);
        const int n = tiles++;
        // blocks that were not loaded: the producer's word (8-bit pools), else the table's
        const Slot& slot = slots[(base + k) % kSlots];
        uint32_t missing = 0;
        bool open = false;                       // every row sees every key of the tile
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (!pipe_wait(bar(B_SFULL + 2 * qt + h), n & 1, abort_flag)) failed = true;
          __syncwarp();
          tc_fence_after();
          uint32_t raw[64];
          float* s_ = reinterpret_cast<float*>(raw);
          tmem_ld32(srow + 64 * h, raw);
          tmem_ld32(srow + 64 * h + 32, raw + 32);
          if (h == 0) {
            if constexpr (CONV) {
              missing = *reinterpret_cast<const volatile uint32_t*>(&slot.missing) & ((1u << NB_T) - 1u);
            } else {
#pragma unroll
              for (int b = 0; b < NB_T; ++b) {
                bool gone = true;
                if (x.all.needs(ts + b * BS, BS)) {
                  const int ph = __ldg(table + ts / BS + b);
                  gone = ph < 0 || ph >= a.num_blocks;
                }
                missing |= gone ? 1u << b : 0u;
              }
            }
            open = missing == 0 && ts + kTile <= pos0 + 1 && (ts >= last_lo || ts + kTile <= a.sinks);
            if (!V8 && !open) {
              // a V row no row of the unit attends meets only zero weights: it must be finite
              // (both query tiles' threads write the zeros, ahead of their own product)
              if (!x.all.needs(ts + r, 1) || ((missing >> (r / BS)) & 1u)) {
                const int seq = 2 * (base + k) + 1, s = seq % kNST;
                if (!pipe_wait(bar(B_FULL + s), (seq / kNST) & 1, abort_flag)) failed = true;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  uint4* z = reinterpret_cast<uint4*>(smem + OFF_KV + s * kOp + hh * kHalf + r * 128);
#pragma unroll
                  for (int c = 0; c < 8; ++c) z[c] = make_uint4(0, 0, 0, 0);
                }
              }
              fence_proxy_async();
            }
            __syncwarp();
          }
          // Scores in the log2 domain, s' = s + log2(V scale) with block scales, are
          // raw f + e with f and e per 16 keys; where some are masked they are formed and
          // masked first, and f = 1, e = 0 from then on.
          float f[4], e[4], lv[4];               // lv: log2 of the V scale
          const float lvmin = BSC ? slot.lvmin : 0.f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int blk = (64 * h + 16 * c) / BS;
            f[c] = BSC ? f0 * slot.ks[blk] : f0;
            e[c] = lv[c] = BSC ? slot.lvs[blk] : 0.f;
          }
          tmem_wait_ld64(raw);
          if (!open) {
            // one bit per key of a 32-key chunk: up to the row's position, from its window
            // on or a first token, in a block that is there
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int t0 = ts + 64 * h + 32 * c;
              auto below = [&](int lim) -> uint32_t {          // keys of the chunk under lim
                const int n = lim - t0;
                return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : ((1u << n) - 1u);
              };
              uint32_t msk = below(pos + 1) & (~below(wlo) | below(a.sinks));
#pragma unroll
              for (int b = 0; b < 32 / BS; ++b)
                if ((missing >> ((64 * h + 32 * c) / BS + b)) & 1u) msk &= ~(kBlkBits << (b * BS));
              if (!row_ok) msk = 0;
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const int q = 2 * c + j / 16;
                s_[32 * c + j] = ((msk >> j) & 1u) ? fmaf(s_[32 * c + j], f[q], e[q]) : -CUDART_INF_F;
              }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              f[c] = 1.f;
              e[c] = 0.f;
            }
          }
          float tm = -CUDART_INF_F, tc[4];       // the half's maximum, and those of 16 keys
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // (f has one sign in all of a launch, but for the masked tiles' f = 1)
            float t0 = s_[16 * c], t1 = s_[16 * c + 1];
            if (f[0] >= 0.f) {
#pragma unroll
              for (int j = 16 * c + 2; j < 16 * c + 16; j += 2) {
                t0 = fmaxf(t0, s_[j]);
                t1 = fmaxf(t1, s_[j + 1]);
              }
              t0 = fmaxf(t0, t1);
            } else {
#pragma unroll
              for (int j = 16 * c + 2; j < 16 * c + 16; j += 2) {
                t0 = fminf(t0, s_[j]);
                t1 = fminf(t1, s_[j + 1]);
              }
              t0 = fminf(t0, t1);
            }
            tc[c] = fmaf(t0, f[c], e[c]);
            tm = fmaxf(tm, tc[c]);
          }
          // the references, in one vote: all of this is rare, but for masked halves
          bool move = tm - m > kMove;
          if constexpr (BSC) move = move || tm - lvmin > m - back_m + kSumMove || lvmin < back_m - 51.f;
          if (first || __any_sync(0xffffffffu, move)) {
            const float mn = tm - kLow, mo = m;
            if (first) {
              m = fmaxf(mn, -FLT_MAX);
            } else if (!BSC || __any_sync(0xffffffffu, tm - m > kMove)) {
              // rescale the row of O, once every product before this half's is in it: those of
              // the last tile's second half (the scores of this tile's come after it), or that
              // of this tile's first half
              const bool resc = tm - m > kMove;
              const float alpha = resc ? ex2(m - mn) : 1.f;
              if (resc) m = mn;
              if (!pipe_wait(bar(h == 0 ? B_SFULL + 2 * qt + 1 : B_OSTEP + qt), n & 1, abort_flag)) failed = true;
              __syncwarp();
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < kD; c += 16) {
                float o[16];
                tmem_ld16(orow_t + c, o);
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * alpha);
                tmem_put16(orow_t + c, w);
              }
              if (!BSC) l *= alpha;
            }
            first = false;
            if constexpr (BSC) {
              const float top = fmaxf(fmaxf(tc[0] - lv[0], tc[1] - lv[1]), fmaxf(tc[2] - lv[2], tc[3] - lv[3]));
              // r stays a whole number of powers of two away from m
              const float ro = mo - back_m, bo = back_m;
              if (top > ro + kSumMove) back_m = rintf(m - top);
              else if (m != mo) back_m = rintf(m - ro);
              l *= ex2(mo - m - (bo - back_m));
              const float rs = m - back_m;
              uint32_t far = 0;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                if (tc[c] < m - 96.f) {
                  if (tc[c] - lv[c] > rs - 45.f) far |= 1u << c;
                  lv[c] = CUDART_INF_F;          // counted below, or nothing to count
                }
              }
              // (a loop over the scores in tensor memory: unrolled over the registers it
              // slowed the prompt, which hardly comes here, by 9%)
              if (__any_sync(0xffffffffu, far != 0)) {
#pragma unroll 1
                for (int j = 64 * h; j < 64 * h + 64; ++j) {
                  const float x = tmem_ld1(srow + j);
                  const int t = ts + j;
                  const bool sees = row_ok && t <= pos && (t >= wlo || t < a.sinks) && !((missing >> (j / BS)) & 1u);
                  if (((far >> ((j >> 4) & 3)) & 1u) && sees) l += ex2(fmaf(x, f0 * slot.ks[j / BS], -rs));
                }
              }
            }
          }
          // weights and the row sum; a 32-key chunk's weights go over its scores, hi parts in
          // its first 16 columns, lo parts in the next 16
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float2 ff = make_float2(f[2 * c + q], f[2 * c + q]);
              const float em = e[2 * c + q] - m;
              const float2 ee = make_float2(em, em);
              float2 sum = make_float2(0.f, 0.f);          // of the 16 keys
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int i = 32 * c + 16 * q + 2 * j;
                float2 p = fma2(make_float2(s_[i], s_[i + 1]), ff, ee);
                p.x = ex2(p.x);
                p.y = ex2(p.y);
                sum = add2(sum, p);
                pack2<FO == 1, LO>(p.x, p.y, hi[8 * q + j], lo[8 * q + j]);
              }
              l = BSC ? fmaf(sum.x + sum.y, pow2_of(back_m - lv[2 * c + q]), l) : l + (sum.x + sum.y);
            }
            tmem_put16(srow + 64 * h + 32 * c, hi);
            if (LO) tmem_put16(srow + 64 * h + 32 * c + 16, lo);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar(B_PREADY + 2 * qt + h));
        }
      }
      // ---- epilogue: O / l of this row to the output
      if (!pipe_wait(bar(B_OFULL + qt), units & 1, abort_flag)) failed = true;
      ++units;
      tc_fence_after();
      if (part.split && qt == 1) {
        // the second part: its maximum and sum to the first, which reads its O
        xch[r] = m;
        xch[128 + r] = BSC ? pack_sum(l, -back_m) : l;
        tc_fence_before();
        mbar_arrive(bar(B_XCH));
        failed = __any_sync(0xffffffffu, failed);
        continue;
      }
      Norm<BSC> na, nb;                          // of this part's O and of the second's
      if (part.split) {
        if (!pipe_wait(bar(B_XCH), splits & 1, abort_flag)) failed = true;
        __syncwarp();
        tc_fence_after();
        const float m2 = xch[r];
        float l2 = xch[128 + r], r1 = BSC ? m - back_m : m, r2 = m2;
        if (BSC) l2 = unpack_sum(l2, r2);
        const float top = fmaxf(r1, r2);
        l = fmaf(l, ex2(r1 - top), l2 * ex2(r2 - top));
        na = norm_of<BSC>(m - top, l, a.v_scale);
        nb = norm_of<BSC>(m2 - top, l, a.v_scale);
        if (!BSC) {                              // (m and m2 are at most top there)
          na.f[0] *= ex2(m - top);
          nb.f[0] *= ex2(m2 - top);
        }
      } else {
        na = norm_of<BSC>(back_m, l, a.v_scale);
      }
      const size_t orow = ((size_t)(x.qrow0 + qs * x.tpt + tl) * a.Hq + (size_t)x.h * G + hg) * kD;
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        tmem_ld32(orow_t + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(na(__uint_as_float(o[e])));
        if (part.split) {
          uint32_t o2[32];
          tmem_ld32(orow_t + kD + c, o2);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(nb(__uint_as_float(o2[e])) + __uint_as_float(o[e]));
        }
        if (row_ok && !failed) {
          if (a.out_dtype == PA_F32) {
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow + c);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          } else {
            uint32_t pk[16], none;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float v0 = __uint_as_float(o[2 * e]), v1 = __uint_as_float(o[2 * e + 1]);
              pack2<FMT == 1, false>(v0, v1, pk[e], none);
            }
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + orow + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(bar(B_ODONE + qt));
      if (part.split) {
        mbar_arrive(bar(B_ODONE + 1));
        ++splits;
      }
      failed = __any_sync(0xffffffffu, failed);
    }
    if (failed) give_up();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kMma) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

namespace {

// Query [T][Hq][128] seen as [T][Hq][2 d-halves][64]: a box of 128 / G tokens x G heads
// x one d-half lands as 128 rows (token-major, then head) of 128 B, 128-byte swizzled.
// 16-bit pools [NB][bs][Hkv][128] seen as [NB][2][Hkv][bs][64]: a box of one block's rows
// of one head and d-half; pools of codes [NB][Hkv][bs][128]: a box of one block's rows of
// one head, a 128-byte line per row.
bool make_maps(const PrefillLaunch& p, int G, CUtensorMap* q, CUtensorMap* k, CUtensorMap* v) {
  auto enc = encode_fn();
  if (!enc || p.num_blocks <= 0) return false;
  const CUtensorMapDataType dt =
      p.dtype == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  auto make = [&](CUtensorMap* m, CUtensorMapDataType t, int rank, const void* base, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box) {
    return enc(m, t, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const cuuint64_t qdims[4] = {64, 2, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
  const cuuint64_t qstr[3] = {128, (cuuint64_t)kD * 2, (cuuint64_t)p.Hq * kD * 2};
  const cuuint32_t qbox[4] = {64, 1, (cuuint32_t)G, (cuuint32_t)(kM / G)};
  if (!make(q, dt, 4, p.q, qdims, qstr, qbox)) return false;
  const cuuint64_t hkv = (cuuint64_t)p.Hkv, bs = (cuuint64_t)p.bs, nb = (cuuint64_t)p.num_blocks;
  const cuuint64_t dims[5] = {64, bs, hkv, 2, nb};
  const cuuint64_t str[4] = {hkv * kD * 2, (cuuint64_t)kD * 2, 128, bs * hkv * kD * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)p.bs, 1, 1, 1};
  const cuuint64_t cdims[4] = {(cuuint64_t)kD, bs, hkv, nb};
  const cuuint64_t cstr[3] = {hkv * kD, (cuuint64_t)kD, bs * hkv * kD};
  const cuuint32_t cbox[4] = {(cuuint32_t)kD, (cuuint32_t)p.bs, 1, 1};
  for (int i = 0; i < 2; ++i) {
    const void* pool = i == 0 ? p.k_cache : p.v_cache;
    CUtensorMap* m = i == 0 ? k : v;
    const bool ok = (i == 0 ? p.k_dtype : p.v_dtype) == PA_FP8_E4M3
                        ? make(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pool, cdims, cstr, cbox)
                        : make(m, dt, 5, pool, dims, str, box);
    if (!ok) return false;
  }
  return true;
}

template <int FMT, int BS, bool K8, bool V8, bool BSC, bool LO>
int launch_t(const Args& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
             cudaStream_t stream) {
  auto kern = prefill_window_kernel<FMT, BS, K8, V8, BSC, LO>;
  // dynamic shared memory above 48 KB needs the attribute, on the current device
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return PA_ERR_CUDA;
  const long long U = (long long)a.B * a.chunks * a.Hkv;
  const long long grid = U < sm_count_cached() ? U : sm_count_cached();
  return launch_k(kern, dim3((unsigned)grid), dim3(Roles<K8 || V8>::kThreads), kSmem, stream, a, q, k, v) ==
                 cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int FMT, bool K8, bool V8, bool BSC, bool LO>
int launch_bs(const Args& a, int bs, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
              cudaStream_t stream) {
  return bs == 16 ? launch_t<FMT, 16, K8, V8, BSC, LO>(a, q, k, v, stream)
                  : launch_t<FMT, 32, K8, V8, BSC, LO>(a, q, k, v, stream);
}

template <bool K8, bool V8, bool BSC>
int launch_kv(const Args& a, int dtype, int bs, const CUtensorMap& q, const CUtensorMap& k,
              const CUtensorMap& v, cudaStream_t stream) {
  if (dtype != PA_BF16) return launch_bs<0, K8, V8, BSC, true>(a, bs, q, k, v, stream);
  // one part: see the head of this file
  if (V8 && a.out_dtype == PA_BF16) return launch_bs<1, K8, V8, BSC, !V8>(a, bs, q, k, v, stream);
  return launch_bs<1, K8, V8, BSC, true>(a, bs, q, k, v, stream);
}

}  // namespace

int launch_prefill_window(const PrefillLaunch& p, cudaStream_t stream) {
  const int G = p.Hq / p.Hkv;
  const bool k8 = p.k_dtype == PA_FP8_E4M3, v8 = p.v_dtype == PA_FP8_E4M3;
  CUtensorMap q, k, v;
  if (!make_maps(p, G, &q, &k, &v)) return PA_ERR_CUDA;
  Args a{};
  a.out = p.out;
  a.out_dtype = p.out_dtype;
  a.block_tables = p.block_tables;
  a.max_blocks = p.max_blocks;
  a.context_lens = p.context_lens;
  a.query_start = p.query_start;
  a.B = p.B; a.T = p.T; a.Hq = p.Hq; a.Hkv = p.Hkv; a.num_blocks = p.num_blocks;
  const int tpu = 2 * kM / G;
  a.chunks = p.max_query_len / tpu + (p.max_query_len % tpu != 0);
  a.scale_log2 = p.scale_log2;
  a.v_scale = v8 ? p.v_scale : 1.f;
  a.max_context_len = p.max_context_len;
  a.err_flag = p.err_flag;
  a.window = p.window; a.sinks = p.sinks;
  a.k_scales = p.k_scales; a.v_scales = p.v_scales;
  a.wait_ns = (uint32_t)tc_wait_ns();           // at most 10^9
  a.test_withhold = tc_test_withhold_q();
  if (p.k_scales) return launch_kv<true, true, true>(a, p.dtype, p.bs, q, k, v, stream);
  if (k8 && v8) return launch_kv<true, true, false>(a, p.dtype, p.bs, q, k, v, stream);
  if (k8) return launch_kv<true, false, false>(a, p.dtype, p.bs, q, k, v, stream);
  if (v8) return launch_kv<false, true, false>(a, p.dtype, p.bs, q, k, v, stream);
  return launch_kv<false, false, false>(a, p.dtype, p.bs, q, k, v, stream);
}

}  // namespace pa
