// decode_window_f32.cu -- windowed decode over fp32 pools, on the CUDA cores (the
// types and shapes are those of decode_window.cu, which holds the 16- and 8-bit
// pools and says how the work is split).
//
// CTA = four warps; a unit is (sequence, KV head, chunk of 4 query heads). The
// warps take a unit's 16-token tiles in turn, each through its own ring of tiles
// in shared memory filled with 16-byte asynchronous copies, and join their sums
// through shared memory at the unit's end. fp32 pools are for exactness, not for speed: a
// tiny batch (four sequences of up to 33 tokens) takes 9.6 us, the two launches and one
// unit's chain of copies, products and sums.
#include "window_common.cuh"

namespace pa {

namespace {

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

// A tile's shared-memory layout: 16 rows, 16-byte chunks swizzled within a row so
// that eight lanes reading one chunk of eight rows touch every bank once.
template <int D> struct Rows {
  static constexpr int ROWB = D * 4, CPR = D / 4, BYTES = kTok * ROWB;
  static __device__ __forceinline__ uint32_t at(int row, int c) {
    return (uint32_t)(row * ROWB + ((c ^ (row & 7)) << 4));
  }
};

// fp32 pools: products on the CUDA cores, 4 query heads. Scores: lane = (token,
// half of the dims); output: a lane owns D / 32 dims of every head.
template <int D>
struct CoreF32 {
  static constexpr int HEADS = 4, WARPS = 4;
  using R = Rows<D>;
  static constexpr int STAGE = 2 * R::BYTES;
  static constexpr int NST = D == 64 ? 4 : 2;   // 16 KB per tile at D = 128, 4 warps: 128 KB
  static constexpr int PER = D / 32;
  float m[HEADS], l[HEADS], o[HEADS][PER];
  const float* q;                               // of the unit; heads past gc read head 0
  int gc;
  float scale;

  __device__ __forceinline__ void start(const WinArgs& a, size_t q0, int gc_, int) {
    q = static_cast<const float*>(a.q) + q0;
    gc = gc_;
    scale = a.scale_log2;
#pragma unroll
    for (int g = 0; g < HEADS; ++g) {
      m[g] = -FLT_MAX;
      l[g] = 0.f;
#pragma unroll
      for (int e = 0; e < PER; ++e) o[g][e] = 0.f;
    }
  }
  __device__ __forceinline__ void tile(uint32_t kst, const Span& sp, int t0, int lane) {
    const uint32_t vst = kst + R::BYTES;
    const int row = lane & 15, hf = lane >> 4;
    float s[HEADS];
#pragma unroll
    for (int g = 0; g < HEADS; ++g) s[g] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const int cc = hf * (D / 8) + c;
      float kv[4];
      widen16<float>(lds16(kst + R::at(row, cc)), kv);
#pragma unroll
      for (int g = 0; g < HEADS; ++g) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(q + (g < gc ? g : 0) * D + 4 * cc));
        s[g] = fmaf(x.x, kv[0], fmaf(x.y, kv[1], fmaf(x.z, kv[2], fmaf(x.w, kv[3], s[g]))));
      }
    }
    const bool sees = sp.sees(t0 + row);
    float p[HEADS];
#pragma unroll
    for (int g = 0; g < HEADS; ++g) {
      s[g] = (s[g] + __shfl_xor_sync(0xffffffffu, s[g], 16)) * scale;
      if (!sees) s[g] = -CUDART_INF_F;
      float mx = s[g];
#pragma unroll
      for (int x = 8; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[g], mx);
      const float alpha = exp2f(m[g] - mn);
      m[g] = mn;
      p[g] = exp2f(s[g] - mn);
      l[g] = l[g] * alpha + p[g];               // lanes 0-15 and 16-31 hold the same tokens
#pragma unroll
      for (int e = 0; e < PER; ++e) o[g][e] *= alpha;
    }
#pragma unroll 4
    for (int r = 0; r < kTok; ++r) {
      float v[4];
      const int d0 = lane * PER;
      const uint32_t at = vst + R::at(r, d0 / 4) + (d0 % 4) * 4;
      if constexpr (PER == 4) {
        widen16<float>(lds16(at), v);
      } else {
        const uint2 w = lds8(at);
        v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y);
      }
#pragma unroll
      for (int g = 0; g < HEADS; ++g) {
        const float pr = __shfl_sync(0xffffffffu, p[g], r);
#pragma unroll
        for (int e = 0; e < PER; ++e) o[g][e] = fmaf(pr, v[e], o[g][e]);
      }
    }
  }
  // this warp's sums: acc[head][d], (m, l) of each head
  __device__ __forceinline__ void leave(float* acc, float* sm, float* sl, int lane) {
#pragma unroll
    for (int g = 0; g < HEADS; ++g) {
#pragma unroll
      for (int x = 8; x >= 1; x >>= 1) l[g] += __shfl_xor_sync(0xffffffffu, l[g], x);
      if (lane == 0) { sm[g] = m[g]; sl[g] = l[g]; }
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[g * D + lane * PER + e] = o[g][e];
    }
  }
};

}  // namespace

template <int D>
__global__ void __launch_bounds__(CoreF32<D>::WARPS * 32, 1)
decode_window_f32_kernel(const WinArgs a) {
  using C = CoreF32<D>;
  using R = Rows<D>;
  constexpr int kWarps = C::WARPS, NST = C::NST, HEADS = C::HEADS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sm_acc[kWarps][HEADS * D];
  __shared__ float sm_m[kWarps][HEADS], sm_l[kWarps][HEADS];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.Hq / a.Hkv;
  const int chunks = (G + HEADS - 1) / HEADS, ny = a.Hkv * chunks;
  const int cta = blockIdx.x;
  Share w = find_share<kWarps * 32>(a, ny, 1, cta, gridDim.x);
  if (cta >= w.shares) return;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * (NST * C::STAGE);
  while (w.p0 < a.B * ny && w.base0 < w.hi) {
    const int p0 = w.p0;
    const Batch u = next_batch(a, w, ny, 1, cta, lane);
    for (int i = 0; i < u.count; ++i) {
      const int b = __shfl_sync(0xffffffffu, u.b, i), y = __shfl_sync(0xffffffffu, u.y, i);
      const int s0 = __shfl_sync(0xffffffffu, u.s0, i), s1 = __shfl_sync(0xffffffffu, u.s1, i);
      const int ctx = __shfl_sync(0xffffffffu, u.ctx, i), n = __shfl_sync(0xffffffffu, u.n, i);
      const int first = __shfl_sync(0xffffffffu, u.first, i), last = __shfl_sync(0xffffffffu, u.last, i);
      const bool starts = __shfl_sync(0xffffffffu, (int)u.starts, i);
      const int h = y / chunks, chunk = y - h * chunks;
      const int gc = min(HEADS, G - chunk * HEADS);
      const size_t row0 = (size_t)b * a.Hq + h * G + chunk * HEADS;
      if (starts && threadIdx.x == 0) a.cuts[p0 + i] = make_int2(first, last);
      if (n == 0) {
        if (!starts) continue;
        // an empty sequence's (or one of a bad length) rows are zeros
        if (y == 0 && threadIdx.x == 0 && ctx != 0) flag_error(a.err_flag, PA_DEV_BAD_CTX);
        for (int x = threadIdx.x; x < gc * D; x += kWarps * 32) store_out(a.out, row0 * D + x, 0.f, a.out_dtype);
        continue;
      }
      if (s0 >= s1) continue;
      const Span sp = span_of(a, ctx);
      const int32_t* table = a.block_tables + (size_t)b * a.max_blocks;
      const int mine = (s1 - s0 - warp + kWarps - 1) / kWarps;
      uint32_t bad = 0;                         // ring stages whose block is bad
      auto issue = [&](int k) {
        if (k < mine) {
          const int t0 = sp.tile(s0 + warp + kWarps * k) * kTok;
          const int st = k % NST;
          const int id = __ldg(table + t0 / a.bs);
          const bool ok = id >= 0 && id < a.num_blocks;
          if (!ok && lane == 0) flag_error(a.err_flag, PA_DEV_BAD_BLOCK_ID);
          bad = ok ? bad & ~(1u << st) : bad | (1u << st);
          const size_t r0 = ((size_t)(ok ? id : 0) * a.bs + (t0 & (a.bs - 1))) * a.Hkv + h;
          const char* kp = static_cast<const char*>(a.k_cache) + (ok ? r0 * R::ROWB : 0);
          const char* vp = static_cast<const char*>(a.v_cache) + (ok ? r0 * R::ROWB : 0);
          for (int x = lane; x < kTok * R::CPR; x += 32) {
            const int row = x / R::CPR, c = x % R::CPR;
            const bool take = ok && sp.sees(t0 + row);       // zeros elsewhere
            const size_t off = take ? (size_t)row * a.Hkv * R::ROWB + c * 16 : 0;
            copy16(ring + st * C::STAGE + R::at(row, c), kp + off, take);
            copy16(ring + st * C::STAGE + R::BYTES + R::at(row, c), vp + off, take);
          }
        }
        copy_commit();
      };
      C core;
      core.start(a, row0 * D, gc, lane);
      __syncwarp();
      for (int k = 0; k < NST - 1; ++k) issue(k);
      for (int k = 0; k < mine; ++k) {
        __syncwarp();                           // every lane has read the stage's last tile
        issue(k + NST - 1);
        copy_wait<NST - 1>();
        __syncwarp();
        if (!((bad >> (k % NST)) & 1u))
          core.tile(ring + (k % NST) * C::STAGE, sp, sp.tile(s0 + warp + kWarps * k) * kTok, lane);
      }
      copy_wait<0>();
      __syncthreads();                          // the last unit's sums have been read
      core.leave(sm_acc[warp], sm_m[warp], sm_l[warp], lane);
      __syncthreads();
      const size_t slot = 2 * (size_t)cta + (cta == first ? 1 : 0);
      for (int x = threadIdx.x; x < HEADS * D; x += kWarps * 32) {
        const int g = x / D;
        float M = -FLT_MAX, L = 0.f, O = 0.f;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) M = fmaxf(M, sm_m[v][g]);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
          const float c = exp2f(sm_m[v][g] - M);
          L = fmaf(sm_l[v][g], c, L);
          O = fmaf(sm_acc[v][x], c, O);
        }
        if (first == last) {
          if (g < gc) store_out(a.out, row0 * D + x, L == 0.f ? 0.f : O / L, a.out_dtype);
        } else {
          a.ws_acc[slot * (HEADS * D) + x] = L == 0.f ? 0.f : O / L;   // (pieces are normalised)
          if (x % D == 0) {
            a.ws_m[slot * HEADS + g] = M;
            a.ws_l[slot * HEADS + g] = L;
          }
        }
      }
    }
  }
}

int launch_decode_window_f32(const WinArgs& a, cudaStream_t stream) {
  auto go = [&](auto kern, int smem) {
    // dynamic shared memory above 48 KB needs the attribute, on the current device
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return (int)PA_ERR_CUDA;
    return launch_k(kern, dim3((unsigned)a.grid), dim3(128), smem, stream, a) == cudaSuccess
               ? (int)PA_OK : (int)PA_ERR_CUDA;
  };
  if (a.D == 64) return go(decode_window_f32_kernel<64>, 4 * CoreF32<64>::NST * CoreF32<64>::STAGE);
  return go(decode_window_f32_kernel<128>, 4 * CoreF32<128>::NST * CoreF32<128>::STAGE);
}

}  // namespace pa
