// prefill_tc.cu -- paged (chunked) prefill attention on the 5th-generation
// tensor cores with the query rows on the MMA's M.
//
// A chunk of a sequence's new query tokens attends, causally, to the
// sequence's cached tokens through its block table ("推理引擎内部机制——
// PagedAttention、连续批处理、分块预填充", chunked prefill: a long prompt is cut
// into chunks that run between decode steps). New token i of a chunk of n at
// the end of a context of ctx tokens sits at position ctx - n + i and attends
// positions 0 .. ctx - n + i.
//
// Work unit = (sequence b, chunk of TPU = 128 / G new tokens, KV head h).
// Its 128 query rows are (token t, query head g of the group of h), row
// r = t * G + g: one TMA box of the query [T][Hq][128] brings them in that
// order. Tile = 128 keys of head h: one TMA box per physical block and 64-wide
// d-half, 128-byte swizzled (block-sized boxes; a head's rows of a block are
// contiguous, the heads of a block are not). Per tile:
//   S[128 rows x 128 keys]  = Q . K_tile^T          (tensor memory, fp32)
//   O[128 rows x 128 d]    += P_hi . V_tile + P_lo . V_tile
// where the weights P (in tensor memory, written over S) enter as two 16-bit
// parts, p = hi + lo, hi = RN(p), lo = RN(p - hi) (~16 significant bits, as
// in the decode kernels), and the A operand of the output products is read
// from tensor memory: each 32-key chunk of S becomes 16 columns of hi parts
// followed by 16 columns of lo parts (two keys per 32-bit column).
//
// Two softmax groups share a unit's 128 query rows: thread (group hf, row r)
// owns row r's keys [64 hf, 64 hf + 64) of every tile and O's columns [64 hf,
// 64 hf + 64), so a row needs only its two threads to agree: they exchange the
// tile's row maximum (and, at the unit's end, their parts of the row sum)
// through shared memory. A thread reads its scores twice, 32 columns at a
// time: once for the maximum, once for the weights, which it writes over the
// chunk it has just read. (Holding all of a row's scores in registers made the
// loop body four times longer; a per-key mask branch inside the loops cost
// more than the rest of the tile's softmax: the mask is one bit per key of a
// 32-key chunk, and whole chunks take a loop without it.) The reference
// maximum of a row is its first tile's maximum
// and moves only when a later tile exceeds it by 2^64 (then the row's O is
// rescaled in tensor memory, each half by its thread); references are
// floored at -FLT_MAX so masked scores (-inf) give weight 0 without a guard.
// Keys past a row's position are masked; the V rows of keys that no row of
// the unit attends (past its last position, or in a block with a bad id) are
// zeroed in shared memory before the output product, so they add exact zeros.
//
// CTA = 10 warps, persistent over rounds of units taken in alternating
// directions (fa_unit_of_cta; the chunks late in their sequences, which
// attend the most keys, come first):
//   warps 0-7  softmax and epilogue, two groups (thread = query row = TMEM
//              lane; warps w and w + 4 reach the same lanes);
//   warp 8     TMA producer: the unit's query (double-buffered by unit), the
//              K and V tiles through a ring of 32 KB stages (its lanes issue
//              the copies of a tile's blocks together);
//   warp 9     MMA issuer and owner of the tensor memory: S(t), then the
//              output product of tile t - 1 (S is double-buffered by tile, O
//              by unit, so a unit's epilogue overlaps the next unit's tiles).
// Every pipeline wait is bounded (1 s); one that gives up sets PA_DEV_TIMEOUT,
// raises the CTA's abort flag, and every role drains its asynchronous work,
// frees tensor memory and returns.
#include "prefill_fa.cuh"

namespace pa {

namespace {

template <int FMT, int BS, bool K8, bool V8>
int launch_fa_g(const FaArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                cudaStream_t stream) {
  switch (a.Hq / a.Hkv) {
    case 1: return launch_fa_t<FMT, BS, 1, K8, V8>(a, q, k, v, stream);
    case 2: return launch_fa_t<FMT, BS, 2, K8, V8>(a, q, k, v, stream);
    case 4: return launch_fa_t<FMT, BS, 4, K8, V8>(a, q, k, v, stream);
    case 8: return launch_fa_t<FMT, BS, 8, K8, V8>(a, q, k, v, stream);
    case 16: return launch_fa_t<FMT, BS, 16, K8, V8>(a, q, k, v, stream);
  }
  return PA_ERR_UNSUPPORTED;
}

template <bool K8, bool V8>
int launch_fa_kv(const FaArgs& a, int dtype, int bs, const CUtensorMap& q, const CUtensorMap& k,
                 const CUtensorMap& v, cudaStream_t stream) {
  if (dtype == PA_BF16)
    return bs == 16 ? launch_fa_g<1, 16, K8, V8>(a, q, k, v, stream)
                    : launch_fa_g<1, 32, K8, V8>(a, q, k, v, stream);
  return bs == 16 ? launch_fa_g<0, 16, K8, V8>(a, q, k, v, stream)
                  : launch_fa_g<0, 32, K8, V8>(a, q, k, v, stream);
}

}  // namespace

bool prefill_fa_supported(int dtype, int Hq, int Hkv, int D, int bs) {
  if (dtype != PA_F16 && dtype != PA_BF16) return false;
  if (D != kD || (bs != 16 && bs != 32) || Hkv <= 0 || Hq % Hkv) return false;
  const int G = Hq / Hkv;
  return G == 1 || G == 2 || G == 4 || G == 8 || G == 16;
}

int launch_prefill_fa(const PrefillLaunch& p, cudaStream_t stream) {
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
  a.chunks = (p.max_query_len + kM / G - 1) / (kM / G);
  a.scale_log2 = p.scale_log2;
  a.v_scale = v8 ? p.v_scale : 1.f;
  a.max_context_len = p.max_context_len;
  a.err_flag = p.err_flag;
  if (k8 && v8) return launch_fa_kv<true, true>(a, p.dtype, p.bs, q, k, v, stream);
  if (k8) return launch_fa_kv<true, false>(a, p.dtype, p.bs, q, k, v, stream);
  if (v8) return launch_fa_kv<false, true>(a, p.dtype, p.bs, q, k, v, stream);
  return launch_fa_kv<false, false>(a, p.dtype, p.bs, q, k, v, stream);
}

}  // namespace pa
