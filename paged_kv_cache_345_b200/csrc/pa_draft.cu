// The cache side of a decode step with drafted tokens: rows with norms and
// rotation written into the cache, verification of the drafted tokens, and the
// move of the accepted rows into place. (The attention between them is
// pa_tree.cu.) "What is paged attention in vLLM, and why does it matter?", Step
// 4: each decoding step writes the new tokens' keys and values into the last
// block; here a step writes several per sequence and keeps some of them.
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <utility>

#include <cooperative_groups.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"

namespace pa {

namespace {

// ------------------------------------------------- rows: norm, rotation, append

struct RowsParams {
  void* q_out;
  const void* q;
  const void* k;
  const void* v;
  int64_t q_out_stride, q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* positions;
  const int64_t* slots;
  const float* cos_sin;  // [max_position][rotary_dim]: cosines, then sines
  const void* q_weight;  // [D] or null: no norm
  const void* k_weight;
  void* k_cache;
  void* v_cache;
  const float* k_scale;  // E4M3 caches
  const float* v_scale;
  unsigned* err;
  int64_t num_slots;
  int num_tokens, num_heads, num_kv_heads, max_position, rotary_dim;
  unsigned units_per_token;
  int q_units, kv_units;  // of a token: of its q heads, of its k heads (and of its v heads)
  float eps;
};

// Rows of T; a lane holds 16 bytes of a head's row, kLanes lanes a row, so a
// warp instruction moves kRows rows. A unit of work is U such instructions of q
// heads, of k heads or of v heads of one token; one warp per unit, all its loads
// first (before the position is known). The bytes bound it (every row is read
// and written once), if the instructions stay few: with the weights folded into
// the cosines and sines once per unit,
//   out[e] = r (x[e] cw[e] + z[e] sw[e]),  r = 1 / sqrt(mean(x^2) + eps),
// z[e] the other element of the pair, all two elements to an instruction. A lane
// holds both elements of its pairs: its 16 bytes are 8 at the pairs' first
// elements and 8 at their second ones (interleaved pairs: 16 in a row), so that
// nothing is exchanged and a cosine or sine is loaded once (with 16 bytes in a row and the
// partner's shuffled 10,578 prompt rows took 52.5 us, issuing 58 % of the time; now
// 49.4, 5.4 TB/s). Four instructions a unit: with 2, 3 or 8 the prompts took 12 to 20 %
// longer, and warps that load the next unit under the current one 58 us (100 registers).
template <typename T, int D>
struct RowsConfig {
  static constexpr int kEPL = ElemTraits<T>::kPer16B;
  static constexpr int kLanes = D / kEPL;
  static constexpr int kRows = 32 / kLanes;
  static constexpr int kU = 4;
  static constexpr int kPer = kRows * kU;  // heads of a unit
  static constexpr int kWarps = 4;         // per CTA
};

// N consecutive floats (N = 2, 4, 8; N * 4 or 16 bytes aligned).
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&x)[N]) {
  if constexpr (N == 2) {
    const float2 f = __ldg(reinterpret_cast<const float2*>(p));
    x[0] = f.x;
    x[1] = f.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
      x[4 * i] = f.x;
      x[4 * i + 1] = f.y;
      x[4 * i + 2] = f.z;
      x[4 * i + 3] = f.w;
    }
  }
}

// 16 bytes of a row as pairs of floats.
template <typename T, int N>
__device__ __forceinline__ void unpack_pairs(const uint4& v, uint64_t (&x)[N]) {
  float f[2 * N];
  ElemTraits<T>::unpack(v, f);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = pair_of(f[2 * i], f[2 * i + 1]);
}

template <typename T, int D, bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(RowsConfig<T, D>::kWarps * 32)
    qk_norm_rope_append_kernel(const RowsParams p) {
  using Cfg = RowsConfig<T, D>;
  constexpr int EPL = Cfg::kEPL, LPR = Cfg::kLanes, U = Cfg::kU, NP = EPL / 2;
  pdl_wait();
  pdl_launch_dependents();
  const unsigned unit = blockIdx.x * Cfg::kWarps + (threadIdx.x >> 5);
  const unsigned tok = unit / p.units_per_token;
  if (tok >= static_cast<unsigned>(p.num_tokens)) return;
  const int part = static_cast<int>(unit - tok * p.units_per_token);
  constexpr int CH = EPL / 2;  // elements of 8 bytes
  const int lane = threadIdx.x & 31, li = lane % LPR;
  const int pos = __ldg(p.positions + tok);
  const int64_t slot = __ldg(p.slots + tok);
  // kind 0 q, 1 k, 2 v (the same for the warp), and its heads
  const int kind = part < p.q_units ? 0 : part < p.q_units + p.kv_units ? 1 : 2;
  const int heads = kind == 0 ? p.num_heads : p.num_kv_heads;
  const int head0 = (part - (kind == 0 ? 0 : kind == 1 ? p.q_units : p.q_units + p.kv_units)) * Cfg::kPer +
                    lane / LPR;
  const T* src = static_cast<const T*>(kind == 0 ? p.q : kind == 1 ? p.k : p.v) +
                 tok * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride) + head0 * D;
  // this lane's elements: ea .. ea + CH - 1 and eb .. eb + CH - 1
  const int half = p.rotary_dim >> 1;
  const bool rotated = INTERLEAVED ? li * EPL < p.rotary_dim : li * CH < half;
  const int ea = INTERLEAVED ? li * EPL : rotated ? li * CH : p.rotary_dim + (li * CH - half) * 2;
  const int eb = INTERLEAVED || !rotated ? ea + CH : ea + half;
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    raw[u] = make_uint4(0, 0, 0, 0);
    // (not the read-only path: q_out may be q)
    if (head0 + u * Cfg::kRows < heads) {
      const T* row = src + u * Cfg::kRows * D;
      if constexpr (INTERLEAVED) {
        raw[u] = __ldcs(reinterpret_cast<const uint4*>(row + ea));
      } else {
        const uint2 a = __ldcs(reinterpret_cast<const uint2*>(row + ea));
        const uint2 b = __ldcs(reinterpret_cast<const uint2*>(row + eb));
        raw[u] = make_uint4(a.x, a.y, b.x, b.y);
      }
    }
  }
  if (pos < 0) return;  // padding
  if (pos >= p.max_position) {
    if (lane == 0 && part == 0) atomicOr(p.err, PA_DEVERR_POSITION);
    return;
  }
  if (slot >= p.num_slots && lane == 0 && part == 0) atomicOr(p.err, PA_DEVERR_SLOT);
  if (kind != 0 && (slot < 0 || slot >= p.num_slots)) return;
  uint8_t* cache = static_cast<uint8_t*>(kind == 1 ? p.k_cache : p.v_cache);
  const int64_t cache_row = slot * p.num_kv_heads + head0;
  T* dst = kind == 0 ? static_cast<T*>(p.q_out) + tok * p.q_out_stride + head0 * D
                     : reinterpret_cast<T*>(cache) + cache_row * D;

  // pairs of elements (2 i, 2 i + 1) of the lane's; the other element of a pair is the
  // neighbour (interleaved), or in the lane's other 8 bytes
  uint64_t cw[NP], sw[NP];
  const T* weight = static_cast<const T*>(kind == 0 ? p.q_weight : p.k_weight);
  if (kind < 2) {
    float c[EPL], n[EPL];
    if (rotated) {
      float cs[CH], sn[CH];
      const float* t = p.cos_sin + static_cast<int64_t>(pos) * p.rotary_dim + (INTERLEAVED ? ea / 2 : ea);
      load_floats<CH>(t, cs);
      load_floats<CH>(t + half, sn);
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        const int angle = INTERLEAVED ? e / 2 : e % CH;
        const bool first = INTERLEAVED ? e % 2 == 0 : e < CH;
        c[e] = cs[angle];
        n[e] = first ? -sn[angle] : sn[angle];
      }
    } else {
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        c[e] = 1.0f;
        n[e] = 0.0f;
      }
    }
    if (weight != nullptr) {
      const uint2 wa = __ldg(reinterpret_cast<const uint2*>(weight + ea));
      const uint2 wb = __ldg(reinterpret_cast<const uint2*>(weight + eb));
      float w[EPL];
      ElemTraits<T>::unpack(make_uint4(wa.x, wa.y, wb.x, wb.y), w);
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        c[e] *= w[e];
        n[e] *= w[INTERLEAVED ? e ^ 1 : (e + CH) % EPL];
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      cw[i] = pair_of(c[2 * i], c[2 * i + 1]);
      sw[i] = pair_of(n[2 * i], n[2 * i + 1]);
    }
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u > 0 && head0 - lane / LPR + u * Cfg::kRows >= heads) break;  // (the same for the warp)
    const bool on = head0 + u * Cfg::kRows < heads;
    uint64_t y[NP];
    if (kind < 2) {
      uint64_t x[NP];
      unpack_pairs<T>(raw[u], x);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint64_t z = x[(i + NP / 2) % NP];
        if constexpr (INTERLEAVED) {
          float lo, hi;
          floats_of(x[i], lo, hi);
          z = pair_of(hi, lo);
        }
        y[i] = mul2(x[i], cw[i]);
        // (elsewhere an infinite x is not a pair of itself)
        if (rotated) y[i] = fma2(z, sw[i], y[i]);
      }
      if (weight != nullptr) {
        uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
        for (int i = 1; i < NP; ++i) sq = fma2(x[i], x[i], sq);
        float s0, s1;
        floats_of(sq, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
        const float r = rsqrtf(ss * (1.0f / D) + p.eps);
        const uint64_t rr = pair_of(r, r);
#pragma unroll
        for (int i = 0; i < NP; ++i) y[i] = mul2(y[i], rr);
      }
    } else {
      unpack_pairs<T>(raw[u], y);
    }
    if (!on) continue;
    float f[EPL];
#pragma unroll
    for (int i = 0; i < NP; ++i) floats_of(y[i], f[2 * i], f[2 * i + 1]);
    if (FP8 && kind != 0) {
      // one rounding: the float32 row divided by its head's scale, to E4M3
      if constexpr (EPL == 8) {
        const float sc = __ldg((kind == 1 ? p.k_scale : p.v_scale) + head0 + u * Cfg::kRows);
        uint32_t r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          r[i] = static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(f[4 * i], sc), __fdiv_rn(f[4 * i + 1], sc))) |
                 (static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(f[4 * i + 2], sc), __fdiv_rn(f[4 * i + 3], sc))) << 16);
        uint8_t* row = cache + (cache_row + u * Cfg::kRows) * D;
        if constexpr (INTERLEAVED) {
          *reinterpret_cast<uint2*>(row + ea) = make_uint2(r[0], r[1]);
        } else {
          *reinterpret_cast<uint32_t*>(row + ea) = r[0];
          *reinterpret_cast<uint32_t*>(row + eb) = r[1];
        }
      }
      continue;
    }
    uint4 o = raw[u];  // v: its own bits
    if (kind != 2) {
      if constexpr (EPL == 8)
        o = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                       pack_bf16x2(f[6], f[7]));
      else
        o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    T* row = dst + u * Cfg::kRows * D;
    if constexpr (INTERLEAVED) {
      *reinterpret_cast<uint4*>(row + ea) = o;
    } else {
      *reinterpret_cast<uint2*>(row + ea) = make_uint2(o.x, o.y);
      *reinterpret_cast<uint2*>(row + eb) = make_uint2(o.z, o.w);
    }
  }
}

template <typename T, int D, bool FP8>
cudaError_t launch_rows_t(RowsParams p, bool interleaved, cudaStream_t stream) {
  using Cfg = RowsConfig<T, D>;
  p.q_units = (p.num_heads + Cfg::kPer - 1) / Cfg::kPer;
  p.kv_units = (p.num_kv_heads + Cfg::kPer - 1) / Cfg::kPer;
  p.units_per_token = static_cast<unsigned>(p.q_units + 2 * p.kv_units);
  const int64_t units = static_cast<int64_t>(p.num_tokens) * p.units_per_token;
  if (units > 0x7fffffff) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned>((units + Cfg::kWarps - 1) / Cfg::kWarps));
  auto kernel = interleaved ? qk_norm_rope_append_kernel<T, D, FP8, true>
                            : qk_norm_rope_append_kernel<T, D, FP8, false>;
  return launch_pdl(kernel, grid, dim3(Cfg::kWarps * 32), 0, stream, p);
}

}  // namespace

cudaError_t launch_qk_norm_rope_append(const QkRowsShape& sh, void* q_out, const void* q,
                                       const void* k, const void* v, const int32_t* positions,
                                       const int64_t* slot_mapping, const float* cos_sin,
                                       const void* q_weight, const void* k_weight, void* k_cache,
                                       void* v_cache, const float* k_scale, const float* v_scale,
                                       cudaStream_t stream) {
  RowsParams p{};
  p.q_out = q_out;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out_stride = sh.q_out_stride;
  p.q_stride = sh.q_stride;
  p.k_stride = sh.k_stride;
  p.v_stride = sh.v_stride;
  p.positions = positions;
  p.slots = slot_mapping;
  p.cos_sin = cos_sin;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_slots = sh.num_slots;
  p.num_tokens = sh.num_tokens;
  p.num_heads = sh.num_heads;
  p.num_kv_heads = sh.num_kv_heads;
  p.max_position = sh.max_position;
  p.rotary_dim = sh.rotary_dim;
  p.eps = sh.eps;
  cudaError_t e = device_error_word(&p.err);
  if (e != cudaSuccess) return e;
  const bool il = sh.interleaved;
  const bool d64 = sh.head_dim == 64;
  if (sh.dtype == PA_F32)
    return d64 ? launch_rows_t<float, 64, false>(p, il, stream) : launch_rows_t<float, 128, false>(p, il, stream);
  if (sh.dtype == PA_BF16)
    return d64 ? launch_rows_t<__nv_bfloat16, 64, false>(p, il, stream)
               : launch_rows_t<__nv_bfloat16, 128, false>(p, il, stream);
  return d64 ? launch_rows_t<__nv_bfloat16, 64, true>(p, il, stream)
             : launch_rows_t<__nv_bfloat16, 128, true>(p, il, stream);
}

// ------------------------------------------------------------- accepted rows

namespace {

// Each warp owns 512 bytes (a lane 16) of a sequence's K or V rows and takes
// the path 32 entries at a time: lane l finds the slots of entry l, then the
// rows move 8 at a time, loads before stores. Sources never lie before their
// targets (the path is increasing), so a batch's stores reach no row that a
// later batch reads, and no two warps share bytes. Latency-bound: a few rows a
// sequence, four loads that follow each other (lengths, path, table, row): the 16 rows of
// 8 sequences appended and moved, two launches, 4.3 us.
__global__ void __launch_bounds__(128)
    kv_accept_kernel(uint4* __restrict__ k_cache, uint4* __restrict__ v_cache,
                     const int32_t* __restrict__ block_tables,
                     const int32_t* __restrict__ context_lens,
                     const int32_t* __restrict__ query_start, const int32_t* __restrict__ path,
                     const int32_t* __restrict__ path_len, int max_path, int num_blocks, int lg,
                     int max_blocks_per_seq, int vec_per_row, unsigned* err) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.x;
  const int w = blockIdx.y * 4 + (threadIdx.x >> 5);  // 512-byte column of the K row, then the V row
  const int wpr = (vec_per_row + 31) / 32;
  if (w >= 2 * wpr) return;
  uint4* cache = w < wpr ? k_cache : v_cache;
  const int col = (w < wpr ? w : w - wpr) * 32 + lane;
  const bool live = col < vec_per_row;
  const bool teller = w == 0 && lane == 0;

  const int L = __ldg(context_lens + s), q0 = __ldg(query_start + s), q1 = __ldg(query_start + s + 1);
  const int len = __ldg(path_len + s);
  const int n = q1 - q0;
  if (q0 < 0 || n < 0 || L < n || L > (static_cast<int64_t>(max_blocks_per_seq) << lg)) {
    if (teller) atomicOr(err, PA_DEVERR_CONTEXT);
    return;
  }
  if (len < 0 || len > max_path || len > n) {
    if (teller) atomicOr(err, PA_DEVERR_DRAFT);
    return;
  }
  const int base = L - n;
  const int32_t* trow = block_tables + static_cast<int64_t>(s) * max_blocks_per_seq;
  const int32_t* prow = path + static_cast<int64_t>(s) * max_path;
  int before = -1;  // the path's entry before this batch
  for (int c = 0; c < len; c += 32) {
    const int j = c + lane;
    int node = j < len ? __ldg(prow + j) : -1;
    int prev = __shfl_up_sync(kFullMask, node, 1);
    if (lane == 0) prev = before;
    // increasing entries within the sequence's rows (so node >= j)
    const bool bad = j < len && (node <= prev || node >= n);
    if (__any_sync(kFullMask, bad)) {
      if (teller) atomicOr(err, PA_DEVERR_DRAFT);
      return;
    }
    int64_t src = -1, dst = -1;
    if (j < len && node != j) {
      const int ps = base + node, pd = base + j;
      const int bsrc = __ldg(trow + (ps >> lg)), bdst = __ldg(trow + (pd >> lg));
      if (static_cast<unsigned>(bsrc) < static_cast<unsigned>(num_blocks) &&
          static_cast<unsigned>(bdst) < static_cast<unsigned>(num_blocks)) {
        src = (static_cast<int64_t>(bsrc) << lg) + (ps & ((1 << lg) - 1));
        dst = (static_cast<int64_t>(bdst) << lg) + (pd & ((1 << lg) - 1));
      } else if (w == 0) {
        atomicOr(err, PA_DEVERR_BLOCK_ID);
      }
    }
    before = __shfl_sync(kFullMask, node, 31);
    const int m = min(32, len - c);
    for (int i = 0; i < m; i += 8) {
      uint4 row[8];
      int64_t to[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {  // (lanes past the path hold -1)
        const int64_t from = __shfl_sync(kFullMask, src, i + e);
        to[e] = __shfl_sync(kFullMask, dst, i + e);
        if (to[e] >= 0 && live) row[e] = cache[from * vec_per_row + col];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (to[e] >= 0 && live) cache[to[e] * vec_per_row + col] = row[e];
    }
  }
}

}  // namespace

cudaError_t launch_kv_accept(void* k_cache, void* v_cache, const int32_t* block_tables,
                             const int32_t* context_lens, const int32_t* query_start,
                             const int32_t* path, const int32_t* path_len, int num_seqs,
                             int max_path, int num_blocks, int log2_block_size,
                             int max_blocks_per_seq, int row_bytes, cudaStream_t stream) {
  unsigned* err = nullptr;
  cudaError_t e = device_error_word(&err);
  if (e != cudaSuccess) return e;
  const int vec = row_bytes / 16, warps = 2 * ((vec + 31) / 32);
  return launch_pdl(kv_accept_kernel, dim3(num_seqs, (warps + 3) / 4), dim3(128), 0, stream,
                    static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), block_tables,
                    context_lens, query_start, path, path_len, max_path, num_blocks,
                    log2_block_size, max_blocks_per_seq, vec, err);
}

// -------------------------------------------------------------- verification

namespace {

struct VerifyParams {
  int32_t* out_tokens;
  int32_t* out_path;
  int32_t* out_len;
  const float* target;
  const float* draft;  // null: the drafted tokens were picked, not sampled
  const int32_t* tokens;
  const int32_t* parents;  // null: chains
  const int32_t* query_start;
  const float* u_accept;
  const float* u_sample;
  int64_t target_stride, draft_stride;
  unsigned* err;
  int total_rows, vocab, max_query_len;
};

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyPart = 8 * kVerifyWarps / 32;  // a lane's share of a cluster's sums
constexpr int kVerifyBatch = 4;  // groups of 128 values that a warp takes at once
constexpr int kVerifyChunk = 128 * kVerifyBatch;
constexpr int kVerifyStages = 3;  // of a warp's ring: a chunk of p and one of q each
constexpr int kVerifyRing = kVerifyWarps * kVerifyStages * kVerifyChunk * 8;

// The mass left of a target row p after rejections at one node,
//   sampled drafts: R_0 = p, Z_0 = 1, R_{k+1} = max(R_k / Z_k - q, 0), Z_k = sum R_k.
// Where R_k > 0 it is A_k (p - t_k q), and where it is 0 the next one is 0 too; with
// F(t) = sum max(p - t q, 0), Z_k = A_k F(t_k), A_{k+1} = 1 / F(t_k) and
// t_{k+1} = t_k + F(t_k) (t_0 = 0, F counted as 1 there). A cancels from every
// comparison: one number t stands for any number of rejections, child x is
// accepted where u q(x) F(t) < max(p(x) - t q(x), 0), and the last token is drawn
// from max(p - t q, 0).
//   picked drafts (q one-hot): R = p without the rejected tokens.
struct Residual {
  double t;  // sampled drafts
  int gone;  // picked drafts: rejected tokens so far (their list is in shared memory)
};

// A float >= 0 as a double times 2^-896: its bits three places down, which holds for
// zero and subnormals too (an infinity becomes 2^128 2^-896). Two shifts, where the
// conversion instruction goes at a quarter of the rate of float64 arithmetic (measured:
// 16 to 62 a clock and SM).
__device__ __forceinline__ double scaled(float x) {
  const unsigned u = __float_as_uint(x);
  return __hiloint2double(static_cast<int>(u >> 3), static_cast<int>(u << 29));
}
constexpr double kUnscale = 0x1p896;

// sum += m where m > 0 (NaN: not), as one predicated addition.
__device__ __forceinline__ void add_positive(double& sum, double m) {
  asm("{\n .reg .pred p;\n setp.gt.f64 p, %1, 0d0000000000000000;\n @p add.f64 %0, %0, %1;\n}"
      : "+d"(sum)
      : "d"(m));
}

// Where a running sum over a warp's values (lane-major, N a lane, on top of `run`)
// first passes `want`: the index and the sum before it; index -1: nowhere. The same for
// the last value above 0. `run` then counts them all.
struct Passed {
  int first, last;
  double first_before, last_before;
};
template <int N>
__device__ __forceinline__ Passed find_passed(const double (&m)[N], double want, double& run, int lane) {
  double c[N];
  c[0] = m[0];
#pragma unroll
  for (int e = 1; e < N; ++e) c[e] = c[e - 1] + m[e];
  double incl = c[N - 1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl += t;
  }
  const double base = run + (incl - c[N - 1]);
  int hit = N, end = -1;
  double hit_before = 0.0, end_before = 0.0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if (!(m[e] > 0.0)) continue;
    const double before = e == 0 ? base : base + c[e - 1];
    if (hit == N && base + c[e] > want) {
      hit = e;
      hit_before = before;
    }
    end = e;
    end_before = before;
  }
  const unsigned hits = __ballot_sync(kFullMask, hit < N), ends = __ballot_sync(kFullMask, end >= 0);
  const int hl = hits ? __ffs(hits) - 1 : 0, el = ends ? 31 - __clz(ends) : 0;
  Passed r;
  r.first = __shfl_sync(kFullMask, lane * N + hit, hl);
  r.first_before = __shfl_sync(kFullMask, hit_before, hl);
  r.last = __shfl_sync(kFullMask, lane * N + end, el);
  r.last_before = __shfl_sync(kFullMask, end_before, el);
  if (!hits) r.first = -1;
  if (!ends) r.last = -1;
  run += __shfl_sync(kFullMask, incl, 31);
  return r;
}

__device__ __forceinline__ uint32_t cluster_address(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// A double into another CTA's shared memory, counted as 8 bytes by its mbarrier.
__device__ __forceinline__ void store_async(uint32_t addr, double v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(addr),
               "l"(__double_as_longlong(v)), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// As mbar_wait, for what other CTAs of the cluster stored.
__device__ __forceinline__ void mbar_wait_cluster(uint32_t bar, uint32_t parity, unsigned* err) {
  if (mbar_try_wait_cluster(bar, parity)) return;
  const uint64_t start = global_timer_ns();
  while (!mbar_try_wait_cluster(bar, parity)) {
    if (global_timer_ns() - start > kWaitLimitNs) {
      atomicOr(err, PA_DEVERR_TIMEOUT);
      return;
    }
  }
}

// One cluster of CTAs per sequence. Every CTA walks the rows in order with the
// same numbers (a row is tried where its parent is the last accepted row, which
// visits the children of each accepted row in order), each row's p and q at its
// token read up front by one thread. Sums over the vocabulary are split over
// the cluster's warps, a contiguous piece each, in 64 bits: a sampled draft's
// mass only when a later child is tried, and the last token's at the end, whose
// piece is then searched. All in float64. The bytes are one row of p and one of q per
// sequence; what bounds it are the sums of a sequence, one after the other: each
// needs the one before (about 2.4 us each over 128,256 values, of which the walk's and
// the exchange's latency is a third). Over 128,256 values: 64 trees of 16 41 us (inputs
// not in L2; 37 to 43 by the drawn numbers), 64 picked trees 30; 64 chains of 5 17.9, of 8
// 18.5, 64 picked chains of 5 15.7; 256 chains of 5 52, picked 43, 256 plain draws (p alone,
// 131 MB) 29. One chain of 5 over 32,000: 6.9 us.
//
// Rows that are not 16-byte aligned (VEC false: a vocabulary of 50,257, say) are read by
// plain loads instead of the rings: bulk copies need the alignment. 64 trees of 16 over
// 50,257 values 39.0 us, over 50,256 31.6; 64 picked chains of 5 10.9 and 10.9.
template <bool VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_draft_kernel(const VerifyParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  extern __shared__ __align__(128) uint8_t smem_raw[];
  // the warps' rings; per row p(token), q(token), u q(token), token, parent; then
  // the rejected tokens' list
  const int cap = p.max_query_len;
  double* s_p = reinterpret_cast<double*>(smem_raw + (VEC ? kVerifyRing : 0));
  double* s_q = s_p + cap;
  double* s_uq = s_q + cap;
  int* s_tok = reinterpret_cast<int*>(s_uq + cap);
  int* s_par = s_tok + cap;
  int* s_gone = s_par + cap;
  // two sets of the cluster's warps' sums, used in turns: a warp sends its part of a
  // sum only when it has read the one before, so a set is read by all before it is
  // written again
  __shared__ double s_warp[kVerifyWarps], s_piece[2][8 * kVerifyWarps];
  __shared__ uint64_t s_bar[kVerifyWarps][kVerifyStages], s_sum_bar[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x / ranks;

  if (VEC && lane == 0) {
    for (int i = 0; i < kVerifyStages; ++i) mbar_init(smem_u32(&s_bar[warp][i]), 1);
    fence_barrier_init();
  }
  const int pieces = ranks * kVerifyWarps;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_sum_bar[i]), 1);
      mbar_arrive_expect_tx(smem_u32(&s_sum_bar[i]), pieces * 8);
    }
    fence_barrier_init();
  }
  // (no CTA writes into another's shared memory before that has set its barriers up)
  auto others = cluster.barrier_arrive();
  pdl_wait();
  pdl_launch_dependents();
  const int q0 = __ldg(p.query_start + s), q1 = __ldg(p.query_start + s + 1);
  int n = q1 - q0;
  if (q0 < 0 || n < 0 || q1 > p.total_rows || n > p.max_query_len) {
    if (rank == 0 && tid == 0) atomicOr(p.err, PA_DEVERR_CONTEXT);
    n = 0;
  }
  int32_t* out_tokens = p.out_tokens + static_cast<int64_t>(s) * p.max_query_len;
  int32_t* out_path = p.out_path + static_cast<int64_t>(s) * p.max_query_len;
  if (n == 0) {  // (the same for the whole cluster)
    if (rank == 0) {
      for (int i = tid; i < p.max_query_len; i += kVerifyThreads) out_tokens[i] = out_path[i] = -1;
      if (tid == 0) p.out_len[s] = 0;
    }
    cluster.barrier_wait(std::move(others));
    return;
  }
  for (int i = 1 + tid; i < n; i += kVerifyThreads) {
    const int row = q0 + i;
    int par = p.parents != nullptr ? __ldg(p.parents + row) : i - 1;
    const int tok = __ldg(p.tokens + row);
    const bool tok_ok = static_cast<unsigned>(tok) < static_cast<unsigned>(p.vocab);
    const bool par_ok = par >= -1 && par < i;
    if (!(tok_ok && par_ok) && rank == 0) atomicOr(p.err, PA_DEVERR_DRAFT);
    if (!(tok_ok && par_ok)) par = -1;  // never tried
    s_par[i] = par;
    s_tok[i] = tok;
    // values not > 0 count as 0 (fmaxf: NaN too)
    const float pt = par >= 0 ? fmaxf(__ldg(p.target + (q0 + par) * p.target_stride + tok), 0.0f) : 0.0f;
    const float qt = par < 0 ? 0.0f : p.draft == nullptr ? 1.0f
                     : fmaxf(__ldg(p.draft + (q0 + par) * p.draft_stride + tok), 0.0f);
    s_p[i] = pt;
    s_q[i] = qt;
    s_uq[i] = static_cast<double>(__ldg(p.u_accept + row)) * static_cast<double>(qt);
  }
  cluster.barrier_wait(std::move(others));
  __syncthreads();

  // this warp's piece of the vocabulary: whole groups of 128 values
  const int groups = (p.vocab + 127) / 128, per = (groups + pieces - 1) / pieces;
  const int piece = rank * kVerifyWarps + warp;
  const int lo = static_cast<int>(min(static_cast<int64_t>(piece) * per * 128, static_cast<int64_t>(p.vocab)));
  const int hi = static_cast<int>(min(static_cast<int64_t>(piece + 1) * per * 128, static_cast<int64_t>(p.vocab)));

  auto load4 = [&](const float* row, int i, int end, float (&x)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = i + e < end ? __ldg(row + i + e) : 0.0f;
  };
  // values of one row: a lane's own of the 128 from i0 on, of the next 128, ... (0 from
  // `end` on). A whole chunk's loads stand without conditions: behind one, the move of
  // each loaded value waits for it before the next load.
  auto load_batch = [&](const float* row, int i0, int end, float (&x)[kVerifyBatch][4]) {
    row += i0 + lane * 4;
    if (i0 + kVerifyChunk <= end) {
#pragma unroll
      for (int u = 0; u < kVerifyBatch; ++u) {
        if constexpr (VEC) {
          const float4 f = __ldg(reinterpret_cast<const float4*>(row + u * 128));
          x[u][0] = f.x;
          x[u][1] = f.y;
          x[u][2] = f.z;
          x[u][3] = f.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[u][e] = __ldg(row + u * 128 + e);
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < kVerifyBatch; ++u) load4(row, u * 128, end - i0 - lane * 4, x[u]);
    }
  };
  // the masses of values i .. i + 3 from their p and q: with sampled drafts unscaled
  // and any not > 0 standing for 0, else scaled and >= 0. Sampled: q by shifts, p by
  // the conversion instruction, so that both pipes carry a part.
  auto masses = [&](auto sampled, const Residual& r, int i, const float (&x)[4], const float (&y)[4],
                    double (&m)[4]) {
    if constexpr (sampled.value) {
      const double t = -r.t * kUnscale;
#pragma unroll
      for (int e = 0; e < 4; ++e) m[e] = fma(t, scaled(fmaxf(y[e], 0.0f)), static_cast<double>(x[e]));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) m[e] = scaled(fmaxf(x[e], 0.0f));
      for (int g = 0; g < r.gone; ++g) {
        const int t = s_gone[g] - i;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t == e) m[e] = 0.0;
      }
    }
  };
  // This warp's ring: chunks arrive by bulk copies while earlier ones are summed (a
  // warp's own loads would hold too few bytes in flight: a pass of 128,256 values
  // took 24 us in one CTA of 512 threads). A chunk's use of the ring goes on from
  // the last one's, over all sums. What a sum leaves in the ring is the last
  // chunks of p and q that it took; another sum over the same piece at the same
  // node starts with them, as they are, and fetches the others meanwhile.
  const uint32_t ring = smem_u32(smem_raw) + warp * kVerifyStages * kVerifyChunk * 8;
  [[maybe_unused]] int ring_st = 0;    // slot of the next chunk
  [[maybe_unused]] uint32_t ring_ph = 0;  // a bit per slot: parity of its next arrival
  [[maybe_unused]] int held = -1, held_at = 0;  // node whose chunks are in the ring; the last sum's first chunk
  auto fetch = [&](int cur, bool both, int i0, int end, int st) {  // (by one lane)
    const uint32_t bytes = static_cast<uint32_t>(min(kVerifyChunk, end - i0) & ~3) * 4;
    const uint32_t bar = smem_u32(&s_bar[warp][st]), dst = ring + st * kVerifyChunk * 8;
    mbar_arrive_expect_tx(bar, both ? 2 * bytes : bytes);
    if (bytes == 0) return;
    bulk_load(dst, p.target + (q0 + cur) * p.target_stride + i0, bytes, bar);
    if (both) bulk_load(dst + kVerifyChunk * 4, p.draft + (q0 + cur) * p.draft_stride + i0, bytes, bar);
  };
  // a warp's sum over values [a, b); `whole`: they are its piece
  auto sum_as = [&](auto sampled, int cur, const Residual& r, int a, int b, bool whole) {
    double acc[kVerifyBatch][4] = {};
    const int chunks = (b - a + kVerifyChunk - 1) / kVerifyChunk;
    [[maybe_unused]] int at = 0, have = 0;  // first chunk taken; chunks in the ring already
    if constexpr (VEC) {
      if (whole && held == cur && chunks > 0) {
        have = min(chunks, kVerifyStages);
        at = held_at - have;
        if (at < 0) at += chunks;
        ring_st -= have;
        if (ring_st < 0) ring_st += kVerifyStages;
      }
      if (lane >= have && lane < min(chunks, kVerifyStages))  // (a lane each: have is 0 or all)
        fetch(cur, sampled.value, a + lane * kVerifyChunk, b, (ring_st + lane) % kVerifyStages);
      held = whole && sampled.value ? cur : -1;
      held_at = at;
    }
    for (int k = 0, c = at; k < chunks; ++k) {
      const int i0 = a + c * kVerifyChunk;
      float x[kVerifyBatch][4] = {}, y[kVerifyBatch][4] = {};
      if constexpr (VEC) {
        if (k >= have) {
          mbar_wait(smem_u32(&s_bar[warp][ring_st]), (ring_ph >> ring_st) & 1, p.err);
          ring_ph ^= 1u << ring_st;
        }
        const uint32_t src = ring + ring_st * kVerifyChunk * 8 + lane * 16;
        if (i0 + kVerifyChunk <= b) {
#pragma unroll
          for (int u = 0; u < kVerifyBatch; ++u) {
            ElemTraits<float>::unpack(lds128(src + u * 512), x[u]);
            if (sampled.value) ElemTraits<float>::unpack(lds128(src + kVerifyChunk * 4 + u * 512), y[u]);
          }
        } else
#pragma unroll
        for (int u = 0; u < kVerifyBatch; ++u) {
          const int i = i0 + u * 128 + lane * 4;
          if (i + 4 <= b) {
            ElemTraits<float>::unpack(lds128(src + u * 512), x[u]);
            if (sampled.value) ElemTraits<float>::unpack(lds128(src + kVerifyChunk * 4 + u * 512), y[u]);
          } else if (i < b) {  // the vocabulary's last one to three values
            load4(p.target + (q0 + cur) * p.target_stride, i, b, x[u]);
            if (sampled.value) load4(p.draft + (q0 + cur) * p.draft_stride, i, b, y[u]);
          }
        }
      } else {
        load_batch(p.target + (q0 + cur) * p.target_stride, i0, b, x);
        if (sampled.value) load_batch(p.draft + (q0 + cur) * p.draft_stride, i0, b, y);
      }
#pragma unroll
      for (int u = 0; u < kVerifyBatch; ++u) {
        double m[4];
        masses(sampled, r, i0 + u * 128 + lane * 4, x[u], y[u], m);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (sampled.value)
            add_positive(acc[u][e], m[e]);
          else
            acc[u][e] += m[e];
        }
      }
      if (++c == chunks) c = 0;
      if constexpr (VEC) {
        __syncwarp();  // every lane has read the chunk
        if (lane == 0 && k + kVerifyStages < chunks) {
          int f = at + k + kVerifyStages;
          if (f >= chunks) f -= chunks;
          fetch(cur, sampled.value, a + f * kVerifyChunk, b, ring_st);
        }
        if (++ring_st == kVerifyStages) ring_st = 0;
      }
    }
    double t = 0.0;
#pragma unroll
    for (int u = 0; u < kVerifyBatch; ++u) t += (acc[u][0] + acc[u][1]) + (acc[u][2] + acc[u][3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFullMask, t, o);
    return sampled.value ? t : t * kUnscale;
  };
  int turn = 0;
  uint32_t turn_ph = 0;  // a bit per set of sums
  // the sum over the vocabulary: every warp sends its piece's to every CTA;
  // a lane then holds those of kVerifyPart pieces
  auto total_mass = [&](double acc, double (&part)[kVerifyPart]) {
    const uint32_t bar = smem_u32(&s_sum_bar[turn]);
    if (lane < ranks)
      store_async(cluster_address(smem_u32(&s_piece[turn][piece]), lane), acc, cluster_address(bar, lane));
    mbar_wait_cluster(bar, (turn_ph >> turn) & 1, p.err);
    turn_ph ^= 1u << turn;
    if (tid == 0) mbar_arrive_expect_tx(bar, pieces * 8);  // for its next use
#pragma unroll
    for (int e = 0; e < kVerifyPart; ++e) {
      const int at = kVerifyPart * lane + e;
      part[e] = at < pieces ? s_piece[turn][at] : 0.0;
    }
    turn ^= 1;
    double z = 0.0;
#pragma unroll
    for (int e = 0; e < kVerifyPart; ++e) z += part[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(kFullMask, z, o);
    return z;
  };

  int cur = 0, len = 1;
  Residual r{0.0, 0};
  double z = 1.0, part[kVerifyPart];
  bool stale = false;  // z has not been summed since the last rejection
  if (rank == 0 && tid == 0) out_path[0] = 0;
  double want = 0.0, run = 0.0;  // of the search: the sum to pass, the sum before [a, b)
  bool good = false;
  // where the running sum passes `want` (by rounding, or with u outside [0, 1),
  // nowhere: the last place with a mass)
  auto narrow = [&](const Passed& f) {
    run = f.first >= 0 ? f.first_before : f.last_before;
    return f.first >= 0 ? f.first : f.last;
  };
  // which warp has it, given every warp's sum of its part
  auto place = [&](double sum) {
    __syncthreads();
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    const double w[1] = {lane < kVerifyWarps ? s_warp[lane] : 0.0};
    return narrow(find_passed(w, want, run, lane));
  };
  // The walk, each sum that it needs, and the search in a long piece go through one
  // loop: the summing code then stands in the program once (in six places it was
  // larger than the instruction cache likes).
  int a = lo, b = hi, step = 0;  // step > 0: searching, a part of that many values a warp
  bool mine = false;             // the place is in this CTA's piece [a, b)
  for (int i = 1;;) {
    if (step == 0) {
      // on to the next child that needs a sum, or to the last row's
      for (;; ++i) {
        // the next row whose parent is `cur`
        unsigned kin = 0;
        for (int base = i & ~31; base < n; base += 32) {
          const int row = base + lane;
          kin = __ballot_sync(kFullMask, row >= i && row < n && s_par[row] == cur);
          if (kin != 0) {
            i = base + __ffs(kin) - 1;
            break;
          }
        }
        if (kin == 0) i = n;
        if (i == n || stale) break;
        double left = fmax(fma(-r.t, s_q[i], s_p[i]), 0.0);
        for (int g = 0; g < r.gone; ++g)
          if (s_gone[g] == s_tok[i]) left = 0.0;
        if (s_uq[i] * z < left) {
          if (rank == 0 && tid == 0) {
            out_tokens[len - 1] = s_tok[i];
            out_path[len] = i;
          }
          cur = i;
          ++len;
          r = Residual{0.0, 0};
          z = 1.0;
        } else if (p.draft != nullptr) {
          r.t += z;
          stale = true;
        } else {
          z = fmax(z - left, 0.0);
          __syncthreads();
          if (tid == 0) s_gone[r.gone] = s_tok[i];
          __syncthreads();
          ++r.gone;
        }
      }
    }
    const int from = step == 0 ? a : min(a + warp * step, b);
    const int to = step == 0 ? b : min(from + step, b);
    const double sum = r.t != 0.0 ? sum_as(std::true_type{}, cur, r, from, to, step == 0)
                                  : sum_as(std::false_type{}, cur, r, from, to, step == 0);
    if (step == 0) {
      z = total_mass(sum, part);
      if (i < n) {
        stale = false;
        continue;
      }
      if (!(z > 0.0) && (r.t != 0.0 || r.gone != 0)) {  // nothing left: the target's own row
        r = Residual{0.0, 0};
        continue;
      }
      // the lowest index whose running sum exceeds u z: its piece, then its place there
      good = z > 0.0 && z < 0x1p127;  // (an infinite value counts 2^128)
      if (!good) break;
      want = static_cast<double>(__ldg(p.u_sample + s)) * z;
      const int at = narrow(find_passed(part, want, run, lane));
      mine = at / kVerifyWarps == rank;
      if (!mine) break;
      a = static_cast<int>(min(static_cast<int64_t>(at) * per * 128, static_cast<int64_t>(p.vocab)));
      b = static_cast<int>(min(static_cast<int64_t>(at + 1) * per * 128, static_cast<int64_t>(p.vocab)));
    } else {
      a = min(a + place(sum) * step, b);
      b = min(a + step, b);
    }
    if (b - a <= kVerifyWarps * kVerifyChunk) break;
    step = ((b - a + 127) / 128 + kVerifyWarps - 1) / kVerifyWarps * 128;
  }
  if (mine) {
    // a chunk each: the warp that has it holds its values
    float x[kVerifyBatch][4], y[kVerifyBatch][4] = {};
    double m[kVerifyBatch][4], sum = 0.0;
    const int i0 = a + warp * kVerifyChunk;
    load_batch(p.target + (q0 + cur) * p.target_stride, i0, b, x);
    if (r.t != 0.0) load_batch(p.draft + (q0 + cur) * p.draft_stride, i0, b, y);
#pragma unroll
    for (int u = 0; u < kVerifyBatch; ++u) {
      if (r.t != 0.0)
        masses(std::true_type{}, r, i0 + u * 128 + lane * 4, x[u], y[u], m[u]);
      else
        masses(std::false_type{}, r, i0 + u * 128 + lane * 4, x[u], y[u], m[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        m[u][e] = m[u][e] > 0.0 ? r.t != 0.0 ? m[u][e] : m[u][e] * kUnscale : 0.0;
        sum += m[u][e];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    if (warp == place(sum)) {
      int chosen = -1, last = -1;
#pragma unroll
      for (int u = 0; u < kVerifyBatch; ++u) {
        const Passed f = find_passed(m[u], want, run, lane);
        if (chosen < 0 && f.first >= 0) chosen = i0 + u * 128 + f.first;
        if (f.last >= 0) last = i0 + u * 128 + f.last;
      }
      if (lane == 0) out_tokens[len - 1] = chosen >= 0 ? chosen : last;
    }
  }
  if (rank == 0) {
    if (!good && tid == 0) {
      atomicOr(p.err, PA_DEVERR_DRAFT);
      out_tokens[len - 1] = -1;
    }
    for (int i = len + tid; i < p.max_query_len; i += kVerifyThreads) out_tokens[i] = out_path[i] = -1;
    if (tid == 0) p.out_len[s] = len;
  }
  // (a CTA may leave: all that others write into its shared memory has been waited for)
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyShape& sh, int32_t* out_tokens, int32_t* out_path,
                                int32_t* out_len, const float* target, const float* draft,
                                const int32_t* tokens, const int32_t* parents,
                                const int32_t* query_start, const float* u_accept,
                                const float* u_sample, cudaStream_t stream) {
  VerifyParams p{};
  p.out_tokens = out_tokens;
  p.out_path = out_path;
  p.out_len = out_len;
  p.target = target;
  p.draft = draft;
  p.tokens = tokens;
  p.parents = parents;
  p.query_start = query_start;
  p.u_accept = u_accept;
  p.u_sample = u_sample;
  p.target_stride = sh.target_stride;
  p.draft_stride = sh.draft_stride;
  p.total_rows = sh.total_rows;
  p.vocab = sh.vocab;
  p.max_query_len = sh.max_query_len;
  cudaError_t e = device_error_word(&p.err);
  if (e != cudaSuccess) return e;
  // CTAs per sequence, up to the portable 8, each with a few thousand values at least.
  // Where rows are summed again after rejections (trees with draft probabilities), 8: a
  // sequence's sums follow each other, and 8 CTAs keep 3/4 of 128,256 values in their
  // rings (7 rejections in each of 64 sequences: 44 us, with 4 CTAs 56; 64 trees of 16:
  // 33.5 and 34.6). Else as many as keep the launch within one wave of resident CTAs, two an
  // SM (one draw a sequence over 128,256 values: 64 sequences 10.2 us with 4 CTAs, 15.3 with
  // 8; 256 sequences 28 us with 1, 53 with 8).
  int ranks = 1;
  const bool again = draft != nullptr && parents != nullptr;
  while (ranks < 8 && (again || sh.num_seqs * ranks <= 148) && sh.vocab / ranks > 4096) ranks *= 2;
  auto vec_ok = [](const float* x, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && stride % 4 == 0;
  };
  const bool vec = vec_ok(target, sh.target_stride) && (draft == nullptr || vec_ok(draft, sh.draft_stride));
  auto kernel = vec ? verify_draft_kernel<true> : verify_draft_kernel<false>;
  const int smem = (vec ? kVerifyRing : 0) + sh.max_query_len * 36;
  static std::atomic<unsigned long long> configured[2] = {{0}, {0}};
  if ((e = ensure_smem(kernel, kVerifyRing + kMaxVerifyRows * 36, configured[vec])) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sh.num_seqs) * ranks);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace pa
