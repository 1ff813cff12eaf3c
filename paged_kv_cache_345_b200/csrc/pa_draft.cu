// The cache side of a decode step with drafted tokens: rows with norms and
// rotation written into the cache, verification of the drafted tokens, and the
// move of the accepted rows into place. (The attention between them is
// pa_tree.cu.) "What is paged attention in vLLM, and why does it matter?", Step
// 4: each decoding step writes the new tokens' keys and values into the last
// block; here a step writes several per sequence and keeps some of them.
#include <cmath>
#include <cstdint>

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
  float eps;
};

// Rows of T; a lane holds 16 bytes of a head's row, kLanes lanes a row, so a
// warp instruction moves kRows rows. A unit of work is U such instructions of
// one token (its q heads, then k, then v heads); one warp per unit, all its
// loads first (before the position is known). HBM-bound: every row is read and written once, the cosines and
// sines of a token once per unit from L1/L2.
template <typename T, int D>
struct RowsConfig {
  static constexpr int kEPL = ElemTraits<T>::kPer16B;
  static constexpr int kLanes = D / kEPL;
  static constexpr int kRows = 32 / kLanes;
  static constexpr int kU = 4;
  static constexpr int kWarps = 4;  // per CTA
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

template <typename T, int D, bool FP8, bool INTERLEAVED>
__global__ void __launch_bounds__(RowsConfig<T, D>::kWarps * 32)
    qk_norm_rope_append_kernel(const RowsParams p) {
  using Cfg = RowsConfig<T, D>;
  constexpr int EPL = Cfg::kEPL, LPR = Cfg::kLanes, U = Cfg::kU;
  pdl_wait();
  pdl_launch_dependents();
  const unsigned unit = blockIdx.x * Cfg::kWarps + (threadIdx.x >> 5);
  const unsigned tok = unit / p.units_per_token;
  if (tok >= static_cast<unsigned>(p.num_tokens)) return;
  const int lane = threadIdx.x & 31, li = lane % LPR;
  const int pos = __ldg(p.positions + tok);
  const int64_t slot = __ldg(p.slots + tok);
  const int row0 = static_cast<int>(unit - tok * p.units_per_token) * (U * Cfg::kRows) + lane / LPR;
  const int hq = p.num_heads, hkv = p.num_kv_heads, total = hq + 2 * hkv;

  // rows of this unit: kind 0 q, 1 k, 2 v, 3 none
  int kind[U], head[U];
  uint4 raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = row0 + u * Cfg::kRows;
    kind[u] = r < hq ? 0 : r < hq + hkv ? 1 : r < total ? 2 : 3;
    head[u] = kind[u] == 0 ? r : kind[u] == 1 ? r - hq : r - hq - hkv;
    raw[u] = make_uint4(0, 0, 0, 0);
    if (kind[u] != 3) {
      const T* base = static_cast<const T*>(kind[u] == 0 ? p.q : kind[u] == 1 ? p.k : p.v);
      const int64_t st = kind[u] == 0 ? p.q_stride : kind[u] == 1 ? p.k_stride : p.v_stride;
      // (not the read-only path: q_out may be q)
      raw[u] = __ldcs(reinterpret_cast<const uint4*>(base + tok * st + head[u] * D + li * EPL));
    }
  }
  if (pos < 0) return;  // padding
  if (pos >= p.max_position || slot >= p.num_slots) {
    if (lane == 0 && row0 == 0)
      atomicOr(p.err, pos >= p.max_position ? PA_DEVERR_POSITION : PA_DEVERR_SLOT);
    if (pos >= p.max_position) return;
  }
  if (slot < 0 || slot >= p.num_slots) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kind[u] != 0) kind[u] = 3;
  }
  // cosines and sines of this lane's elements
  const int half = p.rotary_dim >> 1;
  const int e0 = li * EPL;
  const bool rotated = e0 < p.rotary_dim;
  constexpr int NC = INTERLEAVED ? EPL / 2 : EPL;
  float cs[NC], sn[NC];
  int partner = lane;  // lane that holds the other halves of this lane's pairs
  if (rotated) {
    const float* c = p.cos_sin + static_cast<int64_t>(pos) * p.rotary_dim +
                     (INTERLEAVED ? e0 / 2 : e0 < half ? e0 : e0 - half);
    load_floats<NC>(c, cs);
    load_floats<NC>(c + half, sn);
    if (!INTERLEAVED) {
      partner = e0 < half ? lane + half / EPL : lane - half / EPL;
      if (e0 < half) {
#pragma unroll
        for (int i = 0; i < NC; ++i) sn[i] = -sn[i];
      }
    }
  }
  const int pe0 = (partner % LPR) * EPL;

#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[EPL];
    ElemTraits<T>::unpack(raw[u], x);
    if (__any_sync(kFullMask, kind[u] < 2)) {  // (a v row is copied as it is)
      float rs = 1.0f, w[EPL], wp[EPL];
      const T* weight = static_cast<const T*>(kind[u] == 0 ? p.q_weight : p.k_weight);
      if (__any_sync(kFullMask, weight != nullptr && kind[u] < 2)) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
        if (weight != nullptr) rs = rsqrtf(ss * (1.0f / D) + p.eps);
      }
      if (weight != nullptr) {
        ElemTraits<T>::unpack(__ldg(reinterpret_cast<const uint4*>(weight + e0)), w);
        if (!INTERLEAVED) ElemTraits<T>::unpack(__ldg(reinterpret_cast<const uint4*>(weight + pe0)), wp);
      } else {
#pragma unroll
        for (int e = 0; e < EPL; ++e) w[e] = wp[e] = 1.0f;
      }
      float y[EPL];
#pragma unroll
      for (int e = 0; e < EPL; ++e) y[e] = x[e] * rs * w[e];
      if constexpr (INTERLEAVED) {
        if (rotated) {
#pragma unroll
          for (int i = 0; i < EPL / 2; ++i) {
            const float a = y[2 * i], b = y[2 * i + 1];
            y[2 * i] = a * cs[i] - b * sn[i];
            y[2 * i + 1] = b * cs[i] + a * sn[i];
          }
        }
      } else {
        // the partner's raw 16 bytes (fewer shuffles than its normed floats)
        uint4 o;
        o.x = __shfl_sync(kFullMask, raw[u].x, partner);
        o.y = __shfl_sync(kFullMask, raw[u].y, partner);
        o.z = __shfl_sync(kFullMask, raw[u].z, partner);
        o.w = __shfl_sync(kFullMask, raw[u].w, partner);
        float z[EPL];
        ElemTraits<T>::unpack(o, z);
        if (rotated) {
#pragma unroll
          for (int e = 0; e < EPL; ++e) y[e] = y[e] * cs[e] + z[e] * rs * wp[e] * sn[e];
        }
      }
      if (kind[u] < 2) {
#pragma unroll
        for (int e = 0; e < EPL; ++e) x[e] = y[e];
      }
    }
    if (kind[u] == 3) continue;
    if (FP8 && kind[u] != 0) {
      // one rounding: the float32 row divided by its head's scale, to E4M3
      const float sc = __ldg((kind[u] == 1 ? p.k_scale : p.v_scale) + head[u]);
      uint32_t r[EPL / 4];
#pragma unroll
      for (int i = 0; i < EPL / 4; ++i)
        r[i] = static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], sc), __fdiv_rn(x[4 * i + 1], sc))) |
               (static_cast<uint32_t>(f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], sc), __fdiv_rn(x[4 * i + 3], sc))) << 16);
      uint8_t* dst = static_cast<uint8_t*>(kind[u] == 1 ? p.k_cache : p.v_cache) +
                     (slot * hkv + head[u]) * D + e0;
      if constexpr (EPL == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(r[0], r[1]);
      continue;
    }
    uint4 o;
    if constexpr (EPL == 8) {
      // v: its own bits; q and k: one rounding from float32
      if (kind[u] == 2) {
        o = raw[u];
      } else {
        o = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4 % EPL], x[5 % EPL]),
                       pack_bf16x2(x[6 % EPL], x[7 % EPL]));
      }
    } else {
      o = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    T* dst = kind[u] == 0 ? static_cast<T*>(p.q_out) + tok * p.q_out_stride + head[u] * D + e0
                          : static_cast<T*>(kind[u] == 1 ? p.k_cache : p.v_cache) +
                                (slot * hkv + head[u]) * D + e0;
    *reinterpret_cast<uint4*>(dst) = o;
  }
}

template <typename T, int D, bool FP8>
cudaError_t launch_rows_t(RowsParams p, bool interleaved, cudaStream_t stream) {
  using Cfg = RowsConfig<T, D>;
  const int rows = p.num_heads + 2 * p.num_kv_heads, per = Cfg::kRows * Cfg::kU;
  p.units_per_token = static_cast<unsigned>((rows + per - 1) / per);
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
// sequence.
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

constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyBatch = 4;  // groups of 128 values that a warp loads at once

// The mass left of a target row after the rejections at one node,
//   sampled drafts: R_0 = p, R_{k+1} = max(R_k / Z_k - q, 0), Z_k = sum R_k (Z_0 = 1).
// Where R_k > 0 it is A_k p - B_k q with A_{k+1} = A_k / Z_k, B_{k+1} = B_k / Z_k + 1,
// and where it is 0, A_{k+1} p - B_{k+1} q <= -q <= 0: so R_k = max(A_k p - B_k q, 0)
// for every k, and two numbers stand for any number of rejections.
//   picked drafts (q one-hot): R = p without the rejected tokens.
// Values that are not > 0 count as 0.
struct Residual {
  double a, b;       // sampled drafts
  int gone;          // picked drafts: rejected tokens so far (their list is in shared memory)
};

__device__ __forceinline__ double mass_of(float p, float q, double a, double b) {
  const double x = p > 0.0f ? static_cast<double>(p) : 0.0;
  if (b == 0.0) return x;
  const double y = q > 0.0f ? static_cast<double>(q) : 0.0;
  const double r = a * x - b * y;
  return r > 0.0 ? r : 0.0;
}

// One cluster of CTAs per sequence. Every CTA walks the rows in order with the
// same numbers (a row is tried where its parent is the last accepted row, which
// visits the children of each accepted row in order), each row's p and q at its
// token read up front by one thread. Sums over the vocabulary are split over
// the cluster's warps, a contiguous piece each, in 64 bits: a sampled draft's
// mass only when a later child is tried, and the last token's at the end, whose
// piece is then searched by one warp. Bound by reading one row of p and one of
// q per sequence.
template <bool VEC>
__global__ void __launch_bounds__(kVerifyThreads, 2) verify_draft_kernel(const VerifyParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
  extern __shared__ __align__(16) uint8_t smem_raw[];
  // per row: p(token), q(token), u, token, parent; then the rejected tokens' list
  const int cap = p.max_query_len;
  float* s_p = reinterpret_cast<float*>(smem_raw);
  float* s_q = s_p + cap;
  float* s_u = s_q + cap;
  int* s_tok = reinterpret_cast<int*>(s_u + cap);
  int* s_par = s_tok + cap;
  int* s_gone = s_par + cap;
  __shared__ double s_warp[kVerifyWarps], s_rank[2][8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = blockIdx.x / ranks;

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
    s_u[i] = __ldg(p.u_accept + row);
    s_p[i] = par >= 0 ? __ldg(p.target + (q0 + par) * p.target_stride + tok) : 0.0f;
    s_q[i] = par >= 0 && p.draft != nullptr ? __ldg(p.draft + (q0 + par) * p.draft_stride + tok) : 1.0f;
  }
  cluster.sync();  // (every CTA runs before any writes into another's shared memory)

  // this warp's piece of the vocabulary: whole groups of 128 values
  const int pieces = ranks * kVerifyWarps;
  const int groups = (p.vocab + 127) / 128, per = (groups + pieces - 1) / pieces;
  const int piece = rank * kVerifyWarps + warp;
  const int lo = static_cast<int>(min(static_cast<int64_t>(piece) * per * 128, static_cast<int64_t>(p.vocab)));
  const int hi = static_cast<int>(min(static_cast<int64_t>(piece + 1) * per * 128, static_cast<int64_t>(p.vocab)));

  auto load4 = [&](const float* row, int i, float (&x)[4]) {
    if (VEC && i + 3 < p.vocab) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(row + i));
      x[0] = f.x;
      x[1] = f.y;
      x[2] = f.z;
      x[3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i + e < p.vocab ? __ldg(row + i + e) : 0.0f;
    }
  };
  // the residual's masses of kVerifyBatch groups of 4 values of row `cur`: lane's
  // own of the 128 from i0 on, of the next 128, ... (0 from hi on); all loads first
  auto masses = [&](int cur, const Residual& r, int i0, double (&m)[kVerifyBatch][4]) {
    float x[kVerifyBatch][4], y[kVerifyBatch][4];
    const float* prow = p.target + (q0 + cur) * p.target_stride;
    const float* qrow = p.draft + (q0 + cur) * p.draft_stride;
#pragma unroll
    for (int u = 0; u < kVerifyBatch; ++u) {
      const int i = i0 + u * 128 + lane * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[u][e] = y[u][e] = 0.0f;
      if (i < hi) {
        load4(prow, i, x[u]);
        if (r.b != 0.0) load4(qrow, i, y[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kVerifyBatch; ++u) {
      const int i = i0 + u * 128 + lane * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) m[u][e] = mass_of(x[u][e], y[u][e], r.a, r.b);
      for (int g = 0; g < r.gone; ++g) {
        const int t = s_gone[g] - i;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t == e) m[u][e] = 0.0;
      }
    }
  };
  int turn = 0;
  // the sum over the vocabulary; s_warp then holds the pieces' sums of this
  // CTA and s_rank[which] the CTAs'
  auto total_mass = [&](int cur, const Residual& r, int* which) {
    double acc = 0.0;
    for (int i0 = lo; i0 < hi; i0 += 128 * kVerifyBatch) {
      double m[kVerifyBatch][4];
      masses(cur, r, i0, m);
#pragma unroll
      for (int u = 0; u < kVerifyBatch; ++u) acc += (m[u][0] + m[u][1]) + (m[u][2] + m[u][3]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(kFullMask, acc, o);
    __syncthreads();  // (earlier readers of s_warp are done)
    if (lane == 0) s_warp[warp] = acc;
    __syncthreads();
    *which = turn;
    if (warp == 0) {
      double t = 0.0;
      for (int w = 0; w < kVerifyWarps; ++w) t += s_warp[w];
      if (lane < ranks) *cluster.map_shared_rank(&s_rank[turn][rank], lane) = t;
    }
    cluster.sync();
    double z = 0.0;
    for (int c = 0; c < ranks; ++c) z += s_rank[turn][c];
    turn ^= 1;  // (the next sum's writes to this slot lie behind another cluster.sync)
    return z;
  };

  int cur = 0, len = 1, which = 0;
  Residual r{1.0, 0.0, 0};
  double z = 1.0;
  bool stale = false;  // z has not been summed since the last rejection
  if (rank == 0 && tid == 0) out_path[0] = 0;
  for (int i = 1; i < n; ++i) {
    if (s_par[i] != cur) continue;
    if (stale) {
      z = total_mass(cur, r, &which);
      stale = false;
    }
    double left = mass_of(s_p[i], s_q[i], r.a, r.b);
    for (int g = 0; g < r.gone; ++g)
      if (s_gone[g] == s_tok[i]) left = 0.0;
    const double qx = s_q[i] > 0.0f ? static_cast<double>(s_q[i]) : 0.0;
    if (static_cast<double>(s_u[i]) * qx * z < left) {
      if (rank == 0 && tid == 0) {
        out_tokens[len - 1] = s_tok[i];
        out_path[len] = i;
      }
      cur = i;
      ++len;
      r = Residual{1.0, 0.0, 0};
      z = 1.0;
      continue;
    }
    if (p.draft != nullptr) {
      // (nothing left: stays so)
      r = z > 0.0 ? Residual{r.a / z, r.b / z + 1.0, 0} : Residual{0.0, 1.0, 0};
      stale = true;
    } else {
      z = fmax(z - left, 0.0);
      __syncthreads();
      if (tid == 0) s_gone[r.gone] = s_tok[i];
      __syncthreads();
      ++r.gone;
    }
  }
  z = total_mass(cur, r, &which);
  if (!(z > 0.0)) {  // nothing left: the target's own row
    r = Residual{1.0, 0.0, 0};
    z = total_mass(cur, r, &which);
  }
  // the lowest index whose running sum exceeds u z: its CTA, its warp's piece, its place
  const bool good = z > 0.0 && z < INFINITY;
  const double want = static_cast<double>(__ldg(p.u_sample + s)) * z;
  int chosen = -1;
  {
    double before = 0.0;
    int at = -1, last = -1;
    double at_before = 0.0, last_before = 0.0;
    for (int c = 0; c < ranks; ++c) {
      const double t = s_rank[which][c];
      if (t > 0.0) {
        last = c;
        last_before = before;
      }
      if (at < 0 && before + t > want) {
        at = c;
        at_before = before;
      }
      before += t;
    }
    if (at < 0) {  // rounding, or u outside [0, 1)
      at = last;
      at_before = last_before;
    }
    if (good && rank == at) {
      double b2 = at_before, w_before = 0.0, wl_before = 0.0;
      int aw = -1, lw = -1;
      for (int w = 0; w < kVerifyWarps; ++w) {
        const double t = s_warp[w];
        if (t > 0.0) {
          lw = w;
          wl_before = b2;
        }
        if (aw < 0 && b2 + t > want) {
          aw = w;
          w_before = b2;
        }
        b2 += t;
      }
      if (aw < 0) {
        aw = lw;
        w_before = wl_before;
      }
      if (warp == aw) {
        double run = w_before;
        int last_pos = -1;
        for (int i0 = lo; i0 < hi && chosen < 0; i0 += 128 * kVerifyBatch) {
          double mm[kVerifyBatch][4];
          masses(cur, r, i0, mm);
#pragma unroll
          for (int u = 0; u < kVerifyBatch; ++u) {
            const int i = i0 + u * 128 + lane * 4;
            const double(&m)[4] = mm[u];
            const double c0 = m[0], c1 = c0 + m[1], c2 = c1 + m[2], c3 = c2 + m[3];
            double incl = c3;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const double t = __shfl_up_sync(kFullMask, incl, o);
              if (lane >= o) incl += t;
            }
            const double b = run + (incl - c3);
            const int hit = m[0] > 0.0 && b + c0 > want ? 0 : m[1] > 0.0 && b + c1 > want ? 1
                            : m[2] > 0.0 && b + c2 > want ? 2 : m[3] > 0.0 && b + c3 > want ? 3 : 4;
            const int lastp = m[3] > 0.0 ? 3 : m[2] > 0.0 ? 2 : m[1] > 0.0 ? 1 : m[0] > 0.0 ? 0 : -1;
            const unsigned hits = __ballot_sync(kFullMask, hit < 4);
            const unsigned pos = __ballot_sync(kFullMask, lastp >= 0);
            if (chosen < 0 && hits) chosen = __shfl_sync(kFullMask, i + hit, __ffs(hits) - 1);
            if (pos) last_pos = __shfl_sync(kFullMask, i + lastp, 31 - __clz(pos));
            run += __shfl_sync(kFullMask, incl, 31);
          }
        }
        if (chosen < 0) chosen = last_pos;
        if (lane == 0) out_tokens[len - 1] = chosen;
      }
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
  cluster.sync();  // no CTA leaves while another may still write its shared memory
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
  // CTAs per sequence: as many (up to the portable 8) as keep the launch within
  // one wave of resident CTAs (two an SM) and leave each a few thousand values
  int ranks = 1;
  while (ranks < 8 && sh.num_seqs * ranks <= 148 && sh.vocab / ranks > 4096) ranks *= 2;
  auto vec_ok = [](const float* x, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == 0 && stride % 4 == 0;
  };
  const bool vec = vec_ok(target, sh.target_stride) && (draft == nullptr || vec_ok(draft, sh.draft_stride));
  auto kernel = vec ? verify_draft_kernel<true> : verify_draft_kernel<false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sh.num_seqs) * ranks);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(sh.max_query_len) * 24;
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
