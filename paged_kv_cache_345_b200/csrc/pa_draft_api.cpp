// C-ABI shim of the calls for decode steps with drafted tokens: argument checks
// on the host, then the launches.
#include <cmath>
#include <cstdint>

#include "pa.h"
#include "pa_internal.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
bool known_dtype(int dt) { return dt == PA_F32 || dt == PA_BF16 || dt == PA_FP8_E4M3; }

int cuda_fail(const char* what, cudaError_t e) {
  return pa_fail(PA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int pa_qk_norm_rope_append(void* q_out, const void* q, const void* k, const void* v,
                           int64_t q_out_stride, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                           int num_tokens, const float* cos_sin, int max_position, int rotary_dim,
                           int interleaved, const void* q_weight, const void* k_weight, float eps,
                           void* k_cache, void* v_cache, const float* k_scale,
                           const float* v_scale, int num_blocks, int block_size, int num_heads,
                           int num_kv_heads, int head_dim, pa_dtype dtype, pa_stream_t stream) {
  const char* me = "pa_qk_norm_rope_append";
  if (num_tokens < 0) return pa_fail(PA_ERR_INVALID, "%s: num_tokens < 0", me);
  if (num_tokens == 0) return PA_OK;
  if (!q_out || !q || !k || !v || !positions || !slot_mapping || !cos_sin || !k_cache || !v_cache)
    return pa_fail(PA_ERR_INVALID, "%s: null pointer", me);
  if (!known_dtype(dtype)) return pa_fail(PA_ERR_UNSUPPORTED, "%s: dtype %d", me, dtype);
  const bool fp8 = dtype == PA_FP8_E4M3;
  if (fp8 ? (!k_scale || !v_scale) : (k_scale || v_scale))
    return pa_fail(PA_ERR_INVALID, "%s: k_scale and v_scale go with (and only with) E4M3 caches", me);
  if (num_blocks <= 0 || block_size <= 0 || num_heads <= 0 || num_kv_heads <= 0)
    return pa_fail(PA_ERR_INVALID, "%s: sizes must be positive", me);
  if (num_heads > 65535 || num_kv_heads > 65535)
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: more than 65535 heads", me);
  if (head_dim != 64 && head_dim != 128)
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d (built: 64, 128)", me, head_dim);
  if (max_position <= 0) return pa_fail(PA_ERR_INVALID, "%s: max_position must be positive", me);
  // half of rotary_dim is whole 16-byte pieces of a row
  const int step = dtype == PA_F32 ? 8 : 16;
  if (rotary_dim <= 0 || rotary_dim > head_dim || rotary_dim % step != 0)
    return pa_fail(PA_ERR_INVALID, "%s: rotary_dim %d not a multiple of %d in [%d, %d]", me,
                   rotary_dim, step, step, head_dim);
  if (!std::isfinite(eps) || eps < 0.0f)
    return pa_fail(PA_ERR_INVALID, "%s: eps must be finite and >= 0", me);
  const int per16 = dtype == PA_F32 ? 4 : 8;  // elements of 16 bytes
  const int64_t qrow = static_cast<int64_t>(num_heads) * head_dim;
  const int64_t kvrow = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (num_tokens > 1 && (q_out_stride < qrow || q_stride < qrow || k_stride < kvrow || v_stride < kvrow))
    return pa_fail(PA_ERR_INVALID, "%s: a stride is shorter than its row", me);
  if (q_out_stride % per16 || q_stride % per16 || k_stride % per16 || v_stride % per16)
    return pa_fail(PA_ERR_INVALID, "%s: strides must be multiples of 16 bytes", me);
  if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(cos_sin, 16) ||
      !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(positions, 4) ||
      !aligned(slot_mapping, 8) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
    return pa_fail(PA_ERR_INVALID, "%s: misaligned pointer", me);
  pa::QkRowsShape sh{};
  sh.q_out_stride = q_out_stride;
  sh.q_stride = q_stride;
  sh.k_stride = k_stride;
  sh.v_stride = v_stride;
  sh.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  sh.num_tokens = num_tokens;
  sh.num_heads = num_heads;
  sh.num_kv_heads = num_kv_heads;
  sh.head_dim = head_dim;
  sh.max_position = max_position;
  sh.rotary_dim = rotary_dim;
  sh.interleaved = interleaved != 0;
  sh.eps = eps;
  sh.dtype = dtype;
  cudaError_t e = pa::launch_qk_norm_rope_append(
      sh, q_out, q, k, v, positions, slot_mapping, cos_sin, q_weight, k_weight, k_cache, v_cache,
      k_scale, v_scale, reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return pa_fail(PA_ERR_UNSUPPORTED, "%s: too many rows", me);
  return e == cudaSuccess ? PA_OK : cuda_fail("pa_qk_norm_rope_append launch", e);
}

size_t pa_decode_tree_workspace_bytes(int num_heads, int num_kv_heads, int head_dim,
                                      int max_query_len) {
  if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 || head_dim <= 0 ||
      max_query_len <= 0)
    return 0;
  return pa::tree_workspace(num_heads, num_kv_heads, head_dim, max_query_len).total;
}

int pa_decode_tree(void* out, const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, const int32_t* context_lens,
                   const int32_t* query_start, const int32_t* parents, int num_seqs, int total_q,
                   int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                   int max_blocks_per_seq, int max_query_len, float scale, void* workspace,
                   size_t workspace_bytes, pa_dtype dtype, pa_stream_t stream) {
  const char* me = "pa_decode_tree";
  if (num_seqs < 0 || total_q < 0 || max_query_len < 0)
    return pa_fail(PA_ERR_INVALID, "%s: negative size", me);
  if (num_seqs == 0 || total_q == 0 || max_query_len == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start)
    return pa_fail(PA_ERR_INVALID, "%s: null pointer", me);
  if (dtype != PA_BF16) return pa_fail(PA_ERR_UNSUPPORTED, "%s: dtype %d (built: bf16)", me, dtype);
  if (head_dim != 64 && head_dim != 128)
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d (built: 64, 128)", me, head_dim);
  if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0)
    return pa_fail(PA_ERR_INVALID, "%s: num_heads %d not a multiple of num_kv_heads %d", me,
                   num_heads, num_kv_heads);
  const int group = num_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8)
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: group size %d (built: 1, 2, 4, 8)", me, group);
  if (!pow2(block_size) || block_size < 8 || block_size > 256)
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: block_size %d (built: powers of two 8..256)", me,
                   block_size);
  if (num_blocks <= 0 || max_blocks_per_seq <= 0)
    return pa_fail(PA_ERR_INVALID, "%s: num_blocks and max_blocks_per_seq must be > 0", me);
  if (max_query_len > total_q)
    return pa_fail(PA_ERR_INVALID, "%s: max_query_len %d > total_q %d", me, max_query_len, total_q);
  if (!std::isfinite(scale) || scale <= 0.0f)
    return pa_fail(PA_ERR_INVALID, "%s: scale must be finite and > 0", me);
  if (num_kv_heads > 65535) return pa_fail(PA_ERR_UNSUPPORTED, "%s: num_kv_heads > 65535", me);
  if (static_cast<int64_t>(num_blocks) * block_size * num_kv_heads * head_dim * 2 / 16 >
      (int64_t(1) << 36))
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: cache larger than 1 TiB", me);
  // the kernel counts its work (64-key tiles x KV heads x items of 128 rows) in 31 bits
  const int64_t seq_units = (static_cast<int64_t>(max_blocks_per_seq) * block_size / 64 + 8) *
                            num_kv_heads * ((static_cast<int64_t>(max_query_len) * group + 127) / 128);
  if (seq_units > 0x7fffffff / num_seqs)
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: %d tables of %lld tokens by %d rows are too large", me,
                   num_seqs, static_cast<long long>(max_blocks_per_seq) * block_size, max_query_len);
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4) ||
      !aligned(parents, 4) || !aligned(workspace, 16))
    return pa_fail(PA_ERR_INVALID, "%s: misaligned pointer", me);
  const size_t need = pa_decode_tree_workspace_bytes(num_heads, num_kv_heads, head_dim, max_query_len);
  if (!workspace || workspace_bytes < need)
    return pa_fail(PA_ERR_INVALID, "%s: workspace %zu B < %zu B needed", me,
                   workspace ? workspace_bytes : size_t(0), need);
  pa::TreeShape sh{};
  sh.num_seqs = num_seqs;
  sh.total_q = total_q;
  sh.num_heads = num_heads;
  sh.num_kv_heads = num_kv_heads;
  sh.head_dim = head_dim;
  sh.block_size = block_size;
  sh.num_blocks = num_blocks;
  sh.max_blocks_per_seq = max_blocks_per_seq;
  sh.max_query_len = max_query_len;
  sh.scale = scale;
  cudaError_t e = pa::launch_decode_tree(sh, out, q, k_cache, v_cache, block_tables, context_lens,
                                         query_start, parents, workspace,
                                         reinterpret_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return pa_fail(PA_ERR_UNSUPPORTED, "%s: no kernel for this shape", me);
  return e == cudaSuccess ? PA_OK : cuda_fail("pa_decode_tree launch", e);
}

int pa_verify_draft(int32_t* out_tokens, int32_t* out_path, int32_t* out_len,
                    const float* target_probs, int64_t target_stride, const float* draft_probs,
                    int64_t draft_stride, const int32_t* draft_tokens, const int32_t* parents,
                    const int32_t* query_start, const float* u_accept, const float* u_sample,
                    int num_seqs, int total_q, int vocab_size, int max_query_len,
                    pa_stream_t stream) {
  const char* me = "pa_verify_draft";
  if (num_seqs < 0 || total_q < 0 || max_query_len < 0)
    return pa_fail(PA_ERR_INVALID, "%s: negative size", me);
  if (num_seqs == 0) return PA_OK;
  if (max_query_len == 0 || total_q == 0)
    return pa_fail(PA_ERR_INVALID, "%s: no rows to verify (max_query_len %d, total_q %d)", me,
                   max_query_len, total_q);
  if (!out_tokens || !out_path || !out_len || !target_probs || !draft_tokens || !query_start ||
      !u_accept || !u_sample)
    return pa_fail(PA_ERR_INVALID, "%s: null pointer", me);
  if (vocab_size <= 0 || vocab_size > (1 << 24))
    return pa_fail(PA_ERR_INVALID, "%s: vocab_size %d outside [1, 2^24]", me, vocab_size);
  if (max_query_len > pa::kMaxVerifyRows)
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: max_query_len %d > %d", me, max_query_len, pa::kMaxVerifyRows);
  if (num_seqs > (1 << 24)) return pa_fail(PA_ERR_UNSUPPORTED, "%s: num_seqs > 2^24", me);
  if (total_q > 1 && (target_stride < vocab_size || (draft_probs && draft_stride < vocab_size)))
    return pa_fail(PA_ERR_INVALID, "%s: a stride is shorter than vocab_size", me);
  if (!aligned(out_tokens, 4) || !aligned(out_path, 4) || !aligned(out_len, 4) ||
      !aligned(target_probs, 4) || !aligned(draft_probs, 4) || !aligned(draft_tokens, 4) ||
      !aligned(parents, 4) || !aligned(query_start, 4) || !aligned(u_accept, 4) ||
      !aligned(u_sample, 4))
    return pa_fail(PA_ERR_INVALID, "%s: misaligned pointer", me);
  pa::VerifyShape sh{};
  sh.target_stride = target_stride;
  sh.draft_stride = draft_probs ? draft_stride : 0;
  sh.num_seqs = num_seqs;
  sh.total_rows = total_q;
  sh.vocab = vocab_size;
  sh.max_query_len = max_query_len;
  cudaError_t e = pa::launch_verify_draft(sh, out_tokens, out_path, out_len, target_probs,
                                          draft_probs, draft_tokens, parents, query_start,
                                          u_accept, u_sample, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail("pa_verify_draft launch", e);
}

int pa_kv_accept(void* k_cache, void* v_cache, const int32_t* block_tables,
                 const int32_t* context_lens, const int32_t* query_start, const int32_t* path,
                 const int32_t* path_len, int num_seqs, int max_path_len, int num_blocks,
                 int block_size, int max_blocks_per_seq, int num_kv_heads, int head_dim,
                 pa_dtype dtype, pa_stream_t stream) {
  const char* me = "pa_kv_accept";
  if (num_seqs < 0 || max_path_len < 0) return pa_fail(PA_ERR_INVALID, "%s: negative size", me);
  if (num_seqs == 0 || max_path_len == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !query_start || !path || !path_len)
    return pa_fail(PA_ERR_INVALID, "%s: null pointer", me);
  if (!known_dtype(dtype)) return pa_fail(PA_ERR_UNSUPPORTED, "%s: dtype %d", me, dtype);
  if (num_blocks <= 0 || max_blocks_per_seq <= 0 || num_kv_heads <= 0 || head_dim <= 0)
    return pa_fail(PA_ERR_INVALID, "%s: sizes must be positive", me);
  if (!pow2(block_size))
    return pa_fail(PA_ERR_INVALID, "%s: block_size %d not a power of two", me, block_size);
  const int elem = dtype == PA_F32 ? 4 : dtype == PA_BF16 ? 2 : 1;
  const int64_t row_bytes = static_cast<int64_t>(num_kv_heads) * head_dim * elem;
  if (row_bytes % 16 != 0 || row_bytes > (1 << 24))
    return pa_fail(PA_ERR_UNSUPPORTED, "%s: rows of %lld B (built: multiples of 16 up to 2^24)", me,
                   static_cast<long long>(row_bytes));
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4) || !aligned(query_start, 4) || !aligned(path, 4) ||
      !aligned(path_len, 4))
    return pa_fail(PA_ERR_INVALID, "%s: misaligned pointer", me);
  int lg = 0;
  while ((1 << lg) < block_size) ++lg;
  cudaError_t e = pa::launch_kv_accept(k_cache, v_cache, block_tables, context_lens, query_start,
                                       path, path_len, num_seqs, max_path_len, num_blocks, lg,
                                       max_blocks_per_seq, static_cast<int>(row_bytes),
                                       reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PA_OK : cuda_fail("pa_kv_accept launch", e);
}

}  // extern "C"
