// C ABI entry points of the FP8 block-scaled cache and of kv_qk_norm_rope:
// host-side validation, then the launchers.

#include <cuda_runtime.h>

#include "../../include/kvint4.h"
#include "internal.h"

using namespace kvint4;

namespace {

// sizes of a call over a batch of sequences; KV_INT4_OK or the first error
int check_sizes(int num_seqs, int num_tokens, int max_len, int max_blocks_per_seq, int num_blocks, int block_size,
                int num_kv_heads, int head_size) {
  if (num_seqs < 0 || num_tokens < 0 || max_len < 0 || max_blocks_per_seq < 0 || num_blocks < 0)
    return KV_INT4_ERR_SIZE;
  if (num_kv_heads <= 0) return KV_INT4_ERR_HEADS;
  if (!head_size_ok(head_size)) return KV_INT4_ERR_HEAD_SIZE;
  if (block_size != 16) return KV_INT4_ERR_BLOCK_SIZE;
  if ((int64_t)max_blocks_per_seq * 16 >= (1ll << 31) || (int64_t)num_tokens * 2 * num_kv_heads >= (1ll << 31) ||
      (int64_t)num_blocks * 16 * num_kv_heads >= (1ll << 54))
    return KV_INT4_ERR_SIZE;
  return KV_INT4_OK;
}

int check_cache(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                const int32_t* block_table, const int32_t* seq_lens, const int32_t* start_loc,
                const int32_t* dev_status) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seq_lens || !start_loc) return KV_INT4_ERR_NULL;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(start_loc, 4) || !aligned(dev_status, 4))
    return KV_INT4_ERR_ALIGN;
  return KV_INT4_OK;
}

int do_cache(const CacheFp8Args& a, int block_size, bool write, void* stream) {
  int e = check_sizes(a.num_seqs, a.num_tokens, a.max_len, a.max_blocks_per_seq, a.num_blocks, block_size,
                      a.num_kv_heads, a.head_size);
  if (e != KV_INT4_OK) return e;
  if (a.num_seqs == 0 || a.num_tokens == 0) return KV_INT4_OK;
  if (!a.k || !a.v) return KV_INT4_ERR_NULL;
  e = check_cache(a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.block_table, a.seq_lens, a.start_loc, a.dev_status);
  if (e != KV_INT4_OK) return e;
  if (!aligned16(a.k) || !aligned16(a.v) || !stride_ok(a.k_stride) || !stride_ok(a.v_stride)) return KV_INT4_ERR_ALIGN;
  if (current_device() < 0) return KV_INT4_ERR_CUDA;
  return write ? launch_write_fp8(a, static_cast<cudaStream_t>(stream))
               : launch_read_fp8(a, static_cast<cudaStream_t>(stream));
}

}  // namespace

extern "C" {

int kv_fp8_write(const void* k, int64_t k_token_stride, const void* v, int64_t v_token_stride,
                 const int32_t* block_table, int max_blocks_per_seq, const int32_t* seq_lens,
                 const int32_t* start_loc, int num_seqs, int num_tokens, int max_len, uint8_t* k_cache,
                 uint8_t* v_cache, float* k_scale_cache, float* v_scale_cache, int num_blocks, int block_size,
                 int num_kv_heads, int head_size, int32_t* dev_status, void* stream) {
  return do_cache(CacheFp8Args{const_cast<void*>(k), k_token_stride, const_cast<void*>(v), v_token_stride, block_table,
                               max_blocks_per_seq, seq_lens, start_loc, num_seqs, num_tokens, max_len, k_cache,
                               v_cache, k_scale_cache, v_scale_cache, num_blocks, num_kv_heads, head_size, dev_status},
                  block_size, true, stream);
}

int kv_fp8_read(const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale_cache,
                const float* v_scale_cache, const int32_t* block_table, int max_blocks_per_seq,
                const int32_t* seq_lens, const int32_t* start_loc, int num_seqs, int num_tokens, int max_len, void* k,
                int64_t k_token_stride, void* v, int64_t v_token_stride, int num_blocks, int block_size,
                int num_kv_heads, int head_size, int32_t* dev_status, void* stream) {
  return do_cache(CacheFp8Args{k, k_token_stride, v, v_token_stride, block_table, max_blocks_per_seq, seq_lens,
                               start_loc, num_seqs, num_tokens, max_len, const_cast<uint8_t*>(k_cache),
                               const_cast<uint8_t*>(v_cache), const_cast<float*>(k_scale_cache),
                               const_cast<float*>(v_scale_cache), num_blocks, num_kv_heads, head_size, dev_status},
                  block_size, false, stream);
}

size_t kv_fp8_attention_workspace_size(int num_seqs, int num_q_tokens, int num_q_heads, int num_kv_heads,
                                       int head_size) {
  WorkspaceLayoutFp8 L;
  if (!head_size_ok(head_size) ||
      !workspace_layout_fp8(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_size, false, &L))
    return 0;
  return L.total;
}

int kv_fp8_attention(const void* q, int64_t q_token_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                     const float* k_scale_cache, const float* v_scale_cache, const int32_t* block_table,
                     int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* query_start_loc, int num_seqs,
                     int num_q_tokens, int max_query_len, int max_seq_len, int num_q_heads, int num_kv_heads,
                     int head_size, int block_size, int num_blocks, float softmax_scale, int causal,
                     int sliding_window, void* out, int64_t out_token_stride, void* workspace,
                     size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (max_seq_len < 0 || sliding_window < 0) return KV_INT4_ERR_SIZE;
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > kPrefillRows)
    return KV_INT4_ERR_HEADS;
  int e = check_sizes(num_seqs, num_q_tokens, max_query_len, max_blocks_per_seq, num_blocks, block_size, num_kv_heads,
                      head_size);
  if (e != KV_INT4_OK) return e;
  if ((int64_t)num_q_tokens * num_q_heads >= (1ll << 31)) return KV_INT4_ERR_SIZE;
  if (num_seqs == 0 || num_q_tokens == 0) return KV_INT4_OK;
  if (!workspace) return KV_INT4_ERR_WORKSPACE;
  if (!q || !out) return KV_INT4_ERR_NULL;
  e = check_cache(k_cache, v_cache, k_scale_cache, v_scale_cache, block_table, seq_lens, query_start_loc, dev_status);
  if (e != KV_INT4_OK) return e;
  if (!aligned16(q) || !aligned16(out) || !stride_ok(q_token_stride) || !stride_ok(out_token_stride) ||
      !aligned(workspace, 256))
    return KV_INT4_ERR_ALIGN;
  WorkspaceLayoutFp8 L;
  if (!workspace_layout_fp8(num_seqs, num_q_tokens, num_q_heads, num_kv_heads, head_size, true, &L))
    return KV_INT4_ERR_SIZE;
  if (workspace_bytes < L.total) return KV_INT4_ERR_WORKSPACE;
  if (current_device() < 0) return KV_INT4_ERR_CUDA;
  AttnArgs a{q, q_token_stride, k_cache, v_cache, k_scale_cache, v_scale_cache, block_table, max_blocks_per_seq,
             seq_lens, query_start_loc, num_seqs, num_q_tokens, max_query_len, max_seq_len, num_q_heads,
             num_kv_heads, head_size, block_size, num_blocks, softmax_scale, causal, sliding_window, nullptr, out,
             out_token_stride, workspace, workspace_bytes, dev_status, false,
             block_scale_geo(num_kv_heads, head_size)};
  return launch_attention_fp8(a, static_cast<cudaStream_t>(stream));
}

int kv_qk_norm_rope(const void* q, int64_t q_token_stride, const void* k, int64_t k_token_stride, int num_tokens,
                    int num_q_heads, int num_kv_heads, int head_size, const void* q_weight, const void* k_weight,
                    float eps, const int64_t* positions, const float* cos_sin, int64_t max_position, int rot_dim,
                    int interleaved, void* q_out, int64_t q_out_token_stride, void* k_out,
                    int64_t k_out_token_stride, int32_t* dev_status, void* stream) {
  if (num_tokens < 0 || max_position < 0 || !(eps >= 0.f)) return KV_INT4_ERR_SIZE;
  if (num_q_heads <= 0 || num_kv_heads <= 0) return KV_INT4_ERR_HEADS;
  if (!head_size_ok(head_size)) return KV_INT4_ERR_HEAD_SIZE;
  if (rot_dim < 0 || rot_dim > head_size || rot_dim % 16) return KV_INT4_ERR_ROT;
  if ((int64_t)num_tokens * ((int64_t)num_q_heads + num_kv_heads) >= (1ll << 31)) return KV_INT4_ERR_SIZE;
  if (num_tokens == 0) return KV_INT4_OK;
  if (!q || !k || !q_out || !k_out || !q_weight != !k_weight || (rot_dim > 0 && (!positions || !cos_sin)))
    return KV_INT4_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(q_weight) ||
      !aligned16(k_weight) || !stride_ok(q_token_stride) || !stride_ok(k_token_stride) ||
      !stride_ok(q_out_token_stride) || !stride_ok(k_out_token_stride) || !aligned(dev_status, 4) ||
      (rot_dim > 0 && (!aligned(positions, 8) || !aligned16(cos_sin))))
    return KV_INT4_ERR_ALIGN;
  if (current_device() < 0) return KV_INT4_ERR_CUDA;
  return launch_norm_rope(NormRopeArgs{q, q_token_stride, k, k_token_stride, num_tokens, num_q_heads, num_kv_heads,
                                       head_size, q_weight, k_weight, eps, positions, cos_sin, max_position, rot_dim,
                                       interleaved != 0, q_out, q_out_token_stride, k_out, k_out_token_stride,
                                       dev_status},
                          static_cast<cudaStream_t>(stream));
}

}  // extern "C"
