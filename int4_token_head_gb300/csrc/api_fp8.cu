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

}  // namespace

bool kvint4::shared_layout(int num_seqs, int num_groups, int num_q_tokens, int num_q_heads, int num_kv_heads,
                           int head_size, SharedLayout* L) {
  if (num_seqs < 0 || num_groups < 0 || num_groups > kMostGroups || num_q_tokens < 0 || num_q_tokens >= (1 << 30) ||
      num_seqs > INT32_MAX - num_groups)
    return false;
  const size_t V = (size_t)num_seqs + num_groups;
  // groups' query tokens once more.  The base's own room for decode columns goes by
  // one sequence's, a group's are more: up to 32 per virtual sequence and head here,
  // and they fill more warps' slots than one token's
  const int64_t columns = (int64_t)V * num_kv_heads * kDecodeColsFp8;
  if (!workspace_layout_fp8((int)V, 2 * num_q_tokens, num_q_heads, num_kv_heads, head_size, false, &L->base,
                            num_groups > 0 ? kSharedDecodeWarps : kMaxDecodeWarps,
                            num_groups > 0 && columns <= kSharedRows ? columns : 0))
    return false;
  size_t off = L->base.total;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return at;
  };
  L->vrec = take(V * 32);
  L->dseq2 = take(V * 16);
  L->vinfo = take(V * 8);
  L->tloc = take(L->base.max_pairs * 8);
  const int64_t most = kSharedRows / num_q_heads;
  L->row_tokens = num_groups == 0 ? 0 : (int)(num_q_tokens < most ? num_q_tokens : most);
  const size_t rows = 2 * (size_t)L->row_tokens * num_q_heads;
  L->row_o = take(rows * head_size * 4);
  L->row_ml = take(rows * 2 * 4);
  L->total = off;
  return true;
}

namespace {

// whether rows of len floats at (sequence, head) strides do not overlap
bool rows_apart(int64_t seqs, int64_t seq_stride, int64_t heads, int64_t head_stride, int64_t len) {
  if (seqs <= 1) return heads <= 1 || head_stride >= len;
  if (heads <= 1) return seq_stride >= len;
  const bool by_seq = seq_stride >= head_stride;  // the outer index
  const int64_t outer = by_seq ? seq_stride : head_stride, inner = by_seq ? head_stride : seq_stride;
  return inner >= len && outer >= len && (outer - len) / ((by_seq ? heads : seqs) - 1) >= inner;
}

// the longest sequence that the kernels' loops over positions go through in 32 bits (a
// step of a few thousand positions beyond the end included)
constexpr int64_t kMostPositions = (1ll << 31) - (1 << 16);

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

// both rotary entry points: validation, then the launch
int do_norm_rope(const NormRopeArgs& a, void* stream) {
  if (a.num_tokens < 0 || a.max_position < 0 || !(a.eps >= 0.f)) return KV_INT4_ERR_SIZE;
  if (a.num_q_heads <= 0 || a.num_kv_heads <= 0) return KV_INT4_ERR_HEADS;
  if (!head_size_ok(a.head_size)) return KV_INT4_ERR_HEAD_SIZE;
  if (a.rot_dim < 0 || a.rot_dim > a.head_size || a.rot_dim % 16) return KV_INT4_ERR_ROT;
  if ((int64_t)a.num_tokens * ((int64_t)a.num_q_heads + a.num_kv_heads) >= (1ll << 31)) return KV_INT4_ERR_SIZE;
  if (a.num_tokens == 0) return KV_INT4_OK;
  if (!a.q || !a.k || !a.q_out || !a.k_out || !a.q_weight != !a.k_weight ||
      (a.rot_dim > 0 && (!a.positions || !a.cos_sin)))
    return KV_INT4_ERR_NULL;
  if (!aligned16(a.q) || !aligned16(a.k) || !aligned16(a.q_out) || !aligned16(a.k_out) || !aligned16(a.q_weight) ||
      !aligned16(a.k_weight) || !stride_ok(a.q_stride) || !stride_ok(a.k_stride) || !stride_ok(a.q_out_stride) ||
      !stride_ok(a.k_out_stride) || !aligned(a.dev_status, 4) ||
      (a.rot_dim > 0 && (!aligned(a.positions, 8) || !aligned16(a.cos_sin))))
    return KV_INT4_ERR_ALIGN;
  if (current_device() < 0) return KV_INT4_ERR_CUDA;
  return launch_norm_rope(a, static_cast<cudaStream_t>(stream));
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
  return do_norm_rope(NormRopeArgs{q, q_token_stride, k, k_token_stride, num_tokens, num_q_heads, num_kv_heads,
                                   head_size, q_weight, k_weight, eps, positions, cos_sin, max_position, rot_dim,
                                   interleaved != 0, q_out, q_out_token_stride, k_out, k_out_token_stride,
                                   dev_status, 0, 0, {}},
                      stream);
}

int kv_qk_norm_rope_axes(const void* q, int64_t q_token_stride, const void* k, int64_t k_token_stride, int num_tokens,
                         int num_q_heads, int num_kv_heads, int head_size, const void* q_weight,
                         const void* k_weight, float eps, const int64_t* positions, int64_t position_axis_stride,
                         int num_axes, const uint8_t* pair_axis, const float* cos_sin, int64_t max_position,
                         int rot_dim, int interleaved, void* q_out, int64_t q_out_token_stride, void* k_out,
                         int64_t k_out_token_stride, int32_t* dev_status, void* stream) {
  NormRopeArgs a{q, q_token_stride, k, k_token_stride, num_tokens, num_q_heads, num_kv_heads,
                 head_size, q_weight, k_weight, eps, positions, cos_sin, max_position, rot_dim,
                 interleaved != 0, q_out, q_out_token_stride, k_out, k_out_token_stride,
                 dev_status, num_axes, position_axis_stride, {}};
  if (num_axes < 1 || num_axes > kMaxAxes || rot_dim < 0 || rot_dim > 256) return KV_INT4_ERR_ROT;
  if (position_axis_stride < 0) return KV_INT4_ERR_SIZE;
  if (rot_dim > 0 && num_tokens > 0) {
    if (!pair_axis) return KV_INT4_ERR_NULL;
    for (int i = 0; i < rot_dim / 2; i++) {
      if (pair_axis[i] >= num_axes) return KV_INT4_ERR_ROT;
      a.pair_axis[i / 16] |= (uint32_t)pair_axis[i] << (2 * (i % 16));
    }
  }
  return do_norm_rope(a, stream);
}

size_t kv_fp8_attention_shared_workspace_size(int num_seqs, int num_groups, int num_q_tokens, int num_q_heads,
                                              int num_kv_heads, int head_size) {
  SharedLayout L;
  if (!head_size_ok(head_size) || num_q_heads <= 0 || num_kv_heads <= 0 ||
      !shared_layout(num_seqs, num_groups, num_q_tokens, num_q_heads, num_kv_heads, head_size, &L))
    return 0;
  return L.total;
}

int kv_fp8_attention_shared(const void* q, int64_t q_token_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                            const float* k_scale_cache, const float* v_scale_cache, const int32_t* block_table,
                            int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* query_start_loc, int num_seqs,
                            int num_q_tokens, int max_query_len, int max_seq_len, const int32_t* group_start,
                            const int32_t* prefix_lens, int num_groups, int max_group_tokens, int num_q_heads,
                            int num_kv_heads, int head_size, int block_size, int num_blocks, float softmax_scale, void* out,
                            int64_t out_token_stride, float* lse, int64_t lse_token_stride, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, void* stream) {
  if (max_seq_len < 0 || num_groups < 0 || num_groups > kMostGroups || max_group_tokens < 0) return KV_INT4_ERR_SIZE;
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > kPrefillRows)
    return KV_INT4_ERR_HEADS;
  int e = check_sizes(num_seqs, num_q_tokens, max_query_len, max_blocks_per_seq, num_blocks, block_size, num_kv_heads,
                      head_size);
  if (e != KV_INT4_OK) return e;
  SharedLayout L;
  if ((int64_t)num_q_tokens * num_q_heads >= (1ll << 31) ||
      !shared_layout(num_seqs, num_groups, num_q_tokens, num_q_heads, num_kv_heads, head_size, &L))
    return KV_INT4_ERR_SIZE;
  if (num_seqs == 0 || num_q_tokens == 0) return KV_INT4_OK;
  // query rows that do not overlap, blocks that a tensor map holds
  const int64_t row = (int64_t)num_q_heads * head_size;
  if (num_blocks < 1 || (int64_t)num_blocks * 16 >= (1ll << 31) ||
      (num_q_tokens > 1 && (q_token_stride < row || out_token_stride < row || (lse && lse_token_stride < num_q_heads))))
    return KV_INT4_ERR_SIZE;
  if (!workspace || workspace_bytes < L.total) return KV_INT4_ERR_WORKSPACE;
  if (!q || !out || (num_groups > 0 && (!group_start || !prefix_lens))) return KV_INT4_ERR_NULL;
  e = check_cache(k_cache, v_cache, k_scale_cache, v_scale_cache, block_table, seq_lens, query_start_loc, dev_status);
  if (e != KV_INT4_OK) return e;
  if (!aligned16(q) || !aligned16(out) || !stride_ok(q_token_stride) || !stride_ok(out_token_stride) ||
      !aligned(workspace, 256) || !aligned(group_start, 4) || !aligned(prefix_lens, 4) || !aligned(lse, 4))
    return KV_INT4_ERR_ALIGN;
  if (current_device() < 0) return KV_INT4_ERR_CUDA;
  const AttnArgs a{q, q_token_stride, k_cache, v_cache, k_scale_cache, v_scale_cache, block_table, max_blocks_per_seq,
                   seq_lens, query_start_loc, num_seqs, num_q_tokens, max_query_len, max_seq_len, num_q_heads,
                   num_kv_heads, head_size, block_size, num_blocks, softmax_scale, 1, 0, nullptr, out,
                   out_token_stride, workspace, workspace_bytes, dev_status, false,
                   block_scale_geo(num_kv_heads, head_size)};
  return launch_attention_shared_fp8(SharedAttnArgs{a, group_start, prefix_lens, num_groups, max_group_tokens, lse,
                                                    lse_token_stride},
                                     static_cast<cudaStream_t>(stream));
}

int kv_fp8_attention_mass(const void* q, int64_t q_token_stride, const float* lse, int64_t lse_token_stride,
                          const uint8_t* k_cache, const float* k_scale_cache, const int32_t* block_table,
                          int max_blocks_per_seq, const int32_t* seq_lens, const int32_t* query_start_loc, int num_seqs,
                          int num_q_tokens, int max_query_len, int max_seq_len, int num_q_heads, int num_kv_heads,
                          int head_size, int block_size, int num_blocks, float softmax_scale, float* mass,
                          int64_t mass_seq_stride, int64_t mass_head_stride, int mass_len, int32_t* dev_status,
                          void* stream) {
  if (max_seq_len < 0 || mass_len < 0 || lse_token_stride < 0 || mass_seq_stride < 0 || mass_head_stride < 0)
    return KV_INT4_ERR_SIZE;
  if (num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads || num_q_heads / num_kv_heads > kPrefillRows)
    return KV_INT4_ERR_HEADS;
  int e = check_sizes(num_seqs, num_q_tokens, max_query_len, max_blocks_per_seq, num_blocks, block_size, num_kv_heads,
                      head_size);
  if (e != KV_INT4_OK) return e;
  if ((int64_t)num_q_tokens * num_q_heads >= (1ll << 31) ||
      (max_seq_len > kMostPositions && mass_len > kMostPositions && (int64_t)max_blocks_per_seq * 16 > kMostPositions))
    return KV_INT4_ERR_SIZE;
  if (num_seqs == 0 || num_q_tokens == 0) return KV_INT4_OK;
  if (!q || !lse || !mass) return KV_INT4_ERR_NULL;
  e = check_cache(k_cache, k_cache, k_scale_cache, k_scale_cache, block_table, seq_lens, query_start_loc, dev_status);
  if (e != KV_INT4_OK) return e;
  if (!aligned16(q) || !stride_ok(q_token_stride) || !aligned(lse, 4) || !aligned(mass, 4)) return KV_INT4_ERR_ALIGN;
  if (!rows_apart(num_seqs, mass_seq_stride, num_kv_heads, mass_head_stride, mass_len)) return KV_INT4_ERR_SIZE;
  if (current_device() < 0) return KV_INT4_ERR_CUDA;
  return launch_mass_fp8(MassArgs{q, q_token_stride, lse, lse_token_stride, k_cache, k_scale_cache, block_table,
                                  max_blocks_per_seq, seq_lens, query_start_loc, num_seqs, num_q_tokens, max_query_len,
                                  max_seq_len, num_q_heads, num_kv_heads, head_size, num_blocks, softmax_scale, mass,
                                  mass_seq_stride, mass_head_stride, mass_len, dev_status},
                         static_cast<cudaStream_t>(stream));
}

int kv_fp8_evict(uint8_t* k_cache, uint8_t* v_cache, float* k_scale_cache, float* v_scale_cache, int num_blocks,
                 int block_size, int num_kv_heads, int head_size, const float* mass, int64_t mass_seq_stride,
                 int64_t mass_head_stride, int mass_len, const int32_t* block_table, int max_blocks_per_seq,
                 const int32_t* seq_lens, int num_seqs, int budget, int recent, const int32_t* dst_block_table,
                 int dst_max_blocks_per_seq, float* mass_out, int64_t mass_out_seq_stride, int64_t mass_out_head_stride,
                 int32_t* new_lens, int32_t* kept, int32_t* dev_status, void* stream) {
  if (budget < 1 || recent < 0 || recent > budget || mass_len < 0 || dst_max_blocks_per_seq < 0 ||
      mass_seq_stride < 0 || mass_head_stride < 0 || mass_out_seq_stride < 0 || mass_out_head_stride < 0)
    return KV_INT4_ERR_SIZE;
  int e = check_sizes(num_seqs, 0, 0, max_blocks_per_seq, num_blocks, block_size, num_kv_heads, head_size);
  if (e != KV_INT4_OK) return e;
  // the longest sequence that is worked on, and what is kept of it
  const int64_t table = (int64_t)max_blocks_per_seq * 16, most = table < mass_len ? table : mass_len;
  if (most > kMostPositions || (int64_t)dst_max_blocks_per_seq * 16 < (most < budget ? most : budget) ||
      (int64_t)num_seqs * num_kv_heads >= (1ll << 26))
    return KV_INT4_ERR_SIZE;
  if (num_seqs == 0) return KV_INT4_OK;
  if (!mass || !mass_out || !new_lens || !kept || !dst_block_table) return KV_INT4_ERR_NULL;
  e = check_cache(k_cache, v_cache, k_scale_cache, v_scale_cache, block_table, seq_lens, new_lens, dev_status);
  if (e != KV_INT4_OK) return e;
  if (!aligned(mass, 4) || !aligned(mass_out, 4) || !aligned(kept, 4) || !aligned(dst_block_table, 4))
    return KV_INT4_ERR_ALIGN;
  // in place only row by row
  if (mass_out == mass && ((num_seqs > 1 && mass_out_seq_stride != mass_seq_stride) ||
                           (num_kv_heads > 1 && mass_out_head_stride != mass_head_stride)))
    return KV_INT4_ERR_SIZE;
  if (new_lens == seq_lens || !rows_apart(num_seqs, mass_out_seq_stride, num_kv_heads, mass_out_head_stride,
                                          most < budget ? most : budget))
    return KV_INT4_ERR_SIZE;
  if (current_device() < 0) return KV_INT4_ERR_CUDA;
  return launch_evict_fp8(EvictArgs{k_cache, v_cache, k_scale_cache, v_scale_cache, num_blocks, num_kv_heads, head_size,
                                    mass, mass_seq_stride, mass_head_stride, mass_len, block_table, max_blocks_per_seq,
                                    seq_lens, num_seqs, budget, recent, dst_block_table, dst_max_blocks_per_seq,
                                    mass_out, mass_out_seq_stride, mass_out_head_stride, new_lens, kept, dev_status},
                          static_cast<cudaStream_t>(stream));
}

}  // extern "C"
