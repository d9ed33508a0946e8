// kv_fp8_attention for sm_103a: varlen prefill + decode with GQA over the
// paged E4M3 cache with one power-of-two scale per (block, kv head).
//
// With key p in block b, ks_b = 2^kk, vs_b = 2^kv, codes ck_p and cv_p:
//   s_p = softmax_scale * ks_b * q . ck_p
//   out = sum_p 2^(s_p log2 e) vs_b cv_p / sum_p 2^(s_p log2 e)
// The V scale joins the exponent: with t_p = s_p log2 e + kv_b and the running
// maximum M of t, the weights w_p = 2^(t_p - M) never exceed 1, whatever the
// V scales are, so they fit f16 MMA operands without a range limit on V; the
// denominator in the same units is sum_b 2^-kv_b sum_{p in b} w_p (a block's
// sum times a power of two, fp32; blocks of small kv_b, whose weights beside large
// ones may leave fp32, have theirs summed again in larger units).  A score costs
// one FMA (scale and kv together) and one exp2.
// Weights are rounded to f16 for the product with V (denominators sum them as they
// were): off by 2^-11 of a weight at most, which sums over keys average out, beside
// 2^-8 of the bf16 output.  Against 64 bits outputs are off by as much as with fp32
// weights (0.0017 of their norm); the two differ in last bits, 9e-4 at most.
// Queries are used at full precision: the tensor-core prefill multiplies them
// as they are (bf16, K codes converted to bf16); the warp-MMA kernels divide a
// row by the power of two of its largest magnitude (bf16 to f16, exact but for
// elements 2^-14 of the largest, whose f16 spacing is 2^-24 of it) and multiply
// the fp32 score by that power.  Codes convert exactly to either type.
//
// Launches, all on the caller's stream: the schedule (one CTA), prefill (if a
// sequence may need it), decode, merge (of decode's pieces and of prefill tiles
// split over their keys).  Short batches that only decode: one launch.

#include <cuda.h>
#include <float.h>

#include <type_traits>

#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"
#include "schedule.cuh"

namespace kvint4 {
namespace {

#include "attention_fp8.cuh"

template <int D>
int launch_attention_t(const AttnArgs& a, cudaStream_t stream) {
  WorkspaceLayoutFp8 L;
  if (!workspace_layout_fp8(a.num_seqs, a.num_q_tokens, a.num_q_heads, a.num_kv_heads, a.head_size, false, &L) ||
      a.workspace_bytes < L.total)
    workspace_layout_fp8(a.num_seqs, a.num_q_tokens, a.num_q_heads, a.num_kv_heads, a.head_size, true, &L);
  const PlanView pv = plan_view_fp8(a.workspace, L);
  const int dev = current_device();
  const int sms = sm_count(dev);
  Common c{};
  c.q = static_cast<const uint16_t*>(a.q);
  c.q_stride = a.q_stride;
  c.k_cache = a.k_cache;
  c.v_cache = a.v_cache;
  c.k_scale = a.k_scale;
  c.v_scale = a.v_scale;
  c.geo = a.geo;
  c.block_table = a.block_table;
  c.max_blocks = a.max_blocks_per_seq;
  c.seq_lens = a.seq_lens;
  c.qsl = a.query_start_loc;
  c.num_seqs = a.num_seqs;
  c.num_q_tokens = a.num_q_tokens;
  c.max_qlen = a.max_query_len;
  c.hq = a.num_q_heads;
  c.hkv = a.num_kv_heads;
  c.group = a.num_q_heads / a.num_kv_heads;
  c.gdiv = FastDiv((uint32_t)c.group);
  c.num_blocks = a.num_blocks;
  c.causal = a.causal;
  c.window = a.sliding_window;
  c.qscale = a.softmax_scale * kLog2e;
  c.out = static_cast<uint16_t*>(a.out);
  c.out_stride = a.out_stride;
  c.status = a.dev_status;
  c.max_items = L.max_pairs * a.num_kv_heads;
  // f with the number of blocks per position and of column groups as constants
  auto with_np = [](int np, int cg, auto&& f) {
    using std::integral_constant;
    if (np == 2) return f(integral_constant<int, 2>{}, integral_constant<int, 1>{});
    if (np == 4) return f(integral_constant<int, kFp8Quad<D> ? 4 : 2>{}, integral_constant<int, 1>{});
    if (cg == 2) return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
    if (cg == 4) return f(integral_constant<int, 1>{}, integral_constant<int, 4>{});
    return f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  };
  // decode: blocks per position, kv heads per CTA, CTAs
  c.hg = c.ng = c.nl = c.np = 1;
  // query columns of the batch's decode sequences: paired blocks need at most
  // four, four blocks at most two, column groups take eight each up to 32 (as
  // far as the workspace holds their results).  When the batch also holds longer
  // queries decode is sized for single tokens and the others go to prefill
  const long long mq = (long long)(a.max_query_len > 0 ? a.max_query_len : 1) * c.group;
  const long long cols = mq <= kDecodeColsFp8 ? mq : c.group;
  int cg = cols > 2 * kDecodeCols ? 4 : cols > kDecodeCols ? 2 : 1;
  while (cg > 1 && (long long)a.num_seqs * a.num_kv_heads * kDecodeCols * cg > L.direct_rows) cg /= 2;
  const bool any_decode = c.group <= kDecodeCols * cg;
  int dec_grid = 0, dec_occ = 0;
  if (any_decode) {
    static PerContext<int> occ_cache[5][5];
    int& occ = dec_occ;
    auto take = [&](auto np_tag, auto cg_tag) {
      constexpr int NP = decltype(np_tag)::value, CG = decltype(cg_tag)::value;
      using G = Fp8Dec<D, NP>;
      c.np = NP;
      // the largest divisor of Hkv that gives up to four warps and whose ring
      // leaves room for two CTAs per SM
      for (int h = 4 / CG; h >= 1; h--)
        if (a.num_kv_heads % h == 0 && (h == 1 || 2 * (G::smem_bytes(h) + 1024) <= 228 * 1024)) {
          c.hg = h;
          break;
        }
      return occ_cache[NP == 1 ? CG / 2 : NP / 2 + 2][c.hg].get(dev, [&](int* v) {
        int unused;  // the attribute is raised once, to the largest ring in use
        return configure(decode_fp8_kernel<D, NP, CG, true>, (228 * 1024) / 2 - 1024, 128, &unused) &&
               configure(decode_fp8_kernel<D, NP, CG, false>, (228 * 1024) / 2 - 1024, 128, &unused) &&
               cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, decode_fp8_kernel<D, NP, CG, false>, c.hg * CG * 32,
                                                             G::smem_bytes(c.hg)) == cudaSuccess && *v >= 1;
      }, &occ);
    };
    if (!with_np(cols > 4 ? 1 : cols > 2 || !kFp8Quad<D> ? 2 : 4, cg, take)) return KV_INT4_ERR_CUDA;
    c.ng = a.num_kv_heads / c.hg;
    long long grid = (long long)sms * occ;
    if (grid * c.hg * cg > kMaxDecodeWarps) grid = kMaxDecodeWarps / (c.hg * cg);
    // lanes: as many as divide the head groups, so that the groups' slices of
    // a block's rows are read side by side
    for (int l = (int)(grid < c.ng ? grid : c.ng); l >= 1; l--)
      if (c.ng % l == 0) {
        c.nl = l;
        break;
      }
    dec_grid = (int)(grid / c.nl * c.nl);
  }
  c.dcols = kDecodeCols * cg / c.np;

  const bool may_prefill = c.group > c.dcols || (long long)a.max_query_len * c.group > c.dcols;
  if (!may_prefill) {
    // one launch of clusters where the whole batch runs at once and the shares
    // are short: the largest cluster that leaves every CTA resident, or shares
    // of two positions (1 x 97 keys: 7.4 us against 12.7; 8 x 1024: 13 against
    // 16; shares of more than 16 positions, or a second wave of CTAs, do better
    // with the balanced split)
    const long long tasks = (long long)a.num_seqs * c.ng, room = (long long)sms * dec_occ;
    const long long table = (long long)a.max_blocks_per_seq * 16;
    const long long most = ((a.max_seq_len < table ? a.max_seq_len : table) + 16 * c.np - 1) / (16 * c.np);
    int cl = 1;
    while (cl < 8 && 2 * tasks * cl <= room && most > 2 * cl) cl *= 2;
    if (tasks * cl <= room && most <= 16 * cl) {
      timing_begin(kTimedDecode, stream);
      const int e = with_np(c.np, cg, [&](auto np_tag, auto cg_tag) {
        constexpr int NP = decltype(np_tag)::value, CG = decltype(cg_tag)::value;
        return launch_pdl(decode_fp8_kernel<D, NP, CG, true>, dim3((unsigned)(tasks * cl)), c.hg * CG * 32,
                          Fp8Dec<D, NP>::smem_bytes(c.hg), stream, cl, Fp8DecParams{c, pv, 0, cl, false});
      });
      timing_end(kTimedDecode, stream);
      return e;
    }
  }

  // prefill items: 256 rows on the tensor-core kernel (128 of head size 256: two
  // accumulators would leave no TMEM for scores), 64 on the warp-MMA one, for
  // tensors without a tensor map
  // Keys are split into pieces of at least four steps of the tensor-core kernel
  // (512 keys; 256 at 192), eight of the other (256 keys), where a tile may have
  // four such pieces (looking for splits costs 1 to 3 us per call), two where the
  // query rows fill less than half of the CTAs (2 x 16 tokens against 1322 keys,
  // 64/4 heads of 192: 46 us, in pieces 38; 2 prompts of 1221 tokens, 8/4 heads of
  // 128: 37, 37), and there are fewer tiles than the schedule leaves whole anyway
  // (sequences decoded here have at most dcols / group tokens)
  const long long most_decode = any_decode ? (long long)a.num_seqs * (c.dcols / c.group) : 0;
  auto can_split = [&] {
    const long long tiles = (a.num_q_tokens - most_decode + c.tile_tokens - 1) / c.tile_tokens;
    const long long rows = (long long)a.num_q_tokens * a.num_q_heads;
    const int pieces = rows <= c.split_ctas / 2 * (long long)c.tile_tokens * c.group ? 2 : 4;
    return may_prefill && L.max_pieces > 0 && a.max_seq_len > 16ll * c.step_blocks * c.split_steps * pieces && tiles <= kSplitTiles &&
           tiles * a.num_kv_heads < (long long)kSplitWaves * c.split_ctas;
  };
  bool tc = false, may_split = false;
  const long long pairs = L.max_pairs + L.max_pieces;
  const long long most_items = pairs * a.num_kv_heads;
  {
    using G = Fp8Ws<D>;
    Fp8Maps maps;
    tc = may_prefill && make_maps<D>(a, G::ROWS / c.group, &maps);
    if (tc) {
      c.tile_tokens = G::ROWS / c.group;
      c.step_blocks = G::NB;
      c.split_steps = 4;
      c.split_ctas = sms;
      static PerContext<int> occ_c;
      int occ = 0;
      if (!occ_c.get(dev, [](int* o) { return configure_tmem(prefill_ws_fp8_kernel<D>, G::SMEM, G::THREADS, 512, o); },
                     &occ))
        return KV_INT4_ERR_CUDA;
      may_split = can_split();
      if (int e = launch_plan(c, pv, may_prefill, may_split, stream)) return e;
      const long long grid = sms < most_items ? sms : most_items;
      timing_begin(kTimedPrefill, stream);
      const int e = launch_pdl(prefill_ws_fp8_kernel<D>, dim3((unsigned)grid), G::THREADS, G::SMEM, stream, 1, c, pv, maps);
      timing_end(kTimedPrefill, stream);
      if (e) return e;
    }
  }
  if (!tc) {
    using G = Fp8Pre<D>;
    long long grid = 1;
    c.tile_tokens = kPrefillRows / c.group;
    if (may_prefill) {
      static PerContext<int> occ_c;
      int occ = 0;
      if (!occ_c.get(dev, [](int* o) { return configure(prefill_fp8_kernel<D>, G::SMEM, G::THREADS, o); }, &occ))
        return KV_INT4_ERR_CUDA;
      grid = (long long)sms * occ;
    }
    c.step_blocks = G::NB;
    c.split_steps = 8;
    c.split_ctas = (int)grid;
    may_split = can_split();
    if (int e = launch_plan(c, pv, may_prefill, may_split, stream)) return e;
    if (may_prefill) {
      if (grid > most_items) grid = most_items;
      timing_begin(kTimedPrefill, stream);
      const int e = launch_pdl(prefill_fp8_kernel<D>, dim3((unsigned)grid), G::THREADS, G::SMEM, stream, 1, c, pv);
      timing_end(kTimedPrefill, stream);
      if (e) return e;
    }
  }
  // The merge of pieces has CTAs for a warp per row, as far as they start at once
  // when the prefill's last CTAs leave
  auto merge_ctas = [&](long long segs, int warps) {
    const long long rows = (long long)a.num_q_tokens * a.num_q_heads;
    const long long want = ((rows < kPieceRows / 2 ? rows : kPieceRows / 2) + warps - 1) / warps;
    const long long more = want < sms ? want : sms;
    return may_split && more > segs ? more : segs;
  };
  if (any_decode) {
    const Fp8DecParams prm{c, pv, dec_grid, 1, may_prefill};
    timing_begin(kTimedDecode, stream);
    int e = with_np(c.np, cg, [&](auto np_tag, auto cg_tag) {
      constexpr int NP = decltype(np_tag)::value, CG = decltype(cg_tag)::value;
      return launch_pdl(decode_fp8_kernel<D, NP, CG, false>, dim3(dec_grid), c.hg * CG * 32,
                        Fp8Dec<D, NP>::smem_bytes(c.hg), stream, 1, prm);
    });
    timing_end(kTimedDecode, stream);
    if (e) return e;
    // merge: one or more CTAs per (sequence, kv head) segment, a warp per query
    // column and piece lane; lanes enough that each merges one or two pieces (1 to
    // 3 tokens of 7 heads against up to 9611 keys of one kv head, 2 sequences:
    // 201 us with the 21 columns in one CTA and so one lane each, 24 spread out),
    // as far as all CTAs start at once (more: 55 us instead of 46 for 32 x 1
    // token of group 16, 4 kv heads)
    const long long mcols = (long long)(a.max_query_len > 0 ? a.max_query_len : 1) * c.group;
    const long long segs = (long long)a.num_seqs * a.num_kv_heads;
    const long long pieces = 1 + (long long)dec_grid * c.hg / (segs > 0 ? segs : 1);
    constexpr int kWarps = 32;  // per CTA, and per SM over all CTAs
    int lanes = 1;
    int cols = (int)(mcols < c.dcols ? mcols : c.dcols), parts = 1;
    while (lanes < kWarps && lanes < pieces &&
           (2 * lanes * cols <= kWarps || 2 * lanes * cols * segs <= (long long)kWarps * sms))
      lanes *= 2;
    if (cols * lanes > kWarps) {
      parts = (cols * lanes + kWarps - 1) / kWarps;
      cols = (cols + parts - 1) / parts;
    }
    if (segs * parts > 0x7fffffff) return KV_INT4_ERR_SIZE;
    timing_begin(kTimedReduce, stream);
    e = launch_pdl(may_split ? merge_fp8_kernel<D, true> : merge_fp8_kernel<D, false>,
                   dim3((unsigned)merge_ctas(segs * parts, cols * lanes)), cols * lanes * 32,
                   merge_smem<D>(cols, lanes), stream, 1, Fp8MergeParams{c, pv, dec_grid, cols, lanes, parts, kDecodeCols * cg});
    timing_end(kTimedReduce, stream);
    if (e) return e;
  } else if (may_split) {
    timing_begin(kTimedReduce, stream);
    const int e = launch_pdl(merge_fp8_kernel<D, true>, dim3((unsigned)merge_ctas(1, 8)), 256, 0, stream, 1,
                             Fp8MergeParams{c, pv, 0, 8, 1, 1, kDecodeCols});
    timing_end(kTimedReduce, stream);
    if (e) return e;
  }
  return KV_INT4_OK;
}

}  // namespace

int launch_attention_fp8(const AttnArgs& a, cudaStream_t stream) {
  switch (a.head_size) {
    case 64: return launch_attention_t<64>(a, stream);
    case 96: return launch_attention_t<96>(a, stream);
    case 128: return launch_attention_t<128>(a, stream);
    case 192: return launch_attention_t<192>(a, stream);
    case 256: return launch_attention_t<256>(a, stream);
    default: return KV_INT4_ERR_HEAD_SIZE;
  }
}

}  // namespace kvint4
