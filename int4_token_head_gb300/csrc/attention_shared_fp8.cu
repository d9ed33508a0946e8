// kv_fp8_attention_shared: causal attention over the FP8 cache for batches whose
// groups of sequences share their first positions, and the rows' log-sum-exp.
//
// All queries of a group see all of its shared keys, so the shared part is
// attention without a mask of one sequence with the group's queries: the cache's
// bytes are read once per group, and where the group's rows fill a tensor-core tile
// its keys are converted once for all of them.  What a sequence has behind the
// shared part is attended as ever.  The two are one batch of virtual sequences
// (schedule.cuh) for the kernels of kv_fp8_attention, so that long prefixes and
// short ends are balanced in one launch each, and a row's results are merged by
//   M = max m_i,  l = sum l_i 2^(m_i - M),  out = sum o_i 2^(m_i - M) / l,
//   lse = (M + log2 l) log 2
// over the pieces of both.
//
// Launches: the schedule, prefill (if any rows may need it), decode, merge; short
// batches that only decode: one launch that shares nothing (and reports groups that
// do not ascend, as the schedule does).
//
// A group's rows stay on the decode kernel up to 32 columns per kv head, above that
// they are tensor-core tiles (2 groups over 16384 positions, 8 heads of 128: 16
// columns 42 us on decode and 65 in tiles, 32 columns 61 to 64 and 66 to 70).
// Measured: 64 sequences over one prefix of 8192 positions, 32/8 heads of 128, 59 us
// (schedule 9, tiles 20 with decode on the SMs that they leave and behind them, merge
// 9; every sequence on its own reads 30 times the bytes); 4 x 8 sequences over 32768
// positions 135 (2.3 TB/s of codes, issue and latency of the conversion at two warps
// per scheduler); 16 questions to 16384 positions, 16/4 heads of 192, 103 (a step of
// 64 keys takes 3300 cycles for 1900 of tensor work).

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

constexpr int kMergeWarps = 16;  // per CTA, and about per SM over all CTAs

struct SharedMergeParams {
  Common c;
  PlanView pv;
  int num_ctas;  // of the decode launch
  int cols;      // rows per CTA (warps)
  int lanes;     // warps per row
  int parts;     // CTAs per (sequence, kv head), cols rows each and in turn
  int slot;      // columns of a result slot
  bool prefill;  // whether there was a prefill launch
};

// The results of a virtual sequence for one kv head: pieces of the decode launch,
// of split prefill tiles, or whole tiles' rows
struct Results {
  int kind;         // 0 nothing, 1 decode, 2 prefill
  int index;        // in dseq; first tile
  int ql, first;    // query tokens, first row-buffer token (-1: whole tiles went out by themselves)
  // decode: the direct slot (the piece that starts the segment), then every CTA whose
  // range is not empty and starts strictly inside it; candidates are those CTAs or
  // the positions, whichever are fewer (as merge_fp8_kernel finds them)
  long long seg, sbeg, Tu, w_first;
  int cand, W, lane_g, hl;
  bool by_cta;

  __device__ void find(const Common& c, const PlanView& pv, int num_ctas, int2 info, int4 rec, int4 rec2, int n_dseq,
                       int n_items, int h) {
    kind = info.x == 2 && n_items == 0 ? 0 : info.x;  // more tiles than the workspace holds: none was worked on
    index = info.y;
    ql = rec.y;
    first = rec2.z;
    cand = 0;
    if (kind != 1) return;
    const long long all = pv.dprefix[n_dseq], mine = pv.dprefix[index];
    const int npos = ((rec.z + 15) / 16 + c.np - 1) / c.np;
    const int grp = h / c.hg, gpl = c.ng / c.nl, gs = grp / c.nl;
    hl = h - grp * c.hg;
    lane_g = grp % c.nl;
    seg = (long long)index * c.hkv + h;
    Tu = all * gpl;
    sbeg = mine * gpl + (long long)gs * npos;
    W = num_ctas / c.nl;
    w_first = div_nn((sbeg + 1) * W + Tu - 1, Tu);
    const long long w_end = div_nn((sbeg + npos) * W + Tu - 1, Tu);
    by_cta = w_end - w_first <= npos - 1;
    cand = 1 + (int)(by_cta ? w_end - w_first : (long long)npos - 1);
  }
  // its tile that holds token j, and the pieces of a row of that token
  __device__ __forceinline__ int pieces(const Common& c, const PlanView& pv, int j, int2* tile) const {
    if (kind == 1) return cand;
    if (kind != 2) return 0;
    *tile = pv.tloc[index + j / c.tile_tokens];
    return tile->y > 1 || first >= 0 ? tile->y : 0;
  }
  // piece k of token j's row jj (q head of the group): its values and (maximum, sum); null for none
  __device__ __forceinline__ const float* piece(const Common& c, const PlanView& pv, int D, int slot, int2 tile, int h, int j,
                                                int jj, int k, int sub, const float** ml) const {
    const float *o, *m;
    long long at;
    if (kind == 1) {
      o = k == 0 ? pv.direct_o : pv.warp_o;
      m = k == 0 ? pv.direct_ml : pv.warp_ml;
      at = seg;
      if (k > 0) {
        long long w;
        if (by_cta) {
          w = w_first + k - 1;
          if (div_nn(Tu * (w + 1), W) <= div_nn(Tu * w, W)) return nullptr;
        } else {
          const long long p = sbeg + k;
          w = div_nn((p + 1) * W + Tu - 1, Tu) - 1;  // last CTA starting at or before p
          if (div_nn(Tu * w, W) != p) return nullptr;
        }
        at = (w * c.nl + lane_g) * c.hg + hl;
      }
      at = at * slot + j * c.group + jj + sub * c.dcols;
    } else if (tile.y > 1) {
      const int tok = j / c.tile_tokens * c.tile_tokens, R = min(c.tile_tokens, ql - tok) * c.group;
      at = tile.x + ((long long)h * tile.y + k) * R + (j - tok) * c.group + jj;
      o = pv.piece_o;
      m = pv.piece_ml;
    } else {
      at = (long long)(first + j) * c.hq + h * c.group + jj;
      o = pv.row_o;
      m = pv.row_ml;
    }
    *ml = m + 2 * at;
    return o + at * D;
  }
};

// A row's pieces: a lane finds one and loads its maximum and sum, the warp knows the
// row's maximum and every weight then, and the values are added in the pieces'
// order with several loads under way (a piece at a time, each waiting for its own
// weight, took 16 us instead of the 5 for 64 sequences over one prefix).
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) merge_shared_kernel(SharedMergeParams prm) {
  const Common& c = prm.c;
  const PlanView& pv = prm.pv;
  extern __shared__ __align__(16) float spart[];  // [cols][lanes][D + 2]
  pdl_trigger();
  pdl_wait();
  constexpr int PER = D / 32, VEC = D % 128 == 0 ? 4 : D % 64 == 0 ? 2 : 1;  // values a lane has side by side
  auto element = [](int lane, int e) { return (lane + 32 * (e / VEC)) * VEC + e % VEC; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pl = warp / prm.cols, lcol = warp - pl * prm.cols;
  const int seg = blockIdx.x / prm.parts, part = blockIdx.x - seg * prm.parts;
  const int s = seg / c.hkv, h = seg - s * c.hkv, v = c.sh.num_groups + s;
  const int4 rec = pv.vrec[2 * v], rec2 = pv.vrec[2 * v + 1];
  const int2 info = pv.vinfo[v];
  const int n_dseq = pv.plan[0], n_items = prm.prefill ? pv.plan[1] : 0;
  const int g = rec2.w, q0 = rec.x, ql = rec.y;
  if (ql == 0) return;
  Results own, pre;
  pre.kind = 0;
  int off = 0;  // the sequence's first token in its group
  if (g >= 0) {
    const int4 grec = pv.vrec[2 * g], grec2 = pv.vrec[2 * g + 1];
    pre.find(c, pv, prm.num_ctas, pv.vinfo[g], grec, grec2, n_dseq, n_items, h);
    off = q0 - grec.x;
  }
  own.find(c, pv, prm.num_ctas, info, rec, rec2, n_dseq, n_items, h);
  // paired blocks: columns col and col + dcols of a decode piece hold the same query
  const int own_subs = own.kind == 1 && c.np == 2 ? 2 : 1, pre_subs = pre.kind == 1 && c.np == 2 ? 2 : 1;
#pragma unroll 1
  for (int c0 = part * prm.cols; c0 < ql * c.group; c0 += prm.parts * prm.cols) {
    const int col = c0 + lcol;
    const int j = col / c.group, jj = col - j * c.group;
    float acc[PER], M = -INFINITY, Ls = 0.f;
#pragma unroll
    for (int k = 0; k < PER; k++) acc[k] = 0.f;
    int2 own_tile = make_int2(0, 0), pre_tile = make_int2(0, 0);
    int n_own = 0, n_pre = 0;
    if (col < ql * c.group) {
      if (g >= 0) n_pre = pre.pieces(c, pv, j + off, &pre_tile) * pre_subs;
      n_own = own.pieces(c, pv, j, &own_tile) * own_subs;
    }
    const int n = n_pre + n_own;  // the prefix's first
#pragma unroll 1
    for (int k0 = pl; k0 < n; k0 += 32 * prm.lanes) {
      const int k = k0 + prm.lanes * lane;
      const float *o = nullptr, *ml = nullptr;
      if (k < n_pre) o = pre.piece(c, pv, D, prm.slot, pre_tile, h, j + off, jj, k / pre_subs, k % pre_subs, &ml);
      else if (k < n) o = own.piece(c, pv, D, prm.slot, own_tile, h, j, jj, (k - n_pre) / own_subs, (k - n_pre) % own_subs, &ml);
      float2 x = make_float2(-INFINITY, 0.f);
      if (o) x = *reinterpret_cast<const float2*>(ml);
      float mn = x.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
      mn = fmaxf(M, mn);
      const float mu = mn == -INFINITY ? 0.f : mn;
      const Exp2Pair ea(M - mu), eb(x.x - mu);
      const float scale = ea.both(), w = o ? eb.both() : 0.f;
      const float l = o ? eb.of(x.y) : 0.f;
      M = mn;
      Ls = ea.of(Ls);
#pragma unroll
      for (int e = 0; e < PER; e++) acc[e] *= scale;
      const uint32_t there = __ballot_sync(0xffffffffu, o != nullptr);
      if (!there) continue;
      // absent pieces read the first one there with a weight of 0 (its values are finite)
      const unsigned long long some = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), __ffs(there) - 1);
      const unsigned long long mine = o ? reinterpret_cast<unsigned long long>(o) : some;
      const int count = 32 - __clz(there);
#pragma unroll 4
      for (int kk = 0; kk < count; kk++) {
        const float* src = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, mine, kk));
        const float a = __shfl_sync(0xffffffffu, w, kk);
        Ls += __shfl_sync(0xffffffffu, l, kk);
        float val[PER];
#pragma unroll
        for (int e = 0; e < PER; e += VEC) {
          const float* p = src + element(lane, e);
          if constexpr (VEC == 4) {
            const float4 y = *reinterpret_cast<const float4*>(p);
            val[e] = y.x, val[e + 1] = y.y, val[e + 2] = y.z, val[e + 3] = y.w;
          } else if constexpr (VEC == 2) {
            const float2 y = *reinterpret_cast<const float2*>(p);
            val[e] = y.x, val[e + 1] = y.y;
          } else {
            val[e] = *p;
          }
        }
        // a piece without keys holds zeros (or nothing that its weight of 0 may meet)
#pragma unroll
        for (int e = 0; e < PER; e++) acc[e] = a == 0.f ? acc[e] : fmaf(val[e], a, acc[e]);
      }
    }
    if (prm.lanes > 1) {
      float* mine = spart + (lcol * prm.lanes + pl) * (D + 2);
      if (pl > 0) {
#pragma unroll
        for (int k = 0; k < PER; k++) mine[lane + 32 * k] = acc[k];
        if (lane == 0) {
          mine[D] = M;
          mine[D + 1] = Ls;
        }
      }
      __syncthreads();
      if (pl == 0) {
#pragma unroll 1
        for (int p = 1; p < prm.lanes; p++) {
          const float* o = mine + p * (D + 2);
          const float m = o[D], mn = fmaxf(M, m), mu = mn == -INFINITY ? 0.f : mn;
          const Exp2Pair ea(M - mu), eb(m - mu);
          const float a = ea.both(), b = eb.both();
#pragma unroll
          for (int k = 0; k < PER; k++) acc[k] = acc[k] * a + o[lane + 32 * k] * b;
          Ls = ea.of(Ls) + eb.of(o[D + 1]);
          M = mn;
        }
      }
      __syncthreads();  // read before the next rows' are written
    }
    if (pl > 0 || n == 0) continue;
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;  // no visible key: zeros
    uint16_t* dst = c.out + (long long)(q0 + j) * c.out_stride + (long long)(h * c.group + jj) * D;
#pragma unroll
    for (int e = 0; e < PER; e += VEC) {
      uint16_t* p = dst + element(lane, e);
      if constexpr (VEC == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2_rn(acc[e] * inv, acc[e + 1] * inv),
                                                  pack_bf16x2_rn(acc[e + 2] * inv, acc[e + 3] * inv));
      else if constexpr (VEC == 2)
        *reinterpret_cast<uint32_t*>(p) = pack_bf16x2_rn(acc[e] * inv, acc[e + 1] * inv);
      else
        *p = (uint16_t)(pack_bf16x2_rn(acc[e] * inv, 0.f) & 0xffffu);
    }
    if (c.sh.lse && lane == 0) c.sh.lse[(q0 + j) * c.sh.lse_stride + h * c.group + jj] = log_sum_exp(M, Ls);
  }
}

template <int D>
int launch_t(const SharedAttnArgs& s, cudaStream_t stream) {
  const AttnArgs& a = s.attn;
  SharedLayout L;
  if (!shared_layout(a.num_seqs, s.num_groups, a.num_q_tokens, a.num_q_heads, a.num_kv_heads, D, &L)) return KV_INT4_ERR_SIZE;
  PlanView pv = plan_view_fp8(a.workspace, L.base);
  uint8_t* const ws = static_cast<uint8_t*>(a.workspace);
  pv.vrec = reinterpret_cast<int4*>(ws + L.vrec);
  pv.dseq2 = reinterpret_cast<int4*>(ws + L.dseq2);
  pv.vinfo = reinterpret_cast<int2*>(ws + L.vinfo);
  pv.tloc = reinterpret_cast<int2*>(ws + L.tloc);
  pv.row_o = reinterpret_cast<float*>(ws + L.row_o);
  pv.row_ml = reinterpret_cast<float*>(ws + L.row_ml);
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
  c.causal = 1;
  c.qscale = a.softmax_scale * kLog2e;
  c.out = static_cast<uint16_t*>(a.out);
  c.out_stride = a.out_stride;
  c.status = a.dev_status;
  c.max_items = L.base.max_pairs * a.num_kv_heads;
  c.sh = SharedArgs{s.group_start, s.prefix_lens, s.num_groups, s.max_group_tokens, L.row_tokens, Fp8Ws<D>::ROWS, 64,
                    s.lse, s.lse_stride};
  // f with blocks per position, warps per head and column groups per warp as constants
  using std::integral_constant;
  constexpr int kWide = D <= 128 ? 4 : 2;  // most column groups per warp: registers allow them
  auto with_np = [](int np, int cg, auto&& f) {
    using One = integral_constant<int, 1>;
    using Two = integral_constant<int, 2>;
    if (np == 2) return f(Two{}, One{}, One{});
    if (np == 4) return f(integral_constant<int, kFp8Quad<D> ? 4 : 2>{}, One{}, One{});
    if (cg == 2) return f(One{}, One{}, Two{});
    if (cg == 4) return f(One{}, integral_constant<int, 4 / kWide>{}, integral_constant<int, kWide>{});
    return f(One{}, One{}, One{});
  };
  auto groups_of = [](long long cols) { return cols > 2 * kDecodeCols ? 4 : cols > kDecodeCols ? 2 : 1; };
  auto blocks_of = [](long long cols) { return cols > 4 ? 1 : cols > 2 || !kFp8Quad<D> ? 2 : 4; };
  // the largest divisor of Hkv that gives up to four warps of `warps` each and whose
  // ring leaves room for two CTAs per SM
  auto heads_of = [&](int warps, auto smem_bytes) {
    for (int h = 4 / warps; h > 1; h--)
      if (a.num_kv_heads % h == 0 && 2 * (smem_bytes(h) + 1024) <= 228 * 1024) return h;
    return 1;
  };
  const long long most_own = (long long)(a.max_query_len > 0 ? a.max_query_len : 1) * c.group;

  // one launch of clusters that share nothing where kv_fp8_attention would make it
  if (most_own <= kDecodeColsFp8) {
    auto direct = [&](auto np_tag, auto cg_tag) -> int {  // a status, -1: not here
      constexpr int NP = decltype(np_tag)::value, CG = decltype(cg_tag)::value;
      using G = Fp8Dec<D, NP>;
      constexpr auto kern = decode_fp8_kernel<D, NP, CG, true, true>;
      c.np = NP;
      c.hg = heads_of(CG, [](int h) { return G::smem_bytes(h); });
      c.ng = a.num_kv_heads / c.hg;
      c.dcols = kDecodeCols * CG / NP;
      static PerContext<int> occ_cache[5];
      int occ = 0;
      if (!occ_cache[c.hg].get(dev, [&](int* v) {
            int unused;  // the attribute is raised once, to the largest ring in use
            return configure(kern, (228 * 1024) / 2 - 1024, 128, &unused) &&
                   cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kern, c.hg * CG * 32, G::smem_bytes(c.hg)) == cudaSuccess &&
                   *v >= 1;
          }, &occ))
        return KV_INT4_ERR_CUDA;
      const int checks = s.num_groups > 0;  // a cluster that looks at the groups
      const long long tasks = (long long)a.num_seqs * c.ng, room = (long long)sms * occ;
      const long long table = (long long)a.max_blocks_per_seq * 16;
      const long long most = ((a.max_seq_len < table ? a.max_seq_len : table) + 16 * NP - 1) / (16 * NP);
      int cl = 1;
      while (cl < 8 && 2 * tasks * cl <= room && most > 2 * cl) cl *= 2;
      if (tasks * cl > room || most > 16 * cl) return -1;
      timing_begin(kTimedDecode, stream);
      const int e = launch_pdl(kern, dim3((unsigned)((tasks + checks) * cl)), c.hg * CG * 32, G::smem_bytes(c.hg), stream, cl,
                               Fp8DecParams{c, pv, 0, cl, false});
      timing_end(kTimedDecode, stream);
      return e;
    };
    using One = integral_constant<int, 1>;
    const int np = blocks_of(most_own), cg = groups_of(most_own);
    c.nl = 1;
    const int e = np == 4   ? direct(integral_constant<int, kFp8Quad<D> ? 4 : 2>{}, One{})
                  : np == 2 ? direct(integral_constant<int, 2>{}, One{})
                  : cg == 4 ? direct(One{}, integral_constant<int, 4>{})
                  : cg == 2 ? direct(One{}, integral_constant<int, 2>{})
                            : direct(One{}, One{});
    if (e >= 0) return e;
  }

  // decode, as in kv_fp8_attention; a group's queries count as one sequence's
  c.hg = c.ng = c.nl = c.np = 1;
  const long long most_tokens = s.num_groups > 0 && s.max_group_tokens > a.max_query_len ? s.max_group_tokens : a.max_query_len;
  const long long mq = (most_tokens > 0 ? most_tokens : 1) * c.group;
  const long long cols = mq <= kDecodeColsFp8 ? mq : most_own <= kDecodeColsFp8 ? most_own : c.group;
  int cg = groups_of(cols);
  const long long virt = (long long)a.num_seqs + s.num_groups;
  while (cg > 1 && virt * a.num_kv_heads * kDecodeCols * cg > L.base.direct_rows) cg /= 2;
  const bool any_decode = c.group <= kDecodeCols * cg;
  const int np = blocks_of(cols);
  int dec_grid = 0;
  if (any_decode) {
    int occ = 0;
    auto take = [&](auto np_tag, auto cg_tag, auto gw_tag) {
      constexpr int NP = decltype(np_tag)::value, CG = decltype(cg_tag)::value, GW = decltype(gw_tag)::value;
      using G = Fp8Dec<D, NP>;
      constexpr auto kern = decode_fp8_kernel<D, NP, CG, false, true, GW>;
      c.np = NP;
      c.hg = heads_of(CG, [](int h) { return G::smem_bytes(h, h * CG, GW); });
      static PerContext<int> occ_cache[5];
      return occ_cache[c.hg].get(dev, [&](int* v) {
        int unused;
        return configure(kern, (228 * 1024) / 2 - 1024, 128, &unused) &&
               cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kern, c.hg * CG * 32, G::smem_bytes(c.hg, c.hg * CG, GW)) ==
                   cudaSuccess &&
               *v >= 1;
      }, &occ);
    };
    if (!with_np(np, cg, take)) return KV_INT4_ERR_CUDA;
    c.ng = a.num_kv_heads / c.hg;
    long long grid = (long long)sms * occ;
    const int most_warps = s.num_groups > 0 ? kSharedDecodeWarps : kMaxDecodeWarps;  // as the workspace has slots
    if (grid * c.hg * cg > most_warps) grid = most_warps / (c.hg * cg);
    for (int l = (int)(grid < c.ng ? grid : c.ng); l >= 1; l--)
      if (c.ng % l == 0) {
        c.nl = l;
        break;
      }
    dec_grid = (int)(grid / c.nl * c.nl);
  }
  c.dcols = kDecodeCols * cg / c.np;

  using G = Fp8Ws<D>;
  const bool may_prefill = c.group > c.dcols || most_tokens * c.group > c.dcols;
  c.tile_tokens = G::ROWS / c.group;
  c.step_blocks = G::NB;
  c.split_steps = 4;
  c.split_ctas = sms;
  Fp8Maps maps;
  if (may_prefill) {
    if (!make_maps<D>(a, c.tile_tokens, &maps)) return KV_INT4_ERR_CUDA;
    static PerContext<int> occ_c;
    int occ = 0;
    if (!occ_c.get(dev, [](int* o) { return configure_tmem(prefill_ws_fp8_kernel<D, true>, G::SMEM, G::THREADS, 512, o); },
                   &occ))
      return KV_INT4_ERR_CUDA;
  }
  const bool may_split = may_prefill && a.max_seq_len > 2ll * 16 * c.step_blocks * c.split_steps;
  if (int e = launch_plan<true>(c, pv, may_prefill, may_split, stream)) return e;
  if (may_prefill) {
    const long long items = (L.base.max_pairs + L.base.max_pieces) * a.num_kv_heads;
    const long long grid = sms < items ? sms : items;
    timing_begin(kTimedPrefill, stream);
    const int e = launch_pdl(prefill_ws_fp8_kernel<D, true>, dim3((unsigned)grid), G::THREADS, G::SMEM, stream, 1, c, pv, maps);
    timing_end(kTimedPrefill, stream);
    if (e) return e;
  }
  if (any_decode) {
    timing_begin(kTimedDecode, stream);
    const int e = with_np(np, cg, [&](auto np_tag, auto cg_tag, auto gw_tag) {
      constexpr int NP = decltype(np_tag)::value, CG = decltype(cg_tag)::value;
      constexpr int GW = decltype(gw_tag)::value;
      return launch_pdl(decode_fp8_kernel<D, NP, CG, false, true, GW>, dim3(dec_grid), c.hg * CG * 32,
                        Fp8Dec<D, NP>::smem_bytes(c.hg, c.hg * CG, GW), stream, 1, Fp8DecParams{c, pv, dec_grid, 1, may_prefill});
    });
    timing_end(kTimedDecode, stream);
    if (e) return e;
  }
  // merge: CTAs per (sequence, kv head), a warp per row and piece lane, lanes as
  // far as all CTAs start at once
  const long long segs = (long long)a.num_seqs * a.num_kv_heads, warps = (long long)kMergeWarps * sms;
  int mcols = (int)(most_own < 8 ? most_own : 8), parts = 1, lanes = 1;
  while ((long long)mcols * parts < most_own && segs * parts * mcols < warps) parts *= 2;
  while (mcols * lanes * 2 <= kMergeWarps && 2ll * lanes * mcols * parts * segs <= warps) lanes *= 2;
  if (segs * parts > 0x7fffffff) return KV_INT4_ERR_SIZE;
  timing_begin(kTimedReduce, stream);
  const int e = launch_pdl(merge_shared_kernel<D>, dim3((unsigned)(segs * parts)), mcols * lanes * 32, merge_smem<D>(mcols, lanes),
                           stream, 1, SharedMergeParams{c, pv, dec_grid, mcols, lanes, parts, kDecodeCols * cg, may_prefill});
  timing_end(kTimedReduce, stream);
  return e;
}

}  // namespace

int launch_attention_shared_fp8(const SharedAttnArgs& a, cudaStream_t stream) {
  switch (a.attn.head_size) {
    case 64: return launch_t<64>(a, stream);
    case 96: return launch_t<96>(a, stream);
    case 128: return launch_t<128>(a, stream);
    case 192: return launch_t<192>(a, stream);
    case 256: return launch_t<256>(a, stream);
    default: return KV_INT4_ERR_HEAD_SIZE;
  }
}

}  // namespace kvint4
