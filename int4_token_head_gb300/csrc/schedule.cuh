// The attention launches' shared parameters and their device-built schedule
// (decode sequences with position prefix sums, prefill tiles longest first),
// used by the INT4 / int8 kernels and by the FP8 ones.
#pragma once

#include <limits.h>

#include "common.cuh"
#include "internal.h"

namespace kvint4 {

constexpr float kLog2e = 1.4426950408889634f;

struct PlanView {
  int32_t* plan;      // [0] n_dseq, [1] n_prefill_items, [2] prefill work counter, [3] n_pseq,
                      // FP8: [4] split tiles, [5] the schedule's number in this workspace
  int4* msplit;       // FP8: tiles in pieces: (sequence, tile, first piece row, pieces); plan[4] of them
  struct PrefillPiece* pieces;  // FP8: prefill tiles and pieces of tiles, longest first (in place of plist)
  float* piece_o;
  float* piece_ml;
  int4* dseq;         // decode sequences in order: (sequence id, seq_len, first query token, q_len)
  int64_t* dprefix;
  int2* ptab;         // prefill sequences in order: (seq id, index of its first item); [n_pseq].y = items
  int2* plist;        // prefill (sequence, tile) pairs, longest first; pair i gives items i Hkv .. i Hkv + Hkv - 1
  __half* qrot;
  float* direct_o;
  float* direct_ml;
  float* warp_o;
  float* warp_ml;
  // shared prefixes only (SH below)
  int4* vrec;    // two per virtual sequence: (first query token, query tokens, keys, position of the first query),
                 // (table offset, two words; first row-buffer token or -1; group or -1)
  int4* dseq2;   // with dseq: (table offset, two words; position of the first query; -)
  int2* vinfo;   // per virtual sequence: (0 nothing, 1 decode, 2 prefill; index in dseq, first tile)
  int2* tloc;    // per prefill tile: (first piece row, pieces), (-1, 1) for a whole one
  float* row_o;  // [2][row_tokens][q heads][d] whole tiles' rows: prefixes', then the sequences'
  float* row_ml;
};

// Shared prefixes (kernels with SH set): the batch is worked on as virtual
// sequences, the groups' prefixes (all query tokens of a group against the keys
// that its sequences share, no mask) and then the sequences themselves (their own
// keys, or all of them where nothing is shared).  A row's two results are merged.
struct SharedArgs {
  const int32_t* group_start;
  const int32_t* prefix_lens;
  int num_groups;
  int max_group_tokens;
  int row_tokens;    // query tokens that the row buffer holds
  int max_rows;      // query rows per kv head up to which a sequence shares
  int min_saved;     // key positions that a group must save
  float* lse;
  int64_t lse_stride;
};

// A prefill tile of a sequence, or a piece of its keys: entry i of the list
// gives items i Hkv .. i Hkv + Hkv - 1.  Piece k of kv head h of a tile in P
// pieces of R query rows leaves unnormalised rows row + h P R .. + R - 1.
struct PrefillPiece {
  int seq, tile;
  int kb0, nkb;     // blocks [kb0, nkb) of the sequence
  int row;          // first row of head 0, -1 if the tile is whole
  int head_rows;    // P R
  int unused[2];
};
static_assert(sizeof(PrefillPiece) == 32, "read as two int4");

static PlanView plan_view_fp8(void* ws, const WorkspaceLayoutFp8& L) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  PlanView v{};
  v.plan = reinterpret_cast<int32_t*>(b + L.plan);
  v.dseq = reinterpret_cast<int4*>(b + L.dseq);
  v.dprefix = reinterpret_cast<int64_t*>(b + L.dprefix);
  v.ptab = reinterpret_cast<int2*>(b + L.ptab);
  v.pieces = reinterpret_cast<PrefillPiece*>(b + L.plist);
  v.msplit = reinterpret_cast<int4*>(b + L.msplit);
  v.direct_o = reinterpret_cast<float*>(b + L.direct_o);
  v.direct_ml = reinterpret_cast<float*>(b + L.direct_ml);
  v.warp_o = reinterpret_cast<float*>(b + L.warp_o);
  v.warp_ml = reinterpret_cast<float*>(b + L.warp_ml);
  v.piece_o = reinterpret_cast<float*>(b + L.piece_o);
  v.piece_ml = reinterpret_cast<float*>(b + L.piece_ml);
  return v;
}

static PlanView plan_view(void* ws, const WorkspaceLayout& L) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  PlanView v{};
  v.plan = reinterpret_cast<int32_t*>(b + L.plan);
  v.dseq = reinterpret_cast<int4*>(b + L.dseq);
  v.dprefix = reinterpret_cast<int64_t*>(b + L.dprefix);
  v.ptab = reinterpret_cast<int2*>(b + L.pitems);
  v.plist = reinterpret_cast<int2*>(b + L.plist);
  v.qrot = reinterpret_cast<__half*>(b + L.qrot);
  v.direct_o = reinterpret_cast<float*>(b + L.direct_o);
  v.direct_ml = reinterpret_cast<float*>(b + L.direct_ml);
  v.warp_o = reinterpret_cast<float*>(b + L.warp_o);
  v.warp_ml = reinterpret_cast<float*>(b + L.warp_ml);
  return v;
}

// KV cache formats: INT4 codes of the rotated vectors, two per byte (the
// method), or int8 codes of the unrotated vectors (the int8_per_token_head
// sibling mode).
enum KvFmt { kFmtInt4 = 0, kFmtInt8 = 1 };

struct Common {
  const uint16_t* q;
  int64_t q_stride;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  CacheGeo geo;  // cache strides (separate or in-slot scales)
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seq_lens;
  const int32_t* qsl;
  int num_seqs;
  int num_q_tokens;
  int max_qlen;  // the caller's max_query_len: launch sizes assume no q_len above it
  int hq;
  int hkv;
  int group;
  FastDiv gdiv{1};  // division by group
  int num_blocks;
  int causal;
  int window;    // sliding window (0: none): the query at position p sees no key at p - window or before
  float qscale;  // softmax_scale * log2(e) / b
  const int8_t* signs;
  uint16_t* out;
  int64_t out_stride;
  int32_t* status;
  int tile_tokens;  // prefill: query tokens per 64-row tile
  int hg;           // decode: kv heads per CTA (largest divisor of hkv <= 4)
  int ng;           // decode: head groups per sequence (hkv / hg)
  int nl;           // decode: lanes (a divisor of ng): CTA r serves the head groups g with g mod nl = r mod nl
  int np;           // decode: 16-key blocks per schedule position (1, 2 or 4)
  int dcols;        // decode: query columns per block (8 / np); longer queries go to prefill
  long long max_items;  // capacity of the prefill item list
  int step_blocks;      // FP8 prefill: cache blocks per step
  int split_steps;      // FP8 prefill: least steps of a piece
  int split_ctas;       // FP8 prefill: CTAs that run at once
  SharedArgs sh;        // kernels with SH set
};

// a sequence as attention sees it; with SH set a virtual one
struct SeqView {
  int q0, ql;     // query tokens [q0, q0 + ql)
  int L;          // keys
  int ctx;        // position of the first query: it sees keys up to there, the next ones one more each
  long long tab;  // first entry of its block table
};
template <bool SH>
__device__ __forceinline__ SeqView seq_view(const Common& c, const PlanView& pv, int s) {
  if constexpr (SH) {
    const int4 a = pv.vrec[2 * s], b = pv.vrec[2 * s + 1];
    return SeqView{a.x, a.y, a.z, a.w, (long long)(uint32_t)b.x | (long long)b.y << 32};
  } else {
    const int q0 = c.qsl[s], ql = c.qsl[s + 1] - q0, L = c.seq_lens[s];
    return SeqView{q0, ql, L, L - ql, (long long)s * c.max_blocks};
  }
}

// floor(n / d) for 0 <= n, 0 < d: one 32-bit division when both fit (the
// usual case for schedule arithmetic), the 64-bit routine otherwise
__device__ __forceinline__ long long div_nn(long long n, long long d) {
  return ((n | d) >> 31) == 0 ? (long long)((uint32_t)n / (uint32_t)d) : n / d;
}

// first key position visible to the query at position qpos, which is below 0
// where queries outnumber keys: nothing is subtracted from it then (with a
// window near 2^31 the difference would wrap to a position behind every key)
__device__ __forceinline__ int window_lo(const Common& c, int qpos) {
  return c.window > 0 && qpos >= c.window ? qpos - c.window + 1 : 0;
}
// first 16-key block a sequence's attention reads: blocks wholly before the
// window of its earliest query (position L - q_len) are never visible
__device__ __forceinline__ int first_block(const Common& c, int L, int ql) { return window_lo(c, L - ql) >> 4; }

__device__ __forceinline__ bool is_decode_kind(int qlen, const Common& c) {
  return c.group <= c.dcols && qlen * c.group <= c.dcols;
}

// keys that prefill tile t of a sequence (kv length L, q_len qn) attends:
// up to its last query's causal horizon, or all
__device__ __forceinline__ int prefill_tile_keys(const Common& c, int L, int qn, int t) {
  return c.causal ? L - qn + min(qn, (t + 1) * c.tile_tokens) : L;
}
// prefill item itn in the prep kernel's longest-first order: (sequence, kv
// head, tile, 16-key blocks), or sequence -1 past the last item
__device__ __forceinline__ int4 prefill_item(const Common& c, const PlanView& pv, int itn, int n_items) {
  if (itn >= n_items) return make_int4(-1, 0, 0, 0);
  const int pi = itn / c.hkv;
  const int2 st = pv.plist[pi];
  const int qa = c.qsl[st.x], qn = c.qsl[st.x + 1] - qa;
  const int keys = prefill_tile_keys(c, c.seq_lens[st.x], qn, st.y);
  return make_int4(st.x, itn - pi * c.hkv, st.y, (keys + 15) / 16);
}

// item itn of the FP8 prefill: a tile or a piece of one, for one kv head
struct PrefillItem {
  int seq, h, tile;  // seq -1: past the last item
  int kb0, nkb;      // blocks [kb0, nkb)
  int row;           // first piece row, -1 if the tile is whole
};
__device__ __forceinline__ PrefillItem prefill_piece_item(const Common& c, const PlanView& pv, int itn, int n_items) {
  if (itn >= n_items) return PrefillItem{-1, 0, 0, 0, 0, -1};
  const int pi = itn / c.hkv, h = itn - pi * c.hkv;
  const int4 a = reinterpret_cast<const int4*>(pv.pieces + pi)[0];
  const int2 b = reinterpret_cast<const int2*>(pv.pieces + pi)[2];
  return PrefillItem{a.x, h, a.y, a.z, a.w, b.x < 0 ? -1 : b.x + h * b.y};
}

constexpr int kPrepThreads = 256;  // threads of the CTA that builds the schedule

template <typename T>
__device__ T block_exclusive_scan(T v, T* total, T* sbuf /*[kPrepThreads/32]*/) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sbuf[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T w = lane < kPrepThreads / 32 ? sbuf[lane] : T(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      T y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < kPrepThreads / 32) sbuf[lane] = w;
  }
  __syncthreads();
  T before = warp > 0 ? sbuf[warp - 1] : T(0);
  *total = sbuf[kPrepThreads / 32 - 1];
  __syncthreads();
  return before + x - v;
}

// Whether a sequence's metadata is consistent.  Its queries are its last q_len
// positions, so its length is at least q_len; with ANY_LEN a non-causal call
// may attend keys of another length (none included).  A q_len above
// max_query_len would fall outside the launches sized from it (decode columns,
// the prefill launch, the reduce segments).
template <bool ANY_LEN>
__device__ __forceinline__ bool schedule_seq_ok(const Common& c, int q0, int ql, int L) {
  return !(q0 < 0 || (long long)q0 + ql > c.num_q_tokens || ql < 0 || L < (ANY_LEN && !c.causal ? 0 : ql) ||
           ql > c.max_qlen || (long long)L > (long long)c.max_blocks * 16);
}

// The FP8 prefill's list of tiles, longest first, with tiles split over their
// keys where that shortens the launch (few rows against a long cache: chunked
// prompts, cross attention, queries of a few tokens; 2 x 256 tokens against
// 16384 keys, 32/8 heads of 128: 165 us, whole tiles 281).  A tile of more than
// S steps becomes ceil(steps / S) equal pieces: S is a CTA's share of all steps,
// at least c.split_steps (a piece costs about two steps on top of its own, and
// its rows are merged), twice that where decodes run beside on the SMs that
// whole tiles leave (4 prompts of up to 400 tokens beside 28 decodes: 45.9 us,
// in pieces 55.3; not so beside shared prefixes, whose tiles are most of the work:
// 64 sequences over 8192 positions 63 us, without 59).  If there are fewer tiles than CTAs, an S up to twice as
// large whose pieces all run at once is taken; without one, only tiles of more
// than two shares are worth it.
// With shared prefixes (SH) a few long tiles meet many short ones, a sequence's
// own, which fit beside them: the S is taken whose longest pieces are done first,
// wave by wave (16 questions to one prefix of 16384 positions, 16/4 heads of 192: 80
// pieces of 64 steps and 64 short tiles, which by the rule above must all run at
// once, 144 us; 140 pieces of 37 steps 103).  Everything follows from the call's lengths
// alone, so results do not depend on the order of arrival.  Batches of more
// than kSplitTiles tiles, or of kSplitWaves items per CTA, which the order by
// length balances, keep their tiles whole.  `seqs`: the prefill sequences in
// shared memory, if the batch fits there.  The code is kept short (one loop for
// both passes, none for splits where the host rules them out): a lone CTA that
// runs it once waits for its instructions most of the time (with the loops
// inlined twice 2 to 3 us more per call).
constexpr int kSplitTiles = 1024;
constexpr int kSplitWaves = 6;
template <int BUCKETS, bool SPLIT, bool SH>
__device__ void build_pieces(const Common& c, const PlanView& pv, int n_pseq, int n_tiles, bool with_decode,
                             const int4* seqs, int* hist, int32_t* s_i32) {
  __shared__ int4 tiles[kSplitTiles];  // (sequence, tile, first block, end block)
  __shared__ short tile_rows[kSplitTiles];
  __shared__ int2 s_cand[kPrepThreads / 32];
  __shared__ int next_row, next_split;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // tiles base .. base + kSplitTiles - 1.  A few long sequences: a warp's lanes
  // share a sequence's tiles; many: a thread each
  auto fill = [&](int base) {
    const int lps = n_pseq >= kPrepThreads / 4 ? 1 : 32;
#pragma unroll 1
    for (int p = threadIdx.x / lps; p < n_pseq; p += kPrepThreads / lps) {
      int4 x;  // (sequence, query tokens, keys, index of its first tile)
      if (seqs) {
        x = seqs[p];
      } else {
        const int2 pt = pv.ptab[p];
        const SeqView v = seq_view<SH>(c, pv, pt.x);
        x = make_int4(pt.x, v.ql, v.L, pt.y / c.hkv);
      }
      const bool whole = SH && x.x < c.sh.num_groups;  // every query sees every key
      const int nt = (x.y + c.tile_tokens - 1) / c.tile_tokens;
#pragma unroll 1
      for (int t = threadIdx.x % lps; t < nt; t += lps) {
        const int i = x.w + t - base, tok = t * c.tile_tokens;
        if (i < 0 || i >= kSplitTiles) continue;
        tiles[i] = make_int4(x.x, t, window_lo(c, x.z - x.y + tok) >> 4,
                             ((whole ? x.z : prefill_tile_keys(c, x.z, x.y, t)) + 15) / 16);
        tile_rows[i] = (short)(min(c.tile_tokens, x.y - tok) * c.group);
      }
    }
  };
  auto steps_of = [&](const int4& x) { return max(0, (x.w - x.z + c.step_blocks - 1) / c.step_blocks); };
  if (threadIdx.x == 0) next_row = next_split = 0;
  for (int i = threadIdx.x; i < BUCKETS; i += kPrepThreads) hist[i] = 0;
  __syncthreads();  // the sequence table
  fill(0);
  __syncthreads();
  int S = INT_MAX;
  if (SPLIT && n_tiles <= kSplitTiles && (long long)n_tiles * c.hkv < (long long)kSplitWaves * c.split_ctas) {
    // every warp takes the sum, then one candidate for S: S0 to 2 S0, and 4 S0
    long long sum = 0;
    int longest = 0;
#pragma unroll 1
    for (int i = lane; i < n_tiles; i += 32) {
      const int n = steps_of(tiles[i]);
      sum += n;
      longest = max(longest, n);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    longest = __reduce_max_sync(0xffffffffu, longest);
    const long long share = div_nn(sum * c.hkv + c.split_ctas - 1, c.split_ctas);
    const long long S0 = max(share, (long long)c.split_steps << (with_decode && !SH ? 1 : 0));
    const bool one_wave = (long long)n_tiles * c.hkv < c.split_ctas;
    if (SH && longest > S0) {
      constexpr int W = kPrepThreads / 32;
      constexpr float PIECE = 4.f;  // steps' time that an item takes on top of its own
      const int cand = (int)min(warp == W - 1 ? (long long)longest : warp == W - 2 ? 4 * S0 : S0 + S0 * warp / (W - 3),
                                (long long)longest);
      int r = 0, all = 0, most = 0;  // rows of the pieces, all items, the long ones (of one kv head)
#pragma unroll 1
      for (int i = lane; i < n_tiles; i += 32) {
        const int n = steps_of(tiles[i]), P = n > cand ? min((n - 1) / cand + 1, 2 * kMaxPieces) : 1;
        all += P;
        if (2 * n > P * cand) most += P;
        if (P > 1) r += P * tile_rows[i];
      }
      r = __reduce_add_sync(0xffffffffu, r);
      all = __reduce_add_sync(0xffffffffu, all);
      most = __reduce_add_sync(0xffffffffu, most);
      if (lane == 0) {
        const float heads = (float)c.hkv / c.split_ctas;
        const float time = fmaxf(ceilf(most * heads) * (cand + PIECE), ((float)sum + PIECE * all) * heads);
        s_cand[warp] = make_int2(cand, all > kMaxPieces || (long long)r * c.hkv > kPieceRows ? INT_MAX : __float_as_int(time));
      }
      __syncthreads();
      int best = INT_MAX;
#pragma unroll 1
      for (int i = 0; i < W; i++)
        if (s_cand[i].y < best) {
          best = s_cand[i].y;
          S = s_cand[i].x;
        }
    } else if (!SH && longest > (one_wave ? S0 : 2 * S0)) {  // else every tile stays whole
      constexpr int W = kPrepThreads / 32;
      const int cand = (int)min(warp == W - 1 ? 4 * S0 : S0 + (S0 * warp + W - 3) / (W - 2), (long long)INT_MAX);
      long long p = 0, r = 0, all = 0;  // pieces of split tiles, their rows, all entries
#pragma unroll 1
      for (int i = lane; i < n_tiles; i += 32) {
        const int n = steps_of(tiles[i]), P = n > cand ? (n - 1) / cand + 1 : 1;
        all += P;
        if (P > 1) {
          p += P;
          r += (long long)P * tile_rows[i] * c.hkv;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        p += __shfl_xor_sync(0xffffffffu, p, o);
        r += __shfl_xor_sync(0xffffffffu, r, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
      }
      // 2: fits the workspace and all of it runs at once; 1: fits
      if (lane == 0)
        s_cand[warp] = make_int2(cand, p > kMaxPieces || r > kPieceRows ? 0
                                 : one_wave && all * c.hkv <= c.split_ctas ? 2 : longest > 2 * S0);
      __syncthreads();
      int best = 0;
      for (int i = 0; i < W; i++)
        if (s_cand[i].y > best) {
          best = s_cand[i].y;
          S = s_cand[i].x;
        }
    }
  }

  // counting sort by blocks, descending, within a bucket in arbitrary order
  // (every item computes the same rows either way): pass 0 counts, pass 1
  // writes the list.  Few tiles may have many pieces: a warp each, whose lanes
  // take the pieces
  int sh = 0;
  while ((((long long)c.max_blocks + 1) >> sh) >= BUCKETS) sh++;
  const int lpp = n_tiles <= kPrepThreads / 4 ? 32 : 1;
  int total = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; pass++) {
#pragma unroll 1
    for (int base = 0; base < n_tiles; base += kSplitTiles) {
      if (n_tiles > kSplitTiles) {
        __syncthreads();
        fill(base);
        __syncthreads();
      }
      const int count = min(n_tiles - base, kSplitTiles);
#pragma unroll 1
      for (int i = threadIdx.x / lpp; i < count; i += kPrepThreads / lpp) {
        const int4 x = tiles[i];
        const int rows = tile_rows[i], n = steps_of(x), P = SPLIT && n > S ? (n - 1) / S + 1 : 1;
        int row = 0;
        if (SPLIT && pass && P > 1) {
          if (threadIdx.x % lpp == 0) {
            row = atomicAdd(&next_row, P * rows * c.hkv);
            pv.msplit[atomicAdd(&next_split, 1)] = make_int4(x.x, x.y, row, P);
          }
          if (lpp > 1) row = __shfl_sync(0xffffffffu, row, 0);
        }
        if (SH && pass && threadIdx.x % lpp == 0) pv.tloc[base + i] = make_int2(P > 1 ? row : -1, P);
        const int each = n / P, more = n - each * P;  // the first `more` pieces have a step more
#pragma unroll 1
        for (int k = threadIdx.x % lpp; k < P; k += lpp) {
          const int lo = x.z + c.step_blocks * (k * each + min(k, more));
          const int hi = k + 1 < P ? lo + c.step_blocks * (each + (k < more)) : x.w;
          const int at = atomicAdd(&hist[BUCKETS - 1 - min(BUCKETS - 1, max(0, hi - lo) >> sh)], 1);
          if (pass) {
            int4* dst = reinterpret_cast<int4*>(pv.pieces + at);
            dst[0] = make_int4(x.x, x.y, lo, hi);
            dst[1] = make_int4(P > 1 ? row + k * rows : -1, P * rows, 0, 0);
          }
        }
      }
    }
    __syncthreads();
    if (pass == 0) {
      // exclusive prefix over the buckets: thread j owns buckets [8j, 8j + 8)
      constexpr int PER = BUCKETS / kPrepThreads;
      int mine = 0;
#pragma unroll
      for (int i = 0; i < PER; i++) mine += hist[threadIdx.x * PER + i];
      int run = block_exclusive_scan<int>(mine, &total, s_i32);
#pragma unroll
      for (int i = 0; i < PER; i++) {
        const int hb = hist[threadIdx.x * PER + i];
        hist[threadIdx.x * PER + i] = run;
        run += hb;
      }
      __syncthreads();
    }
  }
  if (threadIdx.x == 0) {
    pv.plan[1] = total * c.hkv;
    pv.plan[4] = next_split;
  }
}

// What a group asks of the row buffer: if it does not fit, one token more than there
// is asks for all the same, and what a round of groups asks for stays in 32 bits
// (groups of a query_start_loc that does not ascend may hold the same tokens each)
__host__ __device__ constexpr int row_claim(int tokens, int room) { return tokens <= room ? tokens : room + 1; }
static_assert((long long)kPrepThreads * row_claim(INT_MAX, kSharedRows) + kSharedRows <= INT_MAX, "claims of a round");

// The virtual sequences of a call with shared prefixes, by the schedule's CTA.  A
// group shares its first P positions, whole blocks of them that come before the
// queries of all its sequences; it does where that saves keys (two sequences with
// queries at least, none of which fills a prefill tile by itself) and where the row
// buffer has room for its rows, in the groups' order.  Else its sequences are
// worked on whole.  group_start is looked at first: one that does not ascend within
// the batch shares nothing.
__device__ inline void build_shared(const Common& c, const PlanView& pv) {
  __shared__ int gs[kMostGroups + 1], least[kMostGroups], first[kMostGroups], count[kMostGroups];
  __shared__ int s_sum[kPrepThreads / 32];
  const SharedArgs& sh = c.sh;
  const int tid = threadIdx.x, NG = sh.num_groups;
  bool bad = false;
  for (int g = tid; NG > 0 && g <= NG; g += kPrepThreads) {
    const int x = sh.group_start[g];
    gs[g] = x;
    bad = bad || x < 0 || x > c.num_seqs || (g > 0 && x < sh.group_start[g - 1]);
    if (g < NG) {
      least[g] = INT_MAX;
      first[g] = INT_MAX;
      count[g] = 0;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && NG > 0) flag(c.status, KV_INT4_DEV_BAD_SEQ);
  // the group of sequence s: the last one that starts at or before it, -1 for none
  auto group_of = [&](int s) {
    if (NG == 0 || bad || s < gs[0] || s >= gs[NG]) return -1;
    int lo = 0, hi = NG;
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (gs[m] <= s) lo = m;
      else hi = m;
    }
    return lo;
  };
  for (int s = tid; s < c.num_seqs; s += kPrepThreads) {
    const int q0 = c.qsl[s], ql = c.qsl[s + 1] - q0, L = c.seq_lens[s], g = group_of(s);
    if (g < 0 || ql == 0) continue;
    if (!schedule_seq_ok<true>(c, q0, ql, L) || (long long)ql * c.group > sh.max_rows) {
      atomicMin(&least[g], 0);
    } else {
      atomicMin(&least[g], L - ql);
      atomicMin(&first[g], s);
      atomicAdd(&count[g], 1);
    }
  }
  __syncthreads();
  int before = 0;  // row-buffer tokens of earlier rounds
  for (int g0 = 0; g0 < NG; g0 += kPrepThreads) {
    const int g = g0 + tid;
    int P = 0, tokens = 0, q0 = 0;
    if (g < NG && !bad && count[g] >= 2) {
      q0 = c.qsl[gs[g]];
      tokens = c.qsl[gs[g + 1]] - q0;
      P = max(0, min(sh.prefix_lens[g], least[g])) & ~15;
      if ((long long)P * (count[g] - 1) < sh.min_saved || q0 < 0 || tokens <= 0 || tokens > sh.max_group_tokens ||
          q0 > c.num_q_tokens - tokens)
        P = 0;
    }
    int total;
    const int at = before + block_exclusive_scan<int>(P > 0 ? row_claim(tokens, sh.row_tokens) : 0, &total, s_sum);
    before = min(before + total, sh.row_tokens);
    if (P > 0 && (long long)at + tokens > sh.row_tokens) P = 0;
    if (g < NG) {
      const long long tab = P > 0 ? (long long)first[g] * c.max_blocks : 0;
      pv.vrec[2 * g] = make_int4(q0, P > 0 ? tokens : 0, P, P);
      pv.vrec[2 * g + 1] = make_int4((int)(uint32_t)tab, (int)(tab >> 32), P > 0 ? at : -1, -1);
      least[g] = P;  // from here on: the shared positions, the group's first token and its place in the row buffer
      first[g] = q0;
      count[g] = at;
    }
  }
  __syncthreads();
  for (int s = tid; s < c.num_seqs; s += kPrepThreads) {
    const int q0 = c.qsl[s], L = c.seq_lens[s], g = group_of(s);
    int ql = c.qsl[s + 1] - q0;
    if (!schedule_seq_ok<true>(c, q0, ql, L)) {
      flag(c.status, KV_INT4_DEV_BAD_SEQ);
      ql = 0;
    }
    const int P = g >= 0 && ql > 0 ? least[g] : 0;
    const long long tab = (long long)s * c.max_blocks + (P >> 4);
    const int v = NG + s;
    pv.vrec[2 * v] = make_int4(q0, ql, L - P, L - P - ql);
    pv.vrec[2 * v + 1] = make_int4((int)(uint32_t)tab, (int)(tab >> 32),
                                   P > 0 ? sh.row_tokens + count[g] + q0 - first[g] : -1, P > 0 ? g : -1);
  }
  __syncthreads();  // the records are read by other threads of the CTA
}

// The schedule, by one CTA of kPrepThreads threads.  PREFILL 0: no sequence of
// the call can be a prefill, 1: none can be split, 2: any (code that is not there
// is not fetched either).
template <bool ANY_LEN, int PREFILL = 1, bool SH = false>
__device__ void build_schedule(const Common& c, const PlanView& pv) {
  const int num_seqs = SH ? c.sh.num_groups + c.num_seqs : c.num_seqs;
  __shared__ int32_t s_i32[kPrepThreads / 32];
  __shared__ long long s_i64[kPrepThreads / 32];
  __shared__ long long s_i64t[ANY_LEN ? kPrepThreads / 32 : 1];
  __shared__ int4 seqs[ANY_LEN && PREFILL > 0 ? kPrepThreads : 1];
  int n_dseq = 0, n_pseq = 0;
  long long dpre = 0, n_items = 0;
  for (int base = 0; base < num_seqs; base += kPrepThreads) {
    const int s = base + threadIdx.x;
    int kind = 0, nblk = 0, ntiles = 0, ql = 0, L = 0, q0 = 0;
    SeqView view{};
    if (s < num_seqs) {
      view = seq_view<SH>(c, pv, s);
      q0 = view.q0;
      L = view.L;
      ql = view.ql;
      if (!SH && !schedule_seq_ok<ANY_LEN>(c, q0, ql, L)) {
        flag(c.status, KV_INT4_DEV_BAD_SEQ);
      } else if (ql > 0) {
        kind = is_decode_kind(ql, c) ? 1 : 2;
        nblk = (L + 15) / 16;
        if (kind == 2) ntiles = (ql + c.tile_tokens - 1) / c.tile_tokens;
      }
    }
    int tot_a, tot_p = 0, ex_a, ex_p = 0;
    long long tot_b, tot_c = 0, ex_b, ex_c = 0;
    const int npos = kind == 1 ? (nblk - first_block(c, L, ql) + c.np - 1) / c.np : 0;
    if constexpr (ANY_LEN) {
      // the four sums in one pass with one barrier, counts in one word
      const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
      int n = (kind == 1) | (kind == 2) << 16;
      long long b = npos, t = (long long)ntiles * c.hkv;
      const int n_in = n;
      const long long b_in = b, t_in = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int yn = __shfl_up_sync(0xffffffffu, n, o);
        const long long yb = __shfl_up_sync(0xffffffffu, b, o);
        const long long yt = PREFILL > 0 ? __shfl_up_sync(0xffffffffu, t, o) : 0;
        if (lane >= o) {
          n += yn;
          b += yb;
          t += yt;
        }
      }
      __syncthreads();  // the last round's sums have been read
      if (lane == 31) {
        s_i32[warp] = n;
        s_i64[warp] = b;
        s_i64t[warp] = t;
      }
      __syncthreads();
      int en = n - n_in, tn = 0;
      ex_b = b - b_in;
      ex_c = t - t_in;
      tot_b = 0;
      for (int w = 0; w < kPrepThreads / 32; w++) {
        if (w == warp) {
          en += tn;
          ex_b += tot_b;
          ex_c += tot_c;
        }
        tn += s_i32[w];
        tot_b += s_i64[w];
        tot_c += s_i64t[w];
      }
      ex_a = en & 0xffff;
      ex_p = en >> 16;
      tot_a = tn & 0xffff;
      tot_p = tn >> 16;
    } else {
      ex_a = block_exclusive_scan<int>(kind == 1, &tot_a, s_i32);
      ex_b = block_exclusive_scan<long long>(npos, &tot_b, s_i64);
      ex_p = block_exclusive_scan<int>(kind == 2, &tot_p, s_i32);
      ex_c = block_exclusive_scan<long long>((long long)ntiles * c.hkv, &tot_c, s_i64);
    }
    if (kind == 1) {
      pv.dseq[n_dseq + ex_a] = make_int4(s, L, q0, ql);
      pv.dprefix[n_dseq + ex_a] = dpre + ex_b;
      if (SH) pv.dseq2[n_dseq + ex_a] = make_int4((int)(uint32_t)view.tab, (int)(view.tab >> 32), view.ctx, 0);
    } else if (PREFILL > 0 && kind == 2) {
      // the prefill kernel expands (tile, kv head) items from this table
      pv.ptab[n_pseq + ex_p] = make_int2(s, (int)min(n_items + ex_c, (long long)INT_MAX));
      if (ANY_LEN && base == 0) seqs[ex_p] = make_int4(s, ql, L, (int)min(ex_c / c.hkv, (long long)INT_MAX));
    }
    if (SH && s < num_seqs)
      pv.vinfo[s] = make_int2(kind, kind == 1 ? n_dseq + ex_a : kind == 2 ? (int)min((n_items + ex_c) / c.hkv, (long long)INT_MAX) : 0);
    n_dseq += tot_a;
    dpre += tot_b;
    n_pseq += tot_p;
    n_items += tot_c;
  }
  if (threadIdx.x == 0) {
    pv.dprefix[n_dseq] = dpre;
    pv.plan[0] = n_dseq;
    if constexpr (PREFILL == 0) return;
    // more items than the workspace was sized for only happens with
    // inconsistent query_start_loc: the prefill part is dropped and flagged
    const bool over = n_items > c.max_items || n_items > INT_MAX;
    if (over) flag(c.status, KV_INT4_DEV_BAD_SEQ);
    pv.ptab[n_pseq] = make_int2(-1, over ? 0 : (int)n_items);
    pv.plan[1] = over ? 0 : (int)n_items;
    pv.plan[2] = 0;
    pv.plan[3] = n_pseq;
    if (ANY_LEN) pv.plan[4] = 0;
  }
  if constexpr (PREFILL == 0) return;
  // the prefill (sequence, tile) pairs, longest first: a counting sort over
  // buckets of 16-key blocks (descending), so that the longest items start
  // first and the shortest fill the end of the launch (within a bucket the
  // order is arbitrary; every item computes the same rows either way)
  constexpr int kBuckets = 2048;
  __shared__ int hist[kBuckets];
  if constexpr (ANY_LEN) {
    if (n_pseq > 0 && n_items <= c.max_items && n_items <= INT_MAX)
      build_pieces<kBuckets, PREFILL == 2, SH>(c, pv, n_pseq, (int)(n_items / c.hkv), n_dseq > 0,
                             num_seqs <= kPrepThreads ? seqs : nullptr, hist, s_i32);
    return;
  }
  if (n_pseq > 0 && n_items <= c.max_items && n_items <= INT_MAX) {
    int sh = 0;
    while ((((long long)c.max_blocks + 1) >> sh) >= kBuckets) sh++;
    auto bucket = [&](int nkb) { return kBuckets - 1 - min(kBuckets - 1, nkb >> sh); };
    for (int i = threadIdx.x; i < kBuckets; i += kPrepThreads) hist[i] = 0;
    __syncthreads();  // the sequence table and the histogram
    // a few long sequences: a warp's lanes share a sequence's tiles; many: a
    // thread each
    const int lps = n_pseq >= kPrepThreads / 4 ? 1 : 32, tl = threadIdx.x % lps;
    for (int p = threadIdx.x / lps; p < n_pseq; p += kPrepThreads / lps) {
      const int sq = pv.ptab[p].x, qn = c.qsl[sq + 1] - c.qsl[sq], Ls = c.seq_lens[sq];
      const int nt = (qn + c.tile_tokens - 1) / c.tile_tokens;
      for (int t = tl; t < nt; t += lps) atomicAdd(&hist[bucket((prefill_tile_keys(c, Ls, qn, t) + 15) / 16)], 1);
    }
    __syncthreads();
    // exclusive prefix over the buckets: thread j owns buckets [8j, 8j + 8)
    constexpr int PER = kBuckets / kPrepThreads;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < PER; i++) mine += hist[threadIdx.x * PER + i];
    int total;
    int run = block_exclusive_scan<int>(mine, &total, s_i32);
#pragma unroll
    for (int i = 0; i < PER; i++) {
      const int hb = hist[threadIdx.x * PER + i];
      hist[threadIdx.x * PER + i] = run;
      run += hb;
    }
    __syncthreads();
    for (int p = threadIdx.x / lps; p < n_pseq; p += kPrepThreads / lps) {
      const int sq = pv.ptab[p].x, qn = c.qsl[sq + 1] - c.qsl[sq], Ls = c.seq_lens[sq];
      const int nt = (qn + c.tile_tokens - 1) / c.tile_tokens;
      for (int t = tl; t < nt; t += lps)
        pv.plist[atomicAdd(&hist[bucket((prefill_tile_keys(c, Ls, qn, t) + 15) / 16)], 1)] = make_int2(sq, t);
    }
  }
}

// ---------------------------------------------------------------------------
// launch settings
// ---------------------------------------------------------------------------
// sets the kernel's shared-memory limit and gives its CTAs per SM
template <typename K>
static bool configure(K kern, int smem, int threads, int* occ_out) {
  if (smem > 48 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return false;
  int o = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&o, kern, threads, smem) != cudaSuccess || o < 1) return false;
  *occ_out = o;
  return true;
}

// CTAs per SM for a kernel that allocates tensor memory: the occupancy API
// answers 1 for any such kernel, so the count is taken from the kernel's
// registers and shared memory and the TMEM columns each CTA holds
template <typename K>
static bool configure_tmem(K kern, int smem, int threads, int tmem_cols, int* occ_out) {
  if (smem > 48 * 1024 && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return false;
  cudaFuncAttributes fa;
  int dev = 0, smem_sm = 0, reserved = 0, regs_sm = 0;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&smem_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&regs_sm, cudaDevAttrMaxRegistersPerMultiprocessor, dev) != cudaSuccess)
    return false;
  const int warps = (threads + 31) / 32;
  const int regs_warp = ((fa.numRegs * 32 + 255) / 256) * 256;  // allocated per warp in 256-register units
  const int by_regs = regs_sm / (regs_warp * ((warps + 3) / 4 * 4));  // and per group of four warps
  const int by_smem = smem_sm / (smem + fa.sharedSizeBytes + reserved);
  const int by_tmem = 512 / tmem_cols;
  const int o = min(by_regs, min(by_smem, by_tmem));
  if (o < 1) return false;
  *occ_out = o;
  return true;
}

}  // namespace kvint4
