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
  int32_t* plan;      // [0] n_dseq, [1] n_prefill_items, [2] prefill work counter, [3] n_pseq
  int4* dseq;         // decode sequences in order: (sequence id, seq_len, first query token, q_len)
  int64_t* dprefix;
  int2* ptab;         // prefill sequences in order: (seq id, index of its first item); [n_pseq].y = items
  int2* plist;        // prefill (sequence, tile) pairs, longest first; pair i gives items i Hkv .. i Hkv + Hkv - 1
  __half* qrot;
  float* direct_o;
  float* direct_ml;
  float* warp_o;
  float* warp_ml;
};

static PlanView plan_view(void* ws, const WorkspaceLayout& L) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  PlanView v;
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
};

// floor(n / d) for 0 <= n, 0 < d: one 32-bit division when both fit (the
// usual case for schedule arithmetic), the 64-bit routine otherwise
__device__ __forceinline__ long long div_nn(long long n, long long d) {
  return ((n | d) >> 31) == 0 ? (long long)((uint32_t)n / (uint32_t)d) : n / d;
}

// first key position visible to the query at position qpos
__device__ __forceinline__ int window_lo(const Common& c, int qpos) {
  return c.window > 0 ? max(0, qpos - c.window + 1) : 0;
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

// The schedule, by one CTA of kPrepThreads threads.
template <bool ANY_LEN>
__device__ void build_schedule(const Common& c, const PlanView& pv) {
  __shared__ int32_t s_i32[kPrepThreads / 32];
  __shared__ long long s_i64[kPrepThreads / 32];
  int n_dseq = 0, n_pseq = 0;
  long long dpre = 0, n_items = 0;
  for (int base = 0; base < c.num_seqs; base += kPrepThreads) {
    const int s = base + threadIdx.x;
    int kind = 0, nblk = 0, ntiles = 0, ql = 0, L = 0, q0 = 0;
    if (s < c.num_seqs) {
      q0 = c.qsl[s];
      L = c.seq_lens[s];
      ql = c.qsl[s + 1] - q0;
      if (!schedule_seq_ok<ANY_LEN>(c, q0, ql, L)) {
        flag(c.status, KV_INT4_DEV_BAD_SEQ);
      } else if (ql > 0) {
        kind = is_decode_kind(ql, c) ? 1 : 2;
        nblk = (L + 15) / 16;
        if (kind == 2) ntiles = (ql + c.tile_tokens - 1) / c.tile_tokens;
      }
    }
    int tot_a, tot_p;
    long long tot_b, tot_c;
    const int ex_a = block_exclusive_scan<int>(kind == 1, &tot_a, s_i32);
    const int npos = kind == 1 ? (nblk - first_block(c, L, ql) + c.np - 1) / c.np : 0;
    const long long ex_b = block_exclusive_scan<long long>(npos, &tot_b, s_i64);
    const int ex_p = block_exclusive_scan<int>(kind == 2, &tot_p, s_i32);
    const long long ex_c = block_exclusive_scan<long long>((long long)ntiles * c.hkv, &tot_c, s_i64);
    if (kind == 1) {
      pv.dseq[n_dseq + ex_a] = make_int4(s, L, q0, ql);
      pv.dprefix[n_dseq + ex_a] = dpre + ex_b;
    } else if (kind == 2) {
      // the prefill kernel expands (tile, kv head) items from this table
      pv.ptab[n_pseq + ex_p] = make_int2(s, (int)min(n_items + ex_c, (long long)INT_MAX));
    }
    n_dseq += tot_a;
    dpre += tot_b;
    n_pseq += tot_p;
    n_items += tot_c;
  }
  if (threadIdx.x == 0) {
    pv.dprefix[n_dseq] = dpre;
    pv.plan[0] = n_dseq;
    // more items than the workspace was sized for only happens with
    // inconsistent query_start_loc: the prefill part is dropped and flagged
    const bool over = n_items > c.max_items || n_items > INT_MAX;
    if (over) flag(c.status, KV_INT4_DEV_BAD_SEQ);
    pv.ptab[n_pseq] = make_int2(-1, over ? 0 : (int)n_items);
    pv.plan[1] = over ? 0 : (int)n_items;
    pv.plan[2] = 0;
    pv.plan[3] = n_pseq;
  }
  // the prefill (sequence, tile) pairs, longest first: a counting sort over
  // buckets of 16-key blocks (descending), so that the longest items start
  // first and the shortest fill the end of the launch (within a bucket the
  // order is arbitrary; every item computes the same rows either way)
  constexpr int kBuckets = 2048;
  __shared__ int hist[kBuckets];
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
