// kv_fp8_evict: per (sequence, kv head), the `budget` positions that stay in an
// FP8 cache (the last `recent` ones and the heaviest others), moved to the front.
//
// Two kernels.  Select finds the positions: a radix select over the masses as
// ordered 32-bit keys (three passes of 11, 11 and 10 bits over histograms in
// shared memory, the masses held there too as far as they fit), then one ordered
// pass that writes the kept positions in ascending order; equal masses go to the
// lowest positions.  Move gathers the kept rows of K and of V, a warp for the 16
// rows of a destination block: their largest magnitude gives the block's scale by
// the rule of kv_fp8_write, and codes follow their new scale by a power of two.
//
// Destination blocks may be the sequence's own.  Row j takes position kept[j] >=
// j, so a row may be overwritten once every destination row at or before it has
// been read: the CTA (or cluster) of a (sequence, kv head, K or V) takes its
// destination blocks in order, a chunk at a time, and no one stores a chunk before
// everyone has loaded it.  The rows of the next chunks lie behind the stores of
// this one and are on their way (cp.async) before them.
//
// Measured: 32 sequences of 6000 to 8192 positions to 2048, 8 heads of 128, to other
// blocks: 73 us.  Select takes 13 of them, instructions of its passes over 7000 masses
// per CTA (18 when the first pass's bin was listed after a count, and the last pass
// compared keys and ranked equals everywhere).  Move takes 59: 268 MB, 4.5 TB/s of
// 128-byte rows gathered; four warps per CTA in clusters of two took 66.

#include <cuda_runtime.h>

#include "../../include/kvint4.h"
#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace kvint4 {
namespace {

// whether sequence i can be worked on
__device__ __forceinline__ bool evict_seq_ok(const EvictArgs& a, int L) {
  return L >= 0 && L <= a.mass_len && (int64_t)L <= (int64_t)a.max_blocks_per_seq * 16;
}

// a mass as a key that orders like it: NaN below everything, both zeros the same
__device__ __forceinline__ uint32_t mass_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 + 0 = 0
  return x != x ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// the mass with a key above 0 (of the zeros: 0)
__device__ __forceinline__ float key_mass(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

constexpr int kBins = 2048;
constexpr int kCachedMasses = 40960;
constexpr int kListed = 1024;

template <int THREADS>
struct Select {
  // histograms by lane: neighbouring masses share their upper bits, and with them a
  // bin (few masses: one, which is sooner cleared and summed)
  static constexpr int COPIES = THREADS > 256 ? 4 : 1;
  static size_t smem(int cached) { return (size_t)(COPIES * kBins + cached) * 4; }
};

template <int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 2 : 4) evict_select_kernel(EvictArgs a, int cached) {
  constexpr int WARPS = THREADS / 32, PER = kBins / THREADS, COPIES = Select<THREADS>::COPIES;
  extern __shared__ __align__(16) uint32_t sdyn[];
  uint32_t* const hist = sdyn;                                            // [COPIES][kBins]
  float* const masses = reinterpret_cast<float*>(sdyn + COPIES * kBins);  // [cached]
  __shared__ uint32_t s_warp[2][32], s_key[kListed];
  __shared__ int s_pos[kListed];
  __shared__ uint32_t s_bin, s_left, s_count, s_listed;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i = blockIdx.x / a.num_kv_heads, h = blockIdx.x - i * a.num_kv_heads;
  const int L = a.seq_lens[i];
  if (!evict_seq_ok(a, L)) {
    if (tid == 0 && h == 0) {
      flag(a.dev_status, KV_INT4_DEV_BAD_SEQ);
      a.new_lens[i] = L;
    }
    return;
  }
  const int n = min(L, a.budget);
  if (tid == 0 && h == 0) a.new_lens[i] = n;
  const float* mass = a.mass + i * a.mass_seq_stride + h * a.mass_head_stride;
  float* out = a.mass_out + i * a.out_seq_stride + h * a.out_head_stride;
  int32_t* kept = a.kept + (int64_t)blockIdx.x * a.budget;
  if (L <= a.budget) {
    for (int p = tid; p < n; p += THREADS) {
      kept[p] = p;
      out[p] = mass[p];
    }
    return;
  }
  const int last = L - a.recent;  // candidates are [0, last); last > take
  const int take = a.budget - a.recent;
  const bool in_smem = L <= cached;
  auto mass_at = [&](int p) { return in_smem ? masses[p] : mass[p]; };
  // histograms of COPIES or, of the list, one: cleared by everyone
  auto clear = [&](int copies) {
    for (int b = tid; b < copies * kBins / 4; b += THREADS) reinterpret_cast<uint4*>(hist)[b] = make_uint4(0, 0, 0, 0);
  };
  uint32_t* const lane_hist = hist + (lane & (COPIES - 1)) * kBins;
  clear(COPIES);
  for (int w = WARPS + tid; w < 32; w += THREADS) s_warp[0][w] = s_warp[1][w] = 0;  // warps that are not there
  if (tid == 0) s_listed = 0;
  __syncthreads();
  // the masses into shared memory, and with them the first pass's counts
  {
    constexpr int U = 8;
#pragma unroll 1
    for (int q = 0; q < L; q += U * THREADS) {
      float x[U];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int p = q + u * THREADS + tid;
        x[u] = p < L ? mass[p] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int p = q + u * THREADS + tid;
        if (in_smem && p < L) masses[p] = x[u];
        if (p < last) atomicAdd(lane_hist + (mass_key(x[u]) >> 21), 1u);
      }
    }
  }
  // sum of x over the warps before this one, of values that lane 0 of each has left
  auto before_warp = [&](const uint32_t* x) {
    const uint32_t mine = x[lane];
    uint32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    return __shfl_sync(0xffffffffu, incl - mine, warp);
  };

  // Each warp owns a run of candidates in the ordered pass at the end.  The
  // take-th largest key and how many of its equals are taken, bin by bin; the keys of
  // the first pass's bin are few as a rule and are listed, so that the other passes
  // touch no more than those
  const int run = (last + WARPS - 1) / WARPS, p0 = min(last, warp * run), p1 = min(last, p0 + run);
  uint32_t prefix = 0, mask = 0, left = take;
  uint32_t listed = 0;  // candidates on the list, 0: there is none
  uint32_t gt = 0, eq = 0;
  if (take > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; pass++) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = pass == 2 ? 1023u : 2047u;
      const int copies = listed ? 1 : COPIES;
      if (pass > 0) {
        clear(copies);
        __syncthreads();
        if (listed) {
          for (uint32_t x = tid; x < listed; x += THREADS) {
            const uint32_t k = s_key[x];
            if ((k & mask) == prefix) atomicAdd(hist + ((k >> shift) & bins), 1u);
          }
        } else {
#pragma unroll 4
          for (int p = tid; p < last; p += THREADS) {
            const uint32_t k = mass_key(mass_at(p));
            if ((k & mask) == prefix) atomicAdd(lane_hist + ((k >> shift) & bins), 1u);
          }
        }
      }
      __syncthreads();
      // thread t owns bins [t PER, t PER + PER) counted from the top: sums of larger bins before it
      uint32_t c[PER], sum = 0;
#pragma unroll
      for (int e = 0; e < PER; e += 4) {
        const uint32_t* const four = hist + kBins - 4 - (tid * PER + e);
        uint4 v = *reinterpret_cast<const uint4*>(four);
        for (int x = 1; x < copies; x++) {
          const uint4 w = *reinterpret_cast<const uint4*>(four + x * kBins);
          v = make_uint4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
        }
        c[e] = v.w, c[e + 1] = v.z, c[e + 2] = v.y, c[e + 3] = v.x;
        sum += v.x + v.y + v.z + v.w;
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_warp[0][warp] = incl;
      __syncthreads();
      uint32_t before = incl - sum + before_warp(s_warp[0]);
#pragma unroll
      for (int e = 0; e < PER; e++) {
        if (before < left && left <= before + c[e]) {
          s_bin = kBins - 1 - (tid * PER + e);
          s_left = left - before;
          s_count = c[e];
        }
        before += c[e];
      }
      __syncthreads();
      prefix |= s_bin << shift;
      mask |= bins << shift;
      left = s_left;
      if (pass == 0 && s_count <= kListed) {
        listed = s_count;
#pragma unroll 4
        for (int p = p0 + lane; p < p1; p += 32) {
          const uint32_t k = mass_key(mass_at(p)), kb = k & mask;
          gt += kb > prefix;
          if (kb == prefix) {
            const uint32_t x = atomicAdd(&s_listed, 1u);
            s_key[x] = k;
            s_pos[x] = p;
          }
        }
        __syncthreads();
      }
    }
  } else {
    prefix = 0xffffffffu;  // above every key (the largest is that of +infinity)
    left = 0;
  }
  __syncthreads();  // the masses in shared memory; the last sums and the list have been read

  // larger and equal keys of every warp's run
  if (!listed) {
#pragma unroll 4
    for (int p = p0 + lane; p < p1; p += 32) {
      const uint32_t k = mass_key(mass_at(p));
      gt += k > prefix;
      eq += k == prefix;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_warp[0][warp] = gt;
    s_warp[1][warp] = eq;
  }
  __syncthreads();
  if (listed) {
    for (uint32_t x = tid; x < listed; x += THREADS)
      if (s_key[x] >= prefix) atomicAdd(&s_warp[s_key[x] == prefix][s_pos[x] / run], 1u);
    __syncthreads();
  }
  const uint32_t gt_before = before_warp(s_warp[0]), eq_before = before_warp(s_warp[1]);
  eq = s_warp[1][warp];
  uint32_t at = gt_before + min(eq_before, left);  // the run's place in what is kept
  const uint32_t below = (1u << lane) - 1;
  const bool all = eq_before + eq <= left, none = eq == 0 || eq_before >= left;
  if (prefix != 0u && (all || none)) {
    // of the run's equal masses all are kept, or none: one comparison of floats.
    // Four masses per lane are loaded before the ballots of the first are used
    const float least = prefix == 0xffffffffu ? __uint_as_float(0x7f800000u) : key_mass(prefix);
    constexpr int U = 4;
#pragma unroll 1
    for (int q = p0 + lane; q - lane < p1; q += 32 * U) {
      float x[U];
      uint32_t m[U];
#pragma unroll
      for (int u = 0; u < U; u++) x[u] = q + 32 * u < p1 ? mass_at(q + 32 * u) : __uint_as_float(0x7fffffffu);
#pragma unroll
      for (int u = 0; u < U; u++) m[u] = __ballot_sync(0xffffffffu, none ? x[u] > least : x[u] >= least);
#pragma unroll
      for (int u = 0; u < U; u++) {
        if (m[u] >> lane & 1) {
          const uint32_t j = at + __popc(m[u] & below);
          kept[j] = q + 32 * u;
          if (in_smem) out[j] = x[u];
        }
        at += __popc(m[u]);
      }
    }
  } else {
    // the run in which the last of the equal masses is kept, or NaN among them
    uint32_t rank = eq_before;
#pragma unroll 1
    for (int q = p0; q < p1; q += 32) {
      const int p = q + lane;
      const float x = p < p1 ? mass_at(p) : 0.f;
      const uint32_t k = p < p1 ? mass_key(x) : 0u;
      const bool e = p < p1 && k == prefix;
      const uint32_t me = __ballot_sync(0xffffffffu, e);
      const bool keep = p < p1 && (k > prefix || (e && rank + __popc(me & below) < left));
      const uint32_t m = __ballot_sync(0xffffffffu, keep);
      if (keep) {
        const uint32_t j = at + __popc(m & below);
        kept[j] = p;
        if (in_smem) out[j] = x;
      }
      at += __popc(m);
      rank += __popc(me);
    }
  }
  for (int p = tid; p < a.recent; p += THREADS) {
    kept[take + p] = last + p;
    if (in_smem) out[take + p] = masses[last + p];
  }
  if (in_smem) return;
  // masses that did not fit go with their positions now; the output may be the input,
  // a chunk is loaded before it is stored
  __syncthreads();  // kept is read below by other threads of the CTA
  constexpr int U = 4;
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += U * THREADS) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int j = j0 + u * THREADS + tid;
      x[u] = j < n ? *const_cast<const volatile float*>(mass + kept[j]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int j = j0 + u * THREADS + tid;
      if (j < n) out[j] = x[u];
    }
  }
}

constexpr int kMoveWarps = 8;

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
// four f16 to E4M3, nearest even, saturating at +-448
__device__ __forceinline__ uint32_t f16x4_to_e4m3(__half2 lo, __half2 hi) {
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n "
      "mov.b32 %0, {a, b};\n}\n"
      : "=r"(r)
      : "r"(*reinterpret_cast<uint32_t*>(&lo)), "r"(*reinterpret_cast<uint32_t*>(&hi)));
  return r;
}

__device__ __forceinline__ void move_barrier(int cluster) {
  if (cluster > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  else
    __syncthreads();
}

// rows in flight per warp, in chunks of a destination block each
constexpr int kMoveAhead = 2;
template <int D>
constexpr int kMovePerSm = D <= 128 ? 4 : 2;
template <int D>
constexpr int kMoveSmem = kMoveWarps * (kMoveAhead + 1) * 16 * D;

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32, kMovePerSm<D>) evict_move_kernel(EvictArgs a, int cluster) {
  constexpr int CH = D / 16;   // 16-byte chunks per row
  constexpr int PER = D / 32;  // chunks per lane (16 rows)
  constexpr int SLOTS = kMoveAhead + 1;
  extern __shared__ __align__(16) uint8_t srows[];  // [warp][SLOTS][16 rows]; a lane reads what it copied
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int task = blockIdx.x / cluster, rank = blockIdx.x - task * cluster;
  const int h = task % a.num_kv_heads, rest = task / a.num_kv_heads;
  const int i = rest >> 1;
  const bool isv = rest & 1;
  const int L = a.seq_lens[i];
  if (!evict_seq_ok(a, L)) return;  // the whole cluster
  const int n = min(L, a.budget);
  const int nblk = (n + 15) >> 4;
  const int32_t* kept = a.kept + ((int64_t)i * a.num_kv_heads + h) * a.budget;
  const int32_t* table = a.block_table + (int64_t)i * a.max_blocks_per_seq;
  const int32_t* into = a.dst_block_table + (int64_t)i * a.dst_max_blocks;
  uint8_t* const codes = (isv ? a.v_cache : a.k_cache) + (int64_t)h * D;
  float* const scales = (isv ? a.v_scale : a.k_scale) + h;
  const int64_t row_bytes = (int64_t)a.num_kv_heads * D;
  const int step = kMoveWarps * cluster;  // blocks per chunk
  const int b0 = rank * kMoveWarps + warp;
  uint8_t* const ring = srows + warp * SLOTS * 16 * D;

  // the pipeline, by chunk: positions, a chunk later their blocks, then the rows
  auto position = [&](int b) { return lane < 16 && b * 16 + lane < n ? kept[b * 16 + lane] : -1; };
  auto block_of = [&](int pos) {
    int blk = -1;
    if (pos >= 0) {
      blk = table[pos >> 4];
      if (blk < 0 || blk >= a.num_blocks) {
        flag(a.dev_status, KV_INT4_DEV_BAD_BLOCK);
        blk = -1;
      }
    }
    return blk;
  };
  auto target = [&](int b) { return b < nblk ? into[b] : -1; };
  // the rows' copies, and of lane r < 16 the scale of row r's block
  auto load = [&](int pos, int block, int slot) {
    float s = 0.f;
    if (block >= 0) s = *const_cast<const volatile float*>(scales + (int64_t)block * a.num_kv_heads);
#pragma unroll
    for (int j = 0; j < PER; j++) {
      const int c = lane + 32 * j, row = c / CH, col = c - row * CH;
      const int blk = __shfl_sync(0xffffffffu, block, row), p = __shfl_sync(0xffffffffu, pos, row);
      const uint8_t* src = codes + (blk >= 0 ? ((int64_t)blk * 16 + (p & 15)) * row_bytes + col * 16 : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_addr(ring + slot * 16 * D + c * 16)), "l"(src),
                   "r"(blk >= 0 ? 16 : 0));
    }
    cp_async_commit();
    return s;
  };

  // chunks now, next, and the one after, whose rows are not yet under way
  int pos0 = position(b0), pos1 = position(b0 + step), pos2 = position(b0 + 2 * step), pos3 = position(b0 + 3 * step);
  int blk0 = block_of(pos0), blk1 = block_of(pos1);
  int to0 = target(b0), to1 = target(b0 + step);
  float sc0 = load(pos0, blk0, 0);
  int blk2 = block_of(pos2);
  float sc1 = load(pos1, blk1, 1);
  int slot = 0;
#pragma unroll 1
  for (int c0 = 0; c0 < nblk; c0 += step) {
    const int b = c0 + b0;
    const float sc2 = load(pos2, blk2, slot == 0 ? 2 : slot - 1);
    const int blk3 = block_of(pos3), to2 = target(b + 2 * step), pos4 = position(b + 4 * step);
    cp_async_wait<kMoveAhead>();  // this chunk's rows
    // ---- the block's largest magnitude, and with it every load of the chunk ----
    const float scale = fp8_scale_exponent(sc0) <= kFp8MaxExp ? sc0 : 0.f;  // 0: the row is zeros
    uint4 x[PER];
    float rs[PER];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < PER; j++) {
      const int row = (lane + 32 * j) / CH;
      rs[j] = __shfl_sync(0xffffffffu, scale, row);
      x[j] = *reinterpret_cast<const uint4*>(ring + slot * 16 * D + (lane + 32 * j) * 16);
      if (rs[j] == 0.f) x[j] = make_uint4(0, 0, 0, 0);
      // code magnitudes order as integers: even and odd bytes as 16-bit lanes
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; e++) m = __vmaxu2(m, __vmaxu2(w[e] & 0x007f007fu, (w[e] >> 8) & 0x007f007fu));
      m = min(max(m & 0xffffu, m >> 16), 0x7eu);  // a NaN code counts as the largest number
      top = max(top, __float_as_uint(__half2float(__low2half(as_half2(e4m3x2_to_f16x2(m)))) * rs[j]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    // smallest k in range with top <= 448 2^k = 1.75 2^(8 + k)
    const int k = min(max((int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u), kFp8MinExp), kFp8MaxExp);
    move_barrier(cluster);  // every row of this chunk has been read
    // rows that all stay where they are are left alone
    const bool here = __all_sync(0xffffffffu, pos0 < 0 || (pos0 == b * 16 + lane && blk0 == to0));
    if (b < nblk && !here) {
      if (to0 < 0 || to0 >= a.num_blocks) {
        if (lane == 0) flag(a.dev_status, KV_INT4_DEV_BAD_BLOCK);
      } else {
        uint8_t* const dst = codes + (int64_t)to0 * 16 * row_bytes;
#pragma unroll
        for (int j = 0; j < PER; j++) {
          const int c = lane + 32 * j, row = c / CH, col = c - row * CH;
          // Codes * 2^shift in f16, exact wherever the code that comes out depends on it:
          // below 2^-24 all become zeros; a row that needs more than 2^15 has codes of
          // 2^-7 at most, and takes two steps
          uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
          const int shift = rs[j] == 0.f ? 0 : max(exp_of(rs[j]) - k, -24);
          if (shift != 0) {
            const __half2 s0 = __float2half2_rn(exp2_int(min(shift, 15)));
            const __half2 s1 = __float2half2_rn(exp2_int(min(max(shift - 15, 0), 15)));
#pragma unroll
            for (int e = 0; e < 4; e++) {
              uint32_t lo, hi;
              e4m3x4_to_f16x2(w[e], lo, hi);
              __half2 l2 = __hmul2(as_half2(lo), s0), h2 = __hmul2(as_half2(hi), s0);
              if (shift > 15) {
                l2 = __hmul2(l2, s1);
                h2 = __hmul2(h2, s1);
              }
              w[e] = f16x4_to_e4m3(l2, h2);
            }
          }
          if (b * 16 + row < n) *reinterpret_cast<uint4*>(dst + row * row_bytes + col * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (lane == 0) scales[(int64_t)to0 * a.num_kv_heads] = exp2_int(k);
      }
    }
    pos0 = pos1, pos1 = pos2, pos2 = pos3, pos3 = pos4;
    blk0 = blk1, blk1 = blk2, blk2 = blk3;
    to0 = to1, to1 = to2;
    sc0 = sc1, sc1 = sc2;
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
  }
  cp_async_wait<0>();
}

template <int D>
int launch_t(const EvictArgs& a, cudaStream_t stream) {
  const int dev = current_device();
  const int sms = sm_count(dev);
  const int64_t pairs = (int64_t)a.num_seqs * a.num_kv_heads;
  const int most = a.mass_len < (int64_t)a.max_blocks_per_seq * 16 ? a.mass_len : a.max_blocks_per_seq * 16;
  const int cached = most < kCachedMasses ? most : kCachedMasses;
  static PerContext<int> attr;
  int set = 0;
  if (!attr.get(dev, [](int* v) {
        *v = 1;
        auto most_smem = [](auto kern, size_t bytes) {
          return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
        };
        return most_smem(evict_move_kernel<D>, kMoveSmem<D>) && most_smem(evict_select_kernel<256>, Select<256>::smem(kCachedMasses)) &&
               most_smem(evict_select_kernel<512>, Select<512>::smem(kCachedMasses));
      }, &set))
    return KV_INT4_ERR_CUDA;
  const bool small = most <= 2048;
  int e = launch_pdl(small ? evict_select_kernel<256> : evict_select_kernel<512>, dim3((unsigned)pairs), small ? 256 : 512,
                     small ? Select<256>::smem(cached) : Select<512>::smem(cached), stream, 1, a, cached);
  if (e) return e;
  // as many CTAs per task as run at once and have a block per warp
  const int64_t tasks = 2 * pairs;
  const int64_t blocks = ((int64_t)(a.budget < most ? a.budget : most) + 15) / 16;
  int cluster = 1;
  while (cluster < 8 && 2 * tasks * cluster <= (int64_t)kMovePerSm<D> * sms && blocks > (int64_t)kMoveWarps * cluster) cluster *= 2;
  return launch_pdl(evict_move_kernel<D>, dim3((unsigned)(tasks * cluster)), kMoveWarps * 32, kMoveSmem<D>, stream, cluster, a, cluster);
}

}  // namespace

int launch_evict_fp8(const EvictArgs& a, cudaStream_t stream) {
  switch (a.head_size) {
    case 64: return launch_t<64>(a, stream);
    case 96: return launch_t<96>(a, stream);
    case 128: return launch_t<128>(a, stream);
    case 192: return launch_t<192>(a, stream);
    case 256: return launch_t<256>(a, stream);
    default: return KV_INT4_ERR_HEAD_SIZE;
  }
}

}  // namespace kvint4
