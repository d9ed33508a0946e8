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
// everyone has loaded it.  The loads of the next chunk lie behind the stores of
// this one and are issued before them.

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

constexpr int kBins = 2048;
constexpr int kCopies = 4;  // histograms by lane: neighbouring masses share their upper bits, and with them a bin
constexpr int kCachedMasses = 40960;

template <int THREADS>
__global__ void __launch_bounds__(THREADS) evict_select_kernel(EvictArgs a, int cached) {
  constexpr int WARPS = THREADS / 32, PER = kBins / THREADS;
  extern __shared__ __align__(16) uint32_t sdyn[];
  uint32_t* const hist = sdyn;                    // [kCopies][kBins]
  uint32_t* const keys = sdyn + kCopies * kBins;  // [cached]
  __shared__ uint32_t s_warp[2][WARPS];
  __shared__ uint32_t s_bin, s_left;
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
  const int last = L - a.recent;        // candidates are [0, last); last > take
  const int take = a.budget - a.recent;
  const bool in_smem = last <= cached;
  auto key_at = [&](int p) { return in_smem ? keys[p] : mass_key(mass[p]); };

  // the take-th largest key and how many of its equals are taken
  uint32_t prefix = 0, mask = 0, left = take;
  if (take > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; pass++) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = pass == 2 ? 1023u : 2047u;
      for (int b = tid; b < kCopies * kBins; b += THREADS) hist[b] = 0;
      __syncthreads();
      uint32_t* const mine = hist + (lane & (kCopies - 1)) * kBins;
      if (pass == 0) {
#pragma unroll 4
        for (int p = tid; p < last; p += THREADS) {
          const uint32_t k = mass_key(mass[p]);
          if (in_smem) keys[p] = k;
          atomicAdd(mine + (k >> shift), 1u);
        }
      } else {
#pragma unroll 4
        for (int p = tid; p < last; p += THREADS) {
          const uint32_t k = key_at(p);
          if ((k & mask) == prefix) atomicAdd(mine + ((k >> shift) & bins), 1u);
        }
      }
      __syncthreads();
      // thread t owns bins [t PER, t PER + PER) counted from the top: sums of larger bins before it
      uint32_t c[PER], sum = 0;
#pragma unroll
      for (int e = 0; e < PER; e++) {
        const int b = kBins - 1 - (tid * PER + e);
        c[e] = 0;
#pragma unroll
        for (int x = 0; x < kCopies; x++) c[e] += hist[x * kBins + b];
        sum += c[e];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_warp[0][warp] = incl;
      __syncthreads();
      uint32_t before = incl - sum;
      for (int w = 0; w < warp; w++) before += s_warp[0][w];
#pragma unroll
      for (int e = 0; e < PER; e++) {
        if (before < left && left <= before + c[e]) {
          s_bin = kBins - 1 - (tid * PER + e);
          s_left = left - before;
        }
        before += c[e];
      }
      __syncthreads();
      prefix |= s_bin << shift;
      mask |= bins << shift;
      left = s_left;
      __syncthreads();
    }
  } else {
    if (in_smem) {
      for (int p = tid; p < last; p += THREADS) keys[p] = 0;
      __syncthreads();
    }
    prefix = 0xffffffffu;  // above every key (the largest is that of +infinity)
    left = 0;
  }

  // the kept positions in order: each warp owns a run of candidates
  const int run = (last + WARPS - 1) / WARPS, p0 = min(last, warp * run), p1 = min(last, p0 + run);
  uint32_t gt = 0, eq = 0;
#pragma unroll 2
  for (int p = p0 + lane; p < p1; p += 32) {
    const uint32_t k = key_at(p);
    gt += k > prefix;
    eq += k == prefix;
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_warp[0][warp] = gt;
    s_warp[1][warp] = eq;
  }
  __syncthreads();
  uint32_t gt_before = 0, eq_before = 0;
  for (int w = 0; w < warp; w++) {
    gt_before += s_warp[0][w];
    eq_before += s_warp[1][w];
  }
  const uint32_t below = (1u << lane) - 1;
#pragma unroll 2
  for (int p = p0; p < p1; p += 32) {
    const uint32_t k = p + lane < p1 ? key_at(p + lane) : 0u;
    const bool g = p + lane < p1 && k > prefix, e = p + lane < p1 && k == prefix;
    const uint32_t mg = __ballot_sync(0xffffffffu, g), me = __ballot_sync(0xffffffffu, e);
    const uint32_t rank = eq_before + __popc(me & below);
    if (g || (e && rank < left)) kept[gt_before + __popc(mg & below) + min(rank, left)] = p + lane;
    gt_before += __popc(mg);
    eq_before += __popc(me);
  }
  for (int p = tid; p < a.recent; p += THREADS) kept[take + p] = last + p;
  __syncthreads();  // kept is read below by other threads of the CTA
  // the masses go with them; the output may be the input, a chunk is loaded before it is stored
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

// what a warp needs to load its destination block of a chunk: lane r < 16 has row r's
struct MoveRow {
  int pos;    // position of the sequence, -1: none
  int block;  // its cache block, -1: none
};

__device__ __forceinline__ void move_barrier(int cluster) {
  if (cluster > 1)
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  else
    __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kMoveWarps * 32) evict_move_kernel(EvictArgs a, int cluster) {
  constexpr int CH = D / 16;   // 16-byte chunks per row
  constexpr int PER = D / 32;  // chunks per lane (16 rows)
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

  // the pipeline: positions two chunks ahead, their blocks and the destination
  // one ahead, then the rows
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
  struct Rows {
    uint4 x[PER];
    float scale;  // lane r < 16: the scale of row r's block; 0: the row is zeros
  };
  auto load = [&](const MoveRow& m, Rows& r) {
    r.scale = 0.f;
    if (m.block >= 0) {
      const float s = *const_cast<const volatile float*>(scales + (int64_t)m.block * a.num_kv_heads);
      if (fp8_scale_exponent(s) <= kFp8MaxExp) r.scale = s;
    }
#pragma unroll
    for (int j = 0; j < PER; j++) {
      const int c = lane + 32 * j, row = c / CH, col = c - row * CH;
      const int blk = __shfl_sync(0xffffffffu, m.block, row), pos = __shfl_sync(0xffffffffu, m.pos, row);
      r.x[j] = make_uint4(0, 0, 0, 0);
      if (blk >= 0)
        r.x[j] = __ldcg(reinterpret_cast<const uint4*>(codes + ((int64_t)blk * 16 + (pos & 15)) * row_bytes + col * 16));
    }
  };

  MoveRow m0{position(b0), -1};
  m0.block = block_of(m0.pos);
  MoveRow m1{position(b0 + step), -1};
  int to = target(b0), to1 = target(b0 + step);
  Rows r;
  load(m0, r);
  m1.block = block_of(m1.pos);
  int pos2 = position(b0 + 2 * step);
#pragma unroll 1
  for (int c0 = 0; c0 < nblk; c0 += step) {
    const int b = c0 + b0;
    // ---- the block's largest magnitude, and with it every load of the chunk ----
    float rs[PER];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < PER; j++) {
      const int row = (lane + 32 * j) / CH;
      rs[j] = __shfl_sync(0xffffffffu, r.scale, row);
      if (rs[j] == 0.f) r.x[j] = make_uint4(0, 0, 0, 0);
      const uint32_t m = __vmaxu4(__vmaxu4(r.x[j].x & 0x7f7f7f7fu, r.x[j].y & 0x7f7f7f7fu),
                                  __vmaxu4(r.x[j].z & 0x7f7f7f7fu, r.x[j].w & 0x7f7f7f7fu));
      uint32_t code = max(max(m & 0xffu, (m >> 8) & 0xffu), max((m >> 16) & 0xffu, m >> 24));
      code = min(code, 0x7eu);  // a NaN code takes no part
      const uint32_t f = e4m3x2_to_f16x2(code);
      top = max(top, __float_as_uint(__half2float(__ushort_as_half((unsigned short)(f & 0xffffu))) * rs[j]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    // smallest k in range with top <= 448 2^k = 1.75 2^(8 + k)
    const int k = min(max((int)(top >> 23) - 127 - 8 + ((top & 0x7fffffu) > 0x600000u), kFp8MinExp), kFp8MaxExp);
    const int pos_of_row = m0.pos;
    Rows next;
    load(m1, next);
    const int blk2 = block_of(pos2), to2 = target(b + 2 * step), pos3 = position(b + 3 * step);
    move_barrier(cluster);  // every row of this chunk has been read
    // rows that all stay where they are are left alone
    const bool here = __all_sync(0xffffffffu, pos_of_row < 0 || (pos_of_row == b * 16 + lane && m0.block == to));
    if (b < nblk && !here) {
      if (to < 0 || to >= a.num_blocks) {
        if (lane == 0) flag(a.dev_status, KV_INT4_DEV_BAD_BLOCK);
      } else {
        uint8_t* const dst = codes + (int64_t)to * 16 * row_bytes;
#pragma unroll
        for (int j = 0; j < PER; j++) {
          const int c = lane + 32 * j, row = c / CH, col = c - row * CH;
          if (b * 16 + row >= n) continue;
          const int shift = rs[j] == 0.f ? 0 : exp_of(rs[j]) - k;
          if (shift != 0) {
            const float f = exp2_int(shift);
            uint32_t* w = reinterpret_cast<uint32_t*>(&r.x[j]);
#pragma unroll
            for (int e = 0; e < 4; e++) {
              uint32_t lo, hi;
              e4m3x4_to_f16x2(w[e], lo, hi);
              const float2 p0 = __half22float2(*reinterpret_cast<__half2*>(&lo));
              const float2 p1 = __half22float2(*reinterpret_cast<__half2*>(&hi));
              w[e] = f32x4_to_e4m3(p0.x * f, p0.y * f, p1.x * f, p1.y * f);
            }
          }
          *reinterpret_cast<uint4*>(dst + row * row_bytes + col * 16) = r.x[j];
        }
        if (lane == 0) scales[(int64_t)to * a.num_kv_heads] = exp2_int(k);
      }
    }
    r = next;
    m0 = m1;
    m1 = MoveRow{pos2, blk2};
    pos2 = pos3;
    to = to1;
    to1 = to2;
  }
}

template <int D>
int launch_t(const EvictArgs& a, cudaStream_t stream) {
  const int dev = current_device();
  const int sms = sm_count(dev);
  const int64_t pairs = (int64_t)a.num_seqs * a.num_kv_heads;
  // few masses: small CTAs (their barriers cost less), many: one CTA's threads share the passes
  const int most = a.mass_len < (int64_t)a.max_blocks_per_seq * 16 ? a.mass_len : a.max_blocks_per_seq * 16;
  const int cached = most < kCachedMasses ? most : kCachedMasses;
  const size_t smem = (size_t)(kCopies * kBins + cached) * 4;
  constexpr int kMostSmem = (kCopies * kBins + kCachedMasses) * 4;
  static PerContext<int> attr;
  int set = 0;
  if (!attr.get(dev, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(evict_select_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) == cudaSuccess &&
               cudaFuncSetAttribute(evict_select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) == cudaSuccess;
      }, &set))
    return KV_INT4_ERR_CUDA;
  int e = launch_pdl(most <= 2048 ? evict_select_kernel<256> : evict_select_kernel<1024>, dim3((unsigned)pairs),
                     most <= 2048 ? 256 : 1024, smem, stream, 1, a, cached);
  if (e) return e;
  // as many CTAs per task as run at once and have a block per warp
  const int64_t tasks = 2 * pairs;
  const int64_t blocks = ((int64_t)(a.budget < most ? a.budget : most) + 15) / 16;
  int cluster = 1;
  while (cluster < 8 && 2 * tasks * cluster <= 2ll * sms && blocks > (int64_t)kMoveWarps * cluster) cluster *= 2;
  return launch_pdl(evict_move_kernel<D>, dim3((unsigned)(tasks * cluster)), kMoveWarps * 32, 0, stream, cluster, a, cluster);
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
