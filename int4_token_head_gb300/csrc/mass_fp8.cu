// kv_fp8_attention_mass: the attention weight that every position of an FP8
// cache receives from the call's queries.
//
//   w_p = sum over the query rows r of the position's kv head that see it of
//         2^(t_rp - lse_r log2 e),  t_rp = softmax_scale log2 e 2^kk_b (q_r . ck_p)
//
// The rows' denominators are known, so nothing is carried from key to key: a
// warp takes 16-key blocks of one kv head and needs no other warp's results.

#include <cuda.h>
#include <cuda_runtime.h>
#include <float.h>

#include <type_traits>

#include "../../include/kvint4.h"
#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"
#include "schedule.cuh"

namespace kvint4 {
namespace {

#include "attention_fp8.cuh"

constexpr int kMassCols = 32;  // query rows staged at once

struct MassParams {
  MassArgs a;
  int group, hg;      // q heads per kv head; kv heads per CTA
  int warp_blocks;    // 16-key blocks per warp
  int few_groups;     // column groups of eight rows that mass_few_kernel stages per head
  float qscale;       // softmax_scale log2 e
  FastDiv by_group{1}, by_groups{1}, by_chunks{1};
};

__device__ __forceinline__ bool mass_seq_ok(const MassArgs& a, int q0, int ql, int L) {
  return q0 >= 0 && ql >= 0 && (int64_t)q0 + ql <= a.num_q_tokens && ql <= a.max_query_len && L >= ql &&
         L <= a.max_seq_len && L <= a.mass_len && (int64_t)L <= (int64_t)a.max_blocks_per_seq * 16;
}

// the sequence's work belongs to the kernel for few query rows
__device__ __forceinline__ bool few_rows(const MassParams& p, int ql) { return (int64_t)ql * p.group <= kMassCols; }

// A column group of eight query rows r0 .. r0 + 7 of kv head `head`, staged by a
// warp as f16 B fragments (a row divided by the power of two of its largest
// magnitude: exact but for elements 2^-14 of it) in the order of dimensions in
// which a lane holds codes: lane (g, cq) word s has row g's elements kdim(cq, s) ..
// + 3.  Rows that are not there get a weight of 0.
template <int D, typename Dim>
__device__ __forceinline__ void stage_rows(const MassParams& p, int q0, int head, int r0, int rows, uint2* frag,
                                           float2* row, Dim&& kdim) {
  const MassArgs& a = p.a;
  constexpr int KSTEPS = D / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, cq = lane & 3;
  const int r = r0 + g;
  const bool ok = r < rows;
  const int j = ok ? r / p.group : 0, jj = ok ? r - j * p.group : 0;
  const int hq = head * p.group + jj;
  const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(q0 + j) * a.q_stride + (int64_t)hq * D;
  const float l = ok ? a.lse[(int64_t)(q0 + j) * a.lse_stride + hq] : INFINITY;
  uint2 v[KSTEPS];
  uint32_t am = 0;
#pragma unroll
  for (int s = 0; s < KSTEPS; s++) v[s] = ok ? *reinterpret_cast<const uint2*>(src + kdim(cq, s)) : make_uint2(0, 0);
#pragma unroll
  for (int s = 0; s < KSTEPS; s++) am = __vmaxu2(am, __vmaxu2(v[s].x & 0x7fff7fffu, v[s].y & 0x7fff7fffu));
  am = max(am & 0xffffu, am >> 16);
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
  am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
  const int e = min(max((int)(am >> 7) - 127, -126), 126);
  const float mul = exp2_int(-e);
#pragma unroll
  for (int s = 0; s < KSTEPS; s++)
    frag[s * 32 + lane] = make_uint2(pack_f16x2(bf16lo_to_f32(v[s].x) * mul, bf16hi_to_f32(v[s].x) * mul),
                                     pack_f16x2(bf16lo_to_f32(v[s].y) * mul, bf16hi_to_f32(v[s].y) * mul));
  if (cq == 0) row[g] = make_float2(p.qscale * exp2_int(e), fabsf(l) == INFINITY ? -INFINITY : -l * kLog2e);
}

// Few query rows (kMassCols per kv head at most): memory-bound.  A warp streams
// 16-key blocks of one kv head from global memory straight into registers: a lane
// holds whole 16-byte chunks cq, cq + 4, ... of rows g and g + 8 (a quarter of the
// row at 96), which are MMA A fragments once converted, as the order of dimensions
// within a product is free.  U blocks are in flight per warp.
// 32 sequences of 32768 positions, 32/8 heads of 128: 190 us, 6.0 TB/s (0.90 of a
// copy's).
template <int D>
struct MassFew {
  static constexpr int KSTEPS = D / 16;
  static constexpr int U = D <= 128 ? 4 : 2;
  static constexpr bool WIDE = D % 64 == 0;
  __device__ static __forceinline__ int kdim(int cq, int s) {
    return WIDE ? 16 * (cq + 4 * (s >> 2)) + 4 * (s & 3) : cq * (D / 4) + 4 * s;
  }
  static size_t smem(int hg, int groups) { return (size_t)hg * groups * 8 * (D * 2 + 8); }
};

template <int D>
__global__ void __launch_bounds__(128, 4) mass_few_kernel(MassParams p) {
  using F = MassFew<D>;
  constexpr int KSTEPS = F::KSTEPS, U = F::U;
  extern __shared__ __align__(16) uint8_t smem[];
  const MassArgs& a = p.a;
  const int HG = p.hg, WPH = 4 / HG;  // warps per head
  const int CG = p.few_groups;
  uint2* const sq = reinterpret_cast<uint2*>(smem);                            // [hg][CG][KSTEPS][32]
  float2* const srow = reinterpret_cast<float2*>(sq + HG * CG * KSTEPS * 32);  // [hg][CG * 8] (factor, -lse log2 e)
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, cq = lane & 3;
  // CTAs of the head groups side by side, then the chunks of a sequence
  const uint32_t xg = p.by_groups.div(blockIdx.x);
  const int grp = (int)(blockIdx.x - xg * p.by_groups.d);
  const int i = (int)p.by_chunks.div(xg), chunk = (int)(xg - (uint32_t)i * p.by_chunks.d);
  const int q0 = a.query_start_loc[i], ql = a.query_start_loc[i + 1] - q0, L = a.seq_lens[i];
  if (!mass_seq_ok(a, q0, ql, L)) {
    if (chunk == 0 && grp == 0 && tid == 0) flag(a.dev_status, KV_INT4_DEV_BAD_SEQ);
    return;
  }
  const int per = p.warp_blocks;
  const int nblk = (L + 15) >> 4, first = chunk * per * WPH;
  if (ql == 0 || first >= nblk || !few_rows(p, ql)) return;
  const int ctx = L - ql, rows = ql * p.group, ncg = (rows + 7) / 8;
  const int hl = warp / WPH, head = grp * HG + hl;
  const int b0 = first + (warp - hl * WPH) * per, nb = min(per, nblk - b0);
  // the warp's block ids, and the first blocks' codes, on their way while the rows are staged
  int id = -1;
  if (lane < nb) {
    id = a.block_table[(int64_t)i * a.max_blocks_per_seq + b0 + lane];
    if (id < 0 || id >= a.num_blocks) {
      id = -1;
      if (head == 0) flag(a.dev_status, KV_INT4_DEV_BAD_BLOCK);
    }
  }
  float* const out = a.mass + i * a.mass_seq_stride + head * a.mass_head_stride;
  struct Block {
    uint32_t x[KSTEPS], y[KSTEPS];  // codes of rows g and g + 8
    float ks, old;                  // 0 without a block; the mass so far of lane cq < 2's position
  };
  const int64_t row = (int64_t)a.num_kv_heads * D;
  auto load = [&](Block& b, int n) {
    const int blk = __shfl_sync(0xffffffffu, id, n & 31);
    const int pos = (b0 + n) * 16 + g;
    b.ks = 0.f;
    b.old = 0.f;
#pragma unroll
    for (int s = 0; s < KSTEPS; s++) b.x[s] = b.y[s] = 0u;
    if (n < nb && blk >= 0) {
      const uint8_t* src = a.k_cache + ((int64_t)blk * 16 * a.num_kv_heads + head) * D + g * row;
      b.ks = a.k_scale[(int64_t)blk * a.num_kv_heads + head];
      // rows behind the sequence's end may hold NaN codes
#pragma unroll
      for (int half = 0; half < 2; half++) {
        uint32_t* w = half ? b.y : b.x;
        if (pos + 8 * half < L) {
          const uint8_t* r = src + half * 8 * row;
          if constexpr (F::WIDE) {
#pragma unroll
            for (int c = 0; c < KSTEPS / 4; c++) {
              const uint4 v = __ldcs(reinterpret_cast<const uint4*>(r + 16 * (cq + 4 * c)));
              w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
            }
          } else {
#pragma unroll
            for (int c = 0; c < KSTEPS / 2; c++) {
              const uint2 v = __ldcs(reinterpret_cast<const uint2*>(r + cq * (D / 4) + 8 * c));
              w[2 * c] = v.x, w[2 * c + 1] = v.y;
            }
          }
        }
      }
    }
    if (n < nb && cq < 2 && pos + 8 * cq < ctx) b.old = out[pos + 8 * cq];
  };
  Block blk[U];
#pragma unroll
  for (int u = 0; u < U; u++) load(blk[u], u);
  for (int u = warp; u < HG * ncg; u += 4) {
    const int h = u / ncg, cgi = u - h * ncg;
    stage_rows<D>(p, q0, grp * HG + h, 8 * cgi, rows, sq + (h * CG + cgi) * KSTEPS * 32, srow + (h * CG + cgi) * 8,
                  [](int c, int s) { return F::kdim(c, s); });
  }
  __syncthreads();
  const uint2* const bq = sq + hl * CG * KSTEPS * 32 + lane;
  const float2* const br = srow + hl * CG * 8 + 2 * cq;
  // positions that this lane's two columns see: up to ctx + row / group; all rows see those up to ctx
#pragma unroll 1
  for (int n0 = 0; n0 < nb; n0 += U) {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int n = n0 + u;
      if (n >= nb) break;
      Block& b = blk[u];
      const int p0 = (b0 + n) * 16 + g, p1 = p0 + 8;
      const bool all = (b0 + n) * 16 + 15 <= ctx;
      float w0 = 0.f, w1 = 0.f;
#pragma unroll 1
      for (int cgi = 0; cgi < ncg; cgi++) {
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KSTEPS; s++) {
          uint32_t f[4];
          e4m3x4_to_f16x2(b.x[s], f[0], f[2]);
          e4m3x4_to_f16x2(b.y[s], f[1], f[3]);
          const uint2 bb = bq[(cgi * KSTEPS + s) * 32];
          mma_16816(s4, f, bb.x, bb.y);
        }
        const float2 ra = br[8 * cgi], rb = br[8 * cgi + 1];
        const float fa = ra.x * b.ks, fb = rb.x * b.ks;
        float e0 = fast_exp2(fmaf(s4[0], fa, ra.y)), e1 = fast_exp2(fmaf(s4[1], fb, rb.y));
        float e2 = fast_exp2(fmaf(s4[2], fa, ra.y)), e3 = fast_exp2(fmaf(s4[3], fb, rb.y));
        if (!all) {
          const int c0 = 8 * cgi + 2 * cq, la = ctx + c0 / p.group, lb = ctx + (c0 + 1) / p.group;
          e0 = p0 <= la ? e0 : 0.f;
          e1 = p0 <= lb ? e1 : 0.f;
          e2 = p1 <= la ? e2 : 0.f;
          e3 = p1 <= lb ? e3 : 0.f;
        }
        w0 += e0 + e1;
        w1 += e2 + e3;
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        w0 += __shfl_xor_sync(0xffffffffu, w0, o);
        w1 += __shfl_xor_sync(0xffffffffu, w1, o);
      }
      const int pos = p0 + 8 * cq;
      if (cq < 2 && pos < L) out[pos] = (b.ks == 0.f ? 0.f : cq ? w1 : w0) + b.old;
      load(b, n + U);
    }
  }
}

// More rows than that, in tiles of kMassCols, where no tensor map holds the queries
// (token rows that overlap: one row for all tokens, say)
template <int D>
__global__ void __launch_bounds__(128) mass_rows_kernel(MassParams p) {
  constexpr int KSTEPS = D / 16, CG = kMassCols / 8;
  extern __shared__ __align__(16) uint8_t smem[];
  const MassArgs& a = p.a;
  const int HG = p.hg, WPH = 4 / HG;  // warps per head
  uint2* const sq = reinterpret_cast<uint2*>(smem);                       // [hg][CG][KSTEPS][32]
  float2* const srow = reinterpret_cast<float2*>(sq + HG * CG * KSTEPS * 32);  // [hg][kMassCols] (factor, -lse log2 e)
  float* const sacc = reinterpret_cast<float*>(srow + HG * kMassCols);    // [warps][warp_blocks * 16]
  pdl_trigger();
  pdl_wait();
  const int nthr = blockDim.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, cq = lane & 3;
  const uint32_t xg = p.by_groups.div(blockIdx.x);
  const int grp = (int)(blockIdx.x - xg * p.by_groups.d);
  const int i = (int)p.by_chunks.div(xg), chunk = (int)(xg - (uint32_t)i * p.by_chunks.d);
  const int q0 = a.query_start_loc[i], ql = a.query_start_loc[i + 1] - q0, L = a.seq_lens[i];
  if (!mass_seq_ok(a, q0, ql, L) || few_rows(p, ql)) return;
  const int per = p.warp_blocks, cta_blocks = per * WPH;
  const int nblk = (L + 15) >> 4, first = chunk * cta_blocks;
  if (first >= nblk) return;
  const int ctx = L - ql, rows = ql * p.group;
  const int hl = warp / WPH, head = grp * HG + hl;
  const int b0 = first + (warp - hl * WPH) * per, b1 = min(b0 + per, nblk);
  const int32_t* table = a.block_table + (int64_t)i * a.max_blocks_per_seq;
  float* const acc = sacc + warp * per * 16;
  for (int x = lane; x < per * 16; x += 32) acc[x] = 0.f;
  // rows before this one see none of the CTA's keys
  const int row0 = max(0, first * 16 - ctx) * p.group / 8 * 8;
#pragma unroll 1
  for (int r0 = row0; r0 < rows; r0 += kMassCols) {
    __syncthreads();
    for (int u = warp; u < HG * CG; u += nthr >> 5) {
      const int h = u / CG, cgi = u - h * CG;
      stage_rows<D>(p, q0, grp * HG + h, r0 + 8 * cgi, rows, sq + u * KSTEPS * 32, srow + h * kMassCols + 8 * cgi,
                    [](int c, int s) { return 16 * s + 4 * c; });
    }
    __syncthreads();
    const int ncg = min(CG, (rows - r0 + 7) / 8);
    const uint2* const bq = sq + hl * CG * KSTEPS * 32 + lane;
#pragma unroll 1
    for (int b = b0; b < b1; b++) {
      const int blk = table[b];
      if (blk < 0 || blk >= a.num_blocks) continue;
      const uint8_t* src = a.k_cache + ((int64_t)blk * 16 * a.num_kv_heads + head) * D + 4 * cq;
      const int64_t row = (int64_t)a.num_kv_heads * D;
      uint32_t x[KSTEPS], y[KSTEPS];
      const bool in0 = b * 16 + g < L, in1 = b * 16 + g + 8 < L;  // rows behind the end may hold NaN codes
#pragma unroll
      for (int s = 0; s < KSTEPS; s++) {
        x[s] = in0 ? *reinterpret_cast<const uint32_t*>(src + g * row + 16 * s) : 0u;
        y[s] = in1 ? *reinterpret_cast<const uint32_t*>(src + (g + 8) * row + 16 * s) : 0u;
      }
      const float ks = a.k_scale[(int64_t)blk * a.num_kv_heads + head];
      float w0 = 0.f, w1 = 0.f;
#pragma unroll 1
      for (int cgi = 0; cgi < ncg; cgi++) {
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KSTEPS; s++) {
          uint32_t f[4];
          e4m3x4_to_f16x2(x[s], f[0], f[2]);
          e4m3x4_to_f16x2(y[s], f[1], f[3]);
          const uint2 bb = bq[(cgi * KSTEPS + s) * 32];
          mma_16816(s4, f, bb.x, bb.y);
        }
        const int c0 = cgi * 8 + 2 * cq;
        const float2 ra = srow[hl * kMassCols + c0], rb = srow[hl * kMassCols + c0 + 1];
        // positions that the rows see: up to ctx + row / group
        const int la = ctx + (r0 + c0) / p.group, lb = ctx + (r0 + c0 + 1) / p.group;
        const int p0 = b * 16 + g, p1 = p0 + 8;
        const float fa = ra.x * ks, fb = rb.x * ks;
        w0 += p0 <= la ? fast_exp2(fmaf(s4[0], fa, ra.y)) : 0.f;
        w0 += p0 <= lb ? fast_exp2(fmaf(s4[1], fb, rb.y)) : 0.f;
        w1 += p1 <= la ? fast_exp2(fmaf(s4[2], fa, ra.y)) : 0.f;
        w1 += p1 <= lb ? fast_exp2(fmaf(s4[3], fb, rb.y)) : 0.f;
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        w0 += __shfl_xor_sync(0xffffffffu, w0, o);
        w1 += __shfl_xor_sync(0xffffffffu, w1, o);
      }
      if (cq < 2) acc[(b - b0) * 16 + g + 8 * cq] += cq ? w1 : w0;
    }
  }
  __syncwarp();
  float* const out = a.mass + i * a.mass_seq_stride + head * a.mass_head_stride;
  for (int x = lane; x < (b1 - b0) * 16; x += 32) {
    const int pos = b0 * 16 + x;
    if (pos < L) out[pos] = acc[x] + (pos < ctx ? out[pos] : 0.f);
  }
  if (hl == 0 && grp == 0)
    for (int b = b0 + lane; b < b1; b += 32)
      if (table[b] < 0 || table[b] >= a.num_blocks) flag(a.dev_status, KV_INT4_DEV_BAD_BLOCK);
}

#include "mass_ws_fp8.cuh"

template <int D>
int launch_t(const MassArgs& a, cudaStream_t stream) {
  const int dev = current_device();
  const int sms = sm_count(dev);
  MassParams p{a, a.num_q_heads / a.num_kv_heads, a.num_kv_heads % 4 == 0 ? 4 : a.num_kv_heads % 2 == 0 ? 2 : 1, 16,
               1, a.softmax_scale * kLog2e};
  p.by_group = FastDiv((uint32_t)p.group);
  const int64_t most_rows = (int64_t)a.max_query_len * p.group;
  p.few_groups = most_rows < 8 ? 1 : most_rows < kMassCols ? (int)(most_rows + 7) / 8 : kMassCols / 8;
  const int64_t table = (int64_t)a.max_blocks_per_seq * 16;
  const int64_t most = a.max_seq_len < table ? a.max_seq_len : table;
  const int64_t nblk = most > 0 ? (most + 15) / 16 : 1;
  const int groups = a.num_kv_heads / p.hg, wph = 4 / p.hg;
  auto grid_of = [&](int warp_blocks, unsigned* grid) {
    const int64_t per = (int64_t)warp_blocks * wph, chunks = (nblk + per - 1) / per;
    if (chunks * a.num_seqs >= (1ll << 31) / groups) return false;
    p.warp_blocks = warp_blocks;
    p.by_groups = FastDiv((uint32_t)groups);
    p.by_chunks = FastDiv((uint32_t)chunks);
    *grid = (unsigned)(chunks * a.num_seqs * groups);
    return true;
  };
  // blocks per warp: as many as leave two rounds of warps
  const int64_t warps = 2ll * 16 * sms, all = nblk * a.num_seqs * a.num_kv_heads;
  int per = MassFew<D>::U;
  while (per < 32 && all >= warps * per * 2) per *= 2;
  static PerContext<int> attr;
  int set = 0;
  if (!attr.get(dev, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(mass_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)MassFew<D>::smem(4, kMassCols / 8)) == cudaSuccess &&
               cudaFuncSetAttribute(mass_rows_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 * 1024) == cudaSuccess;
      }, &set))
    return KV_INT4_ERR_CUDA;
  unsigned grid;
  if (!grid_of(per, &grid)) return KV_INT4_ERR_SIZE;
  if (int e = launch_pdl(mass_few_kernel<D>, dim3(grid), 128, MassFew<D>::smem(p.hg, p.few_groups), stream, 1, p)) return e;
  if (most_rows <= kMassCols) return KV_INT4_OK;
  using W = MassWs<D>;
  const int tile_tokens = W::QR / p.group;
  CUtensorMap qmap;
  if (make_q_map(&qmap, a.q, a.q_stride, a.num_q_tokens, a.num_q_heads, D, p.group, tile_tokens)) {
    static PerContext<int> occ_c;
    int occ = 0;
    if (!occ_c.get(dev, [](int* o) { return configure_tmem(mass_ws_kernel<D>, W::SMEM, W::THREADS, W::S_COLS, o); }, &occ))
      return KV_INT4_ERR_CUDA;
    const int64_t items = (int64_t)a.num_seqs * ((most + 127) / 128) * a.num_kv_heads;
    return launch_pdl(mass_ws_kernel<D>, dim3((unsigned)(items < sms ? (items > 0 ? items : 1) : sms)), W::THREADS, W::SMEM, stream,
                      1, p, tile_tokens, qmap);
  }
  if (!grid_of(16, &grid)) return KV_INT4_ERR_SIZE;
  const size_t smem = (size_t)p.hg * kMassCols * (D * 2 + 8) + 4 * p.warp_blocks * 16 * 4;
  return launch_pdl(mass_rows_kernel<D>, dim3(grid), 128, smem, stream, 1, p);
}

}  // namespace

int launch_mass_fp8(const MassArgs& a, cudaStream_t stream) {
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
