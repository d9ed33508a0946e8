// kv_fp8_attention_mass: the attention weight that every position of an FP8
// cache receives from the call's queries.
//
//   w_p = sum over the query rows r of the position's kv head that see it of
//         2^(t_rp - lse_r log2 e),  t_rp = softmax_scale log2 e 2^kk_b (q_r . ck_p)
//
// The rows' denominators are known, so nothing is carried from key to key: a
// warp takes 16-key blocks of one kv head and needs no other warp's results.

#include <cuda_runtime.h>

#include "../../include/kvint4.h"
#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"
#include "schedule.cuh"

namespace kvint4 {
namespace {

constexpr int kMassCols = 32;  // query rows staged at once

struct MassParams {
  MassArgs a;
  int group, hg;      // q heads per kv head; kv heads per CTA
  int warp_blocks;    // 16-key blocks per warp
  float qscale;       // softmax_scale log2 e
};

__device__ __forceinline__ bool mass_seq_ok(const MassArgs& a, int q0, int ql, int L) {
  return q0 >= 0 && ql >= 0 && (int64_t)q0 + ql <= a.num_q_tokens && ql <= a.max_query_len && L >= ql &&
         L <= a.max_seq_len && L <= a.mass_len && (int64_t)L <= (int64_t)a.max_blocks_per_seq * 16;
}

// one chunk of keys of a sequence for hg kv heads; query rows in tiles of
// kMassCols that the CTA stages in shared memory as f16 fragments (a row divided
// by the power of two of its largest magnitude)
template <int D>
__global__ void __launch_bounds__(128) mass_fp8_kernel(MassParams p) {
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
  const int i = blockIdx.y, grp = blockIdx.z;
  const int q0 = a.query_start_loc[i], ql = a.query_start_loc[i + 1] - q0, L = a.seq_lens[i];
  if (!mass_seq_ok(a, q0, ql, L)) {
    if (blockIdx.x == 0 && grp == 0 && tid == 0) flag(a.dev_status, KV_INT4_DEV_BAD_SEQ);
    return;
  }
  const int per = p.warp_blocks, cta_blocks = per * WPH;
  const int nblk = (L + 15) >> 4, first = blockIdx.x * cta_blocks;
  if (ql == 0 || first >= nblk) return;
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
    // a warp stages a column group (8 rows): lane (g, cq) row g's elements 16 s + 4 cq .. + 3 of k-step s
    for (int u = warp; u < HG * CG; u += nthr >> 5) {
      const int h = u / CG, r = r0 + (u - h * CG) * 8 + g;
      const bool ok = r < rows;
      const int j = ok ? r / p.group : 0, jj = ok ? r - j * p.group : 0;
      const int hq = (grp * HG + h) * p.group + jj;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (int64_t)(q0 + j) * a.q_stride + (int64_t)hq * D;
      uint2 v[KSTEPS];
      uint32_t am = 0;
#pragma unroll
      for (int s = 0; s < KSTEPS; s++) {
        v[s] = ok ? *reinterpret_cast<const uint2*>(src + 16 * s + 4 * cq) : make_uint2(0, 0);
        am = __vmaxu2(am, __vmaxu2(v[s].x & 0x7fff7fffu, v[s].y & 0x7fff7fffu));
      }
      am = max(am & 0xffffu, am >> 16);
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
      const int e = min(max((int)(am >> 7) - 127, -126), 126);
      const float mul = exp2_int(-e);
#pragma unroll
      for (int s = 0; s < KSTEPS; s++)
        sq[(u * KSTEPS + s) * 32 + lane] = make_uint2(pack_f16x2(bf16lo_to_f32(v[s].x) * mul, bf16hi_to_f32(v[s].x) * mul),
                                                      pack_f16x2(bf16lo_to_f32(v[s].y) * mul, bf16hi_to_f32(v[s].y) * mul));
      if (cq == 0) {
        const float l = ok ? a.lse[(int64_t)(q0 + j) * a.lse_stride + hq] : INFINITY;
        srow[u * 8 + g] = make_float2(p.qscale * exp2_int(e), fabsf(l) == INFINITY ? -INFINITY : -l * kLog2e);
      }
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

template <int D>
int launch_t(const MassArgs& a, cudaStream_t stream) {
  const int dev = current_device();
  MassParams p{a, a.num_q_heads / a.num_kv_heads, a.num_kv_heads % 4 == 0 ? 4 : a.num_kv_heads % 2 == 0 ? 2 : 1, 16,
               a.softmax_scale * kLog2e};
  const int64_t table = (int64_t)a.max_blocks_per_seq * 16;
  const int64_t most = a.max_seq_len < table ? a.max_seq_len : table;
  const int64_t nblk = (most + 15) / 16;
  if (nblk == 0) p.warp_blocks = 1;
  const int cta_blocks = p.warp_blocks * (4 / p.hg);
  const int64_t chunks = nblk == 0 ? 1 : (nblk + cta_blocks - 1) / cta_blocks;
  if (a.num_seqs > 65535 || a.num_kv_heads / p.hg > 65535 || chunks > 0x7fffffff) return KV_INT4_ERR_SIZE;
  const size_t smem = (size_t)p.hg * kMassCols * (D * 2 + 8) + 4 * p.warp_blocks * 16 * 4;
  static PerContext<int> attr;
  int set = 0;
  if (!attr.get(dev, [](int* v) {
        *v = 1;
        return cudaFuncSetAttribute(mass_fp8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) == cudaSuccess;
      }, &set))
    return KV_INT4_ERR_CUDA;
  return launch_pdl(mass_fp8_kernel<D>, dim3((unsigned)chunks, (unsigned)a.num_seqs, (unsigned)(a.num_kv_heads / p.hg)), 128,
                    smem, stream, 1, p);
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
