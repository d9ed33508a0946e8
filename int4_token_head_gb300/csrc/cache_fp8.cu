// kv_fp8_write and kv_fp8_read: the paged E4M3 cache with one power-of-two
// scale per (block of 16 tokens, kv head).
//
// Write, per (block, kv head) of K and of V that the call's tokens touch, over
// the values x of the call's rows (NaN counts as 0, magnitudes above
// 448 * 2^60 as that):
//   k  = smallest exponent in [-60, 60] with max |x| <= 448 * 2^k,
//        and at least the stored scale's unless the call writes the block's
//        first row (which begins the block anew)
//   c  = e4m3(x * 2^-k), nearest even; scale = 2^k
//   rows that the block held before: c' = e4m3(c * 2^(k_old - k)) when k grew
//        (a stored scale that is no power of two in range: it held none)
// Read: bf16(c * scale).
//
// Both are HBM-bound (3 d bytes per head vector, write 2 d in and d out, read
// the other way round).  One warp per (block, kv head, K or V): 16 rows are
// d / 16 chunks of 8 elements a lane, all loaded before any is used (2 or 4
// KB in flight per warp at d = 128), so a block's absmax, its rows and its
// scale never leave the warp: no second pass, no atomics, and results that
// depend on neither the launch shape nor the order of warps.  Four-warp CTAs at
// most 72 registers a thread (28 warps per SM) and streaming loads of K and V:
// 65,536 tokens, 8 heads of 128, 403 MB: 66.5 us = 0.89 of the measured copy
// bandwidth (on the same tensors again 65.9; eight-warp CTAs 70.4; streaming
// stores of the codes 65.0, not kept: attention reads them next).  Read: 396 MB in
// 60 us = 0.97.

#include <cuda_runtime.h>

#include "../../include/kvint4.h"
#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace kvint4 {
namespace {

constexpr int kFp8Warps = 4;

struct CacheFp8 {
  Fp8Seqs s;
  const uint16_t* k_in;
  const uint16_t* v_in;
  uint16_t* k_out;
  uint16_t* v_out;
  int64_t k_stride, v_stride;  // elements
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;
  float* v_scale;
  int hkv;
};

template <int D>
__global__ void __launch_bounds__(kFp8Warps * 32, D <= 96 ? 8 : 7) write_fp8_kernel(CacheFp8 a) {
  constexpr int CH = D / 8;   // 16-byte chunks per input row
  constexpr int PER = D / 16; // chunks per lane (16 rows)
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0) fp8_check_seqs(a.s);
  const int lane = threadIdx.x & 31;
  const int task = blockIdx.y * kFp8Warps + (threadIdx.x >> 5);
  if (task >= 2 * a.hkv) return;
  Fp8Unit u;
  if (!fp8_unit(a.s, blockIdx.x, &u)) return;
  if (u.bad) {
    if (task == 0 && lane == 0) flag(a.s.status, KV_INT4_DEV_BAD_BLOCK);
    return;
  }
  const bool isv = task >= a.hkv;
  const int h = isv ? task - a.hkv : task;
  const int64_t stride = isv ? a.v_stride : a.k_stride;
  const uint16_t* src = (isv ? a.v_in : a.k_in) + (u.token0 - u.r0) * stride + (int64_t)h * D;
  float* scale = (isv ? a.v_scale : a.k_scale) + u.block * a.hkv + h;
  const float old = *scale;
  uint4 x[PER];
#pragma unroll
  for (int j = 0; j < PER; j++) {
    const int c = lane + 32 * j, r = c / CH, col = c - r * CH;
    x[j] = make_uint4(0, 0, 0, 0);
    if (r >= u.r0 && r < u.r1) x[j] = __ldcs(reinterpret_cast<const uint4*>(src + r * stride + col * 8));
  }
  auto absmax = [&]() {
    uint32_t m = 0;  // both halves; the sign bits carry nothing
#pragma unroll
    for (int j = 0; j < PER; j++) {
      const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
      for (int i = 0; i < 4; i++) m = __vmaxu2(m, w[i] & 0x7fff7fffu);  // bf16 magnitudes order as integers
    }
    return __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
  };
  uint32_t am = absmax();
  if (am >= 0x7f80u) {
    // infinities become the largest finite value, NaN becomes 0
    if (lane == 0) flag(a.s.status, KV_INT4_DEV_NONFINITE);
#pragma unroll
    for (int j = 0; j < PER; j++) {
      uint32_t* w = reinterpret_cast<uint32_t*>(&x[j]);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        uint32_t r = 0;
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          const uint32_t v = (w[i] >> e) & 0xffffu, mag = v & 0x7fffu;
          r |= (mag > 0x7f80u ? 0u : mag == 0x7f80u ? (v & 0x8000u) | 0x7f7fu : v) << e;
        }
        w[i] = r;
      }
    }
    am = absmax();
  }
  const int k_old = fp8_scale_exponent(old);
  int k = fp8_exponent(am);
  const bool held = u.r0 > 0 && k_old <= kFp8MaxExp;  // rows of an earlier call
  if (held) k = max(k, k_old);
  const float mul = exp2_int(-k);
  uint8_t* codes = (isv ? a.v_cache : a.k_cache) + (u.block * 16 * a.hkv + h) * D;
  const int64_t row = (int64_t)a.hkv * D;
#pragma unroll
  for (int j = 0; j < PER; j++) {
    const int c = lane + 32 * j, r = c / CH, col = c - r * CH;
    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 p = __fmul2_rn(make_float2(bf16lo_to_f32(w[i]), bf16hi_to_f32(w[i])), make_float2(mul, mul));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
    const uint2 q = make_uint2(f32x4_to_e4m3(f[0], f[1], f[2], f[3]), f32x4_to_e4m3(f[4], f[5], f[6], f[7]));
    if (r >= u.r0 && r < u.r1) *reinterpret_cast<uint2*>(codes + r * row + col * 8) = q;
  }
  if (held && k > k_old) {  // they follow the grown scale
    const float shift = exp2_int(k_old - k);
#pragma unroll 2
    for (int c = lane; c < u.r0 * CH; c += 32) {
      const int r = c / CH, col = c - r * CH;
      uint2* p = reinterpret_cast<uint2*>(codes + r * row + col * 8);
      const uint2 w = *p;
      uint32_t o[2];
      const uint32_t in[2] = {w.x, w.y};
#pragma unroll
      for (int i = 0; i < 2; i++) {
        uint32_t lo, hi;
        e4m3x4_to_f16x2(in[i], lo, hi);
        const float2 p0 = __half22float2(*reinterpret_cast<__half2*>(&lo));
        const float2 p1 = __half22float2(*reinterpret_cast<__half2*>(&hi));
        o[i] = f32x4_to_e4m3(p0.x * shift, p0.y * shift, p1.x * shift, p1.y * shift);
      }
      *p = make_uint2(o[0], o[1]);
    }
  }
  if (lane == 0) *scale = exp2_int(k);
}

template <int D>
__global__ void __launch_bounds__(kFp8Warps * 32) read_fp8_kernel(CacheFp8 a) {
  constexpr int CH = D / 8;    // 8-code chunks per row
  constexpr int PER = D / 16;  // chunks per lane (16 rows)
  pdl_trigger();
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0) fp8_check_seqs(a.s);
  const int lane = threadIdx.x & 31;
  const int task = blockIdx.y * kFp8Warps + (threadIdx.x >> 5);
  if (task >= 2 * a.hkv) return;
  Fp8Unit u;
  if (!fp8_unit(a.s, blockIdx.x, &u)) return;
  if (u.bad && task == 0 && lane == 0) flag(a.s.status, KV_INT4_DEV_BAD_BLOCK);
  const bool isv = task >= a.hkv;
  const int h = isv ? task - a.hkv : task;
  const int64_t stride = isv ? a.v_stride : a.k_stride;
  uint16_t* dst = (isv ? a.v_out : a.k_out) + (u.token0 - u.r0) * stride + (int64_t)h * D;
  const uint8_t* codes = (isv ? a.v_cache : a.k_cache) + ((u.bad ? 0 : u.block) * 16 * a.hkv + h) * D;
  const int64_t row = (int64_t)a.hkv * D;
  float s = 0.f;
  uint2 x[PER];
#pragma unroll
  for (int j = 0; j < PER; j++) {
    const int c = lane + 32 * j, r = c / CH, col = c - r * CH;
    x[j] = make_uint2(0, 0);
    if (!u.bad && r >= u.r0 && r < u.r1) x[j] = *reinterpret_cast<const uint2*>(codes + r * row + col * 8);
  }
  if (!u.bad) s = (isv ? a.v_scale : a.k_scale)[u.block * a.hkv + h];
#pragma unroll
  for (int j = 0; j < PER; j++) {
    const int c = lane + 32 * j, r = c / CH, col = c - r * CH;
    uint32_t o[4];
    const uint32_t in[2] = {x[j].x, x[j].y};
#pragma unroll
    for (int i = 0; i < 2; i++) {
      uint32_t lo, hi;
      e4m3x4_to_f16x2(in[i], lo, hi);
      const float2 p0 = __half22float2(*reinterpret_cast<__half2*>(&lo));
      const float2 p1 = __half22float2(*reinterpret_cast<__half2*>(&hi));
      o[2 * i] = pack_bf16x2_rn(p0.x * s, p0.y * s);
      o[2 * i + 1] = pack_bf16x2_rn(p1.x * s, p1.y * s);
    }
    if (r >= u.r0 && r < u.r1)
      *reinterpret_cast<uint4*>(dst + r * stride + col * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <int D>
int launch_t(const CacheFp8& a, bool write, cudaStream_t stream) {
  const int64_t units = fp8_units(a.s.num_seqs, a.s.num_tokens, a.s.max_len);
  const int tasks = 2 * a.hkv;
  const dim3 grid((unsigned)units, (unsigned)((tasks + kFp8Warps - 1) / kFp8Warps));
  if (units > 0x7fffffff || grid.y > 65535) return KV_INT4_ERR_SIZE;
  if (write) timing_begin(kTimedWrite, stream);
  const int e = launch_pdl(write ? write_fp8_kernel<D> : read_fp8_kernel<D>, grid, kFp8Warps * 32, 0, stream, 1, a);
  if (write) timing_end(kTimedWrite, stream);
  return e;
}

int launch(const CacheFp8& a, int head_size, bool write, cudaStream_t stream) {
  switch (head_size) {
    case 64: return launch_t<64>(a, write, stream);
    case 96: return launch_t<96>(a, write, stream);
    case 128: return launch_t<128>(a, write, stream);
    case 192: return launch_t<192>(a, write, stream);
    case 256: return launch_t<256>(a, write, stream);
    default: return KV_INT4_ERR_HEAD_SIZE;
  }
}

CacheFp8 common_args(const CacheFp8Args& w) {
  CacheFp8 a{};
  a.s = Fp8Seqs{w.block_table, w.max_blocks_per_seq, w.seq_lens, w.start_loc, w.num_seqs, w.num_tokens,
                w.max_len, w.num_blocks, w.dev_status};
  a.k_stride = w.k_stride;
  a.v_stride = w.v_stride;
  a.k_cache = w.k_cache;
  a.v_cache = w.v_cache;
  a.k_scale = w.k_scale;
  a.v_scale = w.v_scale;
  a.hkv = w.num_kv_heads;
  return a;
}

}  // namespace

int launch_write_fp8(const CacheFp8Args& w, cudaStream_t stream) {
  CacheFp8 a = common_args(w);
  a.k_in = static_cast<const uint16_t*>(w.k);
  a.v_in = static_cast<const uint16_t*>(w.v);
  return launch(a, w.head_size, true, stream);
}

int launch_read_fp8(const CacheFp8Args& w, cudaStream_t stream) {
  CacheFp8 a = common_args(w);
  a.k_out = static_cast<uint16_t*>(w.k);
  a.v_out = static_cast<uint16_t*>(w.v);
  return launch(a, w.head_size, false, stream);
}

}  // namespace kvint4
