// kv_qk_norm_rope: RMS norm of every query and key head vector and the rotary
// position rotation, in one pass over the heads.
//
//   y = x / sqrt(mean(x^2) + eps) * w            (no norm without weights)
//   (y_i, y_j) <- (y_i cos - y_j sin, y_j cos + y_i sin)   for the rot / 2
//     pairs of the first rot elements: (i, i + rot / 2), or (2 i, 2 i + 1)
// in fp32, rounded once to bf16; squares that leave fp32's range are taken in
// units of the vector's largest element (far_rsqrt).
//
// HBM-bound (2 d bytes in and 2 d out per head vector).  d / 16 lanes hold a
// vector, each lane two 16-byte chunks: pair lanes (lane c < rot / 16) hold
// both halves of eight rotation pairs, so that nothing but the sum of squares
// crosses lanes; a warp takes several heads of one token, whose cosines and
// sines it loads once.  Inputs are loaded as streaming data, and outputs too
// large to wait in L2 for the kernels that read them are stored as such: written
// back in the order they were made they leave the bandwidth to the loads (16384
// tokens, 32/8 heads of 128, 344 MB, a call on the same tensors again: 64.5 us
// without either hint, 55.3 with both; on other tensors in each call 58 to 60 =
// 0.86 of the measured copy bandwidth).

#include <cuda_runtime.h>

#include "../../include/kvint4.h"
#include "common.cuh"
#include "fp8.cuh"
#include "internal.h"

namespace kvint4 {
namespace {

constexpr int kNormWarps = 4;

struct NormRope {
  NormRopeArgs a;
  bool stream_out;  // outputs are stored as streaming data
  int heads;        // q and kv heads
  int parts;        // warps per token
  FastDiv by_parts{1};
};

// sum over the N lanes of a vector (N = 4, 6, 8, 12 or 16, starting at lane base)
template <int N>
__device__ __forceinline__ float vector_sum(float s, int base, int c) {
  int n = N;
#pragma unroll
  for (; n % 2 == 0; n /= 2) s += __shfl_sync(0xffffffffu, s, base + (c % n + n / 2) % n);
  if (n == 3) {
    const float a = __shfl_sync(0xffffffffu, s, base), b = __shfl_sync(0xffffffffu, s, base + 1);
    s = a + b + __shfl_sync(0xffffffffu, s, base + 2);
  }
  return s;
}

// 1 / sqrt(s / D + eps), s the sum of squares, where that is no normal fp32
// number or close to one: from the elements in units of 2^e, e the exponent of
// the largest one
template <int D, int N>
__device__ float far_rsqrt(const float (&f0)[8], const float (&f1)[8], float eps, int base, int c) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i++) m = fmaxf(m, fmaxf(fabsf(f0[i]), fabsf(f1[i])));
#pragma unroll 1
  for (int i = 0; i < N; i++) m = fmaxf(m, __shfl_sync(0xffffffffu, m, base + i));
  const int e = min(max(exp_of(m), -63), 126);
  const float unit = exp2_int(-e);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const float a = f0[i] * unit, b = f1[i] * unit;
    s = fmaf(a, a, fmaf(b, b, s));
  }
  s = vector_sum<N>(s, base, c);
  return rsqrtf(s * (1.f / D) + eps * unit * unit) * unit;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = bf16lo_to_f32(w[i]);
    f[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]), pack_bf16x2_rn(f[4], f[5]),
                    pack_bf16x2_rn(f[6], f[7]));
}

template <int D, int U>
__global__ void __launch_bounds__(kNormWarps * 32, 8) norm_rope_kernel(NormRope p) {
  constexpr int LPV = D / 16;    // lanes per vector
  constexpr int VPW = 32 / LPV;  // vectors per warp step
  const NormRopeArgs& a = p.a;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int gw = blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  const int t = (int)p.by_parts.div((uint32_t)gw);
  if (t >= a.num_tokens) return;
  const int part = gw - t * p.parts;
  const int vsub = lane / LPV, c = lane - vsub * LPV;
  const bool rotated = c < a.rot_dim / 16;
  // the lane's two chunks (of 8 elements)
  const bool split = rotated && !a.interleaved;
  const int c0 = split ? c : 2 * c, c1 = split ? c + a.rot_dim / 16 : 2 * c + 1;

  uint4 x[U][2];
  int head[U];
#pragma unroll
  for (int u = 0; u < U; u++) {
    head[u] = (part * U + u) * VPW + vsub;
    if (vsub >= VPW || head[u] >= p.heads) head[u] = -1;
    x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
    if (head[u] >= 0) {
      const uint16_t* src = head[u] < a.num_q_heads
                                ? static_cast<const uint16_t*>(a.q) + t * a.q_stride + (int64_t)head[u] * D
                                : static_cast<const uint16_t*>(a.k) + t * a.k_stride + (int64_t)(head[u] - a.num_q_heads) * D;
      x[u][0] = __ldcs(reinterpret_cast<const uint4*>(src + 8 * c0));
      x[u][1] = __ldcs(reinterpret_cast<const uint4*>(src + 8 * c1));
    }
  }
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (a.rot_dim > 0) {
    const int64_t pos = a.positions[t];
    if (pos < 0 || pos >= a.max_position) {
      if (part == 0 && lane == 0) flag(a.dev_status, KV_INT4_DEV_BAD_POS);
      return;
    }
    if (rotated) {
      const float* row = a.cos_sin + pos * a.rot_dim + 8 * c;
      const float4* pc = reinterpret_cast<const float4*>(row);
      const float4* ps = reinterpret_cast<const float4*>(row + a.rot_dim / 2);
      const float4 q0 = pc[0], q1 = pc[1], r0 = ps[0], r1 = ps[1];
      cs[0] = q0.x; cs[1] = q0.y; cs[2] = q0.z; cs[3] = q0.w; cs[4] = q1.x; cs[5] = q1.y; cs[6] = q1.z; cs[7] = q1.w;
      sn[0] = r0.x; sn[1] = r0.y; sn[2] = r0.z; sn[3] = r0.w; sn[4] = r1.x; sn[5] = r1.y; sn[6] = r1.z; sn[7] = r1.w;
    }
  }
#pragma unroll
  for (int u = 0; u < U; u++) {
    float f0[8], f1[8];
    unpack8(x[u][0], f0);
    unpack8(x[u][1], f1);
    const bool isq = head[u] < a.num_q_heads;
    if (a.q_weight) {  // both weights or neither
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) s = fmaf(f0[i], f0[i], fmaf(f1[i], f1[i], s));
      const int base = vsub * LPV < 32 - LPV ? vsub * LPV : 32 - LPV;
      s = vector_sum<LPV>(s, base, c);
      const float mean = s * (1.f / D) + a.eps;
      float r = rsqrtf(mean);
      const bool far = mean > 0x1p120f || mean < 0x1p-80f;
      if (__any_sync(0xffffffffu, far)) {
        const float rf = far_rsqrt<D, LPV>(f0, f1, a.eps, base, c);
        if (far) r = rf;
      }
      const uint16_t* w = static_cast<const uint16_t*>(isq ? a.q_weight : a.k_weight);
      float w0[8], w1[8];
      unpack8(*reinterpret_cast<const uint4*>(w + 8 * c0), w0);
      unpack8(*reinterpret_cast<const uint4*>(w + 8 * c1), w1);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        f0[i] = f0[i] * r * w0[i];
        f1[i] = f1[i] * r * w1[i];
      }
    }
    if (rotated) {
      if (!a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float y0 = f0[i], y1 = f1[i];
          f0[i] = y0 * cs[i] - y1 * sn[i];
          f1[i] = y1 * cs[i] + y0 * sn[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const float y0 = f0[2 * i], y1 = f0[2 * i + 1], z0 = f1[2 * i], z1 = f1[2 * i + 1];
          f0[2 * i] = y0 * cs[i] - y1 * sn[i];
          f0[2 * i + 1] = y1 * cs[i] + y0 * sn[i];
          f1[2 * i] = z0 * cs[4 + i] - z1 * sn[4 + i];
          f1[2 * i + 1] = z1 * cs[4 + i] + z0 * sn[4 + i];
        }
      }
    }
    if (head[u] >= 0) {
      uint16_t* dst = isq ? static_cast<uint16_t*>(a.q_out) + t * a.q_out_stride + (int64_t)head[u] * D
                          : static_cast<uint16_t*>(a.k_out) + t * a.k_out_stride + (int64_t)(head[u] - a.num_q_heads) * D;
      uint4* const d0 = reinterpret_cast<uint4*>(dst + 8 * c0);
      uint4* const d1 = reinterpret_cast<uint4*>(dst + 8 * c1);
      if (p.stream_out) {
        __stcs(d0, pack8(f0));
        __stcs(d1, pack8(f1));
      } else {
        *d0 = pack8(f0);
        *d1 = pack8(f1);
      }
    }
  }
}

template <int D>
int launch_t(const NormRopeArgs& a, cudaStream_t stream) {
  constexpr int U = 2, VPW = 32 / (D / 16);
  NormRope p;
  p.a = a;
  p.heads = a.num_q_heads + a.num_kv_heads;
  p.stream_out = (int64_t)a.num_tokens * p.heads * D * 2 > (48ll << 20);  // of 126 MB of L2
  p.parts = (p.heads + VPW * U - 1) / (VPW * U);
  p.by_parts = FastDiv((uint32_t)p.parts);
  const int64_t warps = (int64_t)a.num_tokens * p.parts;
  if (warps >= (1ll << 31) - kNormWarps) return KV_INT4_ERR_SIZE;
  return launch_pdl(norm_rope_kernel<D, U>, dim3((unsigned)((warps + kNormWarps - 1) / kNormWarps)), kNormWarps * 32, 0,
                    stream, 1, p);
}

}  // namespace

int launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
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
