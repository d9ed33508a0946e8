// Device helpers of the FP8 block-scaled cache: E4M3 codes with one
// power-of-two scale per (block of 16 tokens, kv head).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace kvint4 {

// ---------------------------------------------------------------------------
// Programmatic dependent launch: a kernel may be scheduled while the one before
// it on the stream still runs, and waits there (pdl_wait, before it touches
// any memory that another kernel writes or reads) until that one is complete
// and its writes are visible.  A kernel lets the next one start (pdl_trigger)
// once all its CTAs run.  Between short kernels this hides the launch latency.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// A kernel that starts on work before its pdl_wait may use what it has found
// published by st_release with ld_acquire, and what the publisher could see.
__device__ __forceinline__ void st_release(int32_t* p, int32_t v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;\n" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ int32_t ld_acquire(const int32_t* p) {
  int32_t v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// launches on `stream` with that permission, as clusters of `cluster` CTAs;
// KV_INT4_OK or KV_INT4_ERR_CUDA
template <typename... P, typename... A>
inline int launch_pdl(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster,
                      A&&... args) {
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, static_cast<A&&>(args)...) == cudaSuccess) return KV_INT4_OK;
  cudaGetLastError();
  return KV_INT4_ERR_CUDA;
}

// Scales are 2^k with k in [kFp8MinExp, kFp8MaxExp].  E4M3 keeps four
// significant bits at every magnitude, so a power of two loses nothing against
// absmax / 448, and it moves codes between scales by their exponent alone
// (exact unless a code becomes subnormal).
constexpr int kFp8MinExp = -60, kFp8MaxExp = 60;

// Attention's weights carry their block's V scale, 2^(s + kv - M) with M the
// largest s + kv, and the denominator takes it out again, 2^-kv times their sum.
// M <= s_max + 61 (prefill rounds it up), so a key whose score is g below the
// largest has a weight of at least 2^(kv - 61 - g): a normal fp32 number for
// g <= 43 if kv >= -22.  Blocks
// below that (of zeros, say) may weigh too little for fp32 beside a block of large
// V and still count in the denominator: their share is summed from weights in
// units of 2^-22.  Their products with V are below fp32's range then, as they
// should be.
constexpr int kFp8LowExp = -22;

// 2^d, d <= 0, as two factors: a sum in units of 2^-kv times one and then the
// other keeps what 2^d alone would flush to zero
struct Exp2Pair {
  float a, b;
  __device__ __forceinline__ explicit Exp2Pair(float d) : a(fast_exp2(fmaxf(d, -100.f))), b(fast_exp2(fminf(d + 100.f, 0.f))) {}
  __device__ __forceinline__ float both() const { return a * b; }
  __device__ __forceinline__ float of(float x) const { return x * a * b; }
};

// 2^e as fp32, e in [-126, 127]
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }
// the exponent field of a positive normal fp32, unbiased
__device__ __forceinline__ int exp_of(float x) { return (int)(__float_as_uint(x) >> 23) - 127; }

// smallest k in range with a <= 448 * 2^k, a a finite bf16 magnitude (its 15
// bits): a = 1.m * 2^e, 448 = 1.75 * 2^8, and 1.m > 1.75 when m > 96 / 128
__device__ __forceinline__ int fp8_exponent(uint32_t a) {
  const int k = (int)(a >> 7) - 127 - 8 + ((a & 0x7fu) > 96u);
  return min(max(k, kFp8MinExp), kFp8MaxExp);
}
// the exponent of a stored scale; kFp8MaxExp + 1 for anything that no write
// stores (a block that was not begun)
__device__ __forceinline__ int fp8_scale_exponent(float s) {
  const uint32_t b = __float_as_uint(s);
  const int k = (int)(b >> 23) - 127;
  return (b & 0x807fffffu) == 0 && k >= kFp8MinExp && k <= kFp8MaxExp ? k : kFp8MaxExp + 1;
}

// two E4M3 codes (low 16 bits of w, the first in the low byte) as f16x2, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
// the same for both halves of a word
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// four floats to E4M3, nearest even, saturating at +-448
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float x0, float x1, float x2, float x3) {
  uint32_t r;
  asm("{\n .reg .b16 a, b;\n cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n "
      "mov.b32 %0, {a, b};\n}\n"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

// ---------------------------------------------------------------------------
// The tokens of a call by cache block.  Sequence i's tokens are its last
// n_i = start[i + 1] - start[i] positions, so they touch consecutive blocks of
// its table row.  Work unit u is one touched block: sequence i owns the units
// from (start[i] >> 4) + 2 i on, always enough for its blocks
// (n + 30 >> 4 <= 2 + (start[i + 1] >> 4) - (start[i] >> 4)), so a unit finds
// its sequence by a search over start alone and the launch needs no
// schedule; units past a sequence's last block are empty.  With one token per
// sequence at most, unit i is sequence i.
// ---------------------------------------------------------------------------
struct Fp8Seqs {
  const int32_t* block_table;
  int max_blocks;
  const int32_t* seq_lens;
  const int32_t* start;  // query_start_loc
  int num_seqs;
  int num_tokens;
  int max_len;  // bound of n_i
  int num_blocks;
  int32_t* status;
};

inline int64_t fp8_units(int num_seqs, int num_tokens, int max_len) {
  return max_len <= 1 ? num_seqs : (int64_t)(num_tokens >> 4) + 2ll * num_seqs;
}

struct Fp8Unit {
  int64_t block;  // cache block (meaningless when bad)
  int r0, r1;     // rows of the block that the call's tokens fill: [r0, r1)
  int64_t token0; // token of row r0
  bool bad;       // the table's entry is no block
};

__device__ __forceinline__ bool fp8_seq_ok(const Fp8Seqs& a, int q0, int q1, int L) {
  return q0 >= 0 && q1 <= a.num_tokens && q1 >= q0 && L >= q1 - q0 && q1 - q0 <= a.max_len &&
         (int64_t)L <= (int64_t)a.max_blocks * 16;
}

// reports sequences whose metadata is inconsistent (their units are skipped)
__device__ __forceinline__ void fp8_check_seqs(const Fp8Seqs& a) {
  for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x)
    if (!fp8_seq_ok(a, a.start[i], a.start[i + 1], a.seq_lens[i])) flag(a.status, KV_INT4_DEV_BAD_SEQ);
}

// unit u, by a whole warp; false for an empty unit
__device__ __forceinline__ bool fp8_unit(const Fp8Seqs& a, int u, Fp8Unit* out) {
  const int lane = threadIdx.x & 31;
  int i = u, j = 0;
  if (a.max_len > 1) {
    // largest i with (start[i] >> 4) + 2 i <= u (32-ary search)
    int lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
      const int64_t span = hi - lo;
      const int probe = lo + (int)(span * lane / 32);
      const bool le = lane == 0 || (int64_t)(a.start[probe] >> 4) + 2ll * probe <= u;
      const unsigned m = __ballot_sync(0xffffffffu, le);
      const int last = 31 - __clz(m);
      const int nlo = lo + (int)(span * last / 32);
      const int nhi = last == 31 ? hi : lo + (int)(span * (last + 1) / 32);
      lo = nlo;
      hi = nhi > nlo ? nhi : nlo + 1;
    }
    i = lo;
  }
  const int q0 = a.start[i], q1 = a.start[i + 1], L = a.seq_lens[i];
  if (!fp8_seq_ok(a, q0, q1, L) || q0 == q1) return false;
  if (a.max_len > 1) j = u - ((q0 >> 4) + 2 * i);
  const int p0 = L - (q1 - q0);
  const int b = (p0 >> 4) + j;
  if (j < 0 || b > (L - 1) >> 4) return false;
  const int blk = a.block_table[(int64_t)i * a.max_blocks + b];
  out->bad = blk < 0 || blk >= a.num_blocks;
  out->block = blk;
  out->r0 = j == 0 ? p0 & 15 : 0;
  out->r1 = min(16, L - 16 * b);
  out->token0 = (int64_t)q0 + (16 * b + out->r0 - p0);
  return true;
}

}  // namespace kvint4
