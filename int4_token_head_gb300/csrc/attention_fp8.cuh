// The FP8 attention's kernels and launch helpers, included by attention_fp8.cu,
// attention_shared_fp8.cu and mass_fp8.cu in a namespace of their own.
template <int PREFILL, bool SH = false>
__global__ void __launch_bounds__(kPrepThreads) plan_fp8_kernel(Common c, PlanView pv) {
  pdl_trigger();
  pdl_wait();
  // The schedule's number: another one for every schedule built in this
  // workspace, whatever the memory held before.  Who reads it with acquire
  // sees the schedule and all that the kernels before it wrote
  int number = 0;
  if (PREFILL > 0 && threadIdx.x == 0) number = pv.plan[5];
  if constexpr (SH) build_shared(c, pv);
  build_schedule<true, PREFILL, SH>(c, pv);
  if constexpr (PREFILL > 0) {
    __syncthreads();
    if (threadIdx.x == 0) st_release(&pv.plan[5], number + 1);
  }
}

// A query row's power of two from its largest bf16 magnitude bits: rows are
// multiplied by 2^-e (so that |q'| < 2) and scores by 2^e.  Rows of zeros and
// subnormals use the smallest exponent; rows with an infinity or NaN end as NaN.
__device__ __forceinline__ int q_exponent(uint32_t amax_bits) {
  return min(max((int)(amax_bits >> 7) - 127, -126), 126);
}

#include "decode_fp8.cuh"
#include "prefill_fp8.cuh"
#include "prefill_ws_fp8.cuh"

// ---------------------------------------------------------------------------
// host launcher
// ---------------------------------------------------------------------------
// cuTensorMapEncodeTiled, reached through the runtime (the library links the
// static runtime only); null if the driver does not have it
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

template <bool SH = false>
int launch_plan(const Common& c, const PlanView& pv, bool may_prefill, bool may_split, cudaStream_t stream) {
  return launch_pdl(may_split ? plan_fp8_kernel<2, SH> : may_prefill ? plan_fp8_kernel<1, SH> : plan_fp8_kernel<0, SH>, dim3(1),
                    kPrepThreads, 0, stream, 1, c, pv);
}

// the tensor map of query rows: boxes of 64 elements x a kv head's q heads x
// tile_tokens tokens; false where there is none (rows that overlap, say)
bool make_q_map(CUtensorMap* m, const void* q, int64_t q_stride, int tokens, int q_heads, int head_size, int group,
                int tile_tokens) {
  const EncodeTiled enc = encode_tiled();
  const cuuint64_t hq = q_heads, d = head_size;
  if (!enc || (tokens > 1 && q_stride < (int64_t)(hq * d))) return false;
  const cuuint64_t dims[3] = {d, hq, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {d * 2, (tokens > 1 ? (cuuint64_t)q_stride : hq * d) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tile_tokens}, ones[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the tensor maps of a call's prefill; false where its tensors have no such
// map (query rows that overlap, say)
template <int D>
bool make_maps(const AttnArgs& a, int tile_tokens, Fp8Maps* m) {
  using G = Fp8Ws<D>;
  const EncodeTiled enc = encode_tiled();
  const cuuint64_t hkv = a.num_kv_heads, rows = (cuuint64_t)a.num_blocks * 16;
  if (!enc || rows == 0 || rows >= (1ull << 31) ||
      !make_q_map(&m->q, a.q, a.q_stride, a.num_q_tokens, a.num_q_heads, D, a.num_q_heads / a.num_kv_heads, tile_tokens))
    return false;
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  const cuuint64_t dims[4] = {G::W, D / G::W, hkv, rows};
  const cuuint64_t strides[3] = {G::W, D, hkv * D};
  const cuuint32_t box[4] = {G::W, D / G::W, 1, 16};
  const CUtensorMapSwizzle sw = G::W == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                : G::W == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                             : CU_TENSOR_MAP_SWIZZLE_32B;
  for (int i = 0; i < 2; i++)
    if (enc(i ? &m->v : &m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(i ? a.v_cache : a.k_cache), dims,
            strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}
