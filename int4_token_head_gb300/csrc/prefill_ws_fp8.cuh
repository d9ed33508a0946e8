// Warp-specialised prefill over the FP8 cache on the 5th-generation tensor
// cores (tcgen05), included by attention_fp8.cu for head sizes up to 192.
//
// One CTA per SM (all 512 TMEM columns); an item is 256 query rows (query
// token x q head of one kv group) in two halves of 128, the MMA's M.  A step
// is NK keys: 128 for head sizes up to 128 (a 128 x 128 score tile per half,
// full tensor rate), 64 at 192 (the accumulators leave no more TMEM).  Sixteen
// warps in three roles that meet only at mbarriers, each with its own item
// loop:
//   * dequant warps (8-14): claim the next item (longest first) and hand it on
//     through a two-entry ring; stage the step's K and V code rows (coalesced
//     cp.async, K and V apart, so that one's copies run during the other's
//     conversion); load the item's Q rows, divide each by its power of two and
//     store them as f16; convert K into one of two f16 tiles and V into one of
//     two; put the blocks' scales into a three-entry ring;
//   * MMA warp (15, lane 0 issues): S_h = Q_h K^T, then O_h += W_h V with the
//     weights W_h (f16 pairs over S_h's columns) read from TMEM.  Issue order
//     S0 S1 | WV0 S0' | WV1 S1' | ...: a half's softmax runs during the other's MMAs;
//   * softmax warps (0-3 half 0, 4-7 half 1): one query row per thread.  With
//     f_b = 2^e softmax_scale log2 e ks_b >= 0 and kv_b per block, the row's
//     maximum needs only the blocks' largest raw scores, and a weight is
//     exp2(fma(s, f_b, kv_b - m_ref)): one max, one fma and one exp2 per score.
//     m_ref moves (and the row's O in TMEM is rescaled) only when the maximum
//     passes it by more than 8: weights stay below 2^8, inside f16 whatever
//     the V scales.
// Shared operands are K-major (Q, K) or MN-major (V) tiles [D / 64][rows][128
// bytes] with the 16-byte chunk index XORed by row % 8.
//
// Hand-offs: mbarrier pairs, one per K/V tile, half or item ring entry, each
// waited once per completion, every wait bounded (a wait that runs out sets
// KV_INT4_DEV_TIMEOUT and a CTA-wide abort flag that ends every later wait).
//   ifull[e] / ifree[e]  item ring entry e written / read by all
//   kfull[b]  K tile b and the step's ring entry written (first step: Q too)
//   vfull[b]  V tile b written
//   kfree[b]  S0 and S1 that read K tile b complete
//   vfree[b]  WV0 and WV1 that read V tile b complete
//   sfull[h]  S_h complete (and every earlier MMA)
//   pfull[h]  W_h in TMEM, O_h rescaled if it had to be
//   odone     the item's last WV complete
// The ring entry of step j is rewritten at step j + 3, after S of step j + 1,
// which follows both halves' W of step j.  Query exponents are kept per item
// parity: an item's are rewritten two items later, when the item between has
// waited for the first one's last WV.

template <int D>
struct Fp8Ws {
  static constexpr int ROWS = 256;
  static constexpr int NK = D <= 128 ? 128 : 64;  // keys per step
  static constexpr int NB = NK / 16;              // cache blocks per step
  static constexpr int KB = (D + 63) / 64;        // 128-byte blocks of an f16 head vector
  static constexpr int CHR = D / 16;              // 16-byte chunks per code row
  static constexpr int QBYTES = ROWS * 128 * KB;
  static constexpr int KVBYTES = NK * 128 * KB;   // one K or V tile
  // staged code rows: as in the decode, swizzled where the row is a power of
  // two of chunks, else padded to an odd number of them
  static constexpr bool SWZ = Fp8Dec<D, 1>::SWZ;
  static constexpr int SROW = SWZ ? D : D + 16;
  static constexpr int STG = NK * SROW;           // K, then V
  static constexpr int RING = (4 * NB + 4) * 4;   // K scales, log2 V scales, 1 / V scales, block flags, all usable
  static constexpr int NRING = 3;
  static constexpr int NBARS = 18;
  static constexpr int S_COLS = NK, O_COL = 2 * NK;  // TMEM: S_h at h NK, O_h at 2 NK + h D
  static constexpr int SMEM = 1024 + QBYTES + 4 * KVBYTES + 2 * STG + NRING * RING + NBARS * 8 + 48 + 2 * ROWS;
  static constexpr int THREADS = 16 * 32;
  static constexpr int DQ = 7 * 32;  // dequant threads
  static_assert(O_COL + 2 * D <= 512 && SMEM <= 227 * 1024, "TMEM and shared memory");
};

__device__ __forceinline__ uint32_t fp8_sw128(int rows, int r, int c) {
  return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// a bounded wait that gives up at once after any wait of the CTA has run out
__device__ __forceinline__ bool fp8_wait(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  for (int n = 0; n < kMaxWaitIters; n++) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((n & 255) == 255 && *abort) return false;
  }
  *abort = 1;
  flag(status, KV_INT4_DEV_TIMEOUT);
  return false;
}
__device__ __forceinline__ void fp8_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fp8_dq_sync() { asm volatile("bar.sync 1, 224;\n" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(16 * 32, 1) prefill_ws_fp8_kernel(Common c, PlanView pv) {
  using G = Fp8Ws<D>;
  constexpr int KSTEPS = D / 16;
  constexpr int NK = G::NK, NB = G::NB, ROWS = G::ROWS;
  constexpr uint32_t IDESC_S = umma_idesc_f16(128, NK, false);
  constexpr uint32_t IDESC_O = umma_idesc_f16(128, D, true);
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* const sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const sQ = sm;                     // [KB][256 rows][128 B], swizzled
  uint8_t* const sK = sQ + G::QBYTES;         // two K tiles [KB][NK][128 B]
  uint8_t* const sV = sK + 2 * G::KVBYTES;    // two V tiles
  uint8_t* const stg = sV + 2 * G::KVBYTES;   // staged K rows, V rows
  uint8_t* const ring = stg + 2 * G::STG;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ring + G::NRING * G::RING);
  int* const sitem = reinterpret_cast<int*>(bars + G::NBARS);  // item ring [2][4], abort flag
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(sitem + 10);
  volatile int* const abort_flag = sitem + 8;
  int8_t* const sexp = reinterpret_cast<int8_t*>(sitem + 12);  // query exponents [item parity][256]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  enum { KFULL = 0, VFULL = 2, KFREE = 4, VFREE = 6, SFULL = 8, PFULL = 10, ODONE = 12, DRAIN = 13, IFULL = 14, IFREE = 16 };
  auto bar = [&](int i) { return smem_addr(&bars[i]); };
  if (tid == 0) {
    for (int b = 0; b < 2; b++) {
      mbar_init(bar(KFULL + b), 7);
      mbar_init(bar(VFULL + b), 7);
      mbar_init(bar(KFREE + b), 1);
      mbar_init(bar(VFREE + b), 1);
      mbar_init(bar(SFULL + b), 1);
      mbar_init(bar(PFULL + b), 4);
      mbar_init(bar(IFULL + b), 1);
      mbar_init(bar(IFREE + b), 9);  // the eight softmax warps and the MMA warp
    }
    mbar_init(bar(ODONE), 1);
    mbar_init(bar(DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(smem_addr(tslot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const int n_items = pv.plan[1];
  auto item_at = [&](int e) { return make_int4(sitem[4 * e], sitem[4 * e + 1], sitem[4 * e + 2], sitem[4 * e + 3]); };
  // a consumer's wait for ring entry e, warp-uniform
  auto take_item = [&](int e, uint32_t& ph, int4& item) {
    const bool ok = __all_sync(0xffffffffu, fp8_wait(bar(IFULL + e), (ph >> e) & 1, abort_flag, c.status));
    ph ^= 1u << e;
    if (!ok) return false;
    item = item_at(e);
    __syncwarp();
    if (lane == 0) fp8_arrive(bar(IFREE + e));
    return item.x >= 0;
  };
  // registers: 128 a thread at launch (65,536); the softmax warpgroups take
  // 160, the others 96 (2 x 128 x 160 + 2 x 128 x 96 = 65,536)
  if (warp < 8) {
    // ======================= softmax warpgroups =======================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;\n");
    uint32_t ph_sfull = 0, ph_odone = 0, ph_ifull = 0;
    const float qs = fabsf(c.qscale);  // its sign is in Q'
#pragma unroll 1
    for (int itc = 0;; itc++) {
      int4 item;
      const int e = itc & 1;
      if (!take_item(e, ph_ifull, item)) break;
      const int seq = item.x, h = item.y, tile = item.z, nkb = item.w;
      const int q0 = c.qsl[seq], ql = c.qsl[seq + 1] - q0;
      const int L = c.seq_lens[seq], ctx = L - ql;
      const int tok0 = tile * c.tile_tokens;
      const int nrows = min(c.tile_tokens, ql - tok0) * c.group;
      const int kb0 = window_lo(c, ctx + tok0) >> 4;
      const int nsteps = (nkb - kb0 + NB - 1) / NB;
      const int hf = warp >> 2;
      const int r = tid;  // row of the item
      const int j = (int)c.gdiv.div((uint32_t)r);
      const bool rok = r < nrows;
      const int qp = ctx + tok0 + (rok ? j : 0);
      const int lim = c.causal ? min(L, qp + 1) : L;
      const int lo = window_lo(c, qp);
      const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + NK * hf + lane_off, tO = tmem + G::O_COL + hf * D + lane_off;
      float m_ref = -INFINITY, l_run = 0.f, cf = 0.f;
#pragma unroll 1
      for (int st = 0; st < nsteps; st++) {
        const float* re = reinterpret_cast<const float*>(ring + (st % G::NRING) * G::RING);
        const float* kvf = re + NB;
        const float* ivs = re + 2 * NB;
        const int* ok = reinterpret_cast<const int*>(re + 3 * NB);
        fp8_wait(bar(SFULL + hf), ph_sfull, abort_flag, c.status);
        ph_sfull ^= 1;
        tc_fence_after();
        if (st == 0) cf = qs * exp2_int(sexp[e * ROWS + r]);
        const int pos0 = (kb0 + st * NB) * 16;
        // a step wholly inside the row's visible range over usable blocks needs no mask
        const bool full = pos0 >= lo && pos0 + NK <= lim && ok[NB] != 0;
        auto visible = [&](int k) { return ok[k >> 4] != 0 && pos0 + k >= lo && pos0 + k < lim; };
        float mx = -INFINITY;
#pragma unroll
        for (int u = 0; u < NK / 32; u++) {
          float s[32];
          tmem_ld32(tS + 32 * u, s);
          if (!full) {
#pragma unroll
            for (int k = 0; k < 32; k++) s[k] = visible(32 * u + k) ? s[k] : -INFINITY;
          }
#pragma unroll
          for (int b = 0; b < 2; b++) {
            const float* t = s + 16 * b;
            const float a = fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]), fmax3(t[6], t[7], t[8]));
            const float d = fmax3(fmax3(t[9], t[10], t[11]), fmax3(t[12], t[13], t[14]), t[15]);
            const float top = fmaxf(a, d);
            mx = fmaxf(mx, top == -INFINITY ? -INFINITY : fmaf(top, cf * re[2 * u + b], kvf[2 * u + b]));
          }
        }
        const bool grow = m_ref != -INFINITY && mx > m_ref + 8.f;
        const float alpha = grow ? fast_exp2(m_ref - mx) : 1.f;
        if (grow || m_ref == -INFINITY) m_ref = mx;
        if (__any_sync(0xffffffffu, grow)) {
          // O of this half is complete up to the previous step (S_h of this step was issued after it)
#pragma unroll 1
          for (int cc = 0; cc < D / 32; cc++) {
            float o[32];
            tmem_ld32(tO + cc * 32, o);
#pragma unroll
            for (int i = 0; i < 32; i++) o[i] *= alpha;
            tmem_st32(tO + cc * 32, o);
          }
        }
        l_run *= alpha;
        const float mu = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll
        for (int u = 0; u < NK / 32; u++) {
          float s[32];
          tmem_ld32(tS + 32 * u, s);
          uint32_t w[16];
#pragma unroll
          for (int b = 0; b < 2; b++) {
            const float f = cf * re[2 * u + b], o = kvf[2 * u + b] - mu;
            const float2 f2 = make_float2(f, f), o2 = make_float2(o, o);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float2 t = f2fma(make_float2(s[16 * b + k], s[16 * b + k + 1]), f2, o2);
              float2 p = make_float2(fast_exp2(t.x), fast_exp2(t.y));
              if (!full) {
                p.x = visible(32 * u + 16 * b + k) ? p.x : 0.f;
                p.y = visible(32 * u + 16 * b + k + 1) ? p.y : 0.f;
              }
              sum = f2add(sum, p);
              w[8 * b + k / 2] = pack_f16x2(p.x, p.y);
            }
            l_run = fmaf(sum.x + sum.y, ivs[2 * u + b], l_run);
          }
          // the weights over the row's first NK / 2 columns: columns [16 u, 16 u + 16) have been read
          asm volatile(
              "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::
                  "r"(tS + 16 * u),
              "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]),
              "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
              : "memory");
        }
        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) fp8_arrive(bar(PFULL + hf));
      }

      // ---- epilogue: normalise, bf16, stored from registers ----
      fp8_wait(bar(ODONE), ph_odone, abort_flag, c.status);
      ph_odone ^= 1;
      tc_fence_after();
      const bool none = l_run == 0.f;  // the row saw no usable key: zeros
      const float inv = none ? 0.f : 1.f / l_run;
      uint16_t* const orow = c.out + (long long)(q0 + tok0 + (rok ? j : 0)) * c.out_stride +
                             (long long)(h * c.group + (rok ? r - j * c.group : 0)) * D;
      const bool al32 = ((reinterpret_cast<uintptr_t>(c.out) | (uintptr_t)(c.out_stride * 2) | (uintptr_t)(D * 2)) & 31) == 0;
#pragma unroll 1
      for (int base = 0; base < D; base += 32) {
        float o[32];
        tmem_ld32(tO + base, o);
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; i++) w[i] = none ? 0u : pack_bf16x2_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
        if (rok) {
          if (al32) {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(orow + base + 2 * i), "r"(w[i]),
                           "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                           "r"(w[i + 7])
                           : "memory");
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(orow + base + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
          }
        }
      }
    }
  } else {
    // ==================== dequant and MMA warpgroups ====================
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;\n");
    uint32_t ph_kfull = 0, ph_vfull = 0, ph_kfree = 0, ph_vfree = 0, ph_pfull = 0;
    if (warp < 15) {
      // ================= dequant warps =================
      const int dt = tid - 256;
      uint32_t ph_ifree = 0;
      int prev_steps = 0;
      // the previous item's MMA completions that its step loop did not wait
      // for: the S of its last two steps (every read of its Q and K tiles),
      // the last WV of each V tile (every W, so every read of its ring entries)
      auto wait_kfree_tail = [&](int ns) {
        for (int st = ns - 2 < 0 ? 0 : ns - 2; st < ns; st++) {
          fp8_wait(bar(KFREE + (st & 1)), (ph_kfree >> (st & 1)) & 1, abort_flag, c.status);
          ph_kfree ^= 1u << (st & 1);
        }
      };
      auto wait_vfree_tail = [&](int ns) {
        for (int b = 0; b < 2 && b < ns; b++) {
          fp8_wait(bar(VFREE + b), (ph_vfree >> b) & 1, abort_flag, c.status);
          ph_vfree ^= 1u << b;
        }
      };
#pragma unroll 1
      for (int itc = 0;; itc++) {
        const int e = itc & 1;
        if (dt == 0) {
          if (itc >= 2) {
            fp8_wait(bar(IFREE + e), (ph_ifree >> e) & 1, abort_flag, c.status);
            ph_ifree ^= 1u << e;
          }
          const int4 it = prefill_item(c, pv, *abort_flag ? n_items : atomicAdd(&pv.plan[2], 1), n_items);
          sitem[4 * e] = it.x;
          sitem[4 * e + 1] = it.y;
          sitem[4 * e + 2] = it.z;
          sitem[4 * e + 3] = it.w;
          fp8_arrive(bar(IFULL + e));
        }
        fp8_dq_sync();
        const int4 item = item_at(e);
        if (item.x < 0) {
          wait_kfree_tail(prev_steps);
          wait_vfree_tail(prev_steps);
          break;
        }
        const int seq = item.x, h = item.y, tile = item.z, nkb = item.w;
        const int q0 = c.qsl[seq], ql = c.qsl[seq + 1] - q0;
        const int L = c.seq_lens[seq], ctx = L - ql;
        const int tok0 = tile * c.tile_tokens;
        const int nrows = min(c.tile_tokens, ql - tok0) * c.group;
        const int kb0 = window_lo(c, ctx + tok0) >> 4;
        const int nsteps = (nkb - kb0 + NB - 1) / NB;
        // lane b < NB of every warp holds the id of block b of a step (-1: none)
        auto block_of = [&](int st) -> int {
          const int kb = kb0 + st * NB + lane;
          return st < nsteps && lane < NB && kb < nkb ? c.block_table[(long long)seq * c.max_blocks + kb] : -1;
        };
        // copies of the step's K (kv 0) or V (kv 1) rows; rows behind the
        // sequence and unusable blocks are zeros (a NaN code would survive its
        // zero weight)
        auto issue = [&](int st, int kv, int blk) {
          const uint8_t* cache = kv ? c.v_cache : c.k_cache;
          uint8_t* sb = stg + kv * G::STG;
          const int p0 = (kb0 + st * NB) * 16;
#pragma unroll
          for (int q = dt; q < NK * G::CHR; q += G::DQ) {
            const int row = q / G::CHR, col = q - row * G::CHR;
            const int id = __shfl_sync(0xffffffffu, blk, row >> 4);
            const bool in = id >= 0 && id < c.num_blocks && p0 + row < L;
            const uint8_t* src = cache + (in ? (long long)id * c.geo.cblk + (row & 15) * c.geo.crow + (long long)h * D + col * 16 : 0);
            const int pos = G::SWZ ? col ^ Fp8Dec<D, 1>::swz(row & 15) : col;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_addr(sb + row * G::SROW + pos * 16)),
                         "l"(src), "r"(in ? 16 : 0));
          }
          cp_async_commit();
        };
        // the staged K or V codes as f16 into a tile: a thread takes 16 codes
        // of one key, consecutive threads consecutive keys (the eight keys of
        // a load or store phase fall in eight bank groups)
        auto convert = [&](uint8_t* tile_dst, int kv) {
          const uint8_t* sb = stg + kv * G::STG;
#pragma unroll 2
          for (int q = dt; q < NK * G::CHR; q += G::DQ) {
            const int k = q & (NK - 1), g = q / NK;
            const int pos = G::SWZ ? g ^ Fp8Dec<D, 1>::swz(k & 15) : g;
            const uint4 x = *reinterpret_cast<const uint4*>(sb + k * G::SROW + pos * 16);
            uint4 a, b;
            e4m3x4_to_f16x2(x.x, a.x, a.y);
            e4m3x4_to_f16x2(x.y, a.z, a.w);
            e4m3x4_to_f16x2(x.z, b.x, b.y);
            e4m3x4_to_f16x2(x.w, b.z, b.w);
            *reinterpret_cast<uint4*>(tile_dst + fp8_sw128(NK, k, 2 * g)) = a;
            *reinterpret_cast<uint4*>(tile_dst + fp8_sw128(NK, k, 2 * g + 1)) = b;
          }
        };
        int blk = block_of(0), blk_next = block_of(1);
        // the first warp's lanes hold their block's scales a step ahead
        float ks = 0.f, vs = 1.f;
        auto load_scales = [&]() {
          const bool ok = dt < NB && blk >= 0 && blk < c.num_blocks;
          const long long at = ok ? (long long)blk * c.hkv + h : 0;
          ks = ok ? c.k_scale[at] : 0.f;
          vs = ok ? c.v_scale[at] : 1.f;
        };
        load_scales();
        if (nsteps > 0) {  // the staging buffers are free: the previous item's last conversions are done
          issue(0, 0, blk);
          issue(0, 1, blk);
        }
        wait_kfree_tail(prev_steps);
        // the item's Q rows, once every S of the previous item is complete
        {
          constexpr int LPR = D <= 64 ? 8 : D <= 128 ? 16 : 32;  // lanes per row (D / 8 of them with a chunk)
          constexpr int RPW = 32 / LPR;
          const int sub = lane / LPR, ch = lane - sub * LPR;
          const uint32_t neg = c.qscale < 0.f ? 0x80008000u : 0u;
          constexpr int U = 4;
#pragma unroll 1
          for (int r0 = (warp - 8) * RPW; r0 < ROWS; r0 += 7 * RPW * U) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; u++) {
              const int r = r0 + u * 7 * RPW + sub;
              x[u] = make_uint4(0, 0, 0, 0);
              if (r < nrows && ch < D / 8) {
                const int tj = (int)c.gdiv.div((uint32_t)r), tjj = r - tj * c.group;
                x[u] = *reinterpret_cast<const uint4*>(c.q + (long long)(q0 + tok0 + tj) * c.q_stride +
                                                       (long long)(h * c.group + tjj) * D + ch * 8);
              }
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
              const int r = r0 + u * 7 * RPW + sub;
              uint32_t am = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                                     __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
              am = max(am & 0xffffu, am >> 16);
#pragma unroll
              for (int o = 1; o < LPR; o <<= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
              const int qe = q_exponent(am);
              const float mul = exp2_int(-qe);
              const uint32_t w[4] = {x[u].x ^ neg, x[u].y ^ neg, x[u].z ^ neg, x[u].w ^ neg};
              uint32_t o[4];
#pragma unroll
              for (int i = 0; i < 4; i++) o[i] = pack_f16x2(bf16lo_to_f32(w[i]) * mul, bf16hi_to_f32(w[i]) * mul);
              if (r < ROWS && ch < D / 8)
                *reinterpret_cast<uint4*>(sQ + fp8_sw128(ROWS, r, ch)) = make_uint4(o[0], o[1], o[2], o[3]);
              if (r < ROWS && ch == 0) sexp[e * ROWS + r] = (int8_t)qe;
            }
          }
        }
        // V tiles and the first ring entries: every WV of the previous item is complete
        wait_vfree_tail(prev_steps);
#pragma unroll 1
        for (int j = 0; j < nsteps; j++) {
          const int b = j & 1;
          cp_async_wait<1>();
          fp8_dq_sync();  // every thread's K copies of step j have landed
          if (j >= 2) {
            fp8_wait(bar(KFREE + b), (ph_kfree >> b) & 1, abort_flag, c.status);  // S of step j - 2
            ph_kfree ^= 1u << b;
          }
          if (dt < 32) {  // the step's scales
            float* re = reinterpret_cast<float*>(ring + (j % G::NRING) * G::RING);
            const bool ok = blk >= 0 && blk < c.num_blocks;  // lanes < NB
            const int kb = kb0 + j * NB + lane;
            if (lane < NB) {
              re[lane] = ks;
              re[NB + lane] = (float)exp_of(vs);
              re[2 * NB + lane] = __uint_as_float((254u << 23) - (__float_as_uint(vs) & 0x7f800000u));
              reinterpret_cast<int*>(re)[3 * NB + lane] = ok;
              if (!ok && kb < nkb) flag(c.status, KV_INT4_DEV_BAD_BLOCK);
            }
            const bool all = __all_sync(0xffffffffu, ok || lane >= NB);
            if (lane == 0) reinterpret_cast<int*>(re)[4 * NB] = all;
          }
          convert(sK + b * G::KVBYTES, 0);
          fence_proxy_async_smem();  // the tile is read by the tensor cores
          __syncwarp();
          if (lane == 0) fp8_arrive(bar(KFULL + b));
          fp8_dq_sync();  // every thread is done with the staged K rows
          if (j + 1 < nsteps) issue(j + 1, 0, blk_next);
          else cp_async_commit();
          cp_async_wait<1>();
          fp8_dq_sync();  // the V copies of step j have landed
          if (j >= 2) {
            fp8_wait(bar(VFREE + b), (ph_vfree >> b) & 1, abort_flag, c.status);  // WVs of step j - 2
            ph_vfree ^= 1u << b;
          }
          convert(sV + b * G::KVBYTES, 1);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) fp8_arrive(bar(VFULL + b));
          fp8_dq_sync();  // done with the staged V rows
          if (j + 1 < nsteps) issue(j + 1, 1, blk_next);
          else cp_async_commit();
          blk = blk_next;
          load_scales();
          blk_next = block_of(j + 2);
        }
        prev_steps = nsteps;
      }
      cp_async_wait<0>();
    } else {
      // ================= MMA warp =================
      const bool leader = lane == 0;
      uint32_t ph_ifull = 0;
      const uint64_t dq = umma_desc(smem_addr(sQ), 16, 1024);
      const uint64_t dk = umma_desc(smem_addr(sK), 16, 1024);
      const uint64_t dv = umma_desc(smem_addr(sV), NK * 128, 1024);
#pragma unroll 1
      for (int itc = 0;; itc++) {
        int4 item;
        if (!take_item(itc & 1, ph_ifull, item)) break;
        const int seq = item.x, tile = item.z, nkb = item.w;
        const int ql = c.qsl[seq + 1] - c.qsl[seq];
        const int ctx = c.seq_lens[seq] - ql;
        const int kb0 = window_lo(c, ctx + tile * c.tile_tokens) >> 4;
        const int nsteps = (nkb - kb0 + NB - 1) / NB;
        auto issue_s = [&](int hh, int st) {
          if (leader) {
            const uint64_t kt = dk + (uint64_t)((st & 1) * (G::KVBYTES >> 4));
#pragma unroll
            for (int ks = 0; ks < KSTEPS; ks++)
              umma_f16(tmem + NK * hh, dq + (uint64_t)(((ks >> 2) * ROWS * 128 + hh * 128 * 128 + (ks & 3) * 32) >> 4),
                       kt + (uint64_t)(((ks >> 2) * NK * 128 + (ks & 3) * 32) >> 4), IDESC_S, ks > 0);
          }
        };
        auto issue_wv = [&](int hh, int b, bool first) {
          if (leader) {
            const uint64_t vt = dv + (uint64_t)(b * (G::KVBYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < NB; kk++)
              umma_f16_ts(tmem + G::O_COL + hh * D, tmem + NK * hh + kk * 8, vt + (uint64_t)(kk * (2048 >> 4)), IDESC_O,
                          !first || kk > 0);
          }
        };
        auto commit = [&](int i) {
          if (leader) umma_commit(bar(i));
          __syncwarp();
        };
        if (nsteps > 0) {  // kfull of step 0 also covers the item's Q rows
          fp8_wait(bar(KFULL), ph_kfull & 1, abort_flag, c.status);
          ph_kfull ^= 1;
          tc_fence_after();
          issue_s(0, 0);
          commit(SFULL);
          issue_s(1, 0);
          commit(SFULL + 1);
          commit(KFREE);
        }
#pragma unroll 1
        for (int j = 0; j < nsteps; j++) {
          const int b = j & 1, nb = (j + 1) & 1;
          fp8_wait(bar(VFULL + b), (ph_vfull >> b) & 1, abort_flag, c.status);
          ph_vfull ^= 1u << b;
          if (j + 1 < nsteps) {
            fp8_wait(bar(KFULL + nb), (ph_kfull >> nb) & 1, abort_flag, c.status);
            ph_kfull ^= 1u << nb;
          }
          fp8_wait(bar(PFULL), ph_pfull & 1, abort_flag, c.status);
          ph_pfull ^= 1;
          tc_fence_after();
          issue_wv(0, b, j == 0);
          if (j + 1 < nsteps) {
            issue_s(0, j + 1);
            commit(SFULL);
          }
          fp8_wait(bar(PFULL + 1), (ph_pfull >> 1) & 1, abort_flag, c.status);
          ph_pfull ^= 2;
          tc_fence_after();
          issue_wv(1, b, j == 0);
          commit(VFREE + b);
          if (j + 1 < nsteps) {
            issue_s(1, j + 1);
            commit(SFULL + 1);
            commit(KFREE + nb);
          }
        }
        commit(ODONE);
      }
    }
  }
  if (warp == 15) {
    // after a time-out MMAs may still be in flight: they end by themselves
    // and must end before the columns are freed
    if (lane == 0) umma_commit(bar(DRAIN));
    __syncwarp();
    if (!mbar_wait_bounded(bar(DRAIN), 0)) flag(c.status, KV_INT4_DEV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}
