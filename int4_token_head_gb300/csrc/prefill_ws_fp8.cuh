// Warp-specialised prefill over the FP8 cache on the 5th-generation tensor
// cores (tcgen05), included by attention_fp8.cu.
//
// One CTA per SM (all 512 TMEM columns); an item is 256 query rows (query
// token x q head of one kv group) in two halves of 128, the MMA's M.  A step
// is NK keys: 128 for head sizes up to 128 (a 128 x 128 score tile per half,
// full tensor rate), 64 above (the accumulators leave no more TMEM, the K and V
// tiles no more shared memory).  At 256 an item is one half, 128 rows: two
// accumulators would fill TMEM.  Warps in five roles that meet only at mbarriers
// (numbers for two halves):
//   * producer warp (24): claims items (longest first) and hands them on
//     through a two-entry ring; TMA copies of the item's Q rows (bf16, straight
//     into the MMA's swizzled tile) and of the step's K and V code blocks (one
//     box per block; a block that the table does not name is a box outside the
//     tensor, which arrives as zeros); the blocks' scales into a three-entry ring;
//   * convert warps (16-19 K, 20-23 V): K codes into one of two bf16 tiles, V
//     codes into one of two f16 tiles, exactly.  K meets the unconverted bf16
//     queries, so an item starts without any work on Q; V meets the f16 weights;
//   * MMA warp (25, one elected lane issues): S_h = Q_h K^T, then O_h += W_h V with the
//     weights W_h (f16 pairs over S_h's columns) read from TMEM.  Issue order
//     S0 S1 | WV0 S0' | WV1 S1' | ...: a half's softmax runs during the other's MMAs;
//   * softmax warps (0-7 half 0, 8-15 half 1): two threads per query row, one
//     for each half of the step's keys (the half's chain S -> softmax -> WV is
//     what bounds a step; 4700 cycles with one thread per row).  With
//     f_b = |softmax_scale| log2 e ks_b (a negative scale's sign is in K) and
//     kv_b per block, a weight is exp2(fma(s, f_b, kv_b - m_ref)).  m_ref moves to
//     the row's maximum (and its O in TMEM is rescaled) only in the step where the
//     row first sees a usable key and when a step's weights add up to more than
//     2^14: they stay inside f16 whatever the V scales, and most steps need no
//     maximum (one fma, one exp2, one add and half a conversion per score).  The
//     two warps of a row agree on that by a barrier that votes; the weights stay
//     in registers until then, S is whole.
// 8 causal prompts of 512 to 2048 tokens, 32/8 heads of 128: 146 us a call = 0.35
// of the measured bf16 tensor rate (140 us as replays on the same tensors), about
// 4300 cycles per step where the MMAs need 2050; what bounds it is that chain, at
// 53 % of the issue slots.  Of 256, one half whose chain nothing hides: 325 us for
// twice the operations (0.31).  Steps with a V scale below 2^kFp8LowExp take the
// search for the maximum too (all of them: 193 us).
// Shared operands are K-major (Q, K) or MN-major (V) tiles [D / 64][rows][128
// bytes] with the 16-byte chunk index XORed by row % 8.
//
// Steps are counted over all items of a CTA (n).  Hand-offs are mbarriers, each
// waited once per completion by each role that needs it, every wait bounded (a
// wait that runs out sets KV_INT4_DEV_TIMEOUT and a CTA-wide abort flag that
// ends every later wait):
//   ifull[e] / ifree[e]  item ring entry e written / read by all
//   qfull     the item's Q rows have arrived
//   rkfull / rkfree, rvfull / rvfree  staged K / V codes arrived / converted
//   kfull[b]  K tile b = n & 1 and ring entry n % 3 written
//   vfull[b]  V tile b written
//   kfree[b]  S0 and S1 that read K tile b complete
//   vfree[b]  WV0 and WV1 that read V tile b complete
//   sfull[h]  S_h complete (and every earlier MMA)
//   pfull[h]  W_h in TMEM, O_h rescaled if it had to be
//   odone     the item's last WV complete (items with steps)
// Ring entry n % 3 is written once S of step n - 2 is complete: it was issued
// after both halves' W of step n - 3, the entry's last readers.  An item's Q is
// copied once S of the previous item's last step is complete.

template <int D>
struct Fp8Ws {
  static constexpr int H = D <= 192 ? 2 : 1;  // halves of 128 rows: TMEM holds one O of 256 columns beside scores
  static constexpr int ROWS = 128 * H;
  static constexpr int NK = D <= 128 ? 128 : 64;  // keys per step
  static constexpr int NB = NK / 16;              // cache blocks per step
  static constexpr int KB = (D + 63) / 64;        // 128-byte blocks of an f16 head vector
  static constexpr int CHR = D / 16;              // 16-byte chunks per code row
  static constexpr int QBYTES = ROWS * 128 * KB;
  static constexpr int KVBYTES = NK * 128 * KB;   // one K or V tile
  // staged code rows, dense, in the TMA swizzle whose span W divides the row:
  // 16-byte chunk i of the stage at chunk i ^ swizzle(i), which spreads one
  // chunk column of eight rows over all banks for every head size
  static constexpr int W = D % 128 == 0 ? 128 : D % 64 == 0 ? 64 : 32;
  static constexpr int STG = NK * D;              // K, then V
  __host__ __device__ static constexpr int chunk(int i) {
    return W == 128 ? i ^ ((i >> 3) & 7) : W == 64 ? i ^ ((i >> 3) & 3) : i ^ ((i >> 3) & 1);
  }
  // K scales, log2 V scales, 1 / V scales (0 below 2^kFp8LowExp), block flags, step flags (1 all blocks
  // usable, 2 a V scale below)
  static constexpr int RING = (4 * NB + 4) * 4;
  static constexpr int NRING = 3;
  static constexpr int NBARS = 23;
  static constexpr int S_COLS = NK, O_COL = H * NK;  // TMEM: S_h at h NK, O_h at H NK + h D
  static constexpr int XCH = 2 * ROWS * 4;  // a float per row and key half: maxima, sums
  static constexpr int SMEM = QBYTES + 4 * KVBYTES + 2 * STG + NRING * RING + NBARS * 8 + 64 + XCH;
  static constexpr int SM_WARPS = 8 * H;  // softmax
  // two halves: seven warpgroups; the last two warps only give up registers
  static constexpr int THREADS = (H == 2 ? 28 : SM_WARPS + 10) * 32;
  static constexpr int CV_WARPS = 4;       // convert warps for K, and for V
  // byte offset of chunk g of key k in a stage
  __device__ static constexpr int stage_off(int k, int g) {
    return CHR == 8   ? k * 128 + ((g ^ (k & 7)) << 4)
           : CHR == 4 ? k * 64 + ((g ^ ((k >> 1) & 3)) << 4)
                      : chunk(k * CHR + g) * 16;
  }
  static_assert(O_COL + H * D <= 512 && SMEM <= 227 * 1024, "TMEM and shared memory");
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
// MMAs issued by the lane of a converged warp whose `lead` is set.  The code
// around them stays the same for all lanes, so that descriptors live in uniform
// registers: under a branch on the lane, each MMA costs half a dozen moves from
// vector registers, and issuing one half's MMAs of a step takes longer than
// the tensor cores do
__device__ __forceinline__ void fp8_mma(uint32_t lead, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"((int)acc), "r"(lead));
}
__device__ __forceinline__ void fp8_mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                           bool acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"((int)acc), "r"(lead));
}
__device__ __forceinline__ void fp8_commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(lead)
      : "memory");
}
// fp8_wait by a converged warp, for control flow that is the same for all
// lanes; each lane that is not idle may wait for a barrier of its own
__device__ __forceinline__ void fp8_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status,
                                              bool idle = false) {
  for (int n = 0; n < kMaxWaitIters; n++) {
    if (__all_sync(0xffffffffu, idle || mbar_try_wait(bar, parity))) return;
    if ((n & 255) == 255 && __any_sync(0xffffffffu, *abort)) return;
  }
  *abort = 1;
  flag(status, KV_INT4_DEV_TIMEOUT);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// not waited for
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&w)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
      "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
      : "memory");
}
// a tensor-map box at coordinates (0, 0, head, row) into shared memory
__device__ __forceinline__ void tma_box4(uint32_t dst, const CUtensorMap* m, int head, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], "
      "[%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(head), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_box3(uint32_t dst, const CUtensorMap* m, int x, int head, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(head), "r"(row), "r"(bar)
      : "memory");
}
// Four E4M3 codes as two words of two 16-bit floats, exactly but for a power of
// two: with a code byte p = 128 sign + m in the low byte of each half, the
// sign goes to bit 15 (times 256) and m to the format's place (times 16 for
// bf16, 128 for f16) by two multiply-adds, 16 p + 240 sign or 128 p + 128 sign:
// half of the work on the FMA pipe (the converts' ALU work bounded the kernel).
// m then stands for the value * 2^-120 in bf16, which one multiplication undoes
// (f = +-2^120), and for the value * 2^-8 in f16, which the caller undoes.
// E4M3's subnormals are the formats' subnormals.
__device__ __forceinline__ uint32_t mad_u32(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ void e4m3x4_to_bf16x2(uint32_t w, __nv_bfloat162 f, uint32_t& lo, uint32_t& hi) {
  uint32_t r[2];
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const uint32_t p = __byte_perm(w, 0, i ? 0x4342 : 0x4140);
    r[i] = mad_u32(p & 0x00800080u, 240u, mad_u32(p, 16u, 0u));
    const __nv_bfloat162 v = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&r[i]), f);
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  lo = r[0];
  hi = r[1];
}
__device__ __forceinline__ void e4m3x4_to_f16x2_256th(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t p = __byte_perm(w, 0, 0x4140), q = __byte_perm(w, 0, 0x4342);
  lo = mad_u32(p & 0x00800080u, 128u, mad_u32(p, 128u, 0u));
  hi = mad_u32(q & 0x00800080u, 128u, mad_u32(q, 128u, 0u));
}

// tensor maps of a call: q {d, q heads, tokens} bf16, boxes of 64 elements x
// group x tile tokens; the code caches {W, d / W, kv heads, rows}, boxes of one
// head's block
struct Fp8Maps {
  CUtensorMap q, k, v;
};

template <int D>
__global__ void __launch_bounds__(Fp8Ws<D>::THREADS, 1)
    prefill_ws_fp8_kernel(Common c, PlanView pv, const __grid_constant__ Fp8Maps maps) {
  using G = Fp8Ws<D>;
  constexpr int KSTEPS = D / 16;
  constexpr int NK = G::NK, NB = G::NB, ROWS = G::ROWS;
  constexpr uint32_t IDESC_S = umma_idesc_f16(128, NK, false) | (1u << 7) | (1u << 10);  // bf16 operands
  constexpr uint32_t IDESC_O = umma_idesc_f16(128, D, true);
  extern __shared__ __align__(1024) uint8_t smem_ws[];  // the swizzled tiles want 1024-byte bases
  uint8_t* const sQ = smem_ws;                // [KB][256 rows][128 B], swizzled
  uint8_t* const sK = sQ + G::QBYTES;         // two K tiles [KB][NK][128 B]
  uint8_t* const sV = sK + 2 * G::KVBYTES;    // two V tiles
  uint8_t* const stg = sV + 2 * G::KVBYTES;   // staged K codes, V codes
  uint8_t* const ring = stg + 2 * G::STG;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ring + G::NRING * G::RING);
  int* const sitem = reinterpret_cast<int*>(bars + G::NBARS);  // item ring [2][6], abort flag
  uint32_t* const tslot = reinterpret_cast<uint32_t*>(sitem + 14);
  volatile int* const abort_flag = sitem + 12;
  float* const sxch = reinterpret_cast<float*>(sitem + 16);  // [key half][256 rows]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  enum {
    KFULL = 0, VFULL = 2, KFREE = 4, VFREE = 6, SFULL = 8, PFULL = 10, ODONE = 12, DRAIN = 13, IFULL = 14, IFREE = 16,
    QFULL = 18, RKFULL = 19, RVFULL = 20, RKFREE = 21, RVFREE = 22
  };
  auto bar = [&](int i) { return smem_addr(&bars[i]); };
  if (smem_addr(smem_ws) & 1023) {  // dynamic shared memory starts the window: does not occur
    flag(c.status, KV_INT4_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int b = 0; b < 2; b++) {
      mbar_init(bar(KFULL + b), G::CV_WARPS + 1);  // and the producer's ring entry
      mbar_init(bar(VFULL + b), G::CV_WARPS);
      mbar_init(bar(KFREE + b), 1);
      mbar_init(bar(VFREE + b), 1);
      mbar_init(bar(SFULL + b), 1);
      mbar_init(bar(PFULL + b), 8);
      mbar_init(bar(IFULL + b), 1);
      mbar_init(bar(IFREE + b), G::SM_WARPS + 2 * G::CV_WARPS + 1);
      mbar_init(bar(RKFULL + b), 1);  // RKFULL, RVFULL
      mbar_init(bar(RKFREE + b), G::CV_WARPS);
    }
    mbar_init(bar(QFULL), 1);
    mbar_init(bar(ODONE), 1);
    mbar_init(bar(DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // shared memory and TMEM are this CTA's own; the schedule and the caches come
  // from the kernels before.  The next kernel (decode) is let in after the wait,
  // so that it finds the schedule published
  pdl_wait();
  pdl_trigger();
  if (warp == 0) tmem_alloc(smem_addr(tslot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const int n_items = pv.plan[1];
  auto item_at = [&](int e) {
    const int* s = sitem + 6 * e;
    return PrefillItem{s[0], s[1], s[2], s[3], s[4], s[5]};
  };
  // a consumer's wait for ring entry e, warp-uniform
  auto take_item = [&](int e, uint32_t& ph, PrefillItem& item) {
    const bool ok = __all_sync(0xffffffffu, fp8_wait(bar(IFULL + e), (ph >> e) & 1, abort_flag, c.status));
    ph ^= 1u << e;
    if (!ok) return false;
    item = item_at(e);
    __syncwarp();
    if (lane == 0) fp8_arrive(bar(IFREE + e));
    return item.seq >= 0;
  };
  // registers, with two halves: 72 a thread at launch (896 threads, 64,512); the
  // softmax warpgroups take 80, the others 56 (512 x 80 + 384 x 56 = 62,464)
  if (warp < G::SM_WARPS) {
    // ======================= softmax warpgroups =======================
    if constexpr (G::H == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 80;\n");
    uint32_t ph_sfull = 0, ph_odone = 0, ph_ifull = 0;
    const float cf = fabsf(c.qscale);  // its sign is in K
    const int hf = warp >> 3, kh = (warp >> 2) & 1;  // query half, key half
    const int r = hf * 128 + (warp & 3) * 32 + lane;  // row of the item
    const int j = (int)c.gdiv.div((uint32_t)r);
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    constexpr int NC = NK / 2, NBH = NB / 2;  // keys and blocks of a key half
    const uint32_t tS = tmem + NK * hf + NC * kh + lane_off, tO = tmem + G::O_COL + hf * D + lane_off;
    const int pair = 1 + hf * 4 + (warp & 3);  // named barrier of a row's two warps
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;\n" ::"r"(pair) : "memory"); };
    auto pair_any = [&](bool v) -> bool {
      uint32_t any;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(any)
          : "r"((uint32_t)v), "r"(pair)
          : "memory");
      return any != 0;
    };
    int n = 0;  // steps of earlier items
#pragma unroll 1
    for (int itc = 0;; itc++) {
      // both warps of a row go on or neither (after a time-out one may get an
      // item that the other does not)
      PrefillItem item;
      const bool taken = take_item(itc & 1, ph_ifull, item);
      if (pair_any(!taken)) break;
      const int seq = item.seq, h = item.h, tile = item.tile, kb0 = item.kb0, nkb = item.nkb;
      const int q0 = c.qsl[seq], ql = c.qsl[seq + 1] - q0;
      const int L = c.seq_lens[seq], ctx = L - ql;
      const int tok0 = tile * c.tile_tokens;
      const bool rok = r < min(c.tile_tokens, ql - tok0) * c.group;
      const int nsteps = (nkb - kb0 + NB - 1) / NB;
      const int qp = ctx + tok0 + (rok ? j : 0);
      // the row sees positions [lo, lim), counted from this thread's first key
      int lim = (c.causal ? min(L, qp + 1) : L) - kb0 * 16 - NC * kh, lo = window_lo(c, qp) - kb0 * 16 - NC * kh;
      // rows that are not there never ask for a reference: theirs is above everything
      float m_ref = rok ? -INFINITY : INFINITY, l_run = 0.f;
#pragma unroll 1
      for (int st = 0; st < nsteps; st++, n++, lim -= NK, lo -= NK) {
        const float* re = reinterpret_cast<const float*>(ring + (n % G::NRING) * G::RING) + NBH * kh;
        const float* kvf = re + NB;
        const float* ivs = re + 2 * NB;
        const int* ok = reinterpret_cast<const int*>(re + 3 * NB);
        fp8_wait(bar(SFULL + hf), ph_sfull, abort_flag, c.status);
        ph_sfull ^= 1;
        tc_fence_after();
        // the warp's rows all see all its keys: no mask (the usual case)
        const int step_flags = ok[NB - NBH * kh];
        const bool full = __all_sync(0xffffffffu, lo <= 0 && lim >= NC && (step_flags & 1) != 0);
        // the scores of block b, hidden ones -inf, and their factor (never 0, so
        // that -inf stays); seen: whether the row sees a usable key of this thread's
        bool seen = full;
        auto scores = [&](int b, float (&s)[16], float& f) {
          f = fmaxf(cf * re[b], FLT_MIN);
          uint32_t x[16];
          tmem_ld16(tS + 16 * b, x);
#pragma unroll
          for (int k = 0; k < 16; k++) s[k] = __uint_as_float(x[k]);
          if (!full) {
            __syncwarp();  // a branch, not selects in every step
            const int first = lo - 16 * b, last = lim - 16 * b;
            uint32_t vis = first <= 0 ? 0xffffu : first >= 16 ? 0u : 0xffffu << first;
            vis &= last >= 16 ? 0xffffu : last <= 0 ? 0u : 0xffffu >> (16 - last);
            if (!ok[b]) vis = 0;
            seen |= vis != 0;
#pragma unroll
            for (int k = 0; k < 16; k++)
              if (!(vis & (1u << k))) s[k] = -INFINITY;
          }
        };
        uint32_t w[NC / 2];
        float add, tot;
        // find: the reference moves to the row's maximum where it has none or is
        // more than 8 behind; whole numbers, so that O and l move exactly.  Blocks of
        // small V scales (kFp8LowExp) have their share of the denominator taken there
        // too, by a maximum of their own
        bool find = st == 0 || (step_flags & 2) != 0;
#pragma unroll 1
        while (true) {
          if (find) {
            float mx = -INFINITY, top = -INFINITY, lows = 0.f;
#pragma unroll 1
            for (int b = 0; b < NBH; b++) {
              float s[16], f;
              scores(b, s, f);
              float t = s[0];
#pragma unroll
              for (int k = 1; k < 16; k++) t = fmaxf(t, s[k]);
              mx = fmaxf(mx, fmaf(t, f, kvf[b]));
              if (ivs[b] == 0.f) {
                __syncwarp();
                t = fmaxf(top, t * f);
                const float o = t == -INFINITY ? 0.f : t;
                lows *= fast_exp2(top - o);
                top = t;
#pragma unroll
                for (int k = 0; k < 16; k++) lows += fast_exp2(fmaf(s[k], f, -o));
              }
            }
            sxch[kh * ROWS + r] = mx;
            pair_sync();
            mx = ceilf(fmaxf(mx, sxch[(kh ^ 1) * ROWS + r]));
            pair_sync();  // read before anything else is written there
            const bool grow = mx > m_ref + (m_ref == -INFINITY ? 0.f : 8.f);
            const Exp2Pair move(grow && m_ref != -INFINITY ? m_ref - mx : 0.f);
            const float alpha = move.both();
            if (grow) m_ref = mx;
            l_run = move.of(l_run);
            if (lows > 0.f) l_run = fmaf(lows, fast_exp2(top - m_ref), l_run);
            if (__any_sync(0xffffffffu, alpha != 1.f)) {
              // O is complete up to the previous step (S_h of this step was
              // issued after it); each key half rescales its share of the columns
#pragma unroll 1
              for (int cc = kh; cc < D / 16; cc += 2) {
                uint32_t o[16];
                tmem_ld16(tO + 16 * cc, o);
#pragma unroll
                for (int i = 0; i < 16; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st16(tO + 16 * cc, o);
              }
            }
          }
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          add = tot = 0.f;
#pragma unroll
          for (int b = 0; b < NBH; b++) {
            float s[16], f;
            scores(b, s, f);
            const float2 g = make_float2(f, f), o = make_float2(kvf[b] - mu, kvf[b] - mu);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float2 a = f2fma(make_float2(s[k], s[k + 1]), g, o);
              const float2 p = make_float2(fast_exp2(a.x), fast_exp2(a.y));
              sum = f2add(sum, p);
              w[8 * b + k / 2] = pack_f16x2(p.x, p.y);
            }
            const float both = sum.x + sum.y;
            tot += both;
            add = fmaf(both, ivs[b], add);
          }
          // the weights' sum bounds the largest; a row without a reference needs one
          // as soon as it sees a usable key, whatever the weights came to: against 0
          // they vanish where every score is far below it
          if (find || !pair_any(tot > 16384.f || (m_ref == -INFINITY && seen))) break;
          find = true;
        }
        l_run += add;
        // over this thread's own columns, which have been read
#pragma unroll
        for (int b = 0; b < NBH; b += 2) tmem_st16(tS + 8 * b, *reinterpret_cast<uint32_t(*)[16]>(w + 8 * b));
        asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) fp8_arrive(bar(PFULL + hf));
      }

      // ---- epilogue: normalise, bf16, stored from registers; each key half's
      // threads take a share of the columns ----
      sxch[kh * ROWS + r] = l_run;
      pair_sync();
      const float l = l_run + sxch[(kh ^ 1) * ROWS + r];
      pair_sync();  // read before the next item's are written
      if (nsteps > 0) {
        fp8_wait(bar(ODONE), ph_odone, abort_flag, c.status);
        ph_odone ^= 1;
        tc_fence_after();
      }
      constexpr int UNITS = D / 32, FIRST = (UNITS + 1) / 2;  // of 32 columns; the first key half's
      if (item.row >= 0) {
        // a piece: O (V's factor 2^-8 undone), the reference and the sum
        const long long at = item.row + r;
#pragma unroll 1
        for (int u = kh ? 2 * FIRST : 0; u < (kh ? 2 * UNITS : 2 * FIRST); u++) {
          uint32_t o[16];
          tmem_ld16(tO + 16 * u, o);
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            if (rok)
              *reinterpret_cast<float4*>(pv.piece_o + at * D + 16 * u + i) =
                  make_float4(256.f * __uint_as_float(o[i]), 256.f * __uint_as_float(o[i + 1]),
                              256.f * __uint_as_float(o[i + 2]), 256.f * __uint_as_float(o[i + 3]));
        }
        if (rok && kh == 0) *reinterpret_cast<float2*>(pv.piece_ml + 2 * at) = make_float2(m_ref, l);
        continue;
      }
      // a row that saw no usable key is zeros: O is 0 then, but for an item
      // without steps, whose O is not read (V's factor 2^-8 is undone here)
      const float inv = l == 0.f ? 0.f : 256.f / l;
      const float2 inv2 = make_float2(inv, inv);
      uint16_t* const orow = c.out + (long long)(q0 + tok0 + (rok ? j : 0)) * c.out_stride +
                             (long long)(h * c.group + (rok ? r - j * c.group : 0)) * D;
      const bool al32 = ((reinterpret_cast<uintptr_t>(c.out) | (uintptr_t)(c.out_stride * 2) | (uintptr_t)(D * 2)) & 31) == 0;
#pragma unroll 1
      for (int u = kh ? FIRST : 0; u < (kh ? UNITS : FIRST); u++) {
        uint32_t w[16];
#pragma unroll
        for (int hh = 0; hh < 2; hh++) {
          uint32_t o[16];
          if (nsteps > 0) {
            tmem_ld16(tO + 32 * u + 16 * hh, o);
          } else {
#pragma unroll
            for (int i = 0; i < 16; i++) o[i] = 0;
          }
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), inv2);
            w[8 * hh + i] = pack_bf16x2_rn(y.x, y.y);
          }
        }
        if (rok) {
          uint16_t* const dst = orow + 32 * u;
          if (al32) {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst + 2 * i), "r"(w[i]),
                           "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                           "r"(w[i + 7])
                           : "memory");
          } else {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(dst + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
          }
        }
      }
    }
  } else {
    // ============== convert, producer and MMA warps ==============
    if constexpr (G::H == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
    // waits for completions of a barrier pair indexed by step parity, counted
    auto wait_until = [&](int first, int& done, int count) {
      for (; done < count; done++) fp8_wait(bar(first + (done & 1)), (done >> 1) & 1, abort_flag, c.status);
    };
    if (warp < G::SM_WARPS + 2 * G::CV_WARPS) {
      // ================= convert warps =================
      // one team's loop: kv = 0 K codes, 1 V codes
      auto team = [&](auto kv_tag) {
        constexpr int KV = decltype(kv_tag)::value;
        constexpr int FULL = KV ? VFULL : KFULL, FREE = KV ? VFREE : KFREE;
        // a thread takes 16-code chunks of one key, consecutive threads
        // consecutive keys (the eight keys of a load or store phase fall in
        // eight bank groups)
        constexpr int TPK = 128 / NK;  // threads per key
        const int t = tid & 127, k = t & (NK - 1), g0 = t / NK;
        const uint8_t* const src = stg + KV * G::STG;
        uint8_t* const tile = KV ? sV : sK;
        const __nv_bfloat162 kf = __float2bfloat162_rn(c.qscale < 0.f ? -exp2_int(120) : exp2_int(120));
        uint32_t ph_ifull = 0;
        int n = 0, freed = 0;
#pragma unroll 1
        for (int itc = 0;; itc++) {
          PrefillItem item;
          if (!take_item(itc & 1, ph_ifull, item)) break;
          const int nsteps = (item.nkb - item.kb0 + NB - 1) / NB;
          int keys = c.seq_lens[item.seq] - item.kb0 * 16;  // rows of the step that hold keys
#pragma unroll 1
          for (int st = 0; st < nsteps; st++, n++, keys -= NK) {
            uint8_t* const dst = tile + (n & 1) * G::KVBYTES;
            fp8_wait(bar(RKFULL + KV), n & 1, abort_flag, c.status);
            // the step's codes are taken into registers first: the next step's
            // copies (about 2000 cycles) run during the conversion
            constexpr int CH = G::CHR / TPK, U = (CH + 1) / 2;  // chunks, and as a loop of two (instruction caches)
            uint4 x[U], y[U];
#pragma unroll
            for (int i = 0; i < U; i++) {
              x[i] = *reinterpret_cast<const uint4*>(src + G::stage_off(k, i * TPK + (TPK > 1 ? g0 : 0)));
              y[i] = *reinterpret_cast<const uint4*>(src + G::stage_off(k, (U + i) * TPK + (TPK > 1 ? g0 : 0)));
            }
            static_assert(2 * U == CH, "an even number of chunks");
            // ... once they have all arrived: the arrival's address depends on every
            // load (by a mask that is 0), as nothing else orders shared loads in
            // flight before it (TMA then overwrote codes that were still to be
            // read)
            uint32_t seen = 0;
#pragma unroll
            for (int i = 0; i < U; i++) seen |= x[i].x | y[i].x;
            seen = __reduce_or_sync(0xffffffffu, seen & (uint32_t)(c.num_blocks >> 31));
            if (lane == 0) fp8_arrive(bar(RKFREE + KV) + seen);
            wait_until(FREE, freed, n - 1);  // the MMAs of step n - 2 that read this tile
#pragma unroll 1
            for (int i0 = 0; i0 < CH; i0 += U) {
#pragma unroll
              for (int i = 0; i < U; i++) {
                const int g = (i0 + i) * TPK + (TPK > 1 ? g0 : 0);
                uint4 lo, hi;
                if constexpr (KV) {
                  // rows behind the sequence are zeros (a NaN code would survive its zero weight)
                  if (k >= keys) x[i] = make_uint4(0, 0, 0, 0);
                  e4m3x4_to_f16x2_256th(x[i].x, lo.x, lo.y);
                  e4m3x4_to_f16x2_256th(x[i].y, lo.z, lo.w);
                  e4m3x4_to_f16x2_256th(x[i].z, hi.x, hi.y);
                  e4m3x4_to_f16x2_256th(x[i].w, hi.z, hi.w);
                } else {
                  e4m3x4_to_bf16x2(x[i].x, kf, lo.x, lo.y);
                  e4m3x4_to_bf16x2(x[i].y, kf, lo.z, lo.w);
                  e4m3x4_to_bf16x2(x[i].z, kf, hi.x, hi.y);
                  e4m3x4_to_bf16x2(x[i].w, kf, hi.z, hi.w);
                }
                *reinterpret_cast<uint4*>(dst + fp8_sw128(NK, k, 2 * g)) = lo;
                *reinterpret_cast<uint4*>(dst + fp8_sw128(NK, k, 2 * g + 1)) = hi;
              }
#pragma unroll
              for (int i = 0; i < U; i++) x[i] = y[i];
            }
            fence_proxy_async_smem();  // the tile is read by the tensor cores
            __syncwarp();
            if (lane == 0) fp8_arrive(bar(FULL + (n & 1)));
          }
        }
      };
      if (warp < G::SM_WARPS + G::CV_WARPS)
        team(std::integral_constant<int, 0>{});
      else
        team(std::integral_constant<int, 1>{});
    } else if (warp == G::SM_WARPS + 8) {
      // ================= producer warp =================
      uint32_t ph_ifree = 0;
      int n = 0, nq = 0, kfree = 0;
#pragma unroll 1
      for (int itc = 0;; itc++) {
        const int e = itc & 1;
        if (itc >= 2) {
          fp8_wait(bar(IFREE + e), (ph_ifree >> e) & 1, abort_flag, c.status);
          ph_ifree ^= 1u << e;
        }
        int itn = n_items;
        if (lane == 0 && !*abort_flag) itn = atomicAdd(&pv.plan[2], 1);
        const PrefillItem item = prefill_piece_item(c, pv, __shfl_sync(0xffffffffu, itn, 0), n_items);
        if (lane == 0) {
          int* s = sitem + 6 * e;
          s[0] = item.seq;
          s[1] = item.h;
          s[2] = item.tile;
          s[3] = item.kb0;
          s[4] = item.nkb;
          s[5] = item.row;
          fp8_arrive(bar(IFULL + e));
        }
        if (item.seq < 0) break;
        const int seq = item.seq, h = item.h, kb0 = item.kb0, nkb = item.nkb;
        const int q0 = c.qsl[seq], tok0 = item.tile * c.tile_tokens;
        const int nsteps = (nkb - kb0 + NB - 1) / NB;
        // lane b < NB holds block b of a step: its row in the caches (behind
        // their end for a block that the table does not name) and its scales
        const int none = c.num_blocks * 16;
        auto block_of = [&](int st) -> int {
          const int kb = kb0 + st * NB + lane;
          if (st >= nsteps || lane >= NB || kb >= nkb) return -1;
          const int id = c.block_table[(long long)seq * c.max_blocks + kb];
          if (id >= 0 && id < c.num_blocks) return id;
          flag(c.status, KV_INT4_DEV_BAD_BLOCK);
          return -1;
        };
        int blk = block_of(0);
#pragma unroll 1
        for (int st = 0; st < nsteps; st++, n++) {
          if (__any_sync(0xffffffffu, *abort_flag)) break;
          const int b = n & 1;
          const int next = block_of(st + 1);
          const bool ok = blk >= 0;
          const long long at = ok ? (long long)blk * c.hkv + h : 0;
          const float ks = ok ? c.k_scale[at] : 0.f, vs = ok ? c.v_scale[at] : 1.f;
          auto stage = [&](int kv, int full, int free) {
            if (n > 0) fp8_wait(bar(free), (n - 1) & 1, abort_flag, c.status);
            if (lane == 0) mbar_arrive_expect_tx(bar(full), G::STG);
            __syncwarp();
            if (lane < NB)
              tma_box4(smem_addr(stg + kv * G::STG + lane * 16 * D), kv ? &maps.v : &maps.k, h, ok ? blk * 16 : none,
                       bar(full));
          };
          stage(0, RKFULL, RKFREE);
          stage(1, RVFULL, RVFREE);
          if (st == 0) {
            wait_until(KFREE, kfree, n);  // every S of the previous item: its Q has been read
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(QFULL), c.group * c.tile_tokens * 128 * G::KB);
#pragma unroll
              for (int x = 0; x < G::KB; x++)
                tma_box3(smem_addr(sQ + x * ROWS * 128), &maps.q, 64 * x, h * c.group, q0 + tok0, bar(QFULL));
            }
            __syncwarp();
            nq++;
          }
          wait_until(KFREE, kfree, n - 1);  // S of step n - 2: ring entry n % 3 has been read
          float* re = reinterpret_cast<float*>(ring + (n % G::NRING) * G::RING);
          const bool low = vs < exp2_int(kFp8LowExp);
          if (lane < NB) {
            re[lane] = ks;
            re[NB + lane] = (float)exp_of(vs);
            re[2 * NB + lane] =
                low ? 0.f : __uint_as_float((254u << 23) - (__float_as_uint(vs) & 0x7f800000u));
            reinterpret_cast<int*>(re)[3 * NB + lane] = ok;
          }
          const bool all = __all_sync(0xffffffffu, ok || lane >= NB);
          const bool lows = __any_sync(0xffffffffu, low && lane < NB);
          if (lane == 0) reinterpret_cast<int*>(re)[4 * NB] = all | lows << 1;
          __syncwarp();
          if (lane == 0) fp8_arrive(bar(KFULL + b));
          blk = next;
        }
      }
      // the last copy of each kind has landed before the CTA ends, after an
      // abort too
      if (n > 0 && !(mbar_wait_bounded(bar(RKFULL), (n - 1) & 1) && mbar_wait_bounded(bar(RVFULL), (n - 1) & 1) &&
                     mbar_wait_bounded(bar(QFULL), (nq - 1) & 1)))
        flag(c.status, KV_INT4_DEV_TIMEOUT);
    } else if (warp == G::SM_WARPS + 9) {
      // ================= MMA warp =================
      uint32_t lead;
      asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(lead));
      int n = 0, items = 0, pfull = 0;
      const uint64_t dq = umma_desc(smem_addr(sQ), 16, 1024);
      const uint64_t dk = umma_desc(smem_addr(sK), 16, 1024);
      const uint64_t dv = umma_desc(smem_addr(sV), NK * 128, 1024);
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);  // in a uniform register
      auto wait = [&](int i, uint32_t parity) { fp8_wait_warp(bar(i), parity, abort_flag, c.status); };
      auto issue_s = [&](int hh, int b) {
        const uint64_t kt = dk + (uint64_t)(b * (G::KVBYTES >> 4));
#pragma unroll
        for (int ks = 0; ks < KSTEPS; ks++)
          fp8_mma(lead, tm + NK * hh, dq + (uint64_t)(((ks >> 2) * ROWS * 128 + hh * 128 * 128 + (ks & 3) * 32) >> 4),
                  kt + (uint64_t)(((ks >> 2) * NK * 128 + (ks & 3) * 32) >> 4), IDESC_S, ks > 0);
      };
      auto issue_wv = [&](int hh, int b, bool first) {
        const uint64_t vt = dv + (uint64_t)(b * (G::KVBYTES >> 4));
#pragma unroll
        for (int kk = 0; kk < NB; kk++)
          fp8_mma_ts(lead, tm + G::O_COL + hh * D,
                     tm + NK * hh + (kk < NB / 2 ? kk * 8 : NK / 2 + (kk - NB / 2) * 8), vt + (uint64_t)(kk * (2048 >> 4)), IDESC_O,
                     !first || kk > 0);
      };
#pragma unroll 1
      for (int itc = 0;; itc++) {
        wait(IFULL + (itc & 1), (itc >> 1) & 1);
        const PrefillItem item = item_at(itc & 1);
        __syncwarp();
        if (lane == 0) fp8_arrive(bar(IFREE + (itc & 1)));
        __syncwarp();
        // the step count through a warp reduction, whose result is uniform;
        // none once a wait has run out
        int steps = -1;
        if (item.seq >= 0 && !*abort_flag) steps = (item.nkb - item.kb0 + NB - 1) / NB;
        const int nsteps = __reduce_min_sync(0xffffffffu, steps);
        if (nsteps < 0) break;
        if (nsteps > 0) {
          wait(QFULL, items & 1);
          items++;
        }
        // iteration st: for each half, the WV of step st - 1 and the S of step
        // st.  A wait costs the warp some 400 cycles even when it is satisfied,
        // so the first half's three barriers are waited for at once, a lane each
#pragma unroll 1
        for (int st = 0; st <= nsteps; st++) {
          const bool wv = st > 0, sc = st < nsteps;
          {
            // V of step n - 1, the first half's W of it, K of step n
            const int i = lane == 0 ? VFULL + ((n - 1) & 1) : lane == 1 ? PFULL : KFULL + (n & 1);
            const uint32_t ph = lane == 0 ? ((n - 1) >> 1) & 1 : lane == 1 ? pfull & 1 : (n >> 1) & 1;
            const bool idle = lane > 2 || !(lane == 2 ? sc : wv);
            fp8_wait_warp(bar(i), ph, abort_flag, c.status, idle);
          }
#pragma unroll 1
          for (int hh = 0; hh < G::H; hh++) {
            if (wv && hh) wait(PFULL + 1, pfull & 1);
            tc_fence_after();
            if (wv) {
              issue_wv(hh, (n - 1) & 1, st == 1);
              if (hh == G::H - 1) fp8_commit(lead, bar(VFREE + ((n - 1) & 1)));
            }
            if (sc) {
              issue_s(hh, n & 1);
              fp8_commit(lead, bar(SFULL + hh));
            }
          }
          if (wv) pfull++;
          if (sc) {
            fp8_commit(lead, bar(KFREE + (n & 1)));
            n++;
          }
        }
        // none for an item without steps: its completion would follow the last
        // item's at once, before every softmax warp has seen that
        if (nsteps > 0) fp8_commit(lead, bar(ODONE));
      }
    }
  }
  if (warp == G::SM_WARPS + 9) {
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
