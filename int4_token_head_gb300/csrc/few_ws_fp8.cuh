// Attention of few query rows over many keys of the FP8 cache on the
// 5th-generation tensor cores (tcgen05), included by attention_shared_fp8.cu: what
// a group of sequences asks of its shared prefix, 9 to 64 rows per kv head.
//
// The keys are the MMA's M, the rows its N (32 or 64): S^T = K Q^T, O^T += V^T W^T.
// Both cost a fraction of what 128 rows would, and what is left is converting every
// code once (16 warps) beside loading it.  One CTA per SM; an item is a tile of up
// to 64 rows against a piece of the keys (the schedule's list), a step 128 keys.
// Warps:
//   * sums (0-7): a thread is a key, a warpgroup half of the rows.  Weights
//     2^(s f + kv - m) as in prefill_ws_fp8.cuh (references m per row that move when a
//     row first sees a usable key and when a weight outgrows 2^14); a thread adds its
//     keys' shares of the denominators, which meet at the item's end.  W^T goes to
//     shared memory (two tiles) as the second product's K-major operand;
//   * K codes (8-15) into a bf16 tile, V codes (16-23) into one of two f16 tiles, both
//     exact but for V's 2^-8;
//   * producer (24): items, TMA copies of Q and of the code blocks into two stages,
//     scales into a four-entry ring; MMA (25): S of a step is issued before WV of the
//     one before, so that sums run during both.
// Four documents of 32768 positions, eight conversations about each (32 rows per kv
// head), 32/8 heads of 128: TODO us a call; on the decode kernel 150.
template <int D>
struct Few {
  static constexpr int NK = 128, NB = 8, RN = 64;
  static constexpr int KB = (D + 63) / 64, CHR = D / 16;
  static constexpr int KBYTES = NK * 128 * KB;   // K tile [KB][128 keys][128 B]
  static constexpr int VBYTES = NK * 128 * 2;    // V tile [2][128 keys][128 B]: 128 dimensions, the MMA's M
  static constexpr int PBYTES = 2 * RN * 128;    // W^T tile [2][64 rows][128 B]
  static constexpr int QBYTES = KB * RN * 128;
  static constexpr int STG = NK * D;
  static constexpr int W = Fp8Ws<D>::W;
  static constexpr int RING = (4 * NB + 4) * 4, NRING = 4;
  static constexpr int NBARS = 28, BARS = 256;
  static constexpr int SMEM = KBYTES + 2 * VBYTES + 2 * PBYTES + QBYTES + 4 * STG + NRING * RING + BARS + 64 + 64 +
                              3 * RN * 4 + 4 * RN * 4;
  static constexpr int THREADS = 28 * 32;
  static constexpr int O_COL = 2 * RN;           // TMEM: S^T of two steps, O^T
  static_assert(SMEM <= 227 * 1024 && NBARS * 8 <= BARS, "shared memory");
};

template <int D>
__global__ void __launch_bounds__(Few<D>::THREADS, 1)
    few_ws_kernel(Common c, PlanView pv, const __grid_constant__ Fp8Maps maps) {
  using G = Few<D>;
  using P = Fp8Ws<D>;  // the staged codes' layout
  constexpr int KSTEPS = D / 16, NK = G::NK, NB = G::NB, RN = G::RN;
  extern __shared__ __align__(1024) uint8_t smem_few[];
  uint8_t* const sK = smem_few;
  uint8_t* const sV = sK + G::KBYTES;
  uint8_t* const sP = sV + 2 * G::VBYTES;
  uint8_t* const sQ = sP + 2 * G::PBYTES;
  uint8_t* const stg = sQ + G::QBYTES;  // [stage][K, V]
  uint8_t* const ring = stg + 4 * G::STG;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ring + G::NRING * G::RING);
  int* const sitem = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + G::BARS);  // item ring [2][6]
  int* const sctl = sitem + 16;                                                          // abort flag, TMEM address
  volatile int* const abort_flag = sctl;
  float* const sref = reinterpret_cast<float*>(sctl + 16);  // [64] references
  float* const sneg = sref + RN;                            // [64] what is added to an exponent
  float* const smove = sneg + RN;                           // [64] the last move of a reference
  float* const smax = smove + RN;                           // [4 warps][64] maxima, then sums
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  enum {
    IFULL = 0, IFREE = 2, QFULL = 4, RKFULL = 5, RVFULL = 7, RKFREE = 9, RVFREE = 11, KFULL = 13, KFREE = 15, VFULL = 17,
    VFREE = 19, SFULL = 21, PFULL = 23, ODONE = 25, DRAIN = 26
  };
  auto bar = [&](int i) { return smem_addr(&bars[i]); };
  if (smem_addr(smem_few) & 1023) {  // dynamic shared memory starts the window: does not occur
    flag(c.status, KV_INT4_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int b = 0; b < 2; b++) {
      mbar_init(bar(IFULL + b), 1);
      mbar_init(bar(IFREE + b), 25);
      mbar_init(bar(RKFULL + b), 1);
      mbar_init(bar(RVFULL + b), 1);
      mbar_init(bar(RKFREE + b), 8);
      mbar_init(bar(RVFREE + b), 8);
      mbar_init(bar(VFULL + b), 8);
      mbar_init(bar(VFREE + b), 1);
      mbar_init(bar(SFULL + b), 1);
      mbar_init(bar(PFULL + b), 8);
    }
    mbar_init(bar(QFULL), 1);
    // by the step's parity although there is one tile: who waits for a step may come
    // when the one after it is done
    for (int b = 0; b < 2; b++) {
      mbar_init(bar(KFULL + b), 8 + 1);  // and the producer's ring entry
      mbar_init(bar(KFREE + b), 1);
    }
    mbar_init(bar(ODONE), 1);
    mbar_init(bar(DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // rows of Q that no copy writes, and dimensions of V behind D, are zeros
  for (int x = tid; x < (2 * G::VBYTES + 2 * G::PBYTES + G::QBYTES) / 16; x += G::THREADS)
    reinterpret_cast<uint4*>(sV)[x] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  pdl_wait();
  pdl_trigger();
  if (warp == 0) tmem_alloc(smem_addr(sctl + 1), 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)sctl[1];
  const int n_items = pv.plan[1];
  auto item_at = [&](int e) {
    const int* s = sitem + 6 * e;
    return PrefillItem{s[0], s[1], s[2], s[3], s[4], s[5], false};
  };
  auto take_item = [&](int itc, PrefillItem& item) {
    const int e = itc & 1;
    if (!__all_sync(0xffffffffu, fp8_wait(bar(IFULL + e), (itc >> 1) & 1, abort_flag, c.status))) return false;
    item = item_at(e);
    __syncwarp();
    if (lane == 0) fp8_arrive(bar(IFREE + e));
    return item.seq >= 0;
  };
  auto steps_of = [](const PrefillItem& item) { return (item.nkb - item.kb0 + NB - 1) / NB; };
  // registers: 72 a thread at launch (896 threads, 64,512); the sums' warpgroups take
  // 104, the others 56 (256 x 104 + 640 x 56 = 62,464)
  if (warp < 8) {
    // ======================= sums =======================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
    const int wg = warp >> 2, k = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float cf = fabsf(c.qscale);  // its sign is in K
    auto wg_sync = [&]() { asm volatile("bar.sync %0, 128;\n" ::"r"(1 + wg) : "memory"); };
    auto wg_any = [&](bool v) -> bool {
      uint32_t any;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(any)
          : "r"((uint32_t)v), "r"(1 + wg)
          : "memory");
      return any != 0;
    };
    // this key's place in a row of W^T, for the eight swizzles of a row
    uint32_t place[8];
#pragma unroll
    for (int i = 0; i < 8; i++)
      place[i] = smem_addr(sP) + (k >> 6) * RN * 128 + (((((k & 63) >> 3) ^ i)) << 4) + (k & 7) * 2;
    int n = 0, done = 0;  // steps, items with steps
    PrefillItem item;
#pragma unroll 1
    for (int itc = 0;; itc++) {
      // the warpgroup's warps go on together or not at all (after a time-out one may
      // get an item that the others do not)
      const bool taken = take_item(itc, item);
      if (wg_any(!taken)) break;
      const SeqView view = seq_view<true>(c, pv, item.seq);
      const int tok0 = item.tile * c.tile_tokens;
      const int rows = min(c.tile_tokens, view.ql - tok0) * c.group;
      const int N = rows <= 32 ? 32 : 64, nc = N / 2, col0 = wg * nc;  // this warpgroup's rows
      const int nsteps = steps_of(item);
      const int pos0 = item.kb0 * 16 + k;  // this key's position in the first step
      if (k < nc) {  // rows that are not there: their reference is above everything
        const bool there = col0 + k < rows;
        sref[col0 + k] = there ? -INFINITY : INFINITY;
        sneg[col0 + k] = there ? 0.f : -INFINITY;
      }
      float l[32];
#pragma unroll
      for (int i = 0; i < 32; i++) l[i] = 0.f;
      bool unref = true;  // some row has no reference yet
      wg_sync();
#pragma unroll 1
      for (int st = 0; st < nsteps; st++, n++) {
        const float* re = reinterpret_cast<const float*>(ring + (n % G::NRING) * G::RING);
        fp8_wait(bar(SFULL + (n & 1)), (n >> 1) & 1, abort_flag, c.status);
        tc_fence_after();
        const int b = k >> 4, pos = pos0 + st * NK;
        const float f = fmaxf(cf * re[b], FLT_MIN), kvf = re[NB + b], ivs = re[2 * NB + b];
        const bool ok = reinterpret_cast<const int*>(re)[3 * NB + b] != 0 && pos < view.L;
        // rows from `from` on see this key
        const int from = ok ? max(0, (pos - view.ctx - tok0) * c.group) - col0 : 1 << 20;
        const bool full = __all_sync(0xffffffffu, from <= 0);
        const uint32_t ts = tmem + RN * (n & 1) + col0 + lane_off;
        if (n >= 2) fp8_wait(bar(VFREE + (n & 1)), ((n - 2) >> 1) & 1, abort_flag, c.status);  // W^T of step n - 2 has been read
        bool find = unref;
        const uint32_t tile = (n & 1) * G::PBYTES + col0 * 128;
#pragma unroll 1
        while (true) {
          if (find) {
            // the rows' largest exponents over the step's keys
#pragma unroll 1
            for (int c0 = 0; c0 < nc; c0 += 16) {
              uint32_t x[16];
              tmem_ld16(ts + c0, x);
              int mine = INT_MIN;
#pragma unroll
              for (int i = 0; i < 16; i++) {
                int v = c0 + i >= from ? __float_as_int(fmaf(__uint_as_float(x[i]), f, kvf)) : __float_as_int(-INFINITY);
                v ^= (v >> 31) & 0x7fffffff;  // orders as an integer
                v = __reduce_max_sync(0xffffffffu, v);
                if (lane == i) mine = v;
              }
              if (lane < 16) smax[(warp & 3) * RN + col0 + c0 + lane] = __int_as_float(mine ^ ((mine >> 31) & 0x7fffffff));
            }
            wg_sync();
            bool grown = false, none = false;
            if (k < nc) {
              const float* m = smax + col0 + k;
              const float top = ceilf(fmaxf(fmaxf(m[0], m[RN]), fmaxf(m[2 * RN], m[3 * RN])));
              const float old = sref[col0 + k];
              // whole numbers, so that O and l move exactly
              const bool grow = top > old + (old == -INFINITY ? 0.f : 8.f);
              const float now = grow ? top : old;
              smove[col0 + k] = grow && old != -INFINITY ? old - top : 0.f;
              sref[col0 + k] = now;
              sneg[col0 + k] = now == -INFINITY ? 0.f : -now;
              grown = grow && old != -INFINITY;
              none = now == -INFINITY;
            }
            unref = wg_any(none);
            if (wg_any(grown)) {
              // O^T is complete up to the previous step once its WV is
              if (st > 0) fp8_wait(bar(VFREE + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag, c.status);
              tc_fence_after();
#pragma unroll
              for (int c0 = 0; c0 < 32; c0 += 16) {
                if (c0 < nc) {
                  uint32_t o[16];
                  if (st > 0) tmem_ld16(tmem + G::O_COL + col0 + c0 + lane_off, o);
#pragma unroll
                  for (int i = 0; i < 16; i++) {
                    const Exp2Pair move(smove[col0 + c0 + i]);
                    l[c0 + i] = move.of(l[c0 + i]);
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * move.both());
                  }
                  if (st > 0) tmem_st16(tmem + G::O_COL + col0 + c0 + lane_off, o);
                }
              }
              asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
            }
          }
          float big = 0.f;
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 16) {
            if (c0 < nc) {
              uint32_t x[16];
              tmem_ld16(ts + c0, x);
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 m = *reinterpret_cast<const float4*>(sneg + col0 + c0 + i);
                float w[4] = {fast_exp2(fmaf(__uint_as_float(x[i]), f, kvf + m.x)),
                              fast_exp2(fmaf(__uint_as_float(x[i + 1]), f, kvf + m.y)),
                              fast_exp2(fmaf(__uint_as_float(x[i + 2]), f, kvf + m.z)),
                              fast_exp2(fmaf(__uint_as_float(x[i + 3]), f, kvf + m.w))};
                if (!full) {
#pragma unroll
                  for (int e = 0; e < 4; e++) w[e] = c0 + i + e >= from ? w[e] : 0.f;
                }
                big = fmaxf(fmaxf(fmaxf(big, w[0]), fmaxf(w[1], w[2])), w[3]);
                const uint32_t h0 = pack_f16x2(w[0], w[1]), h1 = pack_f16x2(w[2], w[3]);
                const uint32_t at = tile + (c0 + i) * 128;
                asm volatile("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n st.shared.b16 [%0], a;\n st.shared.b16 [%1], b;\n}\n" ::"r"(
                                 place[i & 7] + at),
                             "r"(place[(i + 1) & 7] + at + 128), "r"(h0)
                             : "memory");
                asm volatile("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n st.shared.b16 [%0], a;\n st.shared.b16 [%1], b;\n}\n" ::"r"(
                                 place[(i + 2) & 7] + at + 256),
                             "r"(place[(i + 3) & 7] + at + 384), "r"(h1)
                             : "memory");
              }
            }
          }
          if (find || !wg_any(big > 16384.f)) break;
          find = true;
        }
        // the denominators' shares: a weight without its V scale; those of small V scales
        // may have left fp32 as weights
        {
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 16) {
            if (c0 < nc) {
              uint32_t x[16];
              tmem_ld16(ts + c0, x);
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 m = *reinterpret_cast<const float4*>(sneg + col0 + c0 + i);
                const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                  const float s = __uint_as_float(x[i + e]);
                  const float w = ivs != 0.f ? fast_exp2(fmaf(s, f, kvf + mm[e])) * ivs : fast_exp2(fmaf(s, f, mm[e]));
                  l[c0 + i + e] += c0 + i + e >= from ? w : 0.f;
                }
              }
            }
          }
        }
        tc_fence_before();
        fence_proxy_async_smem();  // W^T is read by the tensor cores
        __syncwarp();
        if (lane == 0) fp8_arrive(bar(PFULL + (n & 1)));
      }
      // ---- epilogue: the denominators over the keys, then O^T with a thread per dimension ----
#pragma unroll
      for (int i = 0; i < 32; i++) {
        if (i < nc) {
          float s = l[i];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == 0) smax[(warp & 3) * RN + col0 + i] = s;
        }
      }
      wg_sync();
      if (nsteps > 0) {
        fp8_wait(bar(ODONE), done & 1, abort_flag, c.status);
        done++;
        tc_fence_after();
      }
      const int first = pv.vrec[2 * item.seq + 1].z;
#pragma unroll 1
      for (int c0 = 0; c0 < nc; c0 += 16) {
        uint32_t o[16];
        if (nsteps > 0) {
          tmem_ld16(tmem + G::O_COL + col0 + c0 + lane_off, o);
        } else {
#pragma unroll
          for (int i = 0; i < 16; i++) o[i] = 0;
        }
#pragma unroll
        for (int i = 0; i < 16; i++) {
          const int r = col0 + c0 + i;
          if (r < rows) {
            const float sum = (smax[r] + smax[RN + r]) + (smax[2 * RN + r] + smax[3 * RN + r]);
            const int j = (int)c.gdiv.div((uint32_t)r), tok = tok0 + j;
            const int head = item.h * c.group + r - j * c.group;
            float *dst = nullptr, *ml = nullptr;
            if (item.row >= 0) {
              dst = pv.piece_o + (long long)(item.row + r) * D;
              ml = pv.piece_ml + 2ll * (item.row + r);
            } else if (first >= 0) {
              const long long at = (long long)(first + tok) * c.hq + head;
              dst = pv.row_o + at * D;
              ml = pv.row_ml + 2 * at;
            }
            // V's factor 2^-8 is undone here
            const float y = __uint_as_float(o[i]) * (dst ? 256.f : sum == 0.f ? 0.f : 256.f / sum);
            if (dst) {
              if (k < D) dst[k] = y;
              if (k == 0) *reinterpret_cast<float2*>(ml) = make_float2(sref[r], sum);
            } else {
              if (k < D) c.out[(long long)(view.q0 + tok) * c.out_stride + (long long)head * D + k] =
                             (uint16_t)(pack_bf16x2_rn(y, 0.f) & 0xffffu);
              if (k == 0 && c.sh.lse) c.sh.lse[(view.q0 + tok) * c.sh.lse_stride + head] = log_sum_exp(sref[r], sum);
            }
          }
        }
      }
      wg_sync();  // the references and sums have been read
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
    // waits for completions of a barrier pair indexed by step parity, counted
    auto wait_until = [&](int first, int& done, int count) {
      for (; done < count; done++) fp8_wait(bar(first + (done & 1)), (done >> 1) & 1, abort_flag, c.status);
    };
    if (warp < 24) {
      // ================= convert warps =================
      auto team = [&](auto kv_tag) {
        constexpr int KV = decltype(kv_tag)::value;
        constexpr int CH = G::CHR / 2;  // a thread takes every other 16-code chunk of a key
        const int t = tid & 255, key = t & 127, g0 = t >> 7;
        const __nv_bfloat162 kf = __float2bfloat162_rn(c.qscale < 0.f ? -exp2_int(120) : exp2_int(120));
        int n = 0, freed = 0;
        PrefillItem item;
#pragma unroll 1
        for (int itc = 0; take_item(itc, item); itc++) {
          const int nsteps = steps_of(item);
          int keys = pv.vrec[2 * item.seq].z - item.kb0 * 16;  // rows of the step that hold keys
#pragma unroll 1
          for (int st = 0; st < nsteps; st++, n++, keys -= NK) {
            const int s = n & 1;
            const uint8_t* const src = stg + (2 * s + KV) * G::STG;
            fp8_wait(bar((KV ? RVFULL : RKFULL) + s), (n >> 1) & 1, abort_flag, c.status);
            uint4 x[CH];
            uint32_t seen = 0;
#pragma unroll
            for (int i = 0; i < CH; i++) x[i] = *reinterpret_cast<const uint4*>(src + P::stage_off(key, 2 * i + g0));
            // the arrival's address depends on every load (by a mask that is 0): nothing else
            // orders shared loads in flight before the copies that come after it
#pragma unroll
            for (int i = 0; i < CH; i++) seen |= x[i].x;
            seen = __reduce_or_sync(0xffffffffu, seen & (uint32_t)(c.num_blocks >> 31));
            if (lane == 0) fp8_arrive(bar((KV ? RVFREE : RKFREE) + s) + seen);
            if constexpr (KV) wait_until(VFREE, freed, n - 1);  // WV of step n - 2, which read this tile
            else wait_until(KFREE, freed, n);                    // S of step n - 1
            uint8_t* const dst = KV ? sV + s * G::VBYTES : sK;
#pragma unroll
            for (int i = 0; i < CH; i++) {
              const int g = 2 * i + g0;
              uint4 lo, hi;
              if constexpr (KV) {
                // rows behind the sequence are zeros (a NaN code would survive its zero weight)
                if (key >= keys) x[i] = make_uint4(0, 0, 0, 0);
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
              *reinterpret_cast<uint4*>(dst + fp8_sw128(NK, key, 2 * g)) = lo;
              *reinterpret_cast<uint4*>(dst + fp8_sw128(NK, key, 2 * g + 1)) = hi;
            }
            fence_proxy_async_smem();  // the tile is read by the tensor cores
            __syncwarp();
            if (lane == 0) fp8_arrive(bar((KV ? VFULL : KFULL) + s));
          }
        }
      };
      if (warp < 16)
        team(std::integral_constant<int, 0>{});
      else
        team(std::integral_constant<int, 1>{});
    } else if (warp == 24) {
      // ================= producer =================
      int n = 0, nq = 0, kfree = 0;
      PrefillItem item;
#pragma unroll 1
      for (int itc = 0;; itc++) {
        const int e = itc & 1;
        if (itc >= 2) fp8_wait(bar(IFREE + e), (itc / 2 - 1) & 1, abort_flag, c.status);
        int itn = n_items;
        if (lane == 0 && !*abort_flag) itn = atomicAdd(&pv.plan[2], 1);
        item = prefill_piece_item(c, pv, __shfl_sync(0xffffffffu, itn, 0), n_items);
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
        const SeqView view = seq_view<true>(c, pv, item.seq);
        const int q0 = view.q0, tok0 = item.tile * c.tile_tokens, h = item.h, nkb = item.nkb;
        const int nsteps = steps_of(item), none = c.num_blocks * 16;
        // lane b < NB holds block b of a step and its scales, a step ahead
        auto block_of = [&](int st) -> int {
          const int kb = item.kb0 + st * NB + lane;
          if (st >= nsteps || lane >= NB || kb >= nkb) return -1;
          const int id = c.block_table[view.tab + kb];
          if (id >= 0 && id < c.num_blocks) return id;
          flag(c.status, KV_INT4_DEV_BAD_BLOCK);
          return -1;
        };
        auto scale_of = [&](const float* scales, int blk, float without) {
          return blk >= 0 ? scales[(long long)blk * c.hkv + h] : without;
        };
        int blk = block_of(0), next = block_of(1);
        float ks = scale_of(c.k_scale, blk, 0.f), vs = scale_of(c.v_scale, blk, 1.f);
#pragma unroll 1
        for (int st = 0; st < nsteps; st++, n++) {
          if (__any_sync(0xffffffffu, *abort_flag)) break;
          const int s = n & 1;
          const int after = block_of(st + 2);
          const float ks1 = scale_of(c.k_scale, next, 0.f), vs1 = scale_of(c.v_scale, next, 1.f);
          const bool ok = blk >= 0;
          auto stage = [&](int kv, int full, int free) {
            if (n > 1) fp8_wait(bar(free + s), ((n - 2) >> 1) & 1, abort_flag, c.status);
            if (lane == 0) mbar_arrive_expect_tx(bar(full + s), G::STG);
            __syncwarp();
            if (lane < NB)
              tma_box4(smem_addr(stg + (2 * s + kv) * G::STG + lane * 16 * D), kv ? &maps.v : &maps.k, h, ok ? blk * 16 : none,
                       bar(full + s));
          };
          stage(0, RKFULL, RKFREE);
          stage(1, RVFULL, RVFREE);
          if (st == 0) {
            wait_until(KFREE, kfree, n);  // every S of the previous item: its Q has been read
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(QFULL), c.group * c.tile_tokens * 128 * G::KB);
#pragma unroll
              for (int x = 0; x < G::KB; x++)
                tma_box3(smem_addr(sQ + x * RN * 128), &maps.q, 64 * x, h * c.group, q0 + tok0, bar(QFULL));
            }
            __syncwarp();
            nq++;
          }
          wait_until(KFREE, kfree, n - 1);  // S of step n - 2: ring entry n % 4 has been read
          float* re = reinterpret_cast<float*>(ring + (n % G::NRING) * G::RING);
          if (lane < NB) {
            const bool low = vs < exp2_int(kFp8LowExp);
            re[lane] = ks;
            re[NB + lane] = (float)exp_of(vs);
            re[2 * NB + lane] = low ? 0.f : __uint_as_float((254u << 23) - (__float_as_uint(vs) & 0x7f800000u));
            reinterpret_cast<int*>(re)[3 * NB + lane] = ok;
          }
          __syncwarp();
          if (lane == 0) fp8_arrive(bar(KFULL + s));
          blk = next;
          next = after;
          ks = ks1;
          vs = vs1;
        }
      }
      // the last copies have landed before the CTA ends, after an abort too
      for (int x = 0; x < 2; x++) {
        const int last = n - 1 - x;
        if (last >= 0 && !(mbar_wait_bounded(bar(RKFULL + (last & 1)), (last >> 1) & 1) &&
                           mbar_wait_bounded(bar(RVFULL + (last & 1)), (last >> 1) & 1)))
          flag(c.status, KV_INT4_DEV_TIMEOUT);
      }
      if (nq > 0 && !mbar_wait_bounded(bar(QFULL), (nq - 1) & 1)) flag(c.status, KV_INT4_DEV_TIMEOUT);
    } else if (warp == 25) {
      // ================= MMA =================
      uint32_t lead;
      asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(lead));
      const uint64_t dk = umma_desc(smem_addr(sK), 16, 1024), dq = umma_desc(smem_addr(sQ), 16, 1024);
      const uint64_t dv = umma_desc(smem_addr(sV), NK * 128, 1024), dp = umma_desc(smem_addr(sP), 16, 1024);
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);  // in a uniform register
      int n = 0, items = 0;
#pragma unroll 1
      for (int itc = 0;; itc++) {
        fp8_wait_warp(bar(IFULL + (itc & 1)), (itc >> 1) & 1, abort_flag, c.status);
        const PrefillItem item = item_at(itc & 1);
        __syncwarp();
        if (lane == 0) fp8_arrive(bar(IFREE + (itc & 1)));
        __syncwarp();
        int steps = -1, rows = 0;
        if (item.seq >= 0 && !*abort_flag) {
          steps = steps_of(item);
          rows = min(c.tile_tokens, pv.vrec[2 * item.seq].y - item.tile * c.tile_tokens) * c.group;
        }
        const int nsteps = __reduce_min_sync(0xffffffffu, steps);
        if (nsteps < 0) break;
        if (nsteps == 0) continue;
        const uint32_t cols = __reduce_max_sync(0xffffffffu, rows) <= 32 ? 32 : 64;
        const uint32_t idesc_s = (umma_idesc_f16(128, 0, false) | (1u << 7) | (1u << 10)) + ((cols >> 3) << 17);  // bf16
        const uint32_t idesc_o = (umma_idesc_f16(128, 0, false) | (1u << 15)) + ((cols >> 3) << 17);  // A (V^T) MN-major
        fp8_wait_warp(bar(QFULL), items & 1, abort_flag, c.status);
        items++;
        // iteration st: S of step st, then WV of the step before, whose sums ran meanwhile
#pragma unroll 1
        for (int st = 0; st <= nsteps; st++) {
          if (st < nsteps) {
            fp8_wait_warp(bar(KFULL + (n & 1)), (n >> 1) & 1, abort_flag, c.status);
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < KSTEPS; ks++)
              fp8_mma(lead, tm + RN * (n & 1), dk + (uint64_t)(((ks >> 2) * NK * 128 + (ks & 3) * 32) >> 4),
                      dq + (uint64_t)(((ks >> 2) * RN * 128 + (ks & 3) * 32) >> 4), idesc_s, ks > 0);
            fp8_commit(lead, bar(SFULL + (n & 1)));
            fp8_commit(lead, bar(KFREE + (n & 1)));
          }
          if (st > 0) {
            const int m = n - 1;  // the step before
            {
              const int i = lane == 0 ? VFULL + (m & 1) : PFULL + (m & 1);
              fp8_wait_warp(bar(i), (m >> 1) & 1, abort_flag, c.status, lane > 1);
            }
            tc_fence_after();
            const uint64_t vt = dv + (uint64_t)((m & 1) * (G::VBYTES >> 4)), pt = dp + (uint64_t)((m & 1) * (G::PBYTES >> 4));
#pragma unroll
            for (int kk = 0; kk < NB; kk++)
              fp8_mma(lead, tm + G::O_COL, vt + (uint64_t)(kk * (2048 >> 4)),
                      pt + (uint64_t)(((kk >> 2) * RN * 128 + (kk & 3) * 32) >> 4), idesc_o, st > 1 || kk > 0);
            fp8_commit(lead, bar(VFREE + (m & 1)));
          }
          if (st < nsteps) n++;
        }
        fp8_commit(lead, bar(ODONE));
      }
      // after a time-out MMAs may still be in flight: they end by themselves
      // and must end before the columns are freed
      if (lane == 0) umma_commit(bar(DRAIN));
      __syncwarp();
      if (!mbar_wait_bounded(bar(DRAIN), 0)) flag(c.status, KV_INT4_DEV_TIMEOUT);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 256);
}
