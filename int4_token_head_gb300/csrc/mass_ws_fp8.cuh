// Attention masses of many query rows on the 5th-generation tensor cores
// (tcgen05), included by mass_fp8.cu.
//
// One CTA per SM; an item is 128 keys of one kv head of a sequence, the MMA's M:
// S = K Q^T with a tile of QR query rows as N, so that a key is a TMEM lane and
// the sum over the rows stays in one thread: per score one fma (the key's factor,
// the row's -lse log2 e), one exp2 and one add, and nothing crosses threads until
// an item's four partial sums meet.  Row tiles are numbered over all items of a
// CTA (g); warps in five roles that meet at mbarriers:
//   * scheduler warp (20): the items of this CTA in an order that it computes by
//     itself (below), through a ring of four;
//   * copy warps (21, 22), even and odd g: TMA copies of the Q tiles that see an
//     item's keys (bf16, straight into the MMA's swizzled tile) into slot g mod NQ;
//   * convert warps (16-19): an item's codes from global memory into one of two bf16
//     tiles, and its blocks' scales into the item's ring entry;
//   * MMA warps (23, 24), even and odd g: a tile into the score buffer of warpgroup g
//     mod 4.  NQ is even, so that a slot's and a buffer's barriers each have one
//     warp that waits for them in turn;
//   * sum warps (0-15): warpgroup g mod 4; the rows' lse are loaded a tile ahead
//     and shared through shared memory.
// Bounds are the exp2 of every score and the MMAs, alike: 512 cycles each for 128 x
// 128 scores at head size 128.  Eight prompts of 512 to 2048 tokens, 32/8 heads: 66.4
// us, a tile every 900 cycles and 1.5 us from an item to the next; both pipes are
// active 0.43 of the time.  A warpgroup sums for 1700 cycles and has its next scores
// 1200 after it has freed its one buffer (TMEM is full).  Not faster: two warpgroups
// with two buffers each 90 us; items of 256 keys, which halve the copies of Q, 81
// (the longest end too late); halves of a buffer freed by themselves, MMAs of 64
// columns, 76; a buffer's scores, the copies or the exponents left out 63 to 73.
//
// Order of items: an item's work is the query rows that see it, which falls with
// the key tile's index where the queries start at the front.  Items are taken by
// their distance from the sequence's end, the longest first, all sequences and
// heads of a distance side by side, and dealt to the CTAs back and forth: no
// counter in memory, nothing left from call to call, and the same sums whatever the
// timing.  Batches of more than kLevelSeqs such sequences, or of more than
// kLevels key tiles, take the sequences one after the other.
constexpr int kMassWindow = 1024;  // sequences whose items are listed at a time
constexpr int kLevelSeqs = 128;
constexpr int kLevels = 1024;

template <int D>
struct MassWs {
  static constexpr int QR = D <= 128 ? 128 : 64;  // query rows per tile
  static constexpr int KB = (D + 63) / 64;        // 128-byte blocks of a bf16 head vector
  static constexpr int QBYTES = QR * 128 * KB, KBYTES = 128 * 128 * KB;
  static constexpr int NQ = D == 256 ? 2 : 4;     // Q slots, an even number
  static constexpr int NI = 4;                    // item ring
  static constexpr int S_COLS = 4 * QR;           // TMEM: a score buffer per warpgroup
  static constexpr int WG = 4;                    // warpgroups that sum
  static constexpr int THREADS = (4 * WG + 9) * 32;
  // item ring entry: 8 ints, 8 scales
  static constexpr int ENTRY = 64;
  static constexpr int NBARS = 2 * NI + 2 * NQ + 4 + 2 * WG + NI + 1;
  static constexpr int BARS = (NBARS * 8 + 15) / 16 * 16;  // what follows is read in 16-byte words
  static constexpr int TAIL = NI * ENTRY + BARS + 16 + WG * 2 * 128 * 4 + NI * (WG - 1) * 128 * 4 + kMassWindow * 8;
  static constexpr int SMEM = 2 * KBYTES + NQ * QBYTES + TAIL;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert((2 * KBYTES + NQ * QBYTES) % 1024 == 0 && (NI * ENTRY + BARS) % 16 == 0, "alignment");
};

struct MassItem {
  int seq, head, kt;         // seq -1: no more
  int tok0, tiles;           // first query token that sees it (of the sequence), Q tiles from there
  int q0, ql, len;
};

__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  // the registers are outputs so that no use of them moves before the wait
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

template <int D>
__global__ void __launch_bounds__(MassWs<D>::THREADS, 1)
    mass_ws_kernel(MassParams p, int tile_tokens, const __grid_constant__ CUtensorMap qmap) {
  using G = MassWs<D>;
  constexpr int KSTEPS = D / 16, QR = G::QR, NQ = G::NQ, NI = G::NI, WG = G::WG, CH = D / 16;
  constexpr uint32_t IDESC = umma_idesc_f16(128, QR, false) | (1u << 7) | (1u << 10);  // bf16 operands
  extern __shared__ __align__(1024) uint8_t smem_mass[];
  uint8_t* const sK = smem_mass;                   // two tiles [KB][128][128 B], swizzled
  uint8_t* const sQ = sK + 2 * G::KBYTES;          // NQ tiles [KB][QR][128 B]
  uint8_t* const ring = sQ + NQ * G::QBYTES;       // items
  uint64_t* const bars = reinterpret_cast<uint64_t*>(ring + NI * G::ENTRY);
  int* const sctl = reinterpret_cast<int*>(ring + NI * G::ENTRY + G::BARS);  // abort flag, TMEM address
  float* const snl = reinterpret_cast<float*>(sctl + 4);      // [warpgroup][2][128]: -lse log2 e of a tile's rows
  float* const spart = snl + WG * 2 * 128;                    // [NI][WG - 1][128]: the other warpgroups' sums
  int2* const slist = reinterpret_cast<int2*>(spart + NI * (WG - 1) * 128);  // [kMassWindow] (sequence, key tiles)
  volatile int* const abort_flag = sctl;
  const MassArgs& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  enum {
    IFULL = 0, IFREE = IFULL + NI, QFULL = IFREE + NI, QFREE = QFULL + NQ, KFULL = QFREE + NQ, KFREE = KFULL + 2,
    SFULL = KFREE + 2, SFREE = SFULL + WG, PART = SFREE + WG, DRAIN = PART + NI
  };
  static_assert(DRAIN + 1 == G::NBARS, "barriers");
  auto bar = [&](int i) { return smem_addr(&bars[i]); };
  if (smem_addr(smem_mass) & 1023) {  // dynamic shared memory starts the window: does not occur
    flag(a.dev_status, KV_INT4_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int b = 0; b < NI; b++) {
      mbar_init(bar(IFULL + b), 1);
      mbar_init(bar(IFREE + b), 4 * WG + 8);
      mbar_init(bar(PART + b), 4 * (WG - 1));
    }
    for (int b = 0; b < NQ; b++) {
      mbar_init(bar(QFULL + b), 1);
      mbar_init(bar(QFREE + b), 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(bar(KFULL + b), 4);
      mbar_init(bar(KFREE + b), 2);
    }
    for (int b = 0; b < WG; b++) {
      mbar_init(bar(SFULL + b), 1);
      mbar_init(bar(SFREE + b), 4);
    }
    mbar_init(bar(DRAIN), 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // rows of a Q slot that no copy writes (groups that do not divide QR) are zeros
  for (int x = tid; x < NQ * G::QBYTES / 16; x += G::THREADS) reinterpret_cast<uint4*>(sQ)[x] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  pdl_trigger();
  pdl_wait();
  if (warp == 0) tmem_alloc(smem_addr(sctl + 1), G::S_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)sctl[1];
  auto entry = [&](int e) { return reinterpret_cast<int*>(ring + e * G::ENTRY); };
  // a consumer's wait for item n, warp-uniform; seq -1 at the end (and after a time-out)
  auto take = [&](int n) {
    const int e = n % NI;
    MassItem it{-1, 0, 0, 0, 0, 0, 0, 0};
    if (__all_sync(0xffffffffu, fp8_wait(bar(IFULL + e), (n / NI) & 1, abort_flag, a.dev_status))) {
      const int4 x = *reinterpret_cast<const int4*>(entry(e)), y = *reinterpret_cast<const int4*>(entry(e) + 4);
      it = MassItem{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    }
    return it;
  };

  if (warp < 4 * WG) {
    // ======================= sums =======================
    const int wg = warp >> 2, r = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int tile_rows = tile_tokens * p.group;
    float* const nls = snl + wg * 2 * 128;
    const int j = (int)p.by_group.div((uint32_t)r), jj = r - j * p.group;  // this thread's column of every tile
    auto row_lse = [&](const MassItem& it, int t) {  // the column's of tile t; infinity for none
      const int tok = it.tok0 + t * tile_tokens + j;
      float l = INFINITY;
      if (it.seq >= 0 && r < tile_rows && tok < it.ql)
        l = a.lse[(int64_t)(it.q0 + tok) * a.lse_stride + it.head * p.group + jj];
      return l;
    };
    // sum of a tile's weights for this key; the columns [lo, hi) see it
    auto sum_tile = [&](auto masked, const float* nl, float f, int lo, int hi) {
      constexpr bool MASKED = decltype(masked)::value;
      const uint32_t ts = tmem + QR * wg + lane_off;
      uint32_t x[2][16];
      tmem_ld16_async(ts, x[0]);
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;
      const float2 ff = make_float2(f, f);
#pragma unroll
      for (int c = 0; c < QR / 16; c++) {
        tmem_ld_wait(x[c & 1]);
        if (c + 1 < QR / 16) {
          tmem_ld16_async(ts + 16 * (c + 1), x[(c + 1) & 1]);
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) fp8_arrive(bar(SFREE + wg));
        }
        const uint32_t (&v)[16] = x[c & 1];
        uint32_t vis = 0xffffu;  // the chunk's columns that see the key
        if (MASKED) {
          const int from = lo - 16 * c, to = hi - 16 * c;
          vis = from <= 0 ? 0xffffu : from >= 16 ? 0u : 0xffffu << from;
          vis &= to >= 16 ? 0xffffu : to <= 0 ? 0u : 0xffffu >> (16 - to);
        }
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 b = *reinterpret_cast<const float4*>(nl + 16 * c + k);
          const float2 t0 = f2fma(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), ff, make_float2(b.x, b.y));
          const float2 t1 = f2fma(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), ff, make_float2(b.z, b.w));
          float2 e0 = make_float2(fast_exp2(t0.x), fast_exp2(t0.y)), e1 = make_float2(fast_exp2(t1.x), fast_exp2(t1.y));
          if (MASKED) {
            e0.x = vis & (1u << k) ? e0.x : 0.f;
            e0.y = vis & (2u << k) ? e0.y : 0.f;
            e1.x = vis & (4u << k) ? e1.x : 0.f;
            e1.y = vis & (8u << k) ? e1.y : 0.f;
          }
          s0 = f2add(s0, e0);
          s1 = f2add(s1, e1);
        }
      }
      return (s0.x + s0.y) + (s1.x + s1.y);
    };
    // the warpgroup's warps go on together or not at all (after a time-out one may
    // get an item that the others do not)
    auto take_all = [&](int n) {
      MassItem x = take(n);
      uint32_t end;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.lt.s32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(end)
          : "r"(x.seq), "r"(1 + wg)
          : "memory");
      if (end) x.seq = -1;
      return x;
    };
    MassItem it = take_all(0);
    int first = wg, before = 0;  // this warpgroup's first tile of the item, row tiles of earlier items
    float l = row_lse(it, first);
    int cnt = 0;  // tiles of this warpgroup
#pragma unroll 1
    for (int n = 0; it.seq >= 0; n++) {
      const int e = n % NI;
      const int ctx = it.len - it.ql, pos = it.kt * 128 + r;
      float* const out = a.mass + it.seq * a.mass_seq_stride + it.head * a.mass_head_stride + pos;
      float old = 0.f;
      if (wg == 0 && pos < ctx) old = *out;
      float w = 0.f, f = 0.f;
      MassItem next{-1, 0, 0, 0, 0, 0, 0, 0};
      before += it.tiles;
      const int next_first = (wg - before) & (WG - 1);
      bool taken = false;
#pragma unroll 1
      for (int t = first; t < it.tiles; t += WG, cnt++) {
        float* const nl = nls + (cnt & 1) * 128;
        nl[r] = fabsf(l) == INFINITY ? -INFINITY : -l * kLog2e;
        if (t + WG < it.tiles) {
          l = row_lse(it, t + WG);
        } else {
          next = take_all(n + 1);
          taken = true;
          l = row_lse(next, next_first);
        }
        asm volatile("bar.sync %0, 128;\n" ::"r"(1 + wg) : "memory");
        fp8_wait(bar(SFULL + wg), cnt & 1, abort_flag, a.dev_status);
        tc_fence_after();
        if (t == first) f = p.qscale * reinterpret_cast<const float*>(entry(e) + 8)[r >> 4];
        const int tok = it.tok0 + t * tile_tokens;
        // this key is hidden from columns before `lo` (0: from none; the distance to a far
        // key times the group is more than 32 bits) and there are none from `hi` on
        const int lo = max(pos - ctx - tok, 0) * p.group, hi = min(tile_tokens, it.ql - tok) * p.group;
        const bool full = __all_sync(0xffffffffu, lo == 0) && hi == tile_rows;
        // two copies of the loop: a branch in it keeps its loads, exponentials and sums
        // from overlapping (2900 cycles a tile)
        w += full ? sum_tile(std::false_type{}, nl, f, lo, hi) : sum_tile(std::true_type{}, nl, f, lo, hi);
      }
      if (!taken) {
        next = take_all(n + 1);
        l = row_lse(next, next_first);
      }
      float* const part = spart + e * (WG - 1) * 128 + r;
      if (wg > 0) {
        part[(wg - 1) * 128] = w;
        __syncwarp();
        if (lane == 0) fp8_arrive(bar(PART + e));
      } else {
        fp8_wait(bar(PART + e), (n / NI) & 1, abort_flag, a.dev_status);
#pragma unroll
        for (int x = 0; x < WG - 1; x++) w += part[x * 128];
        const float ks = reinterpret_cast<const float*>(entry(e) + 8)[r >> 4];
        if (pos < it.len) *out = (ks == 0.f ? 0.f : w) + old;  // a position without a block receives nothing
      }
      __syncwarp();
      if (lane == 0) fp8_arrive(bar(IFREE + e));
      it = next;
      first = next_first;
    }
  } else if (warp < 4 * WG + 4) {
    // ======================= codes =======================
    const int t = tid & 127;
    const __nv_bfloat162 kf = __float2bfloat162_rn(exp2_int(120));
    int freed = 0;
#pragma unroll 1
    for (int n = 0;; n++) {
      const MassItem it = take(n);
      if (it.seq < 0) break;
      const int32_t* const table = a.block_table + (int64_t)it.seq * a.max_blocks_per_seq;
      const int nblk = (it.len + 15) >> 4;
      auto block_at = [&](int b) {
        int id = b < nblk ? table[b] : -1;
        return id >= 0 && id < a.num_blocks ? id : -1;
      };
      if (t < 8) {
        const int b = it.kt * 8 + t, blk = block_at(b);
        reinterpret_cast<float*>(entry(n % NI) + 8)[t] = blk >= 0 ? a.k_scale[(int64_t)blk * a.num_kv_heads + it.head] : 0.f;
        if (b < nblk && blk < 0 && it.head == 0) flag(a.dev_status, KV_INT4_DEV_BAD_BLOCK);
      }
      uint8_t* const dst = sK + (n & 1) * G::KBYTES;
      constexpr int PART_CH = CH < 8 ? CH : CH % 8 ? CH / 2 : 8;  // chunks in flight per thread
#pragma unroll 1
      for (int i0 = 0; i0 < CH; i0 += PART_CH) {
        uint4 x[PART_CH];
        int id[PART_CH];
#pragma unroll
        for (int i = 0; i < PART_CH; i++) id[i] = block_at(it.kt * 8 + ((t + 128 * (i0 + i)) / CH >> 4));
#pragma unroll
        for (int i = 0; i < PART_CH; i++) {
          const int c = t + 128 * (i0 + i), row = c / CH, col = c - row * CH;
          x[i] = make_uint4(0, 0, 0, 0);
          if (id[i] >= 0 && it.kt * 128 + row < it.len)
            x[i] = *reinterpret_cast<const uint4*>(
                a.k_cache + (((int64_t)id[i] * 16 + (row & 15)) * a.num_kv_heads + it.head) * D + 16 * col);
        }
        for (; freed < n - 1; freed++) fp8_wait(bar(KFREE + (freed & 1)), (freed >> 1) & 1, abort_flag, a.dev_status);
#pragma unroll
        for (int i = 0; i < PART_CH; i++) {
          const int c = t + 128 * (i0 + i), row = c / CH, col = c - row * CH;
          uint4 lo, hi;
          e4m3x4_to_bf16x2(x[i].x, kf, lo.x, lo.y);
          e4m3x4_to_bf16x2(x[i].y, kf, lo.z, lo.w);
          e4m3x4_to_bf16x2(x[i].z, kf, hi.x, hi.y);
          e4m3x4_to_bf16x2(x[i].w, kf, hi.z, hi.w);
          *reinterpret_cast<uint4*>(dst + fp8_sw128(128, row, 2 * col)) = lo;
          *reinterpret_cast<uint4*>(dst + fp8_sw128(128, row, 2 * col + 1)) = hi;
        }
      }
      fence_proxy_async_smem();  // the tile is read by the tensor cores
      __syncwarp();
      if (lane == 0) {
        fp8_arrive(bar(KFULL + (n & 1)));
        fp8_arrive(bar(IFREE + n % NI));
      }
    }
  } else if (warp == 4 * WG + 4) {
    // ======================= scheduler =======================
    const int grid = gridDim.x, hkv = a.num_kv_heads;
    int n = 0;  // items handed on
    auto hand_on = [&](const MassItem& it) {
      const int e = n % NI;
      if (n >= NI) fp8_wait(bar(IFREE + e), (n / NI - 1) & 1, abort_flag, a.dev_status);
      if (lane == 0) {
        int4* const x = reinterpret_cast<int4*>(entry(e));
        x[0] = make_int4(*abort_flag ? -1 : it.seq, it.head, it.kt, it.tok0);
        x[1] = make_int4(it.tiles, it.q0, it.ql, it.len);
        fp8_arrive(bar(IFULL + e));
      }
      __syncwarp();
      n++;
    };
    auto item = [&](int seq, int head, int kt) {
      const int q0 = a.query_start_loc[seq], ql = a.query_start_loc[seq + 1] - q0, len = a.seq_lens[seq];
      const int tok0 = max(0, kt * 128 - (len - ql));
      return MassItem{seq, head, kt, tok0, (ql - tok0 + tile_tokens - 1) / tile_tokens, q0, ql, len};
    };
    long long k = 0;     // this CTA's k-th item is number k grid + (its place, back and forth)
    long long base = 0;  // items of earlier windows
    auto number = [&](long long x) { return x * grid + ((x & 1) ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x); };
#pragma unroll 1
    for (int w0 = 0; w0 < a.num_seqs; w0 += kMassWindow) {
      // the window's sequences with many rows, in order
      int count = 0, top = 0;
      for (int s0 = w0; s0 < min(a.num_seqs, w0 + kMassWindow); s0 += 32) {
        int nt = 0;
        const int s = s0 + lane;
        if (s < min(a.num_seqs, w0 + kMassWindow)) {
          const int q0 = a.query_start_loc[s], ql = a.query_start_loc[s + 1] - q0, len = a.seq_lens[s];
          if (mass_seq_ok(a, q0, ql, len) && !few_rows(p, ql)) nt = (len + 127) >> 7;
        }
        const uint32_t m = __ballot_sync(0xffffffffu, nt > 0);
        if (nt > 0) slist[count + __popc(m & ((1u << lane) - 1))] = make_int2(s, nt);
        count += __popc(m);
        top = max(top, (int)__reduce_max_sync(0xffffffffu, nt));
      }
      __syncwarp();
      if (count <= kLevelSeqs && top <= kLevels) {
        int seq[kLevelSeqs / 32], nts[kLevelSeqs / 32];
#pragma unroll
        for (int i = 0; i < kLevelSeqs / 32; i++) {
          const int2 x = 32 * i + lane < count ? slist[32 * i + lane] : make_int2(0, 0);
          seq[i] = x.x;
          nts[i] = x.y;
        }
#pragma unroll 1
        for (int m = top; m > 0; m--) {
          uint32_t has[kLevelSeqs / 32];
          int c = 0;
#pragma unroll
          for (int i = 0; i < kLevelSeqs / 32; i++) {
            has[i] = __ballot_sync(0xffffffffu, nts[i] >= m);
            c += __popc(has[i]);
          }
#pragma unroll 1
          for (; number(k) < base + (long long)c * hkv; k++) {
            const int off = (int)(number(k) - base), which = off / hkv;
            int s = 0, nt = 0, before = 0;
#pragma unroll
            for (int i = 0; i < kLevelSeqs / 32; i++) {
              const int here = __popc(has[i]);
              const int src = which >= before && which < before + here ? (int)__fns(has[i], 0, which - before + 1) : -1;
              const int xs = __shfl_sync(0xffffffffu, seq[i], src & 31), xn = __shfl_sync(0xffffffffu, nts[i], src & 31);
              if (src >= 0) {
                s = xs;
                nt = xn;
              }
              before += here;
            }
            hand_on(item(s, off - which * hkv, nt - m));
          }
          base += (long long)c * hkv;
        }
      } else {
#pragma unroll 1
        for (int x = 0; x < count; x++) {
          const int2 s = slist[x];
          const long long c = (long long)s.y * hkv;
#pragma unroll 1
          for (; number(k) < base + c; k++) {
            const long long off = number(k) - base;
            const int kt = (int)(off / hkv);
            hand_on(item(s.x, (int)(off - (long long)kt * hkv), kt));
          }
          base += c;
        }
      }
      __syncwarp();  // the list is read before the next window's is written
    }
    hand_on(MassItem{-1, 0, 0, 0, 0, 0, 0, 0});
  } else if (warp < 4 * WG + 7) {
    // ============ Q copies: row tiles of even number (over all items), and odd ============
    const int mine = warp - (4 * WG + 5);
    int g = mine, end = 0, last = -1;  // next tile; of lane s: the last fill of slot s
#pragma unroll 1
    for (int n = 0;; n++) {
      const MassItem it = take(n);
      if (it.seq < 0) break;
      const int begin = end;
      end += it.tiles;
#pragma unroll 1
      for (; g < end; g += 2) {
        const int s = g % NQ;
        if (g >= NQ) fp8_wait(bar(QFREE + s), (g / NQ - 1) & 1, abort_flag, a.dev_status);
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(QFULL + s), p.group * tile_tokens * 128 * G::KB);
#pragma unroll
          for (int x = 0; x < G::KB; x++)
            tma_box3(smem_addr(sQ + s * G::QBYTES + x * QR * 128), &qmap, 64 * x, it.head * p.group,
                     it.q0 + it.tok0 + (g - begin) * tile_tokens, bar(QFULL + s));
        }
        if (lane == s) last = g / NQ;
        __syncwarp();
      }
      __syncwarp();
      if (lane == 0) fp8_arrive(bar(IFREE + n % NI));
    }
    // every copy has landed before the CTA ends, after an abort too
    if (last >= 0 && !mbar_wait_bounded(bar(QFULL + lane), last & 1)) flag(a.dev_status, KV_INT4_DEV_TIMEOUT);
  } else {
    // ============ MMA: row tiles of even number, and odd ============
    const int mine = warp - (4 * WG + 7);
    uint32_t lead;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(lead));
    const uint64_t dk = umma_desc(smem_addr(sK), 16, 1024), dq = umma_desc(smem_addr(sQ), 16, 1024);
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);  // in a uniform register
    int g = mine, end = 0;  // next tile
#pragma unroll 1
    for (int n = 0;; n++) {
      const MassItem it = take(n);
      if (it.seq < 0) break;
      fp8_wait_warp(bar(KFULL + (n & 1)), (n >> 1) & 1, abort_flag, a.dev_status);
      const uint64_t kt = dk + (uint64_t)((n & 1) * (G::KBYTES >> 4));
      end += it.tiles;
#pragma unroll 1
      for (; g < end; g += 2) {
        const int s = g % NQ, buf = g % WG;
        // the tile's rows, and its score buffer
        fp8_wait_warp(bar(lane == 0 ? QFULL + s : SFREE + buf), lane == 0 ? (g / NQ) & 1 : (g / WG - 1) & 1, abort_flag,
                      a.dev_status, lane > 1 || (lane == 1 && g < WG));
        tc_fence_after();
        const uint64_t qt = dq + (uint64_t)(s * (G::QBYTES >> 4));
#pragma unroll
        for (int ks = 0; ks < KSTEPS; ks++)
          fp8_mma(lead, tm + QR * buf, kt + (uint64_t)(((ks >> 2) * 128 * 128 + (ks & 3) * 32) >> 4),
                  qt + (uint64_t)(((ks >> 2) * QR * 128 + (ks & 3) * 32) >> 4), IDESC, ks > 0);
        fp8_commit(lead, bar(SFULL + buf));
        fp8_commit(lead, bar(QFREE + s));
      }
      fp8_commit(lead, bar(KFREE + (n & 1)));
      __syncwarp();
      if (lane == 0) fp8_arrive(bar(IFREE + n % NI));
    }
    // after a time-out MMAs may still be in flight: they end by themselves
    // and must end before the columns are freed
    if (lane == 0) umma_commit(bar(DRAIN));
    __syncwarp();
    if (!mbar_wait_bounded(bar(DRAIN), 0)) flag(a.dev_status, KV_INT4_DEV_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, G::S_COLS);
}
