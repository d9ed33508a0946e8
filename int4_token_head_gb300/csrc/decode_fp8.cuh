// Split-KV decode over the FP8 cache and the merge of its pieces, included by
// attention_fp8.cu.
//
// Work: lanes of CTAs over the flattened (decode sequence, head group,
// position) units, each CTA an equal contiguous range of its lane (the
// schedule of decode.cuh; a position is NP consecutive 16-key blocks that
// share the MMA's eight query columns, COLS = 8 / NP each).  A CTA has one
// warp per kv head of its group, or CG warps that take eight query columns each
// (queries of up to 32 columns: a few tokens at once, large groups; the warps
// share the staged blocks, so the cache is still read once); all its threads copy the blocks' codes of the
// group's heads (contiguous runs of the cache) with 16-byte cp.async into a
// ring of block slots.  Rows behind the sequence's end, absent and unusable
// blocks are filled with zeros by the copies, so that no stale byte (E4M3 has
// NaN codes) reaches a product with a zero weight.
//
// Per block and head: S^T = K Q'^T with the 16 keys as the MMA's M, K codes
// straight from shared memory to f16 A fragments (a lane's four consecutive
// codes are one k-step's four elements: head dimensions are permuted the same
// way in q'), then the weights' transpose as B operand of O'^T += V^T W^T, V
// by ldmatrix.trans of byte pairs (one byte permute and two conversions per
// four codes).
//
// Memory-bound: 32 x 32768 keys, 32/8 heads of 128, 2.15 GB of codes: 342 us a
// call = 0.93 of the measured copy bandwidth.  More columns cost issue slots, as
// every warp converts the codes for its own eight: 32 x 1 token of group 16, 4 kv
// heads, against 2048-4096 keys 46 us (floor 15.5; in 256-row prefill tiles 81).
template <int D, int NP>
struct Fp8Dec {
  static constexpr int COLS = kDecodeCols / NP;
  static constexpr int CHR = D / 16;  // 16-byte chunks per code row
  // rows of a power-of-two number of chunks: chunk c of row r at chunk
  // c ^ swz(r), which spreads both an ldmatrix piece (8 rows, one chunk) and a
  // quarter-warp's K loads (2 rows, 4 chunks) over all banks; other row sizes
  // (96 and 192 bytes) do so for K as they are and for V with 16 bytes more
  static constexpr bool SWZ = (CHR & (CHR - 1)) == 0;
  static constexpr int VROW = SWZ ? D : D + 16;
  static constexpr int KTILE = 16 * D;
  static constexpr int VTILE = 16 * VROW;
  // neighbouring heads' rows in different bank halves
  static constexpr int HTILE = (KTILE + VTILE + 63) / 128 * 128 + 64;
  // block slots: the copies in flight per SM set the pace.  Two CTAs of four
  // heads fit an SM with six slots at 128 (two of two heads at 256), with eight
  // at 96 and 192 (32 x 32768 keys, 32/8 heads of 128: five slots 360 us, six
  // 344, seven, one CTA, 443)
  static constexpr int NS = NP == 1 ? 4 : NP == 4 || !SWZ ? 8 : 6;
  static constexpr int WAIT = NS - 2 * NP;                  // copy groups that may stay pending
  static constexpr int KSTEPS = D / 16;
  // head tiles, then the scales [K/V][hg]
  __host__ __device__ static constexpr int slot_bytes(int hg) { return hg * HTILE + 32; }
  __host__ __device__ static constexpr int smem_bytes(int hg) { return NS * slot_bytes(hg) + 32; }
  __host__ __device__ static constexpr int swz(int r) {
    return CHR >= 8 ? ((r & 1) << 2) | ((r >> 1) & 3) : (r >> 1) & 3;
  }
  static_assert(WAIT >= 0 && HTILE % 16 == 0, "ring");
};

template <int D>
constexpr bool kFp8PartsFit = Fp8Dec<D, 1>::smem_bytes(1) >= kDecodeColsFp8 * (D + 2) * 4;  // DIRECT's shares

// head sizes with four blocks per position (queries of at most two columns):
// where the eight-slot ring of four heads leaves room for two CTAs per SM
template <int D>
constexpr bool kFp8Quad = 2 * (Fp8Dec<D, 4>::smem_bytes(4) + 1024) <= 228 * 1024;

struct Fp8Walk {
  int i;     // decode sequence
  int grp;   // head group (grp mod nl = lane)
  int lane;
  int kp;    // position within the sequence
  int npos;  // positions of the sequence
  int fb;    // first block read (the sliding window's)
  int seq;   // sequence id
  int len;   // keys
};

struct Fp8DecParams {
  Common c;
  PlanView pv;
  int num_ctas;
  int cluster;  // DIRECT: CTAs per (sequence, head group)
  bool beside;  // the kernel before is a prefill of the same call
};

template <int NP>
__device__ __forceinline__ void fp8_walk_load(Fp8Walk& w, const Common& c, const PlanView& pv) {
  const int4 di = pv.dseq[w.i];  // (sequence, seq_len, first query token, q_len)
  w.seq = di.x;
  w.len = di.y;
  w.fb = first_block(c, di.y, di.w);
  w.npos = ((di.y + 15) / 16 - w.fb + NP - 1) / NP;
}
// the next unit of the lane (there is one: the caller counts)
template <int NP>
__device__ __forceinline__ void fp8_walk_next(Fp8Walk& w, const Common& c, const PlanView& pv) {
  if (++w.kp == w.npos) {
    w.kp = 0;
    if ((w.grp += c.nl) >= c.ng) {
      w.grp = w.lane;
      do {
        ++w.i;
        fp8_walk_load<NP>(w, c, pv);
      } while (w.npos == 0);  // sequences without keys have no units
    }
  }
}

// head dimension of element 0 of lane quarter cq's k-step s: the lane reads
// whole 16-byte chunks cq, cq + 4, ... of a swizzled row, else its contiguous quarter
template <int D>
__device__ __forceinline__ int fp8_kdim(int cq, int s) {
  if constexpr (Fp8Dec<D, 1>::SWZ) return 16 * (cq + 4 * (s >> 2)) + 4 * (s & 3);
  else return cq * (D / 4) + 4 * s;
}

// this CTA's rank in its cluster, and the cluster's barrier
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// a float of CTA `rank`'s shared memory, at this CTA's address p
__device__ __forceinline__ float ld_cluster(const float* p, int rank) {
  uint32_t a;
  float v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// DIRECT: no schedule, no pieces in the workspace and no merge launch.  A
// cluster of CTAs serves one (sequence, head group), its CTAs equal shares of
// the positions, and merges them through distributed shared memory: one launch
// for batches whose shares are short (latency counts there, not balance).
template <int D, int NP, int CG, bool DIRECT>
__global__ void __launch_bounds__(128) decode_fp8_kernel(Fp8DecParams prm) {
  using G = Fp8Dec<D, NP>;
  static_assert(CG == 1 || (NP == 1 && kFp8PartsFit<D>), "column groups");
  constexpr int SLOT = kDecodeCols * CG;           // columns of a result slot
  constexpr int CPT = (G::CHR + CG - 1) / CG;      // chunks a thread copies per block
  const Common& c = prm.c;
  const PlanView& pv = prm.pv;
  extern __shared__ __align__(16) uint8_t smem[];
  const int HG = c.hg;
  const int tid = threadIdx.x, nthr = HG * CG * 32;
  const int warp = tid >> 5, lane = tid & 31;
  const int hl = CG == 1 ? warp : warp / CG;       // head of the group
  const int cbase = CG == 1 ? 0 : warp % CG * kDecodeCols;  // first query column
  const int g = lane >> 2, cq = lane & 3;
  const int SB = G::slot_bytes(HG);
  pdl_trigger();
  // After a prefill launch decode runs beside it (on the SMs that prefill leaves)
  // and waits for it only at its end, so that what follows comes after both.
  // Before that wait it may rely on nothing but what it acquires: the schedule's
  // number, published by the schedule once that is complete, and with it the
  // schedule and everything written before.  Prefill lets this kernel in after
  // its own wait for the schedule, so that the number read is this call's; the
  // wait at the end shows whether it was, and if not the work is done again
  bool beside = !DIRECT && prm.beside;
  int32_t number = 0;
  if (beside) {
    if (lane == 0) number = ld_acquire(&pv.plan[5]);
    __syncwarp();
    number = __shfl_sync(0xffffffffu, number, 0);
  } else {
    pdl_wait();
  }
  // the end of the kernel: whether the work was done on this call's schedule
  auto done = [&]() -> bool {
    if (!beside) return true;
    pdl_wait();
    beside = false;
    return !__syncthreads_or(*const_cast<volatile int32_t*>(&pv.plan[5]) != number);
  };
again:
  int* sflag = reinterpret_cast<int*>(smem + G::NS * SB);

  Fp8Walk cw;
  int4 dseq0 = make_int4(0, 0, 0, 0);  // DIRECT: the sequence's record (sequence, seq_len, first query token, q_len)
  int nunits;
  const int rank = DIRECT ? cluster_rank() : 0;
  if constexpr (DIRECT) {
    const int task = blockIdx.x / prm.cluster;  // (sequence, head group)
    cw.seq = task / c.ng;
    cw.grp = task - cw.seq * c.ng;
    const int q0 = c.qsl[cw.seq], ql = c.qsl[cw.seq + 1] - q0;
    cw.len = c.seq_lens[cw.seq];
    // the same for the whole cluster
    if (!schedule_seq_ok<true>(c, q0, ql, cw.len)) {
      if (tid == 0 && rank == 0 && cw.grp == 0) flag(c.status, KV_INT4_DEV_BAD_SEQ);
      return;
    }
    if (ql == 0) return;
    dseq0 = make_int4(cw.seq, cw.len, q0, ql);
    cw.i = cw.lane = 0;
    cw.fb = first_block(c, cw.len, ql);
    const int npos = ((cw.len + 15) / 16 - cw.fb + NP - 1) / NP;
    const int first = (int)((long long)npos * rank / prm.cluster), end = (int)((long long)npos * (rank + 1) / prm.cluster);
    nunits = end - first;
    cw.kp = first;
    cw.npos = end;  // the CTA's last position ends its segment
  } else {
    const int n_dseq = pv.plan[0];
    if (n_dseq == 0) {
      if (done()) return;
      goto again;
    }
    const int gpl = c.ng / c.nl;  // head groups per lane
    const int my_lane = blockIdx.x % c.nl, rr = blockIdx.x / c.nl;
    const long long Tu = pv.dprefix[n_dseq] * gpl;
    const int R = prm.num_ctas / c.nl;
    const long long P0 = Tu * rr / R, P1 = Tu * (rr + 1) / R;
    if (P0 >= P1) {
      if (done()) return;
      goto again;
    }
    nunits = (int)(P1 - P0);

    // largest i with dprefix[i] * gpl <= P0 (32-ary search, per warp)
    int lo = 0, hi = n_dseq;
    while (hi - lo > 1) {
      const long long span = hi - lo;
      const int probe = lo + (int)((span * lane) / 32);
      const bool le = lane == 0 || pv.dprefix[probe] * gpl <= P0;
      const unsigned m = __ballot_sync(0xffffffffu, le);
      const int last = 31 - __clz(m);
      const int nlo = lo + (int)((span * last) / 32);
      const int nhi = last == 31 ? hi : lo + (int)((span * (last + 1)) / 32);
      lo = nlo;
      hi = nhi > nlo ? nhi : nlo + 1;
    }
    cw.i = lo;
    cw.lane = my_lane;
    fp8_walk_load<NP>(cw, c, pv);
    {
      const long long off = P0 - pv.dprefix[cw.i] * gpl;
      const int gs = (int)(off / cw.npos);
      cw.grp = gs * c.nl + my_lane;
      cw.kp = (int)(off - (long long)gs * cw.npos);
    }
  }
  Fp8Walk pw = cw;

  // staging: chunk index ((kv * 16 + r) * HG + h) * CHR + col, CPT chunks
  // a thread; consecutive threads read consecutive bytes
  uint32_t c_saddr[CPT];      // shared address within slot 0
  const uint8_t* c_src[CPT];  // cache address within block 0, head group 0
  const bool last_chunk = G::CHR % CG == 0 || tid + nthr * (CPT - 1) < 32 * HG * G::CHR;
#pragma unroll
  for (int j = 0; j < CPT; j++) {
    const int idx = tid + nthr * (j < CPT - 1 || last_chunk ? j : 0);
    const int col = idx % G::CHR, rest = idx / G::CHR;
    const int h = rest % HG, kvr = rest / HG;
    const int kv = kvr / 16, r = kvr % 16;
    const int pos = G::SWZ ? col ^ G::swz(r) : col;
    c_saddr[j] = smem_addr(smem) + h * G::HTILE + (kv ? G::KTILE + r * G::VROW : r * D) + pos * 16;
    c_src[j] = (kv ? c.v_cache : c.k_cache) + r * c.geo.crow + (long long)h * D + col * 16;
  }
  const uint32_t s_saddr = smem_addr(smem) + HG * G::HTILE + tid * 4;  // scale [K/V][h], threads 0 .. 2 hg - 1
  const float* s_src = tid < HG ? c.k_scale + tid : c.v_scale + (tid - HG);

  // block j of a position
  auto block_at = [&](const Fp8Walk& w, int j) {
    const int kb = w.fb + w.kp * NP + j;
    return kb * 16 < w.len ? c.block_table[(long long)w.seq * c.max_blocks + kb] : -1;
  };
  auto issue = [&](int blk, int kb, int len, int grp, int slot) {
    const bool ok = blk >= 0 && blk < c.num_blocks;
    const int rows = ok ? len - kb * 16 : 0;  // rows that hold keys (<= 0: an absent block)
    const uint32_t soff = (uint32_t)(slot * SB);
    const uint64_t base = ok ? (uint64_t)(uint32_t)blk * (uint64_t)c.geo.cblk + (uint64_t)(grp * HG) * D : 0;
    if (rows >= 16) {
#pragma unroll
      for (int j = 0; j < CPT; j++)
        if (j < CPT - 1 || last_chunk)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(c_saddr[j] + soff), "l"(c_src[j] + base));
    } else {
#pragma unroll
      for (int j = 0; j < CPT; j++) {
        if (j == CPT - 1 && !last_chunk) break;
        const int r = (tid + nthr * j) / G::CHR / HG % 16;
        const bool in = r < rows;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(c_saddr[j] + soff),
                     "l"(in ? c_src[j] + base : c.k_cache), "r"(in ? 16 : 0));
      }
    }
    if (tid < 2 * HG) {
      const float* src = ok ? s_src + (uint64_t)(uint32_t)blk * (uint64_t)c.hkv + grp * HG : c.k_scale;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(s_saddr + soff), "l"(src), "r"(ok ? 4 : 0));
    }
    if (tid == 0) {
      sflag[slot] = ok;
      if (!ok && kb * 16 < len) flag(c.status, KV_INT4_DEV_BAD_BLOCK);
    }
  };
  auto next = [&](Fp8Walk& w) {
    if constexpr (DIRECT) ++w.kp;
    else fp8_walk_next<NP>(w, c, pv);
  };
  // producer: one block per call into the next ring slot, the next block id
  // loaded one call ahead; one commit group per call (empty past the range)
  int ppos = 0, pj = 0, ps = 0;
  int pblk = nunits > 0 ? block_at(pw, 0) : -1;
  auto produce = [&]() {
    if (ppos < nunits) {
      issue(pblk, pw.fb + pw.kp * NP + pj, pw.len, pw.grp, ps);
      ps = ps + 1 == G::NS ? 0 : ps + 1;
      if (++pj == NP) {
        pj = 0;
        if (++ppos < nunits) next(pw);
      }
      if (ppos < nunits) pblk = block_at(pw, pj);
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int s = 0; s < G::NS - NP; s++) produce();

  // per-segment state of this warp's head
  uint32_t qb[G::KSTEPS][2];
  float oacc[G::KSTEPS][4];
  float m0, m1, l0, l1;
  float cf0, cf1;  // score factor of columns 2cq, 2cq+1: 2^e of the query row * softmax_scale * log2 e
  int lim0, lim1, lo0, lo1;  // keys visible to the columns: positions [lo, lim)
  int lim_warp, lo_warp;     // smallest limit, largest first position of all columns
  bool first_piece = cw.kp == 0;

  auto begin_segment = [&]() {
    const int head = cw.grp * HG + hl;
    const int4 di = DIRECT ? dseq0 : pv.dseq[cw.i];
    const int q0 = di.z, ql = di.w, L = di.y;
    const int ctx = L - ql;
    // B fragments of this lane's column g, which holds query column cbase + g % COLS
    const int n = cbase + (g & (G::COLS - 1));
    const bool colok = n < ql * c.group;
    const int j = n / c.group, jj = n - j * c.group;
    const uint16_t* qrow = c.q + (long long)(q0 + (colok ? j : 0)) * c.q_stride +
                           (long long)(head * c.group + (colok ? jj : 0)) * D;
    uint2 qv[G::KSTEPS];
    uint32_t am = 0;
#pragma unroll
    for (int s = 0; s < G::KSTEPS; s++) {
      qv[s] = make_uint2(0, 0);
      if (colok) qv[s] = *reinterpret_cast<const uint2*>(qrow + fp8_kdim<D>(cq, s));
      am = __vmaxu2(am, __vmaxu2(qv[s].x & 0x7fff7fffu, qv[s].y & 0x7fff7fffu));
    }
    am = max(am & 0xffffu, am >> 16);
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const int e = q_exponent(am);
    const float mul = exp2_int(-e);
#pragma unroll
    for (int s = 0; s < G::KSTEPS; s++) {
      qb[s][0] = pack_f16x2(bf16lo_to_f32(qv[s].x) * mul, bf16hi_to_f32(qv[s].x) * mul);
      qb[s][1] = pack_f16x2(bf16lo_to_f32(qv[s].y) * mul, bf16hi_to_f32(qv[s].y) * mul);
    }
    const float cf = c.qscale * exp2_int(e);
    cf0 = __shfl_sync(0xffffffffu, cf, 8 * cq);      // column 2 cq is held by lanes 4 (2 cq) ..
    cf1 = __shfl_sync(0xffffffffu, cf, 8 * cq + 4);
    const int col0 = cbase + ((2 * cq) & (G::COLS - 1)), col1 = cbase + ((2 * cq + 1) & (G::COLS - 1));
    const int j0 = min(col0 / c.group, max(ql - 1, 0)), j1 = min(col1 / c.group, max(ql - 1, 0));
    lim0 = c.causal ? min(L, ctx + j0 + 1) : L;
    lim1 = c.causal ? min(L, ctx + j1 + 1) : L;
    lo0 = window_lo(c, ctx + j0);
    lo1 = window_lo(c, ctx + j1);
    lim_warp = __reduce_min_sync(0xffffffffu, min(lim0, lim1));
    lo_warp = __reduce_max_sync(0xffffffffu, max(lo0, lo1));
#pragma unroll
    for (int i = 0; i < G::KSTEPS; i++) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.f;
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
  };

  auto flush = [&]() {
    float a0 = l0, a1 = l1;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      a0 += __shfl_xor_sync(0xffffffffu, a0, o);
      a1 += __shfl_xor_sync(0xffffffffu, a1, o);
    }
    float mm0 = m0, mm1 = m1;
    if constexpr (NP == 4) {
      // the four blocks' columns c, c + 2, c + 4, c + 6 hold the same queries:
      // merged here, so that a piece leaves columns 0 and 1 only
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) {
        const float p0 = __shfl_xor_sync(0xffffffffu, mm0, x), p1 = __shfl_xor_sync(0xffffffffu, mm1, x);
        const float n0 = fmaxf(mm0, p0), n1 = fmaxf(mm1, p1);
        const float u0 = n0 == -INFINITY ? 0.f : n0, u1 = n1 == -INFINITY ? 0.f : n1;
        const Exp2Pair ea0(mm0 - u0), eb0(p0 - u0), ea1(mm1 - u1), eb1(p1 - u1);
        const float sa0 = ea0.both(), sb0 = eb0.both(), sa1 = ea1.both(), sb1 = eb1.both();
        a0 = ea0.of(a0) + eb0.of(__shfl_xor_sync(0xffffffffu, a0, x));
        a1 = ea1.of(a1) + eb1.of(__shfl_xor_sync(0xffffffffu, a1, x));
#pragma unroll
        for (int i = 0; i < G::KSTEPS; i++) {
          oacc[i][0] = oacc[i][0] * sa0 + __shfl_xor_sync(0xffffffffu, oacc[i][0], x) * sb0;
          oacc[i][2] = oacc[i][2] * sa0 + __shfl_xor_sync(0xffffffffu, oacc[i][2], x) * sb0;
          oacc[i][1] = oacc[i][1] * sa1 + __shfl_xor_sync(0xffffffffu, oacc[i][1], x) * sb1;
          oacc[i][3] = oacc[i][3] * sa1 + __shfl_xor_sync(0xffffffffu, oacc[i][3], x) * sb1;
        }
        mm0 = n0;
        mm1 = n1;
      }
      if (cq > 0) return;
    }
    float* dst_o;
    float* dst_ml;
    if constexpr (DIRECT) {  // over the ring: every copy has landed, every warp is done
      dst_o = reinterpret_cast<float*>(smem) + hl * SLOT * (D + 2);
      dst_ml = dst_o + SLOT * D;
    } else if (first_piece) {
      const long long slot = (long long)cw.i * c.hkv + cw.grp * HG + hl;
      dst_o = pv.direct_o + slot * SLOT * D;
      dst_ml = pv.direct_ml + slot * SLOT * 2;
    } else {
      const long long slot = (long long)blockIdx.x * HG + hl;
      dst_o = pv.warp_o + slot * SLOT * D;
      dst_ml = pv.warp_ml + slot * SLOT * 2;
    }
    dst_o += cbase * D;
    dst_ml += cbase * 2;
    // m-tile t holds d = 16 t + 2g (row g) and 16 t + 2g + 1 (row g + 8)
    float* o0 = dst_o + (2 * cq) * D + 2 * g;
    float* o1 = dst_o + (2 * cq + 1) * D + 2 * g;
#pragma unroll
    for (int i = 0; i < G::KSTEPS; i++) {
      *reinterpret_cast<float2*>(o0 + 16 * i) = make_float2(oacc[i][0], oacc[i][2]);
      *reinterpret_cast<float2*>(o1 + 16 * i) = make_float2(oacc[i][1], oacc[i][3]);
    }
    if (g == 0) {
      dst_ml[(2 * cq) * 2 + 0] = mm0;
      dst_ml[(2 * cq) * 2 + 1] = a0;
      dst_ml[(2 * cq + 1) * 2 + 0] = mm1;
      dst_ml[(2 * cq + 1) * 2 + 1] = a1;
    }
  };

  begin_segment();
  const int jb = (cq * NP) >> 2;  // block of this thread's score columns
  const int jv = (g * NP) >> 3;   // block of this lane's W^T column g
  // this lane's ldmatrix row of the V tile: key 8 ((l >> 3) & 1) + (l & 7) of chunk (l >> 4)
  const int vrow = ((lane >> 3) & 1) * 8 + (lane & 7), vchunk = lane >> 4;
  const uint32_t v_lane = smem_addr(smem) + hl * G::HTILE + G::KTILE + vrow * G::VROW;
  const int vx = G::SWZ ? G::swz(vrow) : 0;
  const int kx0 = G::SWZ ? G::swz(g) : 0, kx1 = G::SWZ ? G::swz(g + 8) : 0;
  int cs = 0;
#pragma unroll 1
  for (int it = 0; it < nunits; it++) {
    cp_async_wait<G::WAIT>();
    __syncthreads();  // this position's copies visible; every warp done with the previous slots
#pragma unroll
    for (int j = 0; j < NP; j++) produce();

    int slot[NP];
    slot[0] = cs;
#pragma unroll
    for (int j = 1; j < NP; j++) slot[j] = slot[j - 1] + 1 == G::NS ? 0 : slot[j - 1] + 1;
    bool allok = true;
    int my = slot[0];
#pragma unroll
    for (int j = 0; j < NP; j++) {
      allok = allok && sflag[slot[j]] != 0;
      if (j > 0 && jb == j) my = slot[j];
    }
    const bool bok = sflag[my] != 0;
    const float* sc = reinterpret_cast<const float*>(smem + my * SB + HG * G::HTILE) + hl;
    const float ks = sc[0], vs = sc[HG];

    // ---- S^T = K Q'^T, one accumulator per block ----
    float sacc[NP][4];
#pragma unroll
    for (int j = 0; j < NP; j++) {
      sacc[j][0] = sacc[j][1] = sacc[j][2] = sacc[j][3] = 0.f;
      const uint8_t* x = smem + slot[j] * SB + hl * G::HTILE + g * D;
      const uint8_t* y = x + 8 * D;
      uint32_t xk[G::KSTEPS], yk[G::KSTEPS];
      if constexpr (G::SWZ) {
#pragma unroll
        for (int i = 0; i < G::CHR / 4; i++) {
          const uint4 a = *reinterpret_cast<const uint4*>(x + ((cq + 4 * i) ^ kx0) * 16);
          const uint4 b = *reinterpret_cast<const uint4*>(y + ((cq + 4 * i) ^ kx1) * 16);
          xk[4 * i] = a.x; xk[4 * i + 1] = a.y; xk[4 * i + 2] = a.z; xk[4 * i + 3] = a.w;
          yk[4 * i] = b.x; yk[4 * i + 1] = b.y; yk[4 * i + 2] = b.z; yk[4 * i + 3] = b.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < G::KSTEPS / 2; i++) {
          const uint2 a = *reinterpret_cast<const uint2*>(x + cq * (D / 4) + 8 * i);
          const uint2 b = *reinterpret_cast<const uint2*>(y + cq * (D / 4) + 8 * i);
          xk[2 * i] = a.x; xk[2 * i + 1] = a.y;
          yk[2 * i] = b.x; yk[2 * i + 1] = b.y;
        }
      }
#pragma unroll
      for (int s = 0; s < G::KSTEPS; s++) {
        uint32_t a[4];
        e4m3x4_to_f16x2(xk[s], a[0], a[2]);
        e4m3x4_to_f16x2(yk[s], a[1], a[3]);
        mma_16816(sacc[j], a, qb[s][0], qb[s][1]);
      }
    }
    float sa[4] = {sacc[0][0], sacc[0][1], sacc[0][2], sacc[0][3]};
#pragma unroll
    for (int j = 1; j < NP; j++)
#pragma unroll
      for (int e = 0; e < 4; e++) sa[e] = jb == j ? sacc[j][e] : sa[e];

    const int kb0 = cw.fb + cw.kp * NP;
    const int pos0 = (kb0 + jb) * 16 + g, pos1 = pos0 + 8;
    const float f0 = cf0 * ks, f1 = cf1 * ks;
    const float kvf = (float)exp_of(vs);                                  // log2 of the V scale
    const bool low = vs < exp2_int(kFp8LowExp);
    // its reciprocal; 0 where the denominator's share is taken below
    const float ivs = low ? 0.f : __uint_as_float((254u << 23) - (__float_as_uint(vs) & 0x7f800000u));
    float t00 = fmaf(sa[0], f0, kvf), t01 = fmaf(sa[1], f1, kvf);
    float t10 = fmaf(sa[2], f0, kvf), t11 = fmaf(sa[3], f1, kvf);
    // keys outside a column's visible range (or in an unusable or absent
    // block) only occur in positions that reach past the smallest limit or
    // start before the largest window start
    const bool full = allok && (kb0 + NP) * 16 <= lim_warp && kb0 * 16 >= lo_warp;
    if (!full) {
      t00 = (bok && pos0 < lim0 && pos0 >= lo0) ? t00 : -INFINITY;
      t01 = (bok && pos0 < lim1 && pos0 >= lo1) ? t01 : -INFINITY;
      t10 = (bok && pos1 < lim0 && pos1 >= lo0) ? t10 : -INFINITY;
      t11 = (bok && pos1 < lim1 && pos1 >= lo1) ? t11 : -INFINITY;
    }
    float mx0 = fmaxf(t00, t10), mx1 = fmaxf(t01, t11);
    // exact running max: reduced across the key lanes only when some lane
    // holds a value above its column's current max (or one of a small V scale)
    if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1 || low)) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
      const Exp2Pair e0(mn0 == -INFINITY ? 0.f : m0 - mn0);  // a column with no key yet keeps -inf
      const Exp2Pair e1(mn1 == -INFINITY ? 0.f : m1 - mn1);
      const float al0 = e0.both(), al1 = e1.both();
      m0 = mn0;
      m1 = mn1;
      l0 = e0.of(l0);
      l1 = e1.of(l1);
#pragma unroll
      for (int i = 0; i < G::KSTEPS; i++) {
        oacc[i][0] *= al0;
        oacc[i][1] *= al1;
        oacc[i][2] *= al0;
        oacc[i][3] *= al1;
      }
      if (low) {
        const float up0 = (float)kFp8LowExp - kvf - (m0 == -INFINITY ? 0.f : m0);
        const float up1 = (float)kFp8LowExp - kvf - (m1 == -INFINITY ? 0.f : m1);
        l0 = fmaf(fast_exp2(t00 + up0) + fast_exp2(t10 + up0), exp2_int(-kFp8LowExp), l0);
        l1 = fmaf(fast_exp2(t01 + up1) + fast_exp2(t11 + up1), exp2_int(-kFp8LowExp), l1);
      }
    }
    const float mu0 = m0 == -INFINITY ? 0.f : m0, mu1 = m1 == -INFINITY ? 0.f : m1;
    const float w00 = fast_exp2(t00 - mu0), w01 = fast_exp2(t01 - mu1);
    const float w10 = fast_exp2(t10 - mu0), w11 = fast_exp2(t11 - mu1);
    l0 = fmaf(w00 + w10, ivs, l0);
    l1 = fmaf(w01 + w11, ivs, l1);
    const uint32_t b0 = movmatrix_trans(pack_f16x2(w00, w01)), b1 = movmatrix_trans(pack_f16x2(w10, w11));

    // ---- O'^T += V^T W^T ----
#pragma unroll
    for (int j = 0; j < NP; j++) {
      // block j's weights only: the other blocks' columns are zero
      const uint32_t bj0 = NP == 1 || jv == j ? b0 : 0u, bj1 = NP == 1 || jv == j ? b1 : 0u;
      const uint32_t va = v_lane + slot[j] * SB;
#pragma unroll
      for (int p = 0; p < G::CHR / 2; p++) {
        uint32_t r[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(va + ((2 * p + vchunk) ^ vx) * 16));
        // a word: bytes (2g, 2g + 1) of keys 2cq and 2cq + 1
#pragma unroll
        for (int q = 0; q < 2; q++) {
          uint32_t a[4];
          e4m3x4_to_f16x2(__byte_perm(r[2 * q], 0, 0x3120), a[0], a[1]);
          e4m3x4_to_f16x2(__byte_perm(r[2 * q + 1], 0, 0x3120), a[2], a[3]);
          mma_16816(oacc[2 * p + q], a, bj0, bj1);
        }
      }
    }

    const bool last_in_seg = !DIRECT && cw.kp == cw.npos - 1;
    const bool last_in_range = it + 1 == nunits;
    if (!DIRECT && (last_in_seg || last_in_range)) flush();
    if (!last_in_range) {
      next(cw);
      if (last_in_seg) {
        first_piece = true;
        begin_segment();
      }
    }
    cs += NP;
    if (cs >= G::NS) cs -= G::NS;
  }
  cp_async_wait<0>();
  if (!done()) goto again;
  if constexpr (DIRECT) {
    __syncthreads();
    flush();
    cluster_sync();
    // (head, query column) rows in turn over the cluster's CTAs and their
    // warps; the shares (and with paired blocks a row's two columns) by the
    // log-sum-exp rule, all of a row's values loaded before any is used
    constexpr int PER = D / 32, SUB = NP == 2 ? 2 : 1;
    const int cols = dseq0.w * c.group;
#pragma unroll 1
    for (int p = rank * HG * CG + warp; p < HG * cols; p += prm.cluster * HG * CG) {
      const int h = p / cols, col = p - h * cols;
      const float* base = reinterpret_cast<const float*>(smem) + h * SLOT * (D + 2);
      float M = -INFINITY, Ls = 0.f, acc[PER];
#pragma unroll
      for (int k = 0; k < PER; k++) acc[k] = 0.f;
#pragma unroll 2
      for (int r = 0; r < prm.cluster; r++) {
        float mw[SUB], lw[SUB], o[SUB][PER];
#pragma unroll
        for (int sub = 0; sub < SUB; sub++) {
          const int cc = col + sub * G::COLS;
          mw[sub] = ld_cluster(base + SLOT * D + 2 * cc, r);
          lw[sub] = ld_cluster(base + SLOT * D + 2 * cc + 1, r);
#pragma unroll
          for (int k = 0; k < PER; k++) o[sub][k] = ld_cluster(base + cc * D + lane + 32 * k, r);
        }
#pragma unroll
        for (int sub = 0; sub < SUB; sub++) {
          const float mn = fmaxf(M, mw[sub]);
          const float mu = mn == -INFINITY ? 0.f : mn;
          const Exp2Pair ea(M - mu), eb(mw[sub] - mu);
          const float a = ea.both(), b = eb.both();
#pragma unroll
          for (int k = 0; k < PER; k++) acc[k] = acc[k] * a + o[sub][k] * b;
          Ls = ea.of(Ls) + eb.of(lw[sub]);
          M = mn;
        }
      }
      const float inv = Ls == 0.f ? 0.f : 1.f / Ls;  // no visible key: zeros
      const int j = col / c.group, jj = col - j * c.group;
      uint16_t* dst = c.out + (long long)(dseq0.z + j) * c.out_stride +
                      (long long)((cw.grp * HG + h) * c.group + jj) * D;
#pragma unroll
      for (int k = 0; k < PER; k++)
        dst[lane + 32 * k] = (uint16_t)(pack_bf16x2_rn(acc[k] * inv, 0.f) & 0xffffu);
    }
    cluster_sync();  // no CTA leaves while its shares are read
  }
}

// ---------------------------------------------------------------------------
// merge: the pieces of every segment, normalised and written as bf16
// ---------------------------------------------------------------------------
struct Fp8MergeParams {
  Common c;
  PlanView pv;
  int num_ctas;
  int cols;   // query columns per CTA (warps)
  int lanes;  // piece lanes per column (warps)
  int parts;  // CTAs per segment, cols columns each
  int slot;   // columns of a result slot
};

template <int D>
__host__ __device__ constexpr int merge_smem(int cols, int lanes) {
  return lanes > 1 ? cols * lanes * (D + 2) * 4 : 0;
}

// The rows of prefill tiles that were split over their keys, a warp per row:
// pieces weighted by 2^(m - M), added in their order.
template <int D>
__device__ void merge_prefill_pieces(const Common& c, const PlanView& pv, int first_warp, int num_warps) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const int n_split = pv.plan[4];
  int u = first_warp, base = 0;  // this warp's next row; rows before the 32 tiles in hand
#pragma unroll 1
  for (int e0 = 0; e0 < n_split; e0 += 32) {
    int4 t = make_int4(0, 0, 0, 0);  // (sequence, tile, first piece row, pieces)
    int R = 0, q0 = 0;               // rows per head, the tile's first query token
    if (e0 + lane < n_split) {
      t = pv.msplit[e0 + lane];
      const int qa = c.qsl[t.x], left = c.qsl[t.x + 1] - qa - t.y * c.tile_tokens;
      R = min(c.tile_tokens, left) * c.group;
      q0 = qa + t.y * c.tile_tokens;
    }
    int incl = R * c.hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
#pragma unroll 1
    for (; u < base + total; u += num_warps) {
      const int who = __ffs(__ballot_sync(0xffffffffu, u - base < incl)) - 1;
      const int rows = __shfl_sync(0xffffffffu, R, who), P = __shfl_sync(0xffffffffu, t.w, who);
      const int idx = u - base - (__shfl_sync(0xffffffffu, incl, who) - rows * c.hkv);
      const int h = idx / rows, r = idx - h * rows;
      const long long at = __shfl_sync(0xffffffffu, t.z, who) + (long long)h * P * rows + r;  // piece k: + k rows
      const int tok = __shfl_sync(0xffffffffu, q0, who);
      float M = -INFINITY;
      for (int k = lane; k < P; k += 32) M = fmaxf(M, pv.piece_ml[2 * (at + (long long)k * rows)]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float mu = M == -INFINITY ? 0.f : M;
      float acc[PER], Ls = 0.f;
#pragma unroll
      for (int i = 0; i < PER; i++) acc[i] = 0.f;
#pragma unroll 1
      for (int k0 = 0; k0 < P; k0 += 32) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (k0 + lane < P) ml = *reinterpret_cast<const float2*>(pv.piece_ml + 2 * (at + (long long)(k0 + lane) * rows));
        const Exp2Pair e(ml.x - mu);
        const float a = e.both(), la = e.of(ml.y);
#pragma unroll 4
        for (int k = 0; k < min(32, P - k0); k++) {
          const float ak = __shfl_sync(0xffffffffu, a, k);
          const float* o = pv.piece_o + (at + (long long)(k0 + k) * rows) * D;
#pragma unroll
          for (int i = 0; i < PER; i++) acc[i] = fmaf(o[lane + 32 * i], ak, acc[i]);
          Ls += __shfl_sync(0xffffffffu, la, k);
        }
      }
      const float inv = Ls == 0.f ? 0.f : 1.f / Ls;  // no visible key: zeros
      const int j = (int)c.gdiv.div((uint32_t)r), jj = r - j * c.group;
      uint16_t* dst = c.out + (long long)(tok + j) * c.out_stride + (long long)(h * c.group + jj) * D;
#pragma unroll
      for (int i = 0; i < PER; i++)
        dst[lane + 32 * i] = (uint16_t)(pack_bf16x2_rn(acc[i] * inv, 0.f) & 0xffffu);
    }
    base += total;
  }
}

template <int D, bool PIECES>
__global__ void __launch_bounds__(1024) merge_fp8_kernel(Fp8MergeParams prm) {
  const Common& c = prm.c;
  const PlanView& pv = prm.pv;
  extern __shared__ __align__(16) float spart[];  // [cols][lanes][D + 2]
  pdl_trigger();
  pdl_wait();
  constexpr int PER = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pl = warp / prm.cols;
  const int n_dseq = pv.plan[0];
  const int seg = blockIdx.x / prm.parts;
  const int lcol = warp - pl * prm.cols, col = ((int)blockIdx.x - seg * prm.parts) * prm.cols + lcol;
  if constexpr (PIECES) {  // every CTA's warps take rows in turn, before its segment
    const int warps = blockDim.x >> 5;
    const long long first = (long long)blockIdx.x * warps + warp;
    if (first < kPieceRows) merge_prefill_pieces<D>(c, pv, (int)first, (int)min((long long)gridDim.x * warps, 1ll << 30));
  }
  if (seg >= n_dseq * c.hkv) return;
  const int i = seg / c.hkv, h = seg - i * c.hkv;
  const int4 di = pv.dseq[i];  // (sequence, seq_len, first query token, q_len)
  const int ql = di.w;
  const int npos = ((di.y + 15) / 16 - first_block(c, di.y, ql) + c.np - 1) / c.np;
  const int grp = h / c.hg, hl = h - grp * c.hg;
  const int gpl = c.ng / c.nl, lane_g = grp % c.nl, gs = grp / c.nl;
  const long long Tu = pv.dprefix[n_dseq] * gpl;
  const long long sbeg = pv.dprefix[i] * gpl + (long long)gs * npos, send = sbeg + npos;
  const int W = prm.num_ctas / c.nl;  // the lane's CTAs
  auto wstart = [&](long long w) { return div_nn(Tu * w, W); };
  // pieces: the direct slot (the piece that starts the segment), then every
  // CTA whose range is not empty and starts strictly inside the segment;
  // candidates are those CTAs or the positions, whichever are fewer
  long long w_first = 0, cand = 0;
  bool by_cta = true;
  if (npos > 0) {
    w_first = div_nn((sbeg + 1) * W + Tu - 1, Tu);
    const long long w_end = div_nn(send * W + Tu - 1, Tu);
    by_cta = w_end - w_first <= npos - 1;
    cand = 1 + (by_cta ? w_end - w_first : (long long)npos - 1);
  }
  const int nsub = c.np == 2 ? 2 : 1;  // paired blocks: columns col and col + dcols hold the same query
  const bool used = col < ql * c.group;
  float acc[PER];
#pragma unroll
  for (int k = 0; k < PER; k++) acc[k] = 0.f;
  float M = -INFINITY, Ls = 0.f;
  auto merge = [&](float m, float l, const float (&o)[PER]) {
    const float mn = fmaxf(M, m);
    const float mu = mn == -INFINITY ? 0.f : mn;
    const Exp2Pair ea(M - mu), eb(m - mu);
    const float a = ea.both(), b = eb.both();
#pragma unroll
    for (int k = 0; k < PER; k++) acc[k] = acc[k] * a + o[k] * b;
    Ls = ea.of(Ls) + eb.of(l);
    M = mn;
  };
  if (used) {
    // a candidate's two column sets are loaded together; the lanes of a column
    // keep their candidates' loads in flight side by side
#pragma unroll 2
    for (long long k = pl; k < cand; k += prm.lanes) {
      bool ok = true;
      long long w = 0;
      if (k > 0) {
        if (by_cta) {
          w = w_first + k - 1;
          ok = wstart(w + 1) > wstart(w);
        } else {
          const long long p = sbeg + k;
          w = div_nn((p + 1) * W + Tu - 1, Tu) - 1;  // last CTA starting at or before p
          ok = wstart(w) == p;
        }
      }
      const long long sl = (w * c.nl + lane_g) * c.hg + hl;
      const float* o = k > 0 ? pv.warp_o + sl * prm.slot * D : pv.direct_o + (long long)seg * prm.slot * D;
      const float* ml = k > 0 ? pv.warp_ml + sl * prm.slot * 2 : pv.direct_ml + (long long)seg * prm.slot * 2;
      float mw[2], lw[2], ov[2][PER];
#pragma unroll
      for (int sub = 0; sub < 2; sub++) {
        const bool use = ok && sub < nsub;
        const int cc = col + sub * c.dcols;
        mw[sub] = use ? ml[cc * 2] : -INFINITY;
        lw[sub] = use ? ml[cc * 2 + 1] : 0.f;
#pragma unroll
        for (int e = 0; e < PER; e++) ov[sub][e] = use ? o[cc * D + lane + 32 * e] : 0.f;
      }
#pragma unroll
      for (int sub = 0; sub < 2; sub++) merge(mw[sub], lw[sub], ov[sub]);
    }
  }
  if (prm.lanes > 1) {
    float* mine = spart + (lcol * prm.lanes + pl) * (D + 2);
    if (pl > 0) {
#pragma unroll
      for (int k = 0; k < PER; k++) mine[lane + 32 * k] = acc[k];
      if (lane == 0) {
        mine[D] = M;
        mine[D + 1] = Ls;
      }
    }
    __syncthreads();
    if (pl > 0) return;
#pragma unroll 1
    for (int p = 1; p < prm.lanes; p++) {
      const float* o = mine + p * (D + 2);
      float v[PER];
#pragma unroll
      for (int k = 0; k < PER; k++) v[k] = o[lane + 32 * k];
      merge(o[D], o[D + 1], v);
    }
  }
  if (!used) return;
  const float inv = Ls == 0.f ? 0.f : 1.f / Ls;  // no visible key: zeros
  const int j = col / c.group, jj = col - j * c.group;
  uint16_t* dst = c.out + (long long)(di.z + j) * c.out_stride + (long long)(h * c.group + jj) * D;
#pragma unroll
  for (int k = 0; k < PER; k++)
    dst[lane + 32 * k] = (uint16_t)(pack_bf16x2_rn(acc[k] * inv, 0.f) & 0xffffu);
}
