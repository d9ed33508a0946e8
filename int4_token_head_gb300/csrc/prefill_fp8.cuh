// Prefill over the FP8 cache on warp-level MMAs, included by attention_fp8.cu,
// for queries that no tensor map holds (token rows that overlap: one row for
// all tokens, say; 8 prompts of 512 to 2048 tokens, 32/8 heads of 256: 897 us, on
// the tensor cores 325):
// 64 query rows (query token x q head of one kv group) per item, 16 per warp,
// 32 keys (two cache blocks) per step.  Codes are staged as they are (cp.async,
// three stages) and become f16 B fragments in registers: for S, a lane's four
// consecutive codes of a key are one k-step's four elements (Q' is stored with
// the same permutation within each 16 dimensions); for O, ldmatrix.trans of
// byte pairs, whose even and odd dimensions are two n-tiles.
template <int D>
struct Fp8Pre {
  static constexpr int WARPS = 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROWS = kPrefillRows;
  static constexpr int NB = 2;         // cache blocks per step
  static constexpr int KEYS = 16 * NB;
  static constexpr int STAGES = 3;
  static constexpr int ROW = D + 16;   // code row stride: an odd number of 16-byte units
  static constexpr int TILE = KEYS * ROW;
  static constexpr int STAGE = 2 * TILE + 32;  // K rows, V rows, scales [K/V][NB], block flags [NB]
  static constexpr int QSTRIDE = D + 8;        // halves per Q' row
  static constexpr int SMEM = STAGES * STAGE + ROWS * QSTRIDE * 2 + 32;  // and the item
};

template <int D>
__global__ void __launch_bounds__(Fp8Pre<D>::THREADS) prefill_fp8_kernel(Common c, PlanView pv) {
  using G = Fp8Pre<D>;
  constexpr int NT = D / 8;  // n-tiles of the output
  extern __shared__ __align__(16) uint8_t smem[];
  __half* sQ = reinterpret_cast<__half*>(smem + G::STAGES * G::STAGE);
  int* sitem = reinterpret_cast<int*>(sQ + G::ROWS * G::QSTRIDE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, cq = lane & 3;
  pdl_wait();
  pdl_trigger();  // after the wait: the decode beside this kernel looks for the schedule
  const int n_items = pv.plan[1];

#pragma unroll 1
  while (true) {
    if (tid == 0) {
      const PrefillItem it = prefill_piece_item(c, pv, atomicAdd(&pv.plan[2], 1), n_items);
      sitem[0] = it.seq; sitem[1] = it.h; sitem[2] = it.tile;
      sitem[3] = it.kb0; sitem[4] = it.nkb; sitem[5] = it.row;
    }
    __syncthreads();
    const PrefillItem item{sitem[0], sitem[1], sitem[2], sitem[3], sitem[4], sitem[5]};
    __syncthreads();
    if (item.seq < 0) break;
    const int seq = item.seq, h = item.h, tile = item.tile, kb0 = item.kb0, nkb = item.nkb;
    const int q0 = c.qsl[seq], ql = c.qsl[seq + 1] - q0;
    const int L = c.seq_lens[seq], ctx = L - ql;
    const int tok0 = tile * c.tile_tokens;
    const int nrows = min(c.tile_tokens, ql - tok0) * c.group;
    const int nsteps = (nkb - kb0 + G::NB - 1) / G::NB;

    auto issue = [&](int st, int stage) {
      uint8_t* sb = smem + stage * G::STAGE;
      float* ssc = reinterpret_cast<float*>(sb + 2 * G::TILE);
      int* sfl = reinterpret_cast<int*>(ssc + 2 * G::NB);
#pragma unroll
      for (int b = 0; b < G::NB; b++) {
        const int kb = kb0 + st * G::NB + b;
        const int blk = kb < nkb ? c.block_table[(long long)seq * c.max_blocks + kb] : -1;
        const bool ok = blk >= 0 && blk < c.num_blocks;
        const int rows = ok ? L - kb * 16 : 0;
        const long long base = ok ? (long long)blk * c.geo.cblk + (long long)h * D : 0;
        // rows behind the sequence and unusable blocks are zeros: a NaN code
        // would survive its zero weight
        for (int q = tid; q < 2 * D; q += G::THREADS) {
          const int kv = q >= D, qq = q - kv * D;
          const int r = qq / (D / 16), col = qq - r * (D / 16);
          const bool in = r < rows;
          const uint8_t* src = (kv ? c.v_cache : c.k_cache) + (in ? base + r * c.geo.crow + col * 16 : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                           smem_addr(sb + kv * G::TILE + (b * 16 + r) * G::ROW + col * 16)),
                       "l"(src), "r"(in ? 16 : 0));
        }
        if (tid < 2) {
          const float* src = (tid ? c.v_scale : c.k_scale) + (ok ? (long long)blk * c.hkv + h : 0);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_addr(ssc + tid * G::NB + b)),
                       "l"(src), "r"(ok ? 4 : 0));
        }
        if (tid == 0) {
          sfl[b] = ok;
          if (kb < nkb && !ok) flag(c.status, KV_INT4_DEV_BAD_BLOCK);
        }
      }
    };
    for (int s = 0; s < G::STAGES - 1; s++) {
      if (s < nsteps) issue(s, s);
      cp_async_commit();
    }

    // Q' rows of this warp: divided by their power of two, f16, stored so that
    // k = 2 cq, 2 cq + 1 of k-step s are dimensions 16 s + 4 cq, + 1 and
    // k = 2 cq + 8, + 9 are + 2, + 3
    const int r0 = warp * 16 + g, r1 = r0 + 8;
    float cf0 = 0.f, cf1 = 0.f;
#pragma unroll 1
    for (int rr = 0; rr < 16; rr++) {
      const int r = warp * 16 + rr;
      const int j = (int)c.gdiv.div((uint32_t)r), jj = r - j * c.group;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          c.q + (long long)(q0 + tok0 + j) * c.q_stride + (long long)(h * c.group + jj) * D);
      constexpr int PW = (D / 2 + 31) / 32;  // words per lane
      uint32_t w[PW], am = 0;
#pragma unroll
      for (int i = 0; i < PW; i++) {
        const int p = lane + 32 * i;
        w[i] = r < nrows && p < D / 2 ? src[p] : 0u;
        am = __vmaxu2(am, w[i] & 0x7fff7fffu);
      }
      am = __reduce_max_sync(0xffffffffu, max(am & 0xffffu, am >> 16));
      const int e = q_exponent(am);
      const float mul = exp2_int(-e), cf = c.qscale * exp2_int(e);
#pragma unroll
      for (int i = 0; i < PW; i++) {
        const int p = lane + 32 * i, s = p >> 3, pp = p & 7;
        if (p < D / 2)
          reinterpret_cast<uint32_t*>(sQ + r * G::QSTRIDE)[8 * s + (pp >> 1) + 4 * (pp & 1)] =
              pack_f16x2(bf16lo_to_f32(w[i]) * mul, bf16hi_to_f32(w[i]) * mul);
      }
      if (r == r0) cf0 = cf;
      if (r == r1) cf1 = cf;
    }
    __syncwarp();

    float oacc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; t++) oacc[t][0] = oacc[t][1] = oacc[t][2] = oacc[t][3] = 0.f;
    float mr0 = -INFINITY, mr1 = -INFINITY, lr0 = 0.f, lr1 = 0.f;
    const int qp0 = ctx + tok0 + (r0 < nrows ? (int)c.gdiv.div((uint32_t)r0) : 0);
    const int qp1 = ctx + tok0 + (r1 < nrows ? (int)c.gdiv.div((uint32_t)r1) : 0);
    const int lim0 = c.causal ? min(L, qp0 + 1) : L, lim1 = c.causal ? min(L, qp1 + 1) : L;
    const int lo0 = window_lo(c, qp0), lo1 = window_lo(c, qp1);

#pragma unroll 1
    for (int st = 0; st < nsteps; st++) {
      if (st + G::STAGES - 1 < nsteps) issue(st + G::STAGES - 1, (st + G::STAGES - 1) % G::STAGES);
      cp_async_commit();
      cp_async_wait<G::STAGES - 1>();
      __syncthreads();
      const uint8_t* sb = smem + (st % G::STAGES) * G::STAGE;
      const float* ssc = reinterpret_cast<const float*>(sb + 2 * G::TILE);
      const int* sfl = reinterpret_cast<const int*>(ssc + 2 * G::NB);

      // S = Q' K^T: 16 rows x 32 keys per warp, n-tile n = keys 8 n .. 8 n + 7
      float sacc[2 * G::NB][4];
#pragma unroll
      for (int n = 0; n < 2 * G::NB; n++) sacc[n][0] = sacc[n][1] = sacc[n][2] = sacc[n][3] = 0.f;
#pragma unroll
      for (int s = 0; s < D / 16; s++) {
        uint32_t a[4];
        const int mi = lane >> 3, rr = lane & 7;
        ldmatrix_x4(a, sQ + (warp * 16 + (mi & 1) * 8 + rr) * G::QSTRIDE + 16 * s + (mi >> 1) * 8);
#pragma unroll
        for (int n = 0; n < 2 * G::NB; n++) {
          uint32_t b0, b1;
          e4m3x4_to_f16x2(*reinterpret_cast<const uint32_t*>(sb + (8 * n + g) * G::ROW + 16 * s + 4 * cq), b0, b1);
          mma_16816(sacc[n], a, b0, b1);
        }
      }
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2 * G::NB; n++) {
        const int b = n >> 1;
        const float ks = ssc[b], kvf = (float)exp_of(ssc[G::NB + b]);
        const bool bok = sfl[b] != 0;
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const int pos = (kb0 + st * G::NB) * 16 + 8 * n + 2 * cq + e;
          sacc[n][e] = (bok && pos < lim0 && pos >= lo0) ? fmaf(sacc[n][e], cf0 * ks, kvf) : -INFINITY;
          sacc[n][2 + e] = (bok && pos < lim1 && pos >= lo1) ? fmaf(sacc[n][2 + e], cf1 * ks, kvf) : -INFINITY;
          mx0 = fmaxf(mx0, sacc[n][e]);
          mx1 = fmaxf(mx1, sacc[n][2 + e]);
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
      }
      const float mn0 = fmaxf(mr0, mx0), mn1 = fmaxf(mr1, mx1);
      const float mu0 = mn0 == -INFINITY ? 0.f : mn0, mu1 = mn1 == -INFINITY ? 0.f : mn1;
      const Exp2Pair e0(mr0 - mu0), e1(mr1 - mu1);
      const float al0 = e0.both(), al1 = e1.both();
      mr0 = mn0;
      mr1 = mn1;
      lr0 = e0.of(lr0);
      lr1 = e1.of(lr1);
      uint32_t pa[G::NB][4];  // A fragments of W, one k-step of 16 keys per block
#pragma unroll
      for (int b = 0; b < G::NB; b++) {
        float ivs = __uint_as_float((254u << 23) - (__float_as_uint(ssc[G::NB + b]) & 0x7f800000u));
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int hn = 0; hn < 2; hn++) {
          const float* t = sacc[2 * b + hn];
          const float w0 = fast_exp2(t[0] - mu0), w1 = fast_exp2(t[1] - mu0);
          const float w2 = fast_exp2(t[2] - mu1), w3 = fast_exp2(t[3] - mu1);
          s0 += w0 + w1;
          s1 += w2 + w3;
          pa[b][2 * hn] = pack_f16x2(w0, w1);
          pa[b][2 * hn + 1] = pack_f16x2(w2, w3);
        }
        if (ssc[G::NB + b] < exp2_int(kFp8LowExp)) {
          const float up = (float)(kFp8LowExp - exp_of(ssc[G::NB + b]));
          s0 = s1 = 0.f;
#pragma unroll
          for (int hn = 0; hn < 2; hn++) {
            const float* t = sacc[2 * b + hn];
            s0 += fast_exp2(t[0] - mu0 + up) + fast_exp2(t[1] - mu0 + up);
            s1 += fast_exp2(t[2] - mu1 + up) + fast_exp2(t[3] - mu1 + up);
          }
          ivs = exp2_int(-kFp8LowExp);
        }
        lr0 = fmaf(s0, ivs, lr0);
        lr1 = fmaf(s1, ivs, lr1);
      }
#pragma unroll
      for (int t = 0; t < NT; t++) {
        oacc[t][0] *= al0; oacc[t][1] *= al0; oacc[t][2] *= al1; oacc[t][3] *= al1;
      }
#pragma unroll
      for (int b = 0; b < G::NB; b++) {
        const uint8_t* vt = sb + G::TILE + (b * 16 + ((lane >> 3) & 1) * 8 + (lane & 7)) * G::ROW + (lane >> 4) * 16;
#pragma unroll
        for (int p = 0; p < D / 32; p++) {
          uint32_t r[4];
          ldmatrix_x4_trans(r, vt + 32 * p);
#pragma unroll
          for (int q = 0; q < 2; q++) {
            uint32_t e0, o0, e1, o1;  // even and odd dimensions, keys 0-7 and 8-15
            e4m3x4_to_f16x2(__byte_perm(r[2 * q], 0, 0x3120), e0, o0);
            e4m3x4_to_f16x2(__byte_perm(r[2 * q + 1], 0, 0x3120), e1, o1);
            mma_16816(oacc[2 * (2 * p + q)], pa[b], e0, e1);
            mma_16816(oacc[2 * (2 * p + q) + 1], pa[b], o0, o1);
          }
        }
      }
      __syncthreads();  // every warp is done with this stage
    }
    cp_async_wait<0>();

#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      lr0 += __shfl_xor_sync(0xffffffffu, lr0, o);
      lr1 += __shfl_xor_sync(0xffffffffu, lr1, o);
    }
    if (item.row >= 0) {
      // a piece: O, the running maximum and the sum
      auto store_piece = [&](int r, int e, float m, float l) {
        if (r >= nrows) return;
        const long long at = item.row + r;
#pragma unroll
        for (int ch = 0; ch < D / 16; ch++)
          *reinterpret_cast<float4*>(pv.piece_o + at * D + 16 * ch + 4 * cq) =
              make_float4(oacc[2 * ch][e], oacc[2 * ch + 1][e], oacc[2 * ch][e + 1], oacc[2 * ch + 1][e + 1]);
        if (cq == 0) *reinterpret_cast<float2*>(pv.piece_ml + 2 * at) = make_float2(m, l);
      };
      store_piece(r0, 0, mr0, lr0);
      store_piece(r1, 2, mr1, lr1);
      __syncthreads();  // the next item overwrites the stages
      continue;
    }
    const float inv0 = lr0 == 0.f ? 0.f : 1.f / lr0, inv1 = lr1 == 0.f ? 0.f : 1.f / lr1;
    // dimensions 16 ch + 4 cq .. + 3: even ones in tile 2 ch, odd ones in 2 ch + 1
    auto store = [&](int r, int e, float inv) {
      if (r >= nrows) return;
      const int j = (int)c.gdiv.div((uint32_t)r), jj = r - j * c.group;
      uint16_t* dst = c.out + (long long)(q0 + tok0 + j) * c.out_stride + (long long)(h * c.group + jj) * D;
#pragma unroll
      for (int ch = 0; ch < D / 16; ch++)
        *reinterpret_cast<uint2*>(dst + 16 * ch + 4 * cq) =
            make_uint2(pack_bf16x2_rn(oacc[2 * ch][e] * inv, oacc[2 * ch + 1][e] * inv),
                       pack_bf16x2_rn(oacc[2 * ch][e + 1] * inv, oacc[2 * ch + 1][e + 1] * inv));
    };
    store(r0, 0, inv0);
    store(r1, 2, inv1);
    __syncthreads();  // the next item overwrites the stages
  }
}
