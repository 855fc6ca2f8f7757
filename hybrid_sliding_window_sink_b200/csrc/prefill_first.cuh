// prefill_first.cuh - sm_100a prefill of an SWA layer with window W <= 129, 8 query heads per KV head,
// and the first n_first <= 16 tokens kept visible behind the window.
//
// Row i sees J_i = [lo, i] and [0, min(n_first, lo)), lo = max(0, i - W + 1); the rest of the math, the row blocks, the
// K/V ring, the roles and the precision are those of prefill_swa.cuh (its ring, chunked prefill and
// waits are described there). What differs:
//   * The first tokens sit in one more unit behind the ring, loaded once per (sequence, KV head) run:
//     S has 192 columns, P lies in [0, 96). A key below a row's window counts through that unit, one
//     inside it through the ring, so none counts twice.
//   * The softmax finds its reference on the way (one pass, one slot block per turn).
//   * PV multiplies the window's nine units and the first tokens', not the two slots that may be
//     taking rows of later keys.
//   * Angles: a block's table from one angle per thread, a run's start from one per lane and unit. The
//     first run's units are loaded, converted and rotated by the softmax warps, one each (n = 203, 8/1
//     heads: 15.2 -> 11.8 us with the next).
//   * K has no barrier of its own (Q of a block is handed over after the block's K and V), and a group
//     hands over by one arrival per warp: a thousand arrivals at a run's start, and the nine polls of
//     the issuer, took 2000 cycles.
//   * Every tile masks keys, so in a V row that holds a NaN or an infinity the 16 bytes around it become
//     zeros and its K row a NaN as it enters (see v_row_not_finite in prefill.cuh).
// Bound: bytes at n = 32768 (1.51 GB, 231 us at the measured copy rate); measured 390 us cold, 445 us under
// the power cap (the kernel without first tokens 448 and 500). A trace puts the RoPE group and the two
// softmax groups level at 6200 - 6500 cycles per row block, against 4000 at the byte floor.
#pragma once

#include "ptx.cuh"
#include "prefill_swa.cuh"

namespace mimo {

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

constexpr int kSwaFirst = 16;       // most first tokens (one unit)

struct SwaFirstLayout {
  static constexpr int UNITS = kSwaUnits + 1;          // the ring, and the first tokens
  static constexpr int N = 16 * UNITS;                 // S columns: all units, in slot order
  static constexpr int Q_CHUNK = 128 * 128;
  static constexpr int Q_STAGE = 3 * Q_CHUNK;
  static constexpr int R_CHUNK = N * 128;              // 192 rows x 64 dims
  static constexpr int UNIT_BYTES = 16 * 128;          // one unit inside one 64-dim chunk
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * Q_STAGE;
  static constexpr int OFF_V = OFF_K + 3 * R_CHUNK;
  static constexpr int OFF_TAB = OFF_V + 2 * R_CHUNK;
  static constexpr int TAB_BYTES = kSwaP * 32 * 8;     // 16 positions x 32 frequencies x (cos, sin)
  static constexpr int OFF_MISC = OFF_TAB + 2 * TAB_BYTES;
  static constexpr int MISC_BYTES = 512 + 32 * 8;
  static constexpr int SMEM = OFF_MISC + MISC_BYTES + 1024;
  static constexpr uint32_t IDESC_PV = idesc_f16kind(128, 128, 0, 1, 1);   // P and V in f16
  static constexpr uint32_t IDESC_S = idesc_bf16(128, N, 0, 0);
  static constexpr uint32_t IDESC_S_F16 = idesc_f16kind(128, N, 0, 0, 1);   // rotated dims
  static_assert(R_CHUNK % 1024 == 0, "ring chunks stay on swizzle atoms");
  static_assert(SMEM <= 232448, "shared memory budget");
};

// Barriers beyond those of prefill_swa.cuh.
enum : int {
  kSwFirstFull = kSwNumBars,        // the first tokens' unit: landed, free again
  kSwFirstFree,
  kSwTurn,                          // the turns of a run's start are in the spare table (4 arrivals)
  kSwStart,                         // the softmax warps have the first run's first eight units ready (8)
  kSfNumBars
};

__global__ void __launch_bounds__(kSwaThreads, 1)
    prefill_swa_first_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                             const __grid_constant__ CUtensorMap tmV, const PrefillFirstParams p) {
  using L = SwaFirstLayout;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sQ = sbase + L::OFF_Q;
  const uint32_t sK = sbase + L::OFF_K;
  const uint32_t sV = sbase + L::OFF_V;
  const uint32_t sBar = sbase + L::OFF_MISC;
  auto bar = [&](int i) -> uint32_t { return sBar + 8u * static_cast<uint32_t>(i); };
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::OFF_MISC + 8 * kSfNumBars);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC + 8 * kSfNumBars + 4);
  double* s_invf = reinterpret_cast<double*>(smem + L::OFF_MISC + 512);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned* err = p.err;
  const int half = p.rot_dims >> 1;   // <= 32

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSfNumBars; ++i) {
      // one arrival per warp (of four) where a group hands something over; K needs no barrier of its
      // own here: Q of a block is handed over after the block's K and V
      const bool group = (i >= kSwQReady && i < kSwQReady + 2) || (i >= kSwPReady && i < kSwPReady + 2) ||
                         (i >= kSwTmFree && i < kSwTmFree + 2) || (i >= kSwTab && i < kSwTab + 2) || i == kSwTurn;
      mbar_init(bar(i), i == kSwStart ? 8u : group ? 4u : 1u);
    }
    *s_abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  if (warp >= 2 && warp < 6 && threadIdx.x - 64 < half)
    s_invf[threadIdx.x - 64] = inv_freq(p, threadIdx.x - 64);
  // the ring starts zeroed: slots outside a window are read (masked) before they are filled
  for (int o = threadIdx.x * 16; o < 3 * L::R_CHUNK + 2 * L::R_CHUNK; o += kSwaThreads * 16)
    *reinterpret_cast<uint4*>(smem + L::OFF_K + o) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;

  // this CTA's contiguous run [f0, f1) of the flattened (b, g, block) order
  const long long F = static_cast<long long>(p.num_work);
  const long long f0 = F * blockIdx.x / gridDim.x;
  const long long f1 = F * (blockIdx.x + 1) / gridDim.x;
  const int nqt = p.n_qtiles;

  // the first run's eight units before its block, one by each of the eight softmax warps (idle until
  // the first product): forty copies issued by the producer alone held it for 7000 cycles
  if (warp >= 6 && lane == 0) {
    const int bg = static_cast<int>(f0 / nqt), b = bg / p.Hkv, g = bg - b * p.Hkv;
    const int slot = warp - 6, u = static_cast<int>(f0 % nqt) + (p.q_off >> 4) - 8 + slot;
    mbar_arrive_expect_tx(bar(kSwKVFull + slot), 16 * (kDQK + kDV) * 2);
    for (int c = 0; c < 3; ++c)
      tma_load_4d(sK + c * L::R_CHUNK + slot * L::UNIT_BYTES, &tmK, bar(kSwKVFull + slot), 64 * c, g, 16 * u, b);
    for (int c = 0; c < 2; ++c)
      tma_load_4d(sV + c * L::R_CHUNK + slot * L::UNIT_BYTES, &tmV, bar(kSwKVFull + slot), 64 * c, g, 16 * u, b);
  }
  auto arrive_warp = [&](uint32_t b_) {       // everything this warp wrote before
    __syncwarp();
    if (lane == 0) mbar_arrive(b_);
  };
  // V, sixteen bytes of each half of row x / 8 of a unit (slot) of the ring: bf16 -> f16 in place; sixteen
  // bytes with a value that is not finite become zeros, and dim 64 of the key's K row a NaN (the rotated dims
  // are below it)
  auto v_part = [&](int slot, int x) {
    uint8_t* vb = smem + L::OFF_V + slot * L::UNIT_BYTES;
    uint4 xv[2];
#pragma unroll
    for (int h2 = 0; h2 < 2; ++h2)
      xv[h2] = *reinterpret_cast<const uint4*>(vb + h2 * L::R_CHUNK + x * 16);
    bool bad = false;
    const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
#pragma unroll
    for (int h2 = 0; h2 < 2; ++h2) {
      const uint32_t w[4] = {xv[h2].x, xv[h2].y, xv[h2].z, xv[h2].w};
      __nv_bfloat162 acc = zero;                     // 0, or a NaN (see v_row_not_finite)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]), zero, acc);
      if (!__hbeq2(acc, zero)) {
        xv[h2] = make_uint4(0u, 0u, 0u, 0u);
        bad = true;
      }
    }
    const int row = x >> 3;
    if (bad)
      *reinterpret_cast<uint16_t*>(smem + L::OFF_K + L::R_CHUNK + slot * L::UNIT_BYTES + row * 128 + ((row & 7) << 4)) = kNan16;
#pragma unroll
    for (int h2 = 0; h2 < 2; ++h2)
      *reinterpret_cast<uint4*>(vb + h2 * L::R_CHUNK + x * 16) =
          make_uint4(bf16x2_to_f16x2(xv[h2].x), bf16x2_to_f16x2(xv[h2].y),
                     bf16x2_to_f16x2(xv[h2].z), bf16x2_to_f16x2(xv[h2].w));
  };
  // K row x / 4 of a unit, 16-byte units x % 4 and that + 4: rotated (or, stored rotated, made f16). The
  // angles of the unit's first position lie across the warp (bc, bs: frequency = lane) and are turned by
  // the row's (see `turn`).
  auto k_part = [&](int slot, int x, int kpos0, float bc, float bs, const float* turns) {
    const int row = x >> 2, u = x & 3, kpos = kpos0 + row, ring_row = slot * 16 + row;
    const float4* t4 = reinterpret_cast<const float4*>(turns + row * 64);
    const bool raw = kpos >= p.krot_from && kpos < p.nk, cooked = kpos >= 0 && kpos < p.krot_from;
    uint4* px = reinterpret_cast<uint4*>(smem + L::OFF_K + ring_row * 128 + ((u ^ (row & 7)) << 4));
    uint4* py = reinterpret_cast<uint4*>(smem + L::OFF_K + ring_row * 128 + (((u + 4) ^ (row & 7)) << 4));
    const uint4 xv = *px, yv = *py;
    uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, ys[4] = {yv.x, yv.y, yv.z, yv.w};
#pragma unroll
    for (int e2 = 0; e2 < 4; ++e2) {
      const int k = u * 8 + 2 * e2;
      const float4 t = t4[u * 4 + e2];
      const float c0 = __shfl_sync(0xffffffffu, bc, k), s0 = __shfl_sync(0xffffffffu, bs, k);
      const float c1 = __shfl_sync(0xffffffffu, bc, k + 1), s1 = __shfl_sync(0xffffffffu, bs, k + 1);
      if (raw) {
        rot_pair(xs[e2], ys[e2], make_float4(c0 * t.x - s0 * t.z, c1 * t.y - s1 * t.w,
                                             s0 * t.x + c0 * t.z, s1 * t.y + c1 * t.w));
      } else if (cooked) {
        xs[e2] = bf16x2_to_f16x2(xs[e2]);
        ys[e2] = bf16x2_to_f16x2(ys[e2]);
      }
    }
    if (raw || cooked) {
      *px = make_uint4(xs[0], xs[1], xs[2], xs[3]);
      *py = make_uint4(ys[0], ys[1], ys[2], ys[3]);
    }
  };
  auto angle = [&](int pos, float& sn, float& cs) {   // of frequency `lane`
    const double ang = static_cast<double>(pos) * s_invf[lane];
    const double nrev = rint(ang * 0.15915494309189535);
    __sincosf(static_cast<float>(fma(-nrev, 6.283185307179586, ang)), &sn, &cs);
  };
  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int seq = 8, nq = 0, nfirst = 0;   // (the softmax warps brought the first eight units)
      bool ok = true;
      auto load_unit = [&](int b, int g, int u) -> bool {
        const int slot = seq % kSwaUnits;
        if (seq >= kSwaUnits &&
            !mbar_wait(bar(kSwSlotFree + slot), ((seq / kSwaUnits) - 1) & 1, s_abort, err))
          return false;
        mbar_arrive_expect_tx(bar(kSwKVFull + slot), 16 * (kDQK + kDV) * 2);
        for (int c = 0; c < 3; ++c)
          tma_load_4d(sK + c * L::R_CHUNK + slot * L::UNIT_BYTES, &tmK, bar(kSwKVFull + slot),
                      64 * c, g, 16 * u, b);
        for (int c = 0; c < 2; ++c)
          tma_load_4d(sV + c * L::R_CHUNK + slot * L::UNIT_BYTES, &tmV, bar(kSwKVFull + slot),
                      64 * c, g, 16 * u, b);
        ++seq;
        return true;
      };
      for (long long f = f0; f < f1 && ok; ++f) {
        const int bg = static_cast<int>(f / nqt), t = static_cast<int>(f % nqt);
        const int b = bg / p.Hkv, g = bg - b * p.Hkv;
        const int ua = t + (p.q_off >> 4);   // K/V unit holding the block's own positions
        if (f != f0 && t == 0)
          for (int u = ua - 8; u < ua && ok; ++u) ok = load_unit(b, g, u);
        if (!ok) break;
        const int st = nq & 1;
        if (nq >= 2 && !mbar_wait(bar(kSwQEmpty + st), ((nq >> 1) - 1) & 1, s_abort, err)) { ok = false; break; }
        mbar_arrive_expect_tx(bar(kSwQFull + st), L::Q_STAGE);
        for (int c = 0; c < 3; ++c)
          tma_load_4d(sQ + st * L::Q_STAGE + c * L::Q_CHUNK, &tmQ, bar(kSwQFull + st), 64 * c,
                      g * kSwaG, t * kSwaP, b);
        SWA_TRACE(nq, 9);
        ++nq;
        ok = load_unit(b, g, ua);
        if (ok && (f == f0 || t == 0)) {   // keys 0 .. 15 of this sequence and KV head
          if (nfirst > 0) ok = mbar_wait(bar(kSwFirstFree), (nfirst - 1) & 1, s_abort, err);
          if (ok) {
            mbar_arrive_expect_tx(bar(kSwFirstFull), 16 * (kDQK + kDV) * 2);
            for (int c = 0; c < 3; ++c)
              tma_load_4d(sK + c * L::R_CHUNK + kSwaUnits * L::UNIT_BYTES, &tmK, bar(kSwFirstFull), 64 * c, g, 0, b);
            for (int c = 0; c < 2; ++c)
              tma_load_4d(sV + c * L::R_CHUNK + kSwaUnits * L::UNIT_BYTES, &tmV, bar(kSwFirstFull), 64 * c, g, 0, b);
            ++nfirst;
          }
        }
      }
      // let every issued copy land before the CTA can exit (in any case: a wait that gives up elsewhere
      // leaves none behind)
      for (int s = seq - kSwaUnits < 0 ? 0 : seq - kSwaUnits; s < seq; ++s)
        mbar_wait_drain(bar(kSwKVFull + s % kSwaUnits), (s / kSwaUnits) & 1, err);
      for (int i = nq - 2 < 0 ? 0 : nq - 2; i < nq; ++i)
        mbar_wait_drain(bar(kSwQFull + (i & 1)), (i >> 1) & 1, err);
      if (nfirst > 0) mbar_wait_drain(bar(kSwFirstFull), (nfirst - 1) & 1, err);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const int ntiles = static_cast<int>(f1 - f0);
      int ns = 0, npv = 0, seq = 0;
      int useq_of[4] = {0, 0, 0, 0};
      bool last_of[4] = {false, false, false, false};
      int s_useq = 0;
      bool s_last = false, s_q = false, s_free = false, ok = true;
      bool s_start = false;                    // the softmax warps' units of the first run are ready
      auto prep_s = [&]() {
        const long long f = f0 + ns;
        const int t = static_cast<int>(f % nqt);
        const bool first = (ns == 0 || t == 0);
        s_last = (f == f1 - 1 || t == nqt - 1);
        if (first) seq += 8;
        s_useq = seq++;
        s_q = false;
        s_free = ns < 2;
      };
      if (ntiles > 0) prep_s();
      unsigned long long t_prog = globaltimer_ns();
      uint32_t idle = 0;
      while (npv < ntiles && ok) {
        bool prog = false;
        if (ns < ntiles) {
          const int wg = ns & 1;
          if (!s_q) s_q = mbar_test(bar(kSwQReady + wg), (ns >> 1) & 1);
          if (!s_free) s_free = mbar_test(bar(kSwTmFree + wg), ((ns >> 1) - 1) & 1);
          if (!s_start) s_start = mbar_test(bar(kSwStart), 0);
          if (s_q && s_free && s_start) {
            SWA_TRACE(ns, 17);
            tc_fence_after();
            const uint32_t d = tmem + wg * 256;
#pragma unroll
            for (int kk = 0; kk < 12; ++kk) {
              const uint64_t a =
                  smem_desc(sQ + wg * L::Q_STAGE + (kk >> 2) * L::Q_CHUNK + (kk & 3) * 32, 16, 1024);
              const uint64_t bd = smem_desc(sK + (kk >> 2) * L::R_CHUNK + (kk & 3) * 32, 16, 1024);
              umma_ss(d, a, bd, kk * 16 < p.rot_dims ? L::IDESC_S_F16 : L::IDESC_S, kk > 0 ? 1u : 0u);
            }
            umma_commit(bar(kSwQEmpty + wg));
            umma_commit(bar(kSwSFull + wg));
            SWA_TRACE(ns, 7);
            useq_of[ns & 3] = s_useq;
            last_of[ns & 3] = s_last;
            ++ns;
            if (ns < ntiles) prep_s();
            prog = true;
          }
        }
        if (npv < ns) {
          const int wg = npv & 1;
          if (mbar_test(bar(kSwPReady + wg), (npv >> 1) & 1)) {
            SWA_TRACE(npv, 18);
            tc_fence_after();
            const int uq = useq_of[npv & 3];
            const uint32_t base = tmem + wg * 256;
            // the first tokens' unit, then the nine of the window; not the two slots outside it: they
            // may be taking rows of later keys, which are not f16 yet (and may hold anything)
            umma_ts(base + 128, base + 8 * kSwaUnits, smem_desc(sV + kSwaUnits * L::UNIT_BYTES, L::R_CHUNK, 1024),
                    L::IDESC_PV, 0u);
            const int um = uq % kSwaUnits;
            const uint32_t out2 = (1u << (um + 1 < kSwaUnits ? um + 1 : um + 1 - kSwaUnits)) |
                                  (1u << (um + 2 < kSwaUnits ? um + 2 : um + 2 - kSwaUnits));
#pragma unroll
            for (int s2 = 0; s2 < kSwaUnits; ++s2)
              if (!(out2 >> s2 & 1u))
                umma_ts(base + 128, base + 8 * s2, smem_desc(sV + s2 * L::UNIT_BYTES, L::R_CHUNK, 1024), L::IDESC_PV, 1u);
            umma_commit(bar(kSwPVDone + wg));
            umma_commit(bar(kSwSlotFree + (uq - 8) % kSwaUnits));
            if (last_of[npv & 3])
              for (int s2 = 1; s2 < kSwaWin; ++s2)
                umma_commit(bar(kSwSlotFree + (uq - 8 + s2) % kSwaUnits));
            if (last_of[npv & 3]) umma_commit(bar(kSwFirstFree));
            SWA_TRACE(npv, 8);
            ++npv;
            prog = true;
          }
        }
        if (prog) {
          idle = 0;
        } else if ((++idle & 15u) == 0) {   // look at the clock only now and then
          if (idle == 16u) t_prog = globaltimer_ns();
          if (*s_abort) {
            ok = false;
          } else if (globaltimer_ns() - t_prog > kWaitLimitNs) {
            *s_abort = 1;
            atomicOr(err, kErrWaitTimeout);
            ok = false;
          }
        }
      }
      umma_commit(bar(kSwFinal));
      mbar_wait_drain(bar(kSwFinal), 0, err);
    }
  } else if (warp < 6) {
    // ------------------------------------------------------------ RoPE group
    const int ctid = threadIdx.x - 64;             // 0..127, also the Q row it rotates
    const int nun = p.rot_dims >> 4;
    auto wait_all = [&](uint32_t b_, uint32_t par) -> bool {
      const bool w_ok = mbar_wait(b_, par, s_abort, err);
      return __all_sync(0xffffffffu, w_ok);
    };
    float2 turn[4];   // (cos, sin)(j w_lane) of positions j = warp, warp + 4, .. of a block
    if (half == 32) {
#pragma unroll
      for (int i2 = 0; i2 < 4; ++i2) {
        angle((ctid >> 5) + 4 * i2, turn[i2].y, turn[i2].x);
      }
    }
    // Two tables. Block i writes its angles into table i & 1 and, if it begins a run, the run's turns
    // into the other one, the spare table. Who has read a table before it is written again:
    //   angles of block i over those of block i - 2: all four warps arrived at kSwTab of block i - 1
    //     (waited for there), each behind its last read of block i - 2;
    //   turns of block i over the angles of block i - 1: all four arrived at kSwTab of block i;
    //   angles of block i + 1 over the turns of block i: kSwQReady of block i, one arrival per warp of this
    //     group behind its last read of the turns. It is waited for at the head of block i + 1 only where
    //     block i began a run, and cannot be overtaken there: its next phase is that of block i + 2;
    //   the same over the turns of the first run, which the softmax warps read too: kSwStart.
    int seq = 0, i = 0, runs = 0;
    bool turned = false;                             // the previous block left turns in the spare table
    for (long long f = f0; f < f1; ++f, ++i) {
      const int t = static_cast<int>(f % nqt);
      const bool first = (f == f0 || t == 0);
      if (first) seq += 8;
      const int useq = seq++;
      const int p0 = p.q_off + t * kSwaP;            // absolute position of the block
      if (turned && !wait_all(bar(kSwQReady + ((i - 1) & 1)), ((i - 1) >> 1) & 1)) break;
      turned = first && half == 32;
      float* tab = reinterpret_cast<float*>(smem + L::OFF_TAB + (i & 1) * L::TAB_BYTES);
      if (ctid == 0) SWA_TRACE(i, 0);
      // (the softmax warps' units of the first run: landed, and the turns read, before either is touched:
      // see the tables above)
      if (i == 1 && !wait_all(bar(kSwStart), 0)) break;
      // (cos, sin) of the block's 16 positions (double buffered: tile i - 1 may still read)
      if (half == 32) {
        // one angle per thread (frequency = lane), turned by the four positions the thread serves
        float sn, cs;
        angle(p0, sn, cs);
#pragma unroll
        for (int i2 = 0; i2 < 4; ++i2) {
          float* tk = tab + ((ctid >> 5) + 4 * i2) * 64 + (lane >> 1) * 4 + (lane & 1);
          tk[0] = cs * turn[i2].x - sn * turn[i2].y;
          tk[2] = sn * turn[i2].x + cs * turn[i2].y;
        }
      } else if (half > 0) {
        for (int e = ctid; e < kSwaP * half; e += 128) {
          const int pp = e / half, k = e - pp * half;
          const double ang = static_cast<double>(p0 + pp) * s_invf[k];
          const double nrev = rint(ang * 0.15915494309189535);
          float sn, cs;
          __sincosf(static_cast<float>(fma(-nrev, 6.283185307179586, ang)), &sn, &cs);
          float* tk = tab + pp * 64 + (k >> 1) * 4 + (k & 1);   // (cos k, cos k+1, sin k, sin k+1)
          tk[0] = cs;
          tk[2] = sn;
        }
      }
      if (half > 0) {
        arrive_warp(bar(kSwTab + (i & 1)));   // (bounded waits only: no hardware named barrier)
        if (!wait_all(bar(kSwTab + (i & 1)), (i >> 1) & 1)) break;
      }
      // the turns j w_k of a run's start are handed around in the table that the next block will write
      float* spare = reinterpret_cast<float*>(smem + L::OFF_TAB + ((i + 1) & 1) * L::TAB_BYTES);
      if (first && half == 32) {
#pragma unroll
        for (int i2 = 0; i2 < 4; ++i2) {
          float* tk = spare + ((ctid >> 5) + 4 * i2) * 64 + (lane >> 1) * 4 + (lane & 1);
          tk[0] = turn[i2].x;
          tk[2] = turn[i2].y;
        }
        arrive_warp(bar(kSwTurn));
      }
      if (!wait_all(bar(kSwQFull + (i & 1)), (i >> 1) & 1)) break;
      if (ctid == 0) SWA_TRACE(i, 1);
      if (half > 0 && t * kSwaP + (ctid >> 3) < p.n)
        rope_row_tab(smem + L::OFF_Q + (i & 1) * L::Q_STAGE + ctid * 128, ctid, nun,
                     reinterpret_cast<const float4*>(tab + (ctid >> 3) * 64));
      // K units of this block: the new one, or at the start of a run the whole window (in the first run
      // the softmax warps do the eight before the block's own)
      bool ok = true;
      const int s_first = first ? useq - 8 : useq, s_mine = i == 0 ? useq : s_first;
      for (int s = s_mine; s <= useq && ok; ++s) ok = wait_all(bar(kSwKVFull + s % kSwaUnits), (s / kSwaUnits) & 1);
      if (!ok) break;
      for (int s = s_mine; s <= useq; ++s) v_part(s % kSwaUnits, ctid);   // V units entering the ring
      if (first) {                                 // and the first tokens' unit of a new run
        if (!wait_all(bar(kSwFirstFull), runs & 1)) break;
        v_part(kSwaUnits, ctid);
        if (half == 32) {   // K of the window's units and of the first tokens, two units per turn
          if (!wait_all(bar(kSwTurn), runs & 1)) break;
#pragma unroll 1
          for (int k2 = (i == 0 ? 8 : 0) + (ctid >> 6); k2 <= kSwaWin; k2 += 2) {   // 9: the first tokens'
            const bool own = k2 < kSwaWin;
            const int kpos0 = own ? p0 - 128 + 16 * k2 : 0;
            float bs, bc;
            angle(kpos0, bs, bc);
            k_part(own ? (s_first + k2) % kSwaUnits : kSwaUnits, ctid & 63, kpos0, bc, bs, spare);
          }
        } else if (half > 0 && ctid < 16) {
          const int ring_row = kSwaUnits * 16 + ctid;
          if (ctid >= p.krot_from && ctid < p.nk) rope_row(sK, L::R_CHUNK, ring_row, ctid, p.rot_dims, s_invf);
          else if (ctid < p.krot_from) f16_row(sK, L::R_CHUNK, ring_row, p.rot_dims);
        }
        ++runs;
      }
      if (half > 0) {
        if (first && half == 32) {
          // done above
        } else if (first) {
          for (int rr = (i == 0 ? 128 : 0) + ctid; rr < 16 * kSwaWin; rr += 128) {
            const int kpos = p0 - 128 + rr;
            const int ring_row = ((s_first + rr / 16) % kSwaUnits) * 16 + (rr & 15);
            if (kpos >= p.krot_from && kpos < p.nk) rope_row(sK, L::R_CHUNK, ring_row, kpos, p.rot_dims, s_invf);
            else if (kpos >= 0 && kpos < p.krot_from) f16_row(sK, L::R_CHUNK, ring_row, p.rot_dims);
          }
        } else if (ctid < 64) {   // the 16 new K rows, one (row, unit pair) per thread
          const int rr = ctid >> 2, u = ctid & 3;
          const int ring_row = (useq % kSwaUnits) * 16 + rr;
          if (u < nun && p0 + rr < p.nk)   // a block's own keys lie in the chunk: never stored rotated
            rope_unit(smem + L::OFF_K + ring_row * 128, ring_row, nun,
                      reinterpret_cast<const float4*>(tab + rr * 64), u);
        }
      }
      fence_proxy_async_smem();
      arrive_warp(bar(kSwQReady + (i & 1)));
      if (lane == 0) SWA_TRACE(i, 21 + (ctid >> 5));
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    const int w = (warp - 6) >> 2;                 // group 0 or 1
    const int q4 = warp & 3;
    const int r = q4 * 32 + lane;                  // row == TMEM lane
    const int ctid = (warp - 6 - 4 * w) * 32 + lane;
    const int pl = r >> 3, hl = r & 7;
    const uint32_t trow = tmem + w * 256 + (static_cast<uint32_t>(q4 * 32) << 16);
    auto wait_all = [&](uint32_t b_, uint32_t par) -> bool {
      const bool w_ok = mbar_wait(b_, par, s_abort, err);
      return __all_sync(0xffffffffu, w_ok);
    };
    // the first run's unit that this warp asked for (the RoPE group alone took 5500 cycles for all ten of
    // a run's start, a third of a short call)
    bool started = true;
    {
      const int slot = warp - 6, kpos0 = p.q_off + static_cast<int>(f0 % nqt) * kSwaP - 128 + 16 * slot;
      float bs = 0.f, bc = 0.f;
      if (half == 32) angle(kpos0, bs, bc);
      started = wait_all(bar(kSwKVFull + slot), 0) && (half != 32 || wait_all(bar(kSwTurn), 0));
      if (started) {
#pragma unroll 1
        for (int x = lane; x < 128; x += 32) v_part(slot, x);
        const float* turns = reinterpret_cast<const float*>(smem + L::OFF_TAB + L::TAB_BYTES);
        if (half == 32) {
#pragma unroll 1
          for (int x = lane; x < 64; x += 32) k_part(slot, x, kpos0, bc, bs, turns);
        } else if (half > 0 && lane < 16) {
          const int kpos = kpos0 + lane;
          if (kpos >= p.krot_from && kpos < p.nk) rope_row(sK, L::R_CHUNK, slot * 16 + lane, kpos, p.rot_dims, s_invf);
          else if (kpos >= 0 && kpos < p.krot_from) f16_row(sK, L::R_CHUNK, slot * 16 + lane, p.rot_dims);
        }
        fence_proxy_async_smem();
        arrive_warp(bar(kSwStart));
      }
    }
    int seq = 0, i = 0;
    for (long long f = f0; f < f1 && started; ++f, ++i) {
      const int bg = static_cast<int>(f / nqt), t = static_cast<int>(f % nqt);
      const bool first = (f == f0 || t == 0);
      if (first) seq += 8;
      const int useq = seq++;
      if ((i & 1) != w) continue;
      const int b = bg / p.Hkv, g = bg - b * p.Hkv;
      const int qi = t * kSwaP + pl;                 // query row within the call
      const int p0 = p.q_off + t * kSwaP;            // absolute positions
      const int pos = p.q_off + qi;
      const int hq = g * kSwaG + hl;
      const bool row_ok = qi < p.n;

      // Slot block c < 11 (columns 16c..16c+15) holds the unit d = (useq - c) mod 11 blocks back: keys
      // kb + e with kb = p0 - 16 d; block 11 the first tokens. A block is empty, full or partial for
      // every row of the tile alike (the class depends on p0, W, d and n_first only); only partial
      // blocks mask per element.
      const float sink2 = p.sink ? p.sink[hq] * kLog2e : -INFINITY;
      const int klo = max(0, pos - p.window + 1);          // valid keys of this row: [klo, pos]
      const int klo_min = max(0, p0 - p.window + 1);       // over the tile's rows
      const int klo_max = max(0, p0 + kSwaP - 1 - p.window + 1);
      const int um = useq % kSwaUnits;
      // 0 = empty, 1 = partial, 2 = full; elo/ehi: valid e of this row (partial blocks)
      auto block_class = [&](int c, int& elo, int& ehi) -> int {
        if (c == kSwaUnits) {   // first tokens below this row's window
          elo = 0;
          const int nfirst = first_of(p);
          ehi = min(nfirst, klo) - 1;
          return min(nfirst, klo_max) <= 0 ? 0 : (min(nfirst, klo_min) >= 16 ? 2 : 1);
        }
        int d = um - c;
        d += d < 0 ? kSwaUnits : 0;
        const int kb = p0 - 16 * d;
        elo = max(klo - kb, 0);
        ehi = min(pos - kb, 15);
        if (d >= kSwaWin || kb + 15 < klo_min || kb > p0 + kSwaP - 1) return 0;
        return (kb >= klo_max && kb + 15 <= p0) ? 2 : 1;
      };
      if (!wait_all(bar(kSwSFull + w), (i >> 1) & 1)) break;
      tc_fence_after();
      if (ctid == 0) SWA_TRACE(i, 3);
      float ref = -INFINITY;                                // reference of P (log2 units)
      float sum0 = 0.f, sum1 = 0.f;                         // of its even and odd columns
      const unsigned long long sc2 = f2_pack(p.scale_log2, p.scale_log2);
      // One pass over the slot blocks, one block per turn. The reference is the maximum of the first block that
      // holds a key of the row, rounded up to a whole step, and moves only when a later block lies 2^8 above it
      // (the P written so far are then scaled by a power of two: exact while they stay normal, else off by at
      // most 2^-25, as a weight that small is when it is first written; rare). P = 2^(a - ref) stays within 2^8
      // of 1 at its largest, which f16 carries with all its 11 bits. A pass of its own for the maximum cost six
      // TMEM round trips more; two blocks per turn, in variants for full and partial ones, more code than the
      // instruction caches of an SM that runs four different roles hold (stalls for instructions doubled). n =
      // 32768, 64/8 heads, one after the other under the power cap: two passes 553 us, pairs in one pass 573
      // (cold 515), with their loads ahead 620, this 461 (cold 411).
      uint32_t v[16];
      int elo, ehi;
      tmem_ld16(trow, v);
#pragma unroll 1
      for (int c = 0; c < L::UNITS; ++c) {
        tmem_wait_ld();
        reg_fence16(v);
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(v[e]);
        // the next block's scores are under way while this one is worked on (P of block c ends at
        // column 8 (c + 1), below them)
        if (c + 1 < L::UNITS) tmem_ld16(trow + (c + 1) * 16, v);
        const int kind = block_class(c, elo, ehi);
        if (kind == 0) {                                  // no key for any row (the same for the tile)
          const uint32_t zero[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
          tmem_st8(trow + c * 8, zero);
          continue;
        }
        if (kind == 1) {                                  // masked keys to -inf
          const uint32_t valid = ((1u << (ehi + 1)) - 1u) & ~((1u << elo) - 1u);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = valid >> e & 1u ? x[e] : -INFINITY;
        }
        float ma = fmax3(x[0], x[1], x[2]), mb = fmax3(x[3], x[4], x[5]);
        ma = fmax3(ma, x[6], x[7]);
        mb = fmax3(mb, x[8], x[9]);
        ma = fmax3(ma, x[10], x[11]);
        mb = fmax3(mb, x[12], x[13]);
        const float pm = fmaxf(fmax3(ma, x[14], x[15]), mb) * p.scale_log2;
        const bool move = pm > ref + 8.f;                 // (also the first key of the row)
        const float was = ref;
        ref = move ? ceilf(pm) : ref;                     // whole steps: P is scaled by a power of two
        if (__any_sync(0xffffffffu, move && was != -INFINITY)) {
          const float al = move && was != -INFINITY ? ex2(was - ref) : 1.f;
          sum0 *= al;
          sum1 *= al;
          const __half2 al2 = __float2half2_rn(al);
          tmem_wait_st();
#pragma unroll 1
          for (int c2 = 0; c2 < c; ++c2) {
            uint32_t w2[8];
            tmem_ld8(trow + c2 * 8, w2);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const __half2 a = __hmul2(*reinterpret_cast<const __half2*>(&w2[e]), al2);
              w2[e] = *reinterpret_cast<const uint32_t*>(&a);
            }
            tmem_st8(trow + c2 * 8, w2);
          }
        }
        const float r0 = ref == -INFINITY ? 0.f : ref;
        const unsigned long long nref2 = f2_pack(-r0, -r0);
        uint32_t pk[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 y = f2_unpack(f2_fma(f2_pack(x[2 * e], x[2 * e + 1]), sc2, nref2));
          const float a0 = ex2(y.x), a1 = ex2(y.y);
          sum0 += a0;
          sum1 += a1;
          pk[e] = pack_f16(a0, a1);
        }
        tmem_st8(trow + c * 8, pk);
      }
      ref = ref == -INFINITY ? 0.f : ref;                 // a row without keys
      tmem_wait_st();
      tc_fence_before();
      arrive_warp(bar(kSwPReady + w));
      if (lane == 0) SWA_TRACE(i, 25 + (ctid >> 5));
      const float sum = sum0 + sum1;
      // denominator with the sink: M = max(amax, sink); l = sum 2^(amax-M) + 2^(sink-M)
      const float M = fmaxf(ref, sink2);
      const float sc = ex2(ref - M);
      const float lt = sum * sc + (p.sink ? ex2(sink2 - M) : 0.f);

      // epilogue: o = O sc / lt -> bf16, lse = (M + log2 lt) ln 2
      if (!wait_all(bar(kSwPVDone + w), (i >> 1) & 1)) break;
      tc_fence_after();
      if (ctid == 0) SWA_TRACE(i, 5);
      const bool none = lt == 0.f;                   // no key and no sink (a NaN stays one)
      const float inv_l = none ? 0.f : sc / lt;
      const bool odd = lane & 1;                     // (rows of two lanes: heads of one position)
      __nv_bfloat16* opair = p.out + ((static_cast<long long>(b) * p.n + qi) * p.Hq + (hq & ~1)) * 128 + (odd ? 8 : 0);
      // O columns [128, 192) overlap the S columns of this group's next tile: read them
      // first, release the TMEM region, then finish with columns [192, 256)
#pragma unroll 1
      for (int hh = 0; hh < 4; ++hh) {
        uint32_t v[2][16];
#pragma unroll
        for (int q = 0; q < 2; ++q) tmem_ld16(trow + 128 + (2 * hh + q) * 16, v[q]);
        tmem_wait_ld();
        if (hh == 1) {
          tc_fence_before();
          arrive_warp(bar(kSwTmFree + w));
        }
        const unsigned long long il2 = f2_pack(inv_l, inv_l);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 o = f2_unpack(f2_mul(f2_bits(v[q][2 * e], v[q][2 * e + 1]), il2));
            pk[e] = pack_bf16(o.x, o.y);
          }
          // two lanes write the 32 bytes of the even lane's row, then those of the odd lane's: whole
          // sectors (n = 32768: 410 us with halves of them, 390 so)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? pk[e] : pk[4 + e], 1);
            if (odd) pk[e] = got;
            else pk[4 + e] = got;
          }
          if (row_ok) {
            *reinterpret_cast<uint4*>(opair + (2 * hh + q) * 16) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            *reinterpret_cast<uint4*>(opair + 128 + (2 * hh + q) * 16) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
          }
        }
      }
      if (row_ok && p.lse)
        p.lse[(static_cast<long long>(b) * p.Hq + hq) * p.n + qi] =
            none ? -INFINITY : (M + log2f(lt)) * kLn2;
      if (ctid == 0) SWA_TRACE(i, 6);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace mimo
