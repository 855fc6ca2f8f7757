// decode_paged.cuh - one-token decode over a paged KV cache (bf16 or FP8 pages), optionally
// bounded by a sliding window with the first tokens kept visible, split over the cache's
// length and joined.
//
// Math ("MiMo-V2-Flash: Hybrid Sliding Window Attention Architecture", §4.4): for the query of
// sequence b (position L - 1) and query head h, over the key set
//   J = [0, min(F, lo)) u [lo, L),  lo = max(0, L - W) (W > 0) or 0,
//   a_j = q.k_j * scale, m = max(sink_h, max_j a_j),
//   o = sum_j exp(a_j - m) v_j / (exp(sink_h - m) + sum_j exp(a_j - m)).
// Token t of sequence b lives in row table[b][t / page] * page_stride + t % page of the pool;
// a table entry outside [0, num_pages) names no page and its tokens are masked keys.
//
// Split. The tiles of KT keys of all (sequence, KV head) units form one line, cut into as many
// equal runs as there are CTAs (two per SM, four on FP8 pages, all resident at once): lengths only exist on the
// device, so every CTA sums the units' tile counts itself and finds its run. A run that holds a
// whole unit finishes it in place; at the ends of a run a unit's state (m, l, o) goes to a slot
// of the workspace (two per CTA), and the combine kernel joins the slots of each cut unit with
// the sink. Nothing depends on timing, so results repeat bit for bit.
//
// Tile. Rows arrive by 16-byte cp.async, NS tiles in flight, without a pause where one
// unit ends and the next begins. Four warps share one softmax: warp w scores KT/4 of the keys
// (S = Q K^T, m16n8k16 with the group's heads as rows), the weights P go to shared memory, and
// warp w multiplies all of P with its 32 columns of V. So a warp holds 16 x 32 of O (16 registers
// a thread) instead of 16 x 128, and no state is merged across warps at a unit's end but the row
// sums. The row references move only when a score lies 2^8 above them (and at a unit's first
// tile): a thread checks its own scores, P is written on trust, and the barrier that publishes P
// also says whether some thread disagrees, in which case the maxima meet in shared memory and P
// is written again. So a tile costs two barriers and no exchange of maxima.
// Precision: bf16 products are exact with fp32 sums. P is carried as two bf16 terms (high part
// and remainder, 16 significant bits), so that the only visible rounding is that of the output:
// one bf16 term made the output's error 1.4 times that of the rounding alone. FP8 pages: bytes
// and Q become f16 (exact for 2^-17 <= |q| <= 65504, off by at most 2^-25 below: half of f16's smallest
// step), the K scale multiplies the fp32 score, and the V scale joins the weight in its exponent
// (2^(s + log2|vs| - R) with a running maximum R of its own), so normal scales of any size keep P inside
// f16's normal range where it matters: a weight times its V scale 2^25 and more below the largest of the
// run drops out of O, not out of the denominator, which sums fp32 weights.
#pragma once

#include "ptx.cuh"
#include "decode.cuh"

namespace mimo {

struct PagedParams {
  const __nv_bfloat16* q;     // [B, Hq, 192]
  const void* k;              // [num_pages, page_stride, Hkv, 192] bf16 or E4M3 bytes
  const void* v;              // [num_pages, page_stride, Hkv, 128]
  const float* k_scale;       // [num_pages, page_stride, Hkv] (FP8)
  const float* v_scale;
  const int* table;           // [B, max_pages]
  const int* lengths;         // [B]
  const float* sink;          // [Hq] or null
  __nv_bfloat16* out;         // [B, Hq, 128]
  float* lse;                 // [B, Hq] or null
  int4* hdr;                  // [min(B * Hkv, nctas)]: (unit, first CTA, last CTA, -) of a cut unit
  float* part_ml;             // [2 nctas, G, 2]  (m in log2 units, l)
  float* part_o;              // [2 nctas, G, 128]
  int page_stride;            // tokens between pages
  int B, Hq, Hkv, page_size, max_pages, num_pages, window, n_first, nctas;
  uint32_t div_mul;           // t / page_size = (t * div_mul) >> div_shift for t < 2^31
  int div_shift;
  float scale_log2;           // softmax scale * log2(e)
  unsigned* err;
};

constexpr int kPgThreads = 128;

template <bool FP8>
struct PagedCfg {
  static constexpr int KT = FP8 ? 64 : 32;                  // keys per tile
  // CTAs per SM and stages. bf16 is bound by memory: 60 KB in flight per CTA. FP8 spends more
  // instructions per byte (conversions, two references): more warps to hide them, and Q straight
  // from memory instead of a buffer per stage (two sequences of 100-131k tokens: 60.5 us against
  // 63.3 with two CTAs of four stages; bf16 with three CTAs of three stages: 65.8 against 63.9)
  static constexpr int CTAS = FP8 ? 4 : 2;
  static constexpr int NS = FP8 ? 2 : 4;
  static constexpr int KROW = FP8 ? kKRow8 : kKRow;         // bytes per K row
  static constexpr int VROW = FP8 ? kVRow8 : kVRow;
  static constexpr int TPR = FP8 ? 4 : 8;                   // threads per row while loading
  static constexpr int ROWS = KT / (kPgThreads / TPR);      // rows per thread (2)
  static constexpr int OFF_V = KT * KROW;
  static constexpr int OFF_Q = OFF_V + KT * VROW;           // a unit's 16 query rows (its first tile only)
  static constexpr int OFF_OK = OFF_Q + (FP8 ? 0 : 16 * kKRow);   // float [KT]: 0, or -inf: no cached token
  static constexpr int OFF_SC = OFF_OK + KT * 4;            // float [2][KT] K and V scales
  static constexpr int STAGE = OFF_SC + (FP8 ? KT * 8 : 0);
  static constexpr int PROW = KT * 2 + 16;                  // bytes per row of P (padded: no bank conflicts)
  static constexpr int OFF_P = NS * STAGE;           // P high (or f16), then P low
  static constexpr int OFF_MX = OFF_P + (FP8 ? 1 : 2) * 16 * PROW;   // float [2][16][4] row maxima per warp
  static constexpr int OFF_L = OFF_MX + 2 * 16 * 4 * 4;     // float [16][4] row sums per warp
  static constexpr int SMEM = OFF_L + 16 * 4 * 4;
  static_assert(ROWS == 2, "two rows per thread and tile");
  static_assert(CTAS * (SMEM + 1024 + 256) <= 228 * 1024, "CTAs per SM");
};

// The keys of sequence b: token of key t is t for t < nf, lo + t - nf above.
struct PagedSeq {
  int lo, nf, nkeys;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedParams& p, int b) {
  const long long most = static_cast<long long>(p.max_pages) * p.page_size;   // < 2^31
  int L = __ldg(p.lengths + b);
#ifdef MIMO_DEBUG
  if (L < 0 || L > most) atomicOr(p.err, kErrBadLength);
#endif
  L = L < 0 ? 0 : (L < most ? L : static_cast<int>(most));
  PagedSeq s;
  s.lo = p.window > 0 && L > p.window ? L - p.window : 0;
  s.nf = s.lo < p.n_first ? s.lo : p.n_first;
  s.nkeys = s.nf + L - s.lo;
  return s;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16_bits(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// a / b for a >= 0, b > 0: the 64-bit division costs about 100 instructions more.
__device__ __forceinline__ long long div_ll(long long a, int b) {
  if (static_cast<unsigned long long>(a) >> 32) return a / b;
  return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}
template <int KT>
__device__ __forceinline__ int paged_tiles(int nkeys) {   // an empty unit keeps one (masked) tile
  return nkeys > 0 ? (nkeys - 1) / KT + 1 : 1;
}

template <int G, bool FP8>
__global__ void __launch_bounds__(kPgThreads, PagedCfg<FP8>::CTAS) decode_paged_kernel(const PagedParams p) {
  using C = PagedCfg<FP8>;
  constexpr int KT = C::KT, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ long long s_scan[4];
  __shared__ int s_b0;
  __shared__ long long s_off0;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, tq = lane & 3;   // mma fragment row / column pair
  const uint32_t s_base = smem_u32(smem);

  // ---- this CTA's run [a, e) of the line of tiles, and the unit that a lies in
  const int seg = (p.B + kPgThreads - 1) / kPgThreads;
  const int sb0 = min(tid * seg, p.B), sb1 = min(sb0 + seg, p.B);
  long long mine = 0;
  for (int b = sb0; b < sb1; ++b) mine += paged_tiles<KT>(paged_seq(p, b).nkeys);
  mine *= p.Hkv;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  long long T = 0, before = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < warp) before += s_scan[w];
    T += s_scan[w];
  }
  const int N = T < p.nctas ? static_cast<int>(T) : p.nctas;   // every run holds a tile
  const int cta = blockIdx.x;
  const long long U = static_cast<long long>(p.B) * p.Hkv;
  const bool by_unit = U <= p.nctas;          // headers by unit, else by CTA
  if (cta >= N) return;                       // (only while N = T < nctas, and U <= T: headers are by unit)
  // tile T c / N as c (T div N) + c (T mod N) div N
  const long long quo = div_ll(T, N);
  const int rem = static_cast<int>(T - quo * N);
  const long long a = quo * cta + rem * cta / N, e = quo * (cta + 1) + rem * (cta + 1) / N;
  {
    long long at = before + incl - mine;
    if (a >= at && a < at + mine) {
      for (int b = sb0; b < sb1; ++b) {
        const long long nt = static_cast<long long>(paged_tiles<KT>(paged_seq(p, b).nkeys)) * p.Hkv;
        if (a < at + nt) {
          s_b0 = b;
          s_off0 = a - at;
          break;
        }
        at += nt;
      }
    }
  }
  __syncthreads();

  // ---- the iterator of the loads, NS - 1 tiles ahead of the arithmetic
  int lb = s_b0;
  PagedSeq ls = paged_seq(p, lb);
  int lt = paged_tiles<KT>(ls.nkeys);
  int lg = static_cast<int>(div_ll(s_off0, lt)), lj = static_cast<int>(s_off0 - static_cast<long long>(lg) * lt);
  const int b0 = lb, g0 = lg, j0 = lj, t0 = lt;
  const int* tab = p.table + static_cast<long long>(lb) * p.max_pages;
  const int lrow = tid / C::TPR, lu = tid % C::TPR;
  const uint8_t* kbase = static_cast<const uint8_t*>(p.k) + lu * 16;
  const uint8_t* vbase = static_cast<const uint8_t*>(p.v) + lu * 16;
  int ent[2], off[2];
  bool unit_start = true;                     // the next tile to issue needs its unit's Q
  auto fetch = [&]() {                        // page entries of the iterator's tile
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = lj * KT + i * (KT / 2) + lrow;
      ent[i] = -1;
      off[i] = 0;
      if (key < ls.nkeys) {
        const int tok = key < ls.nf ? key : ls.lo + (key - ls.nf);
        const int pg = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(tok)) * p.div_mul) >> p.div_shift);
        off[i] = tok - pg * p.page_size;
        ent[i] = __ldg(tab + pg);
      }
    }
  };
  auto issue = [&](int stage) {
    const uint32_t st = s_base + stage * C::STAGE;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = i * (KT / 2) + lrow;
      const bool ok = static_cast<unsigned>(ent[i]) < static_cast<unsigned>(p.num_pages);
      const uint32_t sz = ok ? 16u : 0u;
      // (token, KV head) rows of a pool number less than 2^31 (checked by the host)
      const uint32_t r = static_cast<uint32_t>((ok ? ent[i] * p.page_stride + off[i] : 0) * p.Hkv + lg);
      const uint8_t* kg = kbase + static_cast<uint64_t>(r) * C::KROW;
      const uint8_t* vg = vbase + static_cast<uint64_t>(r) * C::VROW;
      if constexpr (FP8) {
        // K rows as they are (192 bytes: eight rows' 16-byte units cover the banks evenly); V
        // rows swizzled for the transposed ldmatrix
#pragma unroll
        for (int pp = 0; pp < 3; ++pp) cp_async16(st + row * C::KROW + (lu + 4 * pp) * 16, kg + pp * 64, sz);
#pragma unroll
        for (int pp = 0; pp < 2; ++pp)
          cp_async16(st + C::OFF_V + row * C::VROW + (((lu + 4 * pp) ^ (row & 7)) << 4), vg + pp * 64, sz);
        if (lu < 2) cp_async4(st + C::OFF_SC + (lu * KT + row) * 4, (lu ? p.v_scale : p.k_scale) + r, ok ? 4u : 0u);
      } else {
        const uint32_t sw = static_cast<uint32_t>((lu ^ (row & 7)) << 4);
#pragma unroll
        for (int pp = 0; pp < 3; ++pp) cp_async16(st + row * C::KROW + pp * 128 + sw, kg + pp * 128, sz);
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) cp_async16(st + C::OFF_V + row * C::VROW + pp * 128 + sw, vg + pp * 128, sz);
      }
      if (lu == 0) *reinterpret_cast<float*>(smem + stage * C::STAGE + C::OFF_OK + row * 4) = ok ? 0.f : -INFINITY;
    }
    if (!FP8 && unit_start) {                 // 16 rows of Q (zero above the group), swizzled
      const uint8_t* qg = reinterpret_cast<const uint8_t*>(p.q + (static_cast<long long>(lb) * p.Hq + lg * G) * kDQK);
      for (int x = tid; x < 16 * 24; x += kPgThreads) {
        const int r = x / 24, u = x - r * 24;
        cp_async16(st + C::OFF_Q + r * kKRow + ((u ^ (r & 7)) << 4), qg + (r < G ? r * kKRow + u * 16 : 0), r < G ? 16u : 0u);
      }
    }
  };
  auto advance = [&]() {                      // to the next tile of the line (the caller knows there is one)
    unit_start = false;
    if (++lj == lt) {
      lj = 0;
      unit_start = true;
      if (++lg == p.Hkv) {
        lg = 0;
        ++lb;
        ls = paged_seq(p, lb);
        lt = paged_tiles<KT>(ls.nkeys);
        tab += p.max_pages;
      }
    }
  };
  const int ntiles = static_cast<int>(e - a);   // (the host keeps runs below 2^31 tiles)
  fetch();
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    if (s < ntiles) {
      issue(s);
      if (s + 1 < ntiles) {
        advance();
        fetch();
      }
    }
    cp_async_commit();
  }

  // ---- the arithmetic
  int cb = b0, cg = g0, cj = j0, ct = t0;
  bool from_start = cj == 0, fresh = true;    // the segment holds its unit's first tile / starts here
  int4 hdr = make_int4(0, -1, -1, 0);
  uint32_t qa[12][4];
  float o[4][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
  float R0 = -INFINITY, R1 = -INFINITY;       // references of O (FP8; those of bf16 are m0, m1)
  float* s_mx = reinterpret_cast<float*>(smem + C::OFF_MX);
  float* s_l = reinterpret_cast<float*>(smem + C::OFF_L);
  const int mi = lane >> 3, r8 = lane & 7;
  int stage = 0;
  for (int it = 0; it < ntiles; ++it) {
    cp_async_wait<NS - 2>();
    __syncthreads();                          // the tile has landed; the previous one is consumed
    {
      const int ahead = stage == 0 ? NS - 1 : stage - 1;
      if (it + NS - 1 < ntiles) {
        issue(ahead);
        if (it + NS < ntiles) {
          advance();
          fetch();
        }
      }
      cp_async_commit();
    }
    const uint32_t sK = s_base + stage * C::STAGE, sV = sK + C::OFF_V, sQ = sK + C::OFF_Q;
    const uint8_t* st_ptr = smem + stage * C::STAGE;
    bool need = fresh;                        // the references have to move
    if (fresh) {
      fresh = false;
      if constexpr (FP8) {
        // k-slot order of a step (j, s): lane tq supplies dims 16 (4 j + tq) + 4 s .. + 3
        const __nv_bfloat16* qg = p.q + (static_cast<long long>(cb) * p.Hq + cg * G) * kDQK;
#pragma unroll
        for (int jj = 0; jj < 3; ++jj)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int r = gq + 8 * hh;
            uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
            if (r < G) {
              const uint4* src = reinterpret_cast<const uint4*>(qg + r * kDQK + 16 * (4 * jj + tq));
              x0 = __ldg(src);
              x1 = __ldg(src + 1);
            }
            const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
            for (int s4 = 0; s4 < 4; ++s4) {
              qa[4 * jj + s4][hh] = pack_f16(bf16_lo(w[2 * s4]), bf16_hi(w[2 * s4]));
              qa[4 * jj + s4][2 + hh] = pack_f16(bf16_lo(w[2 * s4 + 1]), bf16_hi(w[2 * s4 + 1]));
            }
          }
      } else {
        const int r = ((mi & 1) << 3) + r8;
#pragma unroll
        for (int kk = 0; kk < 12; ++kk)
          ldmatrix_x4(sQ + r * kKRow + (((2 * kk + (mi >> 1)) ^ (r & 7)) << 4), qa[kk][0], qa[kk][1], qa[kk][2],
                      qa[kk][3]);
      }
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
      m0 = m1 = R0 = R1 = -INFINITY;
      l0 = l1 = 0.f;
    }

    // S = Q K^T for this warp's KT/4 keys (NT n-tiles of 8)
    constexpr int NT = KT / 32;
    float s[NT][4];
    if constexpr (FP8) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        const int key = warp * 16 + nt * 8 + gq;
#pragma unroll
        for (int jj = 0; jj < 3; ++jj) {
          uint32_t w[4];
          ld_shared_v4(sK + key * C::KROW + (4 * jj + tq) * 16, w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mma_16816_f16(acc[x & 1], qa[4 * jj + x], e4m3x2_to_f16x2(static_cast<uint16_t>(w[x])),
                          e4m3x2_to_f16x2(static_cast<uint16_t>(w[x] >> 16)));
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) s[nt][x] = acc[0][x] + acc[1][x];
      }
    } else {
      float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int key = warp * 8 + r8;
#pragma unroll
      for (int k2 = 0; k2 < 6; ++k2) {
        uint32_t x0, x1, x2, x3;
        ldmatrix_x4(sK + key * C::KROW + (((4 * k2 + mi) ^ (key & 7)) << 4), x0, x1, x2, x3);
        mma_16816(acc[0], qa[2 * k2], x0, x1);
        mma_16816(acc[1], qa[2 * k2 + 1], x2, x3);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) s[0][x] = acc[0][x] + acc[1][x];
    }

    // scores in the log2 domain, masked keys at -inf; does any lie above its reference?
    const float* msk = reinterpret_cast<const float*>(st_ptr + C::OFF_OK);
    const float* ksc = reinterpret_cast<const float*>(st_ptr + C::OFF_SC);
    float lgv[NT][2], vsg[NT][2];             // (FP8) log2 |v scale|, and the scale
    const float lim0 = m0 + 8.f, lim1 = m1 + 8.f, rlim0 = R0 + 8.f, rlim1 = R1 + 8.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int key = warp * (KT / 4) + nt * 8 + tq * 2;
      const float2 mk = *reinterpret_cast<const float2*>(msk + key);
      float f0 = p.scale_log2, f1 = p.scale_log2;
      if constexpr (FP8) {
        const float2 kk = *reinterpret_cast<const float2*>(ksc + key);
        const float2 vv = *reinterpret_cast<const float2*>(ksc + KT + key);
        f0 *= kk.x;
        f1 *= kk.y;
        vsg[nt][0] = vv.x;
        vsg[nt][1] = vv.y;
        lgv[nt][0] = lg2(fabsf(vv.x));
        lgv[nt][1] = lg2(fabsf(vv.y));
      }
      s[nt][0] = fmaf(s[nt][0], f0, mk.x);
      s[nt][1] = fmaf(s[nt][1], f1, mk.y);
      s[nt][2] = fmaf(s[nt][2], f0, mk.x);
      s[nt][3] = fmaf(s[nt][3], f1, mk.y);
      need |= s[nt][0] > lim0 || s[nt][1] > lim0 || s[nt][2] > lim1 || s[nt][3] > lim1;
      if constexpr (FP8)
        need |= s[nt][0] + lgv[nt][0] > rlim0 || s[nt][1] + lgv[nt][1] > rlim0 || s[nt][2] + lgv[nt][0] > rlim1 ||
                s[nt][3] + lgv[nt][1] > rlim1;
    }
    float d0, d1;                             // this tile's share of the row sums
    auto write_p = [&]() {
      const float ref0 = m0 == -INFINITY ? 0.f : m0, ref1 = m1 == -INFINITY ? 0.f : m1;
      const float rr0 = R0 == -INFINITY ? 0.f : R0, rr1 = R1 == -INFINITY ? 0.f : R1;
      d0 = d1 = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float p0 = ex2(s[nt][0] - ref0), p1 = ex2(s[nt][1] - ref0);
        const float p2 = ex2(s[nt][2] - ref1), p3 = ex2(s[nt][3] - ref1);
        d0 += p0 + p1;
        d1 += p2 + p3;
        const uint32_t col = static_cast<uint32_t>(warp * (KT / 4) + nt * 8 + tq * 2) * 2;
        uint32_t* w0 = reinterpret_cast<uint32_t*>(smem + C::OFF_P + gq * C::PROW + col);
        uint32_t* w1 = reinterpret_cast<uint32_t*>(smem + C::OFF_P + (gq + 8) * C::PROW + col);
        if constexpr (FP8) {
          *w0 = f16_bits(copysignf(ex2(s[nt][0] + lgv[nt][0] - rr0), vsg[nt][0]),
                         copysignf(ex2(s[nt][1] + lgv[nt][1] - rr0), vsg[nt][1]));
          *w1 = f16_bits(copysignf(ex2(s[nt][2] + lgv[nt][0] - rr1), vsg[nt][0]),
                         copysignf(ex2(s[nt][3] + lgv[nt][1] - rr1), vsg[nt][1]));
        } else {
          const uint32_t h0 = pack_bf16(p0, p1), h1 = pack_bf16(p2, p3);
          *w0 = h0;
          *w1 = h1;
          w0[16 * C::PROW / 4] = pack_bf16(p0 - bf16_lo(h0), p1 - bf16_hi(h0));
          w1[16 * C::PROW / 4] = pack_bf16(p2 - bf16_lo(h1), p3 - bf16_hi(h1));
        }
      }
    };
    write_p();
    if (__syncthreads_or(need)) {
      // the tile's row maxima move the references; O and the sums follow; P again
      float mx0 = -INFINITY, mx1 = -INFINITY, rx0 = -INFINITY, rx1 = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mx0 = fmaxf(mx0, fmaxf(s[nt][0], s[nt][1]));
        mx1 = fmaxf(mx1, fmaxf(s[nt][2], s[nt][3]));
        if constexpr (FP8) {
          rx0 = fmaxf(rx0, fmaxf(s[nt][0] + lgv[nt][0], s[nt][1] + lgv[nt][1]));
          rx1 = fmaxf(rx1, fmaxf(s[nt][2] + lgv[nt][0], s[nt][3] + lgv[nt][1]));
        }
      }
#pragma unroll
      for (int sh = 1; sh < 4; sh <<= 1) {
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, sh));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, sh));
        if constexpr (FP8) {
          rx0 = fmaxf(rx0, __shfl_xor_sync(0xffffffffu, rx0, sh));
          rx1 = fmaxf(rx1, __shfl_xor_sync(0xffffffffu, rx1, sh));
        }
      }
      if (tq == 0) {
        s_mx[gq * 4 + warp] = mx0;
        s_mx[(gq + 8) * 4 + warp] = mx1;
        if constexpr (FP8) {
          s_mx[64 + gq * 4 + warp] = rx0;
          s_mx[64 + (gq + 8) * 4 + warp] = rx1;
        }
      }
      __syncthreads();
      auto move = [&](float& m, const float* at) -> float {
        const float4 x = *reinterpret_cast<const float4*>(at);
        const float mn = fmaxf(fmaxf(m, fmaxf(x.x, x.y)), fmaxf(x.z, x.w));
        const float al = ex2(m - (mn == -INFINITY ? 0.f : mn));   // 0 from -inf
        m = mn;
        return al;
      };
      const float al0 = move(m0, s_mx + gq * 4), al1 = move(m1, s_mx + (gq + 8) * 4);
      float ao0 = al0, ao1 = al1;
      if constexpr (FP8) {
        ao0 = move(R0, s_mx + 64 + gq * 4);
        ao1 = move(R1, s_mx + 64 + (gq + 8) * 4);
      }
      l0 *= al0;
      l1 *= al1;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        o[nt][0] *= ao0; o[nt][1] *= ao0;
        o[nt][2] *= ao1; o[nt][3] *= ao1;
      }
      write_p();
      __syncthreads();
    }
    l0 += d0;
    l1 += d1;

    // O (this warp's 32 columns) += P V
#pragma unroll
    for (int ks = 0; ks < KT / 16; ++ks) {
      const uint32_t prow = s_base + C::OFF_P + (((mi & 1) << 3) + r8) * C::PROW + ks * 32 + (mi >> 1) * 16;
      uint32_t pa[4];
      ldmatrix_x4(prow, pa[0], pa[1], pa[2], pa[3]);
      const int vrow = ks * 16 + ((mi & 1) << 3) + r8;
      if constexpr (FP8) {
        // a 16-bit element is two adjacent columns of one key: after the transposed load a
        // register holds (key 2 tq, key 2 tq + 1) x (column 2 gq, 2 gq + 1); its even and odd
        // bytes are the B fragments of the even and odd columns
        uint32_t x[4];
        ldmatrix_x4_trans(sV + vrow * C::VROW + (((2 * warp + (mi >> 1)) ^ (vrow & 7)) << 4), x[0], x[1], x[2], x[3]);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const uint32_t sel = odd ? 0x0031u : 0x0020u;
            mma_16816_f16(o[2 * u + odd], pa,
                          e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(x[2 * u], 0u, sel))),
                          e4m3x2_to_f16x2(static_cast<uint16_t>(__byte_perm(x[2 * u + 1], 0u, sel))));
          }
      } else {
        uint32_t pl[4];
        ldmatrix_x4(prow + 16 * C::PROW, pl[0], pl[1], pl[2], pl[3]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t v0, v1, v2, v3;
          ldmatrix_x4_trans(sV + vrow * C::VROW + (((4 * warp + 2 * u + (mi >> 1)) ^ (vrow & 7)) << 4), v0, v1, v2, v3);
          mma_16816(o[2 * u], pa, v0, v1);
          mma_16816(o[2 * u + 1], pa, v2, v3);
          mma_16816(o[2 * u], pl, v0, v1);
          mma_16816(o[2 * u + 1], pl, v2, v3);
        }
      }
    }

    // ---- the end of a unit, or of the run inside one
    const bool at_end = cj == ct - 1;
    if (at_end || it == ntiles - 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      if (tq == 0) {
        s_l[gq * 4 + warp] = l0;
        s_l[(gq + 8) * 4 + warp] = l1;
      }
      __syncthreads();
      const bool direct = from_start && at_end;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int r = gq + 8 * hh;
        if (r < G) {
          const float4 lw = *reinterpret_cast<const float4*>(s_l + r * 4);
          const float l = (lw.x + lw.y) + (lw.z + lw.w);
          const float m = hh ? m1 : m0;
          float f;                            // factor of O
          if (direct) {
            const long long bh = static_cast<long long>(cb) * p.Hq + cg * G + r;
            const float sk = p.sink ? p.sink[cg * G + r] * 1.4426950408889634f : -INFINITY;
            const float M = fmaxf(m, sk), ref = M == -INFINITY ? 0.f : M;
            const float Lt = l * ex2(m - ref) + (p.sink ? ex2(sk - ref) : 0.f);
            f = FP8 ? (hh ? R1 : R0) : m;
            f = Lt == 0.f ? 0.f : ex2(f - ref) / Lt;   // (a NaN stays one)
            uint32_t* orow = reinterpret_cast<uint32_t*>(p.out + bh * kDV);
            if constexpr (FP8) {
#pragma unroll
              for (int u = 0; u < 2; ++u)
                *reinterpret_cast<uint2*>(orow + 16 * warp + 8 * u + 2 * tq) =
                    make_uint2(pack_bf16(o[2 * u][2 * hh] * f, o[2 * u + 1][2 * hh] * f),
                               pack_bf16(o[2 * u][2 * hh + 1] * f, o[2 * u + 1][2 * hh + 1] * f));
            } else {
#pragma unroll
              for (int nt = 0; nt < 4; ++nt)
                orow[16 * warp + 4 * nt + tq] = pack_bf16(o[nt][2 * hh] * f, o[nt][2 * hh + 1] * f);
            }
            if (warp == 0 && tq == 0 && p.lse) p.lse[bh] = Lt == 0.f ? -INFINITY : (ref + log2f(Lt)) * 0.6931471805599453f;
          } else {
            const long long slot = (2LL * cta + (from_start ? 1 : 0)) * G + r;
            // O in the reference of m (FP8: R may lie far from it, but not O 2^(R - m))
            f = 1.f;
            if constexpr (FP8) f = (hh ? R1 : R0) == -INFINITY ? 0.f : ex2((hh ? R1 : R0) - m);
            float* po = p.part_o + slot * kDV + 32 * warp;
            if constexpr (FP8) {
#pragma unroll
              for (int u = 0; u < 2; ++u)
                *reinterpret_cast<float4*>(po + 16 * u + 4 * tq) =
                    make_float4(o[2 * u][2 * hh] * f, o[2 * u + 1][2 * hh] * f, o[2 * u][2 * hh + 1] * f,
                                o[2 * u + 1][2 * hh + 1] * f);
            } else {
#pragma unroll
              for (int nt = 0; nt < 4; ++nt)
                *reinterpret_cast<float2*>(po + 8 * nt + 2 * tq) = make_float2(o[nt][2 * hh], o[nt][2 * hh + 1]);
            }
            if (warp == 0 && tq == 0) {
              p.part_ml[slot * 2] = m;
              p.part_ml[slot * 2 + 1] = l;
            }
          }
        }
      }
      if (from_start && p.hdr) {
        const long long unit = static_cast<long long>(cb) * p.Hkv + cg;
        int4 h = make_int4(static_cast<int>(unit), -1, -1, 0);
        if (!at_end) {
          // CTA c holds tiles [T c / N, T (c + 1) / N): the one with tile x is floor(((x + 1) N - 1) / T)
          const long long x = a + it + (ct - 1 - cj);
          h.y = cta;
          h.z = static_cast<int>(((x + 1) * N - 1) / T);   // (once per CTA at most)
        }
        if (by_unit) {
          if (tid == 0) p.hdr[unit] = h;
        } else if (!at_end) {
          hdr = h;
        }
      }
      fresh = true;
      from_start = true;
      if (at_end && it + 1 < ntiles) {
        cj = -1;
        if (++cg == p.Hkv) {
          cg = 0;
          ++cb;
          ct = paged_tiles<KT>(paged_seq(p, cb).nkeys);
        }
      }
    }
    ++cj;
    stage = stage + 1 == NS ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  if (!by_unit && tid == 0 && p.hdr) p.hdr[cta] = hdr;
}

// Joins the slots of one cut unit (blockIdx.x) for 4 / WARPS query heads of its group
// (blockIdx.y): M = max(sink, max m_c), o = sum o_c 2^(m_c - M) / (2^(sink - M) + sum l_c 2^(m_c - M)).
// Warp w of a head's WARPS takes slots w, w + WARPS, ..., eight of them (state and row together) in
// flight, under a running maximum of its own: two trips to memory, the header's and the slots'. Few
// units are cut into many slots (four warps a head), many into two or three (one warp a head, so
// that all blocks are resident when the main kernel ends).
template <int WARPS>
__global__ void __launch_bounds__(128) decode_paged_combine_kernel(const PagedParams p, int G) {
  __shared__ float4 s_o[4][32];
  __shared__ float2 s_ml[4];
  pdl_wait();
  pdl_trigger();
  const int4 h = p.hdr[blockIdx.x];
  if (h.y < 0) return;
  const int block_warp = threadIdx.x >> 5, warp = block_warp % WARPS, lane = threadIdx.x & 31;
  const int r = blockIdx.y * (4 / WARPS) + block_warp / WARPS;
  if (WARPS == 1 && r >= G) return;
  const int np = h.z - h.y + 1;
  float M = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = warp; i0 < np; i0 += 8 * WARPS) {
    float2 ml[8];
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + WARPS * k;
      ml[k] = make_float2(-INFINITY, 0.f);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < np) {
        const long long s = (2LL * (h.y + i) + (i == 0 ? 1 : 0)) * G + r;
        ml[k] = *reinterpret_cast<const float2*>(p.part_ml + s * 2);
        x[k] = *reinterpret_cast<const float4*>(p.part_o + s * kDV + lane * 4);
      }
    }
    float mn = M;
#pragma unroll
    for (int k = 0; k < 8; ++k) mn = fmaxf(mn, ml[k].x);
    const float ref = mn == -INFINITY ? 0.f : mn, al = ex2(M - ref);
    M = mn;
    l *= al;
    acc.x *= al; acc.y *= al; acc.z *= al; acc.w *= al;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float w = ex2(ml[k].x - ref);
      l += ml[k].y * w;
      acc.x += x[k].x * w;
      acc.y += x[k].y * w;
      acc.z += x[k].z * w;
      acc.w += x[k].w * w;
    }
  }
  const int b = h.x / p.Hkv, head = (h.x - b * p.Hkv) * G + r;
  const float sk = p.sink ? p.sink[head] * 1.4426950408889634f : -INFINITY;
  if constexpr (WARPS > 1) {
    s_o[warp][lane] = acc;
    if (lane == 0) s_ml[warp] = make_float2(M, l);
    __syncthreads();
    if (warp != 0) return;
  }
  float m = fmaxf(sk, M);
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = fmaxf(m, s_ml[w].x);
  }
  const float ref = m == -INFINITY ? 0.f : m;
  float Lt = p.sink ? ex2(sk - ref) : 0.f;
  const float own = ex2(M - ref);
  Lt += l * own;
  acc.x *= own; acc.y *= own; acc.z *= own; acc.w *= own;
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      const float f = ex2(s_ml[w].x - ref);
      const float4 x = s_o[w][lane];
      Lt += s_ml[w].y * f;
      acc.x += x.x * f;
      acc.y += x.y * f;
      acc.z += x.z * f;
      acc.w += x.w * f;
    }
  }
  const float f = Lt == 0.f ? 0.f : 1.f / Lt;
  const long long bh = static_cast<long long>(b) * p.Hq + head;
  *reinterpret_cast<uint2*>(p.out + bh * kDV + lane * 4) =
      make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
  if (lane == 0 && p.lse) p.lse[bh] = Lt == 0.f ? -INFINITY : (ref + log2f(Lt)) * 0.6931471805599453f;
}

}  // namespace mimo
