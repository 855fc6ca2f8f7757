// append_paged.cuh - writes new tokens into a paged KV cache: K rotated at its position, V as
// it is, as bf16 or as E4M3 bytes with one scale per (token, KV head) row.
//
// Rotation ("...MiMo-V2.6-Flash-MOPD混合SWA设计原理" §5): dims (d, d + rot/2), d < rot/2, turn by
// the angle pos * theta^(-2d/rot), reduced modulo 2 pi in double precision. FP8 rows: scale =
// amax / 448 (1 for a row of zeros), byte = e4m3(x / scale), K from its rotated fp32 values.
//
// The bytes bound it (640 read and 640, or 328, written per row). A CTA takes kApTokens tokens
// of one sequence with all their heads: the (cos, sin) of a token is computed once for its heads
// (the frequencies theta^(-2d/rot) come from the host), and a warp writes one row at a time:
// lanes 0-23 the 16-byte units of K (a unit's partner comes from its lane by a shuffle), lanes
// 24-31 two units of V each, so a row's amax is a warp reduction.
#pragma once

#include "ptx.cuh"
#include "decode.cuh"

namespace mimo {

constexpr int kApThreads = 256;

struct AppendPagedParams {
  const __nv_bfloat16* k;     // [B, n, Hkv, 192] un-rotated
  const __nv_bfloat16* v;     // [B, n, Hkv, 128]
  void* kc;                   // pages, as PagedParams
  void* vc;
  float* ks;                  // FP8 scales
  float* vs;
  const int* table;           // [B, max_pages]
  const int* pos;             // [B] position of the chunk's first token
  const int* n_new;           // [B] tokens to write (null: n)
  int page_stride;
  int B, n, Hkv, rot, page_size, max_pages, num_pages, tokens;   // tokens: per CTA
  uint32_t div_mul;           // t / page_size = (t * div_mul) >> div_shift for t < 2^31
  int div_shift;
  double invf[kDQK / 2];      // theta^(-2d/rot)
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ void unpack8(const uint4 x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
// max |x| as bits: magnitudes order as their bits, a NaN above all
__device__ __forceinline__ uint32_t amax8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
  return m;
}
// The scale amax / 448 of a row (1 for zeros) and its reciprocal. Multiplications: the scale is off
// by one rounding (2^-24) and x / scale by 2^-22, far below e4m3's half step (2^-4). Magnitudes
// whose reciprocal may leave fp32's range take the divisions.
__device__ __forceinline__ float row_scale(uint32_t amax_bits, float& inv) {
  const float a = __uint_as_float(amax_bits);
  if (a > 1e-30f && a < 1e30f) {
    inv = __fdividef(448.f, a);
    return a * (1.f / 448.f);
  }
  const float sc = a / 448.f;
  inv = 0.f;                                  // x / scale by division
  return sc == 0.f ? 1.f : sc;
}
__device__ __forceinline__ void scale8(float (&f)[8], float sc, float inv) {
  if (inv != 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] /= sc;
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kApThreads) append_paged_kernel(const __grid_constant__ AppendPagedParams p) {
  extern __shared__ float2 s_cs[];            // [tokens][rot / 2] (cos, sin)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = (p.n - 1) / p.tokens + 1;
  const int b = blockIdx.x / tiles, i0 = (blockIdx.x - b * tiles) * p.tokens;
  const int half = p.rot >> 1, nun = p.rot >> 4;   // nun: 16-byte units per half
  int count = p.n_new ? min(__ldg(p.n_new + b), p.n) : p.n;
  count = min(count - i0, p.tokens);
  if (count <= 0) return;
  const long long pos0 = static_cast<long long>(__ldg(p.pos + b)) + i0;
  const long long most = static_cast<long long>(p.max_pages) * p.page_size;
  for (int x = tid; x < count * half; x += kApThreads) {
    const int t = x / half, d = x - t * half;
    const double ang = static_cast<double>(pos0 + t) * p.invf[d];
    const double turns = rint(ang * 0.15915494309189535);
    float sn, cs;
    sincosf(static_cast<float>(fma(-turns, 6.283185307179586, ang)), &sn, &cs);
    s_cs[x] = make_float2(cs, sn);
  }
  __syncthreads();
  // two rows of the warp at a time, so that both rows' loads are in flight together
  const int rows = count * p.Hkv;
  const bool is_k = lane < 24;
  const int peer = lane < nun ? lane + nun : (lane < 2 * nun ? lane - nun : lane);
  for (int r0 = warp; r0 < rows; r0 += 2 * (kApThreads / 32)) {
    uint32_t dst[2];
    int tok[2];
    bool put[2];
    uint4 x0[2], x1[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = r0 + k * (kApThreads / 32);
      put[k] = r < rows;
      dst[k] = 0;
      x0[k] = x1[k] = make_uint4(0u, 0u, 0u, 0u);
      const int t = r / p.Hkv, g = r - t * p.Hkv;
      tok[k] = put[k] ? t : 0;
      const long long pos = pos0 + t;
      put[k] = put[k] && pos >= 0 && pos < most;     // outside the table: not written
      if (put[k]) {
        const int pg = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(pos)) * p.div_mul) >> p.div_shift);
        const int ent = __ldg(p.table + static_cast<long long>(b) * p.max_pages + pg);
        const long long src = (static_cast<long long>(b) * p.n + i0) * p.Hkv + r;
        if (is_k) {
          x0[k] = *reinterpret_cast<const uint4*>(p.k + src * kDQK + lane * 8);
        } else {
          const uint4* pv = reinterpret_cast<const uint4*>(p.v + src * kDV + (lane - 24) * 16);
          x0[k] = pv[0];
          x1[k] = pv[1];
        }
        put[k] = static_cast<unsigned>(ent) < static_cast<unsigned>(p.num_pages);
        // (token, KV head) rows of a pool number less than 2^31 (checked by the host)
        if (put[k]) dst[k] = static_cast<uint32_t>((ent * p.page_stride + static_cast<int>(pos) - pg * p.page_size) * p.Hkv + g);
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // the partner unit of the rotation, lane + nun or lane - nun
      uint4 y;
      y.x = __shfl_sync(0xffffffffu, x0[k].x, peer);
      y.y = __shfl_sync(0xffffffffu, x0[k].y, peer);
      y.z = __shfl_sync(0xffffffffu, x0[k].z, peer);
      y.w = __shfl_sync(0xffffffffu, x0[k].w, peer);
      if (!put[k]) continue;                         // the same for the whole warp
      float f[8], h[8];
      unpack8(x0[k], f);
      if (lane < 2 * nun) {
        unpack8(y, h);
        const float2* cs = s_cs + tok[k] * half + (lane < nun ? lane : lane - nun) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 w = cs[i];
          f[i] = lane < nun ? f[i] * w.x - h[i] * w.y : f[i] * w.x + h[i] * w.y;
        }
      }
      const uint64_t d = dst[k];
      if constexpr (FP8) {
        unpack8(x1[k], h);                           // V: second unit (zeros on K lanes)
        const uint32_t top = max(amax8(f), amax8(h));
        const uint32_t ak = __reduce_max_sync(0xffffffffu, is_k ? top : 0u);
        const uint32_t av = __reduce_max_sync(0xffffffffu, is_k ? 0u : top);
        float inv;
        const float sc = row_scale(is_k ? ak : av, inv);
        scale8(f, sc, inv);
        const uint2 lo = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
        if (is_k) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.kc) + d * kDQK + lane * 8) = lo;
        } else {
          scale8(h, sc, inv);
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.vc) + d * kDV + (lane - 24) * 16) =
              make_uint4(lo.x, lo.y, e4m3x4(h[0], h[1], h[2], h[3]), e4m3x4(h[4], h[5], h[6], h[7]));
        }
        if (lane == 0) p.ks[d] = sc;
        if (lane == 24) p.vs[d] = sc;
      } else {
        if (is_k) {
          if (lane < 2 * nun)
            x0[k] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.kc) + d * kDQK + lane * 8) = x0[k];
        } else {
          uint4* pv = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.vc) + d * kDV + (lane - 24) * 16);
          pv[0] = x0[k];
          pv[1] = x1[k];
        }
      }
    }
  }
}

}  // namespace mimo
