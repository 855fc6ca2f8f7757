// append_paged.cuh - writes new tokens into a paged KV cache: K rotated at its position, V as
// it is, as bf16 or as E4M3 bytes with one scale per (token, KV head) row.
//
// Rotation ("...MiMo-V2.6-Flash-MOPD混合SWA设计原理" §5): dims (d, d + rot/2), d < rot/2, turn by
// the angle pos * theta^(-2d/rot), reduced modulo 2 pi in double precision. FP8 rows: scale =
// amax / 448 (1 for a row of zeros), byte = e4m3(x / scale), K from its rotated fp32 values.
//
// The bytes bound it (640 read and 640, or 328, written per row). A CTA takes a few tokens (32 rows)
// of one sequence with all their heads: the (cos, sin) of a token is computed once for its heads
// (the frequencies theta^(-2d/rot) come from the host), and half a warp writes a row: lane l its V
// unit l (16 bytes) and, for l < 12, two K units, the partners u and u + rot/16 of the rotation where
// it rotates. So no value crosses lanes but the row's two maxima, and the row's index arithmetic is
// shared by two rows of a warp; the first rows' loads are under way while the angles are worked
// out. 8192 tokens x 4 heads into FP8 pages (31.7 MB, 4.9 us at the copy rate): a row per warp with
// partners by shuffles 16.6 us, this 12.4 (64 registers: four CTAs per SM; three 13.4, five spill, 13.7).
// What is left there is mostly instructions: 7.6 M a call, some 930 a warp for its four rows, are 6.7 us of
// the issue slots (60.8 % of them in use, the math pipe the third of the stalls); then a CTA's chain of
// waits (position, table entry, angles) over two waves of CTAs.
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
// by 2^-23 (1 / 448 and the product round) and x / scale by 2^-22, far below e4m3's half step (2^-4); a
// value that lies in the middle of two e4m3 numbers, as a quotient of two bf16 values often does, may become
// either. Magnitudes whose reciprocal may leave fp32's range take the divisions.
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
__global__ void __launch_bounds__(kApThreads, 4) append_paged_kernel(const __grid_constant__ AppendPagedParams p) {
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
  // two rows per half warp at a time, so that their loads are in flight together
  const int rows = count * p.Hkv;
  const int l = lane & 15, sub = lane >> 4;
  const bool has_k = l < 12, turned = l < nun;
  const int u0 = turned ? l : 2 * l, u1 = turned ? l + nun : 2 * l + 1;
  constexpr int kStep = 2 * (kApThreads / 32);       // rows that all warps take in one go
  uint32_t dst[2];
  int tok[2];
  bool put[2];
  uint4 a[2], b2[2], c[2];
  auto load = [&](int r0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = r0 + k * kStep;
      put[k] = r < rows;
      dst[k] = 0;
      a[k] = b2[k] = c[k] = make_uint4(0u, 0u, 0u, 0u);
      const int t = r / p.Hkv, g = r - t * p.Hkv;
      tok[k] = put[k] ? t : 0;
      const long long pos = pos0 + t;
      put[k] = put[k] && pos >= 0 && pos < most;     // outside the table: not written
      if (put[k]) {
        const int pg = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(pos)) * p.div_mul) >> p.div_shift);
        const int ent = __ldg(p.table + static_cast<long long>(b) * p.max_pages + pg);
        const long long src = (static_cast<long long>(b) * p.n + i0) * p.Hkv + r;
        if (has_k) {
          a[k] = *reinterpret_cast<const uint4*>(p.k + src * kDQK + u0 * 8);
          b2[k] = *reinterpret_cast<const uint4*>(p.k + src * kDQK + u1 * 8);
        }
        c[k] = *reinterpret_cast<const uint4*>(p.v + src * kDV + l * 8);
        put[k] = static_cast<unsigned>(ent) < static_cast<unsigned>(p.num_pages);
        // (token, KV head) rows of a pool number less than 2^31 (checked by the host)
        if (put[k]) dst[k] = static_cast<uint32_t>((ent * p.page_stride + static_cast<int>(pos) - pg * p.page_size) * p.Hkv + g);
      }
    }
  };
  auto work = [&]() {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float f[8], h[8];
      unpack8(a[k], f);
      unpack8(b2[k], h);
      if (turned) {
        const float2* cs = s_cs + tok[k] * half + l * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 w = cs[i];
          const float x = f[i], y = h[i];
          f[i] = x * w.x - y * w.y;
          h[i] = y * w.x + x * w.y;
        }
      }
      const uint64_t d = dst[k];
      if constexpr (FP8) {
        float v[8];
        unpack8(c[k], v);
        uint32_t ak = max(amax8(f), amax8(h)), av = amax8(v);   // zeros on lanes without K
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          ak = max(ak, __shfl_xor_sync(0xffffffffu, ak, o));
          av = max(av, __shfl_xor_sync(0xffffffffu, av, o));
        }
        float ik, iv;
        const float sk = row_scale(ak, ik), sv = row_scale(av, iv);
        scale8(f, sk, ik);
        scale8(h, sk, ik);
        scale8(v, sv, iv);
        if (put[k]) {
          uint8_t* kc = static_cast<uint8_t*>(p.kc) + d * kDQK;
          if (has_k) {
            *reinterpret_cast<uint2*>(kc + u0 * 8) = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
            *reinterpret_cast<uint2*>(kc + u1 * 8) = make_uint2(e4m3x4(h[0], h[1], h[2], h[3]), e4m3x4(h[4], h[5], h[6], h[7]));
          }
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.vc) + d * kDV + l * 8) =
              make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
          if (l == 0) {
            p.ks[d] = sk;
            p.vs[d] = sv;
          }
        }
      } else if (put[k]) {
        __nv_bfloat16* kc = static_cast<__nv_bfloat16*>(p.kc) + d * kDQK;
        if (turned) {
          a[k] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
          b2[k] = make_uint4(pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]), pack_bf16(h[4], h[5]), pack_bf16(h[6], h[7]));
        }
        if (has_k) {
          *reinterpret_cast<uint4*>(kc + u0 * 8) = a[k];
          *reinterpret_cast<uint4*>(kc + u1 * 8) = b2[k];
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.vc) + d * kDV + l * 8) = c[k];
      }
    }
  };
  int r0 = 2 * warp + sub;
  bool more = r0 - sub < rows;                       // the same for the whole warp
  if (more) load(r0);                                // under way while the angles are worked out
  for (int x = tid; x < count * half; x += kApThreads) {
    const int t = x / half, d = x - t * half;
    const double ang = static_cast<double>(pos0 + t) * p.invf[d];
    const double turns = rint(ang * 0.15915494309189535);
    float sn, cs;
    sincosf(static_cast<float>(fma(-turns, 6.283185307179586, ang)), &sn, &cs);
    s_cs[x] = make_float2(cs, sn);
  }
  __syncthreads();
  while (more) {
    work();
    r0 += 2 * kStep;
    more = r0 - sub < rows;
    if (more) load(r0);
  }
}

}  // namespace mimo
