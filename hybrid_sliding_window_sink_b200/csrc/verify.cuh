// verify.cuh - acceptance of drafted tokens against the target's probabilities.
//
// Math (speculative sampling, the step after the MTP verification pass of
// "mimo-mtp-swa-not-mla"). For a sequence with drafts x_0 .. x_{n-1}, target rows p_0 .. p_n,
// draft rows q_0 .. q_{n-1} (one-hot at x_t when none are given: drafts by argmax) and uniform
// numbers u in [0, 1):
//   accepted a = the first t with not (u_t q_t(x_t) < p_t(x_t)), or n;
//   w(v) = max(p_a(v) - q_a(v), 0) for a < n, p_n(v) for a = n;
//   next token = the smallest v with w(0) + .. + w(v) > u_T * sum w.
// u q is exact in double. The sums are pairs of floats (see VfSum) within a lane and double across
// lanes: at V = 131072 an fp32 running sum is off by about as much as one token weighs (1e-5).
//
// Work: one row of p and one of q per sequence, read once (the accepted rows are only probed at
// x_t), so the bytes bound it; for few sequences the latency of the steps does. A cluster of C
// CTAs shares a row: warp k of the cluster sums one contiguous piece and writes the sum into
// every CTA's shared memory, and the CTA of the piece that the target falls into reads that
// piece again (from L2) with all its threads to find the token.
#pragma once

#include <cooperative_groups.h>

#include "ptx.cuh"

namespace mimo {

constexpr int kVfThreads = 256;
constexpr int kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCluster = 8;   // with 256 threads: 5.4 us for one row of 32000 and 17.6 us for 64 of
                                    // 131072; 512 threads 6.4 and 22.0, 1024 threads in clusters of 4 9.2 and 26
                                    // (fewer clusters are resident), clusters of 4 6.0 and 19.9

struct VerifyParams {
  const void* p;              // [B, T + 1, V] fp32 or bf16
  const void* q;              // [B, T, V] or null (one-hot drafts)
  const int* draft;           // [B, T]
  const float* u;             // [B, T + 1]
  const int* n_valid;         // [B] drafts to look at, or null (T)
  int* accepted;              // [B]
  int* tokens;                // [B, T + 1]
  int T, V;
  int piece;                  // elements per warp of the cluster (a multiple of 256)
};

__device__ __forceinline__ float vf_load(const float* x) { return __ldg(x); }
__device__ __forceinline__ float vf_load(const __nv_bfloat16* x) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(x))) << 16);
}
// The weight p - q of one token: differences that are not positive, and values that are not
// finite, weigh nothing.
__device__ __forceinline__ double vf_weight(float p, float q) {
  const double w = static_cast<double>(p) - static_cast<double>(q);
  return w > 0.0 && w <= 1.7976931348623157e308 ? w : 0.0;
}
__device__ __forceinline__ double vf_warp_sum(double x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ double vf_warp_scan(double x) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// W consecutive values of a row as floats, one 16-byte load (rows start on 16 bytes).
template <typename E>
struct VfVec;
template <>
struct VfVec<float> {
  static constexpr int W = 4, U = 4;          // values per load, loads of a row in flight
  static __device__ __forceinline__ void get(const uint4& x, float (&f)[W]) {
    f[0] = __uint_as_float(x.x); f[1] = __uint_as_float(x.y); f[2] = __uint_as_float(x.z); f[3] = __uint_as_float(x.w);
  }
};
template <>
struct VfVec<__nv_bfloat16> {
  static constexpr int W = 8, U = 2;
  static __device__ __forceinline__ void get(const uint4& x, float (&f)[W]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};

// A running sum of weights as two floats, s + c: the difference p - q (error e) and the addition
// to s (its error) are split exactly, and c collects the errors. c itself rounds: after N weights it is at
// most N 2^-24 of the sum, so off by at most N^2 2^-48 of it, and in steps of random sign by about
// N 2^-50. At N <= 256 (kVfSpan) that is 2^-32 at the very worst and 2^-42 as a rule, where a token
// weighs 2^-17; converting every value to double instead made the kernel 2.5 times slower (the
// conversions, at V = 131072).
struct VfSum {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float p, float q) {
    // the weights of vf_weight: p > q, both finite
    const bool ok = p > q && p <= 3.402823466e38f && q >= -3.402823466e38f;
    p = ok ? p : 0.f;
    q = ok ? q : 0.f;
    const float d = p - q, b = d - p, e = (p - (d - b)) - (q + b);
    const float t = s + d, z = t - s;
    c += ((s - (t - z)) + (d - z)) + e;
    s = t;
  }
  __device__ __forceinline__ double get() const { return static_cast<double>(s) + static_cast<double>(c); }
};

// Sixteen bytes that start `off` bytes into two neighbouring vectors.
__device__ __forceinline__ uint4 vf_shift(const uint4& lo, const uint4& hi, int off) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = off & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = off & 4 ? w[i + 1] : w[i];
  const int bits = (off & 3) * 8;
  return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits),
                    __funnelshift_r(w[2], w[3], bits), __funnelshift_r(w[3], w[4], bits));
}

// Sum of the weights of [v0, v1) by one warp (each lane returns its share). VEC: rows start on 16
// bytes (V a multiple of W) and come by 16-byte loads. Otherwise fp32 rows take one value per lane and
// load, eight loads in flight; for bf16 those move too few bytes: its 16-byte loads follow p's
// alignment, a vector of q is put together from the two that hold it, and the ends of the piece (fewer
// than 2 W values each), where a load would reach past the piece, go one value per lane. 64 rows of
// 131071: fp32 18.4 us by values, 21.5 by vectors; bf16 23.6 and 17.2 (16 x 50021 alone: 8.7 and 7.3).
template <typename E, bool VEC>
__device__ __forceinline__ double vf_piece(const E* p, const E* q, int hot, int v0, int v1) {
  using X = VfVec<E>;
  const int lane = threadIdx.x & 31;
  constexpr int W = X::W, U = X::U;
  VfSum sum[2];
  if constexpr (!VEC && sizeof(E) == 4) {
    constexpr int N = 8;
    for (int v = v0 + lane; v < v1; v += 32 * N) {
      float x[N], y[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int at = v + u * 32;
        x[u] = at < v1 ? vf_load(p + at) : 0.f;
        y[u] = at < v1 && q ? vf_load(q + at) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < N; ++u) sum[u & 1].add(x[u], v + u * 32 == hot ? 1.f : y[u]);
    }
    return sum[0].get() + sum[1].get();
  }
  int s0 = v0, s1 = v1, off = 0;              // whole vectors: [s0, s1); bytes q starts after one there
  if constexpr (!VEC) {
    auto past = [](const E* x) { return static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15); };
    s0 += ((16 - past(p + v0)) & 15) / static_cast<int>(sizeof(E));
    int over = 0;                             // values of q's second vector behind the last one of p
    if (q) {
      off = past(q + s0);
      const int before = off / static_cast<int>(sizeof(E));
      if (before) {
        if (s0 - before < v0) s0 += W;
        over = W - before;
      }
    }
    s1 = v1 - s0 - over >= W ? s0 + (v1 - s0 - over) / W * W : s0;
    if (s0 > v1) s0 = s1 = v1;
    for (int part = 0; part < 2; ++part) {
      const int v = (part ? s1 : v0) + lane;
      if (v < (part ? v1 : s0)) sum[part].add(vf_load(p + v), v == hot ? 1.f : q ? vf_load(q + v) : 0.f);
    }
  }
  for (int v = s0 + lane * W; v < s1; v += 32 * W * U) {
    uint4 a[U], b[U], c[VEC ? 1 : U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = v + u * 32 * W;
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
      if constexpr (!VEC) c[u] = make_uint4(0u, 0u, 0u, 0u);
      if (at < s1) {
        a[u] = __ldg(reinterpret_cast<const uint4*>(p + at));
        if constexpr (VEC) {
          if (q) b[u] = __ldg(reinterpret_cast<const uint4*>(q + at));
        } else if (q) {
          const uint4* qa = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(q + at) - off);
          b[u] = __ldg(qa);
          if (off) c[u] = __ldg(qa + 1);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (!VEC) b[u] = vf_shift(b[u], c[u], off);
      float x[W], y[W];
      X::get(a[u], x);
      X::get(b[u], y);
#pragma unroll
      for (int e = 0; e < W; ++e) sum[e & 1].add(x[e], v + u * 32 * W + e == hot ? 1.f : y[e]);
    }
  }
  return sum[0].get() + sum[1].get();
}

// Values that a warp adds before its lanes' sums move into doubles: 256 a lane and sum. Only rows beyond
// 2^20 have longer pieces (without this a row of equal weights, V = 2^27, drifted by a token).
constexpr int kVfSpan = 2 * 32 * 256;

static_assert(kVfMaxCluster * kVfWarps <= 64, "two pieces a lane");

template <typename E, bool VEC>
__global__ void __launch_bounds__(kVfThreads) verify_kernel(const VerifyParams prm) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ double s_sum[kVfMaxCluster * kVfWarps];   // every piece's sum (written by the cluster)
  __shared__ double s_scan[kVfWarps];
  __shared__ int s_acc, s_found;
  cluster.barrier_arrive();                   // every CTA has started (waited for before the first write)
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = prm.T, V = prm.V;
  const E* p0 = static_cast<const E*>(prm.p) + static_cast<long long>(b) * (T + 1) * V;
  const E* q0 = static_cast<const E*>(prm.q) + (prm.q ? static_cast<long long>(b) * T * V : 0);
  const float* u = prm.u + static_cast<long long>(b) * (T + 1);
  const int* draft = prm.draft + static_cast<long long>(b) * T;

  int n = prm.n_valid ? __ldg(prm.n_valid + b) : T;
  n = n < 0 ? 0 : (n < T ? n : T);
  if (warp == 0) {                            // the first rejected draft, 32 at a time
    int a = n;
    for (int t0 = 0; t0 < n; t0 += 32) {
      const int t = t0 + lane;
      bool no = false;
      if (t < n) {
        const int x = __ldg(draft + t);
        double px = 0.0, qx = prm.q ? 0.0 : 1.0;
        if (x >= 0 && x < V) {                // a token outside the vocabulary is rejected
          px = static_cast<double>(vf_load(p0 + static_cast<long long>(t) * V + x));
          if (prm.q) qx = static_cast<double>(vf_load(q0 + static_cast<long long>(t) * V + x));
        }
        no = !(static_cast<double>(__ldg(u + t)) * qx < px);
      }
      const unsigned any = __ballot_sync(0xffffffffu, no);
      if (any) {
        a = t0 + __ffs(any) - 1;
        break;
      }
    }
    if (lane == 0) s_acc = a;
  }
  __syncthreads();
  const int a = s_acc;
  const E* p = p0 + static_cast<long long>(a) * V;
  bool minus = a < n;                         // subtract the draft's row
  const E* q = prm.q && minus ? q0 + static_cast<long long>(a) * V : nullptr;
  int hot = minus && !prm.q ? __ldg(draft + a) : -1;
  const int pieces = C * kVfWarps, mine = rank * kVfWarps + warp;
  const int per = (pieces + 31) / 32;         // pieces a lane scans (at most 2)
  bool started = false;
  for (;;) {
    const long long v0 = static_cast<long long>(mine) * prm.piece;
    double sum = 0.0;
    const int v1 = static_cast<int>(min(v0 + prm.piece, static_cast<long long>(V)));
    for (long long at = v0; at < v1; at += kVfSpan)
      sum += vf_piece<E, VEC>(p, q, hot, static_cast<int>(at), static_cast<int>(min(at + kVfSpan, static_cast<long long>(v1))));
    sum = vf_warp_sum(sum);
    if (!started) cluster.barrier_wait();
    started = true;
    if (lane < C) *cluster.map_shared_rank(&s_sum[mine], lane) = sum;
    cluster.sync();
    // every warp scans the sums of all pieces, lane l those of pieces l per .. l per + per - 1
    double x[2], own = 0.0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = lane * per + k;
      x[k] = k < per && i < pieces ? s_sum[i] : 0.0;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) own += x[k];
    const double incl = vf_warp_scan(own);
    const double total = __shfl_sync(0xffffffffu, incl, 31);
    if (!(total > 0.0)) {
      // nothing is left of p - q (p <= q everywhere): sample p itself; p without mass: no token
      if (!minus) {
        if (rank == 0 && tid == 0) {
          prm.accepted[b] = a;
          prm.tokens[static_cast<long long>(b) * (T + 1) + a] = -1;
        }
        break;
      }
      minus = false;
      q = nullptr;
      hot = -1;
      cluster.sync();                         // the sums are read before they are written again
      continue;
    }
    const double target = static_cast<double>(__ldg(u + T)) * total;
    // the first piece whose running sum passes the target; if none does (u = 1, or the last
    // rounding), the last piece with mass
    const unsigned hit = __ballot_sync(0xffffffffu, own > 0.0 && incl > target);
    const unsigned some = __ballot_sync(0xffffffffu, own > 0.0);
    const int l = hit ? __ffs(hit) - 1 : 31 - __clz(some);
    int found = -1;
    double before = incl - own;
    {
      double at = before;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool passes = x[k] > 0.0 && (found < 0 || !hit) && (!hit || at + x[k] > target);
        if (passes) {
          found = lane * per + k;
          before = at;
        }
        at += x[k];
      }
      if (hit && found < 0) {                 // the lane's own rounding: its last piece with mass
        at = incl - own;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (x[k] > 0.0) {
            found = lane * per + k;
            before = at;
          }
          at += x[k];
        }
      }
    }
    found = __shfl_sync(0xffffffffu, found, l);
    before = __shfl_sync(0xffffffffu, before, l);
    if (found / kVfWarps == rank) {         // (the same for the whole CTA)
      // this CTA holds the piece: four consecutive tokens a thread, and so on until the running
      // sum passes the target (at the first round for a row of up to 2^16 tokens)
      const int w0 = found * prm.piece;
      const int end = static_cast<int>(min(static_cast<long long>(w0) + prm.piece, static_cast<long long>(V)));
      if (tid == 0) s_found = 0x7fffffff;
      int top = -1;                           // this thread's last token with mass
      for (int c0 = w0; c0 < end; c0 += 4 * kVfThreads) {
        const int v0 = c0 + 4 * tid;
        float pv[4], qv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int v = v0 + k;
          pv[k] = v < end ? vf_load(p + v) : 0.f;
          qv[k] = v < end && q ? vf_load(q + v) : 0.f;
        }
        double w[4], own = 0.0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = vf_weight(pv[k], v0 + k == hot ? 1.f : qv[k]);
          own += w[k];
          if (w[k] > 0.0) top = v0 + k;
        }
        const double incl = vf_warp_scan(own);
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        double at = before, all = before;
#pragma unroll
        for (int i = 0; i < kVfWarps; ++i) {
          if (i < warp) at += s_scan[i];
          all += s_scan[i];
        }
        at += incl - own;
        int hit = 0x7fffffff;
#pragma unroll
        for (int k = 3; k >= 0; --k) {
          double upto = at;
          for (int k2 = 0; k2 <= k; ++k2) upto += w[k2];
          if (w[k] > 0.0 && upto > target) hit = v0 + k;
        }
        hit = __reduce_min_sync(0xffffffffu, hit);
        if (lane == 0 && hit != 0x7fffffff) atomicMin(&s_found, hit);
        __syncthreads();
        before = all;
        if (s_found != 0x7fffffff) break;
      }
      if (s_found == 0x7fffffff) {            // the last rounding again: the piece's last token with mass
        __syncthreads();
        if (tid == 0) s_found = -1;
        __syncthreads();
        if (top >= 0) atomicMax(&s_found, top);
        __syncthreads();
      }
      if (tid == 0) {
        prm.accepted[b] = a;
        prm.tokens[static_cast<long long>(b) * (T + 1) + a] = s_found;
      }
    }
    break;
  }
  if (rank == 0) {                            // the accepted drafts, and -1 behind the new token
    for (int t = tid; t <= T; t += kVfThreads)
      if (t != a) prm.tokens[static_cast<long long>(b) * (T + 1) + t] = t < a ? __ldg(draft + t) : -1;
  }
}

}  // namespace mimo
