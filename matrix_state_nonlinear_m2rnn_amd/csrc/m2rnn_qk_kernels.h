// Norm of queries and keys per head with the position rotation in the same pass:
//     xn = gamma (.) x / sqrt(mean_j x_j^2 + eps)           over the K features of one head,
//     (xn_a, xn_b) -> (xn_a cos t - xn_b sin t, xn_b cos t + xn_a sin t),   t = pos * inv_freq[p],
// for the pairs p < R/2 of each head (a = p, b = p + R/2, or interleaved a = 2p, b = 2p + 1); the K - R last
// features are normalised only.  Backward: gn = the upstream gradient rotated by -t, p = gamma gn,
//     dx = r p - (r^2 sum_j(p_j x_j) / K) (r x),   dgamma = sum gn x r,   r = 1 / sqrt(mean x^2 + eps)
// (no r^3: rows of 1e15 keep their projection, rows of zeros with a tiny eps stay finite).
//
// An HBM stream: each value is read and written once.  A lane holds 4 pairs (8 features) of a head, so
// the rotation needs no other lane; K/8 lanes (rounded up to a power of two) hold a head and sum its
// squares; a wave takes 64/lanes heads of one token at a time, the queries' heads first, then the
// keys', and forms its pairs' sines and cosines once per token.  Angles are reduced to a quarter turn
// in fp64 (a position of a million times the first frequency leaves no bit of an fp32 angle), then
// the two series run in fp32.
//
// Measured: B2 T16384, 32 + 32 heads, K = R = 64, bf16: 104 to 108 us for 0.54 GB, 5.0 to 5.2 TB/s, the rate of a large
// copy (4.8 to 5.0); the backward at B4 T4096, 16 + 16 heads, K = 128: 114 to 120 us and 5 us of sums, 5.6 TB/s.
// Eight pairs a lane took 121 us, more waves or a prefetched next head no less.
#pragma once

#include "m2rnn_stream.h"

namespace m2rnn {

struct QkArgs {
  const void *q, *k;              // [B,T,Nq,K], [B,T,Nk,K]
  const float *gq, *gk;           // gamma [K]
  const int* pos;                 // [B,T]
  const double* freq;             // [R/2]
  const float *dqo, *dko;         // backward: upstream [B,T,Nq,K], [B,T,Nk,K]
  void *qo, *ko;                  // forward: outputs in the inputs' type; backward: dq, dk (fp32)
  float* part;                    // backward: [workgroups][2K] partials of dgamma_q, dgamma_k
  long tokens;                    // B T
  int Nq, Nk, K, half;            // half = R/2
  int split;                      // waves per token
  float eps;
};

// cos and sin of pos * freq.
__device__ __forceinline__ void qk_angle(double pos, double freq, float& c, float& s) {
  const double turns = pos * freq * 0.15915494309189533577;  // 1 / (2 pi)
  const double quarter = __builtin_rint(turns * 4.0);
  const float x = (float)((turns - quarter * 0.25) * 6.283185307179586477);  // |x| <= pi/4
  const float x2 = x * x;
  // Taylor series: the first terms left out are below 2^-29 (sin) and 2^-32 (cos) at pi/4
  float ss = 1.0f / 362880.0f;
  ss = __builtin_fmaf(ss, x2, -1.0f / 5040.0f);
  ss = __builtin_fmaf(ss, x2, 1.0f / 120.0f);
  ss = __builtin_fmaf(ss, x2, -1.0f / 6.0f);
  ss = __builtin_fmaf(ss * x2, x, x);
  float cc = -1.0f / 3628800.0f;
  cc = __builtin_fmaf(cc, x2, 1.0f / 40320.0f);
  cc = __builtin_fmaf(cc, x2, -1.0f / 720.0f);
  cc = __builtin_fmaf(cc, x2, 1.0f / 24.0f);
  cc = __builtin_fmaf(cc, x2, -0.5f);
  cc = __builtin_fmaf(cc, x2, 1.0f);
  const int n = (int)(long)quarter;
  const float a = (n & 1) ? ss : cc, b = (n & 1) ? cc : ss;
  c = ((n + 1) & 2) ? -a : a;
  s = (n & 2) ? -b : b;
}

// Sum over the LPH lanes (a power of two, aligned) that hold one head, in each of them.
template <int LPH>
__device__ __forceinline__ float head_sum(float x) {
  if constexpr (LPH >= 2) x += dpp_all<kDppQuadXor1>(x);
  if constexpr (LPH >= 4) x += dpp_all<kDppQuadXor2>(x);
  if constexpr (LPH >= 8) x += dpp_all<kDppRowHalfMirror>(x);
  if constexpr (LPH >= 16) x += dpp_all<kDppRowMirror>(x);
  if constexpr (LPH >= 32) x += __shfl_xor(x, 16);
  return x;
}

// (x[i], x[4 + i]) (or neighbours, interleaved) rotated by the angles; sign -1: the other way.
template <bool INTER>
__device__ __forceinline__ void qk_turn(const float (&x)[8], const float (&c)[4], const float (&s)[4], float sign,
                                        float (&o)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = INTER ? 2 * i : i, b = INTER ? 2 * i + 1 : 4 + i;
    const float t = sign * s[i];
    o[a] = x[a] * c[i] - x[b] * t;
    o[b] = x[b] * c[i] + x[a] * t;
  }
}

template <bool BF16, int LPH, bool INTER, bool BWD>
__global__ void __launch_bounds__(kBlkThreads) m2rnn_qk_norm_rope_kernel(QkArgs A) {
  constexpr int HPW = 64 / LPH;  // heads at a time
  const int lane = threadIdx.x & 63;
  const int unit = lane % LPH, sub = lane / LPH;
  const bool on = unit * 8 < A.K;
  // this lane's features: o1 .. o1 + 3 and o2 .. o2 + 3; pairs past half stay as they are
  const int p0 = 4 * unit;
  const bool turns = on && p0 < A.half;
  const int o1 = (!INTER && turns) ? p0 : 8 * unit, o2 = (!INTER && turns) ? p0 + A.half : 8 * unit + 4;
  float gq[8], gk[8], aq[8], ak[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) gq[i] = gk[i] = aq[i] = ak[i] = 0.0f;
  double fr[4] = {0.0, 0.0, 0.0, 0.0};
  if (on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      gq[i] = A.gq[o1 + i];
      gq[4 + i] = A.gq[o2 + i];
      gk[i] = A.gk[o1 + i];
      gk[4 + i] = A.gk[o2 + i];
      if (turns) fr[i] = A.freq[p0 + i];
    }
  }
  const int heads = A.Nq + A.Nk;
  const float inv = 1.0f / (float)A.K;
  const long waves = (long)gridDim.x * (kBlkThreads / 64);
  const long work = A.tokens * A.split;
  for (long j = (long)blockIdx.x * (kBlkThreads / 64) + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); j < work;
       j += waves) {
    const long tok = j / A.split;
    const int part = (int)(j % A.split);
    float c[4] = {1, 1, 1, 1}, s[4] = {0, 0, 0, 0};
    const double pos = (double)A.pos[tok];
    if (turns) {
#pragma unroll
      for (int i = 0; i < 4; ++i) qk_angle(pos, fr[i], c[i], s[i]);
    }
    for (int h0 = part * HPW; h0 < heads; h0 += A.split * HPW) {
      const int h = h0 + sub;
      const bool live = on && h < heads, isq = h < A.Nq;
      const long at = isq ? (tok * A.Nq + h) * A.K : (tok * A.Nk + (h - A.Nq)) * A.K;
      float x[8] = {0, 0, 0, 0, 0, 0, 0, 0}, g[8], gm[8];
      if (live) {  // (plain loads: the two 8-byte pieces of a lane share lines; non-temporal ones took 120 us, not 110)
        const void* src = isq ? A.q : A.k;
        const float4 x1 = load4<BF16>(src, at + o1), x2 = load4<BF16>(src, at + o2);
        x[0] = x1.x; x[1] = x1.y; x[2] = x1.z; x[3] = x1.w;
        x[4] = x2.x; x[5] = x2.y; x[6] = x2.z; x[7] = x2.w;
      }
      if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = 0.0f;
        if (live) {
          const float* src = isq ? A.dqo : A.dko;
          const float4 g1 = load4_nt<false>(src, at + o1), g2 = load4_nt<false>(src, at + o2);
          g[0] = g1.x; g[1] = g1.y; g[2] = g1.z; g[3] = g1.w;
          g[4] = g2.x; g[5] = g2.y; g[6] = g2.z; g[7] = g2.w;
        }
      }
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = __builtin_fmaf(x[i], x[i], ss);
        gm[i] = isq ? gq[i] : gk[i];
      }
      const float root = sqrtf(head_sum<LPH>(ss) * inv + A.eps);
      const float r = live ? 1.0f / root : 0.0f;  // (eps = 0: lanes without a feature would add 0 times infinity)
      float y[8], o[8];
      if constexpr (!BWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[i] * r * gm[i];
        qk_turn<INTER>(y, c, s, 1.0f, o);
        if (live) {
          void* dst = isq ? A.qo : A.ko;
          const float a4[4] = {o[0], o[1], o[2], o[3]}, b4[4] = {o[4], o[5], o[6], o[7]};
          store4_nt<BF16>(dst, at + o1, a4);
          store4_nt<BF16>(dst, at + o2, b4);
        }
      } else {
        qk_turn<INTER>(g, c, s, -1.0f, y);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float t = y[i] * x[i] * r;
          aq[i] += isq ? t : 0.0f;
          ak[i] += isq ? 0.0f : t;
          y[i] *= gm[i];
          dot = __builtin_fmaf(y[i], x[i], dot);
        }
        const float m = head_sum<LPH>(dot) * inv * r * r;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __builtin_fmaf(r, y[i], -(m * (x[i] * r)));
        if (live) {
          float* dst = (float*)(isq ? A.qo : A.ko);
          const float a4[4] = {o[0], o[1], o[2], o[3]}, b4[4] = {o[4], o[5], o[6], o[7]};
          store4_nt<false>(dst, at + o1, a4);
          store4_nt<false>(dst, at + o2, b4);
        }
      }
    }
  }
  if constexpr (BWD) {
    // the workgroup's sums: lanes of the same unit, then its waves, in a fixed order.  A lane's own sums (of 64
    // heads at most, by the launch plan) and these are fp32, the rows of the workgroups are added in fp64.
    __shared__ float red[kBlkThreads / 64][2][8 * LPH];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int d = LPH; d < 64; d <<= 1) {
        aq[i] += __shfl_xor(aq[i], d);
        ak[i] += __shfl_xor(ak[i], d);
      }
      if (sub == 0) {
        red[threadIdx.x >> 6][0][8 * unit + i] = aq[i];
        red[threadIdx.x >> 6][1][8 * unit + i] = ak[i];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * 8 * LPH; e += kBlkThreads) {
      const int which = e / (8 * LPH), i = e % (8 * LPH), u = i / 8, f = i % 8;
      if (u * 8 >= A.K) continue;
      float t = 0.0f;
#pragma unroll
      for (int wv = 0; wv < kBlkThreads / 64; ++wv) t += red[wv][which][i];
      const bool tu = 4 * u < A.half;
      const int a = (!INTER && tu) ? 4 * u : 8 * u, b = (!INTER && tu) ? 4 * u + A.half : 8 * u + 4;
      A.part[((long)blockIdx.x * 2 + which) * A.K + (f < 4 ? a + f : b + f - 4)] = t;
    }
  }
}

// dgamma_q and dgamma_k from the workgroups' `parts` rows of 2K partial sums: a workgroup takes 16 columns
// (64 bytes of a row), 64 threads every 64th row each, in fp64 and in a fixed order.  One launch of 5 us at
// 1024 rows of 256 columns (the block operators' tree of slices takes two launches of 5 us each).
__global__ void __launch_bounds__(1024) m2rnn_qk_sums_kernel(const float* __restrict__ part, long parts, int K,
                                                             float* __restrict__ dgq, float* __restrict__ dgk) {
  __shared__ double red[64][17];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int j = blockIdx.x * 16 + col;  // 2K is a multiple of 16
  double acc = 0.0;
#pragma unroll 16
  for (long p = row; p < parts; p += 64) acc += (double)part[p * 2 * K + j];
  red[row][col] = acc;
  __syncthreads();
  if (threadIdx.x < 16) {
    double t = 0.0;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) t += red[i][threadIdx.x];
    if (j < K)
      dgq[j] = (float)t;
    else
      dgk[j - K] = (float)t;
  }
}

}  // namespace m2rnn
