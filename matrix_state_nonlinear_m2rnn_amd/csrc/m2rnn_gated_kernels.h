// Gated linear recurrence of channels: per (b, d), from h_0 (zeros, or a given state),
//     s_t = softplus(a_t + beta),  f_t = exp(-alpha s_t),  h_t = f_t h_{t-1} + (1 - f_t) v_t,  y_t = h_t,
// the M²RNN blend with the M²RNN gate, on a vector state and without the tanh.  Backward, with C_{T+1} = dh_T:
//     R_t = dy_t + C_{t+1},  C_t = f_t R_t,  dv_t = (1 - f_t) R_t,  G_t = C_t (h_{t-1} - v_t),
//     da_t = -alpha sigma(a_t + beta) G_t,  dalpha = -sum s G,  dbeta = sum da,  dh_0 = C_1.
//
// The recurrence is linear in h, so a stretch of steps is one map h -> P h + l with P = exp(-sum of alpha s): a
// workgroup takes a chunk of 64 steps of 256 channels (8 waves of 8 steps each; a lane has 4 neighbouring channels), each
// lane runs its 8 steps from zero, the waves' maps are joined in LDS, and the lane runs its steps again from the state that
// enters them.
//
// Precision.  A gate next to 1 keeps its digits as i = 1 - f (a series in alpha s), and f h is then h - i h: f
// itself, rounded to fp32, would be wrong by 2^-25 the same way at every step of a constant gate, 3e-4 of the memory's
// length at i = 1e-4.  Steps with s = 0 (a masked through -infinity or the lowest number, or past the sequence's
// end) hold the state whatever v is.
#pragma once

#include "m2rnn_ssm_device.h"
#include "m2rnn_stream.h"

namespace m2rnn {

constexpr int kGatedSteps = 8;                         // steps of a lane
constexpr int kGatedWaves = 8;                         // waves of a workgroup
constexpr int kGatedChunk = kGatedSteps * kGatedWaves; // steps of a workgroup

struct GatedArgs {
  const void *v, *a;                 // [B,T,D]
  const float *alpha, *beta;         // [D]
  const int* lens;                   // [B] or NULL
  const float* h0;                   // [B,D] or NULL
  float *y, *h_T;                    // [B,T,D], [B,D]
  float2* agg;                       // [chunks][B D]: (sum of alpha s, l) of each chunk; then x = the state that enters it
  long T, cols;                      // cols = B D
  int D, chunks;
  // backward
  const float *yin, *dy, *dh_T;      // the forward's y; dh_T NULL: zeros
  float *dv, *da, *dh0;
  float2* part;                      // [chunks][B D]: dalpha, dbeta of each chunk
};

// What multiplies h: f itself, or i = 1 - f where it is small.
struct Decay {
  float c;
  bool near;
  __device__ __forceinline__ float operator()(float h) const { return __builtin_fmaf(c, h, near ? h : 0.0f); }
};

// The decay of alpha s = x (any sign), and i = 1 - e^-x.
__device__ __forceinline__ Decay decay_of(float x, float& i) {
  Decay d;
  d.near = fabsf(x) < 0.25f;
  // x (1 - x/2 (1 - x/3 (1 - ... x/7))): the first term left out is below 2^-29
  float p = __builtin_fmaf(x, -1.0f / 7.0f, 1.0f);
  p = __builtin_fmaf(x * (-1.0f / 6.0f), p, 1.0f);
  p = __builtin_fmaf(x * (-1.0f / 5.0f), p, 1.0f);
  p = __builtin_fmaf(x * (-1.0f / 4.0f), p, 1.0f);
  p = __builtin_fmaf(x * (-1.0f / 3.0f), p, 1.0f);
  p = __builtin_fmaf(x * (-1.0f / 2.0f), p, 1.0f);
  const float f = exp2_(x * -1.4426950408889634f);
  i = d.near ? x * p : 1.0f - f;
  d.c = d.near ? -i : f;
  return d;
}

// Four neighbouring channels of step t (read at t clamped into the tensor).
template <bool BF16>
__device__ __forceinline__ void gated_load(const void* p, long at, float (&o)[4]) {
  const float4 t = load4<BF16>(p, at);
  o[0] = t.x; o[1] = t.y; o[2] = t.z; o[3] = t.w;
}

// A lane's place: its 4 channels, its sequence and its steps.
struct GatedLane {
  long col;     // b D + d
  long base;    // offset of (b, 0, d)
  int d;
  long len;     // steps of the sequence
  bool on;
};
__device__ __forceinline__ GatedLane gated_lane(const GatedArgs& A, long block) {
  GatedLane L;
  const long c = (block * 64 + (threadIdx.x & 63)) * 4;
  L.on = c < A.cols;
  L.col = L.on ? c : 0;
  const long b = L.col / A.D;
  L.d = (int)(L.col % A.D);
  L.base = b * A.T * A.D + L.d;
  long n = A.lens ? (long)A.lens[b] : A.T;
  n = n < 0 ? 0 : n > A.T ? A.T : n;
  L.len = L.on ? n : 0;
  return L;
}

// The waves' maps in LDS: (sum of alpha s, l) by wave and channel.
struct GatedJoin {
  float x[kGatedWaves][4][64], l[kGatedWaves][4][64];
};

// OUT false: the chunks' maps to agg.  true: y, from the states that enter the chunks (agg.x).
template <bool BF16, bool OUT>
__global__ void __launch_bounds__(64 * kGatedWaves) m2rnn_gated_fwd_kernel(GatedArgs A) {
  __shared__ GatedJoin J;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const long blocks = (A.cols / 4 + 63) / 64;
  const long chunk = blockIdx.x / blocks;
  const GatedLane L = gated_lane(A, blockIdx.x % blocks);
  const long t0 = chunk * kGatedChunk + w * kGatedSteps;
  Decay dec[kGatedSteps][4];
  float b[kGatedSteps][4];
  float al[4], be[4], sum[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    al[e] = A.alpha[L.d + e];
    be[e] = A.beta[L.d + e];
    sum[e] = l[e] = 0.0f;
  }
  const bool some = __builtin_amdgcn_ballot_w64(t0 < L.len) != 0;  // whether any lane has a step in here
  if (some) {
    float va[kGatedSteps][4];
#pragma unroll
    for (int i = 0; i < kGatedSteps; ++i) {
      const long t = t0 + i < A.T ? t0 + i : A.T - 1;
      gated_load<BF16>(A.a, L.base + t * A.D, va[i]);
      gated_load<BF16>(A.v, L.base + t * A.D, b[i]);
    }
#pragma unroll
    for (int i = 0; i < kGatedSteps; ++i) {
      const bool live = t0 + i < L.len;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float s, sg, in;
        softplus_sigma(va[i][e] + be[e], s, sg);
        s = live ? s : 0.0f;
        const float x = s == 0.0f ? 0.0f : al[e] * s;
        dec[i][e] = decay_of(x, in);
        b[i][e] = s == 0.0f ? 0.0f : in * b[i][e];
        sum[e] += x;
        l[e] = dec[i][e](l[e]) + b[i][e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    J.x[w][e][lane] = sum[e];
    J.l[w][e][lane] = l[e];
  }
  __syncthreads();
  if constexpr (!OUT) {
    if (w == 0 && L.on) {
      float4 o[2];
      float* q = (float*)o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = 0.0f, h = 0.0f, in;
#pragma unroll
        for (int j = 0; j < kGatedWaves; ++j) {
          h = decay_of(J.x[j][e][lane], in)(h) + J.l[j][e][lane];
          x += J.x[j][e][lane];
        }
        q[2 * e] = x;
        q[2 * e + 1] = h;
      }
      float4* dst = (float4*)(A.agg + chunk * A.cols + L.col);
      dst[0] = o[0];
      dst[1] = o[1];
    }
    return;
  }
  if (!L.on) return;
  float h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = A.agg[chunk * A.cols + L.col + e].x;
  for (int j = 0; j < w; ++j) {
    float in;
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = decay_of(J.x[j][e][lane], in)(h[e]) + J.l[j][e][lane];
  }
#pragma unroll
  for (int i = 0; i < kGatedSteps; ++i) {
    const long t = t0 + i;
    float o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (some) h[e] = dec[i][e](h[e]) + b[i][e];
      o[e] = t < L.len ? h[e] : 0.0f;
    }
    if (t < A.T) store4_nt<false>(A.y, L.base + t * A.D, o);
  }
}

// The state that enters each chunk, from the chunks' maps (forward: from the first chunk on and h_T at the end;
// backward: from the last chunk on and dh0).  A thread per channel.
template <bool BACK>
__global__ void __launch_bounds__(kBlkThreads) m2rnn_gated_join_kernel(float2* agg, long cols, int chunks,
                                                                       const float* first, float* last) {
  const long c = (long)blockIdx.x * kBlkThreads + threadIdx.x;
  if (c >= cols) return;
  float h = first ? first[c] : 0.0f;
  for (int j = 0; j < chunks; j += 8) {
    float2 m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = j + i < chunks ? j + i : chunks - 1;
      m[i] = agg[(BACK ? chunks - 1 - k : k) * cols + c];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (j + i >= chunks) break;
      float in;
      agg[(BACK ? chunks - 1 - (j + i) : j + i) * cols + c].x = h;
      h = decay_of(m[i].x, in)(h) + m[i].y;
    }
  }
  if (last) last[c] = h;
}

// OUT false: the chunks' reverse maps C -> P C + l to agg.  true: the gradients, from the C that enter the chunks.
template <bool BF16, bool OUT>
__global__ void __launch_bounds__(64 * kGatedWaves) m2rnn_gated_bwd_kernel(GatedArgs A) {
  __shared__ GatedJoin J;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const long blocks = (A.cols / 4 + 63) / 64;
  const long chunk = blockIdx.x / blocks;
  const GatedLane L = gated_lane(A, blockIdx.x % blocks);
  const long t0 = chunk * kGatedChunk + w * kGatedSteps;
  Decay dec[kGatedSteps][4];
  float s[kGatedSteps][4], u[kGatedSteps][4], raw[kGatedSteps][4];
  float al[4], be[4], sum[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    al[e] = A.alpha[L.d + e];
    be[e] = A.beta[L.d + e];
    sum[e] = l[e] = 0.0f;
  }
  const bool some = __builtin_amdgcn_ballot_w64(t0 < L.len) != 0;
  if (some) {
#pragma unroll
    for (int i = 0; i < kGatedSteps; ++i) {
      const long t = t0 + i < A.T ? t0 + i : A.T - 1;
      gated_load<BF16>(A.a, L.base + t * A.D, raw[i]);
      gated_load<false>(A.dy, L.base + t * A.D, u[i]);
    }
#pragma unroll
    for (int i = kGatedSteps - 1; i >= 0; --i) {
      const bool live = t0 + i < L.len;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float sg, in;
        softplus_sigma(raw[i][e] + be[e], s[i][e], sg);
        s[i][e] = live ? s[i][e] : 0.0f;
        u[i][e] = live ? u[i][e] : 0.0f;
        const float x = s[i][e] == 0.0f ? 0.0f : al[e] * s[i][e];
        dec[i][e] = decay_of(x, in);
        sum[e] += x;
        l[e] = dec[i][e](l[e] + u[i][e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    J.x[w][e][lane] = sum[e];
    J.l[w][e][lane] = l[e];
  }
  __syncthreads();
  if constexpr (!OUT) {
    if (w == 0 && L.on) {
      float4 o[2];
      float* q = (float*)o;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = 0.0f, c = 0.0f, in;
#pragma unroll
        for (int j = kGatedWaves - 1; j >= 0; --j) {
          c = decay_of(J.x[j][e][lane], in)(c) + J.l[j][e][lane];
          x += J.x[j][e][lane];
        }
        q[2 * e] = x;
        q[2 * e + 1] = c;
      }
      float4* dst = (float4*)(A.agg + chunk * A.cols + L.col);
      dst[0] = o[0];
      dst[1] = o[1];
    }
    return;
  }
  float C[4], gal[4], gbe[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    C[e] = A.agg[chunk * A.cols + L.col + e].x;
    gal[e] = gbe[e] = 0.0f;
  }
  for (int j = kGatedWaves - 1; j > w; --j) {
    float in;
#pragma unroll
    for (int e = 0; e < 4; ++e) C[e] = decay_of(J.x[j][e][lane], in)(C[e]) + J.l[j][e][lane];
  }
  if (some) {
    float v[kGatedSteps][4], hb[kGatedSteps][4];
#pragma unroll
    for (int i = 0; i < kGatedSteps; ++i) {
      const long t = t0 + i < A.T ? t0 + i : A.T - 1;
      gated_load<BF16>(A.v, L.base + t * A.D, v[i]);
      if (t > 0) {
        gated_load<false>(A.yin, L.base + (t - 1) * A.D, hb[i]);
      } else if (A.h0) {
        gated_load<false>(A.h0, L.col, hb[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) hb[i][e] = 0.0f;
      }
    }
#pragma unroll
    for (int i = kGatedSteps - 1; i >= 0; --i) {
      const long t = t0 + i;
      float dv[4], da[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float sp, sg, in;
        softplus_sigma(raw[i][e] + be[e], sp, sg);
        const bool held = s[i][e] == 0.0f;
        decay_of(held ? 0.0f : al[e] * s[i][e], in);
        const float R = C[e] + u[i][e];
        C[e] = dec[i][e](R);
        const float G = held ? 0.0f : C[e] * (hb[i][e] - v[i][e]);
        dv[e] = held ? 0.0f : in * R;
        da[e] = held ? 0.0f : -al[e] * sg * G;
        gal[e] = __builtin_fmaf(-s[i][e], G, gal[e]);
        gbe[e] += da[e];
      }
      if (L.on && t < A.T) {
        store4_nt<false>(A.dv, L.base + t * A.D, dv);
        store4_nt<false>(A.da, L.base + t * A.D, da);
      }
    }
  } else if (L.on) {
    const float none[4] = {0, 0, 0, 0};
    for (int i = 0; i < kGatedSteps; ++i)
      if (t0 + i < A.T) {
        store4_nt<false>(A.dv, L.base + (t0 + i) * A.D, none);
        store4_nt<false>(A.da, L.base + (t0 + i) * A.D, none);
      }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    J.x[w][e][lane] = gal[e];
    J.l[w][e][lane] = gbe[e];
  }
  __syncthreads();
  if (w < 4 && L.on) {  // wave e adds channel e's sums
    float x = 0.0f, y = 0.0f;
#pragma unroll
    for (int j = 0; j < kGatedWaves; ++j) {
      x += J.x[j][w][lane];
      y += J.l[j][w][lane];
    }
    A.part[chunk * A.cols + L.col + w] = make_float2(x, y);
  }
}

// dalpha and dbeta: the chunks' and the batch's partial sums of a channel, in fp64 and in a fixed order.  A
// workgroup takes 16 channels, 64 threads every 64th row each.
__global__ void __launch_bounds__(1024) m2rnn_gated_sums_kernel(const float2* __restrict__ part, long rows, int D,
                                                                float* __restrict__ dalpha, float* __restrict__ dbeta) {
  __shared__ double ra[64][17], rb[64][17];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int d = blockIdx.x * 16 + col;
  double x = 0.0, y = 0.0;
  if (d < D) {
#pragma unroll 4
    for (long p = row; p < rows; p += 64) {
      const float2 t = part[p * D + d];
      x += (double)t.x;
      y += (double)t.y;
    }
  }
  ra[row][col] = x;
  rb[row][col] = y;
  __syncthreads();
  if (threadIdx.x < 32) {
    const int c = threadIdx.x & 15, j = blockIdx.x * 16 + c;
    if (j < D) {
      double t = 0.0;
      for (int i = 0; i < 64; ++i) t += threadIdx.x < 16 ? ra[i][c] : rb[i][c];
      (threadIdx.x < 16 ? dalpha : dbeta)[j] = (float)t;
    }
  }
}

// One step: h_out = f h + (1 - f) v, four channels a thread.
template <bool BF16>
__global__ void __launch_bounds__(kBlkThreads) m2rnn_gated_step_kernel(const void* v, const void* a, const float* alpha,
                                                                       const float* beta, const float* h, float* h_out,
                                                                       long cols, int D) {
  const long step = (long)gridDim.x * kBlkThreads * 4;
  for (long c = ((long)blockIdx.x * kBlkThreads + threadIdx.x) * 4; c < cols; c += step) {
    const int d = (int)(c % D);
    float va[4], vv[4], hh[4] = {0, 0, 0, 0}, al[4], be[4];
    gated_load<BF16>(a, c, va);
    gated_load<BF16>(v, c, vv);
    if (h) gated_load<false>(h, c, hh);
    gated_load<false>(alpha, d, al);
    gated_load<false>(beta, d, be);
    float4 o;
    float* q = (float*)&o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float s, sg, in;
      softplus_sigma(va[e] + be[e], s, sg);
      const Decay f = decay_of(s == 0.0f ? 0.0f : al[e] * s, in);
      q[e] = f(hh[e]) + (s == 0.0f ? 0.0f : in * vv[e]);
    }
    *(float4*)(h_out + c) = o;
  }
}

}  // namespace m2rnn
