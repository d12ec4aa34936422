// Gated linear recurrence of channels: per (b, d), from h_0 (zeros, or a given state),
//     s_t = softplus(a_t + beta),  f_t = exp(-alpha s_t),  h_t = f_t h_{t-1} + (1 - f_t) v_t,  y_t = h_t,
// the M²RNN blend with the M²RNN gate, on a vector state and without the tanh.  Backward, with C_{T+1} = dh_T:
//     R_t = dy_t + C_{t+1},  C_t = f_t R_t,  dv_t = (1 - f_t) R_t,  G_t = C_t (h_{t-1} - v_t),
//     da_t = -alpha sigma(a_t + beta) G_t,  dalpha = -sum s G,  dbeta = sum da,  dh_0 = C_1.
//
// The recurrence is linear in h, so a stretch of steps is one map h -> P h + l with P = exp(-sum of alpha s): a
// workgroup takes a chunk of 64 steps (backward: 32) of 256 channels, 8 waves of 8 (4) steps each; a lane has 4
// neighbouring channels.  Each lane runs its steps from zero, the waves' maps are joined in LDS, and the lane runs its
// steps again from the state that enters them.  The inputs are read once: a workgroup keeps its chunk in registers until it
// knows the state that enters it.  It leaves its chunk's map in memory, and takes the maps of the chunks before it in its
// group and the state that enters the group, which the last workgroup of the group before leaves; all joins have a
// fixed order.
//
// Workgroups take chunks by a ticket, all channels of a chunk before the next chunk.  One waits only for smaller
// tickets, whose workgroups are running and do not wait for it, so every wait ends.  Each word that is waited for says
// itself whether it has been written (a clearing launch sets all bits of it), so no order of memory operations is needed.
// A wait gives up after kGatedPolls looks (seconds, where microseconds do; only a workspace that two calls share can bring it there): the
// word is then taken as it is, all bits set, so c and l are NaN, and so are the chunk's outputs and the states it hands on.
//
// Measured: 2 x 16384 steps of 2048 channels in bf16 take 131 us with the clearing launch (4.1 TB/s; VALU 80% of the cycles, which the exponentials and
// polynomials of each gate take; 260 us by three launches that read the inputs twice), the backward of 4 x 4096 steps 136 to 138 us
// (5.2 TB/s, v and a read again).
//
// Precision.  A gate next to 1 keeps its digits as i = 1 - f (a series in alpha s), and f h is then h - i h: f
// itself, rounded to fp32, would be wrong by 2^-25 the same way at every step of a constant gate, 3e-4 of the memory's
// length at i = 1e-4.  Steps with i = 0 (a masked through -infinity or the lowest number, or past the sequence's
// end) hold the state whatever v is.
#pragma once

#include "m2rnn_stream.h"

namespace m2rnn {

constexpr int kGatedWaves = 8;                        // waves of a workgroup
constexpr int kGatedStepsFwd = 8, kGatedStepsBwd = 4; // steps of a lane (128 registers: two workgroups a CU)
constexpr int kGatedGroup = 16;                       // chunks of a group at most
constexpr int kGatedLook = 8;                         // maps that are looked at together
constexpr int kGatedPolls = 1 << 22;                  // looks at a word that is waited for

struct GatedArgs {
  const void *v, *a;                 // [B,T,D]
  const float *alpha, *beta;         // [D]
  const int* lens;                   // [B] or NULL
  const float* h0;                   // [B,D] or NULL
  float *y, *h_T;                    // [B,T,D], [B,D]
  unsigned long long* maps;          // [chunks][blocks][4][64]: (P as a Decay, l) of each chunk, by channel and lane
  unsigned long long* entry;         // [groups of chunks][blocks][4][64]: the state that enters each group but the first
  unsigned* ticket;
  long cols, blocks;                 // cols = B D; blocks of 64 lanes of 4 channels
  int T, D, chunks, group;           // group: chunks of a group
  // backward
  const float *yin, *dy, *dh_T;      // the forward's y; dh_T NULL: zeros
  float *dv, *da, *dh0;
  float2* part;                      // [chunks][B D]: dalpha, dbeta of each chunk
  long first_words;                  // words that the clearing launch sets, from maps on
};

// softplus(z) and sigma(z) to a few ulp also where they are small: t = e^-|z| (the exponential's argument in two parts),
// softplus = max(z, 0) + 2 atanh(s), s = t / (2 + t) <= 1/3, atanh(s) / s in s^2 by a polynomial through the Chebyshev
// points (off by less than 2^-25).  SG: sigma too.
template <bool SG>
__device__ __forceinline__ float gated_softplus(float z, float& sg) {
  constexpr float kL = 1.4426950408889634f, kLlo = (float)(1.4426950408889634 - (double)kL);
  const float m = fminf(fabsf(z), 128.0f), x = m * -kL;
  float t = __builtin_amdgcn_exp2f(x);
  t = __builtin_fmaf(t, (__builtin_fmaf(m, -kL, -x) - m * kLlo) * 0.69314718f, t);
  const float s = t * __builtin_amdgcn_rcpf(2.0f + t), s2 = s * s, d = s + s;
  float p = __builtin_fmaf(0.13425749f, s2, 0.141183099f);
  p = __builtin_fmaf(p, s2, 0.200037803f);
  p = __builtin_fmaf(p, s2, 0.333333202f);
  if constexpr (SG) {
    const float r = __builtin_amdgcn_rcpf(1.0f + t);
    sg = z < 0.0f ? t * r : r;
  }
  return (z < 0.0f ? 0.0f : z) + __builtin_fmaf(d, s2 * p, d);  // (NaN stays NaN)
}

// What multiplies h: f itself, or -i = f - 1 where f is next to 1 (its sign bit tells them apart; a mask for each step
// of a lane would not fit the scalar registers).
struct Decay {
  float c;
  __device__ __forceinline__ float operator()(float h) const {
    return __builtin_fmaf(c, h, __float_as_int(c) < 0 ? h : 0.0f);
  }
  __device__ __forceinline__ float i() const { return __float_as_int(c) < 0 ? -c : 1.0f - c; }
};

// The decay of alpha s = x; i = 1 - f next to 1 is x times a polynomial through the Chebyshev points (2^-28).
__device__ __forceinline__ Decay decay_of(float x) {
  float p = __builtin_fmaf(0.00751360622f, x, -0.0414906541f);
  p = __builtin_fmaf(p, x, 0.166651082f);
  p = __builtin_fmaf(p, x, -0.499999515f);
  p = __builtin_fmaf(p, x, 0.999999998f);
  // (made opaque, both sides are formed and one is chosen; the compiler would branch for each value)
  const float near = opaque1(-x * p), far = opaque1(__builtin_amdgcn_exp2f(x * -1.4426950408889634f));
  Decay d;
  d.c = __float_as_uint(x) < __float_as_uint(0.25f) ? near : far;
  return d;
}

// Four neighbouring channels of an array of fp32 or bf16.
template <bool BF16>
__device__ __forceinline__ void gated_load(const void* p, long at, float (&o)[4]) {
  const float4 t = load4<BF16>(p, at);
  o[0] = t.x; o[1] = t.y; o[2] = t.z; o[3] = t.w;
}
// An array as a lane sees it: its own first element, so that a step's offset is the same in all lanes (and stays scalar).
template <bool BF16>
__device__ __forceinline__ const void* lane_base(const void* p, long base) {
  return (const char*)p + base * (BF16 ? 2 : 4);
}

// x y, and 0 where either is 0, whatever the other is.
__device__ __forceinline__ float mul_or_0(float x, float y) {
  float z;
  asm("v_mul_legacy_f32 %0, %1, %2" : "=v"(z) : "v"(x), "v"(y));
  return z;
}

// A lane's place: its 4 channels, its sequence and its steps.
struct GatedLane {
  long col;     // b D + d
  long base;    // offset of (b, 0, d)
  int d;
  int len;      // steps of the sequence
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
  int n = A.lens ? A.lens[b] : A.T;
  n = n < 0 ? 0 : n > A.T ? A.T : n;
  L.len = L.on ? n : 0;
  return L;
}

// The waves' maps in LDS by wave and channel: the sum of alpha s, P, and l, whose place the state that enters the
// wave's steps takes.
struct GatedJoin {
  float x[kGatedWaves][4][64], c[kGatedWaves][4][64], l[kGatedWaves][4][64];
  unsigned ticket;
};

// Sets the words that will be waited for and the ticket's counter.
__global__ void __launch_bounds__(kBlkThreads) m2rnn_gated_clear_kernel(GatedArgs A) {
  const long step = (long)gridDim.x * kBlkThreads;
  for (long i = (long)blockIdx.x * kBlkThreads + threadIdx.x; i < A.first_words; i += step) A.maps[i] = ~0ull;
  if (blockIdx.x == 0 && threadIdx.x == 0) *A.ticket = 0;
}

// A map or a state as a word that is not all ones: its high half is never the NaN with all bits set.
__device__ __forceinline__ unsigned long long gated_word(float c, float l) {
  const uint32_t hi = c != c ? 0x7FC00000u : __float_as_uint(c);
  return (unsigned long long)hi << 32 | __float_as_uint(l);
}
__device__ __forceinline__ void gated_put(unsigned long long* p, unsigned long long w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long gated_get(const unsigned long long* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The chunk of a workgroup in the order of the recurrence (0: first; the backward's first is the last in time), and its block.
__device__ __forceinline__ bool gated_place(const GatedArgs& A, GatedJoin& J, long& order, long& block) {
  long id = blockIdx.x;
  if (A.chunks > 1) {
    if (threadIdx.x == 0) J.ticket = atomicAdd(A.ticket, 1u);
    __syncthreads();
    id = (long)(unsigned)__builtin_amdgcn_readfirstlane((int)J.ticket);
  }
  order = id / A.blocks;
  block = id % A.blocks;
  return order < A.chunks;  // (always, unless two calls share a workspace at once)
}

// The states that enter the waves' steps to J.l, from the waves' maps (BACK: the last wave's steps are the first).
// Waves 0 to 3 take a channel each.
template <bool BACK>
__device__ __forceinline__ void gated_enter(const GatedArgs& A, GatedJoin& J, long order, long block, int lane, int w,
                                            const GatedLane& L, const float* first) {
  if (w < 4) {
    float x = 0.0f, sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kGatedWaves; ++j) {
      const int k = BACK ? kGatedWaves - 1 - j : j;
      x += J.x[k][w][lane];
      sum = Decay{J.c[k][w][lane]}(sum) + J.l[k][w][lane];
    }
    const Decay all = decay_of(x);
    const long at = (block * 4 + w) * 64, row = A.blocks * 256;
    const int group = (int)order / A.group, before = (int)order % A.group;
    const bool end = order + 1 == A.chunks, group_end = before + 1 == A.group;
    if (!end && !group_end) gated_put(A.maps + order * row + at + lane, gated_word(all.c, sum));
    float h = 0.0f;
    if (group > 0) {
      const unsigned long long* src = A.entry + group * row + at;
      unsigned long long word;
      for (int polls = 0; polls < kGatedPolls; ++polls) {
        word = gated_get(src + lane);
        if (__builtin_amdgcn_ballot_w64((uint32_t)(word >> 32) == 0xFFFFFFFFu) == 0) break;
        __builtin_amdgcn_s_sleep(1);
      }
      h = __uint_as_float((uint32_t)word);
    } else if (first && L.on) {
      h = first[L.col + w];
    }
    for (int j0 = 0; j0 < before; j0 += kGatedLook) {
      const unsigned long long* src = A.maps + ((long)group * A.group + j0) * row + at;
      unsigned long long word[kGatedLook];
      for (int polls = 0; polls < kGatedPolls; ++polls) {
        bool there = true;
#pragma unroll
        for (int j = 0; j < kGatedLook; ++j)
          if (j0 + j < before) word[j] = gated_get(src + j * row + lane);
#pragma unroll
        for (int j = 0; j < kGatedLook; ++j)
          if (j0 + j < before) there = there && (uint32_t)(word[j] >> 32) != 0xFFFFFFFFu;
        if (__builtin_amdgcn_ballot_w64(!there) == 0) break;
        __builtin_amdgcn_s_sleep(1);
      }
#pragma unroll
      for (int j = 0; j < kGatedLook; ++j)
        if (j0 + j < before)
          h = Decay{__uint_as_float((uint32_t)(word[j] >> 32))}(h) + __uint_as_float((uint32_t)word[j]);
    }
    if (group_end && !end) gated_put(A.entry + (group + 1) * row + at + lane, gated_word(0.0f, all(h) + sum));
#pragma unroll
    for (int j = 0; j < kGatedWaves; ++j) {
      const int k = BACK ? kGatedWaves - 1 - j : j;
      const float l = J.l[k][w][lane];
      J.l[k][w][lane] = h;
      h = Decay{J.c[k][w][lane]}(h) + l;
    }
  }
  __syncthreads();
}

template <bool BF16>
__global__ void __launch_bounds__(64 * kGatedWaves, 4) m2rnn_gated_fwd_kernel(GatedArgs A) {
  constexpr int NS = kGatedStepsFwd;
  __shared__ GatedJoin J;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  long chunk, block;
  if (!gated_place(A, J, chunk, block)) return;
  const GatedLane L = gated_lane(A, block);
  const int t0 = ((int)chunk * kGatedWaves + w) * NS;
  Decay dec[NS][4];
  float b[NS][4], sum[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = l[e] = 0.0f;
  const bool some = __builtin_amdgcn_ballot_w64(t0 < L.len) != 0;          // whether any lane has a step in here
  const bool all = __builtin_amdgcn_ballot_w64(t0 + NS > L.len) == 0;     // whether all lanes have all of them
  if (some) {
    float va[NS][4], al[4], be[4];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const long at = (long)(t0 + i < A.T ? t0 + i : A.T - 1) * A.D;
      gated_load<BF16>(lane_base<BF16>(A.a, L.base), at, va[i]);
      gated_load<BF16>(lane_base<BF16>(A.v, L.base), at, b[i]);
    }
    gated_load<false>(A.alpha, L.d, al);
    gated_load<false>(A.beta, L.d, be);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const bool live = t0 + i < L.len;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float sg;
        const float s = gated_softplus<false>(va[i][e] + be[e], sg);
        const float xs = opaque1(al[e] * s), x = live ? xs : 0.0f;  // (opaque: no branch)
        dec[i][e] = decay_of(x);
        b[i][e] = mul_or_0(dec[i][e].i(), b[i][e]);  // (0 times anything is 0)
        sum[e] += x;
        l[e] = dec[i][e](l[e]) + b[i][e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    J.x[w][e][lane] = sum[e];
    J.c[w][e][lane] = decay_of(sum[e]).c;
    J.l[w][e][lane] = l[e];
  }
  __syncthreads();
  gated_enter<false>(A, J, chunk, block, lane, w, L, A.h0);
  if (!L.on) return;
  float h[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = J.l[w][e][lane];
  if (all) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) h[e] = dec[i][e](h[e]) + b[i][e];
      store4_nt<false>((void*)lane_base<false>(A.y, L.base), (long)(t0 + i) * A.D, h);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int t = t0 + i;
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (some) h[e] = dec[i][e](h[e]) + b[i][e];
        o[e] = t < L.len ? h[e] : 0.0f;
      }
      if (t < A.T) store4_nt<false>((void*)lane_base<false>(A.y, L.base), (long)t * A.D, o);
    }
  }
  // the wave with the sequence's last step (its first ones, if it has none) has the state behind it: later steps hold it
  const int end = L.len > 0 ? L.len - 1 : 0;
  if (A.h_T && end >= t0 && end < t0 + NS) store4<false>(A.h_T, L.col, make_float4(h[0], h[1], h[2], h[3]));
}

template <bool BF16>
__global__ void __launch_bounds__(64 * kGatedWaves, 4) m2rnn_gated_bwd_kernel(GatedArgs A) {
  constexpr int NS = kGatedStepsBwd;
  __shared__ GatedJoin J;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  long order, block;
  if (!gated_place(A, J, order, block)) return;
  const long chunk = A.chunks - 1 - order;
  const GatedLane L = gated_lane(A, block);
  const int t0 = ((int)chunk * kGatedWaves + w) * NS;
  Decay dec[NS][4];
  float s[NS][4], sg[NS][4], u[NS][4];
  float al[4], sum[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = l[e] = 0.0f;
  const bool some = __builtin_amdgcn_ballot_w64(t0 < L.len) != 0;
  if (some) {
    float be[4];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const long at = (long)(t0 + i < A.T ? t0 + i : A.T - 1) * A.D;
      gated_load<BF16>(lane_base<BF16>(A.a, L.base), at, s[i]);
      gated_load<false>(lane_base<false>(A.dy, L.base), at, u[i]);
    }
    gated_load<false>(A.alpha, L.d, al);
    gated_load<false>(A.beta, L.d, be);
#pragma unroll
    for (int i = NS - 1; i >= 0; --i) {
      const bool live = t0 + i < L.len;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float g;
        const float p = opaque1(gated_softplus<true>(s[i][e] + be[e], g));  // (opaque: no branch)
        g = opaque1(g);
        s[i][e] = live ? p : 0.0f;
        sg[i][e] = live ? g : 0.0f;
        u[i][e] = live ? u[i][e] : 0.0f;
        const float xs = opaque1(al[e] * p), x = live ? xs : 0.0f;
        dec[i][e] = decay_of(x);
        sum[e] += x;
        l[e] = dec[i][e](l[e] + u[i][e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    J.x[w][e][lane] = sum[e];
    J.c[w][e][lane] = decay_of(sum[e]).c;
    J.l[w][e][lane] = l[e];
  }
  __syncthreads();
  gated_enter<true>(A, J, order, block, lane, w, L, A.dh_T);
  float C[4], gal[4], gbe[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    C[e] = J.l[w][e][lane];
    gal[e] = gbe[e] = 0.0f;
  }
  if (some) {
    float v[NS][4], hb[NS][4];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int t = t0 + i < A.T ? t0 + i : A.T - 1;
      gated_load<BF16>(lane_base<BF16>(A.v, L.base), (long)t * A.D, v[i]);
      if (t > 0) {
        gated_load<false>(lane_base<false>(A.yin, L.base), (long)(t - 1) * A.D, hb[i]);
      } else if (A.h0) {
        gated_load<false>(A.h0, L.col, hb[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) hb[i][e] = 0.0f;
      }
    }
#pragma unroll
    for (int i = NS - 1; i >= 0; --i) {
      const int t = t0 + i;
      float dv[4], da[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float R = C[e] + u[i][e];
        C[e] = dec[i][e](R);
        const float G = sg[i][e] == 0.0f ? 0.0f : C[e] * (hb[i][e] - v[i][e]);  // (held: whatever v is)
        dv[e] = dec[i][e].i() * R;
        da[e] = -al[e] * sg[i][e] * G;
        gal[e] = __builtin_fmaf(-s[i][e], G, gal[e]);
        gbe[e] += da[e];
      }
      if (L.on && t < A.T) {
        store4_nt<false>((void*)lane_base<false>(A.dv, L.base), (long)t * A.D, dv);
        store4_nt<false>((void*)lane_base<false>(A.da, L.base), (long)t * A.D, da);
      }
    }
  } else if (L.on) {
    const float none[4] = {0, 0, 0, 0};
    for (int i = 0; i < NS; ++i)
      if (t0 + i < A.T) {
        store4_nt<false>(A.dv, L.base + (long)(t0 + i) * A.D, none);
        store4_nt<false>(A.da, L.base + (long)(t0 + i) * A.D, none);
      }
  }
  if (A.dh0 && L.on && t0 == 0) store4<false>(A.dh0, L.col, make_float4(C[0], C[1], C[2], C[3]));
#pragma unroll
  for (int e = 0; e < 4; ++e) {  // (J.x and J.c were read before the last barrier)
    J.x[w][e][lane] = gal[e];
    J.c[w][e][lane] = gbe[e];
  }
  __syncthreads();
  if (w < 4 && L.on) {  // wave e adds channel e's sums
    float x = 0.0f, y = 0.0f;
#pragma unroll
    for (int j = 0; j < kGatedWaves; ++j) {
      x += J.x[j][w][lane];
      y += J.c[j][w][lane];
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

// A state (NULL: zeros) as it is.
__global__ void __launch_bounds__(kBlkThreads) m2rnn_gated_state_kernel(const float* from, float* to, long n) {
  const long step = (long)gridDim.x * kBlkThreads;
  for (long i = (long)blockIdx.x * kBlkThreads + threadIdx.x; i < n; i += step) to[i] = from ? from[i] : 0.0f;
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
      float sg;
      const Decay f = decay_of(al[e] * gated_softplus<false>(va[e] + be[e], sg));
      q[e] = f(hh[e]) + mul_or_0(f.i(), vv[e]);
    }
    *(float4*)(h_out + c) = o;
  }
}

}  // namespace m2rnn
