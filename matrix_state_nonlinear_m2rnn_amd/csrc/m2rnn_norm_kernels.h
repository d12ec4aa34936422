// The entry of a layer: the residual stream takes the branch's output, and the sum is normalised for the next branch,
//     h = res + x (rounded to the stream's type),   out = gamma (.) h / sqrt(mean_j h_j^2 + eps),
// the output in fp32, bf16, or e4m3 with one scale for each group of features: s = max(amax |out| / 448, 2^-126),
// q = out / s rounded to nearest even (448 is the largest e4m3 number).  The norm is of h as it is kept, so the
// backward, which reads h alone, differentiates what the forward computed:
//     p = gamma (.) dout,   dx = dres = r p - (r^2 sum_j(p_j h_j) / D) (r h) + dh,   dgamma = sum dout (.) (r h),
// r = 1 / sqrt(mean h^2 + eps) and dh the gradient that reaches h down the stream.
//
// HBM streams: a row is read once and kept in registers between its sums and its scaling.  LPR lanes hold a row
// (several rows a wave for narrow ones, a wave or a workgroup for wide ones), a lane 8 neighbouring features at a time, so a
// group of 128 features is 16 lanes (4 at a time, and half a wave, where something read is fp32, D is no multiple of 8, rows are
// narrow, and in the backward).
//
// Measured, rows of 2048: 32768 bf16 rows into an fp32 stream 135 us (6.0 TB/s), into a bf16 stream and out to e4m3 80 us
// (5.9 TB/s); the backward of 16384 rows 97 us and 4 us for dgamma's sums (5.6 TB/s); 128 rows 4 to 5 us.
#pragma once

#include "m2rnn_stream.h"

namespace m2rnn {

struct NormArgs {
  const void *x, *res;  // [rows, D]; res NULL: h = x
  const float* gamma;   // [D]
  void *h, *out;        // h NULL: not kept
  float* scale;         // e4m3: [rows, D / group]
  long rows;
  int D, group;
  bool x_bf16, res_bf16, out_bf16;
  float eps;
};

struct NormBwdArgs {
  const void* h;             // [rows, D]
  const float *gamma, *dout, *dh;  // dh NULL: zeros
  float* dx;
  float* part;               // [workgroups][D] partial sums of dgamma
  long rows;
  int D;
  bool h_bf16;
  float eps;
};

// Sum over the LPR lanes that hold a row, in each of them; 256 lanes: the whole workgroup through LDS.
template <int LPR>
__device__ __forceinline__ float row_sum(float x, float (&red)[2][kBlkThreads / 64], int which) {
  x += dpp_all<kDppQuadXor1>(x);
  x += dpp_all<kDppQuadXor2>(x);
  if constexpr (LPR >= 16) {
    x += dpp_all<kDppRowHalfMirror>(x);
    x += dpp_all<kDppRowMirror>(x);
  }
  if constexpr (LPR >= 64) {
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
  }
  if constexpr (LPR == 256) {
    if ((threadIdx.x & 63) == 0) red[which][threadIdx.x >> 6] = x;
    __syncthreads();
    x = (red[which][0] + red[which][1]) + (red[which][2] + red[which][3]);
  }
  return x;
}

__device__ __forceinline__ uint32_t umax_(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest of the magnitudes' bits over half a wave (a group of 128) or over the whole row.  As whole numbers NaN
// is larger than every magnitude, so it is not lost.
template <int CTRL>
__device__ __forceinline__ uint32_t max_with(uint32_t m) {
  return umax_(m, __float_as_uint(dpp_all<CTRL>(__uint_as_float(m))));
}
__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
  m = max_with<kDppQuadXor1>(m);
  m = max_with<kDppQuadXor2>(m);
  m = max_with<kDppRowHalfMirror>(m);
  return max_with<kDppRowMirror>(m);
}
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  m = row16_max(m);
  return umax_(m, (uint32_t)__shfl_xor((int)m, 16));
}
template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t (&red)[kBlkThreads / 64]) {
  if constexpr (LPR == 4) return max_with<kDppQuadXor2>(max_with<kDppQuadXor1>(m));
  m = row16_max(m);
  if constexpr (LPR >= 64) {
    m = umax_(m, (uint32_t)__shfl_xor((int)m, 16));
    m = umax_(m, (uint32_t)__shfl_xor((int)m, 32));
  }
  if constexpr (LPR == 256) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = umax_(umax_(red[0], red[1]), umax_(red[2], red[3]));
  }
  return m;
}

__device__ __forceinline__ float e4m3_scale(uint32_t amax_bits) {
  const float s = __uint_as_float(amax_bits) / 448.0f;
  return s < 0x1p-126f ? 0x1p-126f : s;  // (NaN stays NaN)
}
// Four values over s as e4m3, in one word: times 1/s with the product's error taken out.
__device__ __forceinline__ uint32_t pack_e4m3(const float (&y)[4], float s, float inv) {
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float t = y[e] * inv;
    q[e] = __builtin_fmaf(__builtin_fmaf(-t, s, y[e]), inv, t);
  }
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
}

template <int NG, int LPR>
__device__ __forceinline__ void load_row(float (&o)[NG][4], const void* p, bool bf16, long at, int unit, int D) {
  if (bf16) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int i = 4 * (g * LPR + unit);
      float4 t = make_float4(0, 0, 0, 0);
      if (i < D) t = load4_nt<true>(p, at + i);
      o[g][0] = t.x; o[g][1] = t.y; o[g][2] = t.z; o[g][3] = t.w;
    }
  } else {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int i = 4 * (g * LPR + unit);
      float4 t = make_float4(0, 0, 0, 0);
      if (i < D) t = load4_nt<false>(p, at + i);
      o[g][0] = t.x; o[g][1] = t.y; o[g][2] = t.z; o[g][3] = t.w;
    }
  }
}
template <int NG, int LPR>
__device__ __forceinline__ void store_row(const float (&v)[NG][4], void* p, bool bf16, long at, int unit, int D) {
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int i = 4 * (g * LPR + unit);
    if (i >= D) continue;
    if (bf16)
      store4_nt<true>(p, at + i, v[g]);
    else
      store4_nt<false>(p, at + i, v[g]);
  }
}

template <int LPR, int NG, bool Q8>
__global__ void __launch_bounds__(kBlkThreads) m2rnn_add_norm_kernel(NormArgs A) {
  constexpr int RPB = kBlkThreads / LPR;  // rows per workgroup
  __shared__ float red[2][kBlkThreads / 64];
  __shared__ uint32_t redm[kBlkThreads / 64];
  const int unit = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float gm[NG][4];
  load_row<NG, LPR>(gm, A.gamma, false, 0, unit, A.D);
  const float inv = 1.0f / (float)A.D;
  int turn = 0;
  for (long r0 = (long)blockIdx.x * RPB; r0 < A.rows; r0 += (long)gridDim.x * RPB, turn ^= 1) {
    const bool on = r0 + sub < A.rows;
    const long row = on ? r0 + sub : A.rows - 1;  // (lanes without a row take the last one and store nothing)
    const long at = row * A.D;
    float h[NG][4];
    load_row<NG, LPR>(h, A.x, A.x_bf16, at, unit, A.D);
    if (A.res) {
      float t[NG][4];
      load_row<NG, LPR>(t, A.res, A.res_bf16, at, unit, A.D);
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[g][e] += t[g][e];
          if (A.res_bf16) h[g][e] = (float)(__bf16)h[g][e];
        }
      if (A.h && on) store_row<NG, LPR>(h, A.h, A.res_bf16, at, unit, A.D);
    }
    float ss = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = __builtin_fmaf(h[g][e], h[g][e], ss);
    const float r = 1.0f / sqrtf(row_sum<LPR>(ss, red, turn) * inv + A.eps);
    uint32_t most = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[g][e] = h[g][e] * r * gm[g][e];
        if constexpr (Q8) most = umax_(most, __float_as_uint(h[g][e]) & 0x7FFFFFFFu);
      }
    if constexpr (!Q8) {
      if (on) store_row<NG, LPR>(h, A.out, A.out_bf16, at, unit, A.D);
    } else {
      uint32_t* q = (uint32_t*)A.out;
      if (A.group == A.D) {
        const float s = e4m3_scale(row_max<LPR>(most, redm)), si = 1.0f / s;  // (the next row writes redm behind row_sum's barrier)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int i = 4 * (g * LPR + unit);
          if (on && i < A.D) q[(at + i) / 4] = pack_e4m3(h[g], s, si);
        }
        if (on && unit == 0) A.scale[row] = s;
      } else {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int i = 4 * (g * LPR + unit);
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) m = umax_(m, __float_as_uint(h[g][e]) & 0x7FFFFFFFu);
          const float s = e4m3_scale(group_max(m)), si = 1.0f / s;
          if (on && i < A.D) {
            q[(at + i) / 4] = pack_e4m3(h[g], s, si);
            if ((unit & 31) == 0) A.scale[row * (A.D / 128) + i / 128] = s;
          }
        }
      }
    }
  }
}

// Eight neighbouring bf16 values as they are in memory.
struct Raw8 {
  uint4 w;
  __device__ __forceinline__ void load(const void* p, long at) {
    typedef unsigned u4v __attribute__((ext_vector_type(4)));
    const u4v t = __builtin_nontemporal_load((const u4v*)((const uint16_t*)p + at));
    w = make_uint4(t[0], t[1], t[2], t[3]);
  }
  __device__ __forceinline__ float operator[](int e) const {
    const uint32_t u = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
    return e & 1 ? bf16_hi_to_f32(u) : bf16_lo_to_f32(u);
  }
};
__device__ __forceinline__ void store8_nt(void* p, bool bf16, long at, const float (&v)[8]) {
  typedef unsigned u4v __attribute__((ext_vector_type(4)));
  if (bf16) {
    const u4v w = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    __builtin_nontemporal_store(w, (u4v*)((uint16_t*)p + at));
  } else {
    const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    __builtin_nontemporal_store(a, (f32x4*)((float*)p + at));
    __builtin_nontemporal_store(b, (f32x4*)((float*)p + at) + 1);
  }
}

// The same for bf16 inputs: 8 features at a time, and a row's loads in flight beside the row before's sums and stores (a
// bf16 row has half the bytes: without this 32768 rows of 2048 in bf16 took 165 us, nearly as long as in fp32).
template <int LPR, int NG, bool RES, bool Q8>
__global__ void __launch_bounds__(kBlkThreads) m2rnn_add_norm8_kernel(NormArgs A) {
  constexpr int RPB = kBlkThreads / LPR;
  __shared__ float red[2][kBlkThreads / 64];
  __shared__ uint32_t redm[kBlkThreads / 64];
  const int unit = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float gm[NG][8];
  Raw8 x[NG] = {}, res[RES ? NG : 1] = {};
  auto fetch = [&](long row) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int i = 8 * (g * LPR + unit);
      if (i < A.D) {
        x[g].load(A.x, row * A.D + i);
        if constexpr (RES) res[g].load(A.res, row * A.D + i);
      }
    }
  };
  long r0 = (long)blockIdx.x * RPB;
  const long step = (long)gridDim.x * RPB;
  fetch(r0 + sub < A.rows ? r0 + sub : A.rows - 1);  // (lanes without a row take the last one and store nothing)
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) gm[g][e] = 8 * (g * LPR + unit) < A.D ? A.gamma[8 * (g * LPR + unit) + e] : 0.0f;
  const float inv = 1.0f / (float)A.D;
  for (int turn = 0; r0 < A.rows; r0 += step, turn ^= 1) {
    const bool on = r0 + sub < A.rows;
    const long row = on ? r0 + sub : A.rows - 1, at = row * A.D;
    float h[NG][8], ss = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[g][e] = x[g][e];
        if constexpr (RES) h[g][e] = (float)(__bf16)(h[g][e] + res[g][e]);
        ss = __builtin_fmaf(h[g][e], h[g][e], ss);
      }
    if (r0 + step < A.rows) fetch(r0 + step + sub < A.rows ? r0 + step + sub : A.rows - 1);
    if (RES && A.h && on) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (8 * (g * LPR + unit) < A.D) store8_nt(A.h, true, at + 8 * (g * LPR + unit), h[g]);
    }
    const float r = 1.0f / sqrtf(row_sum<LPR>(ss, red, turn) * inv + A.eps);
    uint32_t most[NG], all = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      most[g] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[g][e] = h[g][e] * r * gm[g][e];
        if constexpr (Q8) most[g] = umax_(most[g], __float_as_uint(h[g][e]) & 0x7FFFFFFFu);
      }
      all = umax_(all, most[g]);
    }
    if constexpr (!Q8) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (on && 8 * (g * LPR + unit) < A.D) store8_nt(A.out, A.out_bf16, at + 8 * (g * LPR + unit), h[g]);
    } else {
      const bool whole = A.group == A.D;
      float s = 0.0f, si = 0.0f;
      if (whole) {
        s = e4m3_scale(row_max<LPR>(all, redm));  // (the next row writes redm behind row_sum's barrier)
        si = 1.0f / s;
        if (on && unit == 0) A.scale[row] = s;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int i = 8 * (g * LPR + unit);
        if (!whole) {
          s = e4m3_scale(row16_max(most[g]));
          si = 1.0f / s;
          if (on && i < A.D && (unit & 15) == 0) A.scale[row * (A.D / 128) + i / 128] = s;
        }
        const float lo[4] = {h[g][0], h[g][1], h[g][2], h[g][3]}, hi[4] = {h[g][4], h[g][5], h[g][6], h[g][7]};
        if (on && i < A.D) *(uint2*)((uint8_t*)A.out + at + i) = make_uint2(pack_e4m3(lo, s, si), pack_e4m3(hi, s, si));
      }
    }
  }
}

template <int LPR, int NG>
__global__ void __launch_bounds__(kBlkThreads) m2rnn_add_norm_bwd_kernel(NormBwdArgs A) {
  constexpr int RPB = kBlkThreads / LPR;
  __shared__ float red[2][kBlkThreads / 64], red2[2][kBlkThreads / 64];
  __shared__ float cols[RPB][4 * LPR];
  const int unit = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  float gm[NG][4], dg[NG][4];
  load_row<NG, LPR>(gm, A.gamma, false, 0, unit, A.D);
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int e = 0; e < 4; ++e) dg[g][e] = 0.0f;
  const float inv = 1.0f / (float)A.D;
  int turn = 0;
  for (long r0 = (long)blockIdx.x * RPB; r0 < A.rows; r0 += (long)gridDim.x * RPB, turn ^= 1) {
    const bool on = r0 + sub < A.rows;
    const long at = (on ? r0 + sub : A.rows - 1) * A.D;
    float h[NG][4], p[NG][4];
    load_row<NG, LPR>(h, A.h, A.h_bf16, at, unit, A.D);
    load_row<NG, LPR>(p, A.dout, false, at, unit, A.D);
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ss = __builtin_fmaf(h[g][e], h[g][e], ss);
        dot = __builtin_fmaf(p[g][e] * gm[g][e], h[g][e], dot);
      }
    const float r = 1.0f / sqrtf(row_sum<LPR>(ss, red, turn) * inv + A.eps);
    const float m = row_sum<LPR>(dot, red2, turn) * inv * r * r;
    float dh[NG][4];
    if (A.dh) {
      load_row<NG, LPR>(dh, A.dh, false, at, unit, A.D);
    } else {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e) dh[g][e] = 0.0f;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float hn = h[g][e] * r;
        if (on) dg[g][e] = __builtin_fmaf(p[g][e], hn, dg[g][e]);
        h[g][e] = __builtin_fmaf(r, p[g][e] * gm[g][e], __builtin_fmaf(-m, hn, dh[g][e]));
      }
    if (on) store_row<NG, LPR>(h, A.dx, false, at, unit, A.D);
  }
  // the workgroup's sums, its rows in a fixed order
  if constexpr (LPR == 256) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int i = 4 * (g * LPR + unit);
      if (i < A.D) store4<false>(A.part, (long)blockIdx.x * A.D + i, make_float4(dg[g][0], dg[g][1], dg[g][2], dg[g][3]));
    }
  } else {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int e = 0; e < 4; ++e) cols[sub][4 * unit + e] = dg[g][e];
      __syncthreads();
      for (int j = threadIdx.x; j < 4 * LPR && 4 * g * LPR + j < A.D; j += kBlkThreads) {
        float t = 0.0f;
#pragma unroll
        for (int s = 0; s < RPB; ++s) t += cols[s][j];
        A.part[(long)blockIdx.x * A.D + 4 * g * LPR + j] = t;
      }
      __syncthreads();
    }
  }
}

// dgamma from the workgroups' `parts` rows of D partial sums, in fp64 and in a fixed order: a workgroup takes 16
// columns (64 bytes of a row), 64 threads every 64th row each.
__global__ void __launch_bounds__(1024) m2rnn_norm_sums_kernel(const float* __restrict__ part, long parts, int D,
                                                               float* __restrict__ dgamma) {
  __shared__ double red[64][17];
  const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int j = blockIdx.x * 16 + col;
  double acc = 0.0;
  if (j < D) {
#pragma unroll 8
    for (long p = row; p < parts; p += 64) acc += (double)part[p * D + j];
  }
  red[row][col] = acc;
  __syncthreads();
  if (threadIdx.x < 16 && j < D) {
    double t = 0.0;
#pragma unroll 16
    for (int i = 0; i < 64; ++i) t += red[i][threadIdx.x];
    dgamma[j] = (float)t;
  }
}

}  // namespace m2rnn
