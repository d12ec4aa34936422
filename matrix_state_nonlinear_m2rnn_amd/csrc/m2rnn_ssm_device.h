// Device-side building blocks of the selective state space scan (m2rnn_ssm_*): the chunk's decays,
// exact splits of fp32 values into bf16 planes, LDS operand reads and the chunk staging.
//
// Mathematics.  Per (b, n), with D_t = softplus(a_t + beta) and f_t = exp(-alpha D_t),
//     H_t = f_t H_{t-1} + D_t k_t v_t^T,      y_t = H_t^T q_t + w_r (.) v_t.
// Unlike the M²RNN recurrence this one is linear in H, so a chunk of L steps is a handful of matrix
// products.  With c_i = sum_{t <= i} ln f_t inside the chunk and H the state that enters it,
//     y_i  = e^{c_i} H^T q_i + sum_{j <= i} e^{c_i - c_j} D_j (q_i . k_j) v_j + w_r (.) v_i
//     H'   = e^{c_L} H + sum_j e^{c_L - c_j} D_j k_j v_j^T.
// Sums of logarithms are formed in fp64 (64 of them per chunk and head, on one wave), because
// e^{c_i - c_j} of neighbouring steps needs the difference of two long sums; every exponential is
// taken of a difference, so with alpha >= 0 nothing overflows whatever the decay.
//
// Precision.  Products run on the bf16 MFMA with fp32 accumulation.  A computed fp32 operand is
// split into three bf16 planes x = hi + mid + lo by truncation, which is exact (8 + 8 + 8
// significant bits; only a remainder below the smallest bf16 is lost), so a product with a bf16
// input takes three exact passes, and a product of two fp32 operands six (the three terms below
// 2^-24 of the result are left out).  Two rounded planes would take two passes but leave 2e-6
// relative; the passes keep the MFMA busy for 8 to 23% of the kernels' cycles, beside the VALU's work.
#pragma once

#include "m2rnn_device.h"

namespace m2rnn {

constexpr double kLog2e64 = 1.4426950408889634074;

// Steps per chunk: 64 for bf16 inputs, 32 for fp32 ones (three planes of each input in LDS).
template <bool BF16>
constexpr int ssm_chunk() {
  return BF16 ? 64 : 32;
}
// Elements between LDS rows of a [rows][cols] bf16 plane: with 16 more than the columns (8 more for 16
// of them) the 8 rows that a transposing read touches at a time fall on different banks.
constexpr int ssm_stride(int cols) { return cols + (cols > 16 ? 16 : 8); }

// A lane index made opaque at this point.  Addresses formed from it are formed anew here, instead of
// being kept in registers from one phase of a loop to the next.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The same for a wave-uniform number: comparisons with it are made here, not kept as lane masks.
__device__ __forceinline__ int fresh_s(int x) {
  asm volatile("" : "+s"(x));
  return x;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// x = hi + mid + lo exactly; the three bf16 are the high halves of the words.
__device__ __forceinline__ void split3(float x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFF0000u;
  const float r = x - __uint_as_float(hi);
  mid = __float_as_uint(r) & 0xFFFF0000u;
  lo = __float_as_uint(r - __uint_as_float(mid));
}
// The high halves of a and b in one word (a low).
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Four fp32 values as 2 words of each plane.
__device__ __forceinline__ void split3x4(const float (&x)[4], uint2 (&p)[3]) {
  uint32_t h[4], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) split3(x[i], h[i], m[i], l[i]);
  p[0] = make_uint2(pack_hi(h[0], h[1]), pack_hi(h[2], h[3]));
  p[1] = make_uint2(pack_hi(m[0], m[1]), pack_hi(m[2], m[3]));
  p[2] = make_uint2(pack_hi(l[0], l[1]), pack_hi(l[2], l[3]));
}
__device__ __forceinline__ uint4 cat(uint2 a, uint2 b) { return make_uint4(a.x, a.y, b.x, b.y); }

// Eight consecutive slots of an operand as its three planes.
__device__ __forceinline__ void split3x8(const float (&x)[8], uint4 (&o)[3]) {
  const float a[4] = {x[0], x[1], x[2], x[3]}, b[4] = {x[4], x[5], x[6], x[7]};
  uint2 pa[3], pb[3];
  split3x4(a, pa);
  split3x4(b, pb);
#pragma unroll
  for (int p = 0; p < 3; ++p) o[p] = cat(pa[p], pb[p]);
}

// acc += sum of the plane products A[i] B[j], i + j <= 2, the small ones first.  NA, NB planes
// (1: the operand is bf16 itself).
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_planes(const uint4 (&A)[NA], const uint4 (&B)[NB], f32x4 acc) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < NB) acc = mfma_bf16(A[i], B[j], acc);
    }
  return acc;
}

// The same sum with the operands' roles turned: the passes follow in the same order, so the transposed
// tile holds the same bits.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_planes_turned(const uint4 (&A)[NA], const uint4 (&B)[NB], f32x4 acc) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int i = s - j;
      if (i >= 0 && i < NA) acc = mfma_bf16(A[i], B[j], acc);
    }
  return acc;
}

// MFMA operands from a bf16 plane [row][col] in LDS (row stride ST).  Lane l = 16 g + n.
// Row operand: index n along rows r0.., contraction over the columns c0 .. c0 + 31 in order.
__device__ __forceinline__ uint4 lds_row(const uint16_t* p, int ST, int r0, int c0, int g, int n) {
  return *(const uint4*)(p + (r0 + n) * ST + c0 + 8 * g);
}
// The same with the contraction's slots in the accumulator order: lane group g holds columns
// c0 + 4g .. + 3 and c0 + 16 + 4g .. + 3 (two accumulator tiles side by side form such an operand
// without any data movement, so its partner is read like this).
__device__ __forceinline__ uint4 lds_row_acc(const uint16_t* p, int ST, int r0, int c0, int g, int n) {
  const uint16_t* q = p + (r0 + n) * ST + c0 + 4 * g;
  return cat(*(const uint2*)q, *(const uint2*)(q + 16));
}
// Column operand: index n along columns c0.., contraction over the rows r0 .. r0 + 31 in the
// accumulator order, by two transposing reads.
__device__ __forceinline__ uint4 lds_col(const uint16_t* p, int ST, int r0, int c0, int g, int n) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s* lds_v4s;
  const uint16_t* q = p + (r0 + 4 * g + (n >> 2)) * ST + c0 + 4 * (n & 3);
  const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)q);
  const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(q + 16 * ST));
  return cat(__builtin_bit_cast(uint2, a), __builtin_bit_cast(uint2, b));
}

// The column operand with 16 contraction slots: rows r0 .. r0 + 15, lane group g rows r0 + 4g .. + 3.
__device__ __forceinline__ uint2 lds_col16(const uint16_t* p, int ST, int r0, int c0, int g, int n) {
  typedef short v4s __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4s* lds_v4s;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                       (lds_v4s)(p + (r0 + 4 * g + (n >> 2)) * ST + c0 + 4 * (n & 3))));
}

// ------------------------------------------------------------------ cross-lane helpers in fp64

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xF, false);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// The same with every row written and zeros where a lane has no source.
template <int CTRL>
__device__ __forceinline__ double dpp64_all(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Inclusive prefix sum over the wave's 64 lanes (row shifts, then the row totals broadcast on).
__device__ __forceinline__ double prefix64(double x) {
  x += dpp64_all<0x111>(x);
  x += dpp64_all<0x112>(x);
  x += dpp64_all<0x114>(x);
  x += dpp64_all<0x118>(x);
  x += dpp64<0x142, 0xA>(x);
  x += dpp64<0x143, 0xC>(x);
  return x;
}
__device__ __forceinline__ double lane64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// The two words of each of two doubles exchanged between the wave's halves (32) or between the odd rows
// of 16 of the first and the even rows of the second (16), and added.
template <bool HALVES>
__device__ __forceinline__ double swap_add64(double x, double y) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x), v = __builtin_bit_cast(uint64_t, y);
  const auto swap = [](uint32_t p, uint32_t q) {
    if constexpr (HALVES)
      return __builtin_amdgcn_permlane32_swap(p, q, false, false);
    else
      return __builtin_amdgcn_permlane16_swap(p, q, false, false);
  };
  const auto lo = swap((uint32_t)u, (uint32_t)v), hi = swap((uint32_t)(u >> 32), (uint32_t)(v >> 32));
  return __builtin_bit_cast(double, ((uint64_t)hi[0] << 32) | lo[0]) +
         __builtin_bit_cast(double, ((uint64_t)hi[1] << 32) | lo[1]);
}
// Sum over the four lanes n, n + 16, n + 32, n + 48, in each of them.
__device__ __forceinline__ double group_sum64(double x) {
  x = swap_add64<false>(x, x);
  return swap_add64<true>(x, x);
}
// Four such sums at once: lane group g gets the one of x[g].
__device__ __forceinline__ double group_sum64_4(const double (&x)[4]) {
  return swap_add64<false>(swap_add64<true>(x[0], x[2]), swap_add64<true>(x[1], x[3]));
}

// Sum over the wave, in every lane (rotations within the rows of 16, then across them).
__device__ __forceinline__ double total64(double x) {
  x += dpp64_all<0x128>(x);
  x += dpp64_all<0x124>(x);
  x += dpp64_all<0x122>(x);
  x += dpp64_all<0x121>(x);
  return group_sum64(x);
}

// out[16 I + n] = the sum of x[I] over the lane groups.
template <int NI>
__device__ __forceinline__ void put_group_sums(double* out, const double (&x)[NI], int g, int n) {
  if constexpr (NI == 4) {
    out[16 * g + n] = group_sum64_4(x);
  } else {
#pragma unroll
    for (int I = 0; I < NI; ++I) {
      const double t = group_sum64(x[I]);
      if (g == 0) out[16 * I + n] = t;
    }
  }
}

// ------------------------------------------------------------------ the chunk's decays

// softplus(z) and its derivative sigma(z), with a relative error of a few ulp also where they are small (steps of
// 1e-3 are ordinary here, and log(1 + e^z) formed directly would keep 4 digits of them).  With t = e^{-|z|},
// softplus = max(z, 0) + log(1 + t) and log(1 + t) = 2 atanh(s), s = t / (2 + t) <= 1/3, by its series (the first term
// left out is below 2^-29 of the sum); t from the hardware's exponential of |z| log2 e in two parts.  A quarter of
// the instructions of the general functions, for 64 steps of every head in every pass.  t below 2^-126 counts as 0.
__device__ __forceinline__ void softplus_sigma(float z, float& sp, float& sg) {
  constexpr float kL = 1.4426950408889634f, kLlo = (float)(1.4426950408889634 - (double)kL);
  const float m = fminf(fabsf(z), 128.0f);
  const float x = m * -kL, lo = __builtin_fmaf(m, -kL, -x) - m * kLlo;
  float t = exp2_(x);
  t = __builtin_fmaf(t, lo * 0.69314718f, t);
  const auto over = [](float a, float b) {  // a / b, the reciprocal's error taken out
    const float r = __builtin_amdgcn_rcpf(b), q = a * r;
    return __builtin_fmaf(__builtin_fmaf(-q, b, a), r, q);
  };
  const float s = over(t, 2.0f + t), s2 = s * s;
  float p = 1.0f / 17.0f;
  p = __builtin_fmaf(p, s2, 1.0f / 15.0f);
  p = __builtin_fmaf(p, s2, 1.0f / 13.0f);
  p = __builtin_fmaf(p, s2, 1.0f / 11.0f);
  p = __builtin_fmaf(p, s2, 1.0f / 9.0f);
  p = __builtin_fmaf(p, s2, 1.0f / 7.0f);
  p = __builtin_fmaf(p, s2, 1.0f / 5.0f);
  p = __builtin_fmaf(p, s2, 1.0f / 3.0f);
  sp = (z < 0.0f ? 0.0f : z) + __builtin_fmaf(2.0f * s, s2 * p, 2.0f * s);  // (NaN stays NaN)
  sg = over(z < 0.0f ? t : 1.0f, 1.0f + t);
}

// log2 f for a step of size delta, held within +-2^14 so that sums and differences stay finite (2^x
// is 0 or inf in fp32 long before); NaN stays NaN.
__device__ __forceinline__ double log2_decay(float alpha, float delta) {
  double x = -(double)alpha * (double)delta * kLog2e64;
  x = x < -16384.0 ? -16384.0 : x;
  return x > 16384.0 ? 16384.0 : x;
}

// Decay tables of one head's chunk in LDS, by step: e = 2^{c_i}; w = 2^{c_L - c_j}; x = 2^{c_i - c at
// the step before i's 16-step tile}; f[I - 1] = 2^{(c at the step before tile I) - c_j} for j below
// tile I (w and f times D_j if FD, the forward's form); d = D_j; and c itself as a pair of floats (chi + clo) for the diagonal
// tiles, whose factors are formed one by one.
template <int L>
struct SsmTab {
  static constexpr int NI = L / 16;
  float e[L], w[L], x[L], d[L], chi[L], clo[L], f[NI > 1 ? NI - 1 : 1][L];
};
// The backward's also hold sigma(a + beta).
template <int L>
struct SsmTabBwd : SsmTab<L> {
  float s[L];
};

// One wave, lane j = step j of the chunk: its step size D_j and log2 f_j in (both 0 past the sequence's end
// and in the lanes past the chunk).
template <int L, bool FD>
__device__ __forceinline__ void ssm_tables(SsmTab<L>& tab, int lane, float delta, double lg) {
  constexpr int NI = L / 16;
  const double c = prefix64(lg);
  const double cl = lane64(c, L - 1);
  double at[NI];
#pragma unroll
  for (int I = 1; I < NI; ++I) at[I] = lane64(c, 16 * I - 1);
  if (lane >= L) return;
  double ref = 0.0;
#pragma unroll
  for (int I = 1; I < NI; ++I) {
    float fj = exp2_((float)(at[I] - c));
    if constexpr (FD) fj *= delta;
    tab.f[I - 1][lane] = fj;  // meant for lane < 16 I; finite or not, the others are never used
    ref = lane >= 16 * I ? at[I] : ref;
  }
  tab.x[lane] = exp2_((float)(c - ref));
  const float hi = (float)c;
  tab.chi[lane] = hi;
  tab.clo[lane] = (float)(c - (double)hi);
  tab.d[lane] = delta;
  tab.e[lane] = exp2_((float)c);
  tab.w[lane] = (FD ? delta : 1.0f) * exp2_((float)(cl - c));
}

// ------------------------------------------------------------------ staging a chunk

// A thread's share of a [L][CP] block (CP columns in LDS, C of them real) of a row-major source with
// `row_stride` elements between steps: 16-byte pieces held in registers between the load and the
// store to LDS.  Rows at or past `rows` and columns at or past C are zeros and never read.
template <bool BF16, int L, int CP, int NTH>
struct SsmPieces {
  static constexpr int VEC = BF16 ? 8 : 4;
  static constexpr int PR = CP / VEC;  // pieces per row
  static constexpr int NP = (L * PR + NTH - 1) / NTH;
  static constexpr int ST = ssm_stride(CP);
  uint4 r[NP];

  __device__ __forceinline__ void load(const void* base, long row_stride, int C, int rows, int tid) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int i = tid + p * NTH;
      const int row = i / PR, col = (i % PR) * VEC;
      r[p] = make_uint4(0, 0, 0, 0);
      if ((L * PR) % NTH != 0 && i >= L * PR) continue;
      if (row < rows && col < C) {
        if constexpr (BF16)
          r[p] = *(const uint4*)((const uint16_t*)base + row * row_stride + col);
        else
          r[p] = *(const uint4*)((const float*)base + row * row_stride + col);
      }
    }
  }

  // To LDS: one plane for bf16, three for fp32 (plane stride L * ST elements).
  __device__ __forceinline__ void store(uint16_t* lds, int tid) const {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int i = tid + p * NTH;
      const int row = i / PR, col = (i % PR) * VEC;
      if ((L * PR) % NTH != 0 && i >= L * PR) continue;
      uint16_t* d = lds + row * ST + col;
      if constexpr (BF16) {
        *(uint4*)d = r[p];
      } else {
        const float x[4] = {__uint_as_float(r[p].x), __uint_as_float(r[p].y), __uint_as_float(r[p].z),
                            __uint_as_float(r[p].w)};
        uint2 pl[3];
        split3x4(x, pl);
#pragma unroll
        for (int q = 0; q < 3; ++q) *(uint2*)(d + q * L * ST) = pl[q];
      }
    }
  }
};

}  // namespace m2rnn
