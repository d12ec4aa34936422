// Orthogonalised update: X_0 = G / (||G||_F + eps), then `steps` times, with A = X X^T over the shorter side,
//     X <- a X + (b A + c A A) X,
// which takes every singular value s of X to a s + b s^3 + c s^5 and leaves the singular vectors: with the usual
// coefficients all of them end near 1.
//
// Three matrix products a step:
//     (1) A = X X^T (symmetric: its lower tiles, each written twice), (2) B = b A + c A A^T (likewise),
//     (3) X' = a X + B X, whose right operand goes along X's columns (transposing reads).
// Precision.  X is kept in fp32.  What a product multiplies is split into two fp16 planes x = hi + lo (22 bits), and it takes
// three passes of the fp16 MFMA with fp32 accumulation (lo lo, below 2^-22 of the product, is left out): the error is that of
// fp32 products, at eight times the fp32 MFMA's rate over three.
//
// fp16 has no exponents to spare (2^15 down to where lo ends, 2^-24), and rows and columns of a gradient may be far smaller than
// others, so each row and column has a power of two of its own: with D and E no less than the norms of X's rows and columns,
//     R = D^-1 X and C = X E^-1      the operands of (1) and of (3), no entry above 1 (both are planes; with one set, of X
//                                    itself, half the rows times 1e-5 were off by 1e-4, times 1e-12 by all of it),
//     S = R R^T,  D^-1 A = S D       whose rows have the size of R's (entries stay below X's largest singular value),
//     D^-1 B = b (D^-1 A) + c (D^-1 A)(D^-1 A)^T D,   X' = a X + D (D^-1 B) C E.
// So errors of an entry are relative to its row and its column, as fp32 products' are.  Planes are kept times 2^15 (R, C), 2^14
// (D^-1 A) and 2^7 or less (D^-1 B, whose rows are at most |b s + c s^3|).
#pragma once

#include "m2rnn_orth_plan.h"
#include "m2rnn_ssm_device.h"
#include "m2rnn_stream.h"

namespace m2rnn {

constexpr float kOrthX = 32768.0f, kOrthA = 16384.0f;

// The power of two above |x|, from 2^-100 to 2^100 (also of zeros and what is not finite), and its inverse.
__device__ __forceinline__ float pow2_above(float x) {
  const int e = ((int)(__float_as_uint(x) >> 23) & 255) + 1;
  return __uint_as_float((uint32_t)(e < 27 ? 27 : e > 227 ? 227 : e) << 23);
}
__device__ __forceinline__ float pow2_inverse(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }
// The next scale of a row or column whose values, over the scale p, have squares that add up to `squares`, and may grow by 2^grow in the
// step that is being taken: the power of two above their norm, times 2^grow (2^k above the square root: half the exponent).  Less than
// 2^-48 counts as that much: a row of zeros keeps a scale.
__device__ __forceinline__ float next_scale(float p, float squares, int grow) {
  const int k = ((int)(__float_as_uint(fmaxf(squares, 0x1p-48f)) >> 23) - 127) >> 1;
  const int e = (int)(__float_as_uint(p) >> 23) + k + 1 + grow;
  return __uint_as_float((uint32_t)(e < 27 ? 27 : e > 227 ? 227 : e) << 23);
}

// Two fp16 planes of a matrix [rows][ld], in blocks of 16 rows by 32 columns (1 KB, in the order that a product's stage has
// in LDS), so that a wave brings a block as whole lines.
struct Planes {
  uint16_t *hi, *lo;
};
// Within a block, 16-byte unit u of row r is at u ^ plane_turn(r): the lanes that the LDS serves together then touch all
// banks, where an operand is read along its rows (0-3 and 12-15 of one unit with 4-11 of the next: 238 bytes a clock,
// 123 with unit u at u) and by transposing reads (rows r and r + 8 of one half: 137 and 125).
__device__ __forceinline__ int plane_turn(int r) { return (r >> 2) & 2; }
// Where element (r, c) lies.
__device__ __forceinline__ long plane_at(int r, int c, int ld) {
  return ((long)(r >> 4) * (ld >> 5) + (c >> 5)) * 512 + ((r & 15) * 4 + (((c >> 3) & 3) ^ plane_turn(r))) * 8 + (c & 7);
}

__device__ __forceinline__ void split_f16(float x, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)x;
  const _Float16 l = (_Float16)(x - (float)h);
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, l);
}
__device__ __forceinline__ float join_f16(uint16_t hi, uint16_t lo) {
  return (float)__builtin_bit_cast(_Float16, hi) + (float)__builtin_bit_cast(_Float16, lo);
}

// The e-th of four values whose halves are side by side.
__device__ __forceinline__ float half_of(uint2 hi, uint2 lo, int e) {
  const uint32_t h = e < 2 ? hi.x : hi.y, l = e < 2 ? lo.x : lo.y;
  return join_f16((uint16_t)(e & 1 ? h >> 16 : h), (uint16_t)(e & 1 ? l >> 16 : l));
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, long i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  return ((const float*)p)[i];
}

__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  return x;
}

// Partial sums of squares of a matrix in fp64: workgroup (p, matrix) of `parts`.  Four elements a load where a matrix's
// size keeps them aligned, four loads in flight.
template <bool BF16>
__global__ void __launch_bounds__(256) m2rnn_orth_squares_kernel(const void* g, long mn, long each, double* part) {
  __shared__ double red[4];
  const long first = (long)blockIdx.x * each, last = first + each < mn ? first + each : mn;
  const long at = (long)blockIdx.y * mn;
  double acc = 0.0;
  if (mn % 4 == 0) {
#pragma unroll 4
    for (long i = first + 4 * threadIdx.x; i < last; i += 1024) {
      const float4 x = load4<BF16>(g, at + i);
      acc += ((double)x.x * x.x + (double)x.y * x.y) + ((double)x.z * x.z + (double)x.w * x.w);
    }
  } else {
#pragma unroll 8
    for (long i = first + threadIdx.x; i < last; i += 256) {
      const double x = (double)load1<BF16>(g, at + i);
      acc += x * x;
    }
  }
  acc = wave_sum(acc);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
  __syncthreads();
  if (threadIdx.x == 0) part[(long)blockIdx.y * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// A power of two that is no less than the norm of `count` values of X_0 (a row or a column) of magnitude `most` at most: their root's
// share, or 1, which is X_0's own norm.
__device__ __forceinline__ float first_scale(float most, int count) {
  const int root = (33 - __clz(count - 1)) >> 1;  // 2^root >= sqrt(count)
  return fminf(pow2_above(most) * __uint_as_float((uint32_t)(127 + root) << 23), 1.0f);
}

// What X_0's scales come from, over G [rows][cols] as it lies: the partial sums of squares (fp64), and the largest magnitudes of its
// rows and columns within a workgroup's 256 columns and `each` rows (a multiple of 64).
struct OrthNorms {
  double* squares;   // [batch][gridDim.y gridDim.x]
  float *row, *col;  // [batch][gridDim.x][rows], [batch][gridDim.y][cols]
};
// WIDE: columns in multiples of four, of which a lane takes four neighbours; else every 64th.
template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(256) m2rnn_orth_norms_kernel(const void* g, int rows, int cols, int each, OrthNorms N) {
  __shared__ float most[4][256];
  __shared__ double red[4];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const long z = blockIdx.z, at = z * rows * cols;
  const int c0 = blockIdx.x * 256 + (WIDE ? 4 * lane : lane);
  const int first = blockIdx.y * each, last = first + each < rows ? first + each : rows;
  float* of_rows = N.row + (z * gridDim.x + blockIdx.x) * rows;
  float of_col[4] = {0, 0, 0, 0};
  double acc = 0.0;
  for (int r0 = first + 16 * w; r0 < last; r0 += 64) {
    float x[16][4], of_row = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {  // (places past the end take the first column or the last row, and count as zeros)
      const long o = at + (long)(r0 + i < last ? r0 + i : last - 1) * cols;
      if constexpr (WIDE) {
        const float4 t = load4<BF16>(g, o + (c0 < cols ? c0 : 0));
        x[i][0] = t.x; x[i][1] = t.y; x[i][2] = t.z; x[i][3] = t.w;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i][k] = load1<BF16>(g, o + (c0 + 64 * k < cols ? c0 + 64 * k : 0));
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][k] = r0 + i < last && c0 + (WIDE ? 0 : 64 * k) < cols ? x[i][k] : 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc += (double)x[i][k] * (double)x[i][k];
        m = fmaxf(m, fabsf(x[i][k]));
        of_col[k] = fmaxf(of_col[k], fabsf(x[i][k]));
      }
      m = fmaxf(m, dpp_all<kDppQuadXor1>(m));
      m = fmaxf(m, dpp_all<kDppQuadXor2>(m));
      m = fmaxf(m, dpp_all<kDppRowHalfMirror>(m));
      m = fmaxf(m, dpp_all<kDppRowMirror>(m));
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      if (lane == i) of_row = m;
    }
    if (lane < 16 && r0 + lane < last) of_rows[r0 + lane] = of_row;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) most[w][WIDE ? 4 * lane + k : lane + 64 * k] = of_col[k];
  acc = wave_sum(acc);
  if (lane == 0) red[w] = acc;
  __syncthreads();
  const int t = threadIdx.x, c = blockIdx.x * 256 + t;
  if (c < cols) N.col[(z * gridDim.y + blockIdx.y) * cols + c] = fmaxf(fmaxf(most[0][t], most[1][t]), fmaxf(most[2][t], most[3][t]));
  if (t == 0) N.squares[(z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X_0's scale 1 / (||G||_F + eps) for each matrix, and the first scales of its rows (d) and columns (e): a thread each, of the mp rows
// and np columns.  gx, gy: the workgroups that N is of.  m x n is G or, `tall`, its transpose.
__global__ void __launch_bounds__(256) m2rnn_orth_scales_kernel(OrthNorms N, int gx, int gy, int m, int n, int mp, int np, int ma, int na,
                                                                int tall, float eps, double* scale, float* d, float* e) {
  __shared__ double red[4];
  const long z = blockIdx.y;
  double ss = 0.0;
  for (int i = threadIdx.x; i < gx * gy; i += 256) ss += N.squares[z * gx * gy + i];
  ss = wave_sum(ss);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = ss;
  __syncthreads();
  const double f = 1.0 / (sqrt((red[0] + red[1]) + (red[2] + red[3])) + (double)eps);
  if (blockIdx.x == 0 && threadIdx.x == 0) scale[z] = f;
  const int t = blockIdx.x * 256 + threadIdx.x;
  const bool row = t < mp;
  const int i = row ? t : t - mp;
  if (!row && i >= np) return;
  float most = 0.0f;
  if (i < (row ? m : n)) {
    const bool of_rows = row != (tall != 0);  // whether it is a row of G
    const int parts = of_rows ? gx : gy, side = row ? m : n;
    const float* p = (of_rows ? N.row : N.col) + z * parts * side + i;
#pragma unroll 16
    for (int k = 0; k < parts; ++k) most = fmaxf(most, p[(long)k * side]);
  }
  (row ? d + z * ma : e + z * na)[i] = first_scale((float)((double)most * f), row ? n : m);
}

// X_0 in fp32 and as planes R and C, [ma][na], zeros past m x n up to whole workgroups, which take 64 x 64; m x n is G or, `tall`, its
// transpose.
template <bool BF16>
__global__ void __launch_bounds__(256) m2rnn_orth_split_kernel(const void* g, int m, int n, int ma, int na, int tall,
                                                               const double* scale, const float* d, const float* e, float* X, Planes R,
                                                               Planes C) {
  __shared__ float tile[64][65];
  const long z = blockIdx.z;
  const double f = scale[z];
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const long at = z * m * n;
#pragma unroll 8
  for (int i = ty; i < 64; i += 4) {  // (i, tx) along G's own rows
    const int r = tall ? r0 + tx : r0 + i, c = tall ? c0 + i : c0 + tx;
    float x = 0.0f;
    if (r < m && c < n) x = (float)((double)load1<BF16>(g, at + (tall ? (long)c * m + r : (long)r * n + c)) * f);
    tile[tall ? tx : i][tall ? i : tx] = x;
  }
  __syncthreads();
#pragma unroll 8
  for (int i = ty; i < 64; i += 4) X[(z * ma + r0 + i) * na + c0 + tx] = tile[i][tx];
  // 8 blocks of the planes, two of them a wave, a lane the unit that lies at its place
  const int row = tx >> 2, unit = (tx & 3) ^ plane_turn(row);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int id = 2 * ty + k, br = 16 * (id >> 1), bc = 32 * (id & 1);
    const float rd = kOrthX * pow2_inverse(d[z * ma + r0 + br + row]);
    alignas(16) uint16_t hi[8], lo[8], chi[8], clo[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float x = tile[br + row][bc + 8 * unit + q];
      split_f16(x * rd, hi[q], lo[q]);
      split_f16(x * (kOrthX * pow2_inverse(e[z * na + c0 + bc + 8 * unit + q])), chi[q], clo[q]);
    }
    const long o = z * ma * na + plane_at(r0 + br, c0 + bc, na) + tx * 8;
    *(uint4*)(R.hi + o) = *(const uint4*)hi;
    *(uint4*)(R.lo + o) = *(const uint4*)lo;
    *(uint4*)(C.hi + o) = *(const uint4*)chi;
    *(uint4*)(C.lo + o) = *(const uint4*)clo;
  }
}

constexpr int kOrthMaxSteps = 64;
struct OrthCoefs {
  float c[3 * kOrthMaxSteps], unit[kOrthMaxSteps];  // unit: what D^-1 B is kept times
};

// What a product's epilogue does with its tile.
enum { ORTH_GRAM = 0, ORTH_POLY = 1, ORTH_NEXT = 2, ORTH_LAST = 3 };

struct OrthArgs {
  Planes M, N;        // rows x ld and cols x ld (NEXT and LAST: ld x cols), of which the contraction takes K
  Planes E;           // POLY: D^-1 A
  Planes O, C;        // the outputs, rows x cols: GRAM and POLY one, NEXT R and C
  float* X;           // NEXT and LAST: X [rows][cols], the step before's (NEXT: the next one's in its place)
  void* out;          // LAST: [m][n], or [n][m] if tall
  float* part;        // [batch][splits][tiles][waves] wave tiles of partial sums, if the contraction is split
  const float *d, *e; // the scales of X's rows [batch][ma] and columns [batch][na]
  float *dn, *en;     // those of the next X: dn is written by NEXT, en by GRAM
  float* diag;        // [batch][ma]: the diagonal of S = R R^T, written by GRAM, read by NEXT
  float* squares;     // [batch][sums][na]: sums of squares of X E^-1 over some rows each, written by NEXT, read by the next GRAM
  int sums;           // how many there are (0: none yet, the norms are those of the scales)
  int rows, cols, ld; // the arrays' sides: at least what the tiles cover
  int K, gi, gj;      // the contraction's length; rows and columns of tiles
  int m, n, mp;       // X's sides, the shorter one rounded up
  int tall, out_bf16;
  int splits, tiles;
  float ca, cb, cc;   // NEXT and LAST: a.  GRAM: what S D is multiplied by.  POLY: b and c with the planes' units
  float unit;         // NEXT and LAST: 1 over the units of the product's operands
  int grow;           // no row or column grows by more than 2^grow within a step
};

// GRAM and POLY: a lane's part of NJ 16 x 16 tiles side by side, rows r .. r + 3 of the columns c + 16 j.  `mirror`: the
// transposed place is written too.  What the epilogue reads is loaded before anything is stored.
template <int EPI, int NJ>
__device__ __forceinline__ void orth_square(const OrthArgs& A, long z, int r, int c, const f32x4 (&acc)[NJ], bool mirror) {
  const long zo = z * A.rows * A.cols;
  const float* d = A.d + z * A.rows;
  const float4 t4 = *(const float4*)(d + r);
  const float dr[4] = {t4.x, t4.y, t4.z, t4.w};
  float x[NJ][4], dc[NJ];
  uint2 mh[NJ], ml[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) dc[j] = d[c + 16 * j];
  if constexpr (EPI == ORTH_POLY) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const long at = zo + plane_at(r + e, c + 16 * j, A.cols);
        x[j][e] = join_f16(A.E.hi[at], A.E.lo[at]);
      }
    if (mirror) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const long at = zo + plane_at(c + 16 * j, r, A.rows);  // (four neighbours: r is a multiple of 4)
        mh[j] = *(const uint2*)(A.E.hi + at);
        ml[j] = *(const uint2*)(A.E.lo + at);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    float s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] = acc[j][e] * (EPI == ORTH_GRAM ? 1.0f / (kOrthX * kOrthX) : A.cc);
      float y = s[e] * dc[j];
      if constexpr (EPI == ORTH_GRAM) {
        if (r + e == c + 16 * j) A.diag[z * A.rows + r + e] = s[e];
        y *= A.cb;  // (D^-1 A, or D^-1 B of a cubic step)
      } else {
        y = __builtin_fmaf(A.cb, x[j][e], y);
      }
      uint16_t hi, lo;
      split_f16(y, hi, lo);
      const long at = zo + plane_at(r + e, c + 16 * j, A.cols);
      A.O.hi[at] = hi;
      A.O.lo[at] = lo;
    }
    if (mirror) {
      uint16_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y = s[e] * dr[e];
        if constexpr (EPI == ORTH_GRAM)
          y *= A.cb;
        else
          y = __builtin_fmaf(A.cb, half_of(mh[j], ml[j], e), y);
        split_f16(y, hi[e], lo[e]);
      }
      const long at = zo + plane_at(c + 16 * j, r, A.rows);
      *(uint2*)(A.O.hi + at) = make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
      *(uint2*)(A.O.lo + at) = make_uint2(lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16);
    }
  }
}

// GRAM's further workgroups: the scales of the next X's columns, from the norms of this one's.
__device__ __forceinline__ void orth_columns(const OrthArgs& A, long z, int c) {
  if (c >= A.K) return;
  const float* p = A.squares + z * A.sums * A.ld + c;
  float s = A.sums == 0 ? 0.5f : 0.0f;  // (the first scales bound the norms themselves)
#pragma unroll 8
  for (int i = 0; i < A.sums; ++i) s += p[(long)i * A.ld];
  A.en[z * A.ld + c] = next_scale(A.e[z * A.ld + c], s, A.grow);
}

// Sum over the 16 lanes of a row of lanes, in each of them.
__device__ __forceinline__ float row16_sum(float x) {
  x += dpp_all<kDppQuadXor1>(x);
  x += dpp_all<kDppQuadXor2>(x);
  x += dpp_all<kDppRowHalfMirror>(x);
  return x + dpp_all<kDppRowMirror>(x);
}

// NEXT and LAST: a lane's part of NJ 16 x 16 tiles side by side, of row r the columns c + 16 j to c + 16 j + 3, which have the scales
// e and (NEXT) en.  NEXT: adds to sq the squares for the columns' norms; `keep`: writes the row's new scale.
template <int EPI, int NJ>
__device__ __forceinline__ void orth_next(const OrthArgs& A, long z, int r, int c, const f32x4 (&acc)[NJ], const float4 (&e)[NJ],
                                          const float4 (&en)[NJ], f32x4 (&sq)[NJ], bool keep) {
  float* X = A.X + (z * A.rows + r) * A.cols + c;
  const float d = A.d[z * A.rows + r], f = d * A.unit;
  float4 x[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) x[j] = *(const float4*)(X + 16 * j);
  float rd = 0.0f;
  if constexpr (EPI == ORTH_NEXT) {
    const float dn = next_scale(d, A.diag[z * A.rows + r], A.grow);
    if (keep) A.dn[z * A.rows + r] = dn;
    rd = kOrthX * pow2_inverse(dn);
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    float y[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
    const float ec[4] = {e[j].x, e[j].y, e[j].z, e[j].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = __builtin_fmaf(A.ca, y[q], acc[j][q] * f * ec[q]);
    if constexpr (EPI == ORTH_LAST) {
      const int col = c + 16 * j;
      const long o = z * A.m * A.n + (A.tall ? (long)col * A.m + r : (long)r * A.n + col), step = A.tall ? A.m : 1;
      if (!A.tall && A.n % 4 == 0) {  // (aligned)
        if (r < A.m && col < A.n) {
          if (A.out_bf16)
            *(uint2*)((uint16_t*)A.out + o) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
          else
            *(float4*)((float*)A.out + o) = make_float4(y[0], y[1], y[2], y[3]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r < A.m && col + q < A.n) {
            if (A.out_bf16)
              ((__bf16*)A.out)[o + q * step] = (__bf16)y[q];
            else
              ((float*)A.out)[o + q * step] = y[q];
          }
      }
    } else {
      const float en4[4] = {en[j].x, en[j].y, en[j].z, en[j].w};
      uint16_t hi[4], lo[4], chi[4], clo[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float t = y[q] * pow2_inverse(en4[q]);
        const float u = r < A.mp ? t : 0.0f;  // (nothing is known of rows past them)
        sq[j][q] = __builtin_fmaf(u, u, sq[j][q]);
        split_f16(y[q] * rd, hi[q], lo[q]);
        split_f16(t * kOrthX, chi[q], clo[q]);
      }
      *(float4*)(X + 16 * j) = make_float4(y[0], y[1], y[2], y[3]);
      const long at = z * A.rows * A.cols + plane_at(r, c + 16 * j, A.cols);
      *(uint2*)(A.O.hi + at) = make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
      *(uint2*)(A.O.lo + at) = make_uint2(lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16);
      *(uint2*)(A.C.hi + at) = make_uint2(chi[0] | (uint32_t)chi[1] << 16, chi[2] | (uint32_t)chi[3] << 16);
      *(uint2*)(A.C.lo + at) = make_uint2(clo[0] | (uint32_t)clo[1] << 16, clo[2] | (uint32_t)clo[3] << 16);
    }
  }
}

// The place of tile number `id` of TM x TN tiles: those that touch the lower triangle by rows (SYM, Q = TM / TN of them for
// each row before), or bands of four rows, column by column.
template <bool SYM, int Q>
__device__ __forceinline__ void orth_place(int id, int gi, int gj, int& bi, int& bj) {
  if constexpr (SYM) {
    const int k = id / Q;
    bi = (int)((sqrtf(8.0f * (float)k + 1.0f) - 1.0f) * 0.5f);
    while ((bi + 1) * (bi + 2) / 2 * Q <= id) ++bi;
    while (bi * (bi + 1) / 2 * Q > id) --bi;
    bj = id - bi * (bi + 1) / 2 * Q;
  } else {
    const int band = id / (4 * gj), in = id % (4 * gj);
    const int high = gi - 4 * band < 4 ? gi - 4 * band : 4;
    bi = 4 * band + in % high;
    bj = in / high;
  }
}

// Tiles are dealt to the 8 XCDs in turn; each XCD takes a run of neighbouring ones, so that they share rows in its L2.
__device__ __forceinline__ int orth_turn(int id, int total) {
  const int q = total / 8, r = total % 8, x = id % 8;
  return x * q + (x < r ? x : r) + id / 8;
}

// 16 bytes of each lane to LDS, lane after lane from `to` (the same in all lanes) on, past the registers.  The builtin for this
// makes the compiler wait for it before any read of LDS, also of the other buffer; here the caller waits (vmcnt).  Nothing else in
// the kernels that call it uses m0.
__device__ __forceinline__ void load_to_lds(const void* from, const void* to) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)to;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(from) : "memory");
}

// One TM x TN tile of M N^T (NEXT and LAST: M N), or its part of a split contraction (GRAM).  WR x WC waves, 16x16x32 MFMA.  A stage
// is 32 of the contraction: a column of blocks of M's planes, and of N's (M N: two rows of them), brought to LDS past the
// registers.  The three passes of a stage are summed by themselves, from zero, and added to the tile's sum once: one rounding at the sum's
// size for each stage instead of three.
// Measured, of 8192 x 2048: B X by 256 x 256 tiles 183 to 190 us in the last step (1.1 PFLOP/s of the three passes; MFMA 58% of the
// cycles, the card's power) and 216 to 225 in the others, which write X and both operands of the next step at the end, when all
// CUs write (134 MB more than X's two planes alone, 40 us); X X^T 113 to 120.  Of 2176 x 2048: B X 61 to 65 and 66 to 71 us by 96 x 96
// tiles (0.84 and 0.78 PFLOP/s), 41 to 44 for a symmetric product by 64 x 64 (0.62).
// LDS holds BUFS stages, all but the one that is multiplied on their way.  Two where a CU holds several workgroups, or a
// tile leaves no room for more; more for the only workgroup of a CU, whose stages would otherwise each wait for memory.
template <int TM, int TN, int WR, int WC, int BUFS, int EPI, bool SPLIT>
__global__ void __launch_bounds__(64 * WR * WC) m2rnn_orth_product_kernel(OrthArgs A) {
  constexpr bool SYM = EPI == ORTH_GRAM || EPI == ORTH_POLY;  // and M N^T
  constexpr int NI = TM / WR / 16, NJ = TN / WC / 16, WAVES = WR * WC;
  constexpr int BM = TM / 16, BN = TN / 16, PER = 2 * (BM + BN) / WAVES;  // blocks of a plane's stage; those that a wave brings
  constexpr int STAGE = 8 * (TM + TN);                                    // 16-byte units
  static_assert(2 * (BM + BN) % WAVES == 0 && TM % TN == 0, "whole blocks for each wave, whole tiles on the diagonal");
  __shared__ uint4 lds[BUFS * STAGE];  // [buffer][M hi, M lo, N hi, N lo][row][unit]
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const long z = blockIdx.z;
  if constexpr (EPI == ORTH_GRAM) {
    if ((int)blockIdx.x >= A.tiles) {
      if (blockIdx.y == 0) orth_columns(A, z, ((int)blockIdx.x - A.tiles) * 64 * WAVES + (int)threadIdx.x);
      return;
    }
  }
  const int tile = orth_turn(blockIdx.x, A.tiles);
  int bi, bj;
  orth_place<SYM, TM / TN>(tile, A.gi, A.gj, bi, bj);
  const int r0 = bi * TM, c0 = bj * TN;
  const int stages = A.K / kOrthK;
  const int first = SPLIT ? (int)((long)stages * blockIdx.y / A.splits) : 0;
  const int last = SPLIT ? (int)((long)stages * (blockIdx.y + 1) / A.splits) : stages;
  const uint16_t* src[PER];
  long step[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int id = w * PER + i;  // the block's number in a stage, by planes
    const bool right = id >= 2 * BM;
    const int in = right ? id - 2 * BM : id, most = right ? BN : BM;
    const int lo = in >= most, blk = in - lo * most;
    const uint16_t* plane = right ? (lo ? A.N.lo : A.N.hi) : lo ? A.M.lo : A.M.hi;
    long at;
    if (right && !SYM) {  // block 2 j + k: columns 32 j on, rows 16 k on
      at = z * A.ld * A.cols + ((blk & 1) * (A.cols >> 5) + (c0 >> 5) + (blk >> 1)) * 512L;
      step[i] = A.cols * 32L;
    } else {
      at = (z * (right ? A.cols : A.rows) + (right ? c0 : r0) + 16 * blk) * A.ld;
      step[i] = 512;
    }
    src[i] = plane + at + first * step[i] + lane * 8;
  }
  auto fetch = [&](int buf) {  // the next stage
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      load_to_lds(src[i], lds + buf * STAGE + (w * PER + i) * 64);
      src[i] += step[i];
    }
  };
  f32x4 acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  const int n = lane & 15, g = lane >> 4;
  const int wr = (w / WC) * (TM / WR), wc = (w % WC) * (TN / WC);
  const int unit = n * 4 + (g ^ plane_turn(n));  // (16 rows on: the same exchange)
  const uint4 *pm = lds + wr * 4 + unit, *pn = lds + 8 * TM + wc * 4 + unit;
  // M N: a transposing read gives a lane of group g four rows from 8 g on of column n, and the next one the four behind;
  // lane n of the group brings eight bytes of row n / 4.  Even and odd tiles of 16 columns are a block's halves (a wave may
  // begin with either).
  typedef __attribute__((address_space(3))) const char* lds_bytes;
  lds_bytes pt[2];
  {
    const int row = 8 * (g & 1) + (n >> 2), odd = (wc >> 4) & 1;
    const int at = (g >> 1) * 1024 + row * 64 + (((n >> 1) & 1) ^ plane_turn(row)) * 16 + (n & 1) * 8;
#pragma unroll
    for (int p = 0; p < 2; ++p) pt[p] = (lds_bytes)(lds + 8 * TM) + ((wc >> 5) + (p & odd)) * 2048 + (at ^ ((p ^ odd) * 32));
  }
  auto read_n = [&](int buf, int lo, int j) {
    if constexpr (SYM) return pn[buf * STAGE + lo * 4 * TN + j * 64];
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s* lds_v4s;
    const int at = (buf * STAGE + lo * 4 * TN) * 16 + (j >> 1) * 2048;
    const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(pt[j & 1] + at));
    const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(pt[j & 1] + at + 256));  // (plane_turn is the same there)
    return cat(__builtin_bit_cast(uint2, a), __builtin_bit_cast(uint2, b));
  };
  auto times = [&](const uint4& m, const uint4& k, const f32x4& c) { return SYM ? mfma_f16(m, k, c) : mfma_f16(k, m, c); };
  uint4 nh[NJ], nl[NJ], mh[2], ml[2];
  auto read_m = [&](int buf, int i) {
    mh[i & 1] = pm[buf * STAGE + i * 64];
    ml[i & 1] = pm[buf * STAGE + 4 * TM + i * 64];
  };
  constexpr int NT = 2 + NI % 2;  // rows' sums that take turns; the last row's is added in the next stage
  f32x4 t[NT][NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) t[NT - 1][j] = f32x4{0, 0, 0, 0};
  static_assert(NI % NT == 0, "the last row has the last place");
  static_assert((BUFS - 2) * PER < 16, "a wait's count");
#pragma unroll
  for (int i = 0; i < BUFS - 1; ++i)
    if (first + i < last) fetch(i);
  int buf = 0;
  for (int s = first; s < last; ++s, buf = buf + 1 == BUFS ? 0 : buf + 1) {
    if (s + BUFS - 1 <= last)
      __builtin_amdgcn_s_waitcnt(0x0f70 | (BUFS - 2) * PER);  // this wave's blocks have arrived (vmcnt: not those of later stages)
    else
      __builtin_amdgcn_s_waitcnt(0x0f70);  // (fewer are on their way: all of them)
    lds_barrier();  // and all waves'; the buffer of the stage before has been read by all
    if (s + BUFS - 1 < last) fetch(buf == 0 ? BUFS - 1 : buf - 1);
    // in the order in which they are needed: all waves read at once here, and the first products wait for two of these
    ml[0] = pm[buf * STAGE + 4 * TM];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      nh[j] = read_n(buf, 0, j);
      __builtin_amdgcn_sched_barrier(0);
    }
    mh[0] = pm[buf * STAGE];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      nl[j] = read_n(buf, 1, j);
      __builtin_amdgcn_sched_barrier(0);
    }
    // a row of tiles at a time: the next row's operands are read, and the last row's sums added, beside its products
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (i + 1 < NI) read_m(buf, i + 1);
      __builtin_amdgcn_sched_barrier(0);  // reads stay before: the compiler would leave them for the end, to be waited for
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i == 0 ? NI - 1 : i - 1][j] += t[(i + NT - 1) % NT][j];
#pragma unroll
      for (int j = 0; j < NJ; ++j) t[i % NT][j] = times(ml[i & 1], nh[j], f32x4{0, 0, 0, 0});
#pragma unroll
      for (int j = 0; j < NJ; ++j) t[i % NT][j] = times(mh[i & 1], nl[j], t[i % NT][j]);
#pragma unroll
      for (int j = 0; j < NJ; ++j) t[i % NT][j] = times(mh[i & 1], nh[j], t[i % NT][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[NI - 1][j] += t[NT - 1][j];
  if constexpr (SPLIT) {
    float4* dst = (float4*)A.part + (((z * A.splits + blockIdx.y) * A.tiles + tile) * WAVES + w) * (NI * NJ * 64) + lane;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        dst[(i * NJ + j) * 64] = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
  } else if constexpr (SYM) {  // lane (g, n) has rows 4 g + e of column n
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      orth_square<EPI, NJ>(A, z, r0 + wr + 16 * i + 4 * g, c0 + wc + n, acc[i], bj < bi * (TM / TN));
      if constexpr (EPI == ORTH_POLY && NI > 6) __builtin_amdgcn_sched_barrier(0);  // (all rows' loads at once would not fit the registers)
    }
  } else {  // lane (g, n) has columns 4 g + e of row n
    const int c = c0 + wc + 4 * g;
    float4 e[NJ], en[NJ];
    f32x4 sq[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      e[j] = *(const float4*)(A.e + z * A.cols + c + 16 * j);
      en[j] = EPI == ORTH_NEXT ? *(const float4*)(A.en + z * A.cols + c + 16 * j) : e[j];
      sq[j] = f32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
      orth_next<EPI, NJ>(A, z, r0 + wr + 16 * i + n, c, acc[i], e, en, sq, bj == 0 && wc == 0 && g == 0);
    if constexpr (EPI == ORTH_NEXT) {
      float* to = A.squares + (z * A.sums + bi * WR + w / WC) * A.cols + c;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float4 t = make_float4(row16_sum(sq[j][0]), row16_sum(sq[j][1]), row16_sum(sq[j][2]), row16_sum(sq[j][3]));
        if (n == 0) *(float4*)(to + 16 * j) = t;
      }
    }
  }
}

// The parts of X X^T's split contraction added in order, and its epilogue.  A wave takes one row of a wave tile's 16 x 16 tiles.
template <int TM, int TN, int WR, int WC>
__global__ void __launch_bounds__(256) m2rnn_orth_join_kernel(OrthArgs A) {
  constexpr int NI = TM / WR / 16, NJ = TN / WC / 16, WAVES = WR * WC;
  const int lane = threadIdx.x & 63;
  const long z = blockIdx.z;
  const int item = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
  if (item >= A.tiles * WAVES * NI) return;
  const int i = item % NI, w = item / NI % WAVES, tile = item / (NI * WAVES);
  int bi, bj;
  orth_place<true, TM / TN>(tile, A.gi, A.gj, bi, bj);
  const int n = lane & 15, g = lane >> 4;
  const int r = bi * TM + (w / WC) * (TM / WR) + 16 * i, c = bj * TN + (w % WC) * (TN / WC);
  f32x4 acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = f32x4{0, 0, 0, 0};
  for (int s = 0; s < A.splits; ++s) {
    const f32x4* src = (const f32x4*)A.part + (((z * A.splits + s) * A.tiles + tile) * WAVES + w) * (NI * NJ * 64) + i * NJ * 64 + lane;
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] += src[j * 64];
  }
  orth_square<ORTH_GRAM, NJ>(A, z, r + 4 * g, c + n, acc, bj < bi * (TM / TN));
}

// Small matrices (768 of 64 x 64: 39 us, of which 9 are the scales and the second set of planes; the launches of the larger
// ones' kernels took 1253; LDS and VALU at 54 and 62% of the cycles): one workgroup takes a matrix through all its steps, X in
// registers (fp32) and as planes in LDS (R, then C in its place), D^-1 A and then D^-1 B as planes in LDS.  MP x NP the padded
// size; WR x WC waves over the 16 x 16 tiles of A and of X.  A lane holds four rows of a column, which are neighbours in the
// transpose: X lies transposed in LDS (its rows are read by transposing reads), and S = R R^T and (D^-1 A) (D^-1 A)^T are
// symmetric.
template <int MP, int NP, int WR, int WC>
__global__ void __launch_bounds__(64 * WR * WC) m2rnn_orth_small_kernel(const void* gin, void* out, int m, int n, int tall,
                                                                        int bf16, int steps, OrthCoefs coefs, float eps) {
  constexpr int ST = ssm_stride(MP);  // elements between rows of the transpose of X, and of A
  constexpr int AI = MP / 16 / WR, AJ = MP / 16 / WC, XJ = NP / 16 / WC;
  __shared__ __attribute__((aligned(16))) uint16_t xp[2][NP * ST], ap[2][MP * ST];
  __shared__ double red[WR * WC];
  __shared__ __attribute__((aligned(16))) float of_rows[WC][MP], of_cols[WR][NP];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int g = lane >> 4, l = lane & 15;
  const int r0 = (w / WC) * (MP / WR), ca = (w % WC) * (MP / WC), cx = (w % WC) * (NP / WC);
  const long at = (long)blockIdx.x * m * n;
  float x[AI][XJ][4];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < AI; ++i)
#pragma unroll
    for (int j = 0; j < XJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 16 * i + 4 * g + e, c = cx + 16 * j + l;
        float t = 0.0f;
        if (r < m && c < n) {
          const long o = at + (tall ? (long)c * m + r : (long)r * n + c);
          t = bf16 ? load1<true>(gin, o) : load1<false>(gin, o);
        }
        x[i][j][e] = t;
        ss += (double)t * (double)t;
      }
  ss = wave_sum(ss);
  if (lane == 0) red[w] = ss;
  __syncthreads();
  ss = 0.0;
#pragma unroll
  for (int i = 0; i < WR * WC; ++i) ss += red[i];
  const double scale = 1.0 / (sqrt(ss) + (double)eps);
  // four rows of a column as one write for each plane
  auto put4 = [&](const float (&v)[4], uint16_t* hi, uint16_t* lo, int row, int col) {
    uint16_t h[4], t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split_f16(v[e], h[e], t[e]);
    *(uint2*)(hi + row * ST + col) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
    *(uint2*)(lo + row * ST + col) = make_uint2(t[0] | (uint32_t)t[1] << 16, t[2] | (uint32_t)t[3] << 16);
  };
#pragma unroll
  for (int i = 0; i < AI; ++i)
#pragma unroll
    for (int j = 0; j < XJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][j][e] = (float)((double)x[i][j][e] * scale);
  // The scales of this lane's rows and columns.  post: each wave's part of the rows' and columns' largest values (FIRST), or of their
  // sums of squares over the scales that they have; take, behind a barrier: the scales.
  float d[AI][4], ec[XJ];
  auto post = [&](auto first) {
    constexpr bool FIRST = decltype(first)::value;
    auto with = [](float p, float q) { return FIRST ? fmaxf(p, q) : p + q; };
    float rows[AI][4], cols[XJ];
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) rows[i][e] = 0.0f;
#pragma unroll
    for (int j = 0; j < XJ; ++j) {
      cols[j] = 0.0f;
      const float by = FIRST ? 1.0f : pow2_inverse(ec[j]);
#pragma unroll
      for (int i = 0; i < AI; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (FIRST) {
            rows[i][e] = fmaxf(rows[i][e], fabsf(x[i][j][e]));
            cols[j] = fmaxf(cols[j], fabsf(x[i][j][e]));
          } else {
            const float r = x[i][j][e] * pow2_inverse(d[i][e]), c = x[i][j][e] * by;
            rows[i][e] = __builtin_fmaf(r, r, rows[i][e]);
            cols[j] = __builtin_fmaf(c, c, cols[j]);
          }
        }
    }
#pragma unroll
    for (int i = 0; i < AI; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float r = rows[i][e];
        r = with(r, dpp_all<kDppQuadXor1>(r));
        r = with(r, dpp_all<kDppQuadXor2>(r));
        r = with(r, dpp_all<kDppRowHalfMirror>(r));
        rows[i][e] = with(r, dpp_all<kDppRowMirror>(r));
      }
      if (l == 0) *(float4*)&of_rows[w % WC][r0 + 16 * i + 4 * g] = make_float4(rows[i][0], rows[i][1], rows[i][2], rows[i][3]);
    }
#pragma unroll
    for (int j = 0; j < XJ; ++j) {
      float c = cols[j];
      c = with(c, __shfl_xor(c, 16));
      c = with(c, __shfl_xor(c, 32));
      if (g == 0) of_cols[w / WC][cx + 16 * j + l] = c;
    }
  };
  auto take = [&](auto first) {
    constexpr bool FIRST = decltype(first)::value;
    auto with = [](float p, float q) { return FIRST ? fmaxf(p, q) : p + q; };
#pragma unroll
    for (int i = 0; i < AI; ++i) {
      float r[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < WC; ++k) {
        const float4 t = *(const float4*)&of_rows[k][r0 + 16 * i + 4 * g];
        r[0] = with(r[0], t.x);
        r[1] = with(r[1], t.y);
        r[2] = with(r[2], t.z);
        r[3] = with(r[3], t.w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i][e] = FIRST ? first_scale(r[e], NP) : next_scale(d[i][e], r[e], 0);
    }
#pragma unroll
    for (int j = 0; j < XJ; ++j) {
      float c = 0.0f;
#pragma unroll
      for (int k = 0; k < WR; ++k) c = with(c, of_cols[k][cx + 16 * j + l]);
      ec[j] = FIRST ? first_scale(c, MP) : next_scale(ec[j], c, 0);
    }
  };
  // X's planes: R (by rows) or C
  auto put_x = [&](auto by_rows) {
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < XJ; ++j) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = x[i][j][e] * (kOrthX * pow2_inverse(decltype(by_rows)::value ? d[i][e] : ec[j]));
        put4(v, xp[0], xp[1], cx + 16 * j + l, r0 + 16 * i + 4 * g);
      }
  };
  post(std::true_type{});
  __syncthreads();
  take(std::true_type{});
  put_x(std::true_type{});
  // this wave's AI x AJ tiles of R R^T (R's rows read from the transpose's columns) or of (D^-1 A) (D^-1 A)^T
  auto square = [&](auto of_x, f32x4 (&acc)[AI][AJ]) {
    constexpr bool X = decltype(of_x)::value;
    const uint16_t *hi = X ? xp[0] : ap[0], *lo = X ? xp[1] : ap[1];
    auto operand = [&](const uint16_t* p, int r, int k) { return X ? lds_col(p, ST, k, r, g, l) : lds_row(p, ST, r, k, g, l); };
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < AJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    for (int k = 0; k < (X ? NP : MP); k += 32) {
      uint4 nh[AJ], nl[AJ];
#pragma unroll
      for (int j = 0; j < AJ; ++j) {
        nh[j] = operand(hi, ca + 16 * j, k);
        nl[j] = operand(lo, ca + 16 * j, k);
      }
#pragma unroll
      for (int i = 0; i < AI; ++i) {
        const uint4 mh = operand(hi, r0 + 16 * i, k), ml = operand(lo, r0 + 16 * i, k);
        f32x4 t[AJ];
#pragma unroll
        for (int j = 0; j < AJ; ++j) t[j] = mfma_f16(ml, nh[j], f32x4{0, 0, 0, 0});
#pragma unroll
        for (int j = 0; j < AJ; ++j) t[j] = mfma_f16(mh, nl[j], t[j]);
#pragma unroll
        for (int j = 0; j < AJ; ++j) t[j] = mfma_f16(mh, nh[j], t[j]);
#pragma unroll
        for (int j = 0; j < AJ; ++j) acc[i][j] += t[j];
      }
    }
  };
  auto put_a = [&](const float (&v)[AI][AJ][4]) {
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < AJ; ++j) put4(v[i][j], ap[0], ap[1], ca + 16 * j + l, r0 + 16 * i + 4 * g);
  };
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const float fa = coefs.c[3 * s], fb = coefs.c[3 * s + 1], fc = coefs.c[3 * s + 2], unit = coefs.unit[s];
    const float back = 1.0f / (unit * kOrthX);
    f32x4 acc[AI][AJ];
    float a[AI][AJ][4];
    square(std::true_type{}, acc);
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < AJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) a[i][j][e] = acc[i][j][e] * (kOrthA / (kOrthX * kOrthX)) * d[i][e];
    if (fc != 0.0f) {
      put_a(a);
      __syncthreads();
      square(std::false_type{}, acc);
      put_x(std::false_type{});  // (all waves have read R)
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < AJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          a[i][j][e] = __builtin_fmaf(fb * (unit / kOrthA), a[i][j][e],
                                      fc == 0.0f ? 0.0f : fc * (unit / (kOrthA * kOrthA)) * acc[i][j][e] * d[i][e]);
    put_a(a);
    __syncthreads();
    if (fc == 0.0f) {
      put_x(std::false_type{});
      __syncthreads();
    }
    f32x4 y[AI][XJ];
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < XJ; ++j) y[i][j] = f32x4{0, 0, 0, 0};
    for (int k = 0; k < MP; k += 32) {
      uint4 nh[XJ], nl[XJ];
#pragma unroll
      for (int j = 0; j < XJ; ++j) {
        nh[j] = lds_row(xp[0], ST, cx + 16 * j, k, g, l);
        nl[j] = lds_row(xp[1], ST, cx + 16 * j, k, g, l);
      }
#pragma unroll
      for (int i = 0; i < AI; ++i) {
        const uint4 mh = lds_row(ap[0], ST, r0 + 16 * i, k, g, l), ml = lds_row(ap[1], ST, r0 + 16 * i, k, g, l);
        f32x4 t[XJ];
#pragma unroll
        for (int j = 0; j < XJ; ++j) t[j] = mfma_f16(ml, nh[j], f32x4{0, 0, 0, 0});
#pragma unroll
        for (int j = 0; j < XJ; ++j) t[j] = mfma_f16(mh, nl[j], t[j]);
#pragma unroll
        for (int j = 0; j < XJ; ++j) t[j] = mfma_f16(mh, nh[j], t[j]);
#pragma unroll
        for (int j = 0; j < XJ; ++j) y[i][j] += t[j];
      }
    }
#pragma unroll
    for (int i = 0; i < AI; ++i)
#pragma unroll
      for (int j = 0; j < XJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][j][e] = __builtin_fmaf(fa, x[i][j][e], y[i][j][e] * (d[i][e] * back) * ec[j]);
    if (s + 1 < steps) {
      post(std::false_type{});
      __syncthreads();
      take(std::false_type{});
      put_x(std::true_type{});
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < AI; ++i)
#pragma unroll
    for (int j = 0; j < XJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = r0 + 16 * i + 4 * g + e, c = cx + 16 * j + l;
        if (r < m && c < n) {
          const long o = at + (tall ? (long)c * m + r : (long)r * n + c);
          const float v = x[i][j][e];
          if (bf16)
            ((__bf16*)out)[o] = (__bf16)v;
          else
            ((float*)out)[o] = v;
        }
      }
}

// Thin matrices (the shorter side at most 32): the fp32 MFMA, whose rate no longer matters, and no splitting: with few rows the
// 22 bits of split values would show (a single row of 100: 1.5e-6 off where fp32 products are 6e-7).
//
// A wave holds M rows (16 or 32) by 64 columns of X in accumulator order: lane (h, i) has row i, and in register r of
// each M columns column col(r, h).  That is an operand of X X^T over those columns, in some order that is the same on
// both sides.  A comes out in the same order and is symmetric, so its registers are operands of A A, and B's of
// (B X)^T = X^T B, whose other operand, X by columns, comes from LDS; the result has X's order again.
template <int M>
struct Thin {
  static constexpr int H = 64 / M, NR = M * M / 64, NC = 64 / M;  // lanes of a row; registers of M columns; those of a wave
  static constexpr int ST = 68;                                   // floats between rows in LDS
  typedef float acc_t __attribute__((ext_vector_type(NR)));
  static __device__ __forceinline__ acc_t mfma(float a, float b, acc_t c) {
    if constexpr (M == 32)
      return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ acc_t zero() {
    acc_t z;
#pragma unroll
    for (int r = 0; r < NR; ++r) z[r] = 0.0f;
    return z;
  }
  static __device__ __forceinline__ int col(int r, int h) { return 4 * H * (r / 4) + 4 * h + r % 4; }
};

struct ThinArgs {
  const void* g;
  void* out;
  float* X;              // several workgroups: X, [batch][tiles][waves] in the waves' order
  float* part;           // and the partial sums of A, [2][batch][workgroups][lane][NR], the halves in turn
  const double* squares; // and the partial sums of squares [batch][parts]
  int m, n, tall, bf16;  // m x n with m the shorter side; g and out are its transpose if tall
  int tiles, parts, steps;
  float eps, ca, cb, cc;
  int turn;
};

enum { THIN_ALL = 0, THIN_FIRST = 1, THIN_MIDDLE = 2, THIN_LAST = 3 };

// THIN_ALL: one workgroup takes a matrix of up to 64 WAVES columns through all steps.  The others: a step's launch, where a
// workgroup takes every gridDim.x-th tile of 64 WAVES columns: FIRST forms X_0 and its A, MIDDLE applies the step that the
// last launch's A gives and sums the next A, LAST applies the last one.
template <int M, int WAVES, int MODE>
__global__ void __launch_bounds__(64 * WAVES) m2rnn_orth_thin_kernel(ThinArgs A, OrthCoefs coefs) {
  typedef Thin<M> T;
  constexpr int NR = T::NR, NC = T::NC, H = T::H;
  __shared__ float xs[WAVES][M * T::ST];
  __shared__ float4 sums[WAVES][NR / 4][64];
  __shared__ double red[WAVES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int i = lane % M, h = lane / M;
  const long z = blockIdx.y;
  const long at = z * A.m * A.n;
  float x[NC][NR];
  auto place = [&](int tile, int ch, int r) { return (tile * WAVES + w) * 64 + ch * M + T::col(r, h); };  // the column
  auto where = [&](int c) { return at + (A.tall ? (long)c * A.m + i : (long)i * A.n + c); };
  auto load_g = [&](int tile) {
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int c = place(tile, ch, r);
        x[ch][r] = 0.0f;
        if (i < A.m && c < A.n) x[ch][r] = A.bf16 ? load1<true>(A.g, where(c)) : load1<false>(A.g, where(c));
      }
  };
  auto store_out = [&](int tile) {
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int c = place(tile, ch, r);
        if (i < A.m && c < A.n) {
          if (A.bf16)
            ((__bf16*)A.out)[where(c)] = (__bf16)x[ch][r];
          else
            ((float*)A.out)[where(c)] = x[ch][r];
        }
      }
  };
  auto kept = [&](int tile) { return (float4*)A.X + ((z * A.tiles + tile) * WAVES + w) * (NC * NR / 4 * 64) + lane; };
  auto scale_by = [&](double f) {
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
#pragma unroll
      for (int r = 0; r < NR; ++r) x[ch][r] = (float)((double)x[ch][r] * f);
  };
  auto add_gram = [&](typename T::acc_t a) {
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
#pragma unroll
      for (int r = 0; r < NR; ++r) a = T::mfma(x[ch][r], x[ch][r], a);
    return a;
  };
  // the waves' a added, in each of them
  auto over_waves = [&](typename T::acc_t a) {
    if constexpr (WAVES == 1) return a;
    __syncthreads();  // the sums of the time before have been read
#pragma unroll
    for (int q = 0; q < NR / 4; ++q) sums[w][q][lane] = make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
    __syncthreads();
    a = T::zero();
#pragma unroll
    for (int v = 0; v < WAVES; ++v)
#pragma unroll
      for (int q = 0; q < NR / 4; ++q) {
        const float4 t = sums[v][q][lane];
        a[4 * q] += t.x;
        a[4 * q + 1] += t.y;
        a[4 * q + 2] += t.z;
        a[4 * q + 3] += t.w;
      }
    return a;
  };
  auto poly = [&](typename T::acc_t a, float b, float c) {
    typename T::acc_t sq = T::zero();
#pragma unroll
    for (int r = 0; r < NR; ++r) sq = T::mfma(a[r], a[r], sq);
#pragma unroll
    for (int r = 0; r < NR; ++r) a[r] = c == 0.0f ? b * a[r] : __builtin_fmaf(b, a[r], c * sq[r]);
    return a;
  };
  auto apply = [&](typename T::acc_t B, float ca) {
    float* mine = xs[w];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();  // the wave's reads of the time before
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
#pragma unroll
      for (int r = 0; r < NR; r += 4)
        *(float4*)(mine + i * T::ST + ch * M + T::col(r, h)) =
            make_float4(x[ch][r], x[ch][r + 1], x[ch][r + 2], x[ch][r + 3]);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int ch = 0; ch < NC; ++ch) {
      typename T::acc_t y = T::zero();
#pragma unroll
      for (int r = 0; r < NR; ++r) y = T::mfma(mine[T::col(r, h) * T::ST + ch * M + i], B[r], y);
#pragma unroll
      for (int r = 0; r < NR; ++r) x[ch][r] = __builtin_fmaf(ca, x[ch][r], y[r]);
    }
  };
  if constexpr (MODE == THIN_ALL) {
    load_g(0);
    double ss = 0.0;
#pragma unroll
    for (int ch = 0; ch < NC; ++ch)
#pragma unroll
      for (int r = 0; r < NR; ++r) ss += (double)x[ch][r] * (double)x[ch][r];
    ss = wave_sum(ss);
    if (lane == 0) red[w] = ss;
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) ss += red[v];
    scale_by(1.0 / (sqrt(ss) + (double)A.eps));
    for (int s = 0; s < A.steps; ++s)
      apply(poly(over_waves(add_gram(T::zero())), coefs.c[3 * s + 1], coefs.c[3 * s + 2]), coefs.c[3 * s]);
    store_out(0);
  } else {
    const long half = (long)gridDim.y * gridDim.x * 64 * NR;
    typename T::acc_t a = T::zero(), B = T::zero();
    double f = 0.0;
    if constexpr (MODE == THIN_FIRST) {
      for (int k = lane; k < A.parts; k += 64) f += A.squares[z * A.parts + k];
      f = 1.0 / (sqrt(wave_sum(f)) + (double)A.eps);
    } else {
      // the last launch's sums of A: a wave takes every WAVES-th, in fp64
      double t[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) t[r] = 0.0;
      const float4* p = (const float4*)(A.part + (A.turn ^ 1) * half) + z * gridDim.x * (16 * NR) + lane * (NR / 4);
      for (int k = w; k < (int)gridDim.x; k += WAVES)
#pragma unroll
        for (int q = 0; q < NR / 4; ++q) {
          const float4 v = p[k * (16 * NR) + q];
          t[4 * q] += (double)v.x;
          t[4 * q + 1] += (double)v.y;
          t[4 * q + 2] += (double)v.z;
          t[4 * q + 3] += (double)v.w;
        }
#pragma unroll
      for (int r = 0; r < NR; ++r) a[r] = (float)t[r];
      B = poly(over_waves(a), A.cb, A.cc);
      a = T::zero();
    }
    for (int tile = blockIdx.x; tile < A.tiles; tile += gridDim.x) {
      if constexpr (MODE == THIN_FIRST) {
        load_g(tile);
        scale_by(f);
      } else {
        const float4* src = kept(tile);
#pragma unroll
        for (int ch = 0; ch < NC; ++ch)
#pragma unroll
          for (int q = 0; q < NR / 4; ++q) {
            const float4 v = src[(ch * (NR / 4) + q) * 64];
            x[ch][4 * q] = v.x;
            x[ch][4 * q + 1] = v.y;
            x[ch][4 * q + 2] = v.z;
            x[ch][4 * q + 3] = v.w;
          }
        apply(B, A.ca);
      }
      if constexpr (MODE == THIN_LAST) {
        store_out(tile);
      } else {
        a = add_gram(a);
        float4* dst = kept(tile);
#pragma unroll
        for (int ch = 0; ch < NC; ++ch)
#pragma unroll
          for (int q = 0; q < NR / 4; ++q)
            dst[(ch * (NR / 4) + q) * 64] = make_float4(x[ch][4 * q], x[ch][4 * q + 1], x[ch][4 * q + 2], x[ch][4 * q + 3]);
      }
    }
    if constexpr (MODE != THIN_LAST) {
      a = over_waves(a);
      if (w == 0) {
        float4* p = (float4*)(A.part + A.turn * half) + (z * gridDim.x + blockIdx.x) * (16 * NR) + lane * (NR / 4);
#pragma unroll
        for (int q = 0; q < NR / 4; ++q) p[q] = make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
      }
    }
  }
}

}  // namespace m2rnn
