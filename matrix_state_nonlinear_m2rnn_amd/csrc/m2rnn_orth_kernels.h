// Orthogonalised update: X_0 = G / (||G||_F + eps), then `steps` times, with A = X X^T over the shorter side,
//     X <- a X + (b A + c A A) X,
// which takes every singular value s of X to a s + b s^3 + c s^5 and leaves the singular vectors: with the usual
// coefficients all of them end near 1.
//
// Three matrix products a step, all of the form M N^T over rows that are contiguous along the contraction:
//     (1) A = X X^T (symmetric: its lower tiles, each written twice), (2) B = b A + c A A^T (likewise),
//     (3) X' = a X + B (X^T)^T, for which X^T is kept beside X.
// Precision.  Fp32 values are split into two fp16 planes x = hi + lo (22 bits) and a product takes three passes of the
// fp16 MFMA with fp32 accumulation (lo lo, below 2^-22 of the product, is left out): the error is that of fp32
// products, at eight times the fp32 MFMA's rate over three.  Values are kept times a power of two that holds fp16's range:
// X and A times 2^12, B times 2^11.  With singular values up to 1.25 (the usual coefficients' largest) the entries of X
// and A stay below 6.4e3 and those of B below 2.7e4 (fp16 ends at 6.5e4), and entries down to 2^-15 keep both planes whole.
#pragma once

#include "m2rnn_device.h"

namespace m2rnn {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kOrthX = 4096.0f, kOrthA = 4096.0f, kOrthB = 2048.0f;
constexpr int kOrthTile = 128;   // side of a workgroup's tile; sides are padded to it with zeros
constexpr int kOrthK = 32;       // contraction of a stage
constexpr int kOrthThreads = 256;

// Two fp16 planes of a matrix [rows][ld].
struct Planes {
  uint16_t *hi, *lo;
};

__device__ __forceinline__ void split_f16(float x, uint16_t& hi, uint16_t& lo) {
  const _Float16 h = (_Float16)x;
  const _Float16 l = (_Float16)(x - (float)h);
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, l);
}
__device__ __forceinline__ float join_f16(uint16_t hi, uint16_t lo) {
  return (float)__builtin_bit_cast(_Float16, hi) + (float)__builtin_bit_cast(_Float16, lo);
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, long i) {
  if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
  return ((const float*)p)[i];
}

// Partial sums of squares of a matrix in fp64: workgroup (p, matrix) of `parts`.
template <bool BF16>
__global__ void __launch_bounds__(256) m2rnn_orth_squares_kernel(const void* g, long mn, long each, double* part) {
  __shared__ double red[4];
  const long first = (long)blockIdx.x * each, last = first + each < mn ? first + each : mn;
  const long at = (long)blockIdx.y * mn;
  double acc = 0.0;
  for (long i = first + threadIdx.x; i < last; i += 256) {
    const double x = (double)load1<BF16>(g, at + i);
    acc += x * x;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) acc += __shfl_xor(acc, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = acc;
  __syncthreads();
  if (threadIdx.x == 0) part[(long)blockIdx.y * gridDim.x + blockIdx.x] = (red[0] + red[1]) + (red[2] + red[3]);
}

// X_0 times kOrthX as planes [mp][np] and their transposes [np][mp], zeros past m x n; m x n is G or, `tall`, its
// transpose.  A workgroup takes 64 x 64.
template <bool BF16>
__global__ void __launch_bounds__(256) m2rnn_orth_split_kernel(const void* g, int m, int n, int mp, int np, int tall,
                                                               const double* part, int parts, float eps, Planes X, Planes XT) {
  __shared__ float tile[64][65];
  const long z = blockIdx.z;
  double ss = 0.0;
  for (int i = 0; i < parts; ++i) ss += part[z * parts + i];
  const double scale = (double)kOrthX / (sqrt(ss) + (double)eps);
  const int r0 = blockIdx.y * 64, c0 = blockIdx.x * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const long at = z * m * n;
  for (int i = ty; i < 64; i += 4) {  // (i, tx) along G's own rows
    const int r = tall ? r0 + tx : r0 + i, c = tall ? c0 + i : c0 + tx;
    float x = 0.0f;
    if (r < m && c < n) x = (float)((double)load1<BF16>(g, at + (tall ? (long)c * m + r : (long)r * n + c)) * scale);
    tile[tall ? tx : i][tall ? i : tx] = x;
  }
  __syncthreads();
  const long plane = z * mp * np;
  for (int i = ty; i < 64; i += 4) {
    uint16_t hi, lo;
    split_f16(tile[i][tx], hi, lo);
    X.hi[plane + (long)(r0 + i) * np + c0 + tx] = hi;
    X.lo[plane + (long)(r0 + i) * np + c0 + tx] = lo;
    split_f16(tile[tx][i], hi, lo);
    XT.hi[plane + (long)(c0 + i) * mp + r0 + tx] = hi;
    XT.lo[plane + (long)(c0 + i) * mp + r0 + tx] = lo;
  }
}

// What a product's epilogue does with its tile.
enum { ORTH_GRAM = 0, ORTH_POLY = 1, ORTH_NEXT = 2, ORTH_LAST = 3 };

struct OrthArgs {
  Planes M, N;        // [rows][K], [cols][K]
  Planes E;           // POLY: A, NEXT and LAST: X, [rows][cols]
  Planes O, OT;       // outputs [rows][cols] and [cols][rows]
  void* out;          // LAST: [m][n], or [n][m] if tall
  int rows, cols, K;  // padded
  int m, n;
  int tall, out_bf16;
  float ca, cb, cc;
};

__device__ __forceinline__ f32x16 mfma32_f16(uint4 a, uint4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// One 128 x 128 tile of M N^T.  Four waves of 64 x 64, 32x32x16 MFMA.  A stage is 32 of the contraction: 64 bytes of
// each row of the four planes, in 16-byte units; unit u of row r is stored at u ^ ((r >> 1) & 3), so that the eight rows
// that a read touches at a time cover all banks.
template <int EPI>
__global__ void __launch_bounds__(kOrthThreads) m2rnn_orth_product_kernel(OrthArgs A) {
  constexpr bool SYM = EPI == ORTH_GRAM || EPI == ORTH_POLY;
  __shared__ uint4 lds[2][4][kOrthTile * 4];  // [buffer][M hi, M lo, N hi, N lo][row][unit]
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int bi = blockIdx.y, bj = blockIdx.x;
  if constexpr (SYM) {  // tiles of the lower triangle, numbered by rows
    const int id = blockIdx.x;
    bi = (int)((sqrtf(8.0f * (float)id + 1.0f) - 1.0f) * 0.5f);
    while ((bi + 1) * (bi + 2) / 2 <= id) ++bi;
    while (bi * (bi + 1) / 2 > id) --bi;
    bj = id - bi * (bi + 1) / 2;
  }
  const long z = blockIdx.z;
  const int r0 = bi * kOrthTile, c0 = bj * kOrthTile;
  const long mo = z * A.rows * A.K + (long)r0 * A.K, no = z * A.cols * A.K + (long)c0 * A.K;
  const uint16_t* src[4] = {A.M.hi + mo, A.M.lo + mo, A.N.hi + no, A.N.lo + no};
  // this thread's two units of each plane's stage
  const int row = threadIdx.x >> 2, unit = threadIdx.x & 3;
  const int slot0 = row * 4 + (unit ^ ((row >> 1) & 3)), slot1 = slot0 + 64 * 4;  // (64 rows on: the same exchange)
  const long off0 = (long)row * A.K + unit * 8, off1 = off0 + 64L * A.K;
  uint4 pre[8];
  auto fetch = [&](int k) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      pre[2 * p] = *(const uint4*)(src[p] + off0 + k);
      pre[2 * p + 1] = *(const uint4*)(src[p] + off1 + k);
    }
  };
  auto put = [&](int buf) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      lds[buf][p][slot0] = pre[2 * p];
      lds[buf][p][slot1] = pre[2 * p + 1];
    }
  };
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int wr = (w >> 1) * 64, wc = (w & 1) * 64, l32 = lane & 31, half = lane >> 5;
  fetch(0);
  put(0);
  __syncthreads();
  int buf = 0;
  for (int k = 0; k < A.K; k += kOrthK, buf ^= 1) {
    const bool more = k + kOrthK < A.K;
    if (more) fetch(k + kOrthK);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      uint4 mh[2], ml[2], nh[2], nl[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = wr + 32 * i + l32, c = wc + 32 * i + l32;
        const int ur = r * 4 + ((2 * kk + half) ^ ((r >> 1) & 3)), uc = c * 4 + ((2 * kk + half) ^ ((c >> 1) & 3));
        mh[i] = lds[buf][0][ur];
        ml[i] = lds[buf][1][ur];
        nh[i] = lds[buf][2][uc];
        nl[i] = lds[buf][3][uc];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          acc[i][j] = mfma32_f16(mh[i], nl[j], acc[i][j]);
          acc[i][j] = mfma32_f16(ml[i], nh[j], acc[i][j]);
          acc[i][j] = mfma32_f16(mh[i], nh[j], acc[i][j]);
        }
    }
    if (more) put(buf ^ 1);
    __syncthreads();
  }
  // lane l, register 4q + e: row 8q + 4 (l / 32) + e, column l % 32 of a 32 x 32 tile
  const long eo = z * A.rows * A.cols;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = r0 + wr + 32 * i + 8 * q + 4 * half, c = c0 + wc + 32 * j + l32;
        uint16_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = acc[i][j][4 * q + e];
          const long at = eo + (long)(r + e) * A.cols + c;
          if constexpr (EPI == ORTH_GRAM) {
            x *= kOrthA / (kOrthX * kOrthX);
          } else if constexpr (EPI == ORTH_POLY) {
            const float a = join_f16(A.E.hi[at], A.E.lo[at]);
            x = __builtin_fmaf(A.cb * (kOrthB / kOrthA), a, A.cc * (kOrthB / (kOrthA * kOrthA)) * x);
          } else {
            const float x0 = join_f16(A.E.hi[at], A.E.lo[at]);
            x = __builtin_fmaf(A.ca, x0, x * (1.0f / kOrthB));
          }
          if constexpr (EPI == ORTH_LAST) {
            x *= 1.0f / kOrthX;
            if (r + e < A.m && c < A.n) {
              const long o = z * A.m * A.n + (A.tall ? (long)c * A.m + r + e : (long)(r + e) * A.n + c);
              if (A.out_bf16)
                ((__bf16*)A.out)[o] = (__bf16)x;
              else
                ((float*)A.out)[o] = x;
            }
          } else {
            split_f16(x, hi[e], lo[e]);
            A.O.hi[at] = hi[e];
            A.O.lo[at] = lo[e];
          }
        }
        if constexpr (EPI != ORTH_LAST) {
          if (!SYM || bi != bj) {
            const long at = eo + (long)c * A.rows + r;
            *(uint2*)(A.OT.hi + at) = make_uint2(hi[0] | (uint32_t)hi[1] << 16, hi[2] | (uint32_t)hi[3] << 16);
            *(uint2*)(A.OT.lo + at) = make_uint2(lo[0] | (uint32_t)lo[1] << 16, lo[2] | (uint32_t)lo[3] << 16);
          }
        }
      }
}

}  // namespace m2rnn
