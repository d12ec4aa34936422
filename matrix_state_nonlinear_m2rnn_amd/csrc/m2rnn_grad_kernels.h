// Global norm of many gradient tensors, and their clipping:
//     norm = sqrt(sum over all tensors of g^2),   g <- g min(1, max_norm / norm).
//
// HBM streams: one read for the norm, one read and one write for the scaling (no write where nothing
// is to be clipped in place).  The tensors of a launch are its arguments, so nothing is copied to
// the device beforehand and a captured launch keeps its own list.  A workgroup takes one piece of one
// tensor.  Squares are summed in fp64 (a gradient of 1e-25 or 1e25 neither vanishes nor overflows
// when squared), in a fixed order: the same list gives the same bits.
//
// Measured, the gradients of 24 layers (4.07 GB in 288 fp32 tensors, three launches each): norm 0.60 ms, 6.8 TB/s;
// scaling 1.59 ms, 5.1 TB/s read and written.  48 small tensors: 4.4 + 2.3 + 4.7 us, a launch each.
#pragma once

#include "m2rnn_stream.h"

namespace m2rnn {

constexpr int kGradMax = 140;  // tensors per launch: 28 bytes each of the 4 KiB of kernel arguments

struct GradArgs {
  const void* src[kGradMax];
  void* dst[kGradMax];
  long numel[kGradMax];
  int first[kGradMax];  // the tensor's first piece within the launch
  int tensors;
  int piece;            // elements per piece, a multiple of 8 * 256
  unsigned bf16[(kGradMax + 31) / 32];
  double* part;         // norm: one partial per piece of the launch
  const float* norm;    // clip
  float max_norm;
  int in_place;
};

// The tensor that piece i belongs to (first[] is ascending; empty tensors have no piece).
__device__ __forceinline__ int grad_tensor(const GradArgs& A, int i) {
  int lo = 0, hi = A.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (A.first[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float grad_get(const void* p, long i, bool bf) {
  return bf ? bf16_lo_to_f32(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}
__device__ __forceinline__ void grad_put(void* p, long i, float x, bool bf) {
  if (bf)
    ((uint16_t*)p)[i] = (uint16_t)pack_bf16(x, 0.0f);
  else
    ((float*)p)[i] = x;
}

// Elements before the first 16-byte boundary.
__device__ __forceinline__ int grad_head(const void* p, int size) {
  return (int)((16 - ((uintptr_t)p & 15)) & 15) / size;
}

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// f(value) over 16 bytes of fp32 or bf16.
template <bool BF16, typename F>
__device__ __forceinline__ void grad_each(u32x4 v, F&& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f(bf16_lo_to_f32(v[i]));
      f(bf16_hi_to_f32(v[i]));
    } else {
      f(__uint_as_float(v[i]));
    }
  }
}
// The clip factor as c * s, s a power of two: 1, or 2^-64 where the factor itself would be near or below fp32's smallest
// normal number and lose bits (the products are then formed 2^64 larger, which no gradient within the norm overflows).
struct GradFactor {
  float c, s;
  __device__ __forceinline__ float operator()(float x) const { return x * c * s; }
};
__device__ __forceinline__ GradFactor grad_factor(float norm, float max_norm) {
  if (!(norm > max_norm && norm <= 3.4028234e38f)) return {1.0f, 1.0f};
  const double f = (double)max_norm / (double)norm;
  if (f < 0x1p-100) return {(float)(f * 0x1p64), 0x1p-64f};
  return {(float)f, 1.0f};
}

template <bool BF16>
__device__ __forceinline__ u32x4 grad_scaled(u32x4 v, GradFactor c) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16)
      o[i] = pack_bf16(c(bf16_lo_to_f32(v[i])), c(bf16_hi_to_f32(v[i])));
    else
      o[i] = __float_as_uint(c(__uint_as_float(v[i])));
  }
  return o;
}

__device__ __forceinline__ double block_sum64(double x, double* red) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) x += __shfl_xor(x, o);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < (int)blockDim.x / 64; ++i) s += red[i];
  return s;
}

template <bool BF16>
__device__ __forceinline__ double grad_squares(const char* p, long n) {
  constexpr int E = BF16 ? 8 : 4, SZ = BF16 ? 2 : 4;
  double s[2] = {0.0, 0.0};
  long head = grad_head(p, SZ);
  head = head < n ? head : n;
  auto one = [&](long i) {
    const double x = grad_get(p, i, BF16);
    s[0] = __builtin_fma(x, x, s[0]);
  };
  if ((long)threadIdx.x < head) one(threadIdx.x);
  const long vecs = (n - head) / E;
  const u32x4* v = (const u32x4*)(p + head * SZ);
#pragma unroll 4
  for (long i = threadIdx.x; i < vecs; i += kBlkThreads) {
    int k = 0;
    grad_each<BF16>(__builtin_nontemporal_load(v + i), [&](float x) {
      s[k & 1] = __builtin_fma((double)x, (double)x, s[k & 1]);
      ++k;
    });
  }
  const long tail = head + vecs * E + threadIdx.x;
  if (tail < n) one(tail);
  return s[0] + s[1];
}

__global__ void __launch_bounds__(kBlkThreads) m2rnn_grad_norm_kernel(GradArgs A) {
  __shared__ double red[kBlkThreads / 64];
  const int t = grad_tensor(A, blockIdx.x);
  const long i0 = (long)(blockIdx.x - A.first[t]) * A.piece;
  const long n = min((long)A.piece, A.numel[t] - i0);
  const bool bf = (A.bf16[t / 32] >> (t % 32)) & 1;
  const char* p = (const char*)A.src[t] + i0 * (bf ? 2 : 4);
  const double s = bf ? grad_squares<true>(p, n) : grad_squares<false>(p, n);
  const double total = block_sum64(s, red);
  if (threadIdx.x == 0) A.part[blockIdx.x] = total;
}

__global__ void __launch_bounds__(1024) m2rnn_grad_total_kernel(const double* part, long parts, float* norm) {
  __shared__ double red[16];
  double s = 0.0;
#pragma unroll 4
  for (long i = threadIdx.x; i < parts; i += 1024) s += part[i];
  const double total = block_sum64(s, red);
  if (threadIdx.x == 0) *norm = (float)sqrt(total);
}

template <bool BF16>
__device__ __forceinline__ void grad_scale(const char* p, char* o, long n, GradFactor c) {
  constexpr int E = BF16 ? 8 : 4, SZ = BF16 ? 2 : 4;
  long head = grad_head(p, SZ);
  // the vector path needs the same distance to a boundary on both sides
  if (head != grad_head(o, SZ)) {
    for (long i = threadIdx.x; i < n; i += kBlkThreads) grad_put(o, i, c(grad_get(p, i, BF16)), BF16);
    return;
  }
  head = head < n ? head : n;
  if ((long)threadIdx.x < head) grad_put(o, threadIdx.x, c(grad_get(p, threadIdx.x, BF16)), BF16);
  const long vecs = (n - head) / E;
  const u32x4* v = (const u32x4*)(p + head * SZ);
  u32x4* w = (u32x4*)(o + head * SZ);
#pragma unroll 4
  for (long i = threadIdx.x; i < vecs; i += kBlkThreads)
    __builtin_nontemporal_store(grad_scaled<BF16>(__builtin_nontemporal_load(v + i), c), w + i);
  const long tail = head + vecs * E + threadIdx.x;
  if (tail < n) grad_put(o, tail, c(grad_get(p, tail, BF16)), BF16);
}

// A norm that is not finite leaves the gradients as they are (the caller sees it in the norm and
// skips the step), as does one within max_norm.
__global__ void __launch_bounds__(kBlkThreads) m2rnn_grad_clip_kernel(GradArgs A) {
  const GradFactor c = grad_factor(*A.norm, A.max_norm);
  if (c.c == 1.0f && c.s == 1.0f && A.in_place) return;
  const int t = grad_tensor(A, blockIdx.x);
  const long i0 = (long)(blockIdx.x - A.first[t]) * A.piece;
  const long n = min((long)A.piece, A.numel[t] - i0);
  const bool bf = (A.bf16[t / 32] >> (t % 32)) & 1;
  const long off = i0 * (bf ? 2 : 4);
  if (bf)
    grad_scale<true>((const char*)A.src[t] + off, (char*)A.dst[t] + off, n, c);
  else
    grad_scale<false>((const char*)A.src[t] + off, (char*)A.dst[t] + off, n, c);
}

}  // namespace m2rnn
