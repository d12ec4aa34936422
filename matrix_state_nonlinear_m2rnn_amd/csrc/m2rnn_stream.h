// Building blocks of the HBM-bound kernels: their workgroup size, and loads and stores of four
// consecutive fp32 or bf16 values.
#pragma once

#include "m2rnn_device.h"

namespace m2rnn {

constexpr int kBlkThreads = 256;

template <bool BF16>
__device__ __forceinline__ float4 load4(const void* base, long i) {
  if constexpr (BF16) {
    const uint2 r = *(const uint2*)((const uint16_t*)base + i);
    return make_float4(bf16_lo_to_f32(r.x), bf16_hi_to_f32(r.x), bf16_lo_to_f32(r.y), bf16_hi_to_f32(r.y));
  }
  return *(const float4*)((const float*)base + i);
}

// load4 as a non-temporal load, for streams read once.  (It helps the RMSNorm and the conv
// backward by 2-4%; the conv forward, whose x rows are also read by the neighbouring chunk's
// window, runs slower with it.)
template <bool BF16>
__device__ __forceinline__ float4 load4_nt(const void* base, long i) {
  if constexpr (BF16) {
    typedef unsigned u2v __attribute__((ext_vector_type(2)));
    const u2v r = __builtin_nontemporal_load((const u2v*)((const uint16_t*)base + i));
    return make_float4(bf16_lo_to_f32(r[0]), bf16_hi_to_f32(r[0]), bf16_lo_to_f32(r[1]), bf16_hi_to_f32(r[1]));
  }
  const f32x4 t = __builtin_nontemporal_load((const f32x4*)((const float*)base + i));
  return make_float4(t[0], t[1], t[2], t[3]);
}

template <bool BF16>
__device__ __forceinline__ void store4(void* base, long i, float4 v) {
  if constexpr (BF16) {
    *(uint2*)((uint16_t*)base + i) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  } else {
    *(float4*)((float*)base + i) = v;
  }
}

// store4 as a non-temporal store: the caches need not keep a stream written once and not read
// back by the kernel.
template <bool BF16>
__device__ __forceinline__ void store4_nt(void* base, long i, const float (&o)[4]) {
  if constexpr (BF16) {
    typedef unsigned u2v __attribute__((ext_vector_type(2)));
    const u2v v = {pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    __builtin_nontemporal_store(v, (u2v*)((uint16_t*)base + i));
  } else {
    typedef float f4v __attribute__((ext_vector_type(4)));
    const f4v v = {o[0], o[1], o[2], o[3]};
    __builtin_nontemporal_store(v, (f4v*)((float*)base + i));
  }
}

}  // namespace m2rnn
