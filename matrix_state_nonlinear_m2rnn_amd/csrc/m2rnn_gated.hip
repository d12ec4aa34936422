// C entry points of the gated linear recurrence of channels (include/m2rnn.h).
#include <hip/hip_runtime.h>

#include "../../include/m2rnn.h"
#include "m2rnn_gated_kernels.h"

using namespace m2rnn;

namespace m2rnn {
int record_hip_status(hipError_t e);
}  // namespace m2rnn

namespace {

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t round_up256(size_t x) { return (x + 255) & ~(size_t)255; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }

bool meet(const void* a, long na, const void* b, long nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

struct Span {
  const void* p;
  long bytes;
};
// Whether an output shares bytes with an input or with another output.
template <size_t NI, size_t NO>
bool any_meet(const Span (&in)[NI], const Span (&out)[NO]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < NI; ++j)
      if (meet(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
    for (size_t j = 0; j < i; ++j)
      if (meet(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

// Groups of 64 lanes of 4 channels, and chunks of steps.
long blocks(int64_t B, int64_t D) { return ceil_div(B * D / 4, 64); }
long chunks(int64_t T) { return ceil_div(T, kGatedChunk); }

int check_gated(int64_t B, int64_t T, int64_t D, int dtype) {
  if (B < 0 || T < 0 || D <= 0) return M2RNN_EINVAL;
  if (dtype != M2RNN_DTYPE_F32 && dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  if (D % 4 != 0 || D > (1 << 24) || T > (1L << 31) || (double)B * D > 34359738368.0) return M2RNN_EUNSUPPORTED;
  // a launch holds fewer than 2^32 threads
  if ((double)blocks(B, D) * (double)chunks(T) >= 8388608.0) return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

size_t agg_bytes(int64_t B, int64_t T, int64_t D) { return round_up256((size_t)chunks(T) * B * D * sizeof(float2)); }

int launch(const void* kern, long groups, int threads, GatedArgs& A, hipStream_t s) {
  void* args[] = {&A};
  return record_hip_status(hipLaunchKernel(kern, dim3((unsigned)groups), dim3((unsigned)threads), args, 0, s));
}

template <bool BACK>
int join(const GatedArgs& A, const float* first, float* last, hipStream_t s) {
  hipLaunchKernelGGL(m2rnn_gated_join_kernel<BACK>, dim3((unsigned)ceil_div(A.cols, kBlkThreads)), dim3(kBlkThreads), 0, s,
                     A.agg, A.cols, A.chunks, first, last);
  return record_hip_status(hipGetLastError());
}

}  // namespace

extern "C" {

int m2rnn_gated_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D, int dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_gated(B, T, D, dtype);
  if (st) return st;
  *bytes = agg_bytes(B, T, D);
  return M2RNN_OK;
}

int m2rnn_gated_scan_fwd(int64_t B, int64_t T, int64_t D, int dtype, const void* v, const void* a, const float* alpha,
                         const float* beta, const int32_t* lens, const float* h0, float* y, float* h_T, void* workspace,
                         size_t workspace_bytes, void* stream) {
  int st = check_gated(B, T, D, dtype);
  if (st) return st;
  if (B == 0) return M2RNN_OK;
  if (!alpha || !beta || (T > 0 && (!v || !a || !y))) return M2RNN_EINVAL;
  for (const void* p : {v, a, (const void*)alpha, (const void*)beta, (const void*)h0, (const void*)y, (const void*)h_T})
    if (p && !al16(p)) return M2RNN_EINVAL;
  if ((uintptr_t)lens & 3u) return M2RNN_EINVAL;
  const long n = B * T * D, e = dtype == M2RNN_DTYPE_BF16 ? 2 : 4;
  const Span in[] = {{v, n * e}, {a, n * e}, {alpha, 4 * D}, {beta, 4 * D}, {lens, 4 * B}, {h0, 4 * B * D}};
  const Span out[] = {{y, 4 * n}, {h_T, 4 * B * D}};
  if (any_meet(in, out)) return M2RNN_EINVAL;
  const size_t need = agg_bytes(B, T, D);
  if (need > 0 && (!workspace || workspace_bytes < need || !al16(workspace))) return M2RNN_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  GatedArgs A{};
  A.v = v; A.a = a; A.alpha = alpha; A.beta = beta; A.lens = (const int*)lens; A.h0 = h0; A.y = y; A.h_T = h_T;
  A.agg = (float2*)workspace;
  A.T = T; A.cols = B * D; A.D = (int)D; A.chunks = (int)chunks(T);
  const long groups = blocks(B, D) * A.chunks;
  const bool bf16 = dtype == M2RNN_DTYPE_BF16;
  if (groups > 0) {
    st = launch(bf16 ? (const void*)&m2rnn_gated_fwd_kernel<true, false> : (const void*)&m2rnn_gated_fwd_kernel<false, false>,
                groups, 64 * kGatedWaves, A, s);
    if (st) return st;
  }
  st = join<false>(A, h0, h_T, s);
  if (st || groups == 0) return st;
  return launch(bf16 ? (const void*)&m2rnn_gated_fwd_kernel<true, true> : (const void*)&m2rnn_gated_fwd_kernel<false, true>,
                groups, 64 * kGatedWaves, A, s);
}

int m2rnn_gated_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_gated(B, T, D, dtype);
  if (st) return st;
  *bytes = 2 * agg_bytes(B, T, D);
  return M2RNN_OK;
}

int m2rnn_gated_scan_bwd(int64_t B, int64_t T, int64_t D, int dtype, const void* v, const void* a, const float* alpha,
                         const float* beta, const int32_t* lens, const float* h0, const float* y, const float* dy,
                         const float* dh_T, float* dv, float* da, float* dalpha, float* dbeta, float* dh0,
                         void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_gated(B, T, D, dtype);
  if (st) return st;
  const long n = B * T * D, e = dtype == M2RNN_DTYPE_BF16 ? 2 : 4;
  if (!alpha || !beta || !dalpha || !dbeta || (n > 0 && (!v || !a || !y || !dy || !dv || !da))) return M2RNN_EINVAL;
  for (const void* p : {v, a, (const void*)alpha, (const void*)beta, (const void*)h0, (const void*)y, (const void*)dy,
                        (const void*)dh_T, (const void*)dv, (const void*)da, (const void*)dalpha, (const void*)dbeta,
                        (const void*)dh0})
    if (p && !al16(p)) return M2RNN_EINVAL;
  if ((uintptr_t)lens & 3u) return M2RNN_EINVAL;
  const Span in[] = {{v, n * e}, {a, n * e}, {alpha, 4 * D}, {beta, 4 * D}, {lens, 4 * B}, {h0, 4 * B * D}, {y, 4 * n},
                     {dy, 4 * n}, {dh_T, 4 * B * D}};
  const Span out[] = {{dv, 4 * n}, {da, 4 * n}, {dalpha, 4 * D}, {dbeta, 4 * D}, {dh0, 4 * B * D}};
  if (any_meet(in, out)) return M2RNN_EINVAL;
  const size_t half = agg_bytes(B, T, D);
  if (half > 0 && (!workspace || workspace_bytes < 2 * half || !al16(workspace))) return M2RNN_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  GatedArgs A{};
  A.v = v; A.a = a; A.alpha = alpha; A.beta = beta; A.lens = (const int*)lens; A.h0 = h0;
  A.yin = y; A.dy = dy; A.dh_T = dh_T; A.dv = dv; A.da = da; A.dh0 = dh0;
  A.agg = (float2*)workspace;
  A.part = (float2*)((char*)workspace + half);
  A.T = T; A.cols = B * D; A.D = (int)D; A.chunks = (int)chunks(T);
  const long groups = blocks(B, D) * A.chunks;
  const bool bf16 = dtype == M2RNN_DTYPE_BF16;
  if (groups > 0) {
    st = launch(bf16 ? (const void*)&m2rnn_gated_bwd_kernel<true, false> : (const void*)&m2rnn_gated_bwd_kernel<false, false>,
                groups, 64 * kGatedWaves, A, s);
    if (st) return st;
  }
  if (B > 0 && (dh0 || groups > 0)) {
    st = join<true>(A, dh_T, dh0, s);
    if (st) return st;
  }
  if (groups > 0) {
    st = launch(bf16 ? (const void*)&m2rnn_gated_bwd_kernel<true, true> : (const void*)&m2rnn_gated_bwd_kernel<false, true>,
                groups, 64 * kGatedWaves, A, s);
    if (st) return st;
  }
  hipLaunchKernelGGL(m2rnn_gated_sums_kernel, dim3((unsigned)ceil_div(D, 16)), dim3(1024), 0, s, (const float2*)A.part,
                     groups > 0 ? (long)A.chunks * B : 0, (int)D, dalpha, dbeta);
  return record_hip_status(hipGetLastError());
}

int m2rnn_gated_scan_step(int64_t B, int64_t D, int dtype, const void* v, const void* a, const float* alpha,
                          const float* beta, const float* h, float* h_out, void* stream) {
  const int st = check_gated(B, 1, D, dtype);
  if (st) return st;
  if (B == 0) return M2RNN_OK;
  if (!v || !a || !alpha || !beta || !h_out) return M2RNN_EINVAL;
  for (const void* p : {v, a, (const void*)alpha, (const void*)beta, (const void*)h, (const void*)h_out})
    if (p && !al16(p)) return M2RNN_EINVAL;
  const long n = B * D, e = dtype == M2RNN_DTYPE_BF16 ? 2 : 4;
  const Span in[] = {{v, n * e}, {a, n * e}, {alpha, 4 * D}, {beta, 4 * D}, {h == h_out ? nullptr : h, 4 * n}};
  const Span out[] = {{h_out, 4 * n}};
  if (any_meet(in, out)) return M2RNN_EINVAL;
  long groups = ceil_div(n / 4, kBlkThreads);
  groups = groups > (1 << 20) ? (1 << 20) : groups;
  if (dtype == M2RNN_DTYPE_BF16)
    hipLaunchKernelGGL(m2rnn_gated_step_kernel<true>, dim3((unsigned)groups), dim3(kBlkThreads), 0, (hipStream_t)stream, v, a,
                       alpha, beta, h, h_out, n, (int)D);
  else
    hipLaunchKernelGGL(m2rnn_gated_step_kernel<false>, dim3((unsigned)groups), dim3(kBlkThreads), 0, (hipStream_t)stream, v, a,
                       alpha, beta, h, h_out, n, (int)D);
  return record_hip_status(hipGetLastError());
}

}  // extern "C"
