// C entry points of the gated linear recurrence of channels (include/m2rnn.h).
#include <hip/hip_runtime.h>

#include "../../include/m2rnn.h"
#include "m2rnn_gated_kernels.h"

using namespace m2rnn;

namespace m2rnn {
int record_hip_status(hipError_t e);
}  // namespace m2rnn

namespace {

constexpr long kGatedFewChunks = 128;  // up to this many chunks a group is half as long

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
long chunks(int64_t T, int steps) { return ceil_div(T, steps * kGatedWaves); }

int check_gated(int64_t B, int64_t T, int64_t D, int dtype) {
  if (B < 0 || T < 0 || D <= 0) return M2RNN_EINVAL;
  if (dtype != M2RNN_DTYPE_F32 && dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  if (D % 4 != 0 || D > (1 << 24) || T > (1L << 30) || (double)B * D > 34359738368.0) return M2RNN_EUNSUPPORTED;
  // a launch holds fewer than 2^32 threads
  if ((double)blocks(B, D) * (double)chunks(T, kGatedStepsBwd) >= 8388608.0) return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

// The workspace: the chunks' maps, the states that enter the groups of chunks, the ticket; none for one chunk.  The
// backward's has the chunks' partial sums of dalpha and dbeta behind it.
struct Layout {
  size_t maps = 0, entry = 0, ticket = 0;
  int group = 0;
  Layout(int64_t B, int64_t T, int64_t D, int steps) {
    const long n = chunks(T, steps);
    if (n < 2 || B == 0) return;
    const size_t row = (size_t)blocks(B, D) * 256 * 8;
    group = n <= kGatedFewChunks ? kGatedGroup / 2 : kGatedGroup;
    maps = n * row;
    entry = ceil_div(n, group) * row;
    ticket = 256;
  }
  size_t bytes() const { return maps + entry + ticket; }
};
size_t part_bytes(int64_t B, int64_t T, int64_t D) { return round_up256((size_t)chunks(T, kGatedStepsBwd) * B * D * sizeof(float2)); }

int launch(const void* kern, long groups, int threads, GatedArgs& A, hipStream_t s) {
  void* args[] = {&A};
  return record_hip_status(hipLaunchKernel(kern, dim3((unsigned)groups), dim3((unsigned)threads), args, 0, s));
}

// The sizes and the workspace of a call, and the clearing launch.
int begin(GatedArgs& A, int64_t B, int64_t T, int64_t D, int steps, void* workspace, hipStream_t s) {
  const Layout ws(B, T, D, steps);
  A.T = (int)T;
  A.cols = B * D;
  A.blocks = blocks(B, D);
  A.D = (int)D;
  A.chunks = (int)chunks(T, steps);
  A.group = ws.group ? ws.group : 1;
  A.maps = (unsigned long long*)workspace;
  A.entry = (unsigned long long*)((char*)workspace + ws.maps);
  A.ticket = (unsigned*)((char*)workspace + ws.maps + ws.entry);
  A.first_words = (long)((ws.maps + ws.entry) / 8);
  if (A.chunks < 2) return M2RNN_OK;
  const long groups = ceil_div(A.first_words, 8L * kBlkThreads);
  return launch((const void*)&m2rnn_gated_clear_kernel, groups > 2048 ? 2048 : groups, kBlkThreads, A, s);
}

// No steps: the state as it is (NULL: zeros).
int pass_state(const float* from, float* to, long n, hipStream_t s) {
  const long groups = ceil_div(n, 4L * kBlkThreads);
  hipLaunchKernelGGL(m2rnn_gated_state_kernel, dim3((unsigned)(groups > 65536 ? 65536 : groups)), dim3(kBlkThreads), 0, s,
                     from, to, n);
  return record_hip_status(hipGetLastError());
}

}  // namespace

extern "C" {

int m2rnn_gated_scan_fwd_workspace_size(int64_t B, int64_t T, int64_t D, int dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_gated(B, T, D, dtype);
  if (st) return st;
  *bytes = Layout(B, T, D, kGatedStepsFwd).bytes();
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
  const size_t need = Layout(B, T, D, kGatedStepsFwd).bytes();
  if (need > 0 && (!workspace || workspace_bytes < need || !al16(workspace))) return M2RNN_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  GatedArgs A{};
  A.v = v; A.a = a; A.alpha = alpha; A.beta = beta; A.lens = (const int*)lens; A.h0 = h0; A.y = y; A.h_T = h_T;
  const bool bf16 = dtype == M2RNN_DTYPE_BF16;
  if (T == 0)
    return h_T ? pass_state(h0, h_T, B * D, s) : M2RNN_OK;
  st = begin(A, B, T, D, kGatedStepsFwd, workspace, s);
  if (st) return st;
  return launch(bf16 ? (const void*)&m2rnn_gated_fwd_kernel<true> : (const void*)&m2rnn_gated_fwd_kernel<false>,
                A.blocks * A.chunks, 64 * kGatedWaves, A, s);
}

int m2rnn_gated_scan_bwd_workspace_size(int64_t B, int64_t T, int64_t D, int dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_gated(B, T, D, dtype);
  if (st) return st;
  *bytes = Layout(B, T, D, kGatedStepsBwd).bytes() + part_bytes(B, T, D);
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
  const size_t lay = Layout(B, T, D, kGatedStepsBwd).bytes(), need = lay + part_bytes(B, T, D);
  if (need > 0 && (!workspace || workspace_bytes < need || !al16(workspace))) return M2RNN_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  GatedArgs A{};
  A.v = v; A.a = a; A.alpha = alpha; A.beta = beta; A.lens = (const int*)lens; A.h0 = h0;
  A.yin = y; A.dy = dy; A.dh_T = dh_T; A.dv = dv; A.da = da; A.dh0 = dh0;
  A.part = (float2*)((char*)workspace + lay);
  if (n > 0) {
    st = begin(A, B, T, D, kGatedStepsBwd, workspace, s);
    if (st) return st;
    st = launch(dtype == M2RNN_DTYPE_BF16 ? (const void*)&m2rnn_gated_bwd_kernel<true> : (const void*)&m2rnn_gated_bwd_kernel<false>,
                A.blocks * A.chunks, 64 * kGatedWaves, A, s);
    if (st) return st;
  } else if (B > 0 && dh0) {
    st = pass_state(dh_T, dh0, B * D, s);
    if (st) return st;
  }
  hipLaunchKernelGGL(m2rnn_gated_sums_kernel, dim3((unsigned)ceil_div(D, 16)), dim3(1024), 0, s, (const float2*)A.part,
                     n > 0 ? (long)A.chunks * B : 0, (int)D, dalpha, dbeta);
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
