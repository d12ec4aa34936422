// C entry points of the q/k norm with rotation (include/m2rnn.h).
#include <hip/hip_runtime.h>

#include "../../include/m2rnn.h"
#include "m2rnn_qk_kernels.h"

using namespace m2rnn;

namespace m2rnn {
int record_hip_status(hipError_t e);
}  // namespace m2rnn

namespace {

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t round_up256(size_t x) { return (x + 255) & ~(size_t)255; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }

constexpr long kQkWaves = 8192;      // waves that a launch aims for (heads of a token split over waves)
// Workgroups of the backward, each of which writes one row of partial sums: four waves for each SIMD (16K tokens of
// 16 + 16 heads, K = 128: 114 us; with twice as many groups 119 us and longer final sums, with half as many 139 us).
constexpr long kQkMaxGroups = 1024;
// More than these where a lane would otherwise add more heads than this in fp32 (the rows are added in fp64): the sums of long
// batches cancel.  1M tokens of 64 heads, K = 64, take 32 times the rows: 16 MB beside tens of GB of gradients.
constexpr long kQkTerms = 64;

struct QkPlan {
  int LPH = 1, split = 1;
  long groups = 0;
};

int check_qk(int64_t B, int64_t T, int64_t Nq, int64_t Nk, int64_t K, int64_t R, int dtype, float eps) {
  if (B < 0 || T < 0 || Nq < 0 || Nk < 0 || K < 0 || R < 0 || R > K) return M2RNN_EINVAL;
  if (dtype != M2RNN_DTYPE_F32 && dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  if (!(eps >= 0.0f) || eps > 1e30f) return M2RNN_EINVAL;
  if (K == 0 || K % 16 != 0 || K > 256 || R % 8 != 0) return M2RNN_EUNSUPPORTED;
  if (Nq > (1 << 20) || Nk > (1 << 20) || (double)B * T > 1e12) return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

QkPlan plan_qk(long tokens, int heads, int K, bool bwd) {
  QkPlan p;
  while (p.LPH * 8 < K) p.LPH *= 2;
  const long passes = ceil_div(heads, 64 / p.LPH);
  long split = tokens > 0 ? ceil_div(kQkWaves, tokens) : 1;
  split = split > passes ? passes : split;
  p.split = (int)(split < 1 ? 1 : split);
  p.groups = ceil_div(tokens * p.split, kBlkThreads / 64);
  long most = 1L << 22;  // (a launch holds fewer than 2^32 threads)
  if (bwd) {
    const long enough = ceil_div(tokens * passes, kQkTerms * (kBlkThreads / 64));
    most = enough < kQkMaxGroups ? kQkMaxGroups : enough < most ? enough : most;
  }
  p.groups = p.groups > most ? most : p.groups;
  return p;
}

template <bool BF16, int LPH, bool BWD>
const void* pick_inter(bool inter) {
  return inter ? (const void*)&m2rnn_qk_norm_rope_kernel<BF16, LPH, true, BWD>
               : (const void*)&m2rnn_qk_norm_rope_kernel<BF16, LPH, false, BWD>;
}
template <bool BF16, bool BWD>
const void* pick_lanes(int LPH, bool inter) {
  switch (LPH) {
    case 2: return pick_inter<BF16, 2, BWD>(inter);
    case 4: return pick_inter<BF16, 4, BWD>(inter);
    case 8: return pick_inter<BF16, 8, BWD>(inter);
    case 16: return pick_inter<BF16, 16, BWD>(inter);
    default: return pick_inter<BF16, 32, BWD>(inter);
  }
}
template <bool BWD>
const void* pick_qk(bool bf16, int LPH, bool inter) {
  return bf16 ? pick_lanes<true, BWD>(LPH, inter) : pick_lanes<false, BWD>(LPH, inter);
}

int launch_qk(const void* kern, long groups, QkArgs& A, hipStream_t s) {
  void* args[] = {&A};
  return record_hip_status(hipLaunchKernel(kern, dim3((unsigned)groups), dim3(kBlkThreads), args, 0, s));
}

}  // namespace

extern "C" {

int m2rnn_qk_norm_rope_fwd(int64_t B, int64_t T, int64_t Nq, int64_t Nk, int64_t K, int64_t R, int interleaved,
                           int dtype, const void* q, const void* k, const float* gamma_q, const float* gamma_k,
                           const int32_t* pos, const double* inv_freq, float eps, void* q_out, void* k_out,
                           void* stream) {
  const int st = check_qk(B, T, Nq, Nk, K, R, dtype, eps);
  if (st) return st;
  if (B == 0 || T == 0 || Nq + Nk == 0) return M2RNN_OK;
  if (!gamma_q || !gamma_k || !pos || (R > 0 && !inv_freq)) return M2RNN_EINVAL;
  if ((Nq > 0 && (!q || !q_out)) || (Nk > 0 && (!k || !k_out))) return M2RNN_EINVAL;
  const void* ps[] = {q, k, gamma_q, gamma_k, inv_freq, q_out, k_out};
  for (const void* p : ps)
    if (p && !al16(p)) return M2RNN_EINVAL;
  if ((uintptr_t)pos & 3u) return M2RNN_EINVAL;
  const QkPlan p = plan_qk(B * T, (int)(Nq + Nk), (int)K, false);
  QkArgs A{q, k, gamma_q, gamma_k, (const int*)pos, inv_freq, nullptr, nullptr, q_out, k_out, nullptr, B * T,
           (int)Nq, (int)Nk, (int)K, (int)R / 2, p.split, eps};
  return launch_qk(pick_qk<false>(dtype == M2RNN_DTYPE_BF16, p.LPH, interleaved != 0), p.groups, A,
                   (hipStream_t)stream);
}

int m2rnn_qk_norm_rope_bwd_workspace_size(int64_t B, int64_t T, int64_t Nq, int64_t Nk, int64_t K, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_qk(B, T, Nq, Nk, K, 0, M2RNN_DTYPE_F32, 0.0f);
  if (st) return st;
  const QkPlan p = plan_qk(B * T, (int)(Nq + Nk), (int)K, true);
  *bytes = round_up256((size_t)p.groups * 2 * K * sizeof(float));
  return M2RNN_OK;
}

int m2rnn_qk_norm_rope_bwd(int64_t B, int64_t T, int64_t Nq, int64_t Nk, int64_t K, int64_t R, int interleaved,
                           int dtype, const void* q, const void* k, const float* gamma_q, const float* gamma_k,
                           const int32_t* pos, const double* inv_freq, float eps, const float* dq_out,
                           const float* dk_out, float* dq, float* dk, float* dgamma_q, float* dgamma_k,
                           void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_qk(B, T, Nq, Nk, K, R, dtype, eps);
  if (st) return st;
  if (!gamma_q || !gamma_k || !dgamma_q || !dgamma_k) return M2RNN_EINVAL;
  const bool any = B > 0 && T > 0 && Nq + Nk > 0;
  if (any && (!pos || (R > 0 && !inv_freq))) return M2RNN_EINVAL;
  if (any && ((Nq > 0 && (!q || !dq_out || !dq)) || (Nk > 0 && (!k || !dk_out || !dk)))) return M2RNN_EINVAL;
  const void* ps[] = {q, k, gamma_q, gamma_k, inv_freq, dq_out, dk_out, dq, dk, dgamma_q, dgamma_k};
  for (const void* p : ps)
    if (p && !al16(p)) return M2RNN_EINVAL;
  if ((uintptr_t)pos & 3u) return M2RNN_EINVAL;
  const QkPlan p = plan_qk(any ? B * T : 0, (int)(Nq + Nk), (int)K, true);
  size_t need = 0;
  st = m2rnn_qk_norm_rope_bwd_workspace_size(B, T, Nq, Nk, K, &need);
  if (st) return st;
  if (any && (!workspace || workspace_bytes < need || !al16(workspace))) return M2RNN_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  float* part = (float*)workspace;
  if (any) {
    QkArgs A{q, k, gamma_q, gamma_k, (const int*)pos, inv_freq, dq_out, dk_out, dq, dk, part, B * T,
             (int)Nq, (int)Nk, (int)K, (int)R / 2, p.split, eps};
    st = launch_qk(pick_qk<true>(dtype == M2RNN_DTYPE_BF16, p.LPH, interleaved != 0), p.groups, A, s);
    if (st) return st;
  }
  hipLaunchKernelGGL(m2rnn_qk_sums_kernel, dim3((unsigned)(K / 8)), dim3(1024), 0, s, (const float*)part,
                     any ? p.groups : 0, (int)K, dgamma_q, dgamma_k);
  return record_hip_status(hipGetLastError());
}

}  // extern "C"
