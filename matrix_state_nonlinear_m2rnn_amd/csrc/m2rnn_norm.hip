// C entry points of the residual's addition with the RMSNorm (include/m2rnn.h).
#include <hip/hip_runtime.h>

#include "../../include/m2rnn.h"
#include "m2rnn_norm_kernels.h"

using namespace m2rnn;

namespace m2rnn {
int record_hip_status(hipError_t e);
}  // namespace m2rnn

namespace {

constexpr long kNormMaxD = 16384;   // 256 lanes of 64 features
constexpr long kNormFewRows = 2048; // up to this many rows a workgroup takes one row, not one a wave
// Workgroups of a launch: eight for each CU, four where a lane has the next row's loads in flight (85 -> 81 us at 32768 rows
// of 2048, bf16 to e4m3).
constexpr long kNormGroups = 2048, kNormGroups8 = 1024;
constexpr long kNormTerms = 64;     // rows that a lane of the backward adds in fp32, before the sums in fp64

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t round_up256(size_t x) { return (x + 255) & ~(size_t)255; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }
long elem(int dtype) { return dtype == M2RNN_DTYPE_F32 ? 4 : dtype == M2RNN_DTYPE_BF16 ? 2 : 1; }

// Whether two ranges share bytes.
bool meet(const void* a, long na, const void* b, long nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

int check_norm(int64_t rows, int64_t D, float eps) {
  if (rows < 0 || D <= 0) return M2RNN_EINVAL;
  if (!(eps >= 0.0f) || eps > 1e30f) return M2RNN_EINVAL;
  if (D % 4 != 0 || D > kNormMaxD || rows > 2147483647) return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

// Lanes of a row, groups of VEC features of a lane, workgroups.
struct Plan {
  int LPR, NG, VEC;
  long groups;
};

// Eight features at a time (16-byte loads) where everything that is read is bf16: 32768 rows of 2048 with a bf16 stream take 93 us
// instead of 165; in fp32, where a lane's two loads then share their lines with its neighbours', 217 instead of 187.
bool all_bf16(int x_dtype, const void* res, int res_dtype) {
  return x_dtype == M2RNN_DTYPE_BF16 && (!res || res_dtype == M2RNN_DTYPE_BF16);
}

// A wave takes a row of up to wave_most features, else a workgroup: 32768 rows of 2048 take 136 us by workgroups and 158 by waves
// where x is bf16 and the stream fp32, 194 and 187 where both are fp32, 107 and 101 in the backward.
Plan plan_norm(long rows, long D, bool bwd, bool wide, long wave_most) {
  Plan p;
  p.VEC = wide && D % 8 == 0 && D > 64 ? 8 : 4;
  if (p.VEC == 8) {
    p.LPR = D <= 128 ? 16 : D <= 512 || (rows > kNormFewRows && D <= 2048) ? 64 : 256;
  } else {
    p.LPR = D <= 16 ? 4 : D <= 64 ? 16 : (D <= 256 || (rows > kNormFewRows && D <= wave_most)) ? 64 : 256;
  }
  p.NG = 1;
  while ((long)p.VEC * p.LPR * p.NG < D) p.NG *= 2;
  const long all = ceil_div(rows, kBlkThreads / p.LPR);
  const long most = p.VEC == 8 ? kNormGroups8 : kNormGroups;
  p.groups = all < most ? all : most;
  if (bwd) {
    const long enough = ceil_div(all, kNormTerms);
    p.groups = p.groups > 512 ? 512 : p.groups;
    if (p.groups < enough) p.groups = enough;
  }
  return p;
}

template <int LPR, int NG>
struct Fwd {
  static const void* at(bool q8) {
    return q8 ? (const void*)&m2rnn_add_norm_kernel<LPR, NG, true> : (const void*)&m2rnn_add_norm_kernel<LPR, NG, false>;
  }
};
template <int LPR, int NG>
struct Bwd {
  static const void* at(bool) { return (const void*)&m2rnn_add_norm_bwd_kernel<LPR, NG>; }
};

template <template <int, int> class F>
const void* pick(const Plan& p, bool q8) {
  if (p.LPR == 4) return F<4, 1>::at(q8);
  if (p.LPR == 16) return F<16, 1>::at(q8);
  if (p.LPR == 64) {
    switch (p.NG) {
      case 1: return F<64, 1>::at(q8);
      case 2: return F<64, 2>::at(q8);
      case 4: return F<64, 4>::at(q8);
      default: return F<64, 8>::at(q8);
    }
  }
  switch (p.NG) {
    case 1: return F<256, 1>::at(q8);
    case 2: return F<256, 2>::at(q8);
    case 4: return F<256, 4>::at(q8);
    case 8: return F<256, 8>::at(q8);
    default: return F<256, 16>::at(q8);
  }
}

template <int LPR, int NG>
const void* of_types(bool res, bool q8) {
  if (res)
    return q8 ? (const void*)&m2rnn_add_norm8_kernel<LPR, NG, true, true> : (const void*)&m2rnn_add_norm8_kernel<LPR, NG, true, false>;
  return q8 ? (const void*)&m2rnn_add_norm8_kernel<LPR, NG, false, true> : (const void*)&m2rnn_add_norm8_kernel<LPR, NG, false, false>;
}
const void* pick8(const Plan& p, bool res, bool q8) {
  if (p.LPR == 16) return of_types<16, 1>(res, q8);
  if (p.LPR == 64) {
    switch (p.NG) {
      case 1: return of_types<64, 1>(res, q8);
      case 2: return of_types<64, 2>(res, q8);
      default: return of_types<64, 4>(res, q8);
    }
  }
  switch (p.NG) {
    case 1: return of_types<256, 1>(res, q8);
    case 2: return of_types<256, 2>(res, q8);
    case 4: return of_types<256, 4>(res, q8);
    default: return of_types<256, 8>(res, q8);
  }
}

template <typename Args>
int launch(const void* kern, long groups, Args& A, hipStream_t s) {
  void* args[] = {&A};
  return record_hip_status(hipLaunchKernel(kern, dim3((unsigned)groups), dim3(kBlkThreads), args, 0, s));
}

}  // namespace

extern "C" {

int m2rnn_add_norm_fwd(int64_t rows, int64_t D, int x_dtype, const void* x, int res_dtype, const void* res,
                       const float* gamma, float eps, void* h, int out_dtype, int64_t group, void* out, float* scale,
                       void* stream) {
  const int st = check_norm(rows, D, eps);
  if (st == M2RNN_EINVAL) return st;
  for (int t : {x_dtype, res_dtype})
    if (t != M2RNN_DTYPE_F32 && t != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  const bool q8 = out_dtype == M2RNN_DTYPE_E4M3;
  if (!q8 && out_dtype != M2RNN_DTYPE_F32 && out_dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  if (group < 0 || (!q8 && group != 0)) return M2RNN_EINVAL;
  if (st) return st;
  if (group == 0) group = D;
  if (group != D && (group != 128 || D % 128 != 0)) return M2RNN_EUNSUPPORTED;
  if (rows == 0) return M2RNN_OK;
  if (!x || !gamma || !out || (q8 && !scale) || (!res && h)) return M2RNN_EINVAL;
  for (const void* p : {x, res, (const void*)gamma, (const void*)h, (const void*)out})
    if (p && !al16(p)) return M2RNN_EINVAL;
  if ((uintptr_t)scale & 3u) return M2RNN_EINVAL;
  const long n = rows * D;
  const long nx = n * elem(x_dtype), nr = n * elem(res_dtype), no = n * elem(out_dtype), ng = 4 * D;
  const long ns = q8 ? 4 * rows * (D / group) : 0;
  // h may be res, or x of the same type; nothing else that is written may meet anything
  if (meet(h, nr, res, nr) && h != res) return M2RNN_EINVAL;
  if (meet(h, nr, x, nx) && !(h == x && x_dtype == res_dtype)) return M2RNN_EINVAL;
  if (meet(h, nr, gamma, ng) || meet(out, no, x, nx) || meet(out, no, res, nr) || meet(out, no, h, nr) ||
      meet(out, no, gamma, ng) || meet(scale, ns, x, nx) || meet(scale, ns, res, nr) || meet(scale, ns, h, nr) ||
      meet(scale, ns, out, no) || meet(scale, ns, gamma, ng))
    return M2RNN_EINVAL;
  const Plan p = plan_norm(rows, D, false, all_bf16(x_dtype, res, res_dtype), x_dtype == M2RNN_DTYPE_BF16 ? 1024 : 2048);
  NormArgs A{x, res, gamma, h, out, scale, rows, (int)D, (int)group, x_dtype == M2RNN_DTYPE_BF16,
             res_dtype == M2RNN_DTYPE_BF16, out_dtype == M2RNN_DTYPE_BF16, eps};
  const void* kern = p.VEC == 8 ? pick8(p, res != nullptr, q8) : pick<Fwd>(p, q8);
  return launch(kern, p.groups, A, (hipStream_t)stream);
}

int m2rnn_add_norm_bwd_workspace_size(int64_t rows, int64_t D, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_norm(rows, D, 0.0f);
  if (st) return st;
  *bytes = round_up256((size_t)plan_norm(rows, D, true, false, 2048).groups * D * sizeof(float));
  return M2RNN_OK;
}

int m2rnn_add_norm_bwd(int64_t rows, int64_t D, int h_dtype, const void* h, const float* gamma, float eps,
                       const float* dout, const float* dh, float* dx, float* dgamma, void* workspace,
                       size_t workspace_bytes, void* stream) {
  int st = check_norm(rows, D, eps);
  if (st == M2RNN_EINVAL || (h_dtype != M2RNN_DTYPE_F32 && h_dtype != M2RNN_DTYPE_BF16)) return M2RNN_EINVAL;
  if (st) return st;
  if (!gamma || !dgamma || (rows > 0 && (!h || !dout || !dx))) return M2RNN_EINVAL;
  for (const void* p : {h, (const void*)gamma, (const void*)dout, (const void*)dh, (const void*)dx, (const void*)dgamma})
    if (p && !al16(p)) return M2RNN_EINVAL;
  const long n4 = 4 * rows * D, nh = rows * D * elem(h_dtype), ng = 4 * D;
  if ((meet(dx, n4, dout, n4) && dx != dout) || (meet(dx, n4, dh, n4) && dx != dh) || meet(dx, n4, h, nh) ||
      meet(dx, n4, gamma, ng) || meet(dx, n4, dgamma, ng) || meet(dgamma, ng, gamma, ng) || meet(dgamma, ng, h, nh) ||
      meet(dgamma, ng, dout, n4) || meet(dgamma, ng, dh, n4))
    return M2RNN_EINVAL;
  size_t need = 0;
  st = m2rnn_add_norm_bwd_workspace_size(rows, D, &need);
  if (st) return st;
  if (need > 0 && (!workspace || workspace_bytes < need || !al16(workspace))) return M2RNN_EWORKSPACE;
  const Plan p = plan_norm(rows, D, true, false, 2048);
  hipStream_t s = (hipStream_t)stream;
  if (rows > 0) {
    NormBwdArgs A{h, gamma, dout, dh, dx, (float*)workspace, rows, (int)D, h_dtype == M2RNN_DTYPE_BF16, eps};
    st = launch(pick<Bwd>(p, false), p.groups, A, s);
    if (st) return st;
  }
  hipLaunchKernelGGL(m2rnn_norm_sums_kernel, dim3((unsigned)ceil_div(D, 16)), dim3(1024), 0, s, (const float*)workspace,
                     rows > 0 ? p.groups : 0, (int)D, dgamma);
  return record_hip_status(hipGetLastError());
}

}  // extern "C"
