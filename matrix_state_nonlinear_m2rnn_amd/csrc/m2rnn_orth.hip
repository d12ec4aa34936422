// C entry points of the orthogonalised update (include/m2rnn.h).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/m2rnn.h"
#include "m2rnn_orth_kernels.h"

using namespace m2rnn;

namespace m2rnn {
int record_hip_status(hipError_t e);
}  // namespace m2rnn

namespace {

constexpr long kOrthMaxSide = 65536;
constexpr long kOrthMaxSteps = 64;
constexpr long kOrthParts = 256;  // partial sums of squares of a matrix at most

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t round_up256(size_t x) { return (x + 255) & ~(size_t)255; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }

int check_orth(int64_t batch, int64_t m, int64_t n, int dtype) {
  if (batch < 0 || m < 0 || n < 0) return M2RNN_EINVAL;
  if (dtype != M2RNN_DTYPE_F32 && dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  if (m > kOrthMaxSide || n > kOrthMaxSide || batch > 65535) return M2RNN_EUNSUPPORTED;
  // a launch holds fewer than 2^32 threads, one for every 16 padded elements
  if ((double)batch * (double)(ceil_div(m, kOrthTile) * kOrthTile) * (double)(ceil_div(n, kOrthTile) * kOrthTile) >= 68719476736.0)
    return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

// Sizes with m the shorter side, padded, and the workspace's parts.
struct Plan {
  long m, n, mp, np, parts, each;
  size_t part_bytes, x_bytes, a_bytes;  // partial sums; one plane of X; one plane of A
  Plan(int64_t batch, int64_t rows, int64_t cols) {
    m = std::min(rows, cols);
    n = std::max(rows, cols);
    mp = ceil_div(m, kOrthTile) * kOrthTile;
    np = ceil_div(n, kOrthTile) * kOrthTile;
    each = std::max(ceil_div(ceil_div(m * n, kOrthParts), 256), 16L) * 256;
    parts = ceil_div(m * n, each);
    part_bytes = round_up256((size_t)batch * parts * sizeof(double));
    x_bytes = round_up256((size_t)batch * mp * np * 2);
    a_bytes = round_up256((size_t)batch * mp * mp * 2);
  }
  size_t bytes() const { return part_bytes + 8 * x_bytes + 4 * a_bytes; }
};

template <int EPI>
int product(const OrthArgs& A, long batch, hipStream_t s) {
  const unsigned gi = (unsigned)(A.rows / kOrthTile), gj = (unsigned)(A.cols / kOrthTile);
  const dim3 grid = EPI == ORTH_GRAM || EPI == ORTH_POLY ? dim3(gi * (gi + 1) / 2, 1, (unsigned)batch)
                                                         : dim3(gj, gi, (unsigned)batch);
  hipLaunchKernelGGL(m2rnn_orth_product_kernel<EPI>, grid, dim3(kOrthThreads), 0, s, A);
  return record_hip_status(hipGetLastError());
}

}  // namespace

extern "C" {

int m2rnn_orthogonalize_workspace_size(int64_t batch, int64_t m, int64_t n, int dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_orth(batch, m, n, dtype);
  if (st) return st;
  *bytes = batch > 0 && m > 0 && n > 0 ? Plan(batch, m, n).bytes() : 0;
  return M2RNN_OK;
}

int m2rnn_orthogonalize(int64_t batch, int64_t m, int64_t n, int dtype, const void* g, int64_t steps, const float* coefs,
                        float eps, void* out, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_orth(batch, m, n, dtype);
  if (st == M2RNN_EINVAL || steps < 1 || !coefs || !(eps >= 0.0f) || eps > 1e30f) return M2RNN_EINVAL;
  if (st || steps > kOrthMaxSteps) return M2RNN_EUNSUPPORTED;
  if (batch == 0 || m == 0 || n == 0) return M2RNN_OK;
  if (!g || !out || !al16(g) || !al16(out)) return M2RNN_EINVAL;
  const bool bf16 = dtype == M2RNN_DTYPE_BF16;
  const uintptr_t size = (uintptr_t)(batch * m * n * (bf16 ? 2 : 4)), x = (uintptr_t)g, y = (uintptr_t)out;
  if (x != y && x < y + size && y < x + size) return M2RNN_EINVAL;
  const Plan p(batch, m, n);
  if (!workspace || workspace_bytes < p.bytes() || !al16(workspace)) return M2RNN_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  char* at = (char*)workspace;
  double* part = (double*)at;
  at += p.part_bytes;
  auto planes = [&](size_t bytes) {
    Planes q{(uint16_t*)at, (uint16_t*)(at + bytes)};
    at += 2 * bytes;
    return q;
  };
  Planes X = planes(p.x_bytes), XT = planes(p.x_bytes), Y = planes(p.x_bytes), YT = planes(p.x_bytes);
  const Planes P = planes(p.a_bytes), Q = planes(p.a_bytes);
  const int tall = m > n;
  const dim3 parts((unsigned)p.parts, (unsigned)batch);
  const dim3 split((unsigned)(p.np / 64), (unsigned)(p.mp / 64), (unsigned)batch);
  if (bf16) {
    hipLaunchKernelGGL(m2rnn_orth_squares_kernel<true>, parts, dim3(256), 0, s, g, p.m * p.n, p.each, part);
    hipLaunchKernelGGL(m2rnn_orth_split_kernel<true>, split, dim3(256), 0, s, g, (int)p.m, (int)p.n, (int)p.mp, (int)p.np,
                       tall, (const double*)part, (int)p.parts, eps, X, XT);
  } else {
    hipLaunchKernelGGL(m2rnn_orth_squares_kernel<false>, parts, dim3(256), 0, s, g, p.m * p.n, p.each, part);
    hipLaunchKernelGGL(m2rnn_orth_split_kernel<false>, split, dim3(256), 0, s, g, (int)p.m, (int)p.n, (int)p.mp, (int)p.np,
                       tall, (const double*)part, (int)p.parts, eps, X, XT);
  }
  st = record_hip_status(hipGetLastError());
  for (int64_t i = 0; i < steps && !st; ++i) {
    const float *c = coefs + 3 * i;
    OrthArgs A{};
    A.M = A.N = X;
    A.O = A.OT = P;
    A.rows = A.cols = (int)p.mp;
    A.K = (int)p.np;
    st = product<ORTH_GRAM>(A, batch, s);
    if (st) break;
    A.M = A.N = A.E = P;
    A.O = A.OT = Q;
    A.K = (int)p.mp;
    A.cb = c[1];
    A.cc = c[2];
    st = product<ORTH_POLY>(A, batch, s);
    if (st) break;
    A.M = Q;
    A.N = XT;
    A.E = X;
    A.O = Y;
    A.OT = YT;
    A.cols = (int)p.np;
    A.ca = c[0];
    A.out = out;
    A.m = (int)p.m;
    A.n = (int)p.n;
    A.tall = tall;
    A.out_bf16 = bf16;
    st = i + 1 < steps ? product<ORTH_NEXT>(A, batch, s) : product<ORTH_LAST>(A, batch, s);
    std::swap(X, Y);
    std::swap(XT, YT);
  }
  return st;
}

}  // extern "C"
