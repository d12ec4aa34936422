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
constexpr long kOrthParts = 1024;  // partial sums of squares of a matrix at most
constexpr int kOrthPad = 128;     // what the refusals round sides up to
constexpr int kOrthSplits = 16;   // parts of a contraction at most

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t round_up256(size_t x) { return (x + 255) & ~(size_t)255; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }

int check_orth(int64_t batch, int64_t m, int64_t n, int dtype) {
  if (batch < 0 || m < 0 || n < 0) return M2RNN_EINVAL;
  if (dtype != M2RNN_DTYPE_F32 && dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  if (m > kOrthMaxSide || n > kOrthMaxSide || batch > 65535) return M2RNN_EUNSUPPORTED;
  // a launch holds fewer than 2^32 threads, one for every 16 padded elements
  if ((double)batch * (double)(ceil_div(m, kOrthPad) * kOrthPad) * (double)(ceil_div(n, kOrthPad) * kOrthPad) >= 68719476736.0)
    return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

// How a product is cut: tile side, workgroups that a CU holds, and a stage's time when it holds them (us).
struct Shape {
  int T, held;
  double stage;
};
constexpr Shape kShapes[] = {{256, 1, 1.6}, {128, 2, 0.9}, {64, 4, 0.8}};

struct Cut {
  int splits = 1, tiles = 1;
  double us = 0.0;
};
Cut cut_product(const Shape& h, long batch, long rows, long cols, long K, bool sym) {
  const long gi = rows / h.T, gj = cols / h.T, stages = K / kOrthK;
  Cut best;
  best.tiles = (int)(sym ? gi * (gi + 1) / 2 : gi * gj);
  for (int s = 1; s <= kOrthSplits && s <= stages; ++s) {
    const long groups = best.tiles * batch * s;
    if (s > 1 && groups > 2L * 256 * h.held) break;
    double us = (double)ceil_div(groups, 256L * h.held) * ((double)ceil_div(stages, s) * h.stage + 2.0) + 4.0;
    if (s > 1) us += 5.0 + (double)groups * h.T * h.T * 8.0 / 4e6;  // the parts written and read, one more launch
    if (s == 1 || us < best.us) {
      best.splits = s;
      best.us = us;
    }
  }
  return best;
}

// Sizes with m the shorter side, padded, and the workspace's parts.
struct Plan {
  long m, n, mp = 0, np = 0, parts, each;
  int shape = 0;
  Cut gram, poly, next;
  size_t part_bytes, x_bytes, a_bytes, split_bytes;  // partial sums of squares; one fp16 plane of X, of A; split products
  Plan(int64_t batch, int64_t rows, int64_t cols) {
    m = std::min(rows, cols);
    n = std::max(rows, cols);
    double best = 0.0;
    for (int i = 0; i < 3; ++i) {
      const Shape& h = kShapes[i];
      const long a = ceil_div(m, h.T) * h.T, b = ceil_div(n, h.T) * h.T;
      const Cut x = cut_product(h, batch, a, a, b, true), y = cut_product(h, batch, a, a, a, true),
                w = cut_product(h, batch, a, b, a, false);
      const double us = x.us + y.us + w.us;
      if (i == 0 || us < best) {
        best = us;
        shape = i;
        mp = a;
        np = b;
        gram = x;
        poly = y;
        next = w;
      }
    }
    each = std::max(ceil_div(ceil_div(m * n, kOrthParts), 1024), 4L) * 1024;
    parts = ceil_div(m * n, each);
    part_bytes = round_up256((size_t)batch * parts * sizeof(double));
    x_bytes = round_up256((size_t)batch * mp * np * 2);
    a_bytes = round_up256((size_t)batch * mp * mp * 2);
    split_bytes = 0;
    for (const Cut* c : {&gram, &poly, &next})
      if (c->splits > 1)
        split_bytes = std::max(split_bytes, (size_t)batch * c->splits * c->tiles * kShapes[shape].T * kShapes[shape].T * 4);
  }
  size_t bytes() const { return part_bytes + 8 * x_bytes + 4 * a_bytes + split_bytes; }
};

template <int T, int WR, int WC, int EPI>
int product_of(OrthArgs& A, long batch, hipStream_t s) {
  void* args[] = {&A};
  const dim3 grid((unsigned)A.tiles, (unsigned)A.splits, (unsigned)batch), block(64 * WR * WC);
  const void* one = (const void*)&m2rnn_orth_product_kernel<T, WR, WC, EPI, false>;
  if (A.splits == 1) return record_hip_status(hipLaunchKernel(one, grid, block, args, 0, s));
  const void* some = (const void*)&m2rnn_orth_product_kernel<T, WR, WC, EPI, true>;
  const int st = record_hip_status(hipLaunchKernel(some, grid, block, args, 0, s));
  if (st) return st;
  const long items = (long)A.tiles * (T / 16) * WC;
  return record_hip_status(hipLaunchKernel((const void*)&m2rnn_orth_join_kernel<T, WR, WC, EPI>,
                                           dim3((unsigned)ceil_div(items, 4), 1, (unsigned)batch), dim3(256), args, 0, s));
}

template <int EPI>
int product(int shape, const Cut& cut, OrthArgs& A, long batch, hipStream_t s) {
  A.splits = cut.splits;
  A.tiles = cut.tiles;
  switch (shape) {
    case 0: return product_of<256, 2, 4, EPI>(A, batch, s);
    case 1: return product_of<128, 2, 2, EPI>(A, batch, s);
    default: return product_of<64, 2, 2, EPI>(A, batch, s);
  }
}

// The kernel that takes a matrix of m x n (m <= n) through all steps in one workgroup; NULL: none does.
const void* small_kernel(long m, long n, unsigned& threads) {
  threads = 256;
  if (n <= 32) return (const void*)&m2rnn_orth_small_kernel<32, 32, 2, 2>;
  if (n <= 64) return (const void*)&m2rnn_orth_small_kernel<64, 64, 2, 2>;
  if (m <= 64 && n <= 128) return (const void*)&m2rnn_orth_small_kernel<64, 128, 2, 2>;
  threads = 512;
  if (n <= 128) return (const void*)&m2rnn_orth_small_kernel<128, 128, 2, 4>;
  if (m <= 64 && n <= 256) return (const void*)&m2rnn_orth_small_kernel<64, 256, 2, 4>;
  return nullptr;
}

}  // namespace

extern "C" {

int m2rnn_orthogonalize_workspace_size(int64_t batch, int64_t m, int64_t n, int dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_orth(batch, m, n, dtype);
  if (st) return st;
  unsigned threads;
  const bool small = small_kernel(std::min(m, n), std::max(m, n), threads) != nullptr;
  *bytes = batch > 0 && m > 0 && n > 0 && !small ? Plan(batch, m, n).bytes() : 0;
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
  unsigned threads;
  if (const void* small = small_kernel(std::min(m, n), std::max(m, n), threads)) {
    OrthCoefs c{};
    std::copy(coefs, coefs + 3 * steps, c.c);
    int lo = (int)std::min(m, n), hi = (int)std::max(m, n), turned = m > n, half = bf16, count = (int)steps;
    void* args[] = {&g, &out, &lo, &hi, &turned, &half, &count, &c, &eps};
    return record_hip_status(hipLaunchKernel(small, dim3((unsigned)batch), dim3(threads), args, 0, (hipStream_t)stream));
  }
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
  float* X32 = (float*)at;
  at += 2 * p.x_bytes;
  const Planes X = planes(p.x_bytes);
  Planes XT = planes(p.x_bytes), YT = planes(p.x_bytes);
  const Planes P = planes(p.a_bytes), Q = planes(p.a_bytes);
  const int tall = m > n;
  const dim3 parts((unsigned)p.parts, (unsigned)batch);
  const dim3 split((unsigned)(p.np / 64), (unsigned)(p.mp / 64), (unsigned)batch);
  if (bf16) {
    hipLaunchKernelGGL(m2rnn_orth_squares_kernel<true>, parts, dim3(256), 0, s, g, p.m * p.n, p.each, part);
    hipLaunchKernelGGL(m2rnn_orth_split_kernel<true>, split, dim3(256), 0, s, g, (int)p.m, (int)p.n, (int)p.mp, (int)p.np,
                       tall, (const double*)part, (int)p.parts, eps, X32, X, XT);
  } else {
    hipLaunchKernelGGL(m2rnn_orth_squares_kernel<false>, parts, dim3(256), 0, s, g, p.m * p.n, p.each, part);
    hipLaunchKernelGGL(m2rnn_orth_split_kernel<false>, split, dim3(256), 0, s, g, (int)p.m, (int)p.n, (int)p.mp, (int)p.np,
                       tall, (const double*)part, (int)p.parts, eps, X32, X, XT);
  }
  st = record_hip_status(hipGetLastError());
  for (int64_t i = 0; i < steps && !st; ++i) {
    const float* c = coefs + 3 * i;
    OrthArgs A{};
    A.part = (float*)at;
    A.M = A.N = X;
    A.O = A.OT = P;
    A.rows = A.cols = (int)p.mp;
    A.K = (int)p.np;
    st = product<ORTH_GRAM>(p.shape, p.gram, A, batch, s);
    if (st) break;
    A.M = A.N = A.E = P;
    A.O = A.OT = Q;
    A.K = (int)p.mp;
    A.cb = c[1];
    A.cc = c[2];
    st = product<ORTH_POLY>(p.shape, p.poly, A, batch, s);
    if (st) break;
    A.M = Q;
    A.N = XT;
    A.X32 = X32;
    A.O = X;
    A.OT = YT;
    A.cols = (int)p.np;
    A.ca = c[0];
    A.out = out;
    A.m = (int)p.m;
    A.n = (int)p.n;
    A.tall = tall;
    A.out_bf16 = bf16;
    st = i + 1 < steps ? product<ORTH_NEXT>(p.shape, p.next, A, batch, s) : product<ORTH_LAST>(p.shape, p.next, A, batch, s);
    std::swap(XT, YT);
  }
  return st;
}

}  // extern "C"
