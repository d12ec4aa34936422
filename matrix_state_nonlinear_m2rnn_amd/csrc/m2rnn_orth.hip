// C entry points of the orthogonalised update (include/m2rnn.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/m2rnn.h"
#include "m2rnn_orth_kernels.h"

using namespace m2rnn;

namespace m2rnn {
int record_hip_status(hipError_t e);
}  // namespace m2rnn

namespace {

constexpr long kOrthMaxSide = 65536;
constexpr long kOrthParts = 1024;  // partial sums of squares of a thin matrix at most
constexpr long kOrthNorms = 512;   // workgroups that a matrix's norms are dealt to, unless 64 rows each are fewer

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
size_t round_up256(size_t x) { return (x + 255) & ~(size_t)255; }

int check_orth(int64_t batch, int64_t m, int64_t n, int dtype) {
  if (batch < 0 || m < 0 || n < 0) return M2RNN_EINVAL;
  if (dtype != M2RNN_DTYPE_F32 && dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  if (m > kOrthMaxSide || n > kOrthMaxSide || batch > 65535) return M2RNN_EUNSUPPORTED;
  // a launch holds fewer than 2^32 threads, one for every 16 padded elements
  if ((double)batch * (double)(ceil_div(m, kOrthPad) * kOrthPad) * (double)(ceil_div(n, kOrthPad) * kOrthPad) >= 68719476736.0)
    return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

// The arrays' sides (what all products' tiles cover: what lies past the rounded sides is never part of a contraction) and the
// workspace's parts.
struct Plan : OrthCuts {
  long ma, na, gx, gy, each, sums;
  size_t part_bytes, row_bytes, col_bytes, scale_bytes;   // partial sums of squares and largest values, and the matrices' scales
  size_t d_bytes, e_bytes, square_bytes;                  // the rows' and columns' scales; their sums of squares in fp32
  size_t x_bytes, a_bytes, split_bytes;                   // one fp16 plane of X, of A; split products
  Plan(int64_t batch, int64_t rows, int64_t cols) : OrthCuts(batch, rows, cols) {
    ma = na = 0;
    for (const Cut* c : {&gram, &poly, &next}) ma = std::max(ma, (long)c->gi * kShapes[c->shape].TM);
    na = (long)next.gj * kShapes[next.shape].TN;
    gx = ceil_div(cols, 256);
    each = ceil_div(ceil_div(rows, 64), std::max(kOrthNorms / gx, 1L)) * 64;
    gy = ceil_div(rows, each);
    part_bytes = round_up256((size_t)batch * gx * gy * sizeof(double));
    row_bytes = round_up256((size_t)batch * gx * rows * sizeof(float));
    col_bytes = round_up256((size_t)batch * gy * cols * sizeof(float));
    scale_bytes = round_up256((size_t)batch * sizeof(double));
    sums = (long)next.gi * 2;  // (all shapes have two rows of waves)
    d_bytes = round_up256((size_t)batch * ma * sizeof(float));
    e_bytes = round_up256((size_t)batch * na * sizeof(float));
    square_bytes = round_up256((size_t)batch * sums * na * sizeof(float));
    x_bytes = round_up256((size_t)batch * ma * na * 2);
    a_bytes = round_up256((size_t)batch * ma * ma * 2);
    const OrthShape& h = kShapes[gram.shape];
    split_bytes = gram.splits > 1 ? (size_t)batch * gram.splits * gram.tiles * h.TM * h.TN * 4 : 0;
  }
  // X in fp32, R, two of C; the two scales of rows and columns, the diagonal
  size_t bytes() const {
    return part_bytes + row_bytes + col_bytes + scale_bytes + 3 * d_bytes + 2 * e_bytes + square_bytes + 8 * x_bytes + 4 * a_bytes +
           split_bytes;
  }
};

template <int TM, int TN, int WR, int WC, int BUFS, int EPI>
int product_of(OrthArgs& A, long batch, hipStream_t s) {
  void* args[] = {&A};
  static_assert(WR == 2, "Plan::sums");
  const unsigned more = EPI == ORTH_GRAM && A.en ? (unsigned)ceil_div(A.K, 64 * WR * WC) : 0;  // the next columns' scales
  const dim3 grid((unsigned)A.tiles + more, (unsigned)A.splits, (unsigned)batch), block(64 * WR * WC);
  const void* one = (const void*)&m2rnn_orth_product_kernel<TM, TN, WR, WC, BUFS, EPI, false>;
  if constexpr (EPI == ORTH_GRAM) {
    if (A.splits > 1) {
      const void* some = (const void*)&m2rnn_orth_product_kernel<TM, TN, WR, WC, BUFS, EPI, true>;
      const int st = record_hip_status(hipLaunchKernel(some, grid, block, args, 0, s));
      if (st) return st;
      const long items = (long)A.tiles * (TM / 16) * WC;
      return record_hip_status(hipLaunchKernel((const void*)&m2rnn_orth_join_kernel<TM, TN, WR, WC>,
                                               dim3((unsigned)ceil_div(items, 4), 1, (unsigned)batch), dim3(256), args, 0, s));
    }
  }
  return record_hip_status(hipLaunchKernel(one, grid, block, args, 0, s));
}

template <int EPI>
int product(const Cut& cut, OrthArgs& A, long batch, hipStream_t s) {
  A.splits = cut.splits;
  A.tiles = cut.tiles;
  A.gi = cut.gi;
  A.gj = cut.gj;
  switch (cut.shape) {
    case 0: return product_of<256, 256, 2, 4, 2, EPI>(A, batch, s);
    case 1: return product_of<192, 192, 2, 4, 2, EPI>(A, batch, s);
    case 2: return product_of<128, 128, 2, 2, 2, EPI>(A, batch, s);
    case 3: return product_of<128, 64, 2, 2, 2, EPI>(A, batch, s);
    case 4: return product_of<96, 96, 2, 2, 2, EPI>(A, batch, s);
    case 5: return product_of<64, 64, 2, 2, 2, EPI>(A, batch, s);
    default: return product_of<64, 64, 2, 2, 5, EPI>(A, batch, s);
  }
}

// What D^-1 B is kept times: 2^7 leaves |b s + c s^3| up to 500, less for steps whose factors are so large that it could pass that where
// |b s^2 + c s^4| is below 24: with either term below 48, b s is at most sqrt(48 |b|) and c s^3 at most (48^3 |c|)^(1/4).
float orth_unit(float b, float c) {
  const float most = std::sqrt(48.0f * std::fabs(b)) + 18.24f * std::sqrt(std::sqrt(std::fabs(c)));
  float u = 128.0f;
  while (!(most * u < 65000.0f) && u > 0x1p-40f) u *= 0.5f;
  return u;
}
// No row or column of X grows by more than 2^this in a step: they are multiplied by matrices whose singular values are
// |a + b s^2 + c s^4|.
int orth_grow(float a) {
  int k = 5;
  while (std::ldexp(1.0f, k) < std::fabs(a) + 24.0f && k < 40) ++k;
  return k;
}

// The kernel that takes a matrix of m x n (m <= n) through all steps in one workgroup; NULL: none does.
const void* small_kernel(long m, long n, unsigned& threads) {
  threads = 256;
  if (n <= 64) return (const void*)&m2rnn_orth_small_kernel<64, 64, 2, 2>;
  if (m <= 64 && n <= 128) return (const void*)&m2rnn_orth_small_kernel<64, 128, 2, 2>;
  threads = 512;
  if (n <= 128) return (const void*)&m2rnn_orth_small_kernel<128, 128, 2, 4>;
  if (m <= 64 && n <= 256) return (const void*)&m2rnn_orth_small_kernel<64, 256, 2, 4>;
  return nullptr;
}

// Thin matrices: one wave up to 64 columns, one workgroup of 8 up to 512, else tiles of 512 over up to kThinGroups of them.
constexpr long kThinRows = 32, kThinTile = 512, kThinGroups = 64;
struct ThinPlan {
  long tiles, groups, parts, each;
  size_t square_bytes, x_bytes, sum_bytes;
  ThinPlan(int64_t batch, long m, long n) {
    tiles = ceil_div(n, kThinTile);
    groups = std::min(tiles, kThinGroups);
    each = std::max(ceil_div(ceil_div(m * n, kOrthParts), 1024), 4L) * 1024;
    parts = ceil_div(m * n, each);
    const bool one = tiles == 1;
    square_bytes = one ? 0 : round_up256((size_t)batch * parts * sizeof(double));
    x_bytes = one ? 0 : (size_t)batch * tiles * kThinTile * kThinRows * 4;
    sum_bytes = one ? 0 : (size_t)2 * batch * groups * kThinRows * kThinRows * 4;
  }
  size_t bytes() const { return square_bytes + x_bytes + sum_bytes; }
};

template <int M>
int thin_all(ThinArgs& A, OrthCoefs& c, int64_t batch, hipStream_t s) {
  void* args[] = {&A, &c};
  const void* kern = A.n <= 64 ? (const void*)&m2rnn_orth_thin_kernel<M, 1, THIN_ALL> : (const void*)&m2rnn_orth_thin_kernel<M, 8, THIN_ALL>;
  return record_hip_status(hipLaunchKernel(kern, dim3(1, (unsigned)batch), dim3(A.n <= 64 ? 64 : 512), args, 0, s));
}

template <int M>
int thin_steps(ThinArgs& A, OrthCoefs& c, const ThinPlan& p, int64_t batch, hipStream_t s) {
  void* args[] = {&A, &c};
  const dim3 grid((unsigned)p.groups, (unsigned)batch);
  int st = record_hip_status(hipLaunchKernel((const void*)&m2rnn_orth_thin_kernel<M, 8, THIN_FIRST>, grid, dim3(512), args, 0, s));
  for (int i = 0; i < A.steps && !st; ++i) {
    A.turn ^= 1;
    A.ca = c.c[3 * i];
    A.cb = c.c[3 * i + 1];
    A.cc = c.c[3 * i + 2];
    const void* kern = i + 1 < A.steps ? (const void*)&m2rnn_orth_thin_kernel<M, 8, THIN_MIDDLE>
                                       : (const void*)&m2rnn_orth_thin_kernel<M, 8, THIN_LAST>;
    st = record_hip_status(hipLaunchKernel(kern, grid, dim3(512), args, 0, s));
  }
  return st;
}

template <bool BF16>
int squares(const void* g, long mn, long each, long parts, int64_t batch, double* part, hipStream_t s) {
  hipLaunchKernelGGL(m2rnn_orth_squares_kernel<BF16>, dim3((unsigned)parts, (unsigned)batch), dim3(256), 0, s, g, mn, each, part);
  return record_hip_status(hipGetLastError());
}

}  // namespace

extern "C" {

int m2rnn_orthogonalize_workspace_size(int64_t batch, int64_t m, int64_t n, int dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_orth(batch, m, n, dtype);
  if (st) return st;
  *bytes = 0;
  if (batch == 0 || m == 0 || n == 0) return M2RNN_OK;
  const long lo = std::min(m, n), hi = std::max(m, n);
  unsigned threads;
  if (lo <= kThinRows)
    *bytes = ThinPlan(batch, lo, hi).bytes();
  else if (!small_kernel(lo, hi, threads))
    *bytes = Plan(batch, m, n).bytes();
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
  OrthCoefs c{};
  std::copy(coefs, coefs + 3 * steps, c.c);
  for (int64_t i = 0; i < steps; ++i) c.unit[i] = orth_unit(coefs[3 * i + 1], coefs[3 * i + 2]);
  int lo = (int)std::min(m, n), hi = (int)std::max(m, n), turned = m > n, half = bf16, count = (int)steps;
  if (lo <= kThinRows) {
    const ThinPlan p(batch, lo, hi);
    if (p.bytes() > 0 && (!workspace || workspace_bytes < p.bytes() || !al16(workspace))) return M2RNN_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    char* at = (char*)workspace;
    ThinArgs A{};
    A.g = g;
    A.out = out;
    A.squares = (const double*)at;
    A.X = (float*)(at + p.square_bytes);
    A.part = (float*)(at + p.square_bytes + p.x_bytes);
    A.m = lo;
    A.n = hi;
    A.tall = turned;
    A.bf16 = half;
    A.tiles = (int)p.tiles;
    A.parts = (int)p.parts;
    A.steps = count;
    A.eps = eps;
    if (p.tiles == 1) return lo <= 16 ? thin_all<16>(A, c, batch, s) : thin_all<32>(A, c, batch, s);
    st = bf16 ? squares<true>(g, (long)m * n, p.each, p.parts, batch, (double*)at, s)
              : squares<false>(g, (long)m * n, p.each, p.parts, batch, (double*)at, s);
    if (st) return st;
    return lo <= 16 ? thin_steps<16>(A, c, p, batch, s) : thin_steps<32>(A, c, p, batch, s);
  }
  unsigned threads;
  if (const void* small = small_kernel(lo, hi, threads)) {
    void* args[] = {&g, &out, &lo, &hi, &turned, &half, &count, &c, &eps};
    return record_hip_status(hipLaunchKernel(small, dim3((unsigned)batch), dim3(threads), args, 0, (hipStream_t)stream));
  }
  const Plan p(batch, m, n);
  if (!workspace || workspace_bytes < p.bytes() || !al16(workspace)) return M2RNN_EWORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  char* at = (char*)workspace;
  auto take = [&](size_t bytes) {
    char* q = at;
    at += bytes;
    return q;
  };
  auto planes = [&](size_t bytes) { return Planes{(uint16_t*)take(bytes), (uint16_t*)take(bytes)}; };
  const OrthNorms N{(double*)take(p.part_bytes), (float*)take(p.row_bytes), (float*)take(p.col_bytes)};
  double* scale = (double*)take(p.scale_bytes);
  float *d = (float*)take(p.d_bytes), *dn = (float*)take(p.d_bytes), *diag = (float*)take(p.d_bytes);
  float *e = (float*)take(p.e_bytes), *en = (float*)take(p.e_bytes);
  float* sums = (float*)take(p.square_bytes);
  float* X = (float*)take(2 * p.x_bytes);
  const Planes R = planes(p.x_bytes);
  Planes C = planes(p.x_bytes), Cn = planes(p.x_bytes);
  const Planes P = planes(p.a_bytes), Q = planes(p.a_bytes);
  const int tall = m > n;
  const dim3 of_norms((unsigned)p.gx, (unsigned)p.gy, (unsigned)batch);
  const dim3 of_split((unsigned)(p.np / 64), (unsigned)(p.mp / 64), (unsigned)batch);
  const auto norms = n % 4 == 0 ? (bf16 ? &m2rnn_orth_norms_kernel<true, true> : &m2rnn_orth_norms_kernel<false, true>)
                                : (bf16 ? &m2rnn_orth_norms_kernel<true, false> : &m2rnn_orth_norms_kernel<false, false>);
  hipLaunchKernelGGL(norms, of_norms, dim3(256), 0, s, g, (int)m, (int)n, (int)p.each, N);
  st = record_hip_status(hipGetLastError());
  if (st) return st;
  hipLaunchKernelGGL(m2rnn_orth_scales_kernel, dim3((unsigned)ceil_div(p.mp + p.np, 256), (unsigned)batch), dim3(256), 0, s, N, (int)p.gx,
                     (int)p.gy, (int)p.m, (int)p.n, (int)p.mp, (int)p.np, (int)p.ma, (int)p.na, tall, eps, scale, d, e);
  st = record_hip_status(hipGetLastError());
  if (st) return st;
  if (bf16)
    hipLaunchKernelGGL(m2rnn_orth_split_kernel<true>, of_split, dim3(256), 0, s, g, (int)p.m, (int)p.n, (int)p.ma, (int)p.na, tall, scale,
                       d, e, X, R, C);
  else
    hipLaunchKernelGGL(m2rnn_orth_split_kernel<false>, of_split, dim3(256), 0, s, g, (int)p.m, (int)p.n, (int)p.ma, (int)p.na, tall, scale,
                       d, e, X, R, C);
  st = record_hip_status(hipGetLastError());
  for (int64_t i = 0; i < steps && !st; ++i) {
    const float *f = c.c + 3 * i, unit = c.unit[i];
    const bool cubic = f[2] == 0.0f, last = i + 1 == steps;  // cubic: B = b A
    OrthArgs A{};
    A.part = (float*)at;
    A.d = d;
    A.e = e;
    A.en = last ? nullptr : en;
    A.diag = diag;
    A.squares = sums;
    A.sums = i == 0 ? 0 : (int)p.sums;
    A.mp = (int)p.mp;
    A.grow = orth_grow(f[0]);
    A.M = A.N = R;
    A.O = cubic ? Q : P;
    A.rows = A.cols = (int)p.ma;
    A.ld = (int)p.na;
    A.K = (int)p.np;
    A.cb = cubic ? f[1] * unit : kOrthA;
    st = product<ORTH_GRAM>(p.gram, A, batch, s);
    if (!st && !cubic) {
      A.M = A.N = A.E = P;
      A.O = Q;
      A.ld = (int)p.ma;
      A.K = (int)p.mp;
      A.cb = f[1] * (unit / kOrthA);
      A.cc = f[2] * (unit / (kOrthA * kOrthA));
      st = product<ORTH_POLY>(p.poly, A, batch, s);
    }
    if (st) break;
    A.M = Q;
    A.ld = (int)p.ma;
    A.K = (int)p.mp;
    A.N = C;
    A.O = R;
    A.C = Cn;
    A.X = X;
    A.dn = dn;
    A.sums = (int)p.sums;
    A.cols = (int)p.na;
    A.ca = f[0];
    A.unit = 1.0f / (unit * kOrthX);
    A.out = out;
    A.m = (int)p.m;
    A.n = (int)p.n;
    A.tall = tall;
    A.out_bf16 = bf16;
    st = last ? product<ORTH_LAST>(p.next, A, batch, s) : product<ORTH_NEXT>(p.next, A, batch, s);
    std::swap(C, Cn);
    std::swap(d, dn);
    std::swap(e, en);
  }
  return st;
}

}  // extern "C"
