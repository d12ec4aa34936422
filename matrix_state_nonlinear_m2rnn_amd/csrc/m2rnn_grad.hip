// C entry points of the gradient norm and clipping (include/m2rnn.h).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>
#include <vector>

#include "../../include/m2rnn.h"
#include "m2rnn_grad_kernels.h"

using namespace m2rnn;

namespace m2rnn {
int record_hip_status(hipError_t e);
}  // namespace m2rnn

namespace {

constexpr long kPieceMin = 4096, kPieceMax = 65536;  // elements per workgroup
constexpr long kPieces = 4096;                       // workgroups that the piece size aims for
static_assert(kPieceMin % (8 * kBlkThreads) == 0, "pieces keep a tensor's alignment");
static_assert(sizeof(GradArgs) <= 4096, "kernel arguments");

int elem(int64_t dtype) { return dtype == M2RNN_DTYPE_BF16 ? 2 : 4; }

int check_list(const m2rnn_tensor* g, int64_t count) {
  if (count < 0 || (count > 0 && !g)) return M2RNN_EINVAL;
  if (count > (1 << 24)) return M2RNN_EUNSUPPORTED;
  double total = 0.0;
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].dtype != M2RNN_DTYPE_F32 && g[i].dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
    if (g[i].numel < 0 || (g[i].numel > 0 && !g[i].data)) return M2RNN_EINVAL;
    if ((uintptr_t)g[i].data % elem(g[i].dtype)) return M2RNN_EINVAL;
    total += (double)g[i].numel;
  }
  // pieces are numbered with ints
  if (total / kPieceMax + (double)count > 2147483647.0) return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

// Elements per piece: enough pieces to fill the chip, each a power of two within its bounds.
long piece_size(const m2rnn_tensor* g, int64_t count) {
  double total = 0.0;
  for (int64_t i = 0; i < count; ++i) total += (double)g[i].numel;
  long piece = kPieceMin;
  while (piece < kPieceMax && total / (double)piece > (double)kPieces) piece *= 2;
  return piece;
}

long pieces(int64_t numel, long piece) { return (numel + piece - 1) / piece; }

// Calls f(args, workgroups, pieces before this launch) for each launch over the list, from its end if `backwards`.
template <typename F>
int over_launches(const m2rnn_tensor* g, int64_t count, void* const* out, long piece, bool backwards, F&& f) {
  GradArgs A{};
  A.piece = (int)piece;
  long before = 0, here = 0;
  auto flush = [&]() {
    const int st = A.tensors ? f(A, here, before) : M2RNN_OK;
    before += here;
    here = 0;
    A.tensors = 0;
    std::fill(std::begin(A.bf16), std::end(A.bf16), 0u);
    return st;
  };
  for (int64_t j = 0; j < count; ++j) {
    const int64_t i = backwards ? count - 1 - j : j;
    if (g[i].numel == 0) continue;
    const int t = A.tensors++;
    A.src[t] = g[i].data;
    A.dst[t] = out && out[i] ? out[i] : g[i].data;
    A.numel[t] = g[i].numel;
    A.first[t] = (int)here;
    if (g[i].dtype == M2RNN_DTYPE_BF16) A.bf16[t / 32] |= 1u << (t % 32);
    here += pieces(g[i].numel, piece);
    if (A.tensors == kGradMax) {
      const int st = flush();
      if (st) return st;
    }
  }
  return flush();
}

// Whether two outputs share memory, or an output shares memory with the norm, with another tensor's
// input, or only a part of it with its own.
bool overlaps(const m2rnn_tensor* g, int64_t count, void* const* out, const float* norm) {
  struct Span {
    uintptr_t at, end;
    bool written;
  };
  std::vector<Span> s;
  s.reserve(2 * (size_t)count + 1);
  s.push_back({(uintptr_t)norm, (uintptr_t)(norm + 1), false});
  for (int64_t i = 0; i < count; ++i) {
    if (g[i].numel == 0) continue;
    const uintptr_t bytes = (uintptr_t)g[i].numel * elem(g[i].dtype);
    const uintptr_t in = (uintptr_t)g[i].data, o = out && out[i] ? (uintptr_t)out[i] : in;
    s.push_back({o, o + bytes, true});
    if (o != in) s.push_back({in, in + bytes, false});
  }
  std::sort(s.begin(), s.end(), [](const Span& a, const Span& b) { return a.at < b.at; });
  uintptr_t end_any = 0, end_written = 0;
  for (const Span& x : s) {
    if (x.at < (x.written ? end_any : end_written)) return true;
    end_any = std::max(end_any, x.end);
    if (x.written) end_written = std::max(end_written, x.end);
  }
  return false;
}

}  // namespace

extern "C" {

int m2rnn_grad_norm_workspace_size(const m2rnn_tensor* grads, int64_t count, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_list(grads, count);
  if (st) return st;
  const long piece = piece_size(grads, count);
  size_t n = 0;
  for (int64_t i = 0; i < count; ++i) n += (size_t)pieces(grads[i].numel, piece);
  *bytes = n * sizeof(double);
  return M2RNN_OK;
}

int m2rnn_grad_norm(const m2rnn_tensor* grads, int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (!norm || ((uintptr_t)norm & 3u)) return M2RNN_EINVAL;
  size_t need = 0;
  int st = m2rnn_grad_norm_workspace_size(grads, count, &need);
  if (st) return st;
  if (need > 0 && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15u))) return M2RNN_EWORKSPACE;
  for (int64_t i = 0; i < count; ++i) {  // the norm would be written over a gradient
    const uintptr_t at = (uintptr_t)grads[i].data, end = at + (uintptr_t)grads[i].numel * elem(grads[i].dtype);
    if (at < end && (uintptr_t)norm < end && at < (uintptr_t)(norm + 1)) return M2RNN_EINVAL;
  }
  hipStream_t s = (hipStream_t)stream;
  double* part = (double*)workspace;
  st = over_launches(grads, count, nullptr, piece_size(grads, count), false, [&](GradArgs& A, long groups, long before) {
    A.part = part + before;
    hipLaunchKernelGGL(m2rnn_grad_norm_kernel, dim3((unsigned)groups), dim3(kBlkThreads), 0, s, A);
    return record_hip_status(hipGetLastError());
  });
  if (st) return st;
  hipLaunchKernelGGL(m2rnn_grad_total_kernel, dim3(1), dim3(1024), 0, s, (const double*)part,
                     (long)(need / sizeof(double)), norm);
  return record_hip_status(hipGetLastError());
}

int m2rnn_grad_clip(const m2rnn_tensor* grads, int64_t count, void* const* out, const float* norm, float max_norm,
                    void* stream) {
  if (!norm || ((uintptr_t)norm & 3u)) return M2RNN_EINVAL;
  if (!(max_norm >= 0.0f)) return M2RNN_EINVAL;
  const int st = check_list(grads, count);
  if (st) return st;
  bool in_place = true;
  for (int64_t i = 0; out && i < count; ++i) {
    if (!out[i] || grads[i].numel == 0) continue;
    if ((uintptr_t)out[i] % elem(grads[i].dtype)) return M2RNN_EINVAL;
    in_place = in_place && out[i] == grads[i].data;
  }
  try {
    if (overlaps(grads, count, out, norm)) return M2RNN_EINVAL;
  } catch (const std::bad_alloc&) {
    return M2RNN_EUNSUPPORTED;
  }
  hipStream_t s = (hipStream_t)stream;
  // the tensors that the norm read last are the likeliest in the memory-side cache: they come first (4.07 GB: 2.19 ms
  // with the norm, 2.21 in the norm's order)
  return over_launches(grads, count, out, piece_size(grads, count), true, [&](GradArgs& A, long groups, long) {
    A.norm = norm;
    A.max_norm = max_norm;
    A.in_place = in_place;
    hipLaunchKernelGGL(m2rnn_grad_clip_kernel, dim3((unsigned)groups), dim3(kBlkThreads), 0, s, A);
    return record_hip_status(hipGetLastError());
  });
}

}  // extern "C"
