// C entry points of the selective state space scan (include/m2rnn.h): argument checks, the plan
// (time segments, heads per workgroup) and the launches.
#include <hip/hip_runtime.h>

#include "../../include/m2rnn.h"
#include "m2rnn_ssm_select.h"

using namespace m2rnn;

namespace m2rnn {
// Status of a HIP call, recording a failure for m2rnn_last_hip_error() (defined with it).
int record_hip_status(hipError_t e);

// Rows of partial sums that one workgroup adds (a wave 1/16 of them after each other); more go through a second launch.
constexpr long kSsmSlice = 2048;

// The backward's partial sums over `parts` rows: gate [parts][2N] to dbeta, dalpha and wr [parts][N V] to dw_r (W: the type of
// its rows).  A workgroup takes 64 columns (of both arrays, one after the other) of a slice of rows, its 16 waves every
// sixteenth row each; the waves' sums are added in order.  Everything is added in fp64: over a long sequence the terms of
// these sums cancel, and fp32 rows and sums left five times the error of dbeta and dw_r.  With more than one
// slice the slices' sums go to gate_out and wr_out, rows of another call.
template <typename W>
__global__ void __launch_bounds__(1024) m2rnn_ssm_sums_kernel(const double* __restrict__ gate, const W* __restrict__ wr,
                                                              long parts, int N, long NV, double* __restrict__ gate_out,
                                                              double* __restrict__ wr_out, float* __restrict__ dbeta,
                                                              float* __restrict__ dalpha, float* __restrict__ dw_r) {
  __shared__ double red[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const long gate_groups = (2L * N + 63) / 64;
  const bool g = blockIdx.x < gate_groups;
  const long M = g ? 2L * N : NV, j = ((long)blockIdx.x - (g ? 0 : gate_groups)) * 64 + lane;
  const long p0 = (long)blockIdx.y * kSsmSlice, p1 = p0 + kSsmSlice < parts ? p0 + kSsmSlice : parts;
  double acc = 0.0;
  if (j < M && g) {
#pragma unroll 8
    for (long p = p0 + w; p < p1; p += 16) acc += gate[p * M + j];
  } else if (j < M) {
#pragma unroll 8
    for (long p = p0 + w; p < p1; p += 16) acc += (double)wr[p * M + j];
  }
  red[w][lane] = acc;
  __syncthreads();
  if (w == 0 && j < M) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][lane];
    if (gridDim.y > 1)
      (g ? gate_out : wr_out)[(long)blockIdx.y * M + j] = s;
    else if (!g)
      dw_r[j] = (float)s;
    else if (j < N)
      dbeta[j] = (float)s;
    else
      dalpha[j - N] = (float)s;
  }
}

// out = the sum of `planes` planes of `count` floats (count a multiple of 4), for dq and dk of heads that
// share a query/key and were split over workgroups.
__global__ void __launch_bounds__(256) m2rnn_ssm_planes_kernel(const float* __restrict__ dq_part,
                                                               const float* __restrict__ dk_part, int planes,
                                                               long count, float* __restrict__ dq,
                                                               float* __restrict__ dk) {
  const float* src = blockIdx.y ? dk_part : dq_part;
  float* dst = blockIdx.y ? dk : dq;
  for (long i = ((long)blockIdx.x * 256 + threadIdx.x) * 4; i < count; i += (long)gridDim.x * 1024) {
    f32x4 s = *(const f32x4*)(src + i);
    for (int p = 1; p < planes; ++p) s += *(const f32x4*)(src + p * count + i);
    *(f32x4*)(dst + i) = s;
  }
}

}  // namespace m2rnn

namespace {

int status(hipError_t e) { return record_hip_status(e); }

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
size_t round_up256(size_t x) { return (x + 255) & ~(size_t)255; }
long ceil_div(long a, long b) { return (a + b - 1) / b; }

constexpr long kMaxGrid = 2147483647L;
constexpr double kMaxThreads = 4294967295.0;  // of one launch
constexpr int kMaxK = 128;

// Waves that the forward and state launches aim for: three for each of the 1024 SIMDs, which is what registers and LDS
// let a CU hold of the kernels at V = 64 and of the shared V = 16 with K <= 64 (B2 N32 T16384 K=V=64: 226 us; 358 with
// one, 240 with two, 258 with four.  B4 N128 T4096 K=64 V=16 shared: 114; 193, 128, 120).  The kernels at K > 64 hold
// one or two, those at V = 32 two, which the target does not look at: B4 N16 T4096 K=V=128 takes 187 us (366 in fp32), with
// two 165 (318); N64 K=128 V=16 shared 117, with two 94; K=64 V=32 64 us with either (94 in fp32, with two 104).
constexpr long kSsmWaves = 3L * 1024;
// A segment is at least this many chunks: with single ones a prompt of 509 tokens (16 heads, K = V = 128, fp32) takes the
// same time (32 us for its three kernels), with twice the segments' states to write and combine.
constexpr int kSsmMinChunks = 2;
// Workgroups that the backward's launch aims for where a group's heads can be split: two for each CU, which the kernels at
// K <= 64 hold (B4 N128 T4096 K=64 V=16, one query/key: 410 us for the call, 589 with 256, 413 with 1024).  Those at K > 64
// hold one and take about the same (N64 K=128 V=64, one query/key: 1228 us, 1212 with 256, 1242 with 1024).
constexpr long kSsmBwdGroups = 512;

int check_ssm(const m2rnn_dims* d, int dtype) {
  if (!d) return M2RNN_EINVAL;
  if (d->B < 0 || d->T < 0 || d->N < 0 || d->K < 0 || d->V < 0 || d->Nqk < 0) return M2RNN_EINVAL;
  if (dtype != M2RNN_DTYPE_F32 && dtype != M2RNN_DTYPE_BF16) return M2RNN_EINVAL;
  if (d->Nqk != 0 && (d->Nqk > d->N || d->N % d->Nqk != 0)) return M2RNN_EINVAL;
  if (d->V != 16 && d->V != 32 && d->V != 64 && d->V != 128) return M2RNN_EUNSUPPORTED;
  if (d->K <= 0 || d->K % 16 != 0 || d->K > kMaxK) return M2RNN_EUNSUPPORTED;
  // the kernels number steps, heads and workgroups with ints
  if (d->T > kMaxGrid - 128 || d->N > (1 << 20) || d->B > kMaxGrid) return M2RNN_EUNSUPPORTED;
  if ((double)d->B * d->N * (ceil_div(d->T, 32) + 64) * 8 > (double)kMaxGrid) return M2RNN_EUNSUPPORTED;
  return M2RNN_OK;
}

// The backward's further limits: its partial sums are rows per (b, chunk), which two launches of slices add up, and
// it has one workgroup for each (b, query/key, chunk) (and split of its heads, which only small
// launches have).
int check_ssm_bwd(const m2rnn_dims* d, int dtype) {
  const int st = check_ssm(d, dtype);
  if (st) return st;
  const double chunks =
      (double)d->B * ceil_div(d->T, dtype == M2RNN_DTYPE_BF16 ? ssm_chunk<true>() : ssm_chunk<false>());
  if (chunks > 65535.0 * 64.0) return M2RNN_EUNSUPPORTED;
  return chunks * (d->Nqk ? d->Nqk : d->N) * 64 * kSsmBwdWaves > kMaxThreads ? M2RNN_EUNSUPPORTED : M2RNN_OK;
}

struct Plan {
  SsmArgs A{};
  bool bf16 = false;
  int KP = 0, VB = 0, HPW = 0, L = 0;
  long units = 0;     // workgroups that share nothing, per segment
  bool rev = false;
  size_t seg = 0, segdec = 0, rloc = 0, cdec = 0, gate = 0, wr = 0, scratch = 0, planes = 0, total = 0;  // bytes
};

// The launch plan and the workspace's parts.  bwd: the reverse scan's state pass and the backward.
Plan make_plan(const m2rnn_dims* d, int dtype, bool bwd) {
  Plan p;
  SsmArgs& A = p.A;
  A.B = (int)d->B;
  A.T = (int)d->T;
  A.N = (int)d->N;
  A.K = (int)d->K;
  A.V = (int)d->V;
  A.G = d->Nqk ? (int)d->Nqk : A.N;
  p.bf16 = dtype == M2RNN_DTYPE_BF16;
  p.rev = bwd;
  p.L = p.bf16 ? ssm_chunk<true>() : ssm_chunk<false>();
  p.KP = A.K <= 32 ? 32 : (A.K <= 64 ? 64 : 128);
  p.VB = A.V > 64 ? 64 : A.V;
  const int hpg = A.G > 0 ? A.N / A.G : 1;
  p.HPW = (A.V == 16 && hpg > 1) ? 4 : 1;
  A.HB = (int)ceil_div(hpg, p.HPW);
  A.CB = A.V / p.VB;
  A.nch = (int)ceil_div(A.T, p.L);
  p.units = (long)A.B * A.G * A.HB * A.CB;
  const long waves = p.units * (p.HPW * p.VB / 16);
  long S = waves > 0 ? ceil_div(kSsmWaves, waves) : 1;
  const long most = A.nch / kSsmMinChunks;
  S = S > most ? most : S;
  S = S < 1 ? 1 : S;
  A.cps = (int)ceil_div(A.nch > 0 ? A.nch : 1, S);
  A.S = (int)ceil_div(A.nch > 0 ? A.nch : 1, A.cps);
  A.HS = 1;
  const size_t pairs = (size_t)A.B * A.N, KV = (size_t)A.K * A.V, f = sizeof(float);
  if (bwd || A.S > 1) {
    p.seg = round_up256(pairs * A.S * KV * f);
    p.segdec = round_up256(pairs * A.S * f);
  }
  if (bwd) {
    const long groups = (long)A.B * A.G * A.nch;
    if (groups > 0 && groups < kSsmBwdGroups && hpg > 1) {
      const long want = ceil_div(kSsmBwdGroups, groups);
      A.HS = (int)ceil_div(hpg, ceil_div(hpg, want < hpg ? want : hpg));
    }
    const long parts = (long)A.B * A.nch;
    p.rloc = round_up256(pairs * A.nch * KV * f);
    p.cdec = round_up256(pairs * A.nch * f);
    p.gate = round_up256((size_t)parts * 2 * A.N * sizeof(double));
    p.wr = round_up256((size_t)parts * A.N * A.V * f);
    if (parts > kSsmSlice) p.scratch = round_up256((size_t)ceil_div(parts, kSsmSlice) * A.N * (2 + A.V) * sizeof(double));
    if (A.HS > 1) p.planes = round_up256((size_t)2 * A.HS * A.B * A.T * A.G * A.K * f);
  }
  p.total = p.seg + p.segdec + p.rloc + p.cdec + p.gate + p.wr + p.scratch + p.planes;
  return p;
}

const void* pick(const Plan& p, int which) {
  return p.bf16 ? ssm_kernel_bf16(p.KP, p.VB, p.HPW, which) : ssm_kernel_f32(p.KP, p.VB, p.HPW, which);
}

hipError_t launch(const void* kern, long grid, int block, SsmArgs A, hipStream_t s) {
  void* args[] = {&A};
  return hipLaunchKernel(kern, dim3((unsigned)grid), dim3((unsigned)block), args, 0, s);
}

hipError_t launch_combine(const SsmArgs& A, bool rev, hipStream_t s) {
  const long blocks = (long)A.B * A.N * ceil_div((long)A.K * A.V, 256);
  const long grid = blocks < (1L << 22) ? blocks : 1L << 22;  // (a launch holds fewer than 2^32 threads)
  return launch(rev ? (const void*)&m2rnn_ssm_combine_kernel<true> : (const void*)&m2rnn_ssm_combine_kernel<false>,
                grid, 256, A, s);
}

int run_fwd(const m2rnn_dims* d, int dtype, const void* q, const void* k, const void* v, const float* a,
            const float* alpha, const float* beta, const float* w_r, const int32_t* lens, const float* H0, float* y,
            float* H_T, float* ckpt, bool want_ckpt, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_ssm(d, dtype);
  if (st) return st;
  if (d->B == 0 || d->N == 0) return M2RNN_OK;
  if (!alpha || !beta || !w_r) return M2RNN_EINVAL;
  if (d->T > 0 && (!q || !k || !v || !a || !y || (want_ckpt && !ckpt))) return M2RNN_EINVAL;
  const void* p16[] = {q, k, v, w_r, H0, y, H_T, ckpt};
  for (const void* p : p16)
    if (p && !al16(p)) return M2RNN_EINVAL;
  const void* p4[] = {a, alpha, beta, lens};
  for (const void* p : p4)
    if (p && !al4(p)) return M2RNN_EINVAL;
  Plan p = make_plan(d, dtype, false);
  if (p.total > 0 && (!workspace || workspace_bytes < p.total || !al16(workspace))) return M2RNN_EWORKSPACE;
  SsmArgs& A = p.A;
  A.q = q;
  A.k = k;
  A.v = v;
  A.a = a;
  A.alpha = alpha;
  A.beta = beta;
  A.w_r = w_r;
  A.lens = (const int*)lens;
  A.H0 = H0;
  A.y = y;
  A.H_T = H_T;
  A.ckpt = ckpt;
  A.seg = (float*)workspace;
  A.segdec = (float*)((char*)workspace + p.seg);
  if (A.T == 0 && !H_T) return M2RNN_OK;
  hipStream_t s = (hipStream_t)stream;
  const int block = p.HPW * p.VB * 4;
  hipError_t e = hipSuccess;
  if (A.S > 1) {
    e = launch(pick(p, SSM_STATE), p.units * A.S, block, A, s);
    if (e == hipSuccess) e = launch_combine(A, false, s);
  }
  if (e == hipSuccess) e = launch(pick(p, SSM_FWD), p.units * A.S, block, A, s);
  return status(e);
}

template <int V>
const void* step_kernel(bool bf16) {
  return bf16 ? (const void*)&m2rnn_ssm_step_kernel<true, V> : (const void*)&m2rnn_ssm_step_kernel<false, V>;
}

}  // namespace

extern "C" {

int m2rnn_ssm_checkpoint_interval(int qkv_dtype, int64_t* steps) {
  if (!steps || (qkv_dtype != M2RNN_DTYPE_F32 && qkv_dtype != M2RNN_DTYPE_BF16)) return M2RNN_EINVAL;
  *steps = qkv_dtype == M2RNN_DTYPE_BF16 ? ssm_chunk<true>() : ssm_chunk<false>();
  return M2RNN_OK;
}

int m2rnn_ssm_fwd_workspace_size(const m2rnn_dims* dims, int qkv_dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_ssm(dims, qkv_dtype);
  if (st) return st;
  *bytes = make_plan(dims, qkv_dtype, false).total;
  return M2RNN_OK;
}

int m2rnn_ssm_fwd(const m2rnn_dims* dims, int qkv_dtype, const void* q, const void* k, const void* v, const float* a,
                  const float* alpha, const float* beta, const float* w_r, const int32_t* lens, const float* H0,
                  float* y, float* H_T, void* workspace, size_t workspace_bytes, void* stream) {
  return run_fwd(dims, qkv_dtype, q, k, v, a, alpha, beta, w_r, lens, H0, y, H_T, nullptr, false, workspace,
                 workspace_bytes, stream);
}

int m2rnn_ssm_fwd_ckpt(const m2rnn_dims* dims, int qkv_dtype, const void* q, const void* k, const void* v,
                       const float* a, const float* alpha, const float* beta, const float* w_r, const int32_t* lens,
                       const float* H0, float* y, float* H_T, float* ckpt, void* workspace, size_t workspace_bytes,
                       void* stream) {
  return run_fwd(dims, qkv_dtype, q, k, v, a, alpha, beta, w_r, lens, H0, y, H_T, ckpt, true, workspace,
                 workspace_bytes, stream);
}

int m2rnn_ssm_bwd_workspace_size(const m2rnn_dims* dims, int qkv_dtype, size_t* bytes) {
  if (!bytes) return M2RNN_EINVAL;
  const int st = check_ssm_bwd(dims, qkv_dtype);
  if (st) return st;
  *bytes = make_plan(dims, qkv_dtype, true).total;
  return M2RNN_OK;
}

int m2rnn_ssm_bwd(const m2rnn_dims* dims, int qkv_dtype, const void* q, const void* k, const void* v, const float* a,
                  const float* alpha, const float* beta, const float* w_r, const int32_t* lens, const float* ckpt,
                  const float* dy, const float* dH_T, float* dq, float* dk, float* dv, float* da, float* dalpha,
                  float* dbeta, float* dw_r, float* dH0, void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_ssm_bwd(dims, qkv_dtype);
  if (st) return st;
  if (dims->N == 0) return M2RNN_OK;
  if (!alpha || !beta || !w_r || !dalpha || !dbeta || !dw_r) return M2RNN_EINVAL;
  if (dims->B > 0 && dims->T > 0 && (!q || !k || !v || !a || !ckpt || !dy || !dq || !dk || !dv || !da))
    return M2RNN_EINVAL;
  const void* p16[] = {q, k, v, w_r, ckpt, dy, dH_T, dq, dk, dv, dw_r, dH0};
  for (const void* p : p16)
    if (p && !al16(p)) return M2RNN_EINVAL;
  const void* p4[] = {a, alpha, beta, lens, da, dalpha, dbeta};
  for (const void* p : p4)
    if (p && !al4(p)) return M2RNN_EINVAL;
  Plan p = make_plan(dims, qkv_dtype, true);
  if (p.total > 0 && (!workspace || workspace_bytes < p.total || !al16(workspace))) return M2RNN_EWORKSPACE;
  SsmArgs& A = p.A;
  char* ws = (char*)workspace;
  auto part = [&](size_t bytes) {
    char* at = ws;
    ws += bytes;
    return (float*)at;
  };
  A.q = q;
  A.k = k;
  A.v = v;
  A.a = a;
  A.alpha = alpha;
  A.beta = beta;
  A.w_r = w_r;
  A.lens = (const int*)lens;
  A.ckpt = const_cast<float*>(ckpt);  // read only by the backward
  A.dy = dy;
  A.dH_T = dH_T;
  A.dH0 = dH0;
  A.dv = dv;
  A.da = da;
  A.seg = part(p.seg);
  A.segdec = part(p.segdec);
  A.rloc = part(p.rloc);
  A.cdec = part(p.cdec);
  A.part_gate = (double*)part(p.gate);
  A.part_wr = part(p.wr);
  double* scratch = (double*)part(p.scratch);
  float* planes = part(p.planes);
  const long count = (long)A.B * A.T * A.G * A.K;
  A.dq = A.HS > 1 ? planes : dq;
  A.dk = A.HS > 1 ? planes + (long)A.HS * count : dk;
  hipStream_t s = (hipStream_t)stream;
  hipError_t e = hipSuccess;
  const long parts = (long)A.B * A.nch;
  const bool one = A.N == A.G * A.HS && A.CB == 1;  // one head and one block for each workgroup
  if (A.B > 0) {
    e = launch(pick(p, SSM_STATE_REV), p.units * A.S, p.HPW * p.VB * 4, A, s);
    if (e == hipSuccess) e = launch_combine(A, true, s);
    if (e == hipSuccess && A.nch > 0)
      e = launch(p.bf16 ? ssm_bwd_kernel_bf16(p.KP, p.VB, one) : ssm_bwd_kernel_f32(p.KP, p.VB, one),
                 (long)A.B * A.G * A.nch * A.HS, 64 * kSsmBwdWaves, A, s);
    if (e != hipSuccess) return status(e);
    if (A.HS > 1 && count > 0) {
      const long blocks = ceil_div(count, 1024);
      hipLaunchKernelGGL(m2rnn_ssm_planes_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536), 2), dim3(256), 0,
                         s, (const float*)A.dq, (const float*)A.dk, A.HS, count, dq, dk);
    }
  }
  const long NV = (long)A.N * A.V, slices = ceil_div(parts, kSsmSlice);
  const unsigned columns = (unsigned)(ceil_div(2L * A.N, 64) + ceil_div(NV, 64));
  double *gate_sums = scratch, *wr_sums = scratch + slices * 2 * A.N;
  hipLaunchKernelGGL(m2rnn_ssm_sums_kernel<float>, dim3(columns, (unsigned)(slices > 1 ? slices : 1)), dim3(1024), 0, s,
                     (const double*)A.part_gate, (const float*)A.part_wr, parts, A.N, NV, gate_sums, wr_sums, dbeta, dalpha,
                     dw_r);
  if (slices > 1)
    hipLaunchKernelGGL(m2rnn_ssm_sums_kernel<double>, dim3(columns), dim3(1024), 0, s, (const double*)gate_sums,
                       (const double*)wr_sums, slices, A.N, NV, nullptr, nullptr, dbeta, dalpha, dw_r);
  return status(hipGetLastError());
}

int m2rnn_ssm_step(const m2rnn_dims* dims, int qkv_dtype, const void* q, const void* k, const void* v, const float* a,
                   const float* alpha, const float* beta, const float* w_r, const float* H_in, float* H_out, float* y,
                   void* stream) {
  const int st = check_ssm(dims, qkv_dtype);
  if (st) return st;
  if (dims->T != 1) return M2RNN_EINVAL;
  if (dims->B == 0 || dims->N == 0) return M2RNN_OK;
  if (!q || !k || !v || !a || !alpha || !beta || !w_r || !H_out || !y) return M2RNN_EINVAL;
  const void* p16[] = {q, k, v, w_r, H_in, H_out, y};
  for (const void* p : p16)
    if (p && !al16(p)) return M2RNN_EINVAL;
  const void* p4[] = {a, alpha, beta};
  for (const void* p : p4)
    if (!al4(p)) return M2RNN_EINVAL;
  const long pairs = dims->B * dims->N;
  const uintptr_t state = (uintptr_t)pairs * dims->K * dims->V * sizeof(float);
  const uintptr_t in = (uintptr_t)H_in, out = (uintptr_t)H_out;
  if (H_in && in != out && in < out + state && out < in + state) return M2RNN_EINVAL;
  const bool bf = qkv_dtype == M2RNN_DTYPE_BF16;
  const int N = (int)dims->N, G = dims->Nqk ? (int)dims->Nqk : N, K = (int)dims->K, V = (int)dims->V;
  const void* kern = V == 16 ? step_kernel<16>(bf)
                     : V == 32 ? step_kernel<32>(bf)
                     : V == 64 ? step_kernel<64>(bf)
                               : step_kernel<128>(bf);
  void* args[] = {&q, &k, &v, &a, &alpha, &beta, &w_r, &H_in, &H_out, &y, (void*)&N, (void*)&G, (void*)&K};
  return status(hipLaunchKernel(kern, dim3((unsigned)pairs), dim3(256), args, 0, (hipStream_t)stream));
}

}  // extern "C"
