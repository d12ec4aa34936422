// Kernels of the selective state space scan (mathematics and precision: m2rnn_ssm_device.h).
//
//   m2rnn_ssm_state_kernel    what each time segment adds to the state (k, v and a alone), or in the
//                             reverse scan what each chunk and segment adds to the gradient's state
//   m2rnn_ssm_combine_kernel  the states that enter the segments, from those parts and the first state
//   m2rnn_ssm_fwd_kernel      y (and checkpoints and H_T), segment by segment, chunk after chunk
//   m2rnn_ssm_bwd_kernel      all gradients of one chunk, from the states on both of its sides
//   m2rnn_ssm_step_kernel     one token with the state in HBM
//
// Segments.  Within a workgroup the chunks of a segment follow each other with the state in
// registers; the launch cuts the sequence into as many segments as fill the chip.  The extra cost
// is reading k and v a second time (a third of the bytes at K = V); one kernel with a workgroup per
// (b, n) would leave 3/4 of the CUs idle at 64 pairs.
#pragma once

#include "m2rnn_ssm_device.h"

namespace m2rnn {

struct SsmArgs {
  const void *q, *k, *v;                   // [B,T,G,K], [B,T,G,K], [B,T,N,V]
  const float *a, *alpha, *beta, *w_r;     // [B,T,N], [N], [N], [N,V]
  const int* lens;                         // [B] or null (T)
  const float *H0, *dy, *dH_T;             // [B,N,K,V], [B,T,N,V], [B,N,K,V]
  float *y, *H_T, *ckpt;                   // ckpt [B,N,nch,K,V]
  float* seg;                              // [B,N,S,K,V] ([V,K] in the reverse scan)
  // log2 decays are summed in fp64 and kept in fp32: the rounding of x changes 2^x by |x| 2^-25 of it, next to nothing
  // where 2^x still counts
  float* segdec;                           // [B,N,S] log2 decay of each segment
  float* rloc;                             // [B,N,nch,V,K] reverse: the part of the segment's later chunks
  float* cdec;                             // [B,N,nch] reverse: log2 decay from the chunk's end to the segment's
  float *dq, *dk, *dv, *da;                // dq, dk: HS planes of [B,T,G,K]
  double* part_gate;                       // [B nch][2N] (dbeta, dalpha)
  float* part_wr;                          // [B nch][N V]
  float* dH0;
  int B, T, N, G, K, V;
  int S, cps, nch;                         // segments, chunks per segment, chunks
  int HB, CB, HS;                          // head blocks per group, column blocks per head, head splits (backward)
};

// Steps of batch entry b (lens is clamped, so a value out of range cannot lead past the arrays).
__device__ __forceinline__ int ssm_len(const SsmArgs& A, int b) {
  if (!A.lens) return A.T;
  const int n = A.lens[b];
  return n < 0 ? 0 : (n > A.T ? A.T : n);
}

// blockIdx -> (unit, share): the `share` workgroups of a unit read the same q and k rows.  They get
// ids that agree mod 8, which the dispatcher places on one XCD, so its L2 serves them.
__device__ __forceinline__ void ssm_unit(int shares, int units, int& unit, int& share) {
  const int id = blockIdx.x;
  if (shares > 1 && units % 8 == 0) {
    const int r = id / 8;
    share = r % shares;
    unit = (r / shares) * 8 + id % 8;
  } else {
    unit = id / shares;
    share = id % shares;
  }
}

// Row and column tile of the t-th lower-triangular tile (t = I (I + 1) / 2 + J).
__device__ __forceinline__ void tri_tile(int t, int& I, int& J) {
  I = t >= 6 ? 3 : (t >= 3 ? 2 : (t >= 1 ? 1 : 0));
  J = t - I * (I + 1) / 2;
}

// Decay factors 2^{c_i - c_j} of accumulator tile (I, J): lane column i = 16 I + n, rows
// j = 16 J + 4 g + r.  FD: the table's f carries D_j, and the diagonal tile gets it too.
template <int L, bool FD>
__device__ __forceinline__ void ssm_decay(const SsmTab<L>& tab, int I, int J, int g, int n, float (&o)[4]) {
  if (I != J) {
    const float x = tab.x[16 * I + n];
    const float4 f = *(const float4*)&tab.f[I - 1][16 * J + 4 * g];
    o[0] = x * f.x;
    o[1] = x * f.y;
    o[2] = x * f.z;
    o[3] = x * f.w;
  } else {
    const float hi = tab.chi[16 * I + n], lo = tab.clo[16 * I + n];
    const float4 h = *(const float4*)&tab.chi[16 * J + 4 * g];
    const float4 l = *(const float4*)&tab.clo[16 * J + 4 * g];
    float4 d = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if constexpr (FD) d = *(const float4*)&tab.d[16 * J + 4 * g];
    const float hj[4] = {h.x, h.y, h.z, h.w}, lj[4] = {l.x, l.y, l.z, l.w}, dj[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = 4 * g + r <= n ? dj[r] * exp2_((hi - hj[r]) + (lo - lj[r])) : 0.0f;
  }
}

// q k^T of tile (I, J) with the products of later steps replaced by zeros: the factor 0 that they get alone would let
// what is not finite there through, as NaN.
__device__ __forceinline__ f32x4 ssm_causal(f32x4 x, int I, int J, int g, int n) {
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = I != J || 4 * g + r <= n ? x[r] : 0.0f;
  return x;
}

// Four values as NP bf16 planes put together again.
template <int NP>
__device__ __forceinline__ void planes_vals4(const uint2 (&u)[NP], float (&o)[4]) {
#pragma unroll
  for (int i = NP - 1; i >= 0; --i) {
    const float x[4] = {bf16_lo_to_f32(u[i].x), bf16_hi_to_f32(u[i].x), bf16_lo_to_f32(u[i].y), bf16_hi_to_f32(u[i].y)};
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = i == NP - 1 ? x[e] : o[e] + x[e];
  }
}
// Four consecutive values of a bf16 plane set in LDS (NP planes, `plane` elements apart).
template <int NP>
__device__ __forceinline__ void lds_vals4(const uint16_t* p, int plane, float (&o)[4]) {
  uint2 u[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) u[i] = *(const uint2*)(p + i * plane);
  planes_vals4<NP>(u, o);
}

// The step size, its derivative by a and the log2 decay of lane j's step from its gate pre-activation (live:
// within the sequence and the chunk).
__device__ __forceinline__ void ssm_gate(bool live, float a, float alpha, float beta, float& delta, float& sigma,
                                         double& lg) {
  delta = sigma = 0.0f;
  lg = 0.0;
  if (live) {
    softplus_sigma(a + beta, delta, sigma);
    lg = log2_decay(alpha, delta);
  }
}

// ------------------------------------------------------------------ forward

// One workgroup per (b, query/key group, HPW heads or VB columns of one head, segment).  A wave owns
// 16 value columns and their K x 16 part of the state, which stays in registers in the
// accumulator layout; that layout is also the operand layout of H^T q, so the state never moves.
// HPW > 1 (V = 16 heads sharing q and k): one wave per head, q k^T formed once for all of them.
// Otherwise the waves of a head share its masked and decayed q k^T through LDS.
//
// Bound by HBM and issue together: at B2 N32 T16384 K=V=64 (bf16) the kernel takes 158 us at best and 185 on average for
// 0.69 GB, 3.7 to 4.4 TB/s, with a SIMD's VALU busy 61% of the cycles and its MFMA 24%; B4 N128 T4096 K=64 V=16 with one
// query/key takes 101 to 106 us (with checkpoints), VALU 75% (each head's decays and splits for 16 columns).
template <bool BF16, int KP, int VB, int HPW>
__global__ void __launch_bounds__(HPW * VB * 4) m2rnn_ssm_fwd_kernel(SsmArgs A) {
  constexpr int L = ssm_chunk<BF16>(), NI = L / 16, NS = L / 32, KS = KP / 32, KM = KP / 16, NP = BF16 ? 1 : 3;
  constexpr int WPH = VB / 16, NW = HPW * WPH, NTH = 64 * NW, VT = HPW * VB;
  constexpr int STK = ssm_stride(KP), STV = ssm_stride(VT), NT = NI * (NI + 1) / 2;
  constexpr int SETS = (NI / 2) * (NI / 2 + 1);  // (I, s) operand sets of P
  constexpr bool SHARE_P = WPH > 1, SHARE_G = HPW > 1;
  static_assert(!(SHARE_P && SHARE_G), "several heads per workgroup: one wave each");
  __shared__ __attribute__((aligned(16))) uint16_t sq[NP * L * STK];
  __shared__ __attribute__((aligned(16))) uint16_t sk[NP * L * STK];
  __shared__ __attribute__((aligned(16))) uint16_t sv[NP * L * STV];
  __shared__ __attribute__((aligned(16))) SsmTab<L> tab[HPW];
  __shared__ __attribute__((aligned(16))) float4 gbuf[SHARE_G ? NT * 64 : 1];
  __shared__ __attribute__((aligned(16))) uint2 pbuf[SHARE_P ? SETS * 3 * 2 * 64 : 1];

  int tid = threadIdx.x;
  const int lane = tid & 63;
  int g = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int unit, share;
  ssm_unit(A.HB * A.CB, A.B * A.G * A.S, unit, share);
  const int s_ = unit % A.S, bg = unit / A.S;
  const int b = bg / A.G, grp = bg % A.G;
  const int hpg = A.N / A.G;                              // heads per group
  const int h0 = grp * hpg + (share / A.CB) * HPW;        // first head
  const int hn = min(HPW, (grp + 1) * hpg - h0);          // heads here
  const int cb = share % A.CB;
  const int head = h0 + w / WPH;                          // this wave's head
  const bool mine = w / WPH < hn;
  const int c0 = cb * VB + (w % WPH) * 16;                // its first column within the head
  const int lc = w * 16;                                  // and within the workgroup's block
  const int K = A.K, V = A.V, T = A.T;
  const int Tb = ssm_len(A, b);
  const long krow = (long)A.G * K, vrow = (long)A.N * V;
  const char* esz_base_q = (const char*)A.q + (((long)b * T * A.G + grp) * K) * (BF16 ? 2 : 4);
  const char* esz_base_k = (const char*)A.k + (((long)b * T * A.G + grp) * K) * (BF16 ? 2 : 4);
  const char* esz_base_v = (const char*)A.v + ((long)b * T * vrow + (long)h0 * V + cb * VB) * (BF16 ? 2 : 4);
  const int vcols = HPW > 1 ? hn * V : VB;

  // the state that enters the segment
  f32x4 H[KM];
  const float* Hin = A.S > 1 ? A.seg + (((long)b * A.N + head) * A.S + s_) * K * V
                             : (A.H0 ? A.H0 + ((long)b * A.N + head) * K * V : nullptr);
#pragma unroll
  for (int m = 0; m < KM; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int kk = 16 * m + 4 * g + r;
      H[m][r] = (Hin && mine && kk < K) ? Hin[(long)kk * V + c0 + n] : 0.0f;
    }
  float wr[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (mine) {
#pragma unroll
    for (int r = 0; r < 4; ++r) wr[r] = A.w_r[(long)head * V + c0 + 4 * g + r];
  }
  const bool preps = w % WPH == 0;
  const float alpha = mine ? A.alpha[head] : 0.0f, beta = mine ? A.beta[head] : 0.0f;

  SsmPieces<BF16, L, KP, NTH> pq, pk;
  SsmPieces<BF16, L, VT, NTH> pv;
  float pa = 0.0f;
  auto fetch = [&](int ch) {
    const int t0 = ch * L, rows = min(L, Tb - t0);
    pq.load(esz_base_q + (long)t0 * krow * (BF16 ? 2 : 4), krow, K, rows, tid);
    pk.load(esz_base_k + (long)t0 * krow * (BF16 ? 2 : 4), krow, K, rows, tid);
    pv.load(esz_base_v + (long)t0 * vrow * (BF16 ? 2 : 4), vrow, vcols, rows, tid);
    if (preps && mine && lane < rows) pa = A.a[((long)b * T + t0 + lane) * A.N + head];
  };
  const int ch0 = s_ * A.cps, ch1 = min(A.nch, ch0 + A.cps);
  if (ch0 < ch1) fetch(ch0);
  for (int ch = ch0; ch < ch1; ++ch) {
    const int t0 = ch * L;
    if (A.ckpt && mine) {
      float* o = A.ckpt + (((long)b * A.N + head) * A.nch + ch) * K * V;
#pragma unroll
      for (int m = 0; m < KM; ++m) {
        if (16 * m >= K) break;
#pragma unroll
        for (int r = 0; r < 4; ++r) o[(unsigned)((16 * m + 4 * g + r) * V + c0 + n)] = H[m][r];
      }
    }
    if (t0 >= Tb) {  // past the sequence's end (the same for the whole workgroup): zeros, the state as it is
      if (mine) {
#pragma unroll
        for (int I = 0; I < NI; ++I) {
          const int t = t0 + 16 * I + n;
          if (t < T)
            *(float4*)(A.y + ((long)b * T + t) * vrow + (long)head * V + c0 + 4 * g) = make_float4(0, 0, 0, 0);
        }
      }
      continue;
    }
    __syncthreads();  // the previous chunk's reads are done
    tid = fresh(tid);
    g = fresh(g);
    n = fresh(n);
    pq.store(sq, tid);
    pk.store(sk, tid);
    pv.store(sv, tid);
    if (preps) {
      float delta, sigma;
      double lg;
      ssm_gate(lane < L && t0 + lane < Tb, pa, alpha, beta, delta, sigma, lg);
      ssm_tables<L, true>(tab[w / WPH], lane, delta, lg);
    }
    __syncthreads();
    if (ch + 1 < ch1) fetch(ch + 1);

    const SsmTab<L>& tb = tab[w / WPH];
    // q k^T tile (I, J) without later steps: lane column i, rows j
    auto qk_tile = [&](int I, int J) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint4 ko[NP], qo[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          ko[p] = lds_row(sk + p * L * STK, STK, 16 * J, 32 * s, g, n);
          qo[p] = lds_row(sq + p * L * STK, STK, 16 * I, 32 * s, g, n);
        }
        acc = mfma_planes<NP, NP>(ko, qo, acc);
      }
      return ssm_causal(acc, I, J, g, n);
    };
    if constexpr (SHARE_P) {
      for (int t = w; t < NT; t += NW) {
        int I, J;
        tri_tile(t, I, J);
        const f32x4 acc = qk_tile(I, J);
        float d[4], x[4];
        ssm_decay<L, true>(tb, I, J, g, n, d);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = acc[r] * d[r];
        uint2 pl[3];
        split3x4(x, pl);
        const int set = (I / 2) * (I / 2 + 1) + (I & 1) * (I / 2 + 1) + J / 2;
#pragma unroll
        for (int p = 0; p < 3; ++p) pbuf[((set * 3 + p) * 2 + (J & 1)) * 64 + lane] = pl[p];
      }
      __syncthreads();
    } else if constexpr (SHARE_G) {
      for (int t = w; t < NT; t += NW) {
        int I, J;
        tri_tile(t, I, J);
        const f32x4 acc = qk_tile(I, J);
        gbuf[t * 64 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      }
      __syncthreads();
    }

    uint4 vop[NS][NP];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int p = 0; p < NP; ++p) vop[s][p] = lds_col(sv + p * L * STV, STV, 32 * s, lc, g, n);
    // the same values in fp32, in the operand's order
    float vf[NS][8];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      uint2 lo[NP], hi[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        lo[p] = make_uint2(vop[s][p].x, vop[s][p].y);
        hi[p] = make_uint2(vop[s][p].z, vop[s][p].w);
      }
      float a4[4], b4[4];
      planes_vals4<NP>(lo, a4);
      planes_vals4<NP>(hi, b4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        vf[s][e] = a4[e];
        vf[s][4 + e] = b4[e];
      }
    }
    uint4 hp[KS][3];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint2 x[3], y2[3];
      const float h0v[4] = {H[2 * s][0], H[2 * s][1], H[2 * s][2], H[2 * s][3]};
      const float h1v[4] = {H[2 * s + 1][0], H[2 * s + 1][1], H[2 * s + 1][2], H[2 * s + 1][3]};
      split3x4(h0v, x);
      split3x4(h1v, y2);
#pragma unroll
      for (int p = 0; p < 3; ++p) hp[s][p] = cat(x[p], y2[p]);
    }
    // the state that leaves the chunk (the one that entered is in hp)
    const float dl = tb.e[L - 1];
#pragma unroll
    for (int m = 0; m < KM; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) H[m][r] *= dl;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const float4 w0 = *(const float4*)&tb.w[32 * s + 4 * g], w1 = *(const float4*)&tb.w[32 * s + 16 + 4 * g];
      const float x[8] = {vf[s][0] * w0.x, vf[s][1] * w0.y, vf[s][2] * w0.z, vf[s][3] * w0.w,
                          vf[s][4] * w1.x, vf[s][5] * w1.y, vf[s][6] * w1.z, vf[s][7] * w1.w};
      uint4 vs[3];
      split3x8(x, vs);
#pragma unroll
      for (int m = 0; m < KM; ++m) {
        uint4 ko[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) ko[p] = lds_col(sk + p * L * STK, STK, 32 * s, 16 * m, g, n);
        H[m] = mfma_planes<NP, 3>(ko, vs, H[m]);
      }
    }
    // A value of v that is not finite makes its column of the state NaN (also through a weight 0), but must not reach the
    // steps before it, whose zero scores it meets in the same product.  The state shows such a chunk, so the others pay a
    // comparison (0 to 3% of the call's time with the state formed before y): its products are taken without
    // those values, and y is NaN from each column's first one on.
    int bad = L;
    const bool odd = __builtin_amdgcn_ballot_w64(H[0][0] != H[0][0]) != 0;
    if (odd) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (fabsf(vf[s][e]) <= 3.4028234e38f) continue;
          bad = min(bad, 32 * s + 16 * (e / 4) + 4 * g + e % 4);
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            unsigned* word = e / 2 == 0 ? &vop[s][p].x : e / 2 == 1 ? &vop[s][p].y : e / 2 == 2 ? &vop[s][p].z : &vop[s][p].w;
            *word &= e % 2 ? 0x0000FFFFu : 0xFFFF0000u;
          }
        }
      bad = min(bad, __shfl_xor(bad, 16));
      bad = min(bad, __shfl_xor(bad, 32));
    }
#pragma unroll
    for (int I = 0; I < NI; ++I) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint4 qo[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) qo[p] = lds_row_acc(sq + p * L * STK, STK, 16 * I, 32 * s, g, n);
        acc = mfma_planes<3, NP>(hp[s], qo, acc);
      }
      const float e = tb.e[16 * I + n];
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] *= e;
#pragma unroll
      for (int s = 0; s <= I / 2; ++s) {
        uint4 po[3];
        if constexpr (SHARE_P) {
          const int set = (I / 2) * (I / 2 + 1) + (I & 1) * (I / 2 + 1) + s;
#pragma unroll
          for (int p = 0; p < 3; ++p) {
            const uint2* pb = &pbuf[((set * 3 + p) * 2) * 64 + lane];
            po[p] = cat(pb[0], 2 * s + 1 <= I ? pb[64] : make_uint2(0, 0));
          }
        } else {
          // (P is split here, in the wave that uses it.  Feeding the fp32 MFMA instead, which takes the accumulator's
          // registers as they are, saves 24 VALU operations a tile but costs 4 dependent passes of 32 cycles: the
          // padded batch of B4 N128 T4096 V=16 prompts took 83 us instead of 78.)
          uint2 half[2][3];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int J = 2 * s + hf;
            if (J <= I) {
              f32x4 qk;
              if constexpr (SHARE_G) {
                const float4 t4 = gbuf[(I * (I + 1) / 2 + J) * 64 + lane];
                qk = f32x4{t4.x, t4.y, t4.z, t4.w};
              } else {
                qk = qk_tile(I, J);
              }
              float d[4], x[4];
              ssm_decay<L, true>(tb, I, J, g, n, d);
#pragma unroll
              for (int r = 0; r < 4; ++r) x[r] = qk[r] * d[r];
              split3x4(x, half[hf]);
            } else {
#pragma unroll
              for (int p = 0; p < 3; ++p) half[hf][p] = make_uint2(0, 0);
            }
          }
#pragma unroll
          for (int p = 0; p < 3; ++p) po[p] = cat(half[0][p], half[1][p]);
        }
        acc = mfma_planes<NP, 3>(vop[s], po, acc);
      }
      float vv[4];
      lds_vals4<NP>(sv + (16 * I + n) * STV + lc + 4 * g, L * STV, vv);
      const int t = t0 + 16 * I + n;
      if (mine && t < T) {
        const bool live = t < Tb;
        float4 o;
        o.x = live ? acc[0] + wr[0] * vv[0] : 0.0f;
        o.y = live ? acc[1] + wr[1] * vv[1] : 0.0f;
        o.z = live ? acc[2] + wr[2] * vv[2] : 0.0f;
        o.w = live ? acc[3] + wr[3] * vv[3] : 0.0f;
        *(float4*)(A.y + ((long)b * T + t) * vrow + (long)head * V + c0 + 4 * g) = o;
      }
    }
    if (odd && mine) {  // (a lane's own stores to one address keep their order)
      int first[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) first[r] = __shfl(bad, 4 * g + r);
      for (int I = 0; I < NI; ++I) {
        const int t = t0 + 16 * I + n;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * I + n >= first[r] && t < Tb)
            A.y[((long)b * T + t) * vrow + (long)head * V + c0 + 4 * g + r] = __builtin_nanf("");
      }
    }
  }
  if (A.H_T && s_ == A.S - 1 && mine) {
    float* o = A.H_T + ((long)b * A.N + head) * K * V + c0 + n;
#pragma unroll
    for (int m = 0; m < KM; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int kk = 16 * m + 4 * g + r;
        if (kk < K) o[(long)kk * V] = H[m][r];
      }
  }
}

// ------------------------------------------------------------------ what a segment adds to the state

// Both walk their segment's chunks last to first.
// REV = false: seg = sum over the segment's steps of their decayed D_j k_j v_j^T, as [K,V].  A step's weight holds the
// decay to the segment's end, so the sum is never decayed, and the rows read last are those that the forward
// reads first (227 us for the 16K-token prompt, 231 in the forward's order with the state decayed each chunk).
// REV = true: the gradient's state R, seg = sum of the decayed q_i dy_i^T that
// leaves the segment backwards, as [V,K]; before each chunk the part accumulated so far (what the
// segment's later chunks send to it) goes to rloc, and its log2 decay to cdec.
// Work split as in the forward.  The weights multiply v (or dy) in the operand.  dy, in fp32, goes straight
// from HBM into the operands (a lane's column of 16, rows of 64 bytes), since its planes would need three
// times v's LDS.  The decays of the next chunk are formed beside the products of this one.  Bound by
// HBM and its latency: 65 to 72 us for k and v of B2 N32 T16384 K=V=64 (3.8 to 4.2 TB/s), 43 to 45 us for the
// reverse pass of B4 N16 T4096 (0.17 GB read and written).  Two chunks in flight instead of one took 71 us.
template <bool BF16, int KP, int VB, int HPW, bool REV>
__global__ void __launch_bounds__(HPW * VB * 4) m2rnn_ssm_state_kernel(SsmArgs A) {
  constexpr int L = ssm_chunk<BF16>(), NS = L / 32, KM = KP / 16, NP = BF16 ? 1 : 3;
  constexpr int WPH = VB / 16, NW = HPW * WPH, NTH = 64 * NW, VT = HPW * VB;
  constexpr int STK = ssm_stride(KP), STV = ssm_stride(VT);
  __shared__ __attribute__((aligned(16))) uint16_t sk[NP * L * STK];
  __shared__ __attribute__((aligned(16))) uint16_t sv[REV ? 8 : NP * L * STV];
  __shared__ __attribute__((aligned(16))) float weight[2][HPW][L];
  __shared__ float sdec[2][HPW];

  int tid = threadIdx.x;
  const int lane = tid & 63;
  int g = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int unit, share;
  ssm_unit(A.HB * A.CB, A.B * A.G * A.S, unit, share);
  const int s_ = unit % A.S, bg = unit / A.S;
  if (!REV && s_ == A.S - 1) return;  // nothing follows the last segment
  const int b = bg / A.G, grp = bg % A.G;
  const int hpg = A.N / A.G;
  const int h0 = grp * hpg + (share / A.CB) * HPW;
  const int hn = min(HPW, (grp + 1) * hpg - h0);
  const int cb = share % A.CB;
  const int hw = w / WPH, head = h0 + hw;
  const bool mine = hw < hn;
  const int c0 = cb * VB + (w % WPH) * 16, lc = w * 16;
  const int K = A.K, V = A.V, T = A.T;
  const int Tb = ssm_len(A, b);
  const long krow = (long)A.G * K, vrow = (long)A.N * V;
  const char* kbase = (const char*)(REV ? A.q : A.k) + (((long)b * T * A.G + grp) * K) * (BF16 ? 2 : 4);
  const char* vbase = (const char*)A.v + ((long)b * T * vrow + (long)h0 * V + cb * VB) * (BF16 ? 2 : 4);
  const float* ubase = A.dy + (long)b * T * vrow + (long)head * V + c0;
  const int vcols = HPW > 1 ? hn * V : VB;
  const bool preps = w % WPH == 0;
  const float alpha = mine ? A.alpha[head] : 0.0f, beta = mine ? A.beta[head] : 0.0f;
  double dec = 0.0;  // log2 decay of the chunks done (in the preparing waves)

  f32x4 H[KM];
#pragma unroll
  for (int m = 0; m < KM; ++m) H[m] = f32x4{0, 0, 0, 0};
  SsmPieces<BF16, L, KP, NTH> pk;
  SsmPieces<BF16, L, VT, NTH> pv;
  float pu[NS][8];
  float pa = 0.0f;
  auto fetch = [&](int ch) {
    const int t0 = ch * L, rows = min(L, Tb - t0);
    pk.load(kbase + (long)t0 * krow * (BF16 ? 2 : 4), krow, K, rows, tid);
    if constexpr (REV) {
      const float* u = ubase + (long)(t0 + 4 * g) * vrow + n;
      const int last = mine ? rows - 4 * g : 0;
      if (mine && rows == L) {  // (whole chunks without a test for each row)
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int e = 0; e < 8; ++e) pu[s][e] = u[(32 * s + 16 * (e / 4) + e % 4) * vrow];
      } else {
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int j = 32 * s + 16 * (e / 4) + e % 4;
            pu[s][e] = j < last ? u[j * vrow] : 0.0f;
          }
      }
    } else {
      pv.load(vbase + (long)t0 * vrow * (BF16 ? 2 : 4), vrow, vcols, rows, tid);
    }
  };
  auto fetch_a = [&](int ch) {
    const int t = ch * L + lane;
    if (preps && mine && lane < L && t < Tb) pa = A.a[((long)b * T + t) * A.N + head];
  };
  // the weight of each step in the state that leaves chunk ch: D_j 2^{c_L - c_j}, in the reverse scan 2^{c_j}
  double cl = 0.0;
  auto weights = [&](int ch, int buf) {
    if (!preps) return;
    float delta, sigma;
    double lg;
    ssm_gate(lane < L && ch * L + lane < Tb, pa, alpha, beta, delta, sigma, lg);
    const double c = prefix64(lg);
    cl = lane64(c, L - 1);
    if constexpr (REV) {
      if (lane < L) weight[buf][hw][lane] = exp2_((float)c);
      if (lane == 0) sdec[buf][hw] = exp2_((float)cl);
    } else {
      if (lane < L) weight[buf][hw][lane] = delta * exp2_((float)(cl - c + dec));
    }
  };
  const int ch0 = s_ * A.cps, ch1 = min(A.nch, ch0 + A.cps);
  const int last = ch1 - 1, count = ch1 - ch0;
  if (count > 0) {
    fetch_a(last);
    fetch(last);
    weights(last, 0);
    if (count > 1) fetch_a(last - 1);
  }
  for (int c = 0; c < count; ++c) {
    const int ch = last - c, buf = c & 1;
    if constexpr (REV) {
      if (mine) {
        float* o = A.rloc + ((((long)b * A.N + head) * A.nch + ch) * V + c0 + n) * K;
#pragma unroll
        for (int m = 0; m < KM; ++m)
          if (16 * m + 4 * g < K) *(float4*)(o + 16 * m + 4 * g) = make_float4(H[m][0], H[m][1], H[m][2], H[m][3]);
        if (preps && lane == 0 && cb == 0) A.cdec[((long)b * A.N + head) * A.nch + ch] = (float)dec;
      }
    }
    dec += cl;
    __syncthreads();  // the previous chunk's reads are done
    tid = fresh(tid);
    g = fresh(g);
    n = fresh(n);
    pk.store(sk, tid);
    if constexpr (!REV) pv.store(sv, tid);
    float x[NS][8];
    if constexpr (REV) {
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[s][e] = pu[s][e];
    }
    __syncthreads();
    if (c + 1 < count) fetch(ch - 1);
    if constexpr (REV) {
      const float dl = sdec[buf][hw];
#pragma unroll
      for (int m = 0; m < KM; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) H[m][r] *= dl;
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if constexpr (!REV) {
        uint2 lo[NP], hi[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const uint4 t = lds_col(sv + p * L * STV, STV, 32 * s, lc, g, n);
          lo[p] = make_uint2(t.x, t.y);
          hi[p] = make_uint2(t.z, t.w);
        }
        float a4[4], b4[4];
        planes_vals4<NP>(lo, a4);
        planes_vals4<NP>(hi, b4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[s][e] = a4[e];
          x[s][4 + e] = b4[e];
        }
      }
      const float4 w0 = *(const float4*)&weight[buf][hw][32 * s + 4 * g];
      const float4 w1 = *(const float4*)&weight[buf][hw][32 * s + 16 + 4 * g];
      const float ws[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[s][e] *= ws[e];
      uint4 vs[3];
      split3x8(x[s], vs);
#pragma unroll
      for (int m = 0; m < KM; ++m) {
        uint4 ko[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) ko[p] = lds_col(sk + p * L * STK, STK, 32 * s, 16 * m, g, n);
        H[m] = mfma_planes<NP, 3>(ko, vs, H[m]);
      }
    }
    if (c + 1 < count) {
      weights(ch - 1, buf ^ 1);
      if (c + 2 < count) fetch_a(ch - 2);
    }
  }
  if (mine) {
    float* o = A.seg + (((long)b * A.N + head) * A.S + s_) * K * V;
#pragma unroll
    for (int m = 0; m < KM; ++m) {
      if constexpr (REV) {
        if (16 * m + 4 * g < K)
          *(float4*)(o + (long)(c0 + n) * K + 16 * m + 4 * g) = make_float4(H[m][0], H[m][1], H[m][2], H[m][3]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int kk = 16 * m + 4 * g + r;
          if (kk < K) o[(long)kk * V + c0 + n] = H[m][r];
        }
      }
    }
    if (preps && lane == 0 && cb == 0) A.segdec[((long)b * A.N + head) * A.S + s_] = (float)dec;
  }
}

// ------------------------------------------------------------------ the states that enter the segments

// seg[s] <- the state that enters segment s, from the segments' own parts: forwards from H0 (first to
// last), in the reverse scan from dH_T (last to first, [V,K]), which also leaves dH0.  One thread
// per element of a pair's state; the segments are few and their reads independent of the carry.  6 to 10 us,
// a launch and three or four dependent trips to memory.
template <bool REV>
__global__ void __launch_bounds__(256) m2rnn_ssm_combine_kernel(SsmArgs A) {
  const long KV = (long)A.K * A.V;
  const unsigned per = (unsigned)((KV + 255) / 256);
  const long blocks = (long)A.B * A.N * per;
  for (long blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
    const long e = (blk % per) * 256 + threadIdx.x;
    const long pair = blk / per;
    if (e >= KV) continue;
    // the element's place in a [K,V] state
    const long at = REV ? (e % A.K) * A.V + e / A.K : e;
    const float* first = REV ? A.dH_T : A.H0;
    float carry = first ? first[pair * KV + at] : 0.0f;
    float* p = A.seg + pair * A.S * KV + e;
    const float* d = A.segdec + pair * A.S;
    // the segments' parts do not depend on the carry: eight of them in flight at a time
    for (int i = 0; i < A.S; i += 8) {
      float own[8], dec[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int s = REV ? A.S - 1 - i - j : i + j;
        own[j] = i + j < A.S ? p[s * KV] : 0.0f;
        dec[j] = i + j < A.S ? d[s] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int s = REV ? A.S - 1 - i - j : i + j;
        if (i + j < A.S) {
          p[s * KV] = carry;
          carry = __builtin_fmaf(exp2_(dec[j]), carry, own[j]);
        }
      }
    }
    if (REV && A.dH0) A.dH0[pair * KV + at] = carry;
  }
}

// ------------------------------------------------------------------ backward

constexpr int kSsmBwdWaves = 4;

// The factors of ssm_decay with the roles turned: lane column j = 16 J + n, rows i = 16 I + 4 g + r.  The
// same products and differences, so both tiles hold the same numbers.
template <int L>
__device__ __forceinline__ void ssm_decay_col(const SsmTab<L>& tab, int I, int J, int g, int n, float (&o)[4]) {
  if (I != J) {
    const float f = tab.f[I - 1][16 * J + n];
    const float4 x = *(const float4*)&tab.x[16 * I + 4 * g];
    o[0] = x.x * f;
    o[1] = x.y * f;
    o[2] = x.z * f;
    o[3] = x.w * f;
  } else {
    const float hi = tab.chi[16 * J + n], lo = tab.clo[16 * J + n];
    const float4 h = *(const float4*)&tab.chi[16 * I + 4 * g];
    const float4 l = *(const float4*)&tab.clo[16 * I + 4 * g];
    const float hj[4] = {h.x, h.y, h.z, h.w}, lj[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = n <= 4 * g + r ? exp2_((hj[r] - hi) + (lj[r] - lo)) : 0.0f;
  }
}

// All gradients of one chunk of one query/key group (or of a part of its heads).  With u = dy,
// H the state that enters the chunk, R the gradient of the state that leaves it, and
//     P_ij = 2^{c_i - c_j} (q_i . k_j),   X_ij = 2^{c_i - c_j} D_j (u_i . v_j)   (j <= i):
//     dv_j = D_j (sum_i P_ij u_i + 2^{c_L - c_j} R^T k_j) + w_r (.) u_j
//     dq_i = sum_j X_ij k_j + 2^{c_i} H u_i
//     dk_j = sum_i X_ij q_i + D_j 2^{c_L - c_j} R v_j
// and for the decays, with M_ij = 2^{c_i - c_j} (q_i . k_j)(u_i . v_j),
//     g_t = <R_t, f_t H_{t-1}> = sum_{i >= t > j} D_j M_ij + sum_{i >= t} q_i . 2^{c_i} H u_i
//           + sum_{j < t} D_j k_j . 2^{c_L - c_j} R v_j + 2^{c_L} <R, H>
//     dD_t = sum_{i >= t} M_it + k_t . 2^{c_L - c_t} R v_t - alpha g_t.
// The double sum telescopes (row sums less column sums of the strict triangle); both are taken of
// the same M_ij and added in fp64, so what cancels cancels exactly and a decay that forgets at once
// leaves no residue of the terms on the diagonal.
//
// Every chunk has its own workgroup (no chain), which walks its heads one after the other; heads of
// 128 value columns go as two blocks of 64, since all gradients are sums over value columns.
// X is summed over the heads before it meets k and q (one product for all heads that share them).
// A wave owns a 16-step tile of rows (X for dq, row sums of M) and the same tile of columns (X for dk,
// P, column sums of M), five tiles for every wave: formed in both orientations, X needs no exchange
// and only P goes through LDS.  H and R come from HBM straight into operands: each wave takes 16
// of the K rows of H and R for the terms that enter and leave, 16 value columns for dv.
// ONE: the workgroup has one head of one block, so nothing lives from one pass of the loop to the next (B4 N16 T4096
// K=V=64, bf16: 163 to 175 us, 0.58 GB moved at 3.4 TB/s).  Neither HBM nor issue is full (VALU 42%, MFMA 16%, LDS 35% of
// the cycles): two workgroups of four waves a CU, by registers and LDS, wait for their products and barriers.
// With several heads or blocks (!ONE) 22 registers spill at K = VB = 64 in bf16: the call takes 195 us for N16 in groups
// of 4 heads (213 with one query/key each) and 378 us at V = 128, 1.8 times V = 64.
template <bool BF16, int KP, int VB, bool ONE>
__global__ void __launch_bounds__(64 * kSsmBwdWaves, KP == 128 ? 1 : 2) m2rnn_ssm_bwd_kernel(SsmArgs A) {
  constexpr int L = ssm_chunk<BF16>(), NI = L / 16, NS = L / 32, KS = KP / 32, KM = KP / 16, NP = BF16 ? 1 : 3;
  constexpr int NW = kSsmBwdWaves, NTH = 64 * NW;
  static_assert(VB == 32 || VB == 64, "heads of 16 columns have a kernel of their own");
  constexpr int VS = VB / 32, VM = VB / 16;                          // contraction steps over the columns, their tiles
  constexpr int STK = ssm_stride(KP), STV = ssm_stride(VB);
  constexpr int MPW = KM >= NW ? KM / NW : 1;                        // K tiles per wave
  constexpr int TPV = VM * NI / NW;                                  // dv tiles per wave, one V tile
  constexpr bool AHEAD = VB <= 32;                                   // the next block's v and u fit in registers meanwhile
  constexpr int SETS = NI == 4 ? 6 : 2;                              // (J, s) operand sets of P
  constexpr int QW = NP * L * STK, PW = SETS * 3 * 2 * 64 * 4;       // elements of the q and P blocks
  constexpr int XW = (KP * L * 2 > 3 * L * STV ? KP * L * 2 : 3 * L * STV);
  __shared__ __attribute__((aligned(16))) uint16_t sk[NP * L * STK];
  __shared__ __attribute__((aligned(16))) uint16_t sqp[QW > PW ? QW : PW];  // q before and after the heads, P between
  __shared__ __attribute__((aligned(16))) uint16_t sv[NP * L * STV];
  __shared__ __attribute__((aligned(16))) uint16_t su[XW];                 // u; dq's or dk's entering terms at the end
  __shared__ __attribute__((aligned(16))) SsmTabBwd<L> tabs[2];
  __shared__ double rowp[L], colp[L], ap[KM][L], bp[KM][L], rh[KM];
  __shared__ float dgp[L], dwp[NI][VB];
  uint16_t* const sq = sqp;
  uint2* const pbuf = (uint2*)sqp;

  int tid = threadIdx.x;
  const int lane = tid & 63;
  int g = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int unit, hs;
  ssm_unit(A.HS, A.B * A.G * A.nch, unit, hs);
  const int ch = unit % A.nch, bg = unit / A.nch;
  const int b = bg / A.G, grp = bg % A.G;
  const int K = A.K, V = A.V, T = A.T, N = A.N;
  const int hpg = N / A.G, per = (hpg + A.HS - 1) / A.HS;
  const int hb = grp * hpg + hs * per, he = min(grp * hpg + hpg, hb + per);
  const int CB = ONE ? 1 : A.CB, blocks = ONE ? 1 : (he > hb ? he - hb : 0) * CB;
  const int t0 = ch * L;
  const int Tb = ssm_len(A, b);
  const int rows = min(L, Tb - t0);
  const long krow = (long)A.G * K, vrow = (long)N * V, row0 = (long)b * T + t0;

  // this wave's tiles: rows It, columns Jt of the triangle (four tiles: one of each; two: waves 0, 1 the
  // rows, 2, 3 the columns), K tiles m0 .. m0 + MPW - 1 (with two: waves 0, 1 for dq, 2, 3 for dk)
  int It = w, Jt = NI == 4 ? w : w - 2;
  const bool hasI = It < NI, hasJ = Jt >= 0;
  const bool hasdq = KM >= NW || w < KM, hasdk = KM >= NW || w >= NW - KM;
  const int mq = KM >= NW ? w * MPW : w, mk = KM >= NW ? w * MPW : w - (NW - KM);
  const int mv = (w * TPV) / NI, jv0 = (w * TPV) % NI;
  // Every wave has dv tiles.  With one head the test stays, as a branch around R's loads and the products of dv: without
  // it the kernel takes 6% longer; with several heads 6% longer with it (38 registers spilled, not 22).
  const bool hasv = !ONE || w * TPV < VM * NI;

  SsmPieces<BF16, L, VB, NTH> pv;
  SsmPieces<false, L, VB, NTH> pu;
  auto fetch = [&](int blk) {
    const int h = hb + blk / CB;
    const long off = row0 * vrow + (long)h * V + (blk % CB) * VB;
    pv.load(BF16 ? (const void*)((const uint16_t*)A.v + off) : (const void*)((const float*)A.v + off), vrow, VB, rows,
            tid);
    pu.load(A.dy + off, vrow, VB, rows, tid);
  };
  // wave NW - 1 forms the tables of head h (its lanes: the chunk's steps)
  const bool live = lane < L && t0 + lane < Tb;
  float pa = 0.0f, alpha = 0.0f, beta = 0.0f;
  auto fetch_a = [&](int h) {
    pa = live ? A.a[(row0 + lane) * N + h] : 0.0f;
    alpha = A.alpha[h];
    beta = A.beta[h];
  };
  auto tables = [&](SsmTabBwd<L>& tab) {
    float delta, sigma;
    double lg;
    ssm_gate(live, pa, alpha, beta, delta, sigma, lg);
    ssm_tables<L, false>(tab, lane, delta, lg);
    if (lane < L) tab.s[lane] = sigma;
  };
  SsmPieces<BF16, L, KP, NTH> pq;
  auto fetch_q = [&]() {
    const long off = row0 * krow + (long)grp * K;
    pq.load(BF16 ? (const void*)((const uint16_t*)A.q + off) : (const void*)((const float*)A.q + off), krow, K, rows,
            tid);
  };
  // H and R as this wave's products take them: R^T for dv (rows c, contraction kk), H and R for dq and dk (rows
  // kk, contraction c)
  float4 tR[KS][2], tI[KS][2];
  float hx[MPW][VS][8], rx[MPW][VS][8], ix[MPW][VS][8], idec;
  auto fetch_RT = [&](int blk) {
    const long pair = (long)b * N + hb + blk / CB;
    const int cb = blk % CB;
    const float* Rp = A.rloc + ((pair * A.nch + ch) * V + cb * VB) * K;        // [V][K]
    const float* Ip = A.seg + ((pair * A.S + ch / A.cps) * V + cb * VB) * K;   // [V][K]
    idec = A.cdec[pair * A.nch + ch];
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kk = 32 * s + 8 * g + 4 * h;
        tR[s][h] = tI[s][h] = make_float4(0, 0, 0, 0);
        if (hasv && kk < K) {
          tR[s][h] = *(const float4*)(Rp + (unsigned)((16 * mv + n) * K + kk));
          tI[s][h] = *(const float4*)(Ip + (unsigned)((16 * mv + n) * K + kk));
        }
      }
  };
  auto fetch_HR = [&](int blk) {
    const long pair = (long)b * N + hb + blk / CB;
    const int cb = blk % CB;
    const float* Hp = A.ckpt + (pair * A.nch + ch) * K * V + cb * VB;          // [K][V]
    const float* Rp = A.rloc + ((pair * A.nch + ch) * V + cb * VB) * K;        // [V][K]
    const float* Ip = A.seg + ((pair * A.S + ch / A.cps) * V + cb * VB) * K;   // [V][K]
#pragma unroll
    for (int p = 0; p < MPW; ++p)
#pragma unroll
      for (int s = 0; s < VS; ++s) {
        const int c = 32 * s + 8 * g, kr = 16 * (mk + p) + n;
        const int kk = hasdq ? 16 * (mq + p) + n : kr;  // two K tiles: the waves of dk take H for <R, H>
#pragma unroll
        for (int e = 0; e < 8; ++e) hx[p][s][e] = rx[p][s][e] = ix[p][s][e] = 0.0f;
        if ((hasdq || KM < NW) && kk < K) {
          const float4 a4 = *(const float4*)(Hp + (unsigned)(kk * V + c)), b4 = *(const float4*)(Hp + (unsigned)(kk * V + c + 4));
          hx[p][s][0] = a4.x; hx[p][s][1] = a4.y; hx[p][s][2] = a4.z; hx[p][s][3] = a4.w;
          hx[p][s][4] = b4.x; hx[p][s][5] = b4.y; hx[p][s][6] = b4.z; hx[p][s][7] = b4.w;
        }
        if (hasdk && kr < K) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            rx[p][s][e] = Rp[(unsigned)((c + e) * K + kr)];
            ix[p][s][e] = Ip[(unsigned)((c + e) * K + kr)];
          }
        }
      }
  };
  float4 wr = make_float4(0, 0, 0, 0);
  auto fetch_wr = [&](int blk) {
    if (hasv) wr = *(const float4*)(A.w_r + (long)(hb + blk / CB) * V + (blk % CB) * VB + 16 * mv + 4 * g);
  };
  const bool tabler = w == NW - 1 && blocks > 0;
  if (tabler) fetch_a(hb);
  {
    SsmPieces<BF16, L, KP, NTH> pk;
    const long off = row0 * krow + (long)grp * K;
    pk.load(BF16 ? (const void*)((const uint16_t*)A.k + off) : (const void*)((const float*)A.k + off), krow, K, rows,
            tid);
    fetch_q();
    if (blocks > 0) fetch(0);
    if (ONE) {  // in flight until the products take them
      fetch_RT(0);
      fetch_HR(0);
      fetch_wr(0);
    }
    if (tabler) tables(tabs[0]);
    pk.store(sk, tid);
    pq.store(sq, tid);
    if (ONE) {
      pv.store(sv, tid);
      pu.store(su, tid);
    }
  }
  __syncthreads();
  // q k^T of this wave's row and column tiles, and q of its entering terms' rows: the same for all heads
  f32x4 qkr[NI], qkc[NI];
#pragma unroll
  for (int J = 0; J < NI; ++J) {
    qkr[J] = f32x4{0, 0, 0, 0};
    if (hasI && J <= It) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint4 ko[NP], qo[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          ko[i] = lds_row(sk + i * L * STK, STK, 16 * J, 32 * s, g, n);
          qo[i] = lds_row(sq + i * L * STK, STK, 16 * It, 32 * s, g, n);
        }
        qkr[J] = mfma_planes<NP, NP>(ko, qo, qkr[J]);
      }
    }
  }
#pragma unroll
  for (int I = 0; I < NI; ++I) {
    qkc[I] = f32x4{0, 0, 0, 0};
    if (hasJ && I >= Jt) {
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint4 ko[NP], qo[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          ko[i] = lds_row(sk + i * L * STK, STK, 16 * Jt, 32 * s, g, n);
          qo[i] = lds_row(sq + i * L * STK, STK, 16 * I, 32 * s, g, n);
        }
        qkc[I] = mfma_planes_turned<NP, NP>(qo, ko, qkc[I]);
      }
    }
  }
  uint2 qv[MPW][NI][NP];
#pragma unroll
  for (int p = 0; p < MPW; ++p)
#pragma unroll
    for (int I = 0; I < NI; ++I)
#pragma unroll
      for (int i = 0; i < NP; ++i)
        qv[p][I][i] = *(const uint2*)(sq + i * L * STK + (16 * I + n) * STK + 16 * ((hasdq ? mq : 0) + p) + 4 * g);
  f32x4 xr[NI], xc[NI], dqi[MPW][NI], dki[MPW][NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    xr[i] = xc[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < MPW; ++p) dqi[p][i] = dki[p][i] = f32x4{0, 0, 0, 0};
  }
  // wave 0, lane t: what g and dD hold of the head's column blocks done so far
  double gsum = 0.0, dsum = 0.0;

  // da, and the partial sums of dalpha, dbeta and dw_r, of a block whose products are done
  auto finish = [&](int blk) {
    const int head = hb + blk / CB, cb = blk % CB;
    const SsmTabBwd<L>& tab = tabs[(blk / CB) & 1];
    if (w == 0) {
      const int t = lane;
      double row = 0.0, col = 0.0, diag = 0.0, aa = 0.0, bb = 0.0, through = 0.0, delta64 = 0.0;
      if (t < L) {
        row = rowp[t];
        col = colp[t];
        diag = dgp[t];
        delta64 = tab.d[t];
#pragma unroll
        for (int m = 0; m < KM; ++m) {
          aa += ap[m][t];
          bb += bp[m][t];
        }
      }
#pragma unroll
      for (int m = 0; m < KM; ++m) through += rh[m];
      through *= tab.e[L - 1];
      const double x = row - delta64 * (col - diag) + aa, y = delta64 * bb;
      // sum over i >= t of x, sum over j < t of y, each without a subtraction that would leave a residue
      const double sx64 = __shfl(prefix64(__shfl(x, 63 - lane)), 63 - lane);
      gsum += sx64 + prefix64(dpp64<0x138, 0xF>(y)) + through;
      dsum += col + bb;
      if (cb == CB - 1) {
        const double da = live ? (dsum - (double)A.alpha[head] * gsum) * (double)tab.s[t] : 0.0;
        if (t < L && t0 + t < T) A.da[(row0 + t) * N + head] = (float)da;
        const double sb = prefix64(da), sa = prefix64(live ? -delta64 * gsum : 0.0);
        if (lane == 63) {
          double* o = A.part_gate + ((long)b * A.nch + ch) * 2 * N;
          o[head] = sb;
          o[N + head] = sa;
        }
        gsum = dsum = 0.0;
      }
    } else if (w == 1 && lane < VB) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NI; ++i) sum += (double)dwp[i][lane];
      A.part_wr[((long)b * A.nch + ch) * vrow + (long)head * V + cb * VB + lane] = (float)sum;
    }
  };

  for (int blk = 0; blk < blocks; ++blk) {
    const int head = hb + blk / CB, cb = blk % CB;
    const long pair = (long)b * N + head;
    const SsmTabBwd<L>& tab = tabs[(blk / CB) & 1];
    if (!ONE) {
      __syncthreads();  // the previous block's reads are done
      g = fresh(g);
      n = fresh(n);
      tid = fresh(tid);
      pv.store(sv, tid);
      pu.store(su, tid);
      __syncthreads();
      It = fresh_s(It);
      Jt = fresh_s(Jt);
      if (AHEAD && blk + 1 < blocks) fetch(blk + 1);
      fetch_wr(blk);
      if (tabler && cb == CB - 1 && blk + 1 < blocks) fetch_a(head + 1);
    }

    // rows It: X and the row sums of M
    if (hasI) {
      uint4 uo[VS][3];
#pragma unroll
      for (int s = 0; s < VS; ++s)
#pragma unroll
        for (int i = 0; i < 3; ++i) uo[s][i] = lds_row(su + i * L * STV, STV, 16 * It, 32 * s, g, n);
      double row = 0.0;
#pragma unroll
      for (int J = 0; J < NI; ++J) {
        if (J > It) continue;
        f32x4 uv = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < VS; ++s) {
          uint4 vo[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) vo[i] = lds_row(sv + i * L * STV, STV, 16 * J, 32 * s, g, n);
          uv = mfma_planes<NP, 3>(vo, uo[s], uv);
        }
        float d[4];
        ssm_decay<L, false>(tab, It, J, g, n, d);
        const float4 dj = *(const float4*)&tab.d[16 * J + 4 * g];
        const float dl[4] = {dj.x, dj.y, dj.z, dj.w};
        float m[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x0 = uv[r] * d[r];
          m[r] = x0 * qkr[J][r];
          xr[J][r] = __builtin_fmaf(x0, dl[r], xr[J][r]);
        }
        if (It == J) {  // the diagonal apart
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (4 * g + r == n) {
              dgp[16 * It + n] = m[r];
              m[r] = 0.0f;
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) row = __builtin_fma((double)m[r], (double)dl[r], row);
      }
      row = group_sum64(row);
      if (g == 0) rowp[16 * It + n] = row;
    }
    g = fresh(g);
    n = fresh(n);
    if (ONE) __syncthreads();  // q has been read: P takes its place
    // columns Jt: X, P and the column sums of M
    if (hasJ) {
      uint4 vo[VS][NP];
#pragma unroll
      for (int s = 0; s < VS; ++s)
#pragma unroll
        for (int i = 0; i < NP; ++i) vo[s][i] = lds_row(sv + i * L * STV, STV, 16 * Jt, 32 * s, g, n);
      const float dj = tab.d[16 * Jt + n];
      double col = 0.0;
#pragma unroll
      for (int I = 0; I < NI; ++I) {
        if (I < Jt) continue;
        f32x4 uv = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < VS; ++s) {
          uint4 uo[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) uo[i] = lds_row(su + i * L * STV, STV, 16 * I, 32 * s, g, n);
          uv = mfma_planes_turned<3, NP>(uo, vo[s], uv);
        }
        float d[4], pp[4];
        ssm_decay_col<L>(tab, I, Jt, g, n, d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x0 = uv[r] * d[r], m = x0 * qkc[I][r];
          xc[I][r] = __builtin_fmaf(x0, dj, xc[I][r]);
          pp[r] = qkc[I][r] * d[r];
          col += (double)m;
        }
        uint2 pl[3];
        split3x4(pp, pl);
        const int set = NI == 4 ? (Jt < 2 ? 2 * Jt + I / 2 : Jt + 2) : Jt;
#pragma unroll
        for (int i = 0; i < 3; ++i) pbuf[((set * 3 + i) * 2 + (I & 1)) * 64 + lane] = pl[i];
      }
      col = group_sum64(col);
      if (g == 0) colp[16 * Jt + n] = col;
    }
    __syncthreads();

    if (!ONE) fetch_RT(blk);
    const float dec = exp2_(idec);
    g = fresh(g);
    n = fresh(n);
    if (hasv) {
      // dv^T: rows c of tile mv, columns j
      uint4 Ro[KS][3];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const float x[8] = {
            __builtin_fmaf(dec, tI[s][0].x, tR[s][0].x), __builtin_fmaf(dec, tI[s][0].y, tR[s][0].y),
            __builtin_fmaf(dec, tI[s][0].z, tR[s][0].z), __builtin_fmaf(dec, tI[s][0].w, tR[s][0].w),
            __builtin_fmaf(dec, tI[s][1].x, tR[s][1].x), __builtin_fmaf(dec, tI[s][1].y, tR[s][1].y),
            __builtin_fmaf(dec, tI[s][1].z, tR[s][1].z), __builtin_fmaf(dec, tI[s][1].w, tR[s][1].w)};
        split3x8(x, Ro[s]);
      }
      uint4 uo[NS][3];
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 3; ++i) uo[s][i] = lds_col(su + i * L * STV, STV, 32 * s, 16 * mv, g, n);
#pragma unroll
      for (int p = 0; p < TPV; ++p) {
        const int J = jv0 + p;
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint4 ko[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) ko[i] = lds_row(sk + i * L * STK, STK, 16 * J, 32 * s, g, n);
          acc = mfma_planes<3, NP>(Ro[s], ko, acc);
        }
        const float ej = tab.w[16 * J + n], dj = tab.d[16 * J + n];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] *= ej;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          if (s < J / 2) continue;
          const int set = NI == 4 ? (J < 2 ? 2 * J + s : J + 2) : J;
          uint4 po[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const uint2* pb = &pbuf[((set * 3 + i) * 2) * 64 + lane];
            po[i] = cat(2 * s >= J ? pb[0] : make_uint2(0, 0), pb[64]);
          }
          acc = mfma_planes<3, 3>(uo[s], po, acc);
        }
        float uj[4], vj[4];
        lds_vals4<3>(su + (16 * J + n) * STV + 16 * mv + 4 * g, L * STV, uj);
        lds_vals4<NP>(sv + (16 * J + n) * STV + 16 * mv + 4 * g, L * STV, vj);
        const int t = t0 + 16 * J + n;
        if (t < T)
          *(float4*)(A.dv + ((long)b * T + t) * vrow + (long)head * V + cb * VB + 16 * mv + 4 * g) =
              make_float4(dj * acc[0] + wr.x * uj[0], dj * acc[1] + wr.y * uj[1], dj * acc[2] + wr.z * uj[2],
                          dj * acc[3] + wr.w * uj[3]);
        const float sum = row16_sum4(uj[0] * vj[0], uj[1] * vj[1], uj[2] * vj[2], uj[3] * vj[3], lane);
        if ((n & 3) == 0) dwp[J][16 * mv + 4 * g + (n >> 2)] = sum;
      }
    }
    g = fresh(g);
    n = fresh(n);
    if (!ONE) fetch_HR(blk);
#pragma unroll
    for (int p = 0; p < MPW; ++p) {
      // the terms of H and R: rows kk of this wave's K tiles, columns i (j)
      float y[VS][8];
#pragma unroll
      for (int s = 0; s < VS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[s][e] = __builtin_fmaf(dec, ix[p][s][e], rx[p][s][e]);
      if (hasdk) {
        double dot = 0.0;  // <R, H>: every step of the chunk gets it, so its error would add up in dalpha and dbeta
#pragma unroll
        for (int s = 0; s < VS; ++s)
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = __builtin_fma((double)hx[p][s][e], (double)y[s][e], dot);
        dot = total64(dot);
        if (lane == 0) rh[mk + p] = dot;
        uint4 Ro[VS][3];
#pragma unroll
        for (int s = 0; s < VS; ++s) split3x8(y[s], Ro[s]);
        double part[NI];
#pragma unroll
        for (int J = 0; J < NI; ++J) {
          f32x4 acc = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < VS; ++s) {
            uint4 vo[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) vo[i] = lds_row(sv + i * L * STV, STV, 16 * J, 32 * s, g, n);
            acc = mfma_planes<3, NP>(Ro[s], vo, acc);
          }
          const float ej = tab.w[16 * J + n], dj = tab.d[16 * J + n];
          float dot4 = 0.0f;
          float kv[4];
          lds_vals4<NP>(sk + (16 * J + n) * STK + 16 * (mk + p) + 4 * g, L * STK, kv);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            acc[r] *= ej;
            dot4 = __builtin_fmaf(kv[r], acc[r], dot4);
            dki[p][J][r] = __builtin_fmaf(dj, acc[r], dki[p][J][r]);
          }
          part[J] = dot4;
        }
        put_group_sums<NI>(bp[mk + p], part, g, n);
      }
      if (hasdq) {
        uint4 Ho[VS][3];
#pragma unroll
        for (int s = 0; s < VS; ++s) split3x8(hx[p][s], Ho[s]);
        double part[NI];
#pragma unroll
        for (int I = 0; I < NI; ++I) {
          f32x4 acc = {0, 0, 0, 0};
#pragma unroll
          for (int s = 0; s < VS; ++s) {
            uint4 uo[3];
#pragma unroll
            for (int i = 0; i < 3; ++i) uo[i] = lds_row(su + i * L * STV, STV, 16 * I, 32 * s, g, n);
            acc = mfma_planes<3, 3>(Ho[s], uo, acc);
          }
          const float e = tab.e[16 * I + n];
          float dot4 = 0.0f;
          float qf[4];
          planes_vals4<NP>(qv[p][I], qf);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            acc[r] *= e;
            dot4 = __builtin_fmaf(qf[r], acc[r], dot4);
            dqi[p][I][r] += acc[r];
          }
          part[I] = dot4;
        }
        put_group_sums<NI>(ap[mq + p], part, g, n);
      }
    }
    if (!ONE) {
      if (tabler && cb == CB - 1 && blk + 1 < blocks) tables(tabs[(blk / CB + 1) & 1]);
      if (!AHEAD && blk + 1 < blocks) fetch(blk + 1);
      if (blk + 1 == blocks) fetch_q();
      __syncthreads();
      finish(blk);
    }
  }

  // dq and dk: X of all heads times k and q, by step tiles, plus the terms of H and R, by K tiles, through LDS
  if (ONE || blocks == 0) {
    if (!ONE) fetch_q();
    __syncthreads();
  }
  pq.store(sq, tid);
  float* const ex = (float*)su;  // [L][KP]
  const long plane = (long)hs * A.B * T * krow;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which ? hasdk : hasdq) {
#pragma unroll
      for (int p = 0; p < MPW; ++p)
#pragma unroll
        for (int I = 0; I < NI; ++I) {
          const f32x4& t = which ? dki[p][I] : dqi[p][I];
          *(float4*)(ex + (16 * I + n) * KP + 16 * ((which ? mk : mq) + p) + 4 * g) = make_float4(t[0], t[1], t[2], t[3]);
        }
    }
    __syncthreads();
    if (which ? hasJ : hasI) {
      const int own = which ? Jt : It;
      uint4 xo[NS][3];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        uint2 h0[3], h1[3];
        const f32x4 &a4 = which ? xc[2 * s] : xr[2 * s], &b4 = which ? xc[2 * s + 1] : xr[2 * s + 1];
        const float av[4] = {a4[0], a4[1], a4[2], a4[3]}, bv[4] = {b4[0], b4[1], b4[2], b4[3]};
        split3x4(av, h0);
        split3x4(bv, h1);
#pragma unroll
        for (int i = 0; i < 3; ++i) xo[s][i] = cat(h0[i], h1[i]);
      }
      float* out = (which ? A.dk : A.dq) + plane;
      const int t = t0 + 16 * own + n;
#pragma unroll
      for (int m = 0; m < KM; ++m) {
        const float4 t4 = *(const float4*)(ex + (16 * own + n) * KP + 16 * m + 4 * g);
        f32x4 acc = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          uint4 ko[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) ko[i] = lds_col((which ? sq : sk) + i * L * STK, STK, 32 * s, 16 * m, g, n);
          acc = mfma_planes<NP, 3>(ko, xo[s], acc);
        }
        const int kk = 16 * m + 4 * g;
        if (t < T && kk < K)
          *(float4*)(out + ((long)b * T + t) * krow + (long)grp * K + kk) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      }
    }
    if (which == 0) __syncthreads();
  }
  if (ONE) finish(0);
}

// ------------------------------------------------------------------ backward of narrow heads

// The operand with 16 contraction slots (four values a lane): products over the 16 value columns.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma16_planes(const uint2 (&A)[NA], const uint2 (&B)[NB], f32x4 acc) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = s - i;
      if (j >= 0 && j < NB) acc = mfma16_bf16(A[i], B[j], acc);
    }
  return acc;
}
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma16_planes_turned(const uint2 (&A)[NA], const uint2 (&B)[NB], f32x4 acc) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int i = s - j;
      if (i >= 0 && i < NA) acc = mfma16_bf16(A[i], B[j], acc);
    }
  return acc;
}

// The backward of one chunk for heads of 16 value columns (mathematics: m2rnn_ssm_bwd_kernel above), which
// usually share a query/key: the walk over the heads is what counts, so everything in it runs one
// head ahead.  A wave owns the same 16 steps as rows and as columns; with 16 value columns it forms
// its dv tile from its own P, so nothing is exchanged within a head: v, dy and R of the next head
// go to the other half of a double buffer while this one is computed, one barrier a head.  Meanwhile wave 3
// forms the next head's decay tables and wave 0 finishes the previous head's da, so waves 1 and 2 do
// the staging (all four staging: 14.1 thousand cycles a head, of which waves 1 and 2 waited 2.6; every other
// assignment of the three tasks took 14 to 40 us more).  R is read once, as planes in LDS that serve as R (transposing reads) and as R^T; H goes straight into the
// operand of the wave that owns its 16 K rows.  X is summed over the heads in registers.
//
// B4 N128 T4096 K=64 V=16, one query/key: 346 to 405 us, 367 on average, 11.6 thousand cycles a head for the two
// workgroups of a CU.
// Bound by issue and latency at two waves a SIMD (256 VGPRs): VALU 58%, MFMA 18%, LDS 38% of the cycles, HBM at
// 2.4 TB/s.  Of an earlier 366 us the columns with P and dv took a third, the terms of H and R 47 us, the rows 33, loads 27,
// da 25, the tables 8, the fp64 sums 9.
template <bool BF16, int KP>
__global__ void __launch_bounds__(64 * kSsmBwdWaves, KP == 128 ? 1 : 2) m2rnn_ssm_bwd_narrow_kernel(SsmArgs A) {
  constexpr int L = ssm_chunk<BF16>(), NI = L / 16, NS = L / 32, KS = KP / 32, KM = KP / 16, NP = BF16 ? 1 : 3;
  constexpr int NW = kSsmBwdWaves, NTH = 64 * NW, V = 16;
  constexpr int STK = ssm_stride(KP), STV = ssm_stride(V), STR = ssm_stride(KP);
  constexpr int MPW = KM >= NW ? KM / NW : 1;
  constexpr int NST = NTH / 2;                                       // threads that stage: waves 1 and 2
  constexpr int RP = (V * KP / 4 + NST - 1) / NST;                   // pieces of R (4 values) per thread
  constexpr int OV = 0, OU = NP * L * STV, OR = OU + 3 * L * STV, BUF = OR + 3 * V * STR;  // one buffer, in elements
  constexpr int POOL = 2 * BUF * 2 > L * KP * 4 ? 2 * BUF : L * KP * 2;
  struct Small {
    double row[L], col[L], a[KM][L], b[L], rh[KM][64];
    float dg[L], dw[NI][V];
  };
  __shared__ __attribute__((aligned(16))) uint16_t sk[NP * L * STK];
  __shared__ __attribute__((aligned(16))) uint16_t sq[NP * L * STK];
  __shared__ __attribute__((aligned(16))) uint16_t pool[POOL];  // the double buffer; at the end the exchange of dq, dk
  __shared__ __attribute__((aligned(16))) SsmTabBwd<L> tabs[3];
  __shared__ Small small[2];

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  int unit, hs;
  ssm_unit(A.HS, A.B * A.G * A.nch, unit, hs);
  const int ch = unit % A.nch, bg = unit / A.nch;
  const int b = bg / A.G, grp = bg % A.G;
  const int K = A.K, T = A.T, N = A.N;
  // this workgroup's heads: every HS-th of the group's, so that the workgroups of a chunk, which run side by side on
  // one XCD, take the parts of a line of v, dy and dv (32 and 64 bytes a head) at about the same time (two runs of 64
  // heads instead: 570 us for the training step of 128 heads, not 557)
  const int hpg = N / A.G, heads = (hpg - hs + A.HS - 1) / A.HS;
  auto head_of = [&](int it) { return grp * hpg + hs + it * A.HS; };
  const int t0 = ch * L;
  const int Tb = ssm_len(A, b);
  const int rows = min(L, Tb - t0);
  const long krow = (long)A.G * K, vrow = (long)N * V, row0 = (long)b * T + t0;
  const int It = w, Jt = NI == 4 ? w : w - 2;
  const bool hasI = It < NI, hasJ = Jt >= 0;
  const bool hasdq = KM >= NW || w < KM, hasdk = KM >= NW || w >= NW - KM;
  const int mq = KM >= NW ? w * MPW : w, mk = KM >= NW ? w * MPW : w - (NW - KM);
  const int mh = hasdq ? mq : mk;  // the K tiles whose H this wave reads

  const bool stager = w == 1 || w == 2;
  const int sid = tid - 64;
  SsmPieces<BF16, L, V, NST> pv;
  SsmPieces<false, L, V, NST> pu;
  float4 pr[RP], pi[RP];
  float idec;
  auto fetch = [&](int it) {  // v, dy, R of a head
    if (!stager) return;
    const int h = head_of(it);
    const long off = row0 * vrow + (long)h * V;
    pv.load(BF16 ? (const void*)((const uint16_t*)A.v + off) : (const void*)((const float*)A.v + off), vrow, V, rows, sid);
    pu.load(A.dy + off, vrow, V, rows, sid);
    const long pair = (long)b * N + h;
    const float* Rp = A.rloc + (pair * A.nch + ch) * V * K;        // [V][K]
    const float* Ip = A.seg + (pair * A.S + ch / A.cps) * V * K;   // [V][K]
    idec = A.cdec[pair * A.nch + ch];
#pragma unroll
    for (int p = 0; p < RP; ++p) {
      const int i = sid + p * NST, c = i / (KP / 4), kk = (i % (KP / 4)) * 4;
      pr[p] = pi[p] = make_float4(0, 0, 0, 0);
      if (c < V && kk < K) {
        pr[p] = *(const float4*)(Rp + (unsigned)(c * K + kk));
        pi[p] = *(const float4*)(Ip + (unsigned)(c * K + kk));
      }
    }
  };
  auto stage = [&](uint16_t* buf) {
    if (!stager) return;
    pv.store(buf + OV, sid);
    pu.store(buf + OU, sid);
    const float d = exp2_(idec);
#pragma unroll
    for (int p = 0; p < RP; ++p) {
      const int i = sid + p * NST, c = i / (KP / 4), kk = (i % (KP / 4)) * 4;
      if (c < V) {
        const float x[4] = {__builtin_fmaf(d, pi[p].x, pr[p].x), __builtin_fmaf(d, pi[p].y, pr[p].y),
                            __builtin_fmaf(d, pi[p].z, pr[p].z), __builtin_fmaf(d, pi[p].w, pr[p].w)};
        uint2 pl[3];
        split3x4(x, pl);
#pragma unroll
        for (int q = 0; q < 3; ++q) *(uint2*)(buf + OR + (q * V + c) * STR + kk) = pl[q];
      }
    }
  };
  float4 ph[MPW], wr;
  auto fetch_H = [&](int it) {
    const int h = head_of(it);
    wr = *(const float4*)(A.w_r + (long)h * V + 4 * g);
    const float* Hp = A.ckpt + (((long)b * N + h) * A.nch + ch) * K * V;  // [K][V]
#pragma unroll
    for (int p = 0; p < MPW; ++p) {
      const int kk = 16 * (mh + p) + n;
      ph[p] = make_float4(0, 0, 0, 0);
      if (kk < K) ph[p] = *(const float4*)(Hp + (unsigned)(kk * V + 4 * g));
    }
  };
  const bool live = lane < L && t0 + lane < Tb;
  float pa = 0.0f;
  auto fetch_a = [&](int it) { pa = live ? A.a[(row0 + lane) * N + head_of(it)] : 0.0f; };
  auto tables = [&](int it) {
    const int h = head_of(it);
    float delta, sigma;
    double lg;
    SsmTabBwd<L>& tab = tabs[it % 3];
    ssm_gate(live, pa, A.alpha[h], A.beta[h], delta, sigma, lg);
    ssm_tables<L, false>(tab, lane, delta, lg);
    if (lane < L) tab.s[lane] = sigma;
  };
  // da, and the partial sums of dalpha, dbeta and dw_r, of a head whose products are done
  auto finish = [&](int it) {
    const int h = head_of(it);
    const Small& sm = small[it & 1];
    const SsmTabBwd<L>& tab = tabs[it % 3];
    double row = 0.0, col = 0.0, diag = 0.0, aa = 0.0, bb = 0.0, through = 0.0;
    float delta = 0.0f;
    if (lane < L) {
      row = sm.row[lane];
      col = sm.col[lane];
      diag = sm.dg[lane];
      delta = tab.d[lane];
      bb = sm.b[lane];
#pragma unroll
      for (int m = 0; m < KM; ++m) aa += sm.a[m][lane];
    }
    // <R, H>, a term of every g_t, as 64 parts: lane l's part reaches the steps up to l with x and those past l with y
#pragma unroll
    for (int m = 0; m < KM; ++m) through += sm.rh[m][lane];
    through *= tab.e[L - 1];
    const double x = row - (double)delta * (col - diag) + aa + through, y = (double)delta * bb + through;
    const double gs = __shfl(prefix64(__shfl(x, 63 - lane)), 63 - lane) + prefix64(dpp64<0x138, 0xF>(y));
    const double da = live ? (col + bb - (double)A.alpha[h] * gs) * (double)tab.s[lane] : 0.0;
    if (lane < L && t0 + lane < T) A.da[(row0 + lane) * N + h] = (float)da;
    const double sb = prefix64(da), sa = prefix64(live ? -(double)delta * gs : 0.0);
    if (lane == 63) {
      double* o = A.part_gate + ((long)b * A.nch + ch) * 2 * N;
      o[h] = sb;
      o[N + h] = sa;
    }
    if (lane < V) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NI; ++i) sum += (double)sm.dw[i][lane];
      A.part_wr[((long)b * A.nch + ch) * vrow + (long)h * V + lane] = (float)sum;
    }
  };

  fetch(0);
  if (w == NW - 1) fetch_a(0);
  {
    SsmPieces<BF16, L, KP, NTH> pq, pk;
    const long off = row0 * krow + (long)grp * K;
    pk.load(BF16 ? (const void*)((const uint16_t*)A.k + off) : (const void*)((const float*)A.k + off), krow, K, rows, tid);
    pq.load(BF16 ? (const void*)((const uint16_t*)A.q + off) : (const void*)((const float*)A.q + off), krow, K, rows, tid);
    pk.store(sk, tid);
    pq.store(sq, tid);
  }
  if (w == NW - 1) {
    tables(0);
    if (1 < heads) fetch_a(1);
  }
  stage(pool);
  fetch_H(0);
  if (1 < heads) fetch(1);
  __syncthreads();
  // q k^T of this wave's row and column tiles: the same for all heads
  f32x4 qkr[NI], qkc[NI], xr[NI], xc[NI], dqi[MPW][NI], dki[MPW][NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    qkr[i] = qkc[i] = xr[i] = xc[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < MPW; ++p) dqi[p][i] = dki[p][i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      uint4 ko[NP], qo[NP];
      if (hasI && i <= It) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          ko[p] = lds_row(sk + p * L * STK, STK, 16 * i, 32 * s, g, n);
          qo[p] = lds_row(sq + p * L * STK, STK, 16 * It, 32 * s, g, n);
        }
        qkr[i] = mfma_planes<NP, NP>(ko, qo, qkr[i]);
      }
      if (hasJ && i >= Jt) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          ko[p] = lds_row(sk + p * L * STK, STK, 16 * Jt, 32 * s, g, n);
          qo[p] = lds_row(sq + p * L * STK, STK, 16 * i, 32 * s, g, n);
        }
        qkc[i] = mfma_planes_turned<NP, NP>(qo, ko, qkc[i]);
      }
    }
  }

  for (int it = 0; it < heads; ++it) {
    const int h = head_of(it);
    const SsmTabBwd<L>& tab = tabs[it % 3];
    Small& sm = small[it & 1];
    uint16_t* const buf = pool + (it & 1) * BUF;
    const uint16_t *sv = buf + OV, *su = buf + OU, *sr = buf + OR;
    const int n = fresh(lane & 15), g = fresh(lane >> 4);  // (addresses formed per head, not held across them)
    const int It = fresh_s(w), Jt = fresh_s(NI == 4 ? w : w - 2);
    if (w == 0 && it > 0) finish(it - 1);

    // rows It: X and the row sums of M
    if (hasI) {
      uint2 uo[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) uo[i] = *(const uint2*)(su + (i * L + 16 * It + n) * STV + 4 * g);
      double row = 0.0;
#pragma unroll
      for (int J = 0; J < NI; ++J) {
        if (J > It) continue;
        uint2 vo[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) vo[i] = *(const uint2*)(sv + (i * L + 16 * J + n) * STV + 4 * g);
        const f32x4 uv = mfma16_planes<NP, 3>(vo, uo, f32x4{0, 0, 0, 0});
        float d[4];
        ssm_decay<L, false>(tab, It, J, g, n, d);
        const float4 dj = *(const float4*)&tab.d[16 * J + 4 * g];
        const float dl[4] = {dj.x, dj.y, dj.z, dj.w};
        float m[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x0 = uv[r] * d[r];
          m[r] = x0 * qkr[J][r];
          xr[J][r] = __builtin_fmaf(x0, dl[r], xr[J][r]);
        }
        if (It == J) {  // the diagonal apart
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (4 * g + r == n) {
              sm.dg[16 * It + n] = m[r];
              m[r] = 0.0f;
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) row = __builtin_fma((double)m[r], (double)dl[r], row);
      }
      row = group_sum64(row);
      if (g == 0) sm.row[16 * It + n] = row;
    }
    // columns Jt: X, P and the column sums of M, and dv
    if (hasJ) {
      uint2 vo[NP], pl[NI][3];
#pragma unroll
      for (int i = 0; i < NP; ++i) vo[i] = *(const uint2*)(sv + (i * L + 16 * Jt + n) * STV + 4 * g);
      const float dj = tab.d[16 * Jt + n];
      double col = 0.0;
#pragma unroll
      for (int I = 0; I < NI; ++I) {
#pragma unroll
        for (int i = 0; i < 3; ++i) pl[I][i] = make_uint2(0, 0);
        if (I < Jt) continue;
        uint2 uo[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) uo[i] = *(const uint2*)(su + (i * L + 16 * I + n) * STV + 4 * g);
        const f32x4 uv = mfma16_planes_turned<3, NP>(uo, vo, f32x4{0, 0, 0, 0});
        float d[4], pp[4];
        ssm_decay_col<L>(tab, I, Jt, g, n, d);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x0 = uv[r] * d[r], m = x0 * qkc[I][r];
          xc[I][r] = __builtin_fmaf(x0, dj, xc[I][r]);
          pp[r] = qkc[I][r] * d[r];
          col += (double)m;
        }
        split3x4(pp, pl[I]);
      }
      col = group_sum64(col);
      if (g == 0) sm.col[16 * Jt + n] = col;
      // dv^T: the value columns, steps Jt
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint4 ko[NP], ro[3];
#pragma unroll
        for (int i = 0; i < NP; ++i) ko[i] = lds_row(sk + i * L * STK, STK, 16 * Jt, 32 * s, g, n);
#pragma unroll
        for (int i = 0; i < 3; ++i) ro[i] = lds_row(sr + i * V * STR, STR, 0, 32 * s, g, n);
        acc = mfma_planes<3, NP>(ro, ko, acc);
      }
      const float ej = tab.w[16 * Jt + n];
      float uj[4], vj[4];
      lds_vals4<3>(su + (16 * Jt + n) * STV + 4 * g, L * STV, uj);
      lds_vals4<NP>(sv + (16 * Jt + n) * STV + 4 * g, L * STV, vj);
      // k_j . R v_j as v_j . R^T k_j, whose right side is here
      float bj = 0.0f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        acc[r] *= ej;
        bj = __builtin_fmaf(acc[r], vj[r], bj);
      }
      const double bs = group_sum64((double)bj);
      if (g == 0) sm.b[16 * Jt + n] = bs;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        if (2 * s + 1 < Jt) continue;
        uint4 uo[3], po[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          uo[i] = lds_col(su + i * L * STV, STV, 32 * s, 0, g, n);
          po[i] = cat(pl[2 * s][i], pl[2 * s + 1][i]);
        }
        acc = mfma_planes<3, 3>(uo, po, acc);
      }
      const int t = t0 + 16 * Jt + n;
      if (t < T)
        *(float4*)(A.dv + ((long)b * T + t) * vrow + (long)h * V + 4 * g) =
            make_float4(dj * acc[0] + wr.x * uj[0], dj * acc[1] + wr.y * uj[1], dj * acc[2] + wr.z * uj[2],
                        dj * acc[3] + wr.w * uj[3]);
      const float sum = row16_sum4(uj[0] * vj[0], uj[1] * vj[1], uj[2] * vj[2], uj[3] * vj[3], lane);
      if ((n & 3) == 0) sm.dw[Jt][4 * g + (n >> 2)] = sum;
    }
    // the terms of H and R: rows kk of this wave's K tiles, columns i (j)
#pragma unroll
    for (int p = 0; p < MPW; ++p) {
      const float hx[4] = {ph[p].x, ph[p].y, ph[p].z, ph[p].w};
      if (hasdk) {
        uint2 ro[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) ro[i] = lds_col16(sr + i * V * STR, STR, 0, 16 * (mk + p), g, n);
        float rx[4];
        planes_vals4<3>(ro, rx);
        double dot = 0.0;  // <R, H>: every step of the chunk gets it, so its error would add up in dalpha and dbeta
#pragma unroll
        for (int e = 0; e < 4; ++e) dot = __builtin_fma((double)hx[e], (double)rx[e], dot);
        sm.rh[mk + p][lane] = dot;
#pragma unroll
        for (int J = 0; J < NI; ++J) {
          uint2 vo[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) vo[i] = *(const uint2*)(sv + (i * L + 16 * J + n) * STV + 4 * g);
          const f32x4 acc = mfma16_planes<3, NP>(ro, vo, f32x4{0, 0, 0, 0});
          const float ed = tab.w[16 * J + n] * tab.d[16 * J + n];
#pragma unroll
          for (int r = 0; r < 4; ++r) dki[p][J][r] = __builtin_fmaf(ed, acc[r], dki[p][J][r]);
        }
      }
      if (hasdq) {
        uint2 ho[3];
        split3x4(hx, ho);
        double part[NI];
#pragma unroll
        for (int I = 0; I < NI; ++I) {
          uint2 uo[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) uo[i] = *(const uint2*)(su + (i * L + 16 * I + n) * STV + 4 * g);
          const f32x4 acc = mfma16_planes<3, 3>(ho, uo, f32x4{0, 0, 0, 0});
          const float e = tab.e[16 * I + n];
          float qf[4], dot4 = 0.0f;
          lds_vals4<NP>(sq + (16 * I + n) * STK + 16 * (mq + p) + 4 * g, L * STK, qf);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            dot4 = __builtin_fmaf(qf[r], acc[r], dot4);
            dqi[p][I][r] = __builtin_fmaf(e, acc[r], dqi[p][I][r]);
          }
          part[I] = e * dot4;
        }
        put_group_sums<NI>(sm.a[mq + p], part, g, n);
      }
    }
    if (it + 1 < heads) {
      if (w == NW - 1) {
        tables(it + 1);
        if (it + 2 < heads) fetch_a(it + 2);
      }
      stage(pool + ((it + 1) & 1) * BUF);
      fetch_H(it + 1);
      if (it + 2 < heads) fetch(it + 2);
    }
    __syncthreads();
  }
  if (w == 0) finish(heads - 1);

  // dq and dk: X of all heads times k and q, by step tiles, plus the terms of H and R, by K tiles, through LDS
  float* const ex = (float*)pool;  // [L][KP]
  const long plane = (long)hs * A.B * T * krow;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which ? hasdk : hasdq) {
#pragma unroll
      for (int p = 0; p < MPW; ++p)
#pragma unroll
        for (int I = 0; I < NI; ++I) {
          const f32x4& t = which ? dki[p][I] : dqi[p][I];
          *(float4*)(ex + (16 * I + n) * KP + 16 * ((which ? mk : mq) + p) + 4 * g) = make_float4(t[0], t[1], t[2], t[3]);
        }
    }
    __syncthreads();
    if (which ? hasJ : hasI) {
      const int own = which ? Jt : It;
      uint4 xo[NS][3];
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const f32x4 &a4 = which ? xc[2 * s] : xr[2 * s], &b4 = which ? xc[2 * s + 1] : xr[2 * s + 1];
        const float x8[8] = {a4[0], a4[1], a4[2], a4[3], b4[0], b4[1], b4[2], b4[3]};
        split3x8(x8, xo[s]);
      }
      float* out = (which ? A.dk : A.dq) + plane;
      const int t = t0 + 16 * own + n;
#pragma unroll
      for (int m = 0; m < KM; ++m) {
        const float4 t4 = *(const float4*)(ex + (16 * own + n) * KP + 16 * m + 4 * g);
        f32x4 acc = {t4.x, t4.y, t4.z, t4.w};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          uint4 ko[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) ko[i] = lds_col((which ? sq : sk) + i * L * STK, STK, 32 * s, 16 * m, g, n);
          acc = mfma_planes<NP, 3>(ko, xo[s], acc);
        }
        const int kk = 16 * m + 4 * g;
        if (t < T && kk < K)
          *(float4*)(out + ((long)b * T + t) * krow + (long)grp * K + kk) = make_float4(acc[0], acc[1], acc[2], acc[3]);
      }
    }
    if (which == 0) __syncthreads();
  }
}

// ------------------------------------------------------------------ one token

// One step for every (b, n), the state in HBM: reads it, advances it and writes it back, in place or
// not (a thread reads its own elements before it writes them).  One workgroup per pair; a thread owns four
// columns of every (256 / (V / 4))-th row, so a wave's accesses are whole rows, and the readout's sum over
// rows ends in LDS.  Bound by HBM: 128 sequences of 32 heads at K = V = 64 take 23 to 24 us (5.7 to 6.0 TB/s
// of state read and written); one sequence of 128 heads takes 4 us, a launch and two trips to memory.
template <bool BF16, int V>
__global__ void __launch_bounds__(256) m2rnn_ssm_step_kernel(const void* q, const void* k, const void* v,
                                                             const float* a, const float* alpha, const float* beta,
                                                             const float* w_r, const float* H_in, float* H_out,
                                                             float* y, int N, int G, int K) {
  constexpr int VQ = V / 4, RP = 256 / VQ;  // column groups; rows per pass
  __shared__ __attribute__((aligned(16))) float red[4][V];
  const int tid = threadIdx.x, w = tid >> 6;
  const long pair = blockIdx.x;
  const int head = (int)(pair % N);
  const long qk = (pair / N * G + head / (N / G)) * K;
  const int c = (tid % VQ) * 4;
  const int r0 = tid / VQ;
  float delta, sigma;
  double lg;
  ssm_gate(true, a[pair], alpha[head], beta[head], delta, sigma, lg);
  const float f = exp2_((float)lg);
  auto val = [](const void* p, long i) {
    if constexpr (BF16) return bf16_lo_to_f32(((const uint16_t*)p)[i]);
    return ((const float*)p)[i];
  };
  float4 vv;
  if constexpr (BF16) {
    const uint2 u = *(const uint2*)((const uint16_t*)v + pair * V + c);
    vv = make_float4(bf16_lo_to_f32(u.x), bf16_hi_to_f32(u.x), bf16_lo_to_f32(u.y), bf16_hi_to_f32(u.y));
  } else {
    vv = *(const float4*)((const float*)v + pair * V + c);
  }
  const float4 dv = make_float4(delta * vv.x, delta * vv.y, delta * vv.z, delta * vv.w);
  const float* hi = H_in ? H_in + pair * K * V + c : nullptr;
  float* ho = H_out + pair * K * V + c;
  float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll 4
  for (int r = r0; r < K; r += RP) {
    float4 h = hi ? *(const float4*)(hi + (long)r * V) : make_float4(0, 0, 0, 0);
    const float kr = val(k, qk + r), qr = val(q, qk + r);
    h.x = __builtin_fmaf(kr, dv.x, f * h.x);
    h.y = __builtin_fmaf(kr, dv.y, f * h.y);
    h.z = __builtin_fmaf(kr, dv.z, f * h.z);
    h.w = __builtin_fmaf(kr, dv.w, f * h.w);
    *(float4*)(ho + (long)r * V) = h;
    acc.x = __builtin_fmaf(qr, h.x, acc.x);
    acc.y = __builtin_fmaf(qr, h.y, acc.y);
    acc.z = __builtin_fmaf(qr, h.z, acc.z);
    acc.w = __builtin_fmaf(qr, h.w, acc.w);
  }
#pragma unroll
  for (int o = VQ; o < 64; o <<= 1) {
    acc.x += __shfl_xor(acc.x, o);
    acc.y += __shfl_xor(acc.y, o);
    acc.z += __shfl_xor(acc.z, o);
    acc.w += __shfl_xor(acc.w, o);
  }
  if ((tid & 63) < VQ) *(float4*)&red[w][(tid & 63) * 4] = acc;
  __syncthreads();
  if (tid < V)
    y[pair * V + tid] =
        ((red[0][tid] + red[1][tid]) + (red[2][tid] + red[3][tid])) + w_r[(long)head * V + tid] * val(v, pair * V + tid);
}

}  // namespace m2rnn
