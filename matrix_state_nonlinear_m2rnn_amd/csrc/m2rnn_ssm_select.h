// Kernel selection for the selective state space scan: the kernels of each input type are compiled in
// translation units of their own, which export functions mapping the padded key size (32, 64 or
// 128) and the value block to the kernel's host stub.
#pragma once

#include "m2rnn_ssm_kernels.h"

namespace m2rnn {

enum { SSM_FWD = 0, SSM_STATE = 1, SSM_STATE_REV = 2 };

template <bool BF16, int KP, int VB, int HPW>
const void* ssm_pick_kvh(int which) {
  switch (which) {
    case SSM_FWD: return (const void*)&m2rnn_ssm_fwd_kernel<BF16, KP, VB, HPW>;
    case SSM_STATE: return (const void*)&m2rnn_ssm_state_kernel<BF16, KP, VB, HPW, false>;
    default: return (const void*)&m2rnn_ssm_state_kernel<BF16, KP, VB, HPW, true>;
  }
}
template <bool BF16, int KP>
const void* ssm_pick_k(int VB, int HPW, int which) {
  if (VB == 16) return HPW == 4 ? ssm_pick_kvh<BF16, KP, 16, 4>(which) : ssm_pick_kvh<BF16, KP, 16, 1>(which);
  if (VB == 32) return ssm_pick_kvh<BF16, KP, 32, 1>(which);
  return ssm_pick_kvh<BF16, KP, 64, 1>(which);
}
template <bool BF16>
const void* ssm_pick(int KP, int VB, int HPW, int which) {
  if (KP == 32) return ssm_pick_k<BF16, 32>(VB, HPW, which);
  if (KP == 64) return ssm_pick_k<BF16, 64>(VB, HPW, which);
  return ssm_pick_k<BF16, 128>(VB, HPW, which);
}
template <bool BF16, int KP, int VB>
const void* ssm_pick_bwd_kv(bool one) {
  return one ? (const void*)&m2rnn_ssm_bwd_kernel<BF16, KP, VB, true>
             : (const void*)&m2rnn_ssm_bwd_kernel<BF16, KP, VB, false>;
}
template <bool BF16, int KP>
const void* ssm_pick_bwd_k(int VB, bool one) {
  if (VB == 16) return (const void*)&m2rnn_ssm_bwd_narrow_kernel<BF16, KP>;
  if (VB == 32) return ssm_pick_bwd_kv<BF16, KP, 32>(one);
  return ssm_pick_bwd_kv<BF16, KP, 64>(one);
}
template <bool BF16>
const void* ssm_pick_bwd(int KP, int VB, bool one) {
  if (KP == 32) return ssm_pick_bwd_k<BF16, 32>(VB, one);
  if (KP == 64) return ssm_pick_bwd_k<BF16, 64>(VB, one);
  return ssm_pick_bwd_k<BF16, 128>(VB, one);
}

// Defined in m2rnn_ssm_<bf16|f32>.hip and m2rnn_ssm_bwd_<bf16|f32>.hip.
const void* ssm_kernel_bf16(int KP, int VB, int HPW, int which);
const void* ssm_kernel_f32(int KP, int VB, int HPW, int which);
const void* ssm_bwd_kernel_bf16(int KP, int VB, bool one);
const void* ssm_bwd_kernel_f32(int KP, int VB, bool one);

}  // namespace m2rnn
