// The selective scan's backward kernels for bf16 q, k, v.
#include "m2rnn_ssm_select.h"

namespace m2rnn {
const void* ssm_bwd_kernel_bf16(int KP, int VB, bool one) { return ssm_pick_bwd<true>(KP, VB, one); }
}  // namespace m2rnn
