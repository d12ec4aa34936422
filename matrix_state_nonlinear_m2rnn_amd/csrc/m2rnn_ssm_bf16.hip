// The selective scan's forward and state kernels for bf16 q, k, v.
#include "m2rnn_ssm_select.h"

namespace m2rnn {
const void* ssm_kernel_bf16(int KP, int VB, int HPW, int which) { return ssm_pick<true>(KP, VB, HPW, which); }
}  // namespace m2rnn
