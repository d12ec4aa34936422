// The selective scan's forward and state kernels for f32 q, k, v.
#include "m2rnn_ssm_select.h"

namespace m2rnn {
const void* ssm_kernel_f32(int KP, int VB, int HPW, int which) { return ssm_pick<false>(KP, VB, HPW, which); }
}  // namespace m2rnn
