// ct_attention_grad_f32.hip -- the attention gradient's kernels of float32 (see ct_attention_grad.hpp).
#include "ct_attention_grad.hpp"

template void ct::launch_attend_grad<float>(const Attention &, const AttendGradPlan &, char *, hipStream_t);
