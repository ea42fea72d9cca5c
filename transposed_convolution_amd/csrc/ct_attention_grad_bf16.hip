// ct_attention_grad_bf16.hip -- the attention gradient's kernels of bfloat16 (see ct_attention_grad.hpp).
#include "ct_attention_grad.hpp"

template void ct::launch_attend_grad<__bf16>(const Attention &, const AttendGradPlan &, char *, hipStream_t);
