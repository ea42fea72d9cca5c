// ct_attention_grad_f16.hip -- the attention gradient's kernels of float16 (see ct_attention_grad.hpp).
#include "ct_attention_grad.hpp"

template void ct::launch_attend_grad<_Float16>(const Attention &, const AttendGradPlan &, char *, hipStream_t);
