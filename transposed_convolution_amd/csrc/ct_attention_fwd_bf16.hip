// ct_attention_fwd_bf16.hip -- the attention kernels of bfloat16 (see ct_attention_fwd.hpp).
#include "ct_attention_fwd.hpp"

template void ct::launch_attend<__bf16>(const Attention &, const AttendPlan &, float *, hipStream_t);
