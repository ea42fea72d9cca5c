// ct_attention_fwd_f16.hip -- the attention kernels of float16 (see ct_attention_fwd.hpp).
#include "ct_attention_fwd.hpp"

template void ct::launch_attend<_Float16>(const Attention &, const AttendPlan &, float *, hipStream_t);
