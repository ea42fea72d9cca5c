// ct_attention_fwd_f32.hip -- the attention kernels of float32 (see ct_attention_fwd.hpp).
#include "ct_attention_fwd.hpp"

template void ct::launch_attend<float>(const Attention &, const AttendPlan &, float *, hipStream_t);
