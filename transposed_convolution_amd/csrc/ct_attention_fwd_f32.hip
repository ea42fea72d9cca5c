// ct_attention_fwd_f32.hip -- the attention kernels of float32 (see ct_attention_fwd.hpp).
#include "ct_attention_fwd.hpp"

template void ct::launch_attend<float>(Attention, const AttendPlan &, hipStream_t);
