// The float16 instances of the attention kernels.
#include "attention.h"

template gs::AttnPlan gs::attn_plan<_Float16>(const gs::AttnArgs&);
template void gs::attn_fwd<_Float16>(const gs::AttnArgs&, void*, hipStream_t);
template void gs::attn_bwd<_Float16>(const gs::AttnArgs&, void*, hipStream_t);
