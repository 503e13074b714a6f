// The float32 instances of the attention kernels.
#include "attention.h"

template gs::AttnPlan gs::attn_plan<float>(const gs::AttnArgs&);
template void gs::attn_fwd<float>(const gs::AttnArgs&, void*, hipStream_t);
template void gs::attn_bwd<float>(const gs::AttnArgs&, void*, hipStream_t);
