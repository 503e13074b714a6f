// The bfloat16 instances of the attention kernels.
#include "attention.h"

template gs::AttnPlan gs::attn_plan<__bf16>(const gs::AttnArgs&);
template void gs::attn_fwd<__bf16>(const gs::AttnArgs&, void*, hipStream_t);
template void gs::attn_bwd<__bf16>(const gs::AttnArgs&, void*, hipStream_t);
