// The bfloat16 instances of the attention kernels.
#include "attention.h"

template void gs::attn_fwd<__bf16>(const gs::AttnArgs&, hipStream_t);
template void gs::attn_bwd<__bf16>(const gs::AttnArgs&, hipStream_t);
