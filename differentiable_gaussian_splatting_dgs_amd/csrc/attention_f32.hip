// The float32 instances of the attention kernels.
#include "attention.h"

template void gs::attn_fwd<float>(const gs::AttnArgs&, hipStream_t);
template void gs::attn_bwd<float>(const gs::AttnArgs&, hipStream_t);
