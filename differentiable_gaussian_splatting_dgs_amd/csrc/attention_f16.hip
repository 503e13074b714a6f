// The float16 instances of the attention kernels.
#include "attention.h"

template void gs::attn_fwd<_Float16>(const gs::AttnArgs&, hipStream_t);
template void gs::attn_bwd<_Float16>(const gs::AttnArgs&, hipStream_t);
