// The float16 instances of attention's backward.
#include "attention_bwd.h"

template void gs::attn_bwd<_Float16>(const gs::AttnArgs&, void*, hipStream_t);
