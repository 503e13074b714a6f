// The float32 instances of attention's backward.
#include "attention_bwd.h"

template void gs::attn_bwd<float>(const gs::AttnArgs&, void*, hipStream_t);
