// The bfloat16 instances of attention's backward.
#include "attention_bwd.h"

template void gs::attn_bwd<__bf16>(const gs::AttnArgs&, void*, hipStream_t);
