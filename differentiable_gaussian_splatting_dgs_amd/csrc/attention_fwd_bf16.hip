// The bfloat16 instances of attention's forward.
#include "attention_fwd.h"

template gs::AttnBytes gs::attn_bytes<__bf16>(const gs::AttnArgs&);
template void gs::attn_fwd<__bf16>(const gs::AttnArgs&, void*, hipStream_t);
