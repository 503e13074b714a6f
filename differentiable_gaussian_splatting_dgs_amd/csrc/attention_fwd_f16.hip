// The float16 instances of attention's forward.
#include "attention_fwd.h"

template gs::AttnBytes gs::attn_bytes<_Float16>(const gs::AttnArgs&);
template void gs::attn_fwd<_Float16>(const gs::AttnArgs&, void*, hipStream_t);
