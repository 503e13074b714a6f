// The float32 instances of attention's forward.
#include "attention_fwd.h"

template gs::AttnBytes gs::attn_bytes<float>(const gs::AttnArgs&);
template void gs::attn_fwd<float>(const gs::AttnArgs&, void*, hipStream_t);
