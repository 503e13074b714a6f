// The narrow layers' one-pass backward (linear_bwd.h) for __bf16.
#include "linear_bwd.h"

namespace gs {
GS_DEFINE_BWD_NARROW(__bf16)
}  // namespace gs
