// The narrow layers' one-pass backward (linear_bwd.h) for float.
#include "linear_bwd.h"

namespace gs {
GS_DEFINE_BWD_NARROW(float)
}  // namespace gs
