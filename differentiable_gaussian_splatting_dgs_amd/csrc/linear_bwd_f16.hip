// The narrow layers' one-pass backward (linear_bwd.h) for _Float16.
#include "linear_bwd.h"

namespace gs {
GS_DEFINE_BWD_NARROW(_Float16)
}  // namespace gs
