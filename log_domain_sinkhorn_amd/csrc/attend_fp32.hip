// Cross attention, forward: the kernels for fp32 elements.
#include "attend.h"

template void sk::attn::attend<float>(const sk::attn::AttendArgs&, bool, const MassArgs*, hipStream_t);
