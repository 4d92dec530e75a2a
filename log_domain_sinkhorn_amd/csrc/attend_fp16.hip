// Cross attention, forward: the kernels for fp16 elements.
#include "attend.h"

template void sk::attn::attend<_Float16>(const sk::attn::AttendArgs&, bool, const MassArgs*, hipStream_t);
