// Cross attention, forward: the kernels for bf16 elements.
#include "attend.h"

template void sk::attn::attend<__bf16>(const sk::attn::AttendArgs&, bool, const MassArgs*, hipStream_t);
