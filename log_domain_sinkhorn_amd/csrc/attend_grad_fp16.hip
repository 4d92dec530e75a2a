// Cross attention, backward: the kernels for fp16 elements.
#include "attend_grad.h"

template void sk::attn::attend_grad<_Float16>(const sk::attn::GradArgs&, hipStream_t);
