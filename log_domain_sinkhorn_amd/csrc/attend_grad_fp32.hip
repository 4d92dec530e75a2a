// Cross attention, backward: the kernels for fp32 elements.
#include "attend_grad.h"

template void sk::attn::attend_grad<float>(const sk::attn::GradArgs&, hipStream_t);
