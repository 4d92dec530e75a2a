// Cross attention, backward: the kernels for bf16 elements.
#include "attend_grad.h"

template void sk::attn::attend_grad<__bf16>(const sk::attn::GradArgs&, hipStream_t);
