// Gathered attention weight: the kernels for fp16 elements.
#include "attend_mass.h"

template void sk::attn::attend_mass<_Float16>(const sk::attn::MassArgs&, hipStream_t);
