// Gathered attention weight: the kernels for fp32 elements.
#include "attend_mass.h"

template void sk::attn::attend_mass<float>(const sk::attn::MassArgs&, hipStream_t);
