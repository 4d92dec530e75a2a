// Gathered attention weight: the kernels for bf16 elements.
#include "attend_mass.h"

template void sk::attn::attend_mass<__bf16>(const sk::attn::MassArgs&, hipStream_t);
