// Rotary positions, head norms, appending: the kernels for fp32 elements.
#include "rotate.h"

template void sk::attn::rotate<float>(sk::attn::RotateArgs&, int, hipStream_t);
template void sk::attn::rotate_grad<float>(sk::attn::RotateArgs&, int, int, hipStream_t);
