// Rotary positions, head norms, appending: the kernels for fp16 elements.
#include "rotate.h"

template void sk::attn::rotate<_Float16>(sk::attn::RotateArgs&, int, hipStream_t);
template void sk::attn::rotate_grad<_Float16>(sk::attn::RotateArgs&, int, int, hipStream_t);
