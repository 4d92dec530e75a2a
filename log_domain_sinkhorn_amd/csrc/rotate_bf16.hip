// Rotary positions, head norms, appending: the kernels for bf16 elements.
#include "rotate.h"

template void sk::attn::rotate<__bf16>(sk::attn::RotateArgs&, int, hipStream_t);
template void sk::attn::rotate_grad<__bf16>(sk::attn::RotateArgs&, int, int, hipStream_t);
