// Attention over a paged cache: the kernels for fp16 elements.
#include "attend_paged.h"

template void sk::attn::attend_paged<_Float16>(const sk::attn::PagedArgs&, sk::attn::PagedForm, hipStream_t);
