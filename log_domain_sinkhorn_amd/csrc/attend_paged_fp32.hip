// Attention over a paged cache: the kernels for fp32 elements.
#include "attend_paged.h"

template void sk::attn::attend_paged<float>(const sk::attn::PagedArgs&, sk::attn::PagedForm, hipStream_t);
