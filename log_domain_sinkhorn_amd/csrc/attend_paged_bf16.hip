// Attention over a paged cache: the kernels for bf16 elements.
#include "attend_paged.h"

template void sk::attn::attend_paged<__bf16>(const sk::attn::PagedArgs&, sk::attn::PagedForm, hipStream_t);
