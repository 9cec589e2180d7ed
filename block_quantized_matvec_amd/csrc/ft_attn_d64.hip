// ft_attn_d64.hip -- the attention kernels of head dimension 64
#include "ft_attn_kernels.h"

hipError_t ftk_attn_d64(const AttnArgs& a, hipStream_t st) { return ftk::attn_pick<2>(a, st); }
