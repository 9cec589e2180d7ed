// ft_attn_d128.hip -- the attention kernels of head dimension 128
#include "ft_attn_kernels.h"

hipError_t ftk_attn_d128(const AttnArgs& a, hipStream_t st) { return ftk::attn_pick<4>(a, st); }
