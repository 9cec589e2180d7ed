// ft_attn_d96.hip -- the attention kernels of head dimension 96
#include "ft_attn_kernels.h"

hipError_t ftk_attn_d96(const AttnArgs& a, hipStream_t st) { return ftk::attn_pick<3>(a, st); }
