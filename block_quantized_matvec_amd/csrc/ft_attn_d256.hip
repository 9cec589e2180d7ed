// ft_attn_d256.hip -- the attention kernels of head dimension 256
#include "ft_attn_kernels.h"

hipError_t ftk_attn_d256(const AttnArgs& a, hipStream_t st) { return ftk::attn_pick<8>(a, st); }
