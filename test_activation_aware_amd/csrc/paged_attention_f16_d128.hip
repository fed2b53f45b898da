// Paged attention, f16, heads of 128.
#include "paged_attention_impl.h"

namespace ttq {
template hipError_t launch_attn<_Float16, 128>(const AttnArgs& a, hipStream_t s);
}
