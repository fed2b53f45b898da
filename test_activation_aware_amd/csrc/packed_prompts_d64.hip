// Prompts over the fp16 pages of a 4-bit cache with bf16 queries, heads of 64.
#include "paged_attention_impl.h"

namespace ttq {
template hipError_t launch_prompts<64>(const AttnArgs& a, hipStream_t s);
}
