// Prompts over the fp16 pages of a 4-bit cache with bf16 queries, heads of 256.
#include "paged_attention_impl.h"

namespace ttq {
template hipError_t launch_prompts<256>(const AttnArgs& a, hipStream_t s);
}
