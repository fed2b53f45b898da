// Attention over a 4-bit cache, heads of 256.
#include "packed_attention_impl.h"

namespace ttq {
template hipError_t launch_packed<256>(const PackedArgs&, hipStream_t);
}  // namespace ttq
