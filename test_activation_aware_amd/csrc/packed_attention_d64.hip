// Attention over a 4-bit cache, heads of 64.
#include "packed_attention_impl.h"

namespace ttq {
template hipError_t launch_packed<64>(const PackedArgs&, hipStream_t);
}  // namespace ttq
