#include "packed_attention_impl.h"

namespace ttq {
template hipError_t launch_packed<128>(const PackedArgs&, hipStream_t);
}  // namespace ttq
