// Decay-attention walks over float32 activations, key width padded to 128 (kda_decay_attn.h).
#include "kda_decay_attn.h"

namespace kda {
template hipError_t launch_walk_kd<float, 128, false>(const WalkArgs&, bool, hipStream_t);
template hipError_t launch_walk_kd<float, 128, true>(const WalkArgs&, bool, hipStream_t);
template hipError_t launch_segments_kd<float, 128, false>(const SegArgs&, bool, hipStream_t);
template hipError_t launch_segments_kd<float, 128, true>(const SegArgs&, bool, hipStream_t);
}  // namespace kda
