// Decay-attention walks over bfloat16 activations, key width padded to 32 (kda_decay_attn.h).
#include "kda_decay_attn.h"

namespace kda {
template hipError_t launch_walk_kd<bf16_t, 32, false>(const WalkArgs&, bool, hipStream_t);
template hipError_t launch_walk_kd<bf16_t, 32, true>(const WalkArgs&, bool, hipStream_t);
template hipError_t launch_segments_kd<bf16_t, 32, false>(const SegArgs&, bool, hipStream_t);
template hipError_t launch_segments_kd<bf16_t, 32, true>(const SegArgs&, bool, hipStream_t);
}  // namespace kda
