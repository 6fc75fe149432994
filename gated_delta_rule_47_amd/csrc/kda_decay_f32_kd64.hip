// Decay-attention walks over float32 activations, key width padded to 64 (kda_decay_attn.h).
#define KDA_DECAY_INSTANCES
#include "kda_decay_attn.h"

namespace kda {
template hipError_t launch_walk_kd<float, 64>(const WalkArgs&, WalkKind, hipStream_t);
template hipError_t launch_segments_kd<float, 64>(const SegArgs&, const SegArgs*, bool, hipStream_t);
}  // namespace kda
