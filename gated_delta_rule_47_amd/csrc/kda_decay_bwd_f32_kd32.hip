// Decay attention over float32 activations: the backward walks for keys padded to 32 (kda_decay_attn.h).
#include "kda_decay_attn.h"

namespace kda {
KDA_DECAY_BWD_INSTANCES(, float, 32)
}  // namespace kda
