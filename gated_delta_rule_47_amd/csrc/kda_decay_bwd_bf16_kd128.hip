// Decay attention over bfloat16 activations: the backward walks for keys padded to 128 (kda_decay_attn.h).
#include "kda_decay_attn.h"

namespace kda {
KDA_DECAY_BWD_INSTANCES(, bf16_t, 128)
}  // namespace kda
