// Decay attention over bfloat16 activations: the forward walk and the segments' states (kda_decay_attn.h).
#include "kda_decay_attn.h"

namespace kda {
KDA_DECAY_FWD_INSTANCES(, bf16_t, 32)
KDA_DECAY_FWD_INSTANCES(, bf16_t, 64)
KDA_DECAY_FWD_INSTANCES(, bf16_t, 128)
}  // namespace kda
