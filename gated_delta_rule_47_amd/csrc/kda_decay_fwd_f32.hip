// Decay attention over float32 activations: the forward walk and the segments' states (kda_decay_attn.h).
#include "kda_decay_attn.h"

namespace kda {
KDA_DECAY_FWD_INSTANCES(, float, 32)
KDA_DECAY_FWD_INSTANCES(, float, 64)
KDA_DECAY_FWD_INSTANCES(, float, 128)
}  // namespace kda
