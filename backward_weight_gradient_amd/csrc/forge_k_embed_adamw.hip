// The embedding's AdamW step for every supported state format.
#include "forge_embed_step.h"

namespace forge {
FORGE_ADAMW_LIST(FORGE_INSTANTIATE_EMBED)
}  // namespace forge
