// Prompt attention of 16-bit rows, head size 256.
#define XQ_PROMPT_TILE_IMPL
#include "prompt_tile.cuh"

namespace xq {
template struct PromptTileDim<256>;
}  // namespace xq
