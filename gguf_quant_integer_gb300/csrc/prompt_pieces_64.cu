// Prompt attention of fp32 rows, head size 64.
#define XQ_PROMPT_TILE_IMPL
#include "prompt_pieces.cuh"

namespace xq {
template struct PromptPiecesDim<64>;
}  // namespace xq
