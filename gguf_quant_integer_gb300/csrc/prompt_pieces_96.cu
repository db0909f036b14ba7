// Prompt attention of fp32 rows, head size 96.
#define XQ_PROMPT_TILE_IMPL
#include "prompt_pieces.cuh"

namespace xq {
template struct PromptPiecesDim<96>;
}  // namespace xq
