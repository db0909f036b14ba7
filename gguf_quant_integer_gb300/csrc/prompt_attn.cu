// Which kernels a prompt attention call runs, its workspace, the error words.
#include <climits>

#include "prompt_pieces.cuh"
#include "prompt_tile.cuh"

namespace xq {
namespace {

// The workspace of an fp32 call, from `base` on.
PromptPieces pieces(const PromptArgs& a, uint8_t* base) {
  PromptPieces w = {};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* const p = base + at;
    at += (bytes + 255) & ~static_cast<size_t>(255);
    return p;
  };
  const size_t k = static_cast<size_t>(a.tokens) * a.kv_heads, d = a.dim;
  w.slots = a.tokens / prompt_piece_keys(a.dim) + a.batch;
  const size_t tiles = static_cast<size_t>(w.slots) * a.kv_heads;
  w.k = reinterpret_cast<__half*>(take(k * d * 4));
  w.v = reinterpret_cast<__half*>(take(k * d * 4));
  w.k_power = reinterpret_cast<float*>(take(tiles * 4));
  w.v_power = reinterpret_cast<float*>(take(tiles * d * 4));
  w.v_most = reinterpret_cast<float*>(take(tiles * 4));
  w.k_owner = reinterpret_cast<int*>(take(tiles * 4));
  w.v_owner = reinterpret_cast<int*>(take(tiles * 4));
  w.bytes = at;
  return w;
}

// How a call's heads and tokens make row tiles.
PromptTileArgs tiles(const PromptArgs& a) {
  PromptTileArgs p;
  p.a = a;
  const int group = a.heads / a.kv_heads;
  // a group's heads share a tile's rows where that leaves at most a quarter of them empty
  p.pack = group <= kPromptRows && kPromptRows / group * group >= 96 ? group : 1;
  p.tokens_tile = kPromptRows / p.pack;
  p.units = a.heads / p.pack;
  p.sums = nullptr;
  p.wait = prompt_wait_limit(a, kPromptWait);
  p.withhold = false;
  return p;
}

typedef cudaError_t (*TakeTwo)(unsigned int*, unsigned int*);
typedef cudaError_t (*TakeOne)(unsigned int*);

}  // namespace

size_t prompt_attn_workspace(const PromptArgs& a) {
  if (a.tokens <= 0 || a.batch <= 0) return 0;
  if (a.type == kF32) return pieces(a, nullptr).bytes;
  // no row sees more keys than there are tokens
  if (a.tokens <= kPromptRun * kPromptTileKeys) return 0;
  const int row_tiles = prompt_row_tiles(a.dim);
  return static_cast<size_t>(prompt_tile_grid(tiles(a), row_tiles)) * row_tiles * prompt_run_quads(a.dim) * sizeof(float4);
}

cudaError_t launch_prompt_attn(const PromptArgs& a, void* workspace, cudaStream_t s, long long wait, bool withhold) {
  PromptTileArgs p = tiles(a);
  if (wait > 0) p.wait = prompt_wait_limit(a, wait);
  p.withhold = withhold;
  if (a.type == kF32) {
    const PromptPieces w = pieces(a, static_cast<uint8_t*>(workspace));
    const cudaError_t e = launch_prompt_split(a, w, s);
    if (e != cudaSuccess) return e;
    switch (a.dim) {
      case 64: return PromptPiecesDim<64>::launch(p, w, s);
      case 96: return PromptPiecesDim<96>::launch(p, w, s);
      case 128: return PromptPiecesDim<128>::launch(p, w, s);
      default: return PromptPiecesDim<256>::launch(p, w, s);
    }
  }
  p.sums = static_cast<float4*>(workspace);
  switch (a.dim) {
    case 64: return PromptTileDim<64>::launch(p, s);
    case 96: return PromptTileDim<96>::launch(p, s);
    case 128: return PromptTileDim<128>::launch(p, s);
    default: return PromptTileDim<256>::launch(p, s);
  }
}

cudaError_t take_prompt_error(unsigned int* index, unsigned int* wait) {
  const TakeTwo fns[8] = {PromptTileDim<64>::take_error,   PromptTileDim<96>::take_error,   PromptTileDim<128>::take_error,
                          PromptTileDim<256>::take_error,  PromptPiecesDim<64>::take_error, PromptPiecesDim<96>::take_error,
                          PromptPiecesDim<128>::take_error, PromptPiecesDim<256>::take_error};
  *index = *wait = 0;
  for (TakeTwo f : fns) {
    unsigned int i = 0, w = 0;
    const cudaError_t e = f(&i, &w);
    if (e != cudaSuccess) return e;
    if (*index == 0) *index = i;
    if (*wait == 0) *wait = w;
  }
  return cudaSuccess;
}
cudaError_t take_prompt_check(unsigned int* code) {
  const TakeOne fns[8] = {PromptTileDim<64>::take_check,   PromptTileDim<96>::take_check,   PromptTileDim<128>::take_check,
                          PromptTileDim<256>::take_check,  PromptPiecesDim<64>::take_check, PromptPiecesDim<96>::take_check,
                          PromptPiecesDim<128>::take_check, PromptPiecesDim<256>::take_check};
  *code = 0;
  for (TakeOne f : fns) {
    unsigned int c = 0;
    const cudaError_t e = f(&c);
    if (e != cudaSuccess) return e;
    if (*code == 0) *code = c;
  }
  return cudaSuccess;
}

}  // namespace xq
