// The cache attention's tcgen05 kernels at head size 128 (a translation unit of its own).
#define XQ_KV_ATTN_IMPL
#include "kv_tile.cuh"

namespace xq {
template struct KvTileDim<128>;
}
