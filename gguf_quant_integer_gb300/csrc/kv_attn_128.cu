// The cache attention kernels at head size 128 (a translation unit of its own: the four sizes compile in parallel).
#define XQ_KV_ATTN_IMPL
#include "kv_attn.cuh"

namespace xq {
template struct KvAttnDim<128>;
}
