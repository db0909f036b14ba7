// The KV cache part of the C ABI: argument checks and dispatch. Every check
// runs before anything is enqueued; nothing here allocates.
#include <cmath>
#include <cstdint>

#include "kv_common.cuh"
#include "xq.h"

namespace {

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int bits_of(int type) { return type == XQ_TYPE_Q8_0 ? 8 : type == XQ_TYPE_Q4_0 ? 4 : 0; }

bool float_type(int type) { return type == XQ_TYPE_F32 || type == XQ_TYPE_F16 || type == XQ_TYPE_BF16; }

bool cache_shape(int type, int n_pages, int page_size, int heads, int dim) {
  // heads: a page's bytes and a pool's 32-blocks per token stay within an int
  if (n_pages < 0 || page_size < 16 || page_size > 4096 || (page_size & (page_size - 1)) != 0 || heads <= 0 || heads > 1024 ||
      (dim != 64 && dim != 96 && dim != 128 && dim != 256))
    return false;
  // a pool has fewer than 2^32 32-byte pieces
  return static_cast<unsigned long long>(n_pages) * heads * page_size * (dim * bits_of(type) / 8 + dim / 16) < (1ull << 37) - 32;
}

xq_status check_cache(const xq_kv_cache* c) {
  if (!c || !bits_of(c->type)) return XQ_ERR_ARG;
  if (!cache_shape(c->type, c->n_pages, c->page_size, c->heads, c->dim)) return XQ_ERR_SHAPE;
  if (c->n_pages > 0 && (!c->k || !c->v)) return XQ_ERR_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return XQ_ERR_ALIGN;
  return XQ_OK;
}

xq::KvView view_of(const xq_kv_cache* c) {
  xq::KvView v;
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.n_pages = c->n_pages;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c->page_size) ++v.page_shift;
  v.heads = c->heads;
  v.dim = c->dim;
  v.row_bytes = c->dim * bits_of(c->type) / 8;
  const long long lines = static_cast<long long>(c->heads) * c->page_size;
  v.scale_off = static_cast<int>(lines * v.row_bytes);
  v.page_bytes = lines * (v.row_bytes + c->dim / 16);
  return v;
}

// The parts of an attention call's arguments that its workspace depends on.
xq_status check_sizes(const xq_kv_cache* c, const xq_kv_query* q, bool shared) {
  if (!c || !q || !bits_of(c->type) || !float_type(q->type)) return XQ_ERR_ARG;
  if (!cache_shape(c->type, c->n_pages, c->page_size, c->heads, c->dim)) return XQ_ERR_SHAPE;
  if (q->batch < 0 || q->n_q < 0 || q->heads <= 0 || q->heads % c->heads || q->max_pages < 0) return XQ_ERR_SHAPE;
  // positions (own and prefix tokens) and the rows of the call stay within an int
  const long long longest = static_cast<long long>(q->max_pages) * c->page_size + (shared ? q->prefix_len : 0);
  const long long rows = static_cast<long long>(q->batch) * q->n_q;
  if (longest > (1LL << 30) || q->n_q > (1 << 20) || rows > (1LL << 30) || rows * q->heads > (1LL << 30)) return XQ_ERR_SHAPE;
  if (shared && q->prefix_len < 0) return XQ_ERR_SHAPE;
  return XQ_OK;
}

xq::KvAttnArgs args_of(const xq_kv_cache* c, const xq_kv_query* q, bool shared) {
  xq::KvAttnArgs a;
  a.c = view_of(c);
  a.type = q->type;
  a.batch = q->batch;
  a.n_q = q->n_q;
  a.q_heads = q->heads;
  a.group = q->heads / c->heads;
  a.rows = q->n_q * a.group;
  a.q = q->q;
  a.out = q->out;
  a.pages = q->pages;
  a.page_stride = q->page_stride;
  a.max_pages = q->max_pages;
  a.lens = q->lens;
  a.scale = q->scale;
  a.window = shared ? 0 : q->window;
  a.prefix_pages = shared ? q->prefix_pages : nullptr;
  a.prefix_len = shared ? q->prefix_len : 0;
  return a;
}

xq_status attn(const xq_kv_cache* c, const xq_kv_query* q, bool shared, void* ws, size_t ws_bytes, xq_stream stream) {
  xq_status st = check_sizes(c, q, shared);
  if (st == XQ_OK) st = check_cache(c);
  if (st != XQ_OK) return st;
  if (q->page_stride < q->max_pages || q->window < 0 || (shared && q->window != 0) || !std::isfinite(q->scale))
    return XQ_ERR_SHAPE;
  if (q->batch == 0 || q->n_q == 0) return XQ_OK;
  if (!q->q || !q->out || !q->lens || (q->max_pages > 0 && !q->pages)) return XQ_ERR_ARG;
  if (shared && q->prefix_len > 0 && !q->prefix_pages) return XQ_ERR_ARG;
  if (!aligned(q->q, 16) || !aligned(q->out, 16) || !aligned(q->pages, 4) || !aligned(q->lens, 4) ||
      (shared && !aligned(q->prefix_pages, 4)) || !aligned(ws, 16))
    return XQ_ERR_ALIGN;
  const xq::KvAttnArgs a = args_of(c, q, shared);
  const size_t need = xq::kv_attn_workspace(a, bits_of(c->type));
  if (need > ws_bytes || (need > 0 && !ws)) return XQ_ERR_WORKSPACE;
  return xq::launch_kv_attn(a, bits_of(c->type), ws, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? XQ_OK
                                                                                                         : XQ_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t xq_kv_bytes(int type, int n_pages, int page_size, int heads, int dim) {
  const int bits = bits_of(type);
  if (!bits || !cache_shape(type, n_pages, page_size, heads, dim)) return 0;
  return static_cast<size_t>(n_pages) * heads * page_size * (dim * bits / 8 + dim / 16);
}

xq_status xq_kv_write(const xq_kv_cache* cache, int x_type, const void* k, long long k_stride, const void* v,
                      long long v_stride, const int64_t* slots, int n_tokens, xq_stream stream) {
  const xq_status st = check_cache(cache);
  if (st != XQ_OK) return st;
  if (!float_type(x_type)) return XQ_ERR_ARG;
  const long long row = static_cast<long long>(cache->heads) * cache->dim;
  if (n_tokens < 0 || (n_tokens > 1 && (k_stride < row || v_stride < row))) return XQ_ERR_SHAPE;
  if (n_tokens == 0) return XQ_OK;
  if (!k || !v || !slots) return XQ_ERR_ARG;
  const unsigned eb = xq::kv_elt_bytes(x_type);
  if (!aligned(k, eb) || !aligned(v, eb) || !aligned(slots, 8)) return XQ_ERR_ALIGN;
  return xq::launch_kv_write(view_of(cache), bits_of(cache->type), x_type, k, k_stride, v, v_stride, slots, n_tokens,
                             reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? XQ_OK
             : XQ_ERR_CUDA;
}

xq_status xq_kv_read(const xq_kv_cache* cache, const int64_t* slots, int n_tokens, int y_type, void* k, void* v,
                     xq_stream stream) {
  const xq_status st = check_cache(cache);
  if (st != XQ_OK) return st;
  if (!float_type(y_type)) return XQ_ERR_ARG;
  if (n_tokens < 0) return XQ_ERR_SHAPE;
  if (n_tokens == 0) return XQ_OK;
  if (!k || !v || !slots) return XQ_ERR_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return XQ_ERR_ALIGN;
  return xq::launch_kv_read(view_of(cache), bits_of(cache->type), slots, n_tokens, y_type, k, v,
                            reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? XQ_OK
             : XQ_ERR_CUDA;
}

size_t xq_kv_attn_workspace_bytes(const xq_kv_cache* cache, const xq_kv_query* query) {
  if (check_sizes(cache, query, true) != XQ_OK) return 0;
  const xq::KvAttnArgs a = args_of(cache, query, true);
  const size_t need = xq::kv_attn_workspace(a, bits_of(cache->type));
  return need ? need : 16;
}

xq_status xq_kv_attn(const xq_kv_cache* cache, const xq_kv_query* query, void* workspace, size_t ws_bytes,
                     xq_stream stream) {
  return attn(cache, query, false, workspace, ws_bytes, stream);
}

xq_status xq_kv_attn_shared(const xq_kv_cache* cache, const xq_kv_query* query, void* workspace, size_t ws_bytes,
                            xq_stream stream) {
  return attn(cache, query, true, workspace, ws_bytes, stream);
}

}  // extern "C"
