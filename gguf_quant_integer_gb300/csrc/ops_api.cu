// Adapters, norms with rotation and prompt attention in the C ABI: argument
// checks and dispatch. Every check runs before anything is enqueued; nothing
// here allocates.
#include <cmath>
#include <cstdint>

#include "ops_common.cuh"
#include "xq.h"

namespace {

bool aligned(const void* p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool float_type(int type) { return type == XQ_TYPE_F32 || type == XQ_TYPE_F16 || type == XQ_TYPE_BF16; }

bool head_size(int dim) { return dim == 64 || dim == 96 || dim == 128 || dim == 256; }

xq_status status_of(cudaError_t e) { return e == cudaSuccess ? XQ_OK : XQ_ERR_CUDA; }

// The parts of a prompt call's arguments that its workspace depends on.
xq_status check_prompt_sizes(const xq_prompts* p) {
  if (!p || !float_type(p->type)) return XQ_ERR_ARG;
  if (p->tokens < 0 || p->batch < 0 || p->heads <= 0 || p->kv_heads <= 0 || p->heads % p->kv_heads || !head_size(p->dim))
    return XQ_ERR_SHAPE;
  // positions, rows of all heads and sequences stay within an int
  if (p->tokens > (1 << 30) || p->batch > (1 << 24) || static_cast<long long>(p->tokens) * p->heads > (1LL << 30) ||
      p->heads > (1 << 16) || (p->type == XQ_TYPE_F32 && p->tokens >= (1 << 30)))
    return XQ_ERR_SHAPE;
  return XQ_OK;
}

xq::PromptArgs prompt_args(const xq_prompts* p) {
  xq::PromptArgs a;
  a.type = p->type;
  a.tokens = p->tokens;
  a.batch = p->batch;
  a.heads = p->heads;
  a.kv_heads = p->kv_heads;
  a.dim = p->dim;
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.q_stride = p->q_stride;
  a.k_stride = p->k_stride;
  a.v_stride = p->v_stride;
  a.out = p->out;
  a.starts = p->starts;
  a.scale = p->scale;
  a.window = p->window;
  return a;
}

xq_status prompt_attn(const xq_prompts* p, void* workspace, size_t ws_bytes, xq_stream stream, long long wait, bool withhold) {
  const xq_status st = check_prompt_sizes(p);
  if (st != XQ_OK) return st;
  if (p->window < 0 || !std::isfinite(p->scale)) return XQ_ERR_SHAPE;
  const long long wq = static_cast<long long>(p->heads) * p->dim, wk = static_cast<long long>(p->kv_heads) * p->dim;
  if (p->tokens > 1 && (p->q_stride < wq || p->k_stride < wk || p->v_stride < wk)) return XQ_ERR_SHAPE;
  if (p->tokens == 0 || p->batch == 0) return XQ_OK;
  if (!p->q || !p->k || !p->v || !p->out || !p->starts) return XQ_ERR_ARG;
  const long long piece = 16 / xq::kv_elt_bytes(p->type);
  if (!aligned(p->q, 16) || !aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->out, 16) || !aligned(p->starts, 4) ||
      !aligned(workspace, 16) || (p->tokens > 1 && (p->q_stride % piece || p->k_stride % piece || p->v_stride % piece)))
    return XQ_ERR_ALIGN;
  const xq::PromptArgs a = prompt_args(p);
  const size_t need = xq::prompt_attn_workspace(a);
  if (need > ws_bytes || (need > 0 && !workspace)) return XQ_ERR_WORKSPACE;
  return status_of(xq::launch_prompt_attn(a, workspace, reinterpret_cast<cudaStream_t>(stream), wait, withhold));
}

}  // namespace

extern "C" {

xq_status xq_lora_add(const xq_adapters* proj, int n_proj, const float* const* inputs, int n_inputs, int M, const int32_t* ids,
                      xq_stream stream) {
  if (n_proj < 0 || n_proj > xq::kMaxAdapterProj || n_inputs < 0 || n_inputs > 64) return XQ_ERR_ARG;
  if ((n_proj > 0 && !proj) || (n_inputs > 0 && !inputs)) return XQ_ERR_ARG;
  if (M < 0 || M > (1 << 30)) return XQ_ERR_SHAPE;
  xq::LoraArgs a;
  a.n_proj = 0;
  a.M = M;
  a.ids = ids;
  for (int i = 0; i < n_proj; ++i) {
    const xq_adapters& p = proj[i];
    if (!float_type(p.type) || p.input < 0 || p.input >= n_inputs) return XQ_ERR_ARG;
    if (p.n < 0 || p.n > 8192 || p.rank < 8 || p.rank > 256 || p.rank % 8 || p.K <= 0 || p.K % 32 || p.N < 0 ||
        p.N > (1 << 30))  // a cluster's steps over the columns stay within an int
      return XQ_ERR_SHAPE;
    if (M == 0 || p.N == 0) continue;
    const float* const x = inputs[p.input];
    if (!x || !p.y || (p.n > 0 && (!p.a || !p.b))) return XQ_ERR_ARG;
    if (!aligned(x, 16) || !aligned(p.a, 16) || !aligned(p.b, 16) || !aligned(p.y, 4) || !aligned(p.scales, 4)) return XQ_ERR_ALIGN;
    a.p[a.n_proj++] = xq::AdapterProj{p.type, p.n, p.rank, p.K, p.N, p.a, p.b, p.scales, p.y, x};
  }
  if (a.n_proj == 0) return XQ_OK;
  if (!ids) return XQ_ERR_ARG;
  if (!aligned(ids, 4)) return XQ_ERR_ALIGN;
  return status_of(xq::launch_lora(a, reinterpret_cast<cudaStream_t>(stream)));
}

xq_status xq_qk_norm_rope(const xq_qk_rows* r, xq_stream stream) {
  if (!r || !float_type(r->type) || !float_type(r->y_type)) return XQ_ERR_ARG;
  if (r->tokens < 0 || r->heads <= 0 || r->kv_heads <= 0 || r->heads > (1 << 16) || r->kv_heads > (1 << 16) || !head_size(r->dim) ||
      r->rot < 0 || r->rot > r->dim || r->rot % 16 || !(r->eps >= 0.0f) || !std::isfinite(r->eps) || !std::isfinite(r->magnitude))
    return XQ_ERR_SHAPE;
  if (r->pairs != 0 && r->pairs != 1) return XQ_ERR_ARG;
  const long long wq = static_cast<long long>(r->heads) * r->dim, wk = static_cast<long long>(r->kv_heads) * r->dim;
  if (r->tokens > 1 && (r->q_stride < wq || r->k_stride < wk || r->q_out_stride < wq || r->k_out_stride < wk)) return XQ_ERR_SHAPE;
  if (r->tokens == 0) return XQ_OK;
  if (!r->q || !r->k || !r->q_out || !r->k_out || !r->positions || (r->rot > 0 && !r->turns)) return XQ_ERR_ARG;
  const unsigned xb = xq::kv_elt_bytes(r->type), yb = xq::kv_elt_bytes(r->y_type);
  if (!aligned(r->q, xb) || !aligned(r->k, xb) || !aligned(r->q_out, yb) || !aligned(r->k_out, yb) || !aligned(r->q_weight, 4) ||
      !aligned(r->k_weight, 4) || !aligned(r->positions, 8) || !aligned(r->turns, 8))
    return XQ_ERR_ALIGN;
  xq::RopeArgs a;
  a.side[0] = xq::RopeSide{r->q, r->q_out, r->q_stride, r->q_out_stride, r->q_weight, r->heads};
  a.side[1] = xq::RopeSide{r->k, r->k_out, r->k_stride, r->k_out_stride, r->k_weight, r->kv_heads};
  // in place, a row is read whole before it is written; with another type or stride it would meet other rows
  for (const xq::RopeSide& s : a.side)
    if (s.x == s.y && (r->type != r->y_type || (r->tokens > 1 && s.x_stride != s.y_stride))) return XQ_ERR_ARG;
  a.type = r->type;
  a.y_type = r->y_type;
  a.tokens = r->tokens;
  a.dim = r->dim;
  a.rot = r->rot;
  a.pairs = r->pairs;
  a.eps = r->eps;
  a.magnitude = r->magnitude;
  a.positions = r->positions;
  a.turns = r->turns;
  return status_of(xq::launch_qk_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t xq_prompt_attn_workspace_bytes(const xq_prompts* prompts) {
  if (check_prompt_sizes(prompts) != XQ_OK) return 0;
  const size_t need = xq::prompt_attn_workspace(prompt_args(prompts));
  return need ? need : 16;
}

xq_status xq_prompt_attn(const xq_prompts* p, void* workspace, size_t ws_bytes, xq_stream stream) {
  return prompt_attn(p, workspace, ws_bytes, stream, 0, false);
}

xq_status xq_debug_stalled_prompt_attn(const xq_prompts* p, void* workspace, size_t ws_bytes, long long clocks, int withhold,
                                       xq_stream stream) {
  if (clocks < 1 || clocks > (1ll << 32)) return XQ_ERR_ARG;
  return prompt_attn(p, workspace, ws_bytes, stream, clocks, withhold != 0);
}

}  // extern "C"
