// Causal attention over packed prompts.
//
// o_i = sum_j w_ij v_j / sum_j w_ij, w_ij = 2^(s_ij - m_i), s_ij = log2(e) scale q_i.k_j, over the keys j of the
// row's sequence up to its own place (the last `window` of them).
#include "prompt_tile.cuh"

namespace xq {
namespace {

__device__ unsigned int g_prompt_error;

constexpr int kRowWarps = 8;

// Rows and places of sequence b: false, and recorded, if its bounds are no range of the call's rows.
__device__ __forceinline__ bool sequence(const PromptArgs& A, int b, int* first, int* n) {
  const int s0 = A.starts[b], s1 = A.starts[b + 1];
  if (s0 < 0 || s1 < s0 || s1 > A.tokens) {
    atomicCAS(&g_prompt_error, 0u, kOpsBadStart);
    return false;
  }
  *first = s0;
  *n = s1 - s0;
  return true;
}

// One row by one warp, lanes over the head's elements: what every other kernel's results are measured by.
template <int TYPE, int D>
__device__ __noinline__ void one_row(const PromptArgs& A, int first, int place, int head) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, kv = head / (A.heads / A.kv_heads);
  const size_t token = static_cast<size_t>(first) + place;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = load_elt<TYPE>(A.q, token * A.q_stride + static_cast<size_t>(head) * D + lane + 32 * e);
    o[e] = 0.0f;
  }
  const float cs = A.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.0f;
  for (int j = A.window && place >= A.window ? place - A.window + 1 : 0; j <= place; ++j) {
    const size_t key = static_cast<size_t>(first) + j;
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      s = fmaf(q[e], load_elt<TYPE>(A.k, key * A.k_stride + static_cast<size_t>(kv) * D + lane + 32 * e), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s = __fmul_rn(s, cs);
    const float next = fmaxf(m, s);
    const float f = m == next ? 1.0f : exp2f(m - next), w = exp2f(s - next);
    m = next;
    l = fmaf(l, f, w);
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(o[e], f, w * load_elt<TYPE>(A.v, key * A.v_stride + static_cast<size_t>(kv) * D + lane + 32 * e));
  }
#pragma unroll
  for (int e = 0; e < E; ++e) store_elt<TYPE>(A.out, (token * A.heads + head) * D + lane + 32 * e, o[e] / l);
}

template <int TYPE, int D>
__global__ void __launch_bounds__(32 * kRowWarps) prompt_rows_kernel(const __grid_constant__ PromptArgs A) {
  const long long at = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int token = static_cast<int>(at / A.heads), head = static_cast<int>(at % A.heads);
  if (token >= A.tokens) return;
  for (int b = 0; b < A.batch; ++b) {
    int first, n;
    if (sequence(A, b, &first, &n) && token >= first && token < first + n) one_row<TYPE, D>(A, first, token - first, head);
  }
}

template <int TYPE>
cudaError_t launch(const PromptArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.tokens) * a.heads;
  const unsigned blocks = static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps);
  switch (a.dim) {
    case 64: prompt_rows_kernel<TYPE, 64><<<blocks, 32 * kRowWarps, 0, s>>>(a); break;
    case 96: prompt_rows_kernel<TYPE, 96><<<blocks, 32 * kRowWarps, 0, s>>>(a); break;
    case 128: prompt_rows_kernel<TYPE, 128><<<blocks, 32 * kRowWarps, 0, s>>>(a); break;
    default: prompt_rows_kernel<TYPE, 256><<<blocks, 32 * kRowWarps, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace

size_t prompt_attn_workspace(const PromptArgs&) { return 0; }

cudaError_t launch_prompt_attn(const PromptArgs& a, void*, cudaStream_t s) {
  g_kv_launched.store(true, std::memory_order_relaxed);
  if (a.type == kF32) return launch<kF32>(a, s);
  PromptTileArgs p;
  p.a = a;
  const int group = a.heads / a.kv_heads;
  // a group's heads share a tile's rows where that leaves at most a quarter of them empty
  p.pack = group <= kPromptRows && kPromptRows / group * group >= 96 ? group : 1;
  p.tokens_tile = kPromptRows / p.pack;
  p.units = a.heads / p.pack;
  switch (a.dim) {
    case 64: return PromptTileDim<64>::launch(p, s);
    case 96: return PromptTileDim<96>::launch(p, s);
    case 128: return PromptTileDim<128>::launch(p, s);
    default: return PromptTileDim<256>::launch(p, s);
  }
}

cudaError_t take_prompt_error(unsigned int* index, unsigned int* wait) {
  typedef cudaError_t (*TakeTile)(unsigned int*, unsigned int*);
  const TakeTile fns[4] = {PromptTileDim<64>::take_error, PromptTileDim<96>::take_error, PromptTileDim<128>::take_error,
                           PromptTileDim<256>::take_error};
  *wait = 0;
  cudaError_t e = take_record(g_prompt_error, index);
  for (TakeTile f : fns) {
    unsigned int i = 0, w = 0;
    if (e == cudaSuccess) e = f(&i, &w);
    if (*index == 0) *index = i;
    if (*wait == 0) *wait = w;
  }
  return e;
}
cudaError_t take_prompt_check(unsigned int* code) {
  typedef cudaError_t (*TakeFn)(unsigned int*);
  const TakeFn fns[4] = {PromptTileDim<64>::take_check, PromptTileDim<96>::take_check, PromptTileDim<128>::take_check,
                         PromptTileDim<256>::take_check};
  cudaError_t e = take_check_word(code);
  for (TakeFn f : fns) {
    unsigned int c = 0;
    if (e == cudaSuccess) e = f(&c);
    if (*code == 0) *code = c;
  }
  return e;
}

}  // namespace xq
