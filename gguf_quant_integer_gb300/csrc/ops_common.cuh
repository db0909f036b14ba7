// What the operators between a layer's projections and its cache share:
// adapters, norms with rotation, prompt attention.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv_common.cuh"

namespace xq {

constexpr int kMaxAdapterProj = 16;

struct AdapterProj {
  int type, n, rank, K, N;
  const void* a;
  const void* b;
  const float* scales;
  float* y;
  const float* x;
};
struct LoraArgs {
  AdapterProj p[kMaxAdapterProj];
  int n_proj, M;
  const int32_t* ids;
};

struct RopeSide {  // q or k
  const void* x;
  void* y;
  long long x_stride, y_stride;  // elements between tokens
  const float* weight;
  int heads;
};
struct RopeArgs {
  RopeSide side[2];
  int type, y_type, tokens, dim, rot, pairs;
  float eps, magnitude;
  const int64_t* positions;
  const uint64_t* turns;
};

struct PromptArgs {
  int type, tokens, batch, heads, kv_heads, dim;
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  void* out;
  const int32_t* starts;
  float scale;
  int window;
};

enum OpsRecord : unsigned { kOpsBadAdapter = 1, kOpsBadStart = 2 };

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s);
cudaError_t launch_qk_rope(const RopeArgs& a, cudaStream_t s);
size_t prompt_attn_workspace(const PromptArgs& a);
// wait: clocks that a wait lasts at most beside what slow work may take, 0 for the usual; withhold: test hook, no copies are issued.
cudaError_t launch_prompt_attn(const PromptArgs& a, void* workspace, cudaStream_t s, long long wait = 0, bool withhold = false);

// Read and clear the records of invalid indices (0: none), and the checked builds' words.
cudaError_t take_lora_error(unsigned int* code);
cudaError_t take_prompt_error(unsigned int* index, unsigned int* wait);
cudaError_t take_lora_check(unsigned int* code);
cudaError_t take_rope_check(unsigned int* code);
cudaError_t take_prompt_check(unsigned int* code);

// Element i of a row of an activation type, and its store.
template <int TYPE>
__device__ __forceinline__ float load_elt(const void* p, size_t i) {
  if constexpr (TYPE == kF32) return static_cast<const float*>(p)[i];
  if constexpr (TYPE == kF16) return __half2float(static_cast<const __half*>(p)[i]);
  if constexpr (TYPE == kBF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
template <int TYPE>
__device__ __forceinline__ void store_elt(void* p, size_t i, float v) {
  if constexpr (TYPE == kF32) static_cast<float*>(p)[i] = v;
  if constexpr (TYPE == kF16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  if constexpr (TYPE == kBF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

}  // namespace xq
