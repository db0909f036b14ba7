// Low-rank adapters of many requests beside shared projections:
// y[m] += scale[i] * (x[m] A[i]^T) B[i]^T with the row's adapter i.
#include "ops_common.cuh"

namespace xq {
namespace {

__device__ unsigned int g_lora_error;

constexpr int kThreads = 256;

template <int TYPE>
__device__ __forceinline__ void row(const AdapterProj& p, int m, int id, float* t) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < p.rank; r += kThreads / 32) {
    float s = 0.0f;
    for (int k = lane; k < p.K; k += 32)
      s = fmaf(p.x[static_cast<size_t>(m) * p.K + k], load_elt<TYPE>(p.a, (static_cast<size_t>(id) * p.rank + r) * p.K + k), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) t[r] = s * (p.scales ? p.scales[id] : 1.0f);
  }
  __syncthreads();
  for (int n = threadIdx.x; n < p.N; n += kThreads) {
    float s = 0.0f;
    for (int r = 0; r < p.rank; ++r) s = fmaf(t[r], load_elt<TYPE>(p.b, (static_cast<size_t>(id) * p.N + n) * p.rank + r), s);
    p.y[static_cast<size_t>(m) * p.N + n] += s;
  }
}

__global__ void __launch_bounds__(kThreads) lora_kernel(const __grid_constant__ LoraArgs A) {
  __shared__ float t[256];
  const AdapterProj& p = A.p[blockIdx.y];
  const int m = blockIdx.x, id = A.ids[m];
  if (id < 0) return;
  if (id >= p.n) {
    if (threadIdx.x == 0) atomicCAS(&g_lora_error, 0u, kOpsBadAdapter);
    return;
  }
  if (p.type == kF32)
    row<kF32>(p, m, id, t);
  else if (p.type == kF16)
    row<kF16>(p, m, id, t);
  else
    row<kBF16>(p, m, id, t);
}

}  // namespace

cudaError_t launch_lora(const LoraArgs& a, cudaStream_t s) {
  g_kv_launched.store(true, std::memory_order_relaxed);
  lora_kernel<<<dim3(a.M, a.n_proj), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t take_lora_error(unsigned int* code) { return take_record(g_lora_error, code); }
cudaError_t take_lora_check(unsigned int* code) { return take_check_word(code); }

}  // namespace xq
