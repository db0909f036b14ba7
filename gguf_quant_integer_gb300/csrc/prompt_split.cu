// fp32 rows of K and V as two fp16 numbers each, for prompt attention (see prompt_pieces.cuh).
//
// x 2^s = hi + lo: hi = fp16(x 2^s), lo = fp16(x 2^s - hi), with 2^s from the largest finite magnitude of a tile of keys (K)
// or of a column of it (V), which comes to 2^14 .. 2^15: 22 bits for everything down to 2^-17 of that, and an error of 2^-39
// of it below. An element that is not finite is one in hi, and 0 in lo.
//
// Pieces lie at their rows' places, in sizes that go by their slot. With bounds that go back, a sequence that is left out may lie
// between two that have rows in common: slots with such rows get no pieces, and who needs them computes his rows from the
// values themselves.
#include <climits>

#include "prompt_pieces.cuh"

namespace xq {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.0f;
}
__device__ __forceinline__ float4 finite_abs(float4 x) { return make_float4(finite_abs(x.x), finite_abs(x.y), finite_abs(x.z), finite_abs(x.w)); }
__device__ __forceinline__ float largest(float4 x) { return fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)); }
// The power of two that brings `top` to 2^14 .. 2^15 (2^127 at most), and its reciprocal (an exact one, subnormal perhaps).
__device__ __forceinline__ void powers(float top, float* up, float* down) {
  const int e = static_cast<int>(__float_as_uint(top) >> 23);
  const int biased = top == 0.0f ? 127 : min(254, 268 - e);
  *up = __uint_as_float(static_cast<unsigned>(biased) << 23);
  *down = biased == 254 ? __uint_as_float(1u << 22) : __uint_as_float(static_cast<unsigned>(254 - biased) << 23);
}
// A pair as hi and lo pairs; what is not finite is so in hi, and 0 in lo.
__device__ __forceinline__ void split2(float a, float b, uint32_t* hi, uint32_t* lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(fabsf(a) <= 65504.0f ? a - f.x : 0.0f, fabsf(b) <= 65504.0f ? b - f.y : 0.0f);
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split4(float4 x, float4 up, uint2* hi, uint2* lo) {
  split2(x.x * up.x, x.y * up.y, &hi->x, &lo->x);
  split2(x.z * up.z, x.w * up.w, &hi->y, &lo->y);
}
// A slot of K or V: kKeys rows of a sequence, one KV head. K gets one power of two, V one for each column.
template <int D, bool VALUES>
__device__ __forceinline__ void split_tile(const PromptArgs& A, const PromptPieces& W, int slot, int kv) {
  constexpr int kKeys = prompt_piece_keys(D);
  constexpr int kLanes = D == 96 ? 32 : D / 4, kGroups = kThreads / kLanes, kEach = kKeys / kGroups, kRowLanes = kLanes < 32 ? kLanes : 32;
  __shared__ int sh_sequence, sh_back, sh_shared;
  __shared__ __align__(16) float sh_col[kGroups][D], sh_up[D];
  __shared__ unsigned sh_most, sh_least;
  const int tid = threadIdx.x;
  if (tid == 0) {
    sh_sequence = INT_MAX;
    sh_back = sh_shared = 0;
    sh_most = 0u;
    sh_least = 0x7F800000u;
  }
  __syncthreads();
  for (int b = tid; b < A.batch; b += kThreads) {
    const int s0 = A.starts[b], s1 = A.starts[b + 1];
    if (s1 < s0) sh_back = 1;
    if (s0 < 0 || s1 <= s0 || s1 > A.tokens) continue;
    const int at = slot - (s0 / kKeys + b);
    if (at >= 0 && at <= (s1 - s0 - 1) / kKeys) atomicMin(&sh_sequence, b);  // one, but for sequences that overlap
  }
  __syncthreads();
  const int b = sh_sequence;
  const size_t place = static_cast<size_t>(slot) * A.kv_heads + kv;
  int* const owner = VALUES ? W.v_owner : W.k_owner;
  if (b == INT_MAX) {
    if (tid == 0) owner[place] = -1;
    return;
  }
  const int s0 = A.starts[b], n = A.starts[b + 1] - s0, j0 = (slot - (s0 / kKeys + b)) * kKeys;
  if (sh_back) {  // bounds that never go back have no rows in common
    const int r0 = s0 + j0, r1 = s0 + min(n, j0 + kKeys);
    for (int o = tid; o < A.batch; o += kThreads) {
      const int o0 = A.starts[o], o1 = A.starts[o + 1];
      if (o != b && o0 >= 0 && o1 <= A.tokens && max(o0, r0) < min(o1, r1)) sh_shared = 1;
    }
    __syncthreads();
    if (sh_shared) {
      if (tid == 0) owner[place] = -2;
      return;
    }
  }
  const int l = tid % kLanes, g = tid / kLanes;
  const bool in = 4 * l < D;
  const size_t col = static_cast<size_t>(kv) * D + 4 * l;
  const float* const x = static_cast<const float*>(VALUES ? A.v : A.k);
  const long long stride = VALUES ? A.v_stride : A.k_stride;
  // twice over the tile (the second time from L2): kept, its values would take most of a thread's registers
  auto row_at = [&](int i) {
    const int j = j0 + i * kGroups + g;
    return in && j < n ? *reinterpret_cast<const float4*>(x + (static_cast<size_t>(s0) + j) * stride + col) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  float4 top = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float most = 0.0f, least = INFINITY;
#pragma unroll 4
  for (int i = 0; i < kEach; ++i) {
    const float4 a = finite_abs(row_at(i));
    top = make_float4(fmaxf(top.x, a.x), fmaxf(top.y, a.y), fmaxf(top.z, a.z), fmaxf(top.w, a.w));
    float row = largest(a);  // of the row, or of half of it at head size 256
#pragma unroll
    for (int o = kRowLanes / 2; o > 0; o >>= 1) row = fmaxf(row, __shfl_xor_sync(0xffffffffu, row, o));
    most = fmaxf(most, row);
    if (row > 0.0f) least = fminf(least, row);
  }
  if (l % kRowLanes == 0) {
    atomicMax(&sh_most, __float_as_uint(most));
    atomicMin(&sh_least, __float_as_uint(least));
  }
  if (in) *reinterpret_cast<float4*>(&sh_col[g][4 * l]) = top;
  __syncthreads();
  const bool apart = __uint_as_float(sh_most) > 4096.0f * __uint_as_float(sh_least);  // its rows differ much in size
  for (int c = tid; c < D; c += kThreads) {
    float t = 0.0f, down;
    if (VALUES) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i) t = fmaxf(t, sh_col[i][c]);
    } else {
      t = __uint_as_float(sh_most);
    }
    powers(t, &sh_up[c], &down);
    if (VALUES)
      W.v_power[place * D + c] = down;
    else if (c == 0)
      W.k_power[place] = apart ? -down : down;
  }
  if (tid == 0) {
    owner[place] = b;
    if (VALUES) W.v_most[place] = apart ? __uint_as_float(sh_most) : 0.0f;
  }
  __syncthreads();
  if (!in) return;
  const float4 up = *reinterpret_cast<const float4*>(&sh_up[4 * l]);
  const size_t row = static_cast<size_t>(A.kv_heads) * D, piece = static_cast<size_t>(A.tokens) * row;
#pragma unroll 4
  for (int i = 0; i < kEach; ++i) {
    const int j = j0 + i * kGroups + g;
    if (j >= n) break;
    uint2 hi, lo;
    split4(row_at(i), up, &hi, &lo);
    __half* const to = (VALUES ? W.v : W.k) + (static_cast<size_t>(s0) + j) * row + col;
    *reinterpret_cast<uint2*>(to) = hi;
    *reinterpret_cast<uint2*>(to + piece) = lo;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 4) prompt_split_kernel(const __grid_constant__ PromptArgs A, const __grid_constant__ PromptPieces W) {
  const unsigned rest = blockIdx.x >> 1;
  if (blockIdx.x & 1)
    split_tile<D, true>(A, W, rest / A.kv_heads, rest % A.kv_heads);
  else
    split_tile<D, false>(A, W, rest / A.kv_heads, rest % A.kv_heads);
}

template <int D>
cudaError_t launch(const PromptArgs& a, const PromptPieces& w, cudaStream_t s) {
  const long long blocks = 2ll * w.slots * a.kv_heads;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  prompt_split_kernel<D><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, w);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_split(const PromptArgs& a, const PromptPieces& w, cudaStream_t s) {
  switch (a.dim) {
    case 64: return launch<64>(a, w, s);
    case 96: return launch<96>(a, w, s);
    case 128: return launch<128>(a, w, s);
    default: return launch<256>(a, w, s);
  }
}

}  // namespace xq
