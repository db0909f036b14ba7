// fp32 rows of Q, K and V as two fp16 numbers each, for prompt attention (see prompt_pieces.cuh).
//
// x 2^s = hi + lo: hi = fp16(x 2^s), lo = fp16(x 2^s - hi), with 2^s from the largest finite magnitude of the row (Q, K) or
// of the column of a tile of keys (V), which comes to 2^14 .. 2^15: 22 bits for everything down to 2^-17 of that, and an
// error of 2^-39 of it below. An element that is not finite is one in hi, and 0 in lo. One pass over memory.
#include <climits>

#include "prompt_pieces.cuh"

namespace xq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kRowsWarp = 4;

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
__device__ __forceinline__ void split4(float4 x, float4 up, uint2* hi, uint2* lo) {
  const float v[4] = {x.x * up.x, x.y * up.y, x.z * up.z, x.w * up.w};
  __half h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = __float2half_rn(v[i]);
    l[i] = fabsf(v[i]) <= 65504.0f ? __float2half_rn(v[i] - __half2float(h[i])) : __ushort_as_half(0);
  }
  *hi = make_uint2(__half_as_ushort(h[0]) | static_cast<uint32_t>(__half_as_ushort(h[1])) << 16,
                   __half_as_ushort(h[2]) | static_cast<uint32_t>(__half_as_ushort(h[3])) << 16);
  *lo = make_uint2(__half_as_ushort(l[0]) | static_cast<uint32_t>(__half_as_ushort(l[1])) << 16,
                   __half_as_ushort(l[2]) | static_cast<uint32_t>(__half_as_ushort(l[3])) << 16);
}

// Rows of Q, then of K: a warp a row.
template <int D>
__device__ __forceinline__ void split_rows(const PromptArgs& A, const PromptPieces& W, long long first) {
  constexpr int kE = D == 256 ? 2 : 1;  // pieces of 4 elements a lane
  const int lane = threadIdx.x & 31;
  const long long rows_q = static_cast<long long>(A.tokens) * A.heads, rows = rows_q + static_cast<long long>(A.tokens) * A.kv_heads;
  float4 x[kRowsWarp][kE];
#pragma unroll
  for (int u = 0; u < kRowsWarp; ++u) {
    const long long r = first + u;
    const bool key = r >= rows_q;
    const int heads = key ? A.kv_heads : A.heads;
    const long long i = key ? r - rows_q : r, token = i / heads;
    const float* const from = static_cast<const float*>(key ? A.k : A.q) + token * (key ? A.k_stride : A.q_stride) + (i - token * heads) * D;
#pragma unroll
    for (int z = 0; z < kE; ++z)
      x[u][z] = r < rows && lane * 4 < D ? *reinterpret_cast<const float4*>(from + z * 128 + lane * 4) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
#pragma unroll
  for (int u = 0; u < kRowsWarp; ++u) {
    const long long r = first + u;
    if (r >= rows) return;
    const bool key = r >= rows_q;
    const int heads = key ? A.kv_heads : A.heads;
    const long long i = key ? r - rows_q : r, token = i / heads;
    float top = 0.0f;
#pragma unroll
    for (int z = 0; z < kE; ++z) top = fmaxf(top, largest(finite_abs(x[u][z])));
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    float up, down;
    powers(top, &up, &down);
    __half* const to = (key ? W.k : W.q) + i * D;
    const size_t piece = static_cast<size_t>(A.tokens) * heads * D;
    if (lane * 4 < D) {
#pragma unroll
      for (int z = 0; z < kE; ++z) {
        uint2 hi, lo;
        split4(x[u][z], make_float4(up, up, up, up), &hi, &lo);
        *reinterpret_cast<uint2*>(to + z * 128 + lane * 4) = hi;
        *reinterpret_cast<uint2*>(to + piece + z * 128 + lane * 4) = lo;
      }
    }
    if (lane == 0) {
      if (key)
        W.k_power[(i - token * heads) * A.tokens + token] = down;
      else
        W.q_power[i] = down;
    }
  }
}

// A slot of V: kKeys rows of a sequence, one KV head, W columns.
template <int D>
__device__ __forceinline__ void split_values(const PromptArgs& A, const PromptPieces& W, int slot, int kv, int half) {
  constexpr int kKeys = prompt_piece_keys(D), kHalves = prompt_piece_halves(D), kV = D / kHalves;
  constexpr int kLanes = kV == 64 ? 16 : 32, kGroups = kThreads / kLanes, kEach = kKeys / kGroups;
  __shared__ int sh_sequence;
  __shared__ __align__(16) float sh_col[kGroups][kV], sh_up[kV];
  __shared__ unsigned sh_most, sh_least;
  const int tid = threadIdx.x;
  if (tid == 0) {
    sh_sequence = INT_MAX;
    sh_most = 0u;
    sh_least = 0x7F800000u;
  }
  __syncthreads();
  for (int b = tid; b < A.batch; b += kThreads) {
    const int s0 = A.starts[b], s1 = A.starts[b + 1];
    if (s0 < 0 || s1 <= s0 || s1 > A.tokens) continue;
    const int at = slot - (s0 / kKeys + b);
    if (at >= 0 && at <= (s1 - s0 - 1) / kKeys) atomicMin(&sh_sequence, b);  // one, but for sequences that overlap
  }
  __syncthreads();
  const int b = sh_sequence;
  const size_t place = static_cast<size_t>(slot) * A.kv_heads + kv;
  if (b == INT_MAX) {
    if (tid == 0) W.owner[place * kHalves + half] = -1;
    return;
  }
  const int s0 = A.starts[b], n = A.starts[b + 1] - s0, j0 = (slot - (s0 / kKeys + b)) * kKeys;
  const int l = tid % kLanes, g = tid / kLanes;
  const bool in = 4 * l < kV;
  const size_t col = static_cast<size_t>(kv) * D + half * kV + 4 * l;
  float4 x[kEach], top = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = j0 + i * kGroups + g;
    x[i] = in && j < n ? *reinterpret_cast<const float4*>(static_cast<const float*>(A.v) + (static_cast<size_t>(s0) + j) * A.v_stride + col)
                       : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  float most = 0.0f, least = INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const float4 a = finite_abs(x[i]);
    top = make_float4(fmaxf(top.x, a.x), fmaxf(top.y, a.y), fmaxf(top.z, a.z), fmaxf(top.w, a.w));
    float row = largest(a);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) row = fmaxf(row, __shfl_xor_sync(0xffffffffu, row, o));
    most = fmaxf(most, row);
    if (row > 0.0f) least = fminf(least, row);
  }
  if (l == 0) {
    atomicMax(&sh_most, __float_as_uint(most));
    atomicMin(&sh_least, __float_as_uint(least));
  }
  if (in) *reinterpret_cast<float4*>(&sh_col[g][4 * l]) = top;
  __syncthreads();
  for (int c = tid; c < kV; c += kThreads) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) t = fmaxf(t, sh_col[i][c]);
    float down;
    powers(t, &sh_up[c], &down);
    W.v_power[place * D + half * kV + c] = down;
  }
  if (tid == 0) W.owner[place * kHalves + half] = __uint_as_float(sh_most) > 4096.0f * __uint_as_float(sh_least) ? -2 : b;
  __syncthreads();
  if (!in) return;
  const float4 up = *reinterpret_cast<const float4*>(&sh_up[4 * l]);
  const size_t row = static_cast<size_t>(A.kv_heads) * D, piece = static_cast<size_t>(A.tokens) * row;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int j = j0 + i * kGroups + g;
    if (j >= n) break;
    uint2 hi, lo;
    split4(x[i], up, &hi, &lo);
    __half* const to = W.v + (static_cast<size_t>(s0) + j) * row + col;
    *reinterpret_cast<uint2*>(to) = hi;
    *reinterpret_cast<uint2*>(to + piece) = lo;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) prompt_split_kernel(const __grid_constant__ PromptArgs A, const __grid_constant__ PromptPieces W,
                                                                unsigned value_blocks) {
  constexpr int kHalves = prompt_piece_halves(D);
  if (blockIdx.x < value_blocks) {
    const unsigned half = blockIdx.x % kHalves, rest = blockIdx.x / kHalves;
    split_values<D>(A, W, rest / A.kv_heads, rest % A.kv_heads, half);
  } else {
    split_rows<D>(A, W, (static_cast<long long>(blockIdx.x - value_blocks) * kWarps + (threadIdx.x >> 5)) * kRowsWarp);
  }
}

template <int D>
cudaError_t launch(const PromptArgs& a, const PromptPieces& w, cudaStream_t s) {
  const long long values = static_cast<long long>(w.slots) * a.kv_heads * prompt_piece_halves(D);
  const long long rows = static_cast<long long>(a.tokens) * (a.heads + a.kv_heads), each = kWarps * kRowsWarp;
  const long long blocks = values + (rows + each - 1) / each;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  prompt_split_kernel<D><<<static_cast<unsigned>(blocks), kThreads, 0, s>>>(a, w, static_cast<unsigned>(values));
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
