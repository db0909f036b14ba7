// Attention over the quantized KV cache: one CTA per query row.
//
// The plainest form: each warp takes every fourth key, a lane holds dim / 32
// of the row's elements, and each warp keeps the running maximum m and sum l
// of its own keys' softmax, so that one pass over the keys suffices:
//   m' = max(m, s),  l = l e^(m-m') + e^(s-m'),  o = o e^(m-m') + e^(s-m') v.
#include "kv_common.cuh"

namespace xq {
namespace {

__device__ unsigned int g_kv_attn_error;

constexpr int kWarps = 4;

__device__ __forceinline__ float load_elt(const void* p, int type, size_t i) {
  return type == kF32   ? static_cast<const float*>(p)[i]
         : type == kF16 ? __half2float(static_cast<const __half*>(p)[i])
                        : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

template <int BITS>
__global__ void __launch_bounds__(32 * kWarps) kv_attn_row_kernel(const __grid_constant__ KvAttnArgs A) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % A.q_heads, i = blockIdx.x / A.q_heads % A.n_q, b = blockIdx.x / A.q_heads / A.n_q;
  const int kvh = h / A.group, nb = A.c.dim / 32, mask = (1 << A.c.page_shift) - 1;
  int n = A.lens[b];
  const int most = A.max_pages << A.c.page_shift;
  if (n > most) {
    n = most;
    atomicCAS(&g_kv_attn_error, 0u, kKvBadLen);
  }
  n = n < 0 ? 0 : n;
  const int pos = kv_pos(A.prefix_len, n, A.n_q, i);
  const int first = A.window && pos - A.window + 1 > 0 ? pos - A.window + 1 : 0;
  const size_t at = static_cast<size_t>(blockIdx.x) * A.c.dim;
  float q[8], o[8];
  for (int e = 0; e < nb; ++e) {
    q[e] = load_elt(A.q, A.type, at + 32 * e + lane) * A.scale;
    o[e] = 0.0f;
  }
  float m = -1e30f, l = 0.0f;
  for (int j = first + warp; j <= pos; j += kWarps) {
    const bool pre = j < A.prefix_len;
    const int t = pre ? j : j - A.prefix_len;
    const int page = pre ? A.prefix_pages[t >> A.c.page_shift]
                         : A.pages[static_cast<size_t>(b) * A.page_stride + (t >> A.c.page_shift)];
    if (page < 0 || page >= A.c.n_pages) {
      atomicCAS(&g_kv_attn_error, 0u, kKvBadPage);
      continue;
    }
    const long long line = (static_cast<long long>(kvh) << A.c.page_shift) + (t & mask);
    const uint8_t* kp = A.c.k + page * A.c.page_bytes;
    const uint8_t* vp = A.c.v + page * A.c.page_bytes;
    float s = 0.0f, v[8];
    for (int e = 0; e < nb; ++e) {
      int kc, vc;
      if (BITS == 8) {
        kc = kp[line * A.c.row_bytes + 32 * e + lane] - 128;
        vc = vp[line * A.c.row_bytes + 32 * e + lane] - 128;
      } else {
        kc = ((kp[line * A.c.row_bytes + 16 * e + (lane & 15)] >> (lane & 16 ? 4 : 0)) & 15) - 8;
        vc = ((vp[line * A.c.row_bytes + 16 * e + (lane & 15)] >> (lane & 16 ? 4 : 0)) & 15) - 8;
      }
      const long long so = A.c.scale_off + (line * nb + e) * 2;
      s += q[e] * (kc * __half2float(*reinterpret_cast<const __half*>(kp + so)));
      v[e] = vc * __half2float(*reinterpret_cast<const __half*>(vp + so));
    }
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float top = fmaxf(m, s), keep = expf(m - top), p = expf(s - top);
    l = l * keep + p;
    for (int e = 0; e < nb; ++e) o[e] = o[e] * keep + p * v[e];
    m = top;
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][256];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int e = 0; e < nb; ++e) so[warp][32 * e + lane] = o[e];
  __syncthreads();
  float top = sm[0];
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  for (int e = threadIdx.x; e < A.c.dim; e += 32 * kWarps) {
    float sum = 0.0f, acc = 0.0f;
    for (int w = 0; w < kWarps; ++w) {
      const float f = expf(sm[w] - top);
      sum += sl[w] * f;
      acc += so[w][e] * f;
    }
    const float y = sum > 0.0f || sum != sum ? acc / sum : 0.0f;
    if (A.type == kF32)
      static_cast<float*>(A.out)[at + e] = y;
    else if (A.type == kF16)
      static_cast<__half*>(A.out)[at + e] = __float2half_rn(y);
    else
      static_cast<__nv_bfloat16*>(A.out)[at + e] = __float2bfloat16_rn(y);
  }
}

}  // namespace

size_t kv_attn_workspace(const KvAttnArgs&, int) { return 0; }

cudaError_t launch_kv_attn(const KvAttnArgs& a, int bits, void*, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * a.n_q * a.q_heads);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bits == 8 ? cudaLaunchKernelEx(&cfg, kv_attn_row_kernel<8>, a) : cudaLaunchKernelEx(&cfg, kv_attn_row_kernel<4>, a);
}

cudaError_t take_kv_attn_error(unsigned int* code) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv_attn_error, sizeof(v));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_kv_attn_error, &z, sizeof(z));
  *code = v;
  return e;
}
cudaError_t take_kv_attn_check(unsigned int* code) { return take_check_word(code); }

}  // namespace xq
