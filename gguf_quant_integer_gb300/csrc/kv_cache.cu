// Writing the quantized KV cache and reading it back (block formulas and the
// page layout in the public header).
//
// Both kernels move each byte once. What bounds them: launch latency up to a
// few hundred tokens (one token 3 us for a write and a read); then, for reads,
// HBM (16383 tokens of 8 heads of 128, Q8_0 to fp32: 28 us, 6.1 TB/s; 65536
// Q4_0 tokens to bf16: 52 us, 6.6 TB/s); for writes the instructions, some 25
// a value in all, as fp32's 16-byte pieces hold four values only (fp32 to Q8_0
// 32 us, 5.3 TB/s, 68 % of the issue slots; bf16 to Q4_0 29 us, 2.9 TB/s).
// A 32-value block belongs to a group of neighbouring lanes of one warp, each
// with 16 bytes of float values (8 lanes for fp32, 4 for 16-bit types): the
// loads and stores of a warp are then whole 128-byte lines, and the block's
// maximum takes two or three shuffles and no shared memory. A thread handles
// the same block of K and of V, which doubles the loads in flight.
#include <climits>
#include <type_traits>

#include "kv_common.cuh"
#include "xq_common.cuh"

namespace xq {
namespace {

__device__ unsigned int g_kv_cache_error;

constexpr int kThreads = 256;

// A token's row of K (and of V) is row_blocks blocks of 32 in heads order; a
// warp takes `span` pieces of it, each as many blocks as it has lane groups.
struct RowArgs {
  KvView c;
  const int64_t* slots;
  unsigned warps;         // in this launch
  unsigned warps_row;     // a token's
  unsigned span;          // pieces of a row a warp
  unsigned row_blocks;    // heads * dim / 32
};
struct WriteArgs {
  RowArgs r;
  const void* x[2];       // K and V rows
  long long stride[2];    // elements between tokens
  bool wide;              // every 16-byte piece of x is 16-byte aligned
};
struct ReadArgs {
  RowArgs r;
  void* y[2];
};

// This thread's blocks: the first, and the step to the next (blocks a piece).
struct BlockAt {
  unsigned hb, h, b;      // of the row; head and block of the head
  __device__ __forceinline__ BlockAt(unsigned first, unsigned nb) : hb(first), h(first / nb), b(first - first / nb * nb) {}
  __device__ __forceinline__ void step(unsigned by, unsigned nb) {
    hb += by;
    b += by;
    while (b >= nb) {
      b -= nb;
      ++h;
    }
  }
};

template <typename X>
__device__ __forceinline__ float to_float(X v);
template <>
__device__ __forceinline__ float to_float(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_float(__half v) {
  return __half2float(v);
}
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

// 16 bytes of row elements as floats.
template <typename X, int N>
__device__ __forceinline__ void load_piece(const X* p, bool wide, float (&f)[N]) {
  static_assert(N * sizeof(X) == 16, "a piece is 16 bytes");
  union {
    uint4 u;
    X e[N];
  } r;
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.u.x), "=r"(r.u.y), "=r"(r.u.z), "=r"(r.u.w)
                 : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.e[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = to_float<X>(r.e[i]);
}

// The page row of a slot, or false (recorded) if the cache has no such slot.
__device__ __forceinline__ bool slot_row(const KvView& c, long long slot, long long* page, int* row) {
  *page = slot >> c.page_shift;
  *row = static_cast<int>(slot & ((1 << c.page_shift) - 1));
  if (slot < 0) return false;
  if (*page >= c.n_pages) {
    atomicCAS(&g_kv_cache_error, 0u, kKvBadSlot);
    return false;
  }
  return true;
}

// round(x / d), halves away from zero, clamped; a quotient that is not a
// number (0 / 0 never reaches here; inf / inf) gives 0.
__device__ __forceinline__ int quant(float x, float d, float low, float top) {
  float y = roundf(__fdiv_rn(x, d));
  y = (y != y) ? 0.0f : y;
  return static_cast<int>(fminf(fmaxf(y, low), top));
}

// The larger magnitude (a NaN if there is one).
__device__ __forceinline__ float max_abs(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}

// fp16(top / 127). The product with 1 / 127 is within 3 steps of the quotient,
// so fp16 rounds both alike unless the product lies that near the middle of two
// fp16 numbers (one block in a thousand) or below fp16's normal ones.
__device__ __forceinline__ __half scale_q8(float top) {
  float q = top * (1.0f / 127.0f);
  if (!(q >= 6.1035156e-5f) || ((__float_as_uint(q) - 0x0FFCu) & 0x1FFFu) <= 8u) q = __fdiv_rn(top, 127.0f);
  return __float2half_rn(q);
}

// The codes of N values, a byte each (q + 128, or q + 8 for BITS = 4), by
// x * (1 / d), within 2^-15 of x / d: adding 1.5 * 2^23 + offset leaves the
// nearest whole number in the low bits. What is left is which side of a half
// the quotient is on.
//   16-bit inputs: with x and d of 11 bits, a quotient is a half or 2^-12 from
//     one at least (2 x - (2 n + 1) d is a multiple of the smaller of 2 ulp(x)
//     and ulp(d), 2^-11 d or more), so a step of 2^-13 away from zero takes
//     the halves outwards and no other quotient past one.
//   fp32: a piece with a product within 1e-4 of a half is divided out, about
//     one warp in forty.
// CLAMP: Q8_0's quotients pass 127.5 only where d is below fp16's normal numbers.
// 4 to 8 instructions a value where a division takes 25.
template <int BITS, int N, bool CLAMP>
__device__ __forceinline__ void codes_by_product(const float (&f)[N], float d, uint32_t (&code)[N / 4]) {
  constexpr float low = BITS == 8 ? -127.0f : -8.0f, top = BITS == 8 ? 127.0f : 7.0f;
  constexpr float shift = 12582912.0f + (BITS == 8 ? 128.0f : 8.0f);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  float off = 0.0f;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    uint32_t b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float y = f[4 * i + k] * inv;
      if (N == 8) y = __fadd_rn(y, copysignf(1.220703125e-4f, y));
      if (CLAMP) y = fminf(fmaxf(y, low), top);
      const float z = __fadd_rn(y, shift);
      if (N == 4) off = max_abs(off, __fadd_rn(y, -__fadd_rn(z, -shift)));
      b[k] = __float_as_uint(z);
    }
    code[i] = prmt(prmt(b[0], b[1], 0x0040u), prmt(b[2], b[3], 0x0040u), 0x5410u);
  }
  if (N == 4 && !(off < 0.4999f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned q = quant(f[i], d, low, top) + (BITS == 8 ? 128 : 8);
      code[i / 4] = (i & 3) ? (code[i / 4] | (q << (8 * (i & 3)))) : q;
    }
  }
}
template <int BITS, int N>
__device__ __forceinline__ void codes_of(const float (&f)[N], float d, uint32_t (&code)[N / 4]) {
  constexpr uint32_t zeros = BITS == 8 ? 0x80808080u : 0x08080808u;
  if (BITS == 8 && d >= 6.1035156e-5f && d <= 65504.0f) {
    codes_by_product<BITS, N, false>(f, d, code);
  } else if (!(fabsf(d) <= 65504.0f) || d == 0.0f) {  // finite / infinite, and what is not a number: 0
#pragma unroll
    for (int i = 0; i < N / 4; ++i) code[i] = zeros;
  } else {
    codes_by_product<BITS, N, true>(f, d, code);
  }
}

// The block of N values in each of 32 / N neighbouring lanes: scale, and this
// lane's codes as stored. Q4_0: lanes of the block's first half return the
// bytes of elements (own, own + 16), the others nothing of use.
template <int BITS, int N>
__device__ __forceinline__ float quantize_piece(const float (&f)[N], int lane, uint32_t (&code)[N / 4]) {
  constexpr int G = 32 / N;
  __half dh;
  if (BITS == 8) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) top = max_abs(top, f[i]);
#pragma unroll
    for (int o = 1; o < G; o *= 2) top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, o));
    dh = scale_q8(top);
  } else {
    float m = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i)
      if (__float_as_uint(fabsf(f[i])) > __float_as_uint(fabsf(m))) m = f[i];
#pragma unroll
    for (int o = 1; o < G; o *= 2) {
      const float other = __shfl_xor_sync(0xffffffffu, m, o);
      const unsigned a = __float_as_uint(fabsf(m)), b = __float_as_uint(fabsf(other));
      // elements are in lane order, so of two equal magnitudes the lower lane's is the first
      if (b > a || (b == a && (lane & o))) m = other;
    }
    dh = __float2half_rn(m * -0.125f);
  }
  const float d = __half2float(dh);
  codes_of<BITS, N>(f, d, code);
  if (BITS == 4) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) code[i] |= __shfl_xor_sync(0xffffffffu, code[i], G / 2) << 4;
  }
  return d;
}

template <int BITS, typename X>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const __grid_constant__ WriteArgs A) {
  constexpr int N = 16 / sizeof(X), G = 32 / N, kBlocks = 32 / G;  // blocks of a warp's piece
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned w = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int lane = static_cast<int>(threadIdx.x & 31), piece = lane % G;
  if (w >= A.r.warps) return;
  const unsigned t = w / A.r.warps_row, first = (w - t * A.r.warps_row) * A.r.span * kBlocks;
  const unsigned nb = A.r.c.dim / 32, end = min(first + A.r.span * kBlocks, A.r.row_blocks);
  BlockAt at(first + lane / G, nb);
  const X* x[2];
  float f[2][N];
  auto load = [&](unsigned hb) {
#pragma unroll
    for (int z = 0; z < 2; ++z) load_piece<X, N>(x[z] + hb * 32, A.wide, f[z]);
  };
#pragma unroll
  for (int z = 0; z < 2; ++z) x[z] = static_cast<const X*>(A.x[z]) + static_cast<long long>(t) * A.stride[z] + piece * N;
  load(at.hb < end ? at.hb : first);  // beside the slot, whatever it turns out to be
  long long page;
  int row;
  if (!slot_row(A.r.c, A.r.slots[t], &page, &row)) return;
  uint8_t* const base = A.r.c.k + page * A.r.c.page_bytes;
  const long long v_off = A.r.c.v - A.r.c.k;
  for (unsigned from = first; from < end; from += kBlocks) {
    const bool live = at.hb < end;
    const long long line = (static_cast<long long>(at.h) << A.r.c.page_shift) + row;
    const unsigned b = at.b;
    uint32_t code[2][N / 4];
    float d[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) d[z] = quantize_piece<BITS, N>(f[z], lane, code[z]);
    at.step(kBlocks, nb);
    if (from + kBlocks < end) load(at.hb < end ? at.hb : first);
    if (!live || !XQ_IN(line, static_cast<long long>(A.r.c.heads) << A.r.c.page_shift, kChkKvRow)) continue;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      uint8_t* const pool = z ? base + v_off : base;
      // Q8_0: every lane N bytes; Q4_0: the lanes of the first half N bytes (two elements each)
      if (BITS == 8 || piece < G / 2) {
        uint8_t* to = pool + line * A.r.c.row_bytes + b * (4 * BITS) + piece * N;
        if (N == 8)
          *reinterpret_cast<uint2*>(to) = make_uint2(code[z][0], code[z][N / 4 - 1]);
        else
          *reinterpret_cast<uint32_t*>(to) = code[z][0];
      }
      if (piece == 0) *reinterpret_cast<__half*>(pool + A.r.c.scale_off + (line * nb + b) * 2) = __float2half_rn(d[z]);
    }
  }
}

// 16 bytes of float values from N codes.
template <typename Y, int N>
__device__ __forceinline__ void store_piece(Y* p, const float (&f)[N]) {
  union {
    uint4 u;
    Y e[N];
  } r;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (sizeof(Y) == 4)
      r.e[i] = f[i];
    else if constexpr (sizeof(Y) == 2 && std::is_same<Y, __half>::value)
      r.e[i] = __float2half_rn(f[i]);
    else
      r.e[i] = __float2bfloat16_rn(f[i]);
  }
  *reinterpret_cast<uint4*>(p) = r.u;
}

// A thread takes N code bytes of K and of V: N values of a Q8_0 block, or the
// N low and N high halves (elements j and j + 16) of a Q4_0 block.
template <int BITS, typename Y>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ ReadArgs A) {
  constexpr int N = 16 / sizeof(Y), G = 4 * BITS / N, kBlocks = 32 / G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const unsigned w = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int lane = static_cast<int>(threadIdx.x & 31), piece = lane % G;
  if (w >= A.r.warps) return;
  const unsigned t = w / A.r.warps_row, first = (w - t * A.r.warps_row) * A.r.span * kBlocks;
  const unsigned nb = A.r.c.dim / 32, end = min(first + A.r.span * kBlocks, A.r.row_blocks);
  BlockAt at(first + lane / G, nb);
  long long page;
  int row;
  const bool ok = slot_row(A.r.c, A.r.slots[t], &page, &row);
  const uint8_t* const base = A.r.c.k + page * A.r.c.page_bytes;
  const long long v_off = A.r.c.v - A.r.c.k;
  constexpr int kAhead = 2;  // pieces a thread has in flight
  for (unsigned from = first; from < end; from += kAhead * kBlocks) {
    uint32_t code[kAhead][2][N / 4];
    float d[kAhead][2];
    unsigned hb[kAhead];
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      hb[p] = at.hb;
      const long long line = (static_cast<long long>(at.h) << A.r.c.page_shift) + row;
      const bool there = ok && at.hb < end && XQ_IN(line, static_cast<long long>(A.r.c.heads) << A.r.c.page_shift, kChkKvRow);
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        d[p][z] = 0.0f;
        code[p][z][0] = code[p][z][N / 4 - 1] = 0u;
        if (!there) continue;
        const uint8_t* const pool = z ? base + v_off : base;
        const uint8_t* const src = pool + line * A.r.c.row_bytes + at.b * (4 * BITS) + piece * N;
        if (N == 8) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
          code[p][z][0] = v.x;
          code[p][z][N / 4 - 1] = v.y;
        } else {
          code[p][z][0] = __ldg(reinterpret_cast<const uint32_t*>(src));
        }
        d[p][z] = __half2float(
            __ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(pool + A.r.c.scale_off + (line * nb + at.b) * 2))));
      }
      at.step(kBlocks, nb);
    }
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      if (hb[p] >= end) continue;
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        Y* const to = static_cast<Y*>(A.y[z]) + (static_cast<size_t>(t) * A.r.row_blocks + hb[p]) * 32 + piece * N;
        constexpr float off = BITS == 8 ? 8388736.0f : 8388616.0f;  // 2^23 + 128, 2^23 + 8
#pragma unroll
        for (int half = 0; half < (BITS == 8 ? 1 : 2); ++half) {
          float f[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            // a byte u as the float 2^23 + u; int-to-float conversions would keep the slow pipe busy
            const uint32_t v = BITS == 8 ? code[p][z][i / 4] : (code[p][z][i / 4] >> (4 * half)) & 0x0F0F0F0Fu;
            f[i] = ok ? __fmul_rn(d[p][z], __fadd_rn(__uint_as_float(prmt(v, 0x4B000000u, 0x7440u + (i & 3))), -off)) : 0.0f;
          }
          store_piece<Y, N>(to + 16 * half, f);
        }
      }
    }
  }
}

template <typename K, typename Args>
cudaError_t launch(K kernel, Args& A, long long tokens, int lanes, cudaStream_t s) {
  const unsigned blocks = 32 / lanes, pieces = (A.r.row_blocks + blocks - 1) / blocks;
  // Few tokens: a warp a piece, for the least latency. Many: a warp several
  // pieces of a row, which share the slot's and the addresses' arithmetic
  // (16383 fp32 tokens of 8 heads of 128, Q8_0: writes 43.3, 32.6, 31.8 and
  // 31.9 us with 1, 4, 8 and 16 pieces, reads 42.7, 27.9, 29.3 and 29.4).
  constexpr unsigned kMost = std::is_same<Args, WriteArgs>::value ? 8 : 4;
  const long long most = 64LL * kNumSMs;
  unsigned span = tokens * pieces > 2 * most ? kMost : tokens * pieces > most ? 2 : 1;
  span = span < pieces ? span : pieces;
  A.r.span = span;
  A.r.warps_row = (pieces + span - 1) / span;
  A.r.warps = static_cast<unsigned>(tokens) * A.r.warps_row;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((A.r.warps + kThreads / 32 - 1) / (kThreads / 32));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  g_kv_launched.store(true, std::memory_order_relaxed);
  return cudaLaunchKernelEx(&cfg, kernel, A);
}

// Tokens per launch: warp indices stay within 31 bits.
int tokens_per_launch(const KvView& c) {
  const long long most = (1LL << 27) / (static_cast<long long>(c.heads) * (c.dim / 32));
  return most < 1 ? 1 : most > INT_MAX ? INT_MAX : static_cast<int>(most);
}

}  // namespace

cudaError_t launch_kv_write(const KvView& c, int bits, int x_type, const void* k, long long k_stride, const void* v,
                            long long v_stride, const int64_t* slots, int n_tokens, cudaStream_t s) {
  const int eb = kv_elt_bytes(x_type), step = tokens_per_launch(c);
  WriteArgs A;
  A.r.c = c;
  A.stride[0] = k_stride;
  A.stride[1] = v_stride;
  A.r.row_blocks = static_cast<unsigned>(c.heads) * (c.dim / 32);
  A.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | static_cast<uintptr_t>(k_stride * eb) |
             static_cast<uintptr_t>(v_stride * eb)) & 15u) == 0;
  for (long long t0 = 0; t0 < n_tokens; t0 += step) {
    const long long n = n_tokens - t0 < step ? n_tokens - t0 : step;
    A.x[0] = static_cast<const char*>(k) + t0 * k_stride * eb;
    A.x[1] = static_cast<const char*>(v) + t0 * v_stride * eb;
    A.r.slots = slots + t0;
    cudaError_t e;
    if (x_type == kF32)
      e = bits == 8 ? launch(kv_write_kernel<8, float>, A, n, 8, s) : launch(kv_write_kernel<4, float>, A, n, 8, s);
    else if (x_type == kF16)
      e = bits == 8 ? launch(kv_write_kernel<8, __half>, A, n, 4, s) : launch(kv_write_kernel<4, __half>, A, n, 4, s);
    else
      e = bits == 8 ? launch(kv_write_kernel<8, __nv_bfloat16>, A, n, 4, s) : launch(kv_write_kernel<4, __nv_bfloat16>, A, n, 4, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_kv_read(const KvView& c, int bits, const int64_t* slots, int n_tokens, int y_type, void* k, void* v,
                           cudaStream_t s) {
  const int eb = kv_elt_bytes(y_type), step = tokens_per_launch(c);
  const long long row = static_cast<long long>(c.heads) * c.dim * eb;
  ReadArgs A;
  A.r.c = c;
  A.r.row_blocks = static_cast<unsigned>(c.heads) * (c.dim / 32);
  for (long long t0 = 0; t0 < n_tokens; t0 += step) {
    const long long n = n_tokens - t0 < step ? n_tokens - t0 : step;
    A.y[0] = static_cast<char*>(k) + t0 * row;
    A.y[1] = static_cast<char*>(v) + t0 * row;
    A.r.slots = slots + t0;
    cudaError_t e;  // code bytes a thread: 4 for fp32, 8 for 16-bit values
    if (y_type == kF32)
      e = bits == 8 ? launch(kv_read_kernel<8, float>, A, n, 8, s) : launch(kv_read_kernel<4, float>, A, n, 4, s);
    else if (y_type == kF16)
      e = bits == 8 ? launch(kv_read_kernel<8, __half>, A, n, 4, s) : launch(kv_read_kernel<4, __half>, A, n, 2, s);
    else
      e = bits == 8 ? launch(kv_read_kernel<8, __nv_bfloat16>, A, n, 4, s) : launch(kv_read_kernel<4, __nv_bfloat16>, A, n, 2, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t take_kv_cache_error(unsigned int* code) { return take_record(g_kv_cache_error, code); }
cudaError_t take_kv_cache_check(unsigned int* code) { return take_check_word(code); }

}  // namespace xq
