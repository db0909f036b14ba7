// Norms of queries and keys for each head with the position rotation, in one
// pass over both.
//
// Mathematics: r = x * w / sqrt(mean(x^2) + eps); pair (a, b) of r turns by
// the angle of its position. An angle is position * turns mod 2^64 in units of
// 2^-64 of a full turn: an integer product whose overflow drops whole turns, so
// it is exact at any position (position * frequency in fp32 is off by 0.004
// at 131071). What is left after the nearest quarter turn is at most an eighth
// of a turn and enters sincospi with 2^-33.
//
// A lane has 8 elements of a row, so a row of 64, 128 or 256 takes 8, 16 or 32
// lanes (96: 12 of 16) and its sum 3 to 5 shuffles; a warp takes several heads
// of one token, as the cosines are the token's. Element i and its partner
// i + rot / 2 lie the same number of lanes apart for all (rot is a multiple of
// 16), neighbouring pairs in one lane.
#include "ops_common.cuh"

namespace xq {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsAhead = 4;  // rows a lane group loads before it works on them

// 8 elements from p + at; wide: a 16-byte boundary.
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, size_t at, bool wide, float (&x)[8]) {
  if constexpr (TYPE == kF32) {
    if (wide) {
      const float4* const f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
      const float4 a = f[0], b = f[1];
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
      return;
    }
  } else if (wide) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (TYPE == kF16)
        f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      else
        f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = load_elt<TYPE>(p, at + i);
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, size_t at, bool wide, const float (&x)[8]) {
  if constexpr (TYPE == kF32) {
    if (wide) {
      float4* const f = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
      f[0] = make_float4(x[0], x[1], x[2], x[3]);
      f[1] = make_float4(x[4], x[5], x[6], x[7]);
      return;
    }
  } else if (wide) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (TYPE == kF16) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) store_elt<TYPE>(p, at + i, x[i]);
}

__device__ __forceinline__ void cos_sin(uint64_t phase, float* c, float* s) {
  const uint64_t quarter = (phase + (1ull << 61)) >> 62;
  const int rest = static_cast<int>(static_cast<int64_t>(phase - (quarter << 62)) >> 30);  // -2^31 .. 2^31 - 1: an eighth
  float sn, cn;
  sincospif(static_cast<float>(rest) * 1.16415321826934814453125e-10f, &sn, &cn);  // 2^-33 half turns
  *c = quarter == 0 ? cn : quarter == 1 ? -sn : quarter == 2 ? -cn : sn;
  *s = quarter == 0 ? sn : quarter == 1 ? cn : quarter == 2 ? -sn : -cn;
}

struct RopeGrid {
  int span;         // row groups a warp takes
  int warps_token;
  bool wide_x, wide_y;
};

// W: lanes a row.
template <int XT, int YT, int W>
__global__ void __launch_bounds__(kThreads) qk_rope_kernel(const __grid_constant__ RopeArgs A, const RopeGrid G) {
  constexpr int kGroups = 32 / W;
  const int lane = threadIdx.x & 31, li = lane & (W - 1), group = lane / W;
  const long long warp = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const long long token = warp / G.warps_token;
  if (token >= A.tokens) return;
  const int heads = A.side[0].heads, rows = heads + A.side[1].heads;
  const int first = static_cast<int>(warp - token * G.warps_token) * G.span;  // row group
  const int e0 = 8 * li, half = A.rot / 2;
  const bool in = e0 < A.dim, turns = e0 < A.rot;
  // the 8 elements' cosines and sines, these negated for a pair's first element; the lane that has their partners
  float cs[8], sn[8];
  int from = lane;
  if (turns) {
    const uint64_t position = static_cast<uint64_t>(A.positions[token]);
    if (A.pairs) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float c, s;
        cos_sin(position * A.turns[e0 / 2 + i], &c, &s);
        cs[2 * i] = cs[2 * i + 1] = c * A.magnitude;
        sn[2 * i + 1] = s * A.magnitude;
        sn[2 * i] = -sn[2 * i + 1];
      }
    } else {
      const bool high = e0 >= half;
      from = high ? lane - half / 8 : lane + half / 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float c, s;
        cos_sin(position * A.turns[(high ? e0 - half : e0) + i], &c, &s);
        cs[i] = c * A.magnitude;
        sn[i] = (high ? s : -s) * A.magnitude;
      }
    }
  }
  for (int b = 0; b < G.span; b += kRowsAhead) {
    float x[kRowsAhead][8];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int row = (first + b + u) * kGroups + group;
      const bool there = in && b + u < G.span && row < rows;
      const RopeSide& side = A.side[row < heads ? 0 : 1];
      const size_t at = static_cast<size_t>(token) * side.x_stride + static_cast<size_t>(row < heads ? row : row - heads) * A.dim + e0;
      if (there && XQ_CHECKED(token < A.tokens && e0 + 8 <= A.dim, kChkRope))
        load8<XT>(side.x, at, G.wide_x, x[u]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      if (b + u >= G.span) break;
      const int row = (first + b + u) * kGroups + group;
      const RopeSide& side = A.side[row < heads ? 0 : 1];
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[u][i], x[u][i], ss);
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (side.weight && in) {
        const float inv = 1.0f / sqrtf(ss / static_cast<float>(A.dim) + A.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = x[u][i] * inv * side.weight[e0 + i];
      }
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float near = x[u][i ^ 1];
        const float other = __shfl_sync(0xffffffffu, x[u][i], from);
        y[i] = turns ? fmaf(x[u][i], cs[i], (A.pairs ? near : other) * sn[i]) : x[u][i];
      }
      if (in && row < rows)
        store8<YT>(side.y, static_cast<size_t>(token) * side.y_stride + static_cast<size_t>(row < heads ? row : row - heads) * A.dim + e0,
                   G.wide_y, y);
    }
  }
}

bool on16(const void* p, long long stride, int bytes, bool one) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (one || (stride * bytes) % 16 == 0);
}

template <int XT, int YT>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int lanes = a.dim <= 64 ? 8 : a.dim <= 128 ? 16 : 32, groups = 32 / lanes;
  const int row_groups = (a.side[0].heads + a.side[1].heads + groups - 1) / groups;
  RopeGrid g;
  g.span = 1;
  g.warps_token = (row_groups + g.span - 1) / g.span;
  const int xb = kv_elt_bytes(a.type), yb = kv_elt_bytes(a.y_type);
  g.wide_x = on16(a.side[0].x, a.side[0].x_stride, xb, a.tokens == 1) && on16(a.side[1].x, a.side[1].x_stride, xb, a.tokens == 1);
  g.wide_y = on16(a.side[0].y, a.side[0].y_stride, yb, a.tokens == 1) && on16(a.side[1].y, a.side[1].y_stride, yb, a.tokens == 1);
  const long long warps = static_cast<long long>(a.tokens) * g.warps_token;
  const unsigned blocks = static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32));
  if (lanes == 8)
    qk_rope_kernel<XT, YT, 8><<<blocks, kThreads, 0, s>>>(a, g);
  else if (lanes == 16)
    qk_rope_kernel<XT, YT, 16><<<blocks, kThreads, 0, s>>>(a, g);
  else
    qk_rope_kernel<XT, YT, 32><<<blocks, kThreads, 0, s>>>(a, g);
  return cudaGetLastError();
}

template <int XT>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  return a.y_type == kF32 ? launch<XT, kF32>(a, s) : a.y_type == kF16 ? launch<XT, kF16>(a, s) : launch<XT, kBF16>(a, s);
}

}  // namespace

cudaError_t launch_qk_rope(const RopeArgs& a, cudaStream_t s) {
  return a.type == kF32 ? launch<kF32>(a, s) : a.type == kF16 ? launch<kF16>(a, s) : launch<kBF16>(a, s);
}

cudaError_t take_rope_check(unsigned int* code) { return take_check_word(code); }

}  // namespace xq
