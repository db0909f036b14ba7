// Norms of queries and keys for each head with the position rotation, in one
// pass over both.
//
// Mathematics: r = x * w / sqrt(mean(x^2) + eps); pair (a, b) of r turns by
// the angle of its position. An angle is position * turns mod 2^64 in units of
// 2^-64 of a full turn: an integer product whose overflow drops whole turns, so
// it is exact at any position for the turns it is given, which a table rounds
// to 2^-65 (at position 2^40 that is 2e-7; position * frequency in fp32 is off
// by 0.004 at 131071). What is left after the nearest quarter turn is at most an eighth
// of a turn, known to 2^-34 of one.
//
// A lane has 8 elements of a row, so a row of 64, 128 or 256 takes 8, 16 or 32
// lanes (96: 12 of 16) and its sum 3 to 5 shuffles; a warp takes several heads
// of one token, as the cosines are the token's. Element i and its partner
// i + rot / 2 lie the same number of lanes apart for all (rot is a multiple of
// 16), neighbouring pairs in one lane. Weights go into the cosines and sines,
// which the block's threads work out once a token.
//
// What bounds it: HBM, 82 % of the copy rate (16383 tokens of 32 + 8 heads of
// 128, fp32 to bf16: 90 us, 5.6 TB/s; 327 us with the angles worked out by every
// warp); with few tokens the launch and one round trip (2.9 to 3.1 us).
#include "ops_common.cuh"

namespace xq {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
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

// Cosine and sine of a phase, 2^-64 of a full turn: the nearest quarter turn, and an angle of at most pi / 4 beside it by the
// power series (the first terms left out are 2e-9 and 2e-9 of 1).
__device__ __forceinline__ void cos_sin(uint64_t phase, float* c, float* s) {
  const uint64_t quarter = (phase + (1ull << 61)) >> 62;
  const int rest = static_cast<int>(static_cast<int64_t>(phase - (quarter << 62)) >> 30);  // in 2^-34 of a turn
  const float x = static_cast<float>(rest) * 3.657295198e-10f, x2 = x * x;                   // 2 pi 2^-34
  float sn = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, 1/7!
  sn = fmaf(sn, x2, 8.3333333e-3f);
  sn = fmaf(sn, x2, -0.16666667f);
  sn = fmaf(sn * x2, x, x);
  float cn = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);  // 1/10!, 1/8!
  cn = fmaf(cn, x2, -1.3888889e-3f);
  cn = fmaf(cn, x2, 4.1666667e-2f);
  cn = fmaf(cn, x2, -0.5f);
  cn = fmaf(cn, x2, 1.0f);
  const float a = quarter & 1 ? sn : cn, b = quarter & 1 ? cn : sn;
  *c = (quarter + 1) & 2 ? -a : a;
  *s = quarter & 2 ? -b : b;
}

struct RopeGrid {
  int span;         // row groups a warp takes
  int warps_token;  // 1, 2, 4 or a multiple of the warps of a block
  int tokens_block;
  bool wide_x, wide_y;
};

// W: lanes a row.
template <int XT, int YT, int W>
__global__ void __launch_bounds__(kThreads, 3) qk_rope_kernel(const __grid_constant__ RopeArgs A, const RopeGrid G) {
  constexpr int kGroups = 32 / W;
  __shared__ __align__(16) float sh_cos[kWarps][128], sh_sin[kWarps][128];  // of the block's tokens
  const int lane = threadIdx.x & 31, li = lane & (W - 1), group = lane / W;
  const long long warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long token = warp / G.warps_token, token0 = static_cast<long long>(blockIdx.x) * kWarps / G.warps_token;
  // row groups: q's, then k's
  const int groups_q = (A.side[0].heads + kGroups - 1) / kGroups, groups = groups_q + (A.side[1].heads + kGroups - 1) / kGroups;
  int next = static_cast<int>(warp - token * G.warps_token) * G.span;
  const int end = min(next + G.span, groups);
  const int e0 = 8 * li, half = A.rot / 2;
  const bool in = e0 < A.dim && token < A.tokens, turns = e0 < A.rot;
  float x[kRowsAhead][8];
  // rows of one side from row group `first` on; `n` of them at most
  auto load = [&](const RopeSide& side, int first, int n) {
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const int row = (first + u) * kGroups + group;
      if (in && u < n && row < side.heads && XQ_CHECKED(token < A.tokens && e0 + 8 <= A.dim, kChkRope))
        load8<XT>(side.x, static_cast<size_t>(token) * side.x_stride + static_cast<size_t>(row) * A.dim + e0, G.wide_x, x[u]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) x[u][i] = 0.0f;
    }
  };
  // the first rows are on their way while the angles are worked out
  if (next < groups_q)
    load(A.side[0], next, min(end, groups_q) - next);
  else
    load(A.side[1], next - groups_q, end - next);
  for (int i = threadIdx.x; i < G.tokens_block * half; i += kThreads) {
    const int t = i / half, pair = i - t * half;
    if (token0 + t < A.tokens) {
      float c, s;
      cos_sin(static_cast<uint64_t>(A.positions[token0 + t]) * A.turns[pair], &c, &s);
      sh_cos[t][pair] = c * A.magnitude;
      sh_sin[t][pair] = s * A.magnitude;
    }
  }
  __syncthreads();
  if (token >= A.tokens) return;
  bool loaded = true;
#pragma unroll 1
  for (int z = 0; z < 2; ++z) {
    const RopeSide& side = A.side[z];
    const int before = z ? groups_q : 0, stop = z ? end : min(end, groups_q);
    if (next >= stop) continue;
    // y = inv * (x * near + (its partner's x) * other), weights in the factors: w cos, and the partner's w times sin, negated
    // for a pair's first element; the lane that has the partners
    float near[8], other[8];
    int from = lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) near[i] = side.weight && in ? side.weight[e0 + i] : 1.0f;
    if (turns && in) {
      const float *const c = sh_cos[token - token0], *const s = sh_sin[token - token0];
      if (A.pairs) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float cn = c[(e0 + i) / 2], sn = s[(e0 + i) / 2], w0 = near[i], w1 = near[i + 1];
          other[i] = -(w1 * sn), other[i + 1] = w0 * sn;
          near[i] = w0 * cn, near[i + 1] = w1 * cn;
        }
      } else {
        const bool high = e0 >= half;
        from = high ? lane - half / 8 : lane + half / 8;
        const int at = high ? e0 - half : e0, partner = high ? at : e0 + half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float sn = side.weight ? side.weight[partner + i] * s[at + i] : s[at + i];
          other[i] = high ? sn : -sn;
          near[i] *= c[at + i];
        }
      }
    }
    const float over_dim = 1.0f / static_cast<float>(A.dim);
    for (; next < stop; next += kRowsAhead) {
      if (!loaded) load(side, next - before, stop - next);
      loaded = false;
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        if (next + u >= stop) break;
        const int row = (next - before + u) * kGroups + group;
        float inv = 1.0f;
        if (side.weight) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(x[u][i], x[u][i], ss);
#pragma unroll
          for (int o = W / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          inv = rsqrtf(fmaf(ss, over_dim, A.eps));
        }
        float y[8];
        if (A.pairs) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = turns ? fmaf(x[u][i], near[i], x[u][i ^ 1] * other[i]) : x[u][i] * near[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float partner = __shfl_sync(0xffffffffu, x[u][i], from);
            y[i] = turns ? fmaf(x[u][i], near[i], partner * other[i]) : x[u][i] * near[i];
          }
        }
        if (side.weight) {
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] *= inv;
        }
        if (in && row < side.heads)
          store8<YT>(side.y, static_cast<size_t>(token) * side.y_stride + static_cast<size_t>(row) * A.dim + e0, G.wide_y, y);
      }
    }
    next = stop;
  }
}

bool on16(const void* p, long long stride, int bytes, bool one) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (one || (stride * bytes) % 16 == 0);
}

template <int XT, int YT>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
  const int lanes = a.dim <= 64 ? 8 : a.dim <= 128 ? 16 : 32, groups = 32 / lanes;
  const int row_groups = (a.side[0].heads + groups - 1) / groups + (a.side[1].heads + groups - 1) / groups;
  RopeGrid g;
  // warps a token: one takes all its rows where that fills the device (three blocks an SM); few tokens are shared out. Measured
  // with 1, 2, 4, 8, 16, 24: 16383 tokens of 32 + 8 heads 90, 94, 114, 165, 208, 278 us, 257 tokens of 12 + 2 heads 5.3,
  // 3.8, 2.9, 2.9, 4.2, 4.8, one token of 32 + 8 heads 9.4, 6.0, 4.5, 4.1, 3.2, 3.0.
  const long long enough = 152 * 3 * kWarps;
  g.warps_token = 1;
  while (g.warps_token < row_groups && static_cast<long long>(g.warps_token) * a.tokens < enough)
    g.warps_token = g.warps_token < kWarps ? 2 * g.warps_token : g.warps_token + kWarps;
  g.span = (row_groups + g.warps_token - 1) / g.warps_token;
  g.tokens_block = g.warps_token < kWarps ? kWarps / g.warps_token : 1;
  const int xb = kv_elt_bytes(a.type), yb = kv_elt_bytes(a.y_type);
  g.wide_x = on16(a.side[0].x, a.side[0].x_stride, xb, a.tokens == 1) && on16(a.side[1].x, a.side[1].x_stride, xb, a.tokens == 1);
  g.wide_y = on16(a.side[0].y, a.side[0].y_stride, yb, a.tokens == 1) && on16(a.side[1].y, a.side[1].y_stride, yb, a.tokens == 1);
  const long long warps = static_cast<long long>(a.tokens) * g.warps_token;
  const unsigned blocks = static_cast<unsigned>((warps + kWarps - 1) / kWarps);
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
