// What the prompt attention's kernels share: items of work, one row by itself, operand helpers.
#pragma once

#include "ops_common.cuh"
#include "xq_common.cuh"
#include "xq_ptx.cuh"

namespace xq {

constexpr int kPromptRows = 128;  // of a row tile
constexpr long long kPromptWait = 1ll << 32;
// A wait's limit in clocks: `base`, and what slow work of the CTA that it may be a wait for can take. That is up to 32 rows by
// themselves, one behind the other (one_row; 32 keys take up to 18000 clocks at head size 128, with all SMs at it; 131000 are allowed),
// and a search of the next item (at most 304 levels, as each has an item at least; 32 sequences are a memory round trip, some 600
// clocks; 2048 are allowed). (Limits that begin anew while some word in shared memory counts on cost 5 to 11 % in the loops that poll.)
inline long long prompt_wait_limit(const PromptArgs& a, long long base) {
  return base + 1024ll * a.tokens * a.dim + 2048ll * 306 * (a.batch / 32 + 1);
}

struct PromptTileArgs {
  PromptArgs a;
  int pack;      // query heads of a KV head in a tile's rows
  int tokens_tile;  // of a row tile: 128 / pack
  int units;     // head units: heads / pack
  CUtensorMap q, k, v;
  long long wait;  // clocks that a wait lasts at most
  bool withhold;   // test hook: no copies
  float4* sums;  // 16-bit rows: a CTA's row tiles' sums of outputs over runs of key tiles, [dim / 4][128 rows], and references, [128]
};

// 16-bit rows: keys of a tile, and tiles whose outputs the tensor cores add up. 16, 32, 64 tiles, all: 12287 tokens 934, 891, 876,
// 862 us; lost towards 0 at 32767 keys 0, 6e-6, 1.9e-5, 1.9e-4, where fp16's half step is 4.9e-4.
constexpr int kPromptTileKeys = 128, kPromptRun = 32;
// CTAs of a call with `tiles` row tiles each: no more than items, which are whole groups of tokens and a part of one for each sequence.
inline int prompt_tile_grid(const PromptTileArgs& p, int tiles) {
  const long long items = (p.a.tokens / (tiles * p.tokens_tile) + static_cast<long long>(p.a.batch)) * p.units;
  return static_cast<int>(items < 152 ? (items < 1 ? 1 : items) : 152);
}

#ifdef XQ_PROMPT_TILE_IMPL

namespace {

__device__ unsigned int g_prompt_error;  // invalid indices
__device__ unsigned int g_prompt_wait;   // a wait that ran out
constexpr int kRows = kPromptRows;
constexpr int kWalkKept = 2;  // sequences a lane keeps in registers

struct Item {
  int first, n;     // the sequence's first row and its rows
  int sequence;
  int place;        // of row tile 0's first token
  int head;         // first query head
  int half;         // of V's columns, where a CTA takes half of them
  int begin[2], end[2];  // key tiles of the row tiles
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  uint32_t d;
  if constexpr (TYPE == kF16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
        "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

// 4 elements from p + at.
template <int TYPE>
__device__ __forceinline__ float4 load4(const void* p, size_t at) {
  if constexpr (TYPE == kF32) {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
    if constexpr (TYPE == kF16) {
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
      return make_float4(a.x, a.y, b.x, b.y);
    } else {
      return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                         __uint_as_float(v.y & 0xFFFF0000u));
    }
  }
}

// One row by one warp, in fp32: 32 keys' scores at a time, a lane each, then their values, lanes over the head's elements.
// Sums go 32 keys at a time, with what an addition rounds off kept beside them, as a long row's would be far off (fp32, 131071 equal
// weights one after the other: 5e-4).
// Writes columns c0 .. c1 - 1, multiples of 32 or, with lanes left out, of 16.
template <int TYPE, int D>
__device__ __noinline__ void one_row(const PromptArgs& A, int first, int place, int head, int c0, int c1) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, kv = head / (A.heads / A.kv_heads);
  const size_t token = static_cast<size_t>(first) + place, q0 = token * A.q_stride + static_cast<size_t>(head) * D;
  float o[E], o_rest[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = o_rest[e] = 0.0f;
  // sum += x
  auto add = [](float& sum, float& rest, float x) {
    const float next = sum + x, kept = next - sum;
    rest += (sum - (next - kept)) + (x - kept);
    sum = next;
  };
  const float cs = A.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.0f, l_rest = 0.0f;
  for (int j0 = A.window && place >= A.window ? place - A.window + 1 : 0; j0 <= place; j0 += 32) {
    const int n = min(32, place - j0 + 1);
    float s = -INFINITY;
    if (lane < n) {
      const size_t k0 = (static_cast<size_t>(first) + j0 + lane) * A.k_stride + static_cast<size_t>(kv) * D;
      s = 0.0f;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        const float4 q = load4<TYPE>(A.q, q0 + c), k = load4<TYPE>(A.k, k0 + c);
        s = fmaf(q.w, k.w, fmaf(q.z, k.z, fmaf(q.y, k.y, fmaf(q.x, k.x, s))));
      }
      s = __fmul_rn(s, cs);
    }
    float top = s;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float next = fmaxf(m, top);
    // an infinite score above all others leaves NaN, as infinity minus infinity does; none above minus infinity, no weight
    const float f = m == next ? 1.0f : exp2f(m - next);
    const float w = lane >= n || (s == -INFINITY && next == s) ? 0.0f : exp2f(s - next);
    m = next;
    float sum = w;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (sum != sum) {  // a NaN among the scores is the whole row's
      l = sum;
      break;
    }
    l *= f, l_rest *= f;
    add(l, l_rest, sum);
    float part[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f, o_rest[e] *= f, part[e] = 0.0f;
    const size_t v0 = (static_cast<size_t>(first) + j0) * A.v_stride + static_cast<size_t>(kv) * D + lane;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
#pragma unroll
      for (int e = 0; e < E; ++e) part[e] = fmaf(wj, load_elt<TYPE>(A.v, v0 + j * A.v_stride + 32 * e), part[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) add(o[e], o_rest[e], part[e]);
  }
  const size_t row = token * A.heads + head;
  if (XQ_IN(row, static_cast<size_t>(A.tokens) * A.heads, kChkPromptRow))
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (lane + 32 * e >= c0 && lane + 32 * e < c1) store_elt<TYPE>(A.out, row * D + lane + 32 * e, (isfinite(o[e]) ? o[e] + o_rest[e] : o[e]) / (l + l_rest));
}

// Sequence b's rows and their number; 0, and recorded, if its bounds are no range of the call's rows.
__device__ __forceinline__ int sequence(const PromptArgs& A, int b, int* first) {
  if (b >= A.batch) return 0;
  const int s0 = A.starts[b], s1 = A.starts[b + 1];
  *first = s0;
  if (s0 < 0 || s1 < s0 || s1 > A.tokens) {
    atomicCAS(&g_prompt_error, 0u, kOpsBadStart);
    return 0;
  }
  return s1 - s0;
}

// Items in descending order of their work. An item is a head unit of a group of `step` tokens of a sequence; group L of any
// sequence has the keys up to it, so all groups L of all sequences (a level) are alike. A warp walks down the levels,
// counting the sequences that reach each.
struct Walk {
  int level;        // of the current one
  long long before; // groups in the levels before it
  int count;        // sequences that reach it
  int n[kWalkKept], first[kWalkKept];  // of sequences lane, lane + 32, ...: a level costs no memory round trip
};
// Rows (and the first) of the lane's i-th sequence.
__device__ __forceinline__ int walk_sequence(const PromptArgs& A, const Walk& w, int i, int* first) {
  int n = 0;
  if (i >= kWalkKept) return sequence(A, i * 32 + (threadIdx.x & 31), first);
#pragma unroll
  for (int k = 0; k < kWalkKept; ++k)
    if (k == i) n = w.n[k], *first = w.first[k];
  return n;
}
__device__ __forceinline__ int walk_count(const PromptArgs& A, const Walk& w, int level, int step) {
  const int beyond = level * step;
  int c = 0;
#pragma unroll
  for (int k = 0; k < kWalkKept; ++k) c += w.n[k] > beyond;
  for (int i = kWalkKept; i * 32 < A.batch; ++i) {
    int first;
    c += sequence(A, i * 32 + (threadIdx.x & 31), &first) > beyond;
  }
  return __reduce_add_sync(0xffffffffu, c);
}
__device__ __forceinline__ void walk_begin(const PromptArgs& A, int step, Walk& w) {
  int most = 0;
#pragma unroll
  for (int k = 0; k < kWalkKept; ++k) {
    w.first[k] = 0;
    w.n[k] = sequence(A, k * 32 + (threadIdx.x & 31), &w.first[k]);
    most = max(most, w.n[k]);
  }
  for (int i = kWalkKept; i * 32 < A.batch; ++i) {
    int first;
    most = max(most, sequence(A, i * 32 + (threadIdx.x & 31), &first));
  }
  most = __reduce_max_sync(0xffffffffu, most);
  w.level = (most + step - 1) / step - 1;
  w.before = 0;
  w.count = w.level >= 0 ? walk_count(A, w, w.level, step) : 0;
}
// The item of this rank; false behind the last. Ranks come in ascending order. KEYS: of a tile.
template <int KEYS, int HALVES>
__device__ __forceinline__ bool next_item(const PromptTileArgs& P, int tiles, long long rank, Walk& w, Item& it) {
  const PromptArgs& A = P.a;
  const int step = tiles * P.tokens_tile, units = P.units * HALVES;
  const long long group = rank >> 32 ? rank / units : static_cast<unsigned>(rank) / static_cast<unsigned>(units);
  const int unit = static_cast<int>(rank - group * units);
  while (w.level >= 0 && group >= w.before + w.count) {
    w.before += w.count;
    --w.level;
    if (w.level >= 0) w.count = walk_count(A, w, w.level, step);
  }
  if (w.level < 0) return false;
  int left = static_cast<int>(group - w.before);  // sequences to pass over, of those that reach the level
  for (int i = 0; i * 32 < A.batch; ++i) {
    int first = 0;
    const int n = walk_sequence(A, w, i, &first);
    unsigned reach = __ballot_sync(0xffffffffu, n > w.level * step);
    const int c = __popc(reach);
    if (left >= c) {
      left -= c;
      continue;
    }
    for (; left > 0; --left) reach &= reach - 1;
    const int at = __ffs(reach) - 1;
    it.first = __shfl_sync(0xffffffffu, first, at);
    it.n = __shfl_sync(0xffffffffu, n, at);
    it.sequence = i * 32 + at;
    break;
  }
  it.place = w.level * step;
  it.head = unit / HALVES * P.pack;
  it.half = unit % HALVES;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int p0 = it.place + r * P.tokens_tile, p1 = min(p0 + P.tokens_tile, it.n) - 1;  // first and last row's
    const int k0 = A.window ? max(0, p0 - A.window + 1) : 0;
    it.begin[r] = r < tiles && p1 >= p0 ? k0 / KEYS : 0;
    it.end[r] = r < tiles && p1 >= p0 ? p1 / KEYS + 1 : 0;
  }
  return true;
}

// Whether some row of row tile r does not see some key of a tile from `key` on.
template <int KEYS>
__device__ __forceinline__ bool masked(const PromptTileArgs& P, int place, int key) {
  return key + KEYS > place + 1 || (P.a.window && key < place + P.tokens_tile - P.a.window);
}

// Bit 15 of each half: it is an infinity or NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  constexpr uint32_t field = TYPE == kF16 ? 0x7C007C00u : 0x7F807F80u, one = TYPE == kF16 ? 0x04000400u : 0x00800080u;
  return ((w & field) + one) & 0x80008000u;
}


}  // namespace

#endif  // XQ_PROMPT_TILE_IMPL

}  // namespace xq
