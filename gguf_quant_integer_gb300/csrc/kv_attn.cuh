// Attention over the quantized KV cache for few query rows a KV head: a
// split-KV kernel on the warp-level tensor cores, and the join of its parts.
//
// Mathematics. A CTA holds up to R query rows that read one KV head (grouped
// heads and neighbouring query tokens) and streams that head's keys through
// four independent warps, 16 keys at a time:
//   scores    s = c * sum_b dk_b * (codes_b . q_b)   over the 32-value blocks b
//   weights   p = 2^(s - e),   w_b = p * dv_b
//   outputs   o = sum_keys w_b * codes_b,   l = sum_keys p
// The codes are small integers, exact in fp16, so both products run on
// m16n8k16 with the codes as the A operand (16 keys x 16 elements, then 16
// elements x 16 keys) and block scales applied in fp32: dk to a block's sum,
// dv to the weight. q and w enter as fp16: 16-bit queries as one number,
// fp32 ones as two (hi + lo, 22 bits, one column each), so that a column pair
// adds up to the fp32 product. fp32 outputs are summed in fp32 additions every
// kAttnRun tiles.
// e is a running reference per query instead of the exact running maximum: it
// moves only when some weight w would pass 2^15 (it then restarts at 2^11), which also keeps w inside
// fp16 whatever the sizes of V. One vote per 16 keys; the rescale is rare.
// A V scale that is not finite stops there too: its block becomes NaN in the
// rows that see the key, and the scale 0 for the products.
// Score columns become weight columns by movmatrix, whose 8x8 transpose takes
// an accumulator's (key, query pair) registers to the B operand.
//
// What bounds it. One key of dim 128 is 272 bytes of Q8_0 (144 of Q4_0) and
// 512 multiply-adds a query; an SM has about 24 bytes a clock to itself,
// against 4 instructions. A warp's 16 keys cost some 420 instructions, so long
// Q8_0 caches are bound by HBM and Q4_0's nearly as much by instructions: 64
// sequences, 230000 tokens in all, 8 KV heads, fp32: 84 us, 5.9 TB/s with the
// join; one sequence of 131071 Q4_0 tokens, bf16: 38 us, 4.0 TB/s, of which 4
// are the join and 5 pass before the first tile's products. Short calls are
// bound by latency: one sequence of 97 tokens 5.5 us (10000 clocks: 3000 to
// find the work, 3000 for queries and the first tile, 1000 to 1500 a tile).
//
// Work split. Sequences differ in length, so the keys of all (sequence, KV
// head, row chunk) pairs are one line of 64-key units that is cut evenly over
// the resident CTAs. A CTA that does not cover a pair alone writes a partial
// (o, e, l); the CTA where the pair begins leaves a record and the join kernel
// adds the parts in order, so results do not depend on timing.
#pragma once

#include <climits>
#include <type_traits>

#include "kv_common.cuh"
#include "xq_common.cuh"
#include "xq_ptx.cuh"

namespace xq {

constexpr int kAttnWarps = 4;
// A weight's second fp16 number, w - hi, is stored 2^11 larger (its column has
// accumulators of its own, scaled back at the end): small weights, whose hi
// is a subnormal fp16, keep their bits.
constexpr float kLoUp = 2048.0f;
constexpr float kWeightTop = 32768.0f, kWeightLow = 1.220703125e-4f;  // 2^15, 2^-13
// The reference of a row that has seen no key: below every finite score, and itself finite (a masked score is -infinity, and
// the difference of two would not be a number).
constexpr float kNoKey = -3.402823466e38f;
constexpr int kAttnUnit = 16 * kAttnWarps;  // keys a unit
// Units of time that a CTA spends on a pair besides its keys (queries, page
// ids, filling the pipeline, merging): the cut counts them, or CTAs with many
// short sequences would finish last. With two n-tiles more, as each row's
// query is split. (64 sequences of 211 to 8192 tokens: 87.9, 84.0, 84.0, 84.3,
// 84.6 us with 2, 3, 4, 5, 6; two n-tiles, 16 sequences of 300 to 4099: 18.7,
// 18.5, 18.6, 18.6 us with 4, 5, 6, 8, and 8 KV heads' 1000-token prefix for 8
// sequences 16.7, 16.7, 16.5, 16.5.)
constexpr int kAttnHead = 4, kAttnHead2 = 6;
// Pairs that can have no more units than this are not cut. A CTA takes about
// 0.5 us a unit, the join's launch 4 us (one 97-token sequence, 8 KV heads:
// 8.5 us cut, 6.6 us whole).
constexpr int kAttnWhole = 4;
// The same for the own pages of a call with a prefix, whose pass runs beside
// the prefix's and then needs no join of its own.
constexpr int kAttnWholeOwn = 16;

// Kernel arguments. A pair's rows are `tokens` query tokens x group heads;
// token and head select q's and out's row. Own pages: sequence b has the
// tokens b * n_q .. + n_q - 1. Prefix (flat): one sequence of prefix_len keys
// whose tokens are all batch * n_q of the call.
struct SplitArgs {
  KvView c;
  int type, group, q_heads, n_q;
  int seqs;     // sequences (1 when flat)
  int rows;     // query rows of a pair
  int chunks;   // row chunks of a pair
  bool flat;
  const void* q;
  const int32_t* pages;
  int page_stride, max_pages;
  const int32_t* lens;
  int prefix_len;
  float scale;
  int window;
  long long units;  // upper bound of the launch's units
  int ctas;         // of the launch: as many as run at a time, or one a unit
  bool whole;       // pairs are not cut: no join
  bool counted;     // whole, and each counts as one unit of the line
  int head;         // units that a pair counts besides its keys
  float* part_o;    // [2 * ctas][R][dim]
  float* part_el;   // [2 * ctas][R][2]
  int4* record;     // [ctas]: sequence, head * chunks + chunk, last CTA (or -1)
  // Results: out rows (o / l in the call's type). A call with a prefix runs
  // the own pages first, whose pass stores o and (e, l) of each (token, query
  // head), and then the prefix, whose pass merges them.
  void* out;
  float* pre_o;
  float* pre_el;
  bool store, merge;
  bool late;  // starts beside the call's first pass: waits for it only where it merges, and at its end
  // What the checked build measures against: rows of partial results and records that the workspace holds.
  long long part_rows;
  int records;
};

template <int BITS, int D, bool EX, int NP, int NT>
struct SplitShape {
  static constexpr int NB = D / 32;
  static constexpr int kRow = D * BITS / 8;
  static constexpr int kChunks = kRow / 16;          // 16-byte chunks a row
  static constexpr int kSteps = (kChunks + 1) / 2;   // copies of 32 chunks a tile
  static constexpr bool kPow2 = (kChunks & (kChunks - 1)) == 0;
  // The swizzle of step x's rows (x * 32 / kChunks further down) against the
  // first step's, on the chunk's byte offset.
  static constexpr uint32_t turn(int x) {
    return kChunks == 8 ? (x & 1) * 64u : kChunks == 16 ? (x & 3) * 32u : 0u;
  }
  static constexpr int R = NT * 8 / NP;              // query rows of a CTA
  static constexpr int kCodes = 16 * kRow;
  static constexpr int kScales = 16 * NB * 2;
  static constexpr int kStage = 2 * (kCodes + kScales);
  // Stages of 16 keys a warp: about 13 KB (three 4.25 KB stages of Q8_0 at dim
  // 128), so that 12 warps an SM keep 100 KB in flight. (18 KB: 4 us more on
  // the batch above.)
  // Two where a third and the fp32 sums below would leave the SM one CTA.
  static constexpr int kStages = EX && kStage > 8192 ? 2 : kStage * 3 > 13312 ? 3 : 13312 / kStage > 6 ? 6 : 13312 / kStage;
  static constexpr int kWarpBytes = kStages * kStage > R * D * 4 ? kStages * kStage : R * D * 4;
  // fp32: a warp's sums (a lane's own, four floats a step) and their references.
  static constexpr int kSums = R * D * 4, kSumBytes = EX ? kSums + NT * 32 * 4 : 0;
  static constexpr int kSmem = kAttnWarps * (kWarpBytes + kSumBytes);
  // A warp's results fit one stage: the next pair's first tiles can be on
  // their way into the others while the warps are merged.
  static constexpr bool kOverlap = R * D * 4 <= kStage;
  // Resident CTAs an SM, by registers (168 a thread, 255 with two n-tiles): a
  // fourth (128 registers, some spilled) costs more than its latency hiding
  // gives (64-sequence Q8_0 fp32 batch 92 against 86 us, 131071-token Q4_0
  // bf16 sequence 46 against 42 us; two n-tiles, 16 sequences of 5 tokens: 28
  // against 26 us).
  static constexpr int kCtas = D == 256 || NT == 2 ? 2 : 3;
};

// Tiles of a warp after which fp32 outputs leave the tensor cores' accumulators for sums in shared memory. An accumulator
// cuts off what an fp32 addition would round, and always towards 0: some 1.2e-8 of the output a tile, 6e-6 over the 512 tiles a
// warp of 64 sequences behind 32768 keys, where the same in fp32 operations has 5e-7. With 32 tiles the error is 3.5e-7 to
// 5.8e-7 at any length. 64 sequences of 8000 keys, fp32: 173 us with and without; two n-tiles 399 and 399, head size 256 with
// 4-bit codes 38.6 for 36.6. (Inside the tiles' loop instead of around it: two n-tiles 428.)
constexpr int kAttnRun = 32;

// One dim's kernels, in a translation unit of their own.
template <int D>
struct KvAttnDim {
  static cudaError_t launch(SplitArgs& a, int bits, bool exact, int np, int nt, cudaStream_t s);
  static cudaError_t take_error(unsigned int* code);
  static cudaError_t take_check(unsigned int* code);
};

#ifdef XQ_KV_ATTN_IMPL

namespace {

__device__ unsigned int g_kv_attn_error;

__device__ __forceinline__ void kv_record(unsigned what) { atomicCAS(&g_kv_attn_error, 0u, what); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// lo in the low half
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
  return d;
}
__device__ __forceinline__ uint32_t hfma2_of(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The larger of two, or a NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// fp16 pairs of codes. A stored byte u put under 0x64 is the fp16 number
// 1024 + u, so one subtraction gives u - 128 (and u - 8 for a low nibble); a
// high nibble in place is 1024 + 16 u, brought to u - 8 by one fma. All exact.
__device__ __forceinline__ uint32_t bytes02(uint32_t v) { return ptx::hsub2(prmt(v, 0x64646464u, 0x4240u), 0x64806480u); }
__device__ __forceinline__ uint32_t bytes13(uint32_t v) { return ptx::hsub2(prmt(v, 0x64646464u, 0x4341u), 0x64806480u); }
__device__ __forceinline__ uint32_t nib_low(uint32_t v) { return ptx::hsub2(and_or(v, 0x000F000Fu, 0x64006400u), 0x64086408u); }
__device__ __forceinline__ uint32_t nib_high(uint32_t v) {
  return hfma2_of(and_or(v, 0x00F000F0u, 0x64006400u), 0x2C002C00u, 0xD480D480u);  // x / 16 - 72
}

// The same codes as stored, u = q + 128 or q + 8: a zero-extended byte or nibble is the subnormal fp16 u * 2^-24, exact in
// the tensor cores, one instruction for two values. 16-bit queries (EX = false) take K this way, and the offset out of a
// block's score through the block's sum of q: the sums then pass through values larger than their result by the offset over
// a typical code, which costs a few of fp32's bits. fp32 queries, which have to keep them, subtract from each code, and V
// always does (its sum runs over keys, and a small output beside a large weight on a zero code would be lost).
// A high nibble in place is 16 u * 2^-24: its query elements are stored 16 times smaller.
__device__ __forceinline__ uint32_t raw02(uint32_t v) { return prmt(v, 0u, 0x4240u); }
__device__ __forceinline__ uint32_t raw13(uint32_t v) { return prmt(v, 0u, 0x4341u); }
__device__ __forceinline__ uint32_t raw_low(uint32_t v) { return v & 0x000F000Fu; }
__device__ __forceinline__ uint32_t raw_high(uint32_t v) { return v & 0x00F000F0u; }

// Byte offset of 16-byte chunk c of row r in a staged tile. The xor spreads a
// chunk's 8 rows over all banks, for ldmatrix.
template <int NCH>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  const int x = NCH % 8 == 0 ? c ^ (r & 7) : NCH == 4 ? c ^ ((r >> 1) & 3) : NCH % 2 == 0 ? c ^ ((r >> 2) & 1) : c;
  return static_cast<uint32_t>(r * NCH + x) * 16;
}

// N halves at p (4-byte aligned when N is even) as floats, and their largest magnitude (a NaN if there is one).
template <int N>
__device__ __forceinline__ float load_scales(const __half* p, float (&f)[N]) {
  if constexpr (N % 2 == 0) {
    uint32_t w[N / 2];
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const uint2 v = *reinterpret_cast<const uint2*>(p + 4 * i);
        w[2 * i] = v.x;
        w[2 * i + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + 2 * i);
    }
    __half2 top = __habs2(*reinterpret_cast<const __half2*>(&w[0]));
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __half2 h = *reinterpret_cast<const __half2*>(&w[i]);
      const float2 v = __half22float2(h);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
      if (i) top = __hmax2_nan(top, __habs2(h));
    }
    return __half2float(__hmax_nan(__low2half(top), __high2half(top)));
  } else {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      f[i] = __half2float(p[i]);
      top = max_nan(top, fabsf(f[i]));
    }
    return top;
  }
}

__device__ __forceinline__ void store4(void* p, int type, size_t i, float4 v) {
  if (type == kF32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
  } else {
    uint2 w;
    if (type == kF16) {
      w.x = half2_of(v.x, v.y);
      w.y = half2_of(v.z, v.w);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
      w.x = *reinterpret_cast<const uint32_t*>(&a);
      w.y = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = w;
  }
}

// ---- extents, for the checked build
__device__ __forceinline__ int table_len(const SplitArgs& A) {
  return A.flat ? (A.prefix_len + (1 << A.c.page_shift) - 1) >> A.c.page_shift : A.max_pages;
}
__device__ __forceinline__ long long out_rows(const SplitArgs& A) { return static_cast<long long>(A.seqs) * A.rows * A.c.heads; }
// bytes at byte `at` of a pool, both multiples of 16
__device__ __forceinline__ bool in_pool(const SplitArgs& A, long long at, long long bytes) {
  return at >= 0 && at + bytes <= A.c.n_pages * A.c.page_bytes && ((at | bytes) & 15) == 0;
}

// Tokens of sequence b that its table can hold.
__device__ __forceinline__ int seq_len(const SplitArgs& A, int b) {
  if (A.flat) return A.prefix_len;
  if (!XQ_IN(b, A.seqs, kChkKvLens)) return 0;
  const int n = A.lens[b];
  const long long most = static_cast<long long>(A.max_pages) << A.c.page_shift;
  return n < 0 ? 0 : n > most ? static_cast<int>(most) : n;
}
// First unit with a key that some query of the sequence sees (a window hides
// earlier ones), and how many units follow. At least one, so that every row
// has a CTA that writes it. A pair counts kAttnHead more.
__device__ __forceinline__ int first_unit(const SplitArgs& A, int n) {
  if (!A.window) return 0;
  const long long k = static_cast<long long>(n) - A.n_q - A.window + 1;
  return k > 0 ? static_cast<int>(k / kAttnUnit) : 0;
}
__device__ __forceinline__ int unit_count(const SplitArgs& A, int n) {
  const int u = (n + kAttnUnit - 1) / kAttnUnit - first_unit(A, n);
  return u > 1 ? u : 1;
}

// A pair's row r of chunk base: its query token and head.
// a / b for a >= 0 (signed division takes more instructions).
__device__ __forceinline__ int quot(int a, int b) { return static_cast<unsigned>(a) / static_cast<unsigned>(b); }
__device__ __forceinline__ size_t row_at(const SplitArgs& A, int seq, int head, int r) {
  const int token = quot(r, A.group);
  return (static_cast<size_t>(seq) * A.n_q + token) * A.q_heads + head * A.group + (r - token * A.group);
}

// Last key + 1 and first key that row r of a pair sees.
__device__ __forceinline__ void row_range(const SplitArgs& A, int seq, int n, int r, int* start, int* end) {
  const int token = quot(r, A.group);
  if (A.flat) {
    const int b = quot(token, A.n_q);
    int own = XQ_IN(r, A.rows, kChkKvLens) ? A.lens[b] : 0;
    const long long most = static_cast<long long>(A.max_pages) << A.c.page_shift;
    own = own < 0 ? 0 : own > most ? static_cast<int>(most) : own;
    const int pos = kv_pos(A.prefix_len, own, A.n_q, token - b * A.n_q);
    *start = 0;
    *end = pos + 1 < A.prefix_len ? pos + 1 : A.prefix_len;
  } else {
    const int pos = kv_pos(0, n, A.n_q, token);
    *start = A.window && pos >= A.window ? pos - A.window + 1 : 0;
    *end = pos + 1;
  }
}

// Row (token, head) `at` of the result: sums o and l relative to 2^e.
__device__ __forceinline__ void finish4(const SplitArgs& A, int D, size_t at, int d, float4 o, float e, float l) {
  if (!XQ_IN(at, out_rows(A), kChkKvQuery)) return;
  if (A.store) {
    *reinterpret_cast<float4*>(A.pre_o + at * D + d) = o;
    if (d == 0) *reinterpret_cast<float2*>(A.pre_el + at * 2) = make_float2(e, l);
    return;
  }
  if (A.merge) {
    const float4 po = *reinterpret_cast<const float4*>(A.pre_o + at * D + d);
    const float2 pel = *reinterpret_cast<const float2*>(A.pre_el + at * 2);
    const float top = fmaxf(e, pel.x), f = ex2(e - top), g = ex2(pel.x - top);
    o = make_float4(o.x * f + po.x * g, o.y * f + po.y * g, o.z * f + po.z * g, o.w * f + po.w * g);
    l = l * f + pel.y * g;
  }
  // no visible key: l = 0 and the row is 0 (a NaN stays one)
  const float4 y = l != 0.0f ? make_float4(__fdiv_rn(o.x, l), __fdiv_rn(o.y, l), __fdiv_rn(o.z, l), __fdiv_rn(o.w, l))
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  store4(A.out, A.type, at * D + d, y);
}

// The kernel before: waited for at the start, or (late) where its results are
// needed and before the last thread ends, as the kernel after this one waits
// for this one alone. The kernel after may take its place from here on: the
// join, which waits, or a late pass, which needs nothing of this one yet but
// that what came before it is done.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_begin(bool late) {
  if (!late) grid_wait();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---- the line of units and this CTA's stretch of it

struct Line {
  long long total, per;  // units of the line; pairs of a sequence
  long long u, u1;       // the stretch left
  long long off;         // units into sequence seq
  int seq, ctas;
};
struct LineShared {
  int seq, scan[32];
  long long before;
};
// A part of a pair: units k0 .. k1-1 of its keys' nu.
struct Part {
  int seq, n, nu, pair, k0, k1;
  long long first;  // where the pair begins on the line
};

// The stretch of CTA blockIdx.x, found by all threads of its WARPS warps.
// False (with an empty record left): there are fewer units than CTAs.
template <int WARPS>
__device__ __forceinline__ bool line_begin(const SplitArgs& A, LineShared& sh, Line* out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Sum of `x` over the CTA's threads up to this one, and over all of them.
  auto scan = [&](int x, int* all) {
    int sum = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) sh.scan[warp] = sum;
    __syncthreads();
    *all = 0;
    int add = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      add += w < warp ? sh.scan[w] : 0;
      *all += sh.scan[w];
    }
    return sum + add;
  };
  auto cost = [&](int b) { return b < A.seqs ? A.counted ? 1 : unit_count(A, seq_len(A, b)) + A.head : 0; };
  Line L;
  L.per = static_cast<long long>(A.c.heads) * A.chunks;
  int mine = cost(tid), part, more;
  int upto = scan(mine, &part);
  long long sum = part;
  for (int base = 32 * WARPS; base < A.seqs; base += 32 * WARPS) {
    scan(cost(base + tid), &more);
    sum += more;
  }
  L.total = sum * L.per;
  L.ctas = L.total < A.ctas ? static_cast<int>(L.total) : A.ctas;
  const int cta = blockIdx.x;
  if (cta >= L.ctas) {
    if (tid == 0 && !A.whole && XQ_IN(cta, A.records, kChkKvPart)) A.record[cta] = make_int4(0, 0, -1, 0);
    return false;
  }
  L.u = L.total * cta / L.ctas;
  L.u1 = L.total * (cta + 1) / L.ctas;
  const long long v = L.u / L.per;
  long long before = 0;
  for (int base = 0;;) {
    const long long end = before + upto;
    if (mine && end - mine <= v && v < end) {
      sh.seq = base + tid;
      sh.before = end - mine;
    }
    before += part;
    base += 32 * WARPS;
    if (base >= A.seqs || before > v) break;
    mine = cost(base + tid);
    upto = scan(mine, &part);
  }
  __syncthreads();
  L.seq = sh.seq;
  L.off = L.u - sh.before * L.per;
  *out = L;
  return true;
}

// The next part of the stretch. A CTA that gets only from a pair's head
// leaves the pair to the next.
__device__ __forceinline__ bool line_next(const SplitArgs& A, Line& L, Part& x) {
  while (L.u < L.u1) {
    const int n = seq_len(A, L.seq), nu = unit_count(A, n), nv = A.counted ? 1 : nu + A.head;
    if (!A.flat && threadIdx.x == 0 && A.lens[L.seq] > n) kv_record(kKvBadLen);
    const int pair = static_cast<int>(L.off / nv), at = static_cast<int>(L.off - static_cast<long long>(pair) * nv);
    // a whole pair is the CTA's in whose stretch it begins
    const int did = A.whole || nv - at < L.u1 - L.u ? nv - at : static_cast<int>(L.u1 - L.u);
    x = {L.seq, n, nu, pair, at > A.head ? at - A.head : 0, A.whole ? (at ? 0 : nu) : at + did - A.head, L.u - at};
    L.u += did;
    L.off += did;
    if (L.off == nv * L.per) {
      L.off = 0;
      ++L.seq;
    }
    if (x.k1 > 0) return true;
  }
  return false;
}

// The CTA of the last unit of x's pair: the largest c with total * c / ctas <= that unit.
__device__ __forceinline__ int line_last(const SplitArgs& A, const Line& L, const Part& x) {
  const long long last = x.first + x.nu + A.head - 1;
  return static_cast<int>(((last + 1) * L.ctas - 1) / L.total);
}

template <int NT, int M>
__device__ __forceinline__ void scale_all(float (&o)[NT][M][4], float f) {
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int m = 0; m < M; ++m) {
      o[j][m][0] *= f;
      o[j][m][1] *= f;
      o[j][m][2] *= f;
      o[j][m][3] *= f;
    }
}

// A lane's share of a query row as it lies in memory, elements 16 k + 0 .. 3: fp32 (EX) or 16-bit ones.
template <bool EX, int D>
struct RawQuery {
  using Piece = std::conditional_t<EX, float4, uint2>;
  Piece x[D / 16];
  __device__ __forceinline__ void load(const SplitArgs& A, size_t at, bool live) {
    const Piece* const p = reinterpret_cast<const Piece*>(static_cast<const uint8_t*>(A.q) + at * (EX ? 4 : 2));
#pragma unroll
    for (int k = 0; k < D / 16; ++k) x[k] = live ? p[4 * k] : Piece{};
  }
  __device__ __forceinline__ void floats(bool f16, float4 (&v)[D / 16]) const {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      if constexpr (EX) {
        v[k] = x[k];
      } else {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x[k].x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&x[k].y));
        v[k] = f16 ? make_float4(a.x, a.y, b.x, b.y)
                   : make_float4(__uint_as_float(x[k].x << 16), __uint_as_float(x[k].x & 0xFFFF0000u),
                                 __uint_as_float(x[k].y << 16), __uint_as_float(x[k].y & 0xFFFF0000u));
      }
    }
  }
};

template <int BITS, int D, bool EX, int NP, int NT>
__global__ void __launch_bounds__(32 * kAttnWarps, SplitShape<BITS, D, EX, NP, NT>::kCtas)
    kv_split_kernel(const __grid_constant__ SplitArgs A) {
  using S = SplitShape<BITS, D, EX, NP, NT>;
  constexpr int NB = S::NB, R = S::R, kStages = S::kStages, NS = NP == 2 ? 2 : 4, NQ = NP == 2 ? 1 : 2;
  extern __shared__ __align__(256) uint8_t smem[];  // stage and matrix addresses are put together by xor
  __shared__ LineShared sh_line;
  __shared__ float sh_el[kAttnWarps][R][2];
  __shared__ uint32_t sh_at[kAttnWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  grid_begin(A.late);

  const int cta = blockIdx.x;
  Line line;
  if (!line_begin<kAttnWarps>(A, sh_line, &line)) {
    if (A.late) grid_wait();
    return;
  }

  uint8_t* const stages = smem + warp * S::kWarpBytes;
  uint8_t* const sums = smem + kAttnWarps * S::kWarpBytes + warp * S::kSumBytes;  // fp32: this warp's
  const uint32_t stage0 = ptx::smem_addr(stages);
  // Where this lane's copies of a tile go and come from. Scales: the first
  // lanes take K's, the next ones V's.
  const uint32_t code_to = chunk_at<S::kChunks>(lane / S::kChunks, lane % S::kChunks);
  const bool v_scale = lane >= S::kScales / 16;
  const int scale_lane = (v_scale ? lane - S::kScales / 16 : lane) * 16;
  const uint32_t scale_to = S::kCodes + scale_lane + (v_scale ? S::kCodes + S::kScales : 0);
  // A tile's place in a pool, in 32-byte steps (16 rows of codes or scales are
  // a multiple; a pool has fewer than 2^32), is added to these.
  const uint8_t* const k_from = A.c.k + lane * 16;
  const uint8_t* const v_from = A.c.v + lane * 16;
  const uint8_t* const scale_from = (v_scale ? A.c.v : A.c.k) + scale_lane;
  bool left_record = false;
  // ---- the warp's tiles of 16 keys of a part: warp, warp + 4, ... of its units
  int tile0 = 0, tiles = 0, line0 = 0, stage = 0;
  const int32_t* table = nullptr;
  const int shift = A.c.page_shift - 4;  // tiles a page
  // Where the codes and the scales of the next 32 tiles lie, one tile a lane (all ones if its page id is invalid). The page
  // ids after them are on their way.
  uint32_t code_at = 0, scales_at = 0;
  int next_page = 0;
  unsigned bad = 0;      // stages whose page id was invalid
  unsigned clean_n = 0;  // tiles from `clean` on that hold only keys which every row sees
  auto page_of = [&](int i) {
    const int at = (tile0 + i * kAttnWarps) >> shift;
    return i < tiles && XQ_IN(at, table_len(A), kChkKvTable) ? table[at] : 0;
  };
  auto locate = [&](int i, int page) {
    const int line = line0 + (((tile0 + i * kAttnWarps) & ((1 << shift) - 1)) << 4);
    const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(A.c.n_pages);
    const uint32_t at = static_cast<uint32_t>(page) * static_cast<uint32_t>(A.c.page_bytes >> 5);
    code_at = ok ? at + static_cast<uint32_t>(line / 16) * (S::kRow / 2) : ~0u;
    scales_at = at + static_cast<uint32_t>(A.c.scale_off + line * (NB * 2)) / 32;
  };
  auto issue = [&](int i, int stage) {
    if (i < tiles) {
      if ((i & 31) == 0 && i > 0) {
        locate(i + lane, next_page);
        next_page = page_of(i + 32 + lane);
      }
      const uint32_t at = __shfl_sync(0xffffffffu, code_at, i & 31), so = __shfl_sync(0xffffffffu, scales_at, i & 31);
      if (at != ~0u && !XQ_CHECKED(in_pool(A, 32ll * at, 16 * S::kRow) && in_pool(A, 32ll * so, S::kScales), kChkKvTile)) {
      } else if (at != ~0u) {
        const uint8_t* const kc = k_from + static_cast<size_t>(at) * 32;
        const uint8_t* const vc = v_from + static_cast<size_t>(at) * 32;
        const uint32_t base = stage0 + stage * S::kStage, dst = base + code_to;
#pragma unroll
        for (int x = 0; x < S::kSteps; ++x) {
          // 32 chunks a step; a step's rows differ from the first one's in the swizzle by a constant
          const uint32_t to = S::kPow2 ? (dst ^ S::turn(x)) + x * 512
                                       : base + chunk_at<S::kChunks>((x * 32 + lane) / S::kChunks, (x * 32 + lane) % S::kChunks);
          if (S::kChunks % 2 == 0 || x * 32 + lane < 16 * S::kChunks) {
            cp16(to, kc + x * 512);
            cp16(to + S::kCodes + S::kScales, vc + x * 512);
          }
        }
        if (lane < 2 * S::kScales / 16) cp16(base + scale_to, scale_from + static_cast<size_t>(so) * 32);
      } else {
        bad |= 1u << stage;
        clean_n = 0;
        if (lane == 0) kv_record(kKvBadPage);
      }
    }
    cp_commit();
  };

  // Start on a part: its first tiles into the stages from `stage` on.
  auto begin_part = [&](const Part& x) {
    const int all = (x.n + 15) / 16;
    tile0 = (first_unit(A, x.n) + x.k0) * kAttnWarps + warp;
    tiles = all > tile0 ? (all - tile0 + kAttnWarps - 1) / kAttnWarps : 0;
    tiles = tiles < x.k1 - x.k0 ? tiles : x.k1 - x.k0;
    line0 = quot(x.pair, A.chunks) << A.c.page_shift;
    table = A.flat ? A.pages : A.pages + static_cast<size_t>(x.seq) * A.page_stride;
    const int page = page_of(lane);
    next_page = page_of(32 + lane);
    locate(lane, page);
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue(i, stage + i < kStages ? stage + i : stage + i - kStages);
  };

  Part cur;
  bool have = line_next(A, line, cur), begun = false;
  while (have) {
    const int sq = cur.seq, n = cur.n, nu = cur.nu, pair = cur.pair, k0 = cur.k0, k1 = cur.k1;
    const int head = quot(pair, A.chunks), chunk = pair - head * A.chunks;
    const int row0 = chunk * R, rows = A.rows - row0 < R ? A.rows - row0 : R;
    // ---- the queries' loads, all before the first use, and ahead of the first tiles'
    RawQuery<EX, D> raw[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = NP == 2 ? 4 * j + (g >> 1) : 8 * j + g;
      const size_t at = r < rows ? row_at(A, sq, head, row0 + r) : 0;
      raw[j].load(A, at * D + 4 * t, r < rows && XQ_IN(at, out_rows(A), kChkKvQuery));
    }
    if (!begun) begin_part(cur);
    // ---- queries as B operands. Column g of n-tile j: NP = 2: row 4 j + g/2, piece g & 1; NP = 1: row 8 j + g.
    uint32_t qf[NT][D / 16][2];
    float cs[NT][NQ], qs[NT][NB][NQ];  // score factor, and -(128 or 8) sum(q) of each block, of this lane's columns
    int lim0[NT][NQ], lim1[NT][NQ];
    int all0 = 0, all1 = INT_MAX;  // keys that every row of the chunk sees
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float4 v[D / 16];
      raw[j].floats(A.type == kF16, v);
      float top = 0.0f;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        top = fmaxf(fmaxf(top, fmaxf(fabsf(v[k].x), fabsf(v[k].y))), fmaxf(fabsf(v[k].z), fabsf(v[k].w)));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // a power of two that takes the row's largest element to 2^12 .. 2^13
      int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      ex = ex < -100 ? -100 : ex;
      const float up = __uint_as_float(static_cast<unsigned>(127 + 12 - ex) << 23);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        // the elements of high nibbles 16 times smaller
        const float f = !EX && BITS == 4 && (k & 1) ? up * 0.0625f : up;
        const float x = v[k].x * f, y = v[k].y * f, z = v[k].z * f, w = v[k].w * f;
        uint32_t b0 = half2_of(x, z), b1 = half2_of(y, w);
        if (NP == 2 && (g & 1)) {  // lo = q - hi, exact in fp32
          const float2 h0 = __half22float2(*reinterpret_cast<const __half2*>(&b0));
          const float2 h1 = __half22float2(*reinterpret_cast<const __half2*>(&b1));
          b0 = half2_of(x - h0.x, z - h0.y);
          b1 = half2_of(y - h1.x, w - h1.y);
        }
        qf[j][k][0] = b0;
        qf[j][k][1] = b1;
      }
      float block_sum[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float sum2[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 u0 = __half22float2(*reinterpret_cast<const __half2*>(&qf[j][2 * b + x][0]));
          const float2 u1 = __half22float2(*reinterpret_cast<const __half2*>(&qf[j][2 * b + x][1]));
          sum2[x] = (u0.x + u0.y) + (u1.x + u1.y);
        }
        float sum = BITS == 4 ? fmaf(sum2[1], 16.0f, sum2[0]) : sum2[0] + sum2[1];
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        block_sum[b] = sum * (BITS == 4 ? -8.0f * 5.9604645e-8f : -128.0f * 5.9604645e-8f);
      }
      // in two steps: of 2^(ex + 12) alone the exponent would pass fp32's for bf16 queries of 2^116 and more
      const float down = A.scale * 1.4426950408889634f * __uint_as_float(static_cast<unsigned>(127 + ex) << 23) *
                         (EX ? 2.44140625e-4f : 4096.0f);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        if (NP == 2) {  // both pieces
          qs[j][b][0] = __shfl_sync(0xffffffffu, block_sum[b], 8 * t) + __shfl_sync(0xffffffffu, block_sum[b], 8 * t + 4);
        } else {
          qs[j][b][0] = __shfl_sync(0xffffffffu, block_sum[b], 8 * t);
          qs[j][b][NQ - 1] = __shfl_sync(0xffffffffu, block_sum[b], 8 * t + 4);
        }
      }
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        // the lane that holds this accumulator column's row as column g
        cs[j][i] = __shfl_sync(0xffffffffu, down, 8 * t + 4 * i);
        const int rr = NP == 2 ? 4 * j + t : 8 * j + 2 * t + i;
        lim0[j][i] = 0;
        lim1[j][i] = 0;
        if (rr < rows) {
          row_range(A, sq, n, row0 + rr, &lim0[j][i], &lim1[j][i]);
          all0 = max(all0, lim0[j][i]);
          all1 = min(all1, lim1[j][i]);
        }
      }
    }
#pragma unroll
    for (int x = 1; x < 4; x <<= 1) {
      all0 = max(all0, __shfl_xor_sync(0xffffffffu, all0, x));
      all1 = min(all1, __shfl_xor_sync(0xffffffffu, all1, x));
    }

    // tiles clean .. clean + clean_n - 1 hold only keys that every row sees (none, once a page id was invalid)
    int clean = ((all0 + 15) / 16 - tile0 + kAttnWarps - 1) / kAttnWarps;
    clean = clean > 0 ? clean : 0;
    clean_n = all1 / 16 > tile0 ? static_cast<unsigned>((all1 / 16 - tile0 + kAttnWarps - 1) / kAttnWarps) : 0u;
    clean_n = clean_n > static_cast<unsigned>(clean) && !bad ? clean_n - clean : 0u;

    float o[NT][D / 16][4], er[NT][NQ], l[NT][NQ];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int m = 0; m < D / 16; ++m) o[j][m][0] = o[j][m][1] = o[j][m][2] = o[j][m][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        er[j][i] = kNoKey;
        l[j][i] = 0.0f;
      }
    }
    // ldmatrix row addresses: matrix m of 4 covers rows 8 (m & 1) .. + 7, chunk m >> 1
    const int lrow = (lane & 7) + (lane & 8), lch = lane >> 4;
    const uint32_t code_from = chunk_at<S::kChunks>(lrow, lch);
    // chunk c + lch (c even) of the lane's row
    auto from = [&](uint32_t base, int c) {
      return S::kPow2 ? (base + code_from) ^ (c * 16) : base + chunk_at<S::kChunks>(lrow, (c + lch) % S::kChunks);
    };
    // fp32: the accumulators into this lane's sums, in fp32 additions, relative to the references of now.
    auto to_sums = [&](bool first) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float* const ref = reinterpret_cast<float*>(sums + S::kSums) + j * 32 + lane;
        const float f = first ? 0.0f : ex2(*ref - er[j][0]);
        *ref = er[j][0];
#pragma unroll
        for (int m = 0; m < D / 16; m += 2) {
          float4* const sum = reinterpret_cast<float4*>(sums) + (j * (D / 32) + m / 2) * 32 + lane;
          float4 y;
          y.x = fmaf(o[j][m][1], 1.0f / kLoUp, o[j][m][0]);
          y.y = fmaf(o[j][m][3], 1.0f / kLoUp, o[j][m][2]);
          y.z = fmaf(o[j][m + 1][1], 1.0f / kLoUp, o[j][m + 1][0]);
          y.w = fmaf(o[j][m + 1][3], 1.0f / kLoUp, o[j][m + 1][2]);
          if (!first) {
            const float4 x = *sum;
            y = make_float4(fmaf(x.x, f, y.x), fmaf(x.y, f, y.y), fmaf(x.z, f, y.z), fmaf(x.w, f, y.w));
          }
          *sum = y;
#pragma unroll
          for (int x = 0; x < 4; ++x) o[j][m][x] = o[j][m + 1][x] = 0.0f;
        }
      }
    };
    const bool summed = EX && tiles > kAttnRun;
    for (int i = 0, run = 0; run < tiles; run += kAttnRun) {
      for (const int end = EX && tiles - run > kAttnRun ? run + kAttnRun : tiles; i < end; ++i) {
        cp_wait<kStages - 2>();
        __syncwarp();  // this tile has landed for every lane, and the one before has been read by every lane
        issue(i + kStages - 1, stage == 0 ? kStages - 1 : stage - 1);
        const uint32_t kb = stage0 + stage * S::kStage, vb = kb + S::kCodes + S::kScales;
        const __half* ks = reinterpret_cast<const __half*>(stages + stage * S::kStage + S::kCodes);
        const __half* vs = ks + (S::kCodes + S::kScales) / 2;
        // ---- scores of keys g and g + 8
        float s[NT][NS];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < NS; ++x) s[j][x] = 0.0f;
        {
          float d0[NB], d1[NB];
          load_scales<NB>(ks + g * NB, d0);
          load_scales<NB>(ks + (g + 8) * NB, d1);
          uint32_t w[4];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t a0[4], a1[4];  // operands of the block's two 16-element halves
            if (BITS == 8) {
              ldm4(from(kb, 2 * b), w);
              a0[0] = EX ? bytes02(w[0]) : raw02(w[0]);
              a0[1] = EX ? bytes02(w[1]) : raw02(w[1]);
              a0[2] = EX ? bytes13(w[0]) : raw13(w[0]);
              a0[3] = EX ? bytes13(w[1]) : raw13(w[1]);
              a1[0] = EX ? bytes02(w[2]) : raw02(w[2]);
              a1[1] = EX ? bytes02(w[3]) : raw02(w[3]);
              a1[2] = EX ? bytes13(w[2]) : raw13(w[2]);
              a1[3] = EX ? bytes13(w[3]) : raw13(w[3]);
            } else {
              // one load holds two blocks (16 bytes each); an odd last one is paired with the first
              if (b % 2 == 0) ldm4(from(kb, b), w);
              const uint32_t x = w[2 * (b & 1)], y = w[2 * (b & 1) + 1], x8 = x >> 8, y8 = y >> 8;
              a0[0] = EX ? nib_low(x) : raw_low(x);
              a0[1] = EX ? nib_low(y) : raw_low(y);
              a0[2] = EX ? nib_low(x8) : raw_low(x8);
              a0[3] = EX ? nib_low(y8) : raw_low(y8);
              a1[0] = EX ? nib_high(x) : raw_high(x);
              a1[1] = EX ? nib_high(y) : raw_high(y);
              a1[2] = EX ? nib_high(x8) : raw_high(x8);
              a1[3] = EX ? nib_high(y8) : raw_high(y8);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float c[4];
              mma16_first(c, a0, qf[j][2 * b][0], qf[j][2 * b][1]);
              mma16(c, a1, qf[j][2 * b + 1][0], qf[j][2 * b + 1][1]);
              if (!EX) {  // the offset's share
                s[j][0] = fmaf(d0[b], qs[j][b][0], s[j][0]);
                s[j][NS / 2] = fmaf(d1[b], qs[j][b][0], s[j][NS / 2]);
                if (NP == 1) {
                  s[j][1] = fmaf(d0[b], qs[j][b][NQ - 1], s[j][1]);
                  s[j][NS - 1] = fmaf(d1[b], qs[j][b][NQ - 1], s[j][NS - 1]);
                }
              }
              if (NP == 2) {
                s[j][0] = fmaf(d0[b], c[0] + c[1], s[j][0]);
                s[j][1] = fmaf(d1[b], c[2] + c[3], s[j][1]);
              } else {
                s[j][0] = fmaf(d0[b], c[0], s[j][0]);
                s[j][1] = fmaf(d0[b], c[1], s[j][1]);
                s[j][NS - 2] = fmaf(d1[b], c[2], s[j][NS - 2]);
                s[j][NS - 1] = fmaf(d1[b], c[3], s[j][NS - 1]);
              }
            }
          }
        }
        float v0[NB], v1[NB];
        float m0 = load_scales<NB>(vs + g * NB, v0), m1 = load_scales<NB>(vs + (g + 8) * NB, v1);
        // ---- scale, and mask where the tile holds keys that some row does not see
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < NS; ++x) s[j][x] *= cs[j][NP == 2 ? 0 : (x & 1)];
        if (static_cast<unsigned>(i - clean) >= clean_n) {
          const bool gone = (bad >> stage) & 1;
          bad &= ~(1u << stage);
          const int ka = (tile0 + i * kAttnWarps) * 16 + g, kb8 = ka + 8;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int x = 0; x < NS; ++x) {
              const int col = NP == 2 ? 0 : (x & 1), kk = x < NS / 2 ? ka : kb8;
              if (gone || kk < lim0[j][col] || kk >= lim1[j][col]) s[j][x] = -INFINITY;
            }
          // what lies past the sequence may be anything: its scales must not reach a product
          if (gone || ka >= n) {
#pragma unroll
            for (int b = 0; b < NB; ++b) v0[b] = 0.0f;
            m0 = 0.0f;
          }
          if (gone || kb8 >= n) {
#pragma unroll
            for (int b = 0; b < NB; ++b) v1[b] = 0.0f;
            m1 = 0.0f;
          }
        }
        // ---- weights p = 2^(s - e). w: p times the key's largest V scale (no less than the least fp16 step). e moves if some
        // w passes 2^15 or is not a number, as with a V scale that is not finite; the fp32 form also looks for weights below 2^-13.
        constexpr float kLeast = 5.9604645e-8f;
        m0 = max_nan(m0, kLeast);
        m1 = max_nan(m1, kLeast);
        float p[NT][NS];
        bool odd = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < NS; ++x) {
            p[j][x] = ex2(s[j][x] - er[j][NP == 2 ? 0 : (x & 1)]);
            const float w = p[j][x] * (x < NS / 2 ? m0 : m1);
            odd |= !(w <= kWeightTop && (!EX || w >= kWeightLow));
          }
        const bool any_odd = __any_sync(0xffffffffu, odd);
        if (any_odd) {
          bool move = false;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int x = 0; x < NS; ++x) move |= !(p[j][x] * (x < NS / 2 ? m0 : m1) <= kWeightTop);
          odd = __any_sync(0xffffffffu, move);
        }
        if (any_odd && odd) {
          if (__any_sync(0xffffffffu, !(m0 <= 65504.0f) || !(m1 <= 65504.0f))) {
            // V blocks that are not finite: their elements become NaN in the rows that see the key. The scale itself must not
            // reach a product: a row that does not see it has the weight 0, and 0 times infinity is NaN.
            m0 = m1 = kLeast;
            unsigned spoilt = 0;  // blocks, by row
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const bool b0 = !(fabsf(v0[b]) <= 65504.0f), b1 = !(fabsf(v1[b]) <= 65504.0f);
              v0[b] = b0 ? 0.0f : v0[b];
              v1[b] = b1 ? 0.0f : v1[b];
              m0 = fmaxf(m0, fabsf(v0[b]));
              m1 = fmaxf(m1, fabsf(v1[b]));
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < NQ; ++c)
                  if ((b0 && s[j][c] != -INFINITY) || (b1 && s[j][NS / 2 + c] != -INFINITY)) spoilt |= 1u << ((b * NT + j) * NQ + c);
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) spoilt |= __shfl_xor_sync(0xffffffffu, spoilt, x);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < NQ; ++c)
                  if (spoilt >> ((b * NT + j) * NQ + c) & 1) {
                    o[j][2 * b][c] = o[j][2 * b][2 + c] = __int_as_float(0x7FC00000);
                    o[j][2 * b + 1][c] = o[j][2 * b + 1][2 + c] = __int_as_float(0x7FC00000);
                  }
          }
          const float lg0 = __log2f(m0), lg1 = __log2f(m1);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
              float top = fmaxf(s[j][c] + lg0, s[j][NS / 2 + c] + lg1) - 11.0f;
              // scores of 2^27, where fp32's step is 16, can leave a weight of 2^24 so
              const float z = fmaxf((s[j][c] - top) + lg0, (s[j][NS / 2 + c] - top) + lg1);
              top = z > 15.0f ? top + z : top;
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
              top = fmaxf(top, er[j][c]);
              const float f = ex2(er[j][c] - top);
              er[j][c] = top;
              l[j][c] *= f;
#pragma unroll
              for (int m = 0; m < D / 16; ++m) {
                if (NP == 2) {
                  o[j][m][0] *= f;
                  o[j][m][1] *= f;
                  o[j][m][2] *= f;
                  o[j][m][3] *= f;
                } else {
                  o[j][m][c] *= f;
                  o[j][m][2 + c] *= f;
                }
              }
              p[j][c] = ex2(s[j][c] - top);
              p[j][NS / 2 + c] = ex2(s[j][NS / 2 + c] - top);
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < NQ; ++c) l[j][c] += p[j][c] + p[j][NS / 2 + c];
        // ---- outputs, block by block. fp32: weights below 2^-13 would lose bits in fp16 (they count only where the larger
        // ones meet zero codes); they follow 2^24 larger, on accumulators scaled alike, at most three times: 2^-85.
        for (int level = 0;; ++level) {
          float rest[NT][NS];
          bool more = false;
          if (EX && any_odd) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
              for (int x = 0; x < NS; ++x) {
                const bool later = level < 3 && p[j][x] * (x < NS / 2 ? m0 : m1) < kWeightLow;
                rest[j][x] = later ? p[j][x] * 16777216.0f : 0.0f;
                p[j][x] = later ? 0.0f : p[j][x];
                more |= rest[j][x] > 0.0f;
              }
          }
          uint32_t w[4];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            uint32_t a0[4], a1[4];
            if (BITS == 8) {
              ldm4t(from(vb, 2 * b), w);
              a0[0] = bytes02(w[0]);
              a0[1] = bytes13(w[0]);
              a0[2] = bytes02(w[1]);
              a0[3] = bytes13(w[1]);
              a1[0] = bytes02(w[2]);
              a1[1] = bytes13(w[2]);
              a1[2] = bytes02(w[3]);
              a1[3] = bytes13(w[3]);
            } else {
              if (b % 2 == 0) ldm4t(from(vb, b), w);
              const uint32_t x = w[2 * (b & 1)], y = w[2 * (b & 1) + 1], x8 = x >> 8, y8 = y >> 8;
              a0[0] = nib_low(x);
              a0[1] = nib_low(x8);
              a0[2] = nib_low(y);
              a0[3] = nib_low(y8);
              a1[0] = nib_high(x);
              a1[1] = nib_high(x8);
              a1[2] = nib_high(y);
              a1[3] = nib_high(y8);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              uint32_t b0, b1;
              if (NP == 2) {
                const ptx::f2 up = ptx::pk(kLoUp, kLoUp), down = ptx::pk(-kLoUp, -kLoUp);
                const ptx::f2 x = ptx::mul2(ptx::pk(p[j][0], p[j][1]), ptx::pk(v0[b], v1[b]));
                const uint32_t hi = half2_of(ptx::lo32(x), ptx::hi32(x));
                const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                const ptx::f2 r = ptx::fma2(ptx::pk(h.x, h.y), down, ptx::mul2(x, up));  // (w - hi) * 2^11, exact
                const uint32_t lo = half2_of(ptx::lo32(r), ptx::hi32(r));
                b0 = transpose8(prmt(hi, lo, 0x5410u));
                b1 = transpose8(prmt(hi, lo, 0x7632u));
              } else {
                b0 = transpose8(half2_of(p[j][0] * v0[b], p[j][1] * v0[b]));
                b1 = transpose8(half2_of(p[j][NS - 2] * v1[b], p[j][NS - 1] * v1[b]));
              }
              mma16(o[j][2 * b], a0, b0, b1);
              mma16(o[j][2 * b + 1], a1, b0, b1);
            }
          }
          if (!EX || !any_odd) break;
          if (!__any_sync(0xffffffffu, more)) {
            if (level > 0) scale_all(o, level == 1 ? 5.9604645e-8f : level == 2 ? 3.5527137e-15f : 2.1175824e-22f);
            break;
          }
          scale_all(o, 16777216.0f);
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int x = 0; x < NS; ++x) p[j][x] = rest[j][x];
        }
        stage = stage + 1 == kStages ? 0 : stage + 1;
      }
      if (!EX) break;
      if (summed) to_sums(run == 0);
    }
    // ---- merge the four warps in shared memory. Each puts its results where its last tile was; the next part's tiles go
    // elsewhere until the barrier after the merge.
    __syncwarp();  // every lane has read that tile
    const uint32_t at = S::kOverlap ? (stage == 0 ? kStages - 1 : stage - 1) * S::kStage : 0;
    float* const mine_o = reinterpret_cast<float*>(stages + at);
    if (lane == 0) sh_at[warp] = warp * S::kWarpBytes + at;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < NQ; ++c) {
        float sum_l = l[j][c];
        sum_l += __shfl_xor_sync(0xffffffffu, sum_l, 4);
        sum_l += __shfl_xor_sync(0xffffffffu, sum_l, 8);
        sum_l += __shfl_xor_sync(0xffffffffu, sum_l, 16);
        const int r = NP == 2 ? 4 * j + t : 8 * j + 2 * t + c;
        if (g == 0) {
          sh_el[warp][r][0] = er[j][c];
          sh_el[warp][r][1] = sum_l;
        }
#pragma unroll
        for (int m = 0; m < D / 16; ++m) {
          float2 y = NP == 2 ? make_float2(fmaf(o[j][m][1], 1.0f / kLoUp, o[j][m][0]),
                                                 fmaf(o[j][m][3], 1.0f / kLoUp, o[j][m][2]))
                                   : make_float2(o[j][m][c], o[j][m][2 + c]);
          if (summed) y = reinterpret_cast<const float2*>(sums)[((j * (D / 32) + m / 2) * 32 + lane) * 2 + m % 2];
          *reinterpret_cast<float2*>(mine_o + r * D + 16 * m + 2 * g) = y;
        }
      }
    Part next;
    const bool more_parts = line_next(A, line, next);
    begun = S::kOverlap && more_parts;
    if (begun) begin_part(next);
    __syncthreads();
    const bool whole = k0 == 0 && k1 == nu;
    if (A.late && whole) grid_wait();
    for (int x = tid * 4; x < rows * D; x += 32 * kAttnWarps * 4) {
      const int r = x / D, d = x - r * D;
      float e = sh_el[0][r][0];
#pragma unroll
      for (int w = 1; w < kAttnWarps; ++w) e = fmaxf(e, sh_el[w][r][0]);
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float ll = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) {
        const float f = ex2(sh_el[w][r][0] - e);
        const float4 z = *reinterpret_cast<const float4*>(smem + sh_at[w] + x * 4);
        y = make_float4(fmaf(z.x, f, y.x), fmaf(z.y, f, y.y), fmaf(z.z, f, y.z), fmaf(z.w, f, y.w));
        ll = fmaf(sh_el[w][r][1], f, ll);
      }
      if (whole) {
        finish4(A, D, row_at(A, sq, head, row0 + r), d, y, e, ll);
      } else {
        // a pair that began in an earlier CTA goes to the first slot, one that goes on in the next to the second
        const size_t ps = (static_cast<size_t>(cta) * 2 + (k0 == 0 ? 1 : 0)) * R + r;
        if (!XQ_IN(ps, A.part_rows, kChkKvPart)) continue;
        *reinterpret_cast<float4*>(A.part_o + ps * D + d) = y;
        if (d == 0) *reinterpret_cast<float2*>(A.part_el + ps * 2) = make_float2(e, ll);
      }
    }
    if (!whole && k0 == 0) {
      left_record = true;
      if (tid == 0 && XQ_IN(cta, A.records, kChkKvPart)) A.record[cta] = make_int4(sq, pair, line_last(A, line, cur), 0);
    }
    __syncthreads();
    cur = next;
    have = more_parts;
  }
  if (!left_record && tid == 0 && !A.whole && XQ_IN(cta, A.records, kChkKvPart)) A.record[cta] = make_int4(0, 0, -1, 0);
  if (A.late) grid_wait();
}

// The parts of the pairs that begin in a block's stretch of CTAs (of neighbours: pairs often begin at equal distances, which
// a step of gridDim.x may divide), RB of their R rows from RB * blockIdx.y on. A thread holds one float4 of the rows; each
// team of threads takes every kTeams-th part, several loads at a time, then the teams are merged. COLS: the parts' outputs
// are stored [dim / 4][R], not [R][dim / 4].
// Two blocks an SM, with 6 loads in flight a thread (one block with 8: 64 sequences of 211 to 8192 tokens 85.8 us instead
// of 83.9, a prefix of 32768 tokens for 64 sequences 96.6 instead of 91.6; three with 2 to 4 help or cost as much).
constexpr int kJoinThreads = 512, kJoinBlocks = 2, kJoinBatch = 6;
// Parts a pair from which a block takes one row (57 parts: 37.2 us for 38.5 of a 131071-token sequence; 9 parts of 8 rows:
// 17.9 for 16.8 of 8 sequences behind a 1000-token prefix).
constexpr int kJoinMany = 24;
template <int D, int R, int RB, bool COLS>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks) kv_join_kernel(const __grid_constant__ SplitArgs A) {
  constexpr int kLanes = RB * D / 4;
  constexpr int kTeams = kJoinThreads / kLanes;
  static_assert(kTeams >= 1, "a part's rows are one pass of the block");
  __shared__ float2 sel[kTeams][RB];
  __shared__ float4 so[kTeams][kLanes];
  grid_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int team = tid / kLanes, at = tid - team * kLanes;
  const int r = COLS ? at % RB : at / (D / 4), d = (COLS ? at / RB : at % (D / 4)) * 4;
  const int row = RB * blockIdx.y + r;
  int4 mine = make_int4(0, 0, -1, 0);  // the records, one a lane
  const int per = (A.ctas + gridDim.x - 1) / gridDim.x, c = blockIdx.x * per + lane;
  if (lane < per && c < A.ctas && XQ_IN(c, A.records, kChkKvPart)) mine = A.record[c];
  for (unsigned left = __ballot_sync(0xffffffffu, mine.z >= 0); left; left &= left - 1) {
    const int from = __ffs(left) - 1, c0 = blockIdx.x * per + from;
    const int seq = __shfl_sync(0xffffffffu, mine.x, from), pair = __shfl_sync(0xffffffffu, mine.y, from);
    const int parts = __shfl_sync(0xffffffffu, mine.z, from) - c0 + 1;
    const int head = pair / A.chunks, pair_row = (pair - head * A.chunks) * R + row;
    float e = kNoKey, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const bool live = team < kTeams && pair_row < A.rows;
    if (live) {
      for (int base = team; base < parts; base += kTeams * kJoinBatch) {
        float2 el[kJoinBatch];
        float4 z[kJoinBatch];
        float top = e;
#pragma unroll
        for (int x = 0; x < kJoinBatch; ++x) {
          const int i = base + x * kTeams;
          if (i < parts) {
            // part i: the second slot of the CTA where the pair begins, the first of those after it
            const size_t slot = (static_cast<size_t>(c0 + i) * 2 + (i == 0 ? 1 : 0)) * R + row;
            el[x] = make_float2(kNoKey, 0.0f);
            z[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (!XQ_IN(slot, A.part_rows, kChkKvPart)) continue;
            el[x] = *reinterpret_cast<const float2*>(A.part_el + slot * 2);
            z[x] = *reinterpret_cast<const float4*>(A.part_o + (COLS ? (slot - row) * D + d * R + row * 4 : slot * D + d));
          }
        }
#pragma unroll
        for (int x = 0; x < kJoinBatch; ++x)
          if (base + x * kTeams < parts) top = fmaxf(top, el[x].x);
        const float keep = ex2(e - top);
        o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
        l *= keep;
        e = top;
#pragma unroll
        for (int x = 0; x < kJoinBatch; ++x)
          if (base + x * kTeams < parts) {
            const float f = ex2(el[x].x - top);
            o = make_float4(fmaf(z[x].x, f, o.x), fmaf(z[x].y, f, o.y), fmaf(z[x].z, f, o.z), fmaf(z[x].w, f, o.w));
            l = fmaf(el[x].y, f, l);
          }
      }
      if (team > 0) so[team][at] = o;
      if (d == 0) sel[team][r] = make_float2(e, l);
    }
    __syncthreads();
    if (live && team == 0) {
      const int used = parts < kTeams ? parts : kTeams;
      const float own = e;
      for (int w = 1; w < used; ++w) e = fmaxf(e, sel[w][r].x);
      float f = ex2(own - e);
      o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
      l *= f;
      for (int w = 1; w < used; ++w) {
        const float2 el = sel[w][r];
        const float4 z = so[w][at];
        f = ex2(el.x - e);
        o = make_float4(fmaf(z.x, f, o.x), fmaf(z.y, f, o.y), fmaf(z.z, f, o.z), fmaf(z.w, f, o.w));
        l = fmaf(el.y, f, l);
      }
      finish4(A, D, row_at(A, seq, head, pair_row), d, o, e, l);
    }
    __syncthreads();  // the sums have been read
  }
}

// Its grid: about as many blocks as run at a time, at most 32 records each.
template <int R, int RB>
dim3 join_grid(int ctas) {
  const int rows = R / RB, want = 4 * kNumSMs / rows, least = (ctas + 31) / 32;
  const int x = want < least ? least : want < ctas ? want : ctas;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(rows));
}

template <int BITS, int D, bool EX, int NP, int NT>
cudaError_t launch_split(SplitArgs& a, cudaStream_t s) {
  using S = SplitShape<BITS, D, EX, NP, NT>;
  constexpr int kResident = S::kCtas * kNumSMs;
  a.ctas = a.units < kResident ? static_cast<int>(a.units) : kResident;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared(kv_split_kernel<BITS, D, EX, NP, NT>, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
  cfg.blockDim = dim3(32 * kAttnWarps);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  g_kv_launched.store(true, std::memory_order_relaxed);
  e = cudaLaunchKernelEx(&cfg, kv_split_kernel<BITS, D, EX, NP, NT>, a);
  if (e != cudaSuccess || a.whole) return e;
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  // A block a row where pairs have many parts, for more of them at a time.
  if (a.ctas >= kJoinMany * static_cast<long long>(a.seqs) * a.c.heads * a.chunks) {
    cfg.gridDim = join_grid<S::R, 1>(a.ctas);
    return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, S::R, 1, false>, a);
  }
  cfg.gridDim = join_grid<S::R, S::R>(a.ctas);
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, S::R, S::R, false>, a);
}

}  // namespace

template <int D>
cudaError_t KvAttnDim<D>::launch(SplitArgs& a, int bits, bool exact, int np, int nt, cudaStream_t s) {
  constexpr int N2 = D == 256 ? 1 : 2;  // two n-tiles of dim 256 would not fit the registers
  if (exact)
    return bits == 8 ? (nt == 1 ? launch_split<8, D, true, 2, 1>(a, s) : launch_split<8, D, true, 2, N2>(a, s))
                     : (nt == 1 ? launch_split<4, D, true, 2, 1>(a, s) : launch_split<4, D, true, 2, N2>(a, s));
  if (np == 2) return bits == 8 ? launch_split<8, D, false, 2, 1>(a, s) : launch_split<4, D, false, 2, 1>(a, s);
  return bits == 8 ? (nt == 1 ? launch_split<8, D, false, 1, 1>(a, s) : launch_split<8, D, false, 1, N2>(a, s))
                   : (nt == 1 ? launch_split<4, D, false, 1, 1>(a, s) : launch_split<4, D, false, 1, N2>(a, s));
}

template <int D>
cudaError_t KvAttnDim<D>::take_error(unsigned int* code) {
  return take_record(g_kv_attn_error, code);
}

template <int D>
cudaError_t KvAttnDim<D>::take_check(unsigned int* code) {
  return take_check_word(code);
}

#endif  // XQ_KV_ATTN_IMPL

}  // namespace xq
