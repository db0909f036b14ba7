// Attention over the quantized KV cache for many 16-bit query rows a KV head
// (a prefix that a whole batch shares, a long run of query tokens): tiles of
// 128 rows x 64 keys on the tcgen05 tensor cores.
//
// Mathematics: as in kv_attn.cuh, o = sum_j 2^(s_j - e) v_j and l alike, per
// row, with a reference e that moves only when a weight would leave its
// range. Both products take their A operand from tensor memory (queries,
// 128 rows = lanes; then weights, which a row's thread writes where it read
// the scores: no shuffles, no shared memory) and their B operand, the
// dequantized tile, from shared memory. Everything enters as fp16; K and V are
// code * d / 2^x, where 2^x, from the part's largest finite block scale (for V
// of each 32 elements), keeps them in range. Scales more than 2^21 (8-bit codes)
// or 2^25 (4-bit) below that largest one lose a bit for each factor of 2. For
// bf16 queries the products are rounded to one number (11 bits, 8 finer than the
// output's). For fp16 ones they are two, P = 2, which hold all 19 bits of a code
// times its scale: one would nearly double the output's error (4.1e-4 against
// 2.8e-4 relative, of which rounding the output is 2.1e-4). fp32 queries never come here: a tensor
// core's accumulator loses a little at each product added to it, and the 24
// products of a tile in three bf16 pieces brought errors to 2.5e-6 .. 4e-6,
// growing with the length, where the split kernel's are 4e-7.
//
// Roles: 8 warps for the softmax (a thread a row), 8 that unpack, in two groups
// with a tile each in turn, and one that issues the products. Scores are
// computed two tiles ahead of the outputs where tensor memory has the columns
// (128 rows), else one. Raw tiles come by bulk copies, two of a group's ahead.
//
// Not finite: a K scale gives its key's column NaN, which the rows that do not
// see the key mask; a V scale is 0 in the operand, and the rows that see its key
// are told which block to end as NaN (kOddV). Large scores: see `far`.
//
// What bounds it, in clocks a tile at dim 128, Q8_0 (the tensor cores need 1024
// with two row tiles and one piece; taken before what the paragraph above adds, 3 %):
//   256 rows: 2600, most of it a softmax thread's 64 scores (tensor memory
//     there and back, maximum, exponentials); 3500 with two pieces. Twice the
//     softmax warps would have 72 registers a thread: slower (104 us for 74 of
//     a 64-sequence batch over 32768 shared keys).
//   128 rows: 1600, the unpacking warps', of which a group spends 2800 on its
//     tile (5400 with 16-byte copies by every thread).
// Before a part's first scores come some 20000 (page ids, the part's scales,
// the first tile, and instructions seen for the first time: hence the rolled
// loops outside the tiles'), after its last weights 6000 for the results.
// Whole calls, 8 KV heads over 32768 keys: 256 bf16 rows 69 us (34 GFLOP, 500
// TFLOP/s), 128 bf16 rows 48 us, 256 fp16 rows 81 us.
// Work is cut as in kv_attn.cuh: units of 64 keys, one CTA an SM.
#pragma once

#include "kv_attn.cuh"

namespace xq {

constexpr int kTileRows = 128;  // of one accumulator
constexpr int kTileChunk = 2 * kTileRows;  // rows of a pair's chunk, two tiles
constexpr int kTileKeys = 64;
static_assert(kTileKeys == kAttnUnit, "both kernels cut the line in the same units");
constexpr int kTileSoft = 4, kTileConv = 8;  // warps: of a row tile's softmax; that unpack
constexpr int kTileWarps = 2 * kTileSoft + kTileConv + 1;
constexpr int kTileHead = 6;  // units of time a pair costs besides its keys

// P: fp16 pieces of K and of V, 2 where outputs are fp16.
template <int BITS, int D, int P>
struct TileShape {
  static constexpr int NB = D / 32;
  static constexpr int kRow = D * BITS / 8, kChunks = kRow / 16, kWords = kRow / 4;
  // Operands in 8 x 16-byte core matrices. Neighbours in N are 144 bytes apart, K's in K 16 more than 8 of those, so that
  // the unpacking warps' 16-byte stores spread over the banks.
  static constexpr int kSbo = 144;
  static constexpr int kKLbo = kTileKeys / 8 * kSbo + 16, kVLbo = D / 8 * kSbo;
  static constexpr int kOperand = D / 8 * kKLbo;  // one piece of K or of V: 64 keys x dim
  static_assert(kOperand >= kTileKeys / 8 * kVLbo && kOperand % 16 == 0, "V's is the smaller");
  static constexpr int kBufs = 2;  // of K and of V
  static constexpr int kRawCodes = kTileKeys * kRow, kRawScales = kTileKeys * NB * 2;
  static constexpr int kRaw = 2 * (kRawCodes + kRawScales);
  static constexpr int kOffV = kBufs * P * kOperand, kOffRaw = kOffV + kBufs * P * kOperand;
  // The tile's scales, ready for use: K's [64][NB], V's [NB][64], fp16.
  static constexpr int kScaleK = kTileKeys * NB * 2, kScales = 2 * kScaleK;  // a table for each group
  // The part's largest scale comes to 2^kUp .. 2^(kUp + 1): with codes of 128 or 8 at most, products stay within 2^15, and
  // scales down to 2^-(14 + kUp) of it are normal fp16 numbers, 11 bits as stored. (2^0: 2^-14 of it, and 3 % errors at 2^-20.)
  static constexpr int kUp = BITS == 8 ? 7 : 11;
  static constexpr int kRawStages = 2;  // of a group of unpacking warps
  static constexpr int kOffScale = kOffRaw + 2 * kRawStages * kRaw;
  static constexpr int kSmem = kOffScale + 2 * kScales;
  // Tensor memory columns: queries and scores of the two row tiles (or two buffers of scores of one), outputs. The weights
  // take the scores' columns, which the row's thread has read by then.
  static constexpr int kColS = D, kColO = kColS + 2 * kTileKeys, kCols = kColO + 2 * D;
  static constexpr int kAlloc = kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512 && kSmem <= 227 * 1024 - 1536, "one CTA fits the SM");  // and its static shared memory
};

template <int D>
struct KvTileDim {
  static cudaError_t launch(SplitArgs& a, int bits, bool two_pieces, cudaStream_t s);
  static cudaError_t take_error(unsigned int* index, unsigned int* wait);
  static cudaError_t take_check(unsigned int* code);
};

#ifdef XQ_KV_ATTN_IMPL

namespace {

__device__ unsigned int g_kv_tile_error;  // a wait that ran out
constexpr long long kTileWait = 1ll << 32;

constexpr unsigned kOddV = 16;  // the tile has V blocks that are not finite

// Barriers: of each row tile (Q), of each scores buffer (S; P and O, its weights and their products) and of each
// operand buffer and raw stage, as a barrier's parity tells a phase only from the next.
enum TileBar { kBarDrain, kBarQ, kBarS = kBarQ + 2, kBarP = kBarS + 2, kBarO = kBarP + 2, kBarK = kBarO + 2, kBarKFree = kBarK + 2,
               kBarV = kBarKFree + 2, kBarVFree = kBarV + 2, kBarRaw = kBarVFree + 2, kBars = kBarRaw + 4 };

// Barrier of `threads` threads that gives the or of their predicates.
__device__ __forceinline__ bool group_any(int id, int threads, bool p) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.s32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<int>(p)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// Loads and stores of tensor memory are a whole warp's: hence __syncwarp() where its threads may have parted.

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Magnitudes of an fp16 pair, 0 for what is not finite.
__device__ __forceinline__ __half2 finite_abs(uint32_t w) {
  const __half2 h = __habs2(*reinterpret_cast<const __half2*>(&w));
  const uint32_t m = *reinterpret_cast<const uint32_t*>(&h) & __hle2_mask(h, __float2half2_rn(65504.0f));
  return *reinterpret_cast<const __half2*>(&m);
}

// Biased exponent of a largest scale (fp32 bits), at least that of fp16's least number: 103 .. 142.
__device__ __forceinline__ unsigned kv_top_exponent(unsigned bits) { return max(bits >> 23, 103u); }

// Bytes (0, 1) and (2, 3) of w as fp16 pairs u - 128 or u - 8.
template <int BITS>
__device__ __forceinline__ void code_halves(uint32_t w, uint32_t (&h)[2]) {
  constexpr uint32_t off = BITS == 8 ? 0x64806480u : 0x64086408u;
  h[0] = ptx::hsub2(prmt(w, 0x64646464u, 0x4140u), off);
  h[1] = ptx::hsub2(prmt(w, 0x64646464u, 0x4342u), off);
}

template <int BITS, int D, int P>
__global__ void __launch_bounds__(32 * kTileWarps, 1) kv_tile_kernel(const __grid_constant__ SplitArgs A) {
  using S = TileShape<BITS, D, P>;
  constexpr int NB = S::NB;
  extern __shared__ __align__(256) uint8_t smem[];
  __shared__ LineShared sh_line;
  __shared__ __align__(8) uint64_t bars[kBars];
  __shared__ uint32_t sh_tmem;
  __shared__ unsigned sh_bad[4];            // tile's 16-key groups without a valid page, and kOddV, by tile & 3
  __shared__ unsigned sh_odd[4][NB][2];     // keys whose V block is not finite, by tile & 3: only where kOddV says so
  __shared__ unsigned sh_top[4][1 + NB];    // largest finite |scale| of the part: K's, V's blocks (fp32 bits), by part & 3
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return ptx::smem_addr(&bars[i]); };
  if (tid == 0) {
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar(kBarQ + b), kTileSoft);
      ptx::mbar_init(bar(kBarS + b), 1);
      ptx::mbar_init(bar(kBarP + b), kTileSoft);
      ptx::mbar_init(bar(kBarO + b), 1);
      ptx::mbar_init(bar(kBarK + b), kTileConv / 2);
      ptx::mbar_init(bar(kBarKFree + b), 1);
      ptx::mbar_init(bar(kBarV + b), kTileConv / 2);
      ptx::mbar_init(bar(kBarVFree + b), 1);
      ptx::mbar_init(bar(kBarRaw + b), 1);
      ptx::mbar_init(bar(kBarRaw + 2 + b), 1);
    }
    ptx::mbar_init(bar(kBarDrain), 1);
    ptx::mbar_init_fence();
  }
  grid_begin(A.late);
  Line line;
  if (!line_begin<kTileWarps>(A, sh_line, &line)) {
    if (A.late) grid_wait();
    return;
  }
  if (warp == kTileWarps - 1) ptx::tmem_alloc(ptx::smem_addr(&sh_tmem), S::kAlloc);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh_tmem;
  auto wait = [&](int i, unsigned parity, unsigned code) {
    return ptx::mbar_wait(bar(i), parity & 1, &g_kv_tile_error, code, kTileWait);
  };
  auto wait_sleep = [&](int i, unsigned parity, unsigned code) {
    return ptx::mbar_wait_sleep(bar(i), parity & 1, &g_kv_tile_error, code, kTileWait);
  };
  const uint32_t base = ptx::smem_addr(smem);
  // Two buffers of scores: of the two row tiles, or taken in turn by the only one. The buffer of row tile r's n-th tile, and
  // how often it was used before.
  const bool two = A.rows > kTileRows;
  auto buffer = [&](int r, unsigned n) { return two ? r : static_cast<int>(n & 1); };
  auto turn = [&](unsigned n) { return two ? n : n >> 1; };
  Part part;

  if (warp == kTileWarps - 1) {
    // ------------------------------------------------ products (issued by one thread). The whole warp walks through the tiles,
    // so that the operands' addresses are its uniform values when the thread comes to the products: one a product, added to
    // a tile's descriptor, not built anew (77 clocks a product otherwise, more than the 32 to 64 it takes).
    constexpr uint32_t idS = ptx::idesc_f16(kTileRows, kTileKeys, false), idO = ptx::idesc_f16(kTileRows, D, false);
    // Scores are computed this many tiles ahead of the outputs.
    const unsigned ahead = two ? 1 : 2;
    const bool lead = ptx::elect_one();
    const uint64_t k_desc = ptx::smem_desc(base, S::kKLbo, S::kSbo), v_desc = ptx::smem_desc(base + S::kOffV, S::kVLbo, S::kSbo);
    const uint32_t at = __shfl_sync(0xffffffffu, tmem, 0);
    auto wait_all = [&](int i, unsigned parity, unsigned code) { return __all_sync(0xffffffffu, wait(i, parity, code)) != 0; };
    bool ok = true;
    unsigned it = 0, scored[2] = {0u, 0u}, done[2] = {0u, 0u}, parts[2] = {0u, 0u};  // tiles so far; of each row tile
    // Row tile r's scores of tile i; last: of the part's row tiles.
    auto scores = [&](int r, unsigned i, bool last) {
      const unsigned b = i % S::kBufs;
      if (r == 0 && !wait_all(kBarK + b, i / S::kBufs, 1)) return false;
      ptx::tc_fence_after();
      const int to = buffer(r, scored[r]++);
      const uint32_t d = __shfl_sync(0xffffffffu, at + S::kColS + to * kTileKeys, 0);
      const uint32_t a = __shfl_sync(0xffffffffu, at + r * (D / 2), 0);
      const uint64_t kd = k_desc + __shfl_sync(0xffffffffu, b * (P * S::kOperand / 16), 0);
      if (lead) {
#pragma unroll
        for (int p = P - 1; p >= 0; --p)  // the smaller piece first
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            ptx::mma_f16_ts(d, a + 8 * k, kd + (p * S::kOperand + 2 * k * S::kKLbo) / 16, idS, p < P - 1 || k > 0);
        if (last) ptx::tc_commit(bar(kBarKFree + b));
        ptx::tc_commit(bar(kBarS + to));
      }
      __syncwarp();
      return true;
    };
    while (ok && line_next(A, line, part)) {
      const int tiles = part.k1 - part.k0;
      const int chunk = part.pair % A.chunks;
      const int last = A.rows - chunk * kTileChunk > kTileRows ? 1 : 0;
      for (int r = 0; r <= last && ok; ++r) ok = wait_all(kBarQ + r, parts[r]++, 2) && scores(r, it, r == last);
      if (ahead == 2 && ok && tiles > 1) ok = scores(0, it + 1, true);
      for (int i = 0; i < tiles && ok; ++i, ++it) {
        const unsigned b = it % S::kBufs;
        for (int r = 0; r <= last && ok; ++r) {
          const int from = buffer(r, done[r]);  // the weights'
          ok = wait_all(kBarP + from, turn(done[r]), 3);
          ++done[r];
          if (r == 0) ok = ok && wait_all(kBarV + b, it / S::kBufs, 4);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t d = __shfl_sync(0xffffffffu, at + S::kColO + r * D, 0);
          const uint32_t a = __shfl_sync(0xffffffffu, at + S::kColS + from * kTileKeys, 0);
          const uint64_t vd = v_desc + __shfl_sync(0xffffffffu, b * (P * S::kOperand / 16), 0);
          if (lead) {
#pragma unroll
            for (int p = P - 1; p >= 0; --p)
#pragma unroll
              for (int k = 0; k < kTileKeys / 16; ++k)
                ptx::mma_f16_ts(d, a + 8 * k, vd + (p * S::kOperand + 2 * k * S::kVLbo) / 16, idO, i > 0 || p < P - 1 || k > 0);
            if (r == last) ptx::tc_commit(bar(kBarVFree + b));
            ptx::tc_commit(bar(kBarO + from));
          }
          __syncwarp();
          if (i + static_cast<int>(ahead) < tiles) ok = scores(r, it + ahead, r == last);
        }
      }
    }
    if (lead) ptx::tc_commit(bar(kBarDrain));  // nothing is in flight when tensor memory is freed
    wait(kBarDrain, 0, 5);
  } else if (warp < 2 * kTileSoft) {
    // ------------------------- softmax, two row tiles: a thread is a row; no thread needs another
    constexpr float kTop = 15.0f, kStart = 11.0f;  // log2 of weights: the largest, and where the reference starts anew
    const int r = warp >> 2, row = r * kTileRows + (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t to = tl + S::kColO + r * D;
    unsigned it = 0, done = 0, parts = 0;
    bool ok = true, left_record = false;
    for (; ok && line_next(A, line, part); ++parts) {
      const int head = part.pair / A.chunks, chunk = part.pair - head * A.chunks;
      const int row0 = chunk * kTileChunk, tiles = part.k1 - part.k0;
      if (row0 + r * kTileRows >= A.rows) {  // not this row tile's
        it += tiles;
        continue;
      }
      const bool mine = row0 + row < A.rows;
      const size_t at = mine ? row_at(A, part.seq, head, row0 + row) : 0;
      const bool live = mine && XQ_IN(at, out_rows(A), kChkKvQuery);
      int lim0 = 0, lim1 = 0;
      if (live) row_range(A, part.seq, part.n, row0 + row, &lim0, &lim1);
      // ---- the row's query into tensor memory: fp16, its largest element at 2^12 .. 2^13; negated for a negative scale (so
      // that cs > 0)
      const uint4* const from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(A.q) + at * D);
      const bool f16 = A.type == kF16;
      auto both = [&](uint32_t w) {
        return f16 ? __half22float2(*reinterpret_cast<const __half2*>(&w))
                   : make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
      };
      uint4 qv[D / 8];  // all of it at once: one round trip to memory
      unsigned mag = 0;  // magnitudes compare as integers
#pragma unroll
      for (int x = 0; x < D / 8; ++x) qv[x] = live ? from[x] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int x = 0; x < D / 8; ++x)
        mag = __vmaxu2(__vmaxu2(__vmaxu2(mag, qv[x].x & 0x7FFF7FFFu), __vmaxu2(qv[x].y & 0x7FFF7FFFu, qv[x].z & 0x7FFF7FFFu)),
                       qv[x].w & 0x7FFF7FFFu);
      const float2 tops2 = both(mag);
      float top = fmaxf(tops2.x, tops2.y);
      int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      ex = ex < -100 ? -100 : ex;
      const float up = (A.scale < 0.0f ? -1.0f : 1.0f) * __uint_as_float(static_cast<unsigned>(127 + 12 - ex) << 23);
      float cs = fabsf(A.scale) * 1.4426950408889634f * __uint_as_float(static_cast<unsigned>(127 - 12 + ex) << 23);
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 16) {
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint4 q = live ? from[c / 4 + x] : make_uint4(0u, 0u, 0u, 0u);
          const float2 a = both(q.x), b = both(q.y), g = both(q.z), d = both(q.w);
          w[4 * x] = half2_of(a.x * up, a.y * up);
          w[4 * x + 1] = half2_of(b.x * up, b.y * up);
          w[4 * x + 2] = half2_of(g.x * up, g.y * up);
          w[4 * x + 3] = half2_of(d.x * up, d.y * up);
        }
        __syncwarp();
        ptx::tmem_st16(tl + r * (D / 2) + c, w);
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(kBarQ + r));

      int key = (first_unit(A, part.n) + part.k0) * kTileKeys;
      float e = kNoKey;
      ptx::f2 l = ptx::pk(0.0f, 0.0f);
      bool far = false;  // some reference of the warp's is past 2^20
      unsigned vx = 0;  // exponents of V's powers of two, 8 bits a block (all ones: the row's elements are NaN)
      for (int i = 0; i < tiles; ++i, ++it, ++done, key += kTileKeys) {
        ok = __all_sync(0xffffffffu, wait(kBarS + buffer(r, done), turn(done), 6));
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t ts = tl + S::kColS + buffer(r, done) * kTileKeys;
        if (i == 0) {  // the part's powers of two, known once its first tile is there (and until its weights are)
          auto power = [&](int x) { return kv_top_exponent(sh_top[parts & 3][x]) - S::kUp; };
          cs = fmaxf(cs * __uint_as_float(power(0) << 23), 1.17549435e-38f);
#pragma unroll
          for (int b = 0; b < NB; ++b) vx |= power(1 + b) << (8 * b);
        }
        const unsigned bad = sh_bad[it & 3];
        if (bad & kOddV) {  // V blocks that are not finite: their elements become NaN in the rows that see the key
          const int from = lim0 > key ? lim0 - key : 0, to = lim1 - key < kTileKeys ? lim1 - key : kTileKeys;
          const unsigned long long sees = from < to ? (~0ull >> (kTileKeys - (to - from))) << from : 0ull;
#pragma unroll 1
          for (int b = 0; b < NB; ++b)
            if (sees & (sh_odd[it & 3][b][0] | static_cast<unsigned long long>(sh_odd[it & 3][b][1]) << 32)) vx |= 0xFFu << (8 * b);
        }
        const bool edge = key < lim0 || key + kTileKeys > lim1 || bad;
        uint32_t sv[2][16];
        // 32 scores from column c on, those that the row does not see as -infinity
        auto load = [&](int c) {
          __syncwarp();
          ptx::tmem_ld16(ts + c, sv[0]);
          ptx::tmem_ld16(ts + c + 16, sv[1]);
          ptx::tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (key + c + x < lim0 || key + c + x >= lim1 || (bad >> ((c + x) >> 4) & 1)) sv[x >> 4][x & 15] = 0xFF800000u;
          }
        };
        float tops4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four chains
        auto largest = [&] {
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 8; y += 2)
              tops4[x] = max3(tops4[x], __uint_as_float(sv[x >> 1][8 * (x & 1) + y]), __uint_as_float(sv[x >> 1][8 * (x & 1) + y + 1]));
        };
        load(32);
        largest();
        load(0);
        largest();
        const float tile_top = fmaxf(fmaxf(tops4[0], tops4[1]), fmaxf(tops4[2], tops4[3])) * cs;
        if (__any_sync(0xffffffffu, tile_top - e > kTop)) {  // the reference of some rows moves
          float next = tile_top - e > kTop ? tile_top - kStart : e;
          next = tile_top - next > kTop ? tile_top : next;  // at 2^27, where fp32's step is 16, 11 less is 16 less
          const float f = ex2(e - next);
          e = next;
          far = __any_sync(0xffffffffu, fabsf(e) > 1048576.0f && e != kNoKey);
          l = ptx::mul2(l, ptx::pk(f, f));
          if (i > 0) {
            ok = __all_sync(0xffffffffu, wait(kBarO + buffer(r, done - 1), turn(done - 1), 7));
            if (!ok) break;
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t w[16];
              ptx::tmem_ld16(to + c, w);
              ptx::tmem_wait_ld();
#pragma unroll
              for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(__uint_as_float(w[x]) * f);
              ptx::tmem_st16(to + c, w);
            }
          }
        }
        // A weight's score times cs minus e is one operation, whose product is not rounded as the one that gave e was. Where that
        // difference counts, with scores past 2^20, the products take the scores' place first.
        float factor = cs;
        if (far) {
          factor = 1.0f;
          __syncwarp();
#pragma unroll 1
          for (int c = 0; c < kTileKeys; c += 16) {
            ptx::tmem_ld16(ts + c, sv[0]);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) sv[0][x] = __float_as_uint(__fmul_rn(__uint_as_float(sv[0][x]), cs));
            ptx::tmem_st16(ts + c, sv[0]);
          }
          ptx::tmem_wait_st();
          load(0);
        }
        const ptx::f2 c2 = ptx::pk(factor, factor), e2 = ptx::pk(-e, -e);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h) load(32);
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const ptx::f2 z =
                ptx::fma2(ptx::pk(__uint_as_float(sv[x >> 4][x & 15]), __uint_as_float(sv[x >> 4][(x & 15) + 1])), c2, e2);
            const float a = ex2(ptx::lo32(z)), d = ex2(ptx::hi32(z));
            l = ptx::add2(l, ptx::pk(a, d));
            w[x / 2] = half2_of(a, d);
          }
          __syncwarp();
          ptx::tmem_st16(ts + 16 * h, w);  // into columns already read
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kBarP + buffer(r, done)));
      }
      if (!ok) break;
      // ---- the part's results
      ok = __all_sync(0xffffffffu, wait_sleep(kBarO + buffer(r, done - 1), turn(done - 1), 9));
      if (!ok) break;
      ptx::tc_fence_after();
      const float sum = ptx::lo32(l) + ptx::hi32(l);
      const bool whole = part.k0 == 0 && part.k1 == part.nu;
      if (A.late && whole) grid_wait();
      const size_t slot = (static_cast<size_t>(blockIdx.x) * 2 + (part.k0 == 0 ? 1 : 0)) * kTileChunk + row;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t w[16];
        __syncwarp();
        ptx::tmem_ld16(to + c, w);
        ptx::tmem_wait_ld();
        const unsigned x2 = vx >> (8 * (c / 32)) & 0xFFu;
        const float f = __uint_as_float(x2 == 0xFFu ? 0x7FC00000u : x2 << 23);
        if (live) {
#pragma unroll
          for (int x = 0; x < 16; x += 4) {
            const float4 y = make_float4(__uint_as_float(w[x]) * f, __uint_as_float(w[x + 1]) * f, __uint_as_float(w[x + 2]) * f,
                                         __uint_as_float(w[x + 3]) * f);
            if (whole)
              finish4(A, D, at, c + x, y, e, sum);
            else if (XQ_IN(slot, A.part_rows, kChkKvPart))
              *reinterpret_cast<float4*>(A.part_o + (slot - row) * D + (c + x) * kTileChunk + row * 4) = y;
          }
        }
      }
      if (live && !whole && XQ_IN(slot, A.part_rows, kChkKvPart))
        *reinterpret_cast<float2*>(A.part_el + slot * 2) = make_float2(e, sum);
      if (!whole && part.k0 == 0) {
        left_record = true;
        if (tid == 0 && XQ_IN(blockIdx.x, A.records, kChkKvPart))
          A.record[blockIdx.x] = make_int4(part.seq, part.pair, line_last(A, line, part), 0);
      }
      ptx::tc_fence_before();
    }
    if (!left_record && tid == 0 && !A.whole && XQ_IN(blockIdx.x, A.records, kChkKvPart))
      A.record[blockIdx.x] = make_int4(0, 0, -1, 0);
  } else {
    // ------------------------------------------------ copying and unpacking
    // Two groups of four warps, each a tile: one's copies and barriers pass while the other unpacks.
    constexpr int kThreads = 32 * kTileConv, kGroup = kThreads / 2, kBarrier = 2;
    const int ct = tid - 64 * kTileSoft, group = ct / kGroup, gt = ct - group * kGroup;
    const int group_shift = A.c.page_shift - 4, groups_page = 1 << group_shift;  // 16-key groups a page
    const int run = groups_page < 4 ? groups_page : 4;                          // those of a tile that lie in one page
    unsigned filled = 0, coming = 0;  // of the raw stages: phases' parities, copies on their way
    const long long v_off = reinterpret_cast<long long>(A.c.v) - reinterpret_cast<long long>(A.c.k);
    unsigned it = 0, parts = 0;
    bool fail = false;
    while (line_next(A, line, part)) {
      const int tiles = part.k1 - part.k0, unit0 = first_unit(A, part.n) + part.k0;
      const int32_t* const table = A.flat ? A.pages : A.pages + static_cast<size_t>(part.seq) * A.page_stride;
      const int line0 = (part.pair / A.chunks) << A.c.page_shift;
      const int groups = (part.n + 15) / 16;  // of the sequence
      // Address of 16-key group gi's page, or 0; its first row within the head's rows.
      auto page_at = [&](int gi) -> long long {
        if (gi >= groups || !XQ_IN(gi >> group_shift, table_len(A), kChkKvTable)) return 0;
        const int page = table[gi >> group_shift];
        if (static_cast<unsigned>(page) < static_cast<unsigned>(A.c.n_pages))
          return reinterpret_cast<long long>(A.c.k) + page * A.c.page_bytes;
        kv_record(kKvBadPage);
        return 0;
      };
      auto row_of = [&](int gi) { return line0 + ((gi & (groups_page - 1)) << 4); };

      // ---- the groups take tiles in turn. Raw tiles come one of its own tiles ahead, page ids one further. A page's rows of a
      // head follow each other: a copy is what a tile has of a page, and each of the group's warps makes those of one kind
      // (K's codes, V's, K's scales, V's; all from one warp, 16 keys each, took some 1900 clocks a tile)
      auto id_at = [&](int i) {
        const int gi = (unit0 + i) * 4 + (lane & 3);
        return i < tiles && gi < groups && XQ_IN(gi >> group_shift, table_len(A), kChkKvTable) ? table[gi >> group_shift] : -1;
      };
      int next_id = id_at(group);
      unsigned miss = 0, next_miss = 0;  // 16-key groups without a valid page: of this tile, of the one on its way
      auto issue = [&](int i, int stage) {
        if (i < tiles) {
          const int gi0 = (unit0 + i) * 4;
          const bool there = static_cast<unsigned>(next_id) < static_cast<unsigned>(A.c.n_pages);
          if (!there && gi0 + (lane & 3) < groups) kv_record(kKvBadPage);
          const long long page = there ? reinterpret_cast<long long>(A.c.k) + next_id * A.c.page_bytes : 0;
          next_id = id_at(i + 2);
          next_miss = __ballot_sync(0xffffffffu, !there) & 15u;
          coming |= 1u << stage;
          constexpr unsigned kCodes = 16 * S::kRow, kScale = 16 * NB * 2;  // of 16 keys
          const uint32_t full = bar(kBarRaw + 2 * group + stage);
          if (gt == 0) ptx::mbar_expect_tx(full, (4 - __popc(next_miss)) * 2 * (kCodes + kScale));
          // a run's 16-key groups before the sequence's end: those after it are in next_miss
          const int have = groups - gi0 < 4 ? groups - gi0 : 4, n = have - lane < run ? have - lane : run;
          if (lane < have && (lane & (run - 1)) == 0 && there) {
            const int kind = gt >> 5, v = kind & 1, row = row_of(gi0 + lane);
            const uint32_t to = base + S::kOffRaw + (S::kRawStages * group + stage) * S::kRaw;
            const uint8_t* const from = reinterpret_cast<const uint8_t*>(page + (v ? v_off : 0));
            if (!XQ_CHECKED(in_pool(A, page - reinterpret_cast<long long>(A.c.k) + (kind < 2 ? row * S::kRow : A.c.scale_off + row * (2 * NB)),
                                    n * (kind < 2 ? kCodes : kScale)), kChkKvTile)) {
            } else if (kind < 2) {
              ptx::bulk_load(to + v * S::kRawCodes + lane * kCodes, from + row * S::kRow, n * kCodes, full);
            } else {
              ptx::bulk_load(to + 2 * S::kRawCodes + v * S::kRawScales + lane * kScale, from + A.c.scale_off + row * (2 * NB),
                             n * kScale, full);
            }
          }
        }
      };
      issue(group, 0);

      float kf = 1.0f, vf[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) vf[b] = 1.0f;
      {
        // ---- the part's largest finite scales (one that is not belongs to the rows that see its key: in the others' way it
        // would leave no power of two for the finite ones): 1 / 17 or 1 / 9 of its bytes, which its tiles then find in L2
        unsigned* const tops = sh_top[parts & 3];
        if (ct <= NB) tops[ct] = 0u;
        if (group_any(kBarrier, kThreads, fail)) break;
        __half2 kt = __float2half2_rn(0.0f), vt[NB % 2 ? NB : NB / 2];  // running maxima; V's by block, pairs of them if even
#pragma unroll
        for (int b = 0; b < (NB % 2 ? NB : NB / 2); ++b) vt[b] = kt;
        const int pieces = tiles * 4 * 2 * NB;  // 16-byte pieces of K's scales, 2 NB a group
        constexpr int kAhead = 4;               // pieces a thread has in flight
        for (int x0 = ct; x0 < pieces; x0 += kThreads * kAhead) {
          long long page[kAhead];
          uint4 k4[kAhead], v4[kAhead];
#pragma unroll
          for (int y = 0; y < kAhead; ++y) {
            const int x = x0 + y * kThreads;
            page[y] = x < pieces ? page_at(unit0 * 4 + x / (2 * NB)) : 0;
          }
#pragma unroll
          for (int y = 0; y < kAhead; ++y) {
            const int x = x0 + y * kThreads, gl = x / (2 * NB), piece = x - gl * 2 * NB, gi = unit0 * 4 + gl;
            k4[y] = v4[y] = make_uint4(0u, 0u, 0u, 0u);
            if (!page[y]) continue;
            const uint8_t* const p = reinterpret_cast<const uint8_t*>(page[y]) + A.c.scale_off + row_of(gi) * (2 * NB) + piece * 16;
            if (!XQ_CHECKED(in_pool(A, p - A.c.k, 16), kChkKvTile)) continue;
            k4[y] = *reinterpret_cast<const uint4*>(p);
            v4[y] = *reinterpret_cast<const uint4*>(p + v_off);
          }
#pragma unroll
          for (int y = 0; y < kAhead; ++y) {
            const int x = x0 + y * kThreads, gl = x / (2 * NB), piece = x - gl * 2 * NB;
            uint32_t kw[4] = {k4[y].x, k4[y].y, k4[y].z, k4[y].w}, vw[4] = {v4[y].x, v4[y].y, v4[y].z, v4[y].w};
            const int left = (part.n - (unit0 * 4 + gl) * 16) * NB - piece * 8;  // scales of the sequence from the piece on
            if (left < 8) {
#pragma unroll
              for (int h = 0; h < 8; ++h)
                if (h >= left) {
                  kw[h / 2] &= h & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                  vw[h / 2] &= h & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                }
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              kt = __hmax2(kt, finite_abs(kw[h]));
              const __half2 a = finite_abs(vw[h]);
              if (NB % 2 == 0) {
                vt[h % (NB / 2 > 0 ? NB / 2 : 1)] = __hmax2(vt[h % (NB / 2 > 0 ? NB / 2 : 1)], a);
              } else {
#pragma unroll
                for (int q = 0; q < NB; ++q) {
                  if ((piece * 8 + 2 * h) % NB == q) vt[q] = __hmax2(vt[q], __half2half2(__low2half(a)));
                  if ((piece * 8 + 2 * h + 1) % NB == q) vt[q] = __hmax2(vt[q], __half2half2(__high2half(a)));
                }
              }
            }
          }
        }
#pragma unroll
        for (int b = 0; b <= NB; ++b) {
          // magnitudes order like their bits
          const __half2 h = b == 0 ? kt : vt[NB % 2 ? b - 1 : (b - 1) / 2];
          const float lo = __half2float(__low2half(h)), hi = __half2float(__high2half(h));
          const unsigned bits = b == 0 || NB % 2 ? max(__float_as_uint(lo), __float_as_uint(hi))
                                                 : __float_as_uint((b - 1) % 2 ? hi : lo);
          const unsigned m = __reduce_max_sync(0xffffffffu, bits);
          if (lane == 0) atomicMax(&tops[b], m);
        }
        if (group_any(kBarrier, kThreads, fail)) break;
        auto down = [](unsigned t) { return __uint_as_float((254 + S::kUp - kv_top_exponent(t)) << 23); };
        kf = down(tops[0]);
#pragma unroll
        for (int b = 0; b < NB; ++b) vf[b] = down(tops[1 + b]);
      }

      uint8_t* const scales = smem + S::kOffScale + group * S::kScales;
      const unsigned it0 = it;
      for (int i = group, stage = 0; i < tiles; i += 2, stage ^= 1) {
        it = it0 + i;
        fail |= !wait_sleep(kBarRaw + 2 * group + stage, filled >> stage, 12);
        filled ^= 1u << stage;
        coming &= ~(1u << stage);
        // the group's last tile has been unpacked
        if (group_any(kBarrier + 1 + group, kGroup, fail)) break;
        miss = next_miss;
        issue(i + 2, stage ^ 1);
        const uint8_t* const raw = smem + S::kOffRaw + (S::kRawStages * group + stage) * S::kRaw;
        const int left = part.n - (unit0 + i) * kTileKeys;  // keys of the sequence from the tile's first on
        // ---- scales: scaled, and 0 for keys that are not there (whose codes may be anything). A V scale that is not finite
        // is 0 too, as the product takes it to all rows, and the rows that see its key are told
        auto key_gone = [&](int key) { return key >= left || (miss >> (key >> 4) & 1); };
        auto finite = [](__half h) { return (__half_as_ushort(h) & 0x7C00u) != 0x7C00u; };
        const __half* const kd = reinterpret_cast<const __half*>(raw + 2 * S::kRawCodes);
        const __half* const vd = kd + S::kRawScales / 2;
        bool odd = false;
        for (int x = gt; x < kTileKeys * NB; x += kGroup) {
          const int key = x / NB, blk = x - key * NB;
          const bool gone = key_gone(key), zero = gone || !finite(vd[x]);
          odd |= zero && !gone;
          float f = vf[0];
#pragma unroll
          for (int q = 1; q < NB; ++q) f = blk == q ? vf[q] : f;
          const float dk = gone ? 0.0f : __half2float(kd[x]) * kf, dv = zero ? 0.0f : __half2float(vd[x]) * f;
          reinterpret_cast<__half*>(scales)[x] = __float2half_rn(dk);
          reinterpret_cast<__half*>(scales + S::kScaleK)[blk * kTileKeys + key] = __float2half_rn(dv);
        }
        if (group_any(kBarrier + 1 + group, kGroup, odd)) {
          unsigned* const keys = &sh_odd[it & 3][0][0];
          if (gt < 2 * NB) keys[gt] = 0u;
          group_any(kBarrier + 1 + group, kGroup, false);
#pragma unroll 1
          for (int x = gt; x < kTileKeys * NB; x += kGroup) {
            const int key = x / NB, blk = x - key * NB;
            if (!key_gone(key) && !finite(vd[x])) atomicOr(&keys[2 * blk + (key >> 5)], 1u << (key & 31));
          }
          miss |= kOddV;
        }
        // ---- K: operand rows are keys. A task is a key's 16-byte chunk
        const unsigned b = it % S::kBufs, turn = it / S::kBufs;  // tiles take the buffers, and the groups the tiles, in turn
        if (turn > 0) fail |= !wait_sleep(kBarKFree + b, turn - 1, 10);
        if (gt == 0) sh_bad[it & 3] = miss;
        uint8_t* const ko = smem + b * P * S::kOperand;
#pragma unroll
        for (int x = 0; x < (kTileKeys * S::kChunks + kGroup - 1) / kGroup; ++x) {
          const int c = x * kGroup + gt, key = c / S::kChunks, ch = c - key * S::kChunks;
          if (key < kTileKeys) {
            const uint4 u4 = *reinterpret_cast<const uint4*>(raw + c * 16);
            const uint32_t u[4] = {u4.x, u4.y, u4.z, u4.w};
            const int si = key * NB + (BITS == 8 ? ch / 2 : ch);
            const uint32_t dd = reinterpret_cast<const uint16_t*>(scales)[si] * 0x10001u;
            uint8_t* const to = ko + (key >> 3) * S::kSbo + (key & 7) * 16;
#pragma unroll
            for (int z = 0; z < (BITS == 8 ? 2 : 4); ++z) {  // 8 elements each
              const uint32_t w0 = BITS == 8 ? u[2 * z] : (u[2 * (z & 1)] >> (z & 2 ? 4 : 0)) & 0x0F0F0F0Fu;
              const uint32_t w1 = BITS == 8 ? u[2 * z + 1] : (u[2 * (z & 1) + 1] >> (z & 2 ? 4 : 0)) & 0x0F0F0F0Fu;
              uint8_t* const cell = to + (ch * (BITS == 8 ? 2 : 4) + z) * S::kKLbo;
              uint32_t h[4], v[4];
              code_halves<BITS>(w0, *reinterpret_cast<uint32_t(*)[2]>(&h[0]));
              code_halves<BITS>(w1, *reinterpret_cast<uint32_t(*)[2]>(&h[2]));
#pragma unroll
              for (int q = 0; q < 4; ++q) v[q] = ptx::hmul2(h[q], dd);
              *reinterpret_cast<uint4*>(cell) = make_uint4(v[0], v[1], v[2], v[3]);
              if (P == 2) {  // what the rounding left, exact
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = hfma2_of(h[q], dd, v[q] ^ 0x80008000u);
                *reinterpret_cast<uint4*>(cell + S::kOperand) = make_uint4(v[0], v[1], v[2], v[3]);
              }
            }
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kBarK + b));
        // ---- V: operand rows are elements. A task is a word (4 code bytes) of 8 keys
        if (turn > 0) fail |= !wait_sleep(kBarVFree + b, turn - 1, 11);
        uint8_t* const vo = smem + S::kOffV + b * P * S::kOperand;
#pragma unroll 1
        for (int x = 0; x < (8 * S::kWords + kGroup - 1) / kGroup; ++x) {
          const int c = x * kGroup + gt, kg = c / S::kWords, word = c - kg * S::kWords;
          if (kg < 8) {
            const int blk = BITS == 8 ? word / 8 : word / 4;
            uint32_t u[8];
            const uint4 d4 = *reinterpret_cast<const uint4*>(scales + S::kScaleK + (blk * kTileKeys + kg * 8) * 2);
            const uint32_t d2[4] = {d4.x, d4.y, d4.z, d4.w};  // the 8 keys' scales of the block
#pragma unroll
            for (int k = 0; k < 8; ++k)
              u[k] = *reinterpret_cast<const uint32_t*>(raw + S::kRawCodes + (kg * 8 + k) * S::kRow + word * 4);
            // elements 4 word + i; of a 4-bit block 32 blk + 4 (word % 4) + i, and 16 further on those of the high halves
#pragma unroll
            for (int z = 0; z < (BITS == 8 ? 1 : 2); ++z) {
              const int e0 = BITS == 8 ? 4 * word : 32 * blk + 4 * (word & 3) + 16 * z;
              uint8_t* const to = vo + kg * S::kVLbo + (e0 >> 3) * S::kSbo + (e0 & 7) * 16;
              uint32_t v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = BITS == 8 ? u[k] : (u[k] >> (4 * z)) & 0x0F0F0F0Fu;
              uint32_t r[P][4][4];  // [piece][element][key pair]
#pragma unroll
              for (int k = 0; k < 8; k += 2) {
                const uint32_t lo = prmt(v[k], v[k + 1], 0x5140u), hi = prmt(v[k], v[k + 1], 0x7362u);
                const uint32_t dd = d2[k / 2];
                uint32_t h[4];
                code_halves<BITS>(lo, *reinterpret_cast<uint32_t(*)[2]>(&h[0]));
                code_halves<BITS>(hi, *reinterpret_cast<uint32_t(*)[2]>(&h[2]));
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  r[0][y][k / 2] = ptx::hmul2(h[y], dd);
                  if (P == 2) r[P - 1][y][k / 2] = hfma2_of(h[y], dd, r[0][y][k / 2] ^ 0x80008000u);
                }
              }
#pragma unroll
              for (int q = 0; q < P; ++q)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  *reinterpret_cast<uint4*>(to + q * S::kOperand + y * 16) =
                      make_uint4(r[q][y][0], r[q][y][1], r[q][y][2], r[q][y][3]);
            }
          }
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kBarV + b));
      }
      it = it0 + tiles;
      ++parts;
      // the raw stages are free for the next part once every thread is here
      if (group_any(kBarrier, kThreads, fail)) break;
    }
    for (int s = 0; s < 2; ++s)  // no copy is in flight when the CTA ends, even after a wait that ran out
      if (coming >> s & 1) wait_sleep(kBarRaw + 2 * group + s, filled >> s, 12);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kTileWarps - 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, S::kAlloc);
  }
  if (A.late) grid_wait();
}

template <int BITS, int D, int P>
cudaError_t launch_tile_attn(SplitArgs& a, cudaStream_t s) {
  using S = TileShape<BITS, D, P>;
  a.ctas = a.units < kNumSMs ? static_cast<int>(a.units) : kNumSMs;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = allow_shared(kv_tile_kernel<BITS, D, P>, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.ctas));
  cfg.blockDim = dim3(32 * kTileWarps);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  g_kv_launched.store(true, std::memory_order_relaxed);
  e = cudaLaunchKernelEx(&cfg, kv_tile_kernel<BITS, D, P>, a);
  if (e != cudaSuccess || a.whole) return e;
  constexpr int kRowsBlock = 4;
  cfg.gridDim = join_grid<kTileChunk, kRowsBlock>(a.ctas);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, kTileChunk, kRowsBlock, true>, a);
}

}  // namespace

template <int D>
cudaError_t KvTileDim<D>::launch(SplitArgs& a, int bits, bool two_pieces, cudaStream_t s) {
  if (bits == 8) return two_pieces ? launch_tile_attn<8, D, 2>(a, s) : launch_tile_attn<8, D, 1>(a, s);
  return two_pieces ? launch_tile_attn<4, D, 2>(a, s) : launch_tile_attn<4, D, 1>(a, s);
}

template <int D>
cudaError_t KvTileDim<D>::take_error(unsigned int* index, unsigned int* wait) {
  const cudaError_t e = take_record(g_kv_attn_error, index);
  return e == cudaSuccess ? take_record(g_kv_tile_error, wait) : e;
}

template <int D>
cudaError_t KvTileDim<D>::take_check(unsigned int* code) {
  return take_check_word(code);
}

#endif  // XQ_KV_ATTN_IMPL

}  // namespace xq
