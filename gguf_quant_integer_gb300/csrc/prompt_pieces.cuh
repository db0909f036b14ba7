// Prompt attention of fp32 rows on the tcgen05 tensor cores: every operand as two fp16 numbers.
//
// x = 2^-s (hi + lo) with hi and lo of 11 bits each, so a product takes three: hi hi, hi lo, lo hi (what is left out is
// 2^-21 of it at most, in the mean 2^-24). A first kernel (prompt_split) makes the pieces of K and V in the workspace, a
// row's thread those of its query in tensor memory. Powers of two keep them in fp16's range: one for a row of Q and for a
// tile of K, which the softmax applies to the scores, and for V one for each column of a tile, which is applied to the
// tile's output.
//
// Sums: a tensor core's accumulator cuts off, towards 0, what an fp32 addition rounds, so it only ever holds one tile's sum,
// small products first; outputs are added up in registers. Scores of large and small weights: a weight is 2^(z - e), its
// reference e as in prompt_tile.cuh, hi cut off and lo the rest.
//
// Pieces below fp16's normal range are off by 2^-39 of the tile's largest (K) or the column's (V). Where a tile's rows differ by
// more than 2^12 in size, that may show: in K, for scores that could pass 2^20, of which it is 2^-20 or more (c_tile below); in V,
// for results below 2^-15 of the tile's largest row, which has no weight there. Such rows, as those that see something not
// finite, or keys that belong to two sequences (which bounds out of order allow), are computed by themselves (one_row).
//
// A CTA has 128 rows. Q and the weights are the products' first operands in tensor memory (Q in shared memory was read at
// 107 clocks a product, of which the tensor cores need 64), scores are double-buffered there, so that the products of a
// tile pass beside the softmax of the two before it. With head size 256 a CTA has half of V's columns, and tiles of 64
// keys. Roles: two groups of 4 warps share a tile's softmax (a thread has half a row's keys; the halves' maxima are
// exchanged), 4 warps add up outputs (a thread a row), then one that issues the products of Q and K, one those of weights
// and V, one that copies, and one that brings the tiles' powers of two and looks through V. Items as in prompt_tile.cuh.
//
// Loops are rolled wherever registers allow: many roles' code at once does not fit the instruction caches (unrolled, the
// softmax's two passes alone made 5 sequences of 33 to 1500 take 195 us instead of 156).
//
// What bounds it, at head size 128: a tile's 48 products take the tensor cores some 3100 clocks; the outputs' way out of tensor
// memory, which has no room for a second one beside them, and the scores', softmax and weights' make it some 4000. An item
// costs some 12000 more (queries, first scores, results). 5 sequences of 33 to 1500, 32/8 heads: 136 us and 15 for the split,
// 252 TFLOP/s of fp32 work (760 of the tensor cores'), error against 64 bits 4.9e-7 to 5.5e-7 (plain fp32 5.7e-7 to 6.9e-7).
// Tried and slower: a softmax group a tile (156 us for 154), queries by threads from memory (18000 clocks an item), outputs in
// two column groups with barriers of their own (160: products of 64 columns are not twice as fast), eight output warps (154
// for 149), the next item's queries before the last tile's softmax (157).
#pragma once

#include "prompt_items.cuh"

namespace xq {

// The workspace.
struct PromptPieces {
  __half *k, *v;           // [2][tokens][kv_heads][dim], hi and lo
  float *k_power, *v_power;  // [slots][kv_heads] (negative: rows far apart), [slots][kv_heads][dim]: what the pieces are to be multiplied by
  float* v_most;           // [slots][kv_heads]: the largest value, 0 unless rows are far apart
  int *k_owner, *v_owner;  // [slots][kv_heads]: the slot's sequence; -1: none, -2: another sequence's too
  int slots;               // tiles of keys of all sequences: tile j of sequence b has slot starts[b] / keys + b + j
  size_t bytes;
};
constexpr int prompt_piece_keys(int dim) { return dim == 256 ? 64 : 128; }
constexpr int prompt_piece_halves(int dim) { return dim == 256 ? 2 : 1; }

cudaError_t launch_prompt_split(const PromptArgs& a, const PromptPieces& w, cudaStream_t s);

template <int D>
struct PromptPiecesDim {
  static cudaError_t launch(PromptTileArgs& a, const PromptPieces& w, cudaStream_t s);
  static cudaError_t take_error(unsigned int* index, unsigned int* wait);
  static cudaError_t take_check(unsigned int* code);
};

#ifdef XQ_PROMPT_TILE_IMPL

namespace {

template <int D>
struct PieceShape {
  static constexpr int kKeys = prompt_piece_keys(D), kHalves = prompt_piece_halves(D), kV = D / kHalves;
  static constexpr int kBox = D % 64 == 0 ? 64 : 32, kLine = kBox * 2, kBoxes = kV / kBox;  // of a part: kV elements of a row
  static constexpr int kStage = kKeys * kV * 2;  // a part of a piece of a tile
  // Stages of K parts and of V parts. A tile's are K's lo parts, then K's hi parts (all of these are needed at a time);
  // V lo, V hi.
  static constexpr int kKParts = 2 * kHalves, kKStages = D == 128 ? 4 : D == 96 ? 5 : 8, kVStages = D == 128 || D == 96 ? 2 : 4;
  // An item's queries come through K's stages before its first tile: boxes of 128 rows x 32 fp32 columns.
  static constexpr int kQBoxes = kStage / (kRows * 128), kQParts = D / 32 / kQBoxes;
  static constexpr int kStages = kKStages + kVStages;
  static constexpr int kRowsOut = 4 * 4096;  // results on their way out: 32 rows x 128 bytes of each output warp
  static constexpr int kSmem = kStages * kStage + kRowsOut + 1024;
  static constexpr int kColO = 2 * kKeys, kColQ = kColO + kV, kAlloc = 512;  // scores twice, outputs, Q's hi and lo
  static constexpr int kWarps = 16;
  // registers a thread: of the softmax, the outputs, the others; four warps each, launched with 128
  static constexpr int kRegsSoft = 112, kRegsOut = 208, kRegsRest = 80;
  static_assert(2 * kRegsSoft + kRegsOut + kRegsRest <= 4 * 128, "an increase beyond what was launched with waits forever");
  static_assert(D / 32 % kQBoxes == 0 && kKStages >= kQParts && kKStages > kHalves && kVStages >= 2 && kColQ + D <= kAlloc && kSmem <= 227 * 1024 - 8 * 1024, "one CTA fits the SM");
  static constexpr uint64_t kSwizzle = kLine == 128 ? 2ull : 4ull;
  static constexpr uint64_t kCommon = (1ull << 46) | (kSwizzle << 61) | (static_cast<uint64_t>(8 * kLine / 16) << 32);
  static constexpr uint64_t kDescK = kCommon | (1ull << 16);
  static constexpr uint64_t kDescV = kCommon | (static_cast<uint64_t>(kKeys * kLine / 16) << 16);
};

enum PieceBar { kQbDrain, kQbQ, kQbTop, kQbItem, kQbItemFree = kQbItem + 2, kQbS = kQbItemFree + 2, kQbP = kQbS + 2,
                kQbO = kQbP + 2, kQbOFree = kQbO + 2, kQbPower = kQbOFree + 2, kQbPowerFree = kQbPower + 2, kQbChecked = kQbPowerFree + 2,
                kQbSum = kQbChecked + 2, kQbFull = kQbSum + 2 };  // then a stage's full and free: K's, V's

// Two fp32 numbers as fp16 pairs: hi (each cut off to 11 bits; exact above 2^-14) and what is left.
__device__ __forceinline__ void halves_of(float a, float b, uint32_t* hi, uint32_t* lo) {
  const float ah = __uint_as_float(__float_as_uint(a) & 0xFFFFE000u), bh = __uint_as_float(__float_as_uint(b) & 0xFFFFE000u);
  *hi = pack2<kF16>(ah, bh);
  const ptx::f2 rest = ptx::add2(ptx::pk(a, b), ptx::pk(-ah, -bh));
  *lo = pack2<kF16>(ptx::lo32(rest), ptx::hi32(rest));
}

template <int D>
__global__ void __launch_bounds__(32 * PieceShape<D>::kWarps, 1)
    prompt_pieces_kernel(const __grid_constant__ PromptTileArgs P, const __grid_constant__ PromptPieces W) {
  using S = PieceShape<D>;
  constexpr int kKeys = S::kKeys, kStages = S::kStages, kQbFree = kQbFull + kStages, kOut = 8, kScores = 12, kOutputs = 13, kLoad = 14, kAux = 15;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kQbFull + 2 * kStages];
  __shared__ uint32_t sh_tmem;
  __shared__ Item sh_item[2];
  __shared__ unsigned sh_odd[2];                        // rows of the item have to be looked at (1) or computed by themselves (2)
  __shared__ unsigned sh_most[2];                       // largest value of the item's tiles whose V rows are far apart, as bits
  __shared__ float sh_k[2];                             // the tile's powers of two, by tile & 1
  __shared__ __align__(16) float sh_v[2][S::kV];
  __shared__ float sh_ref[2][kRows];                    // the rows' references, by tile & 1
  __shared__ float sh_top[2][2][kRows];                 // largest scores of the halves, by tile & 1 and half
  __shared__ float sh_sum[2][2][kRows];                 // sums of weights, by item & 1 and half
  const PromptArgs& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return ptx::smem_addr(&bars[i]); };
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u, stages = base, rows_out = base + kStages * S::kStage;
  if (tid == 0) {
    ptx::mbar_init(bar(kQbDrain), 2);
    ptx::mbar_init(bar(kQbQ), 8);
    ptx::mbar_init(bar(kQbTop), 8);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar(kQbItem + b), 1);
      ptx::mbar_init(bar(kQbItemFree + b), 15);
      ptx::mbar_init(bar(kQbS + b), 1);
      ptx::mbar_init(bar(kQbP + b), 8);
      ptx::mbar_init(bar(kQbO + b), 1);
      ptx::mbar_init(bar(kQbOFree + b), 4);
      ptx::mbar_init(bar(kQbPower + b), 1);
      ptx::mbar_init(bar(kQbPowerFree + b), 12);
      ptx::mbar_init(bar(kQbChecked + b), 1);
      ptx::mbar_init(bar(kQbSum + b), 8);
    }
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(bar(kQbFull + i), 1);
      ptx::mbar_init(bar(kQbFree + i), 1);
    }
    ptx::mbar_init_fence();
  }
  if (warp == kScores) ptx::tmem_alloc(ptx::smem_addr(&sh_tmem), S::kAlloc);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh_tmem;
  auto wait = [&](int i, unsigned parity, unsigned code) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar(i), parity & 1, &g_prompt_wait, code, P.wait)) != 0;
  };
  auto arrive = [&](int i) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(i));
  };
  unsigned items = 0;  // taken so far
  auto take = [&](Item& it) {  // false: the last one is done (or a wait ran out)
    if (!wait(kQbItem + (items & 1), items >> 1, 1)) return false;
    it = sh_item[items & 1];
    return it.n >= 0;
  };
  auto leave = [&] {  // its last use of the item's place
    arrive(kQbItemFree + (items & 1));
    ++items;
  };
  const int group = A.heads / A.kv_heads;
  unsigned n = 0;  // tiles before this one
  bool ok = true;
  Item it;

  if (warp >= kScores) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsRest));
  if (warp == kLoad) {
    // ------------------------------------------------ copies
    Walk w;
    walk_begin(A, P.tokens_tile, w);
    const bool lead = ptx::elect_one();
    unsigned loaded[2] = {0u, 0u};  // parts of K, of V
    // the next stage of a ring, its last contents done with; -1 if a wait ran out
    auto stage = [&](int v) {
      const unsigned ring = v ? S::kVStages : S::kKStages, turn = loaded[v] / ring, st = (v ? S::kKStages : 0) + loaded[v] % ring;
      if (turn > 0) ok = ok && wait(kQbFree + st, turn - 1, 4);
      ++loaded[v];
      return ok ? static_cast<int>(st) : -1;
    };
    // a part of a piece: kV elements of kKeys rows
    auto load = [&](int v, const CUtensorMap* map, int x, int y, int z) {
      const int st = stage(v);
      if (st < 0 || !lead) return;
      ptx::mbar_expect_tx(bar(kQbFull + st), S::kStage);
#pragma unroll
      for (int b = 0; b < S::kBoxes; ++b)
        tma_load_3d(stages + st * S::kStage + b * (kKeys * S::kLine), map, x + b * S::kBox, y, z, bar(kQbFull + st));
    };
    Item next;
    auto find = [&](unsigned round) {
      const long long rank = static_cast<long long>(round) * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      if (!next_item<kKeys, S::kHalves>(P, 1, rank, w, next)) next.n = -1;
    };
    find(0);
    for (unsigned round = 0; ok; ++round) {
      it = next;
      const bool there = it.n >= 0;
      if (round >= 2 && !wait(kQbItemFree + (round & 1), (round >> 1) + 1, 2)) break;
      if (lead) {
        sh_item[round & 1] = it;
        sh_odd[round & 1] = 0u;
        sh_most[round & 1] = 0u;
        ptx::mbar_arrive(bar(kQbItem + (round & 1)));
      }
      __syncwarp();
      if (!there || P.withhold) break;
      for (int i = 0; i < S::kQParts && ok; ++i) {
        const int st = stage(0);
        if (st < 0 || !lead) continue;
        ptx::mbar_expect_tx(bar(kQbFull + st), S::kQBoxes * P.pack * P.tokens_tile * 128);
#pragma unroll
        for (int b = 0; b < S::kQBoxes; ++b)
          tma_load_3d(stages + st * S::kStage + b * (kRows * 128), &P.q, (i * S::kQBoxes + b) * 32, it.head, it.first + it.place, bar(kQbFull + st));
      }
      __syncwarp();
      // in the order of the products: K a tile before V
      const int kv = it.head / group;
      for (int j = it.begin[0]; j <= it.end[0] && ok; ++j) {
        const int row = it.first + j * kKeys;
        for (int c = 0; c < S::kKParts && j < it.end[0]; ++c)
          load(0, &P.k, c % S::kHalves * S::kV, kv, c < S::kHalves ? row + A.tokens : row);
        if (j == it.begin[0]) find(round + 1);  // while the first copies are on their way
        for (int p = 1; p >= 0 && j > it.begin[0]; --p) load(1, &P.v, it.half * S::kV, kv, row - kKeys + p * A.tokens);
      }
      __syncwarp();
    }
    // copies in flight land before the CTA ends
    for (int v = 0; v < 2; ++v) {
      const unsigned ring = v ? S::kVStages : S::kKStages;
      for (unsigned i = loaded[v] > ring ? loaded[v] - ring : 0; i < loaded[v]; ++i)
        if (!wait(kQbFull + (v ? S::kKStages : 0) + i % ring, i / ring, 5)) break;
    }
  } else if (warp == kScores) {
    // ------------------------------------------------ products of Q and K, issued by one thread
    constexpr uint32_t idS = ptx::idesc_f16(kRows, kKeys, false);
    constexpr int kSteps = S::kBox / 16;
    const bool lead = ptx::elect_one();
    const uint32_t at = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t stage0 = stages >> 4;
    auto full = [&](unsigned i) { return wait(kQbFull + i % S::kKStages, i / S::kKStages, 7); };
    // Q piece p, part c x the K part number i
    auto qk = [&](uint32_t d, int p, int c, unsigned i, bool first, bool last) {
      const uint64_t kd = S::kDescK | (stage0 + __shfl_sync(0xffffffffu, i % S::kKStages * (S::kStage / 16), 0));
      const uint32_t q = __shfl_sync(0xffffffffu, at + S::kColQ + p * (D / 2) + c * (S::kV / 2), 0);
      if (lead) {
#pragma unroll
        for (int k = 0; k < S::kV / 16; ++k)
          ptx::mma_f16_ts(d, q + 8 * k, kd + k / kSteps * (kKeys * S::kLine / 16) + k % kSteps * 2, idS, !first || k > 0);
        if (last) ptx::tc_commit(bar(kQbFree + i % S::kKStages));
      }
      __syncwarp();
    };
    while (ok && take(it)) {
      ok = wait(kQbQ, items, 6);
      for (int i = 0; i < S::kQParts && lead; ++i) ptx::mbar_arrive(bar(kQbFree + (items * S::kQParts + n * S::kKParts + i) % S::kKStages));
      __syncwarp();
      leave();
      for (int j = it.begin[0]; j < it.end[0] && ok; ++j, ++n) {
        const unsigned lo = items * S::kQParts + n * S::kKParts, hi = lo + S::kHalves;
        const uint32_t d = __shfl_sync(0xffffffffu, at + (n & 1) * kKeys, 0);
        // the weights that lay there are done with
        ok = n < 2 || wait(kQbO + (n & 1), (n >> 1) - 1, 8);
#pragma unroll
        for (int c = 0; c < S::kHalves; ++c) {
          ok = ok && full(lo + c);
          if (!ok) break;
          ptx::tc_fence_after();
          qk(d, 0, c, lo + c, c == 0, true);
        }
#pragma unroll
        for (int c = 0; c < S::kHalves; ++c) {
          ok = ok && full(hi + c);
          if (!ok) break;
          ptx::tc_fence_after();
          qk(d, 1, c, hi + c, false, false);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < S::kHalves; ++c) qk(d, 0, c, hi + c, false, true);
        if (lead) ptx::tc_commit(bar(kQbS + (n & 1)));
        __syncwarp();
      }
    }
    if (lead) ptx::tc_commit(bar(kQbDrain));  // nothing is in flight when tensor memory is freed
    wait(kQbDrain, 0, 10);
  } else if (warp == kOutputs) {
    // ------------------------------------------------ products of weights and V: a warp of its own, so that its waits and the
    // other's pass beside each other's products
    constexpr uint32_t idO = ptx::idesc_f16(kRows, S::kV, false) | (1u << 16);
    const bool lead = ptx::elect_one();
    const uint32_t at = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t stage0 = stages >> 4;
    auto full = [&](unsigned i) { return wait(kQbFull + S::kKStages + i % S::kVStages, i / S::kVStages, 9); };
    while (ok && take(it)) {
      leave();
      for (int j = it.begin[0]; j < it.end[0] && ok; ++j, ++n) {
        const unsigned b = n & 1, lo = 2 * n, hi = lo + 1, st_lo = S::kKStages + lo % S::kVStages, st_hi = S::kKStages + hi % S::kVStages;
        ok = wait(kQbChecked + b, n >> 1, 14) && full(lo) && full(hi) && (n == 0 || wait(kQbOFree + ((n - 1) & 1), (n - 1) >> 1, 16)) &&
             wait(kQbP + b, n >> 1, 8);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t d = __shfl_sync(0xffffffffu, at + S::kColO, 0), a = __shfl_sync(0xffffffffu, at + b * kKeys, 0);
        const uint64_t lo_d = S::kDescV | (stage0 + __shfl_sync(0xffffffffu, st_lo * (S::kStage / 16), 0));
        const uint64_t hi_d = S::kDescV | (stage0 + __shfl_sync(0xffffffffu, st_hi * (S::kStage / 16), 0));
        if (lead) {
          // weights of 32 keys: 16 columns of hi, 16 of lo
          auto pv = [&](int p, uint64_t vd, bool first) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              ptx::mma_f16_ts(d, a + k / 2 * 32 + p * 16 + k % 2 * 8, vd + k * (2 * 8 * S::kLine / 16), idO, !first || k > 0);
          };
          pv(0, lo_d, true);
          ptx::tc_commit(bar(kQbFree + st_lo));
          pv(1, hi_d, false);
          pv(0, hi_d, false);
          ptx::tc_commit(bar(kQbFree + st_hi));
          ptx::tc_commit(bar(kQbO + b));
        }
        __syncwarp();
      }
    }
    if (lead) ptx::tc_commit(bar(kQbDrain));
    wait(kQbDrain, 0, 10);
  } else if (warp >= kAux) {
    // ------------------------------------------------ powers of two, and V's elements that are not finite
    for (; ok && take(it); leave()) {
      const int kv = it.head / group;
      for (int j = it.begin[0]; j < it.end[0]; ++j, ++n) {
        const unsigned b = n & 1;
        const int slot = it.first / kKeys + it.sequence + j;
        const bool known = XQ_IN(slot, W.slots, kChkPromptSlot);
        const size_t place = (known ? static_cast<size_t>(slot) * A.kv_heads : 0) + kv;
        float vp[S::kV / 32];
#pragma unroll
        for (int x = 0; x < S::kV / 32; ++x) vp[x] = W.v_power[place * D + it.half * S::kV + x * 32 + lane];
        const float kp = W.k_power[place], most = W.v_most[place];
        const bool whole = known && W.k_owner[place] == it.sequence && W.v_owner[place] == it.sequence;
        ok = n < 2 || wait(kQbPowerFree + b, (n >> 1) - 1, 17);
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < S::kV / 32; ++x) sh_v[b][x * 32 + lane] = vp[x];
        if (lane == 0) {
          sh_k[b] = kp;
          if (!whole) atomicOr(&sh_odd[items & 1], 2u);
          if (most > 0.0f) atomicMax(&sh_most[items & 1], __float_as_uint(most));
        }
        arrive(kQbPower + b);
        const unsigned st[2] = {S::kKStages + 2 * n % S::kVStages, S::kKStages + (2 * n + 1) % S::kVStages};  // V's lo and hi
        ok = wait(kQbFull + st[0], 2 * n / S::kVStages, 15) && wait(kQbFull + st[1], (2 * n + 1) / S::kVStages, 15);
        if (!ok) break;
        if (masked<kKeys>(P, it.place, j * kKeys)) {
          constexpr int kBlock = kKeys * S::kLine;  // bytes of a column block
          const int end = min(it.n - j * kKeys, kKeys) * S::kLine;  // of the sequence's rows in each; the pieces behind are anyone's
          const uint32_t from = stages + st[1] * S::kStage + lane * 16;
          bool found = false;
          for (int x = end + lane * 16; x < kBlock; x += 32 * 16) {
#pragma unroll
            for (int i = 0; i < 2 * S::kBoxes; ++i)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(stages + st[i % 2] * S::kStage + i / 2 * kBlock + x),
                           "r"(0u) : "memory");
          }
#pragma unroll 8
          for (int x = 0; x < S::kStage; x += 32 * 16) {
            if ((x + lane * 16) % kBlock >= end) continue;
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from + x));
            if (odd_halves<kF16>(w[0]) | odd_halves<kF16>(w[1]) | odd_halves<kF16>(w[2]) | odd_halves<kF16>(w[3])) {
              found = true;
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] &= ~((odd_halves<kF16>(w[i]) >> 15) * 0xFFFFu);
              asm volatile("st.shared.v4.b32 [%4], {%0, %1, %2, %3};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(from + x) : "memory");
            }
          }
          if (found) atomicOr(&sh_odd[items & 1], 1u);
          ptx::fence_proxy_async_smem();
        }
        arrive(kQbChecked + b);
      }
      if (!ok) break;
    }
  } else {
    const int row = (warp & 3) * 32 + lane, token = row / P.pack, part = row - token * P.pack;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    if (warp < kOut) {
      // ---------------------------------------------- softmax: a thread has half a row's keys of a tile, the other group of warps the other
      // half
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsSoft));
      const int half = warp >> 2;
      float cq = 0.0f;  // the row's: of the scale and its query's power of two
      constexpr float kTop = 15.0f, kStart = 11.0f;  // log2 of weights: the largest, and where the reference starts anew
      const bool turned = !(A.scale > 0.0f);  // as in prompt_tile.cuh
      const float sign = A.scale < 0.0f ? -1.0f : 0.0f, cs = A.scale == 0.0f ? 1.0f : fabsf(A.scale) * 1.4426950408889634f;
      // An item's queries into tensor memory (the scores of the last tile before, which the group has had, were the last
      // product of those there): hi and lo, the row's largest at 2^14 .. 2^15, half of the columns by each group. (In unrolled
      // loops, whose instructions are waited for at every item: 20000 clocks instead of 4000.)
      auto query = [&](const Item& q) {
        const bool there = token < P.tokens_tile && q.place + token < q.n;
        const unsigned first = items * S::kQParts + n * S::kKParts;  // of the ring's parts
        for (int i = 0; i < S::kQParts && ok; ++i) ok = wait(kQbFull + (first + i) % S::kKStages, (first + i) / S::kKStages, 22);
        if (!ok) return;
        // columns 4 c .. 4 c + 3
        auto chunk = [&](int c) {
          const unsigned box = c / 8, st = (first + box / S::kQBoxes) % S::kKStages;
          float4 x;
          asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                       : "r"(stages + st * S::kStage + box % S::kQBoxes * (kRows * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)));
          return x;
        };
        unsigned top = 0u;
#pragma unroll 4
        for (int c = 0; c < D / 4; ++c) {
          const float4 x = chunk(c);
          top = max(top, max(max(__float_as_uint(x.x) & 0x7FFFFFFFu, __float_as_uint(x.y) & 0x7FFFFFFFu),
                             max(__float_as_uint(x.z) & 0x7FFFFFFFu, __float_as_uint(x.w) & 0x7FFFFFFFu)));
        }
        // a row that is not finite is computed by itself: its pieces need not hold it
        const unsigned biased = !there || top == 0u ? 127u : min(254u, max(1u, 268u - min(267u, top >> 23)));
        const float up = there ? __uint_as_float(biased << 23) : 0.0f;
        cq = cs * (biased == 254u ? __uint_as_float(1u << 22) : __uint_as_float((254u - biased) << 23));
#pragma unroll 1
        for (int c = half * (D / 8); c < (half + 1) * (D / 8); c += 4) {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float4 x = chunk(c + i);
            x = there ? make_float4(x.x * up, x.y * up, x.z * up, x.w * up) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            halves_of(x.x, x.y, &hi[2 * i], &lo[2 * i]);
            halves_of(x.z, x.w, &hi[2 * i + 1], &lo[2 * i + 1]);
          }
          __syncwarp();
          tmem_st8(tl + S::kColQ + 2 * c, hi);
          tmem_st8(tl + S::kColQ + D / 2 + 2 * c, lo);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        arrive(kQbQ);
      };
      for (; ok && take(it); leave()) {
        query(it);
        if (!ok) break;
        const int place = it.place + token;
        const int lim1 = place + 1, lim0 = A.window ? max(0, lim1 - A.window) : 0;
        float e = -3.402823466e38f, l = 0.0f;
        for (int j = it.begin[0]; j < it.end[0]; ++j, ++n) {
          const unsigned b = n & 1;
          const int key = j * kKeys + half * (kKeys / 2);
          ok = wait(kQbPower + b, n >> 1, 18) && wait(kQbS + b, n >> 1, 11);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t ts = tl + b * kKeys + half * (kKeys / 2);
          const float kp = sh_k[b], c_tile = cq * fabsf(kp);
          // rows far apart: what K's pieces leave out comes to this much of a score (2^15 2^-25 for each product)
          if (kp < 0.0f && !(c_tile * (D * 0x1p-10f) < 0x1p-20f)) l = NAN;
          const bool edge = masked<kKeys>(P, it.place, j * kKeys);
          // 32 scores from column c on, those that the row does not see as -infinity
          ptx::f2 s[16];
          auto load = [&](int c) {
            uint32_t v[32];
            __syncwarp();
            tmem_ld32(ts + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 2) s[x / 2] = ptx::pk(__uint_as_float(v[x]), __uint_as_float(v[x + 1]));
            if (turned) {
#pragma unroll
              for (int x = 0; x < 16; ++x) s[x] = ptx::mul2(s[x], ptx::pk(sign, sign));
            }
            if (edge) {
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const int k = key + c + 2 * x;
                s[x] = ptx::pk(k < lim0 || k >= lim1 ? -INFINITY : ptx::lo32(s[x]), k + 1 < lim0 || k + 1 >= lim1 ? -INFINITY : ptx::hi32(s[x]));
              }
            }
          };
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c = 0; c < kKeys / 2; c += 32) {
            load(c);
#pragma unroll
            for (int x = 0; x < 16; ++x) tops[x & 3] = max3(tops[x & 3], ptx::lo32(s[x]), ptx::hi32(s[x]));
          }
          float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * c_tile;
          sh_top[b][half][row] = top;
          arrive(kQbTop);
          ok = wait(kQbTop, n, 23);
          if (!ok) break;
          top = fmaxf(top, sh_top[b][half ^ 1][row]);
          if (top - e > kTop) {  // the row's reference moves
            const float next = top - kStart;
            l *= ex2(e - next);
            e = next;
          }
          if (half == 0) {
            ok = n < 2 || wait(kQbOFree + b, (n >> 1) - 1, 19);
            if (!ok) break;
            sh_ref[b][row] = e;
          }
          const ptx::f2 c2 = ptx::pk(c_tile, c_tile), e2 = ptx::pk(-e, -e);
          ptx::f2 sum[2] = {ptx::pk(0.0f, 0.0f), ptx::pk(0.0f, 0.0f)};
#pragma unroll 1
          for (int c = 0; c < kKeys / 2; c += 32) {
            load(c);
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const ptx::f2 z = ptx::fma2(s[x], c2, e2);
              const float u = ex2(ptx::lo32(z)), v = ex2(ptx::hi32(z));
              sum[x & 1] = ptx::add2(sum[x & 1], ptx::pk(u, v));
              halves_of(u, v, &hi[x], &lo[x]);
            }
            __syncwarp();
            ptx::tmem_st16(ts + c, hi);  // into columns already read
            ptx::tmem_st16(ts + c + 16, lo);
          }
          sum[0] = ptx::add2(sum[0], sum[1]);
          l += ptx::lo32(sum[0]) + ptx::hi32(sum[0]);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          arrive(kQbP + b);
          if (lane == 0) ptx::mbar_arrive(bar(kQbPowerFree + b));
        }
        if (!ok) break;
        sh_sum[items & 1][half][row] = l;
        arrive(kQbSum + (items & 1));
      }
    } else {
      // ---------------------------------------------- outputs: a thread is a row
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsOut));
      for (; ok && take(it); leave()) {
        const int place = it.place + token, kv = it.head / group;
        const bool live = token < P.tokens_tile && place < it.n;
        ptx::f2 o[S::kV / 2];
#pragma unroll
        for (int x = 0; x < S::kV / 2; ++x) o[x] = ptx::pk(0.0f, 0.0f);
        float e = -3.402823466e38f;  // the outputs' reference
        for (int j = it.begin[0]; j < it.end[0]; ++j, ++n) {
          const unsigned b = n & 1;
          ok = wait(kQbP + b, n >> 1, 20) && wait(kQbO + b, n >> 1, 12) && wait(kQbPower + b, n >> 1, 21);
          if (!ok) break;
          ptx::tc_fence_after();
          const float ref = sh_ref[b][row];
          if (__any_sync(0xffffffffu, ref != e)) {
            const float g = ex2(e - ref);
            e = ref;
#pragma unroll
            for (int x = 0; x < S::kV / 2; ++x) o[x] = ptx::mul2(o[x], ptx::pk(g, g));
          }
          const uint32_t from = tl + S::kColO;
#pragma unroll
          for (int c = 0; c < S::kV; c += 32) {
            uint32_t v[32];
            tmem_ld32(from + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 p = *reinterpret_cast<const float4*>(&sh_v[b][c + x]);
              o[(c + x) / 2] = ptx::fma2(ptx::pk(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), ptx::pk(p.x, p.y), o[(c + x) / 2]);
              o[(c + x) / 2 + 1] =
                  ptx::fma2(ptx::pk(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), ptx::pk(p.z, p.w), o[(c + x) / 2 + 1]);
            }
          }
          ptx::tc_fence_before();
          if (j + 1 < it.end[0]) arrive(kQbOFree + b);  // behind the last tile the results go through it
          arrive(kQbPowerFree + b);
        }
        if (!ok) break;
        // ---- the rows' results
        ok = wait(kQbSum + (items & 1), items >> 1, 13);
        if (!ok) break;
        const float sum = sh_sum[items & 1][0][row] + sh_sum[items & 1][1][row], inv = 1.0f / sum;
        const int at = (it.first + place) * A.heads + it.head + part;
        const int to = live && XQ_IN(at, static_cast<size_t>(A.tokens) * A.heads, kChkPromptRow) ? at : -1;
        ptx::f2 odd = ptx::pk(sum * 0.0f, 0.0f);  // NaN if anything is not finite
#pragma unroll
        for (int x = 0; x < S::kV / 2; ++x) odd = ptx::fma2(o[x], ptx::pk(0.0f, 0.0f), odd);
        float top = 0.0f;  // the row's largest result
        // Back into tensor memory, and from there 32 columns at a time in a rolled loop (see above), through shared memory, so
        // that a store has 4 rows' lines, not 32.
#pragma unroll
        for (int c = 0; c < S::kV; c += 16) {
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            const ptx::f2 u = ptx::mul2(o[(c + x) / 2], ptx::pk(inv, inv));
            w[x] = __float_as_uint(ptx::lo32(u)), w[x + 1] = __float_as_uint(ptx::hi32(u));
            top = max3(top, fabsf(ptx::lo32(u)), fabsf(ptx::hi32(u)));
          }
          ptx::tmem_st16(tl + S::kColO + c, w);
        }
        ptx::tmem_wait_st();
        const uint32_t mine = rows_out + (warp & 3) * 4096 + lane * 128, other = rows_out + (warp & 3) * 4096 + (lane >> 3) * 128;
#pragma unroll 1
        for (int c = 0; c < S::kV; c += 32) {
          uint32_t v[32];
          tmem_ld32(tl + S::kColO + c, v);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((i ^ (lane & 7)) << 4)), "r"(v[4 * i]), "r"(v[4 * i + 1]),
                         "r"(v[4 * i + 2]), "r"(v[4 * i + 3])
                         : "memory");
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float4 y;
            asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(y.x), "=f"(y.y), "=f"(y.z), "=f"(y.w)
                         : "r"(other + i * 512 + (((lane & 7) ^ ((4 * i + (lane >> 3)) & 7)) << 4))
                         : "memory");
            const int row_to = __shfl_sync(0xffffffffu, to, 4 * i + (lane >> 3));
            if (row_to >= 0)
              *reinterpret_cast<float4*>(static_cast<float*>(A.out) + static_cast<size_t>(row_to) * D + it.half * S::kV + c + (lane & 7) * 4) = y;
          }
          __syncwarp();
        }
        ptx::tc_fence_before();
        arrive(kQbOFree + ((n - 1) & 1));
        const unsigned look = sh_odd[items & 1];
        bool meets = (look & 2u) != 0;  // pieces that do not hold the values, or an element that was put to 0
        const float most = __uint_as_float(sh_most[items & 1]);
        meets |= most > 0.0f && !(top >= most * 0x1p-15f);
        if (look & 1u) {
          const int lim1 = place + 1, lim0 = A.window ? max(0, lim1 - A.window) : 0;
#pragma unroll 1
          for (int j = it.begin[0]; j < it.end[0]; ++j)
            if (masked<kKeys>(P, it.place, j * kKeys))
#pragma unroll 1
              for (int key = j * kKeys; key < min((j + 1) * kKeys, it.n); ++key) {
                bool odd_v = false;
                for (int x = lane; x < D; x += 32)
                  odd_v |= !isfinite(static_cast<const float*>(A.v)[(static_cast<size_t>(it.first) + key) * A.v_stride + static_cast<size_t>(kv) * D + x]);
                if (__any_sync(0xffffffffu, odd_v)) meets |= key >= lim0 && key < lim1;
              }
        }
        unsigned again = __ballot_sync(0xffffffffu, live && (meets || !(ptx::lo32(odd) + ptx::hi32(odd) == 0.0f && sum > 0.0f)));
        while (again) {
          const int src = __ffs(again) - 1;
          again &= again - 1;
          one_row<kF32, D>(A, it.first, __shfl_sync(0xffffffffu, place, src), it.head + __shfl_sync(0xffffffffu, part, src), it.half * S::kV, (it.half + 1) * S::kV);
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kScores) ptx::tmem_dealloc(tmem, S::kAlloc);
}

}  // namespace

template <int D>
cudaError_t PromptPiecesDim<D>::launch(PromptTileArgs& p, const PromptPieces& w, cudaStream_t s) {
  using S = PieceShape<D>;
  g_kv_launched.store(true, std::memory_order_relaxed);
  const PromptArgs& a = p.a;
  const long long ks = static_cast<long long>(a.kv_heads) * D;
  if (!encode_tma_heads_f32(&p.q, a.q, D, a.heads, a.tokens, a.tokens == 1 ? static_cast<long long>(a.heads) * D : a.q_stride, p.pack, p.tokens_tile) ||
      !encode_tma_heads(&p.k, false, w.k, D, a.kv_heads, 2 * a.tokens, ks, S::kBox, 1, S::kKeys) ||
      !encode_tma_heads(&p.v, false, w.v, D, a.kv_heads, 2 * a.tokens, ks, S::kBox, 1, S::kKeys))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> allowed{0};
  static std::atomic<int> registers{0};
  cudaError_t e = allow_shared(prompt_pieces_kernel<D>, S::kSmem, allowed);
  if (e == cudaSuccess && registers.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, prompt_pieces_kernel<D>);
    if (e == cudaSuccess) registers.store(f.numRegs, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  // the split of registers goes by 128 a thread at launch: with fewer its increase would wait forever
  if (registers.load(std::memory_order_relaxed) != 128) return cudaErrorInvalidConfiguration;
  const long long items = (a.tokens / p.tokens_tile + static_cast<long long>(a.batch)) * p.units * S::kHalves;
  prompt_pieces_kernel<D><<<static_cast<int>(items < 152 ? items : 152), 32 * S::kWarps, S::kSmem, s>>>(p, w);
  return cudaGetLastError();
}

template <int D>
cudaError_t PromptPiecesDim<D>::take_error(unsigned int* index, unsigned int* wait) {
  const cudaError_t e = take_record(g_prompt_error, index);
  return e != cudaSuccess ? e : take_record(g_prompt_wait, wait);
}
template <int D>
cudaError_t PromptPiecesDim<D>::take_check(unsigned int* code) {
  return take_check_word(code);
}

#endif  // XQ_PROMPT_TILE_IMPL

}  // namespace xq
