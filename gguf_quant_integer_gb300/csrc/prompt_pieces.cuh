// Prompt attention of fp32 rows on the tcgen05 tensor cores: every operand as two fp16 numbers.
//
// x = 2^-s (hi + lo) with hi and lo of 11 bits each, so a product takes three: hi hi, hi lo, lo hi (what is left out is
// 2^-21 of it at most, in the mean 2^-24). A first kernel (prompt_split) makes the pieces of Q, K and V in the workspace.
// Powers of two keep them in fp16's range: one for each row of Q and of K, which the softmax applies to the scores, and for
// V one for each column of a tile of keys, which is applied to the tile's output.
//
// Sums: a tensor core's accumulator cuts off, towards 0, what an fp32 addition rounds, so it only ever holds one tile's sum,
// small products first; outputs are added up in registers. Scores of large and small weights: a weight is 2^(z - e), its
// reference e as in prompt_tile.cuh, hi cut off and lo the rest.
//
// V rows of a tile that differ by more than 2^12 in size would cost the small ones bits where no large one has a weight;
// rows of such tiles (as those that see something not finite) are computed by themselves (one_row).
//
// A CTA has 128 rows; scores and a tile's output are double-buffered in tensor memory, so that the products of tile j + 1
// pass beside the softmax of tile j and the addition of tile j - 1. With head size 256 it has half of V's columns, and
// tiles of 64 keys. Roles: warps 0-3 softmax (a thread a row), 4-7 outputs (a thread a row), then products, copies, and two
// warps that bring the tiles' powers of two and look through V. Items as in prompt_tile.cuh.
#pragma once

#include "prompt_items.cuh"

namespace xq {

// The workspace.
struct PromptPieces {
  __half *q, *k, *v;       // [2][tokens][heads][dim], hi and lo
  float *q_power, *k_power;  // [tokens][heads], [kv_heads][tokens]: what a row's pieces are to be multiplied by
  float* v_power;          // [slots][kv_heads][dim]
  int* owner;              // [slots][kv_heads][halves]: the slot's sequence; -1: none, -2: rows too far apart
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
  static constexpr int kQPart = kRows * kV * 2, kQ = kHalves * kQPart;                      // of a piece
  static constexpr int kStage = kKeys * kV * 2;  // a part of a piece of a tile
  static constexpr int kStages = D == 128 ? 4 : D == 64 ? 11 : D == 96 ? 6 : 5;
  static constexpr int kLoads = 2 * kHalves + 2;  // of a tile: K's lo parts, K's hi parts, V lo, V hi
  // A tile's scores are computed before the outputs of the one before it. Its K parts then come while V's two are there: with
  // head size 256 the stages for that do not fit.
  static constexpr bool kAhead = kStages >= 2 * kHalves + 2;
  static constexpr int kSmem = 2 * kQ + kStages * kStage + 1024;
  static constexpr int kColO = 2 * kKeys, kAlloc = 512;
  static constexpr int kWarps = 12;
  static_assert(kColO + 2 * kV <= kAlloc && kSmem <= 227 * 1024 - 6 * 1024, "one CTA fits the SM");
  static constexpr uint64_t kSwizzle = kLine == 128 ? 2ull : 4ull;
  static constexpr uint64_t kCommon = (1ull << 46) | (kSwizzle << 61) | (static_cast<uint64_t>(8 * kLine / 16) << 32);
  static constexpr uint64_t kDescK = kCommon | (1ull << 16);
  static constexpr uint64_t kDescV = kCommon | (static_cast<uint64_t>(kKeys * kLine / 16) << 16);
};

enum PieceBar { kQbDrain, kQbQ, kQbQFree, kQbItem, kQbItemFree = kQbItem + 2, kQbS = kQbItemFree + 2, kQbP = kQbS + 2, kQbO = kQbP + 2,
                kQbOFree = kQbO + 2, kQbPower = kQbOFree + 2, kQbPowerFree = kQbPower + 2, kQbChecked = kQbPowerFree + 2,
                kQbSum = kQbChecked + 2, kQbFull = kQbSum + 2 };

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
  constexpr int kKeys = S::kKeys, kStages = S::kStages, kQbFree = kQbFull + kStages, kMma = 8, kLoad = 9, kAux = 10;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kQbFull + 2 * kStages];
  __shared__ uint32_t sh_tmem;
  __shared__ Item sh_item[2];
  __shared__ unsigned sh_odd[2];                        // rows of the item have to be looked at (1) or computed by themselves (2)
  __shared__ __align__(16) float sh_k[2][kKeys];        // the tile's powers of two, by tile & 1
  __shared__ __align__(16) float sh_v[2][S::kV];
  __shared__ float sh_move[2][kRows];                   // factor of what a row summed up before the tile, by tile & 1
  __shared__ float sh_sum[2][kRows];                    // sums of weights, by item & 1
  const PromptArgs& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto bar = [&](int i) { return ptx::smem_addr(&bars[i]); };
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u, stages = base + 2 * S::kQ;
  if (tid == 0) {
    ptx::mbar_init(bar(kQbDrain), 1);
    ptx::mbar_init(bar(kQbQ), 1);
    ptx::mbar_init(bar(kQbQFree), 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar(kQbItem + b), 1);
      ptx::mbar_init(bar(kQbItemFree + b), 11);
      ptx::mbar_init(bar(kQbS + b), 1);
      ptx::mbar_init(bar(kQbP + b), 4);
      ptx::mbar_init(bar(kQbO + b), 1);
      ptx::mbar_init(bar(kQbOFree + b), 4);
      ptx::mbar_init(bar(kQbPower + b), 2);
      ptx::mbar_init(bar(kQbPowerFree + b), 8);
      ptx::mbar_init(bar(kQbChecked + b), 2);
      ptx::mbar_init(bar(kQbSum + b), 4);
    }
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(bar(kQbFull + i), 1);
      ptx::mbar_init(bar(kQbFree + i), 1);
    }
    ptx::mbar_init_fence();
  }
  if (warp == kMma) ptx::tmem_alloc(ptx::smem_addr(&sh_tmem), S::kAlloc);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh_tmem;
  auto wait = [&](int i, unsigned parity, unsigned code) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar(i), parity & 1, &g_prompt_wait, code, kPromptWait)) != 0;
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

  if (warp == kLoad) {
    // ------------------------------------------------ copies
    Walk w;
    walk_begin(A, P.tokens_tile, w);
    const bool lead = ptx::elect_one();
    unsigned loaded = 0;
    auto load = [&](const CUtensorMap* map, int x, int y, int z) {  // a part of a piece: kV elements of kKeys rows
      const unsigned st = loaded % kStages;
      if (loaded >= kStages) ok = ok && wait(kQbFree + st, loaded / kStages - 1, 4);
      ++loaded;
      if (!ok || !lead) return;
      ptx::mbar_expect_tx(bar(kQbFull + st), S::kStage);
#pragma unroll
      for (int b = 0; b < S::kBoxes; ++b)
        tma_load_3d(stages + st * S::kStage + b * (kKeys * S::kLine), map, x + b * S::kBox, y, z, bar(kQbFull + st));
    };
    for (unsigned round = 0; ok; ++round) {
      const long long rank = static_cast<long long>(round) * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      const bool there = next_item<kKeys, S::kHalves>(P, 1, rank, w, it);
      if (!there) it.n = -1;
      if (round >= 2 && !wait(kQbItemFree + (round & 1), (round >> 1) + 1, 2)) break;
      if (lead) {
        sh_item[round & 1] = it;
        sh_odd[round & 1] = 0u;
        ptx::mbar_arrive(bar(kQbItem + (round & 1)));
      }
      __syncwarp();
      if (!there) break;
      if (round > 0 && !wait(kQbQFree, round - 1, 3)) break;
      if (lead) {
        ptx::mbar_expect_tx(bar(kQbQ), 2 * P.pack * P.tokens_tile * D * 2);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int b = 0; b < D / S::kBox; ++b)
            tma_load_3d(base + p * S::kQ + b * (kRows * S::kLine), &P.q, b * S::kBox, it.head, p * A.tokens + it.first + it.place, bar(kQbQ));
      }
      const int kv = it.head / group;
      for (int j = it.begin[0]; j < it.end[0] && ok; ++j) {
        const int row = it.first + j * kKeys;
        for (int c = 0; c < S::kHalves; ++c) load(&P.k, c * S::kV, kv, row + A.tokens);
        for (int c = 0; c < S::kHalves; ++c) load(&P.k, c * S::kV, kv, row);
        load(&P.v, it.half * S::kV, kv, row + A.tokens);
        load(&P.v, it.half * S::kV, kv, row);
      }
      __syncwarp();
    }
    // copies in flight land before the CTA ends
    for (unsigned i = loaded > kStages ? loaded - kStages : 0; i < loaded; ++i)
      if (!wait(kQbFull + i % kStages, i / kStages, 5)) break;
  } else if (warp == kMma) {
    // ------------------------------------------------ products, issued by one thread
    constexpr uint32_t idS = ptx::idesc_f16(kRows, kKeys, false), idO = ptx::idesc_f16(kRows, S::kV, false) | (1u << 16);
    constexpr int kSteps = S::kBox / 16;
    const bool lead = ptx::elect_one();
    const uint32_t at = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t stage0 = stages >> 4, q0 = base >> 4;
    auto full = [&](unsigned ld, unsigned code) { return wait(kQbFull + ld % kStages, ld / kStages, code); };
    auto release = [&](unsigned ld) {
      if (lead) ptx::tc_commit(bar(kQbFree + ld % kStages));
      __syncwarp();
    };
    // Q piece p, part c x the K part of load ld
    auto qk = [&](uint32_t d, int p, int c, unsigned ld, bool first) {
      const uint64_t kd = S::kDescK | (stage0 + __shfl_sync(0xffffffffu, (ld % kStages) * (S::kStage / 16), 0));
      const uint64_t qd = S::kDescK | (q0 + (p * S::kQ + c * S::kQPart) / 16);
      if (lead) {
#pragma unroll
        for (int k = 0; k < S::kV / 16; ++k) {
          const int step = k % kSteps * 2, box = k / kSteps;
          ptx::mma_f16_ss(d, qd + box * (kRows * S::kLine / 16) + step, kd + box * (kKeys * S::kLine / 16) + step, idS, !first || k > 0);
        }
      }
      __syncwarp();
    };
    auto scores = [&](unsigned t, bool last) {
      const unsigned ld = t * S::kLoads;
      const uint32_t d = __shfl_sync(0xffffffffu, at + (t & 1) * kKeys, 0);
      for (int c = 0; c < S::kHalves && ok; ++c) {
        ok = full(ld + c, 7);
        if (!ok) return;
        ptx::tc_fence_after();
        qk(d, 0, c, ld + c, c == 0);
        release(ld + c);
      }
      for (int c = 0; c < S::kHalves && ok; ++c) {
        ok = full(ld + S::kHalves + c, 7);
        if (!ok) return;
        ptx::tc_fence_after();
        qk(d, 1, c, ld + S::kHalves + c, false);
      }
      for (int c = 0; c < S::kHalves; ++c) {
        qk(d, 0, c, ld + S::kHalves + c, false);
        release(ld + S::kHalves + c);
      }
      if (lead) {
        ptx::tc_commit(bar(kQbS + (t & 1)));
        if (last) ptx::tc_commit(bar(kQbQFree));
      }
      __syncwarp();
    };
    auto outputs = [&](unsigned t) {
      const unsigned ld = t * S::kLoads + 2 * S::kHalves;
      ok = wait(kQbP + (t & 1), t >> 1, 8) && wait(kQbChecked + (t & 1), t >> 1, 14) && full(ld, 9) && full(ld + 1, 9) &&
           (t < 2 || wait(kQbOFree + (t & 1), (t >> 1) - 1, 16));
      if (!ok) return;
      ptx::tc_fence_after();
      const uint32_t d = __shfl_sync(0xffffffffu, at + S::kColO + (t & 1) * S::kV, 0);
      const uint32_t a = __shfl_sync(0xffffffffu, at + (t & 1) * kKeys, 0);
      const uint64_t lo = S::kDescV | (stage0 + __shfl_sync(0xffffffffu, ld % kStages * (S::kStage / 16), 0));
      const uint64_t hi = S::kDescV | (stage0 + __shfl_sync(0xffffffffu, (ld + 1) % kStages * (S::kStage / 16), 0));
      if (lead) {
        // weights of 32 keys: 16 columns of hi, 16 of lo
        auto pv = [&](int p, uint64_t vd, bool first) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            ptx::mma_f16_ts(d, a + k / 2 * 32 + p * 16 + k % 2 * 8, vd + k * (2 * 8 * S::kLine / 16), idO, !first || k > 0);
        };
        pv(0, lo, true);
        ptx::tc_commit(bar(kQbFree + ld % kStages));
        pv(1, hi, false);
        pv(0, hi, false);
        ptx::tc_commit(bar(kQbFree + (ld + 1) % kStages));
        ptx::tc_commit(bar(kQbO + (t & 1)));
      }
      __syncwarp();
    };
    for (; ok && take(it);) {
      ok = wait(kQbQ, items, 6);
      leave();
      const int tiles = it.end[0] - it.begin[0];
      if (S::kAhead && ok) scores(n, tiles == 1);
      for (int i = 0; i < tiles && ok; ++i, ++n) {
        if (!S::kAhead) scores(n, i + 1 == tiles);
        if (S::kAhead && i + 1 < tiles) scores(n + 1, i + 2 == tiles);
        if (ok) outputs(n);
      }
    }
    if (lead) ptx::tc_commit(bar(kQbDrain));  // nothing is in flight when tensor memory is freed
    wait(kQbDrain, 0, 10);
  } else if (warp >= kAux) {
    // ------------------------------------------------ powers of two, and V's elements that are not finite
    const int at = (warp - kAux) * 32 + lane;
    for (; ok && take(it); leave()) {
      const int kv = it.head / group;
      for (int j = it.begin[0]; j < it.end[0]; ++j, ++n) {
        const unsigned b = n & 1;
        const int key = it.first + j * kKeys, slot = it.first / kKeys + it.sequence + j;
        const bool known = XQ_IN(slot, W.slots, kChkPromptSlot);
        float kp[kKeys / 64], vp[(S::kV + 63) / 64];
#pragma unroll
        for (int x = 0; x < kKeys / 64; ++x)
          kp[x] = key + x * 64 + at < A.tokens ? W.k_power[static_cast<size_t>(kv) * A.tokens + key + x * 64 + at] : 0.0f;
#pragma unroll
        for (int x = 0; x < (S::kV + 63) / 64; ++x)
          vp[x] = x * 64 + at < S::kV && known
                      ? W.v_power[(static_cast<size_t>(slot) * A.kv_heads + kv) * D + it.half * S::kV + x * 64 + at]
                      : 0.0f;
        const int owner = known ? W.owner[(static_cast<size_t>(slot) * A.kv_heads + kv) * S::kHalves + it.half] : -1;
        ok = n < 2 || wait(kQbPowerFree + b, (n >> 1) - 1, 17);
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < kKeys / 64; ++x) sh_k[b][x * 64 + at] = kp[x];
#pragma unroll
        for (int x = 0; x < (S::kV + 63) / 64; ++x)
          if (x * 64 + at < S::kV) sh_v[b][x * 64 + at] = vp[x];
        if (owner != it.sequence && at == 0) atomicOr(&sh_odd[items & 1], 2u);
        arrive(kQbPower + b);
        const unsigned ld = n * S::kLoads + 2 * S::kHalves;  // V lo's, hi's is the next
        ok = wait(kQbFull + ld % kStages, ld / kStages, 15) && wait(kQbFull + (ld + 1) % kStages, (ld + 1) / kStages, 15);
        if (!ok) break;
        if (masked<kKeys>(P, it.place, j * kKeys)) {
          constexpr int kBlock = kKeys * S::kLine;  // bytes of a column block
          const int end = min(it.n - j * kKeys, kKeys) * S::kLine;  // of the sequence's rows in each; the pieces behind are anyone's
          const uint32_t from = stages + (ld + 1) % kStages * S::kStage + at * 16;
          bool found = false;
          for (int x = end + at * 16; x < kBlock; x += 64 * 16) {
#pragma unroll
            for (int i = 0; i < 2 * S::kBoxes; ++i)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(stages + (ld + i % 2) % kStages * S::kStage + i / 2 * kBlock + x),
                           "r"(0u) : "memory");
          }
#pragma unroll 8
          for (int x = 0; x < S::kStage; x += 64 * 16) {
            if ((x + at * 16) % kBlock >= end) continue;
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
    if (warp < 4) {
      // ---------------------------------------------- softmax: a thread is a row
      constexpr float kTop = 15.0f, kStart = 11.0f;  // log2 of weights: the largest, and where the reference starts anew
      const bool turned = !(A.scale > 0.0f);  // as in prompt_tile.cuh
      const float sign = A.scale < 0.0f ? -1.0f : 0.0f, cs = A.scale == 0.0f ? 1.0f : fabsf(A.scale) * 1.4426950408889634f;
      for (; ok && take(it); leave()) {
        const int place = it.place + token;
        const bool live = token < P.tokens_tile && place < it.n;
        const int lim1 = place + 1, lim0 = A.window ? max(0, lim1 - A.window) : 0;
        const float cq = live ? cs * W.q_power[(static_cast<size_t>(it.first) + place) * A.heads + it.head + part] : 0.0f;
        float e = -3.402823466e38f, l = 0.0f;
        for (int j = it.begin[0]; j < it.end[0]; ++j, ++n) {
          const unsigned b = n & 1;
          const int key = j * kKeys;
          ok = wait(kQbPower + b, n >> 1, 18) && wait(kQbS + b, n >> 1, 11);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t ts = tl + b * kKeys;
          const bool edge = masked<kKeys>(P, it.place, key);
          // 32 scores from column c on, those that the row does not see as -infinity
          ptx::f2 s[16];
          auto load = [&](int c) {
            uint32_t v[32];
            __syncwarp();
            tmem_ld32(ts + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; x += 4) {
              const float4 k = *reinterpret_cast<const float4*>(&sh_k[b][c + x]);
              s[x / 2] = ptx::mul2(ptx::pk(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), ptx::pk(k.x, k.y));
              s[x / 2 + 1] = ptx::mul2(ptx::pk(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), ptx::pk(k.z, k.w));
            }
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
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            load(c);
#pragma unroll
            for (int x = 0; x < 16; ++x) tops[x & 3] = max3(tops[x & 3], ptx::lo32(s[x]), ptx::hi32(s[x]));
          }
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * cq;
          float f = 1.0f;
          if (top - e > kTop) {  // the row's reference moves
            const float next = top - kStart;
            f = ex2(e - next);
            e = next;
            l *= f;
          }
          ok = n < 2 || wait(kQbOFree + b, (n >> 1) - 1, 19);
          if (!ok) break;
          sh_move[b][row] = f;
          const ptx::f2 c2 = ptx::pk(cq, cq), e2 = ptx::pk(-e, -e);
          ptx::f2 sum = ptx::pk(0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < kKeys; c += 32) {
            load(c);
            uint32_t hi[16], lo[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const ptx::f2 z = ptx::fma2(s[x], c2, e2);
              const float u = ex2(ptx::lo32(z)), v = ex2(ptx::hi32(z));
              sum = ptx::add2(sum, ptx::pk(u, v));
              halves_of(u, v, &hi[x], &lo[x]);
            }
            __syncwarp();
            ptx::tmem_st16(ts + c, hi);  // into columns already read
            ptx::tmem_st16(ts + c + 16, lo);
          }
          l += ptx::lo32(sum) + ptx::hi32(sum);
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          arrive(kQbP + b);
          if (lane == 0) ptx::mbar_arrive(bar(kQbPowerFree + b));
        }
        if (!ok) break;
        sh_sum[items & 1][row] = l;
        arrive(kQbSum + (items & 1));
      }
    } else {
      // ---------------------------------------------- outputs: a thread is a row
      for (; ok && take(it); leave()) {
        const int place = it.place + token, kv = it.head / group;
        const bool live = token < P.tokens_tile && place < it.n;
        ptx::f2 o[S::kV / 2];
#pragma unroll
        for (int x = 0; x < S::kV / 2; ++x) o[x] = ptx::pk(0.0f, 0.0f);
        for (int j = it.begin[0]; j < it.end[0]; ++j, ++n) {
          const unsigned b = n & 1;
          ok = wait(kQbP + b, n >> 1, 20) && wait(kQbO + b, n >> 1, 12) && wait(kQbPower + b, n >> 1, 21);
          if (!ok) break;
          ptx::tc_fence_after();
          const float f = sh_move[b][row];
          if (__any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll
            for (int x = 0; x < S::kV / 2; ++x) o[x] = ptx::mul2(o[x], ptx::pk(f, f));
          }
          const uint32_t from = tl + S::kColO + b * S::kV;
#pragma unroll
          for (int c = 0; c < S::kV; c += 16) {
            uint32_t v[16];
            ptx::tmem_ld16(from + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; x += 4) {
              const float4 p = *reinterpret_cast<const float4*>(&sh_v[b][c + x]);
              o[(c + x) / 2] = ptx::fma2(ptx::pk(__uint_as_float(v[x]), __uint_as_float(v[x + 1])), ptx::pk(p.x, p.y), o[(c + x) / 2]);
              o[(c + x) / 2 + 1] =
                  ptx::fma2(ptx::pk(__uint_as_float(v[x + 2]), __uint_as_float(v[x + 3])), ptx::pk(p.z, p.w), o[(c + x) / 2 + 1]);
            }
          }
          ptx::tc_fence_before();
          arrive(kQbOFree + b);
          if (lane == 0) ptx::mbar_arrive(bar(kQbPowerFree + b));
        }
        if (!ok) break;
        // ---- the rows' results
        ok = wait(kQbSum + (items & 1), items >> 1, 13);
        if (!ok) break;
        const float sum = sh_sum[items & 1][row], inv = 1.0f / sum;
        const size_t at = (static_cast<size_t>(it.first) + place) * A.heads + it.head + part;
        const bool store = live && XQ_IN(at, static_cast<size_t>(A.tokens) * A.heads, kChkPromptRow);
        float4* const out = reinterpret_cast<float4*>(static_cast<float*>(A.out) + at * D + it.half * S::kV);
        ptx::f2 odd = ptx::pk(sum * 0.0f, 0.0f);  // NaN if anything is not finite
#pragma unroll
        for (int x = 0; x < S::kV / 2; x += 2) {
          odd = ptx::fma2(o[x], ptx::pk(0.0f, 0.0f), odd);
          odd = ptx::fma2(o[x + 1], ptx::pk(0.0f, 0.0f), odd);
          if (store)
            out[x / 2] = make_float4(ptx::lo32(o[x]) * inv, ptx::hi32(o[x]) * inv, ptx::lo32(o[x + 1]) * inv, ptx::hi32(o[x + 1]) * inv);
        }
        const unsigned look = sh_odd[items & 1];
        bool meets = (look & 2u) != 0;  // pieces that do not hold the values, or an element that was put to 0
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
          one_row<kF32, D>(A, it.first, __shfl_sync(0xffffffffu, place, src), it.head + __shfl_sync(0xffffffffu, part, src));
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMma) ptx::tmem_dealloc(tmem, S::kAlloc);
}

}  // namespace

template <int D>
cudaError_t PromptPiecesDim<D>::launch(PromptTileArgs& p, const PromptPieces& w, cudaStream_t s) {
  using S = PieceShape<D>;
  g_kv_launched.store(true, std::memory_order_relaxed);
  const PromptArgs& a = p.a;
  const long long qs = static_cast<long long>(a.heads) * D, ks = static_cast<long long>(a.kv_heads) * D;
  if (!encode_tma_heads(&p.q, false, w.q, D, a.heads, 2 * a.tokens, qs, S::kBox, p.pack, p.tokens_tile) ||
      !encode_tma_heads(&p.k, false, w.k, D, a.kv_heads, 2 * a.tokens, ks, S::kBox, 1, S::kKeys) ||
      !encode_tma_heads(&p.v, false, w.v, D, a.kv_heads, 2 * a.tokens, ks, S::kBox, 1, S::kKeys))
    return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_shared(prompt_pieces_kernel<D>, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
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
