// Prompt attention of 16-bit rows on the tcgen05 tensor cores.
//
// o_i = sum_j w_ij v_j / sum_j w_ij with w_ij = 2^(s_ij - e_i), s_ij = log2(e) scale q_i.k_j. The reference e_i of a row
// moves only when a weight would leave its range, so outputs are rescaled rarely.
//
// w enters the second product rounded to the call's type, and the divisor is the fp32 sum of the weights as rounded: what all of a
// row's weights lose alike cancels, so a row that one key takes, or values that are much alike, come back with the result's own
// rounding only. Else the roundings of the weights add 1.1e-3 (bf16) or 1.6e-4 (fp16) of a row's spread at random, beside the
// result's 1.6e-3 and 2.0e-4. Weights as two numbers of the type would add nothing; their products are half as many again, and
// measured 12287 bf16 tokens 1117 us for 825 and 16 sequences of 17 to 2048 297 for 219 (as low as with any order of waits and
// products that was tried), so they are left at one.
//
// A tile is 128 rows x 128 keys. Rows are the query heads of a KV head that lie side by side, times tokens: row r is token
// r / pack, head r % pack, so that K and V are read once for all of them. A CTA has two row tiles (one with head size 256,
// whose outputs fill tensor memory), so that one's softmax passes under the other's products. Q, K and V come by TMA with
// the swizzle that the products read; V is the K-outer operand as it lies in memory. Scores go to tensor memory, a softmax
// thread takes a row of them and leaves the weights in the same columns, the second product's A operand.
//
// Roles: warps 0-3 and 4-7 softmax and results of a row tile, then one that issues products, one that copies, two that
// look through V (below). CTAs are persistent and take items (row tiles of a sequence and heads) longest first, in rounds of
// alternating direction; the copying warp finds them from the sequences' bounds (see next_item) an item ahead, so Q, K and V
// of the next item are on their way, and its first scores are computed, while one ends.
//
// Sums: a tensor core's accumulator cuts off, towards 0, what an fp32 addition rounds, so an output that stayed there over a long
// sequence would be too small by 8e-9 a key (fp16, V of one sign, 131071 keys: 1e-3, two half steps of the result). So after
// kPromptRun key tiles the outputs are added to the row's sum in the workspace, in fp32, and the accumulator begins anew. The sum of
// weights goes tile by tile, with what each addition rounds off kept beside it (one after the other, equal weights of 524287 keys
// were all rounded the same way: 3e-3).
//
// What is not finite: scores of keys that a row does not see are replaced, but such a key's V would meet a weight of 0 in
// the product, where an infinity or NaN spoils the row. So two warps look through the V tiles of which some row does not see
// all keys, before the product, and put 0 in the place of such elements. Rows that do see one of them, and rows whose result
// or sum is not finite (a score, a V that all rows see), are computed again by themselves (one_row).
//
// What bounds it, at head size 128: the tensor cores have 2048 clocks of work for the two row tiles' 128 keys, which take
// some 3600: a tile's scores (107 clocks a product, with both operands in shared memory), softmax (1700), weights and outputs follow each
// other, and two of them do not fill the pipe. 12287 bf16 tokens of 32/8 heads 891 us, 1.39 PFLOP/s; 16 sequences of 17 to 2048
// 209 us (1.03; masked halves of tiles count as nothing), where an item of some 9 tiles ends and begins in about 8000 clocks.
// Tried and slower: 32 scores at a time in rolled loops (long 974 us for 935), products issued by two warps (one is then left
// to look through V: 241 us for 229, packed), masks as bits of a word (247 for 229), results stored from registers (258 for
// 235: a store of 32 rows takes 32 lines' turns), the scan of V unrolled eight times instead of twice (234 for 229).
#pragma once

#include "prompt_items.cuh"

namespace xq {

constexpr int prompt_row_tiles(int dim) { return dim == 256 ? 1 : 2; }  // of a CTA: head size 256's outputs fill tensor memory
constexpr int prompt_run_quads(int dim) { return kPromptRows * (dim + 1) / 4; }  // a row tile's sums and references, in 16 bytes

template <int D>
struct PromptTileDim {
  static cudaError_t launch(PromptTileArgs& a, cudaStream_t s);
  static cudaError_t take_error(unsigned int* index, unsigned int* wait);
  static cudaError_t take_check(unsigned int* code);
};

#ifdef XQ_PROMPT_TILE_IMPL

namespace {

constexpr int kKeys = kPromptTileKeys;

template <int D>
struct PromptShape {
  static constexpr int kTiles = prompt_row_tiles(D);            // row tiles
  static constexpr int kBox = D % 64 == 0 ? 64 : 32;            // elements of a swizzled row
  static constexpr int kLine = kBox * 2, kBoxes = D / kBox;
  static constexpr int kQ = kRows * D * 2, kStage = kKeys * D * 2;  // bytes: Q of a row tile; K or V of a tile
  static constexpr int kStages = D == 256 ? 2 : D == 128 ? 4 : D == 96 ? 6 : 9;
  static constexpr int kRowsOut = 4 * kTiles * 2048;  // results on their way out: 32 rows x 64 bytes of each softmax warp
  static constexpr int kSmem = kTiles * kQ + kStages * kStage + kRowsOut + 1024;
  static constexpr int kColS = 0, kColO = 2 * kKeys, kAlloc = 512;
  static constexpr int kWarps = 4 * kTiles + 4;
  static_assert(kColO + kTiles * D <= kAlloc && kSmem <= 227 * 1024 - 1024, "one CTA fits the SM");
  // Operand descriptors. Q and K: rows of kLine bytes are the K extent, 8 of them 8 * kLine apart. V: rows are keys, the
  // N extent runs along them, blocks of kBox elements kKeys * kLine apart.
  static constexpr uint64_t kSwizzle = kLine == 128 ? 2ull : 4ull;
  static constexpr uint64_t kCommon = (1ull << 46) | (kSwizzle << 61) | (static_cast<uint64_t>(8 * kLine / 16) << 32);
  static constexpr uint64_t kDescK = kCommon | (1ull << 16);
  static constexpr uint64_t kDescV = kCommon | (static_cast<uint64_t>(kKeys * kLine / 16) << 16);
};
enum PromptBar { kPbDrain, kPbItem, kPbItemFree = kPbItem + 2, kPbQ = kPbItemFree + 2, kPbQFree = kPbQ + 2, kPbS = kPbQFree + 2,
                 kPbP = kPbS + 2, kPbO = kPbP + 2, kPbFull = kPbO + 2 };



// A row's sum over runs of tiles and the reference that it goes by (a row's 4 columns lie beside the other rows', the references
// behind all columns). Functions of their own, that find these again each time, so that the softmax loop keeps its registers: written
// into it they cost 16 sequences of 17 to 2048, which have no use for them, 208 -> 243 us.
template <int D>
__device__ __forceinline__ float4* run_sum(float4* sums, float** reference) {
  const int r = threadIdx.x >> 7, row = threadIdx.x & 127;
  float4* const sum = sums + (static_cast<size_t>(blockIdx.x) * prompt_row_tiles(D) + r) * prompt_run_quads(D);
  *reference = reinterpret_cast<float*>(sum + D / 4 * kRows) + row;
  return sum + row;
}
// JOIN: outputs += sum 2^(reference - e), else sum = sum 2^(reference - e) + outputs; `there`: there is a sum.
template <int D, bool JOIN>
__device__ __noinline__ void run_add(float4* sums, uint32_t outputs, float e, bool there) {
  float* reference;
  float4* const sum = run_sum<D>(sums, &reference);
  const float f = there ? ex2(*reference - e) : 0.0f;
  if (!JOIN) *reference = e;
  float4 o[8], next[8];
  auto load = [&](int c) {
#pragma unroll
    for (int x = 0; x < 8; ++x) next[x] = there ? sum[(c / 4 + x) * kRows] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  load(0);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
#pragma unroll
    for (int x = 0; x < 8; ++x) o[x] = next[x];
    if (c + 32 < D) load(c + 32);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[16];
      __syncwarp();
      ptx::tmem_ld16(outputs + c + 16 * h, w);
      ptx::tmem_wait_ld();
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float4 s = o[4 * h + x];
        const float4 y = make_float4(fmaf(s.x, f, __uint_as_float(w[4 * x])), fmaf(s.y, f, __uint_as_float(w[4 * x + 1])),
                                     fmaf(s.z, f, __uint_as_float(w[4 * x + 2])), fmaf(s.w, f, __uint_as_float(w[4 * x + 3])));
        if (!JOIN) sum[(c / 4 + 4 * h + x) * kRows] = y;
        w[4 * x] = __float_as_uint(y.x), w[4 * x + 1] = __float_as_uint(y.y), w[4 * x + 2] = __float_as_uint(y.z), w[4 * x + 3] = __float_as_uint(y.w);
      }
      if (JOIN) ptx::tmem_st16(outputs + c + 16 * h, w);
    }
  }
  if (JOIN) ptx::tmem_wait_st();
}

template <int TYPE, int D>
__global__ void __launch_bounds__(32 * PromptShape<D>::kWarps, 1) prompt_tile_kernel(const __grid_constant__ PromptTileArgs P) {
  using S = PromptShape<D>;
  constexpr int kTiles = S::kTiles, kStages = S::kStages, kPbFree = kPbFull + kStages, kPbChecked = kPbFree + kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kPbFull + 3 * kStages];
  __shared__ uint32_t sh_tmem;
  __shared__ Item sh_item[2];
  __shared__ unsigned sh_odd[2];  // elements of V that are not finite were put to 0, by item & 1
  const PromptArgs& A = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kMma = 4 * kTiles, kLoad = kMma + 1, kCheck = kMma + 2;
  auto bar = [&](int i) { return ptx::smem_addr(&bars[i]); };
  const uint32_t base = (ptx::smem_addr(smem_raw) + 1023u) & ~1023u;
  if (tid == 0) {
    ptx::mbar_init(bar(kPbDrain), 1);
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar(kPbItem + b), 1);
      ptx::mbar_init(bar(kPbItemFree + b), 4 * kTiles + 3);
      ptx::mbar_init(bar(kPbQ + b), 1);
      ptx::mbar_init(bar(kPbQFree + b), 1);
      ptx::mbar_init(bar(kPbS + b), 1);
      ptx::mbar_init(bar(kPbP + b), 4);
      ptx::mbar_init(bar(kPbO + b), 1);
    }
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(bar(kPbFull + i), 1);
      ptx::mbar_init(bar(kPbFree + i), 1);
      ptx::mbar_init(bar(kPbChecked + i), 2);
    }
    ptx::mbar_init_fence();
  }
  if (warp == kMma) ptx::tmem_alloc(ptx::smem_addr(&sh_tmem), S::kAlloc);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = sh_tmem;
  auto wait = [&](int i, unsigned parity, unsigned code) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar(i), parity & 1, &g_prompt_wait, code, P.wait)) != 0;
  };
  // buffer of scores of row tile r's n-th tile, and how often it was used before
  auto buffer = [](int r, unsigned n) { return kTiles == 2 ? r : static_cast<int>(n & 1); };
  auto turn = [](unsigned n) { return kTiles == 2 ? n : n >> 1; };
  unsigned items = 0;  // taken so far
  auto take = [&](Item& it) {  // false: the last one is done (or a wait ran out)
    if (!wait(kPbItem + (items & 1), items >> 1, 1)) return false;
    it = sh_item[items & 1];
    return it.n >= 0;
  };
  auto leave = [&] {  // its last use of the item's place
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar(kPbItemFree + (items & 1)));
    ++items;
  };

  if (warp == kLoad) {
    // ------------------------------------------------ copies
    Walk w;
    walk_begin(A, kTiles * P.tokens_tile, w);
    const bool lead = ptx::elect_one();
    unsigned loaded = 0, q_done[2] = {0u, 0u};
    bool ok = true;
    Item next;
    auto find = [&](unsigned round) {
      const long long rank = static_cast<long long>(round) * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      if (!next_item<kKeys, 1>(P, kTiles, rank, w, next)) next.n = -1;
    };
    find(0);
    for (unsigned round = 0; ok; ++round) {
      const Item it = next;
      const bool there = it.n >= 0;
      if (round >= 2 && !wait(kPbItemFree + (round & 1), (round >> 1) + 1, 2)) break;
      if (lead) {
        sh_item[round & 1] = it;
        sh_odd[round & 1] = 0u;
        ptx::mbar_arrive(bar(kPbItem + (round & 1)));
      }
      __syncwarp();
      if (!there || P.withhold) break;
      const int kv = it.head / (A.heads / A.kv_heads);
      const bool second = kTiles == 2 && it.end[1] > 0;
      // the first K before the queries, whose place is free later
      auto queries = [&] {
        for (int r = 0; r < (second ? 2 : 1) && ok; ++r) {
          if (q_done[r] > 0) ok = wait(kPbQFree + r, q_done[r] - 1, 3);
          ++q_done[r];
          if (ok && lead) {
            ptx::mbar_expect_tx(bar(kPbQ + r), P.pack * P.tokens_tile * D * 2);
#pragma unroll
            for (int x = 0; x < S::kBoxes; ++x)
              tma_load_3d(base + r * S::kQ + x * (kRows * S::kLine), &P.q, x * S::kBox, it.head, it.first + it.place + r * P.tokens_tile,
                          bar(kPbQ + r));
          }
        }
      };
      const int last = second ? it.end[1] : it.end[0];
      for (int j = it.begin[0]; j < last && ok; ++j) {
#pragma unroll 1
        for (int v = 0; v < 2 && ok; ++v) {
          const unsigned st = loaded % kStages;
          if (loaded >= kStages) ok = wait(kPbFree + st, loaded / kStages - 1, 4);
          if (!ok) break;
          ++loaded;
          if (lead) {
            ptx::mbar_expect_tx(bar(kPbFull + st), S::kStage);
#pragma unroll
            for (int x = 0; x < S::kBoxes; ++x)
              tma_load_3d(base + kTiles * S::kQ + st * S::kStage + x * (kKeys * S::kLine), v ? &P.v : &P.k, x * S::kBox, kv,
                          it.first + j * kKeys, bar(kPbFull + st));
          }
          if (v == 0 && j == it.begin[0]) queries();
        }
        if (j == it.begin[0]) find(round + 1);  // while the first copies are on their way
      }
      __syncwarp();
    }
    // copies in flight land before the CTA ends
    for (unsigned i = loaded > kStages ? loaded - kStages : 0; i < loaded; ++i)
      if (!wait(kPbFull + i % kStages, i / kStages, 5)) break;
  } else if (warp == kMma) {
    // ------------------------------------------------ products, issued by one thread
    constexpr uint32_t idS = ptx::idesc_f16(kRows, kKeys, TYPE == kBF16), idO = ptx::idesc_f16(kRows, D, TYPE == kBF16) | (1u << 16);
    const bool lead = ptx::elect_one();
    const uint32_t at = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t stage0 = static_cast<uint64_t>((base + kTiles * S::kQ) >> 4), q0 = static_cast<uint64_t>(base >> 4);
    unsigned used = 0;  // loads of the items before
    unsigned scored[2] = {0u, 0u}, done[2] = {0u, 0u}, parts[2] = {0u, 0u};
    bool ok = true;
    Item it, next;
    bool more = take(it), begun = false;  // begun: the item's first scores of row tile 0 were issued before the last outputs of the one before
    if (more) leave();
    while (ok && more) {
      const bool second = kTiles == 2 && it.end[1] > 0;
      const int first = it.begin[0], last = second ? it.end[1] : it.end[0];
      auto k_load = [&](int j) { return used + 2 * (j - first); };  // V's is the next
      auto scores_of = [&](const Item& it, int r, int j, unsigned ld) {
        if (j == it.begin[r]) {
          ok = wait(kPbQ + r, parts[r]++, 6);
          if (!ok) return;
        }
        const unsigned st = ld % kStages;
        ok = wait(kPbFull + st, ld / kStages, 7);
        if (!ok) return;
        ptx::tc_fence_after();
        const int to = buffer(r, scored[r]++);
        const uint32_t d = __shfl_sync(0xffffffffu, at + S::kColS + to * kKeys, 0);
        const uint64_t kd = S::kDescK | (stage0 + __shfl_sync(0xffffffffu, st * (S::kStage / 16), 0));
        const uint64_t qd = S::kDescK | (q0 + r * (S::kQ / 16));
        if (lead) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            constexpr int kSteps = S::kBox / 16;
            const int off = (k / kSteps) * (kRows * S::kLine / 16) + (k % kSteps) * 2;
            ptx::mma_f16_ss(d, qd + off, kd + off, idS, k > 0);
          }
          ptx::tc_commit(bar(kPbS + to));
          if (j + 1 == it.end[r]) ptx::tc_commit(bar(kPbQFree + r));
        }
        __syncwarp();
      };
      auto scores = [&](int r, int j) { scores_of(it, r, j, k_load(j)); };
      auto outputs = [&](int r, int j) {
        const int from = buffer(r, done[r]);
        ok = wait(kPbP + from, turn(done[r]), 8);
        ++done[r];
        if (!ok) return;
        const unsigned ld = k_load(j) + 1, st = ld % kStages;
        ok = wait(kPbFull + st, ld / kStages, 9) && wait(kPbChecked + ld / 2 % kStages, ld / 2 / kStages, 14);
        if (!ok) return;
        ptx::tc_fence_after();
        const uint32_t d = __shfl_sync(0xffffffffu, at + S::kColO + r * D, 0);
        const uint32_t a = __shfl_sync(0xffffffffu, at + S::kColS + from * kKeys, 0);
        const uint64_t vd = S::kDescV | (stage0 + __shfl_sync(0xffffffffu, st * (S::kStage / 16), 0));
        if (lead) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            ptx::mma_f16_ts(d, a + 8 * k, vd + k * (2 * 8 * S::kLine / 16), idO, (j - it.begin[r]) % kPromptRun > 0 || k > 0);
          ptx::tc_commit(bar(kPbO + from));
        }
        __syncwarp();
      };
      auto release = [&](unsigned ld) {
        if (lead) ptx::tc_commit(bar(kPbFree + ld % kStages));
        __syncwarp();
      };
      for (int j = first - 1; j < last && ok; ++j) {
        // behind the last scores of row tile 0 come the next item's first
        auto begin_next = [&] {
          more = take(next);
          if (!more) return;
          leave();
          scores_of(next, 0, next.begin[0], used + 2 * (last - first));
        };
        if (kTiles == 2) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            if (r == 1 && ok && j + 1 == last) begin_next();
            if (ok && j >= it.begin[r] && j < it.end[r]) outputs(r, j);
            if (ok && j + 1 >= it.begin[r] && j + 1 < it.end[r] && !(r == 0 && begun && j + 1 == first)) scores(r, j + 1);
          }
        } else {
          if (j + 1 == last)
            begin_next();
          else if (!(begun && j + 1 == first))
            scores(0, j + 1);
          if (ok && j >= first) outputs(0, j);
        }
        if (!ok) break;
        if (j + 1 < last) release(k_load(j + 1));
        if (j >= first) release(k_load(j) + 1);
      }
      used += 2 * (last - first);
      it = next;
      begun = true;
    }
    if (lead) ptx::tc_commit(bar(kPbDrain));  // nothing is in flight when tensor memory is freed
    wait(kPbDrain, 0, 10);
  } else if (warp >= kCheck) {
    // ------------------------------------------------ V's elements that are not finite
    unsigned tiles = 0;  // V tiles so far
    bool ok = true;
    Item it;
    while (ok && take(it)) {
      const bool second = kTiles == 2 && it.end[1] > 0;
      const int last = second ? it.end[1] : it.end[0];
      for (int j = it.begin[0]; j < last; ++j, ++tiles) {
        const unsigned ld = 2 * tiles + 1, st = ld % kStages;
        ok = wait(kPbFull + st, ld / kStages, 15);
        if (!ok) break;
        if (masked<kKeys>(P, it.place, j * kKeys) || (second && masked<kKeys>(P, it.place + P.tokens_tile, j * kKeys))) {
          const uint32_t from = base + kTiles * S::kQ + st * S::kStage + ((warp - kCheck) * 32 + lane) * 16;
          bool found = false;
#pragma unroll 2
          for (int x = 0; x < S::kStage; x += 64 * 16) {
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from + x));
            if (odd_halves<TYPE>(w[0]) | odd_halves<TYPE>(w[1]) | odd_halves<TYPE>(w[2]) | odd_halves<TYPE>(w[3])) {
              found = true;
#pragma unroll
              for (int i = 0; i < 4; ++i) w[i] &= ~((odd_halves<TYPE>(w[i]) >> 15) * 0xFFFFu);
              asm volatile("st.shared.v4.b32 [%4], {%0, %1, %2, %3};" ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(from + x) : "memory");
            }
          }
          if (found) {
            sh_odd[items & 1] = 1u;
            ptx::fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kPbChecked + tiles % kStages));
      }
      leave();
    }
  } else {
    // ------------------------------------------------ softmax and results: a thread is a row
    // log2 of weights: the largest, and where the reference starts anew. fp16 keeps 2^-24 at least, so its weights begin above 1.
    constexpr float kTop = TYPE == kF16 ? 15.0f : 20.0f, kStart = TYPE == kF16 ? 8.0f : 0.0f;
    constexpr float kLowest = -3.402823466e38f;
    const int r = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16), to = tl + S::kColO + r * D;
    // a scale that is not positive goes to the scores first, so that cs > 0 and what is masked stays -infinity
    const bool turned = !(A.scale > 0.0f);
    const float sign = A.scale < 0.0f ? -1.0f : 0.0f, cs = A.scale == 0.0f ? 1.0f : fabsf(A.scale) * 1.4426950408889634f;
    const int token = row / P.pack, part = row - token * P.pack;
    unsigned done = 0;
    bool ok = true;
    Item it;
    while (ok && take(it)) {
      const int tiles = it.end[r] - it.begin[r];
      if (tiles <= 0) {
        leave();
        continue;
      }
      const int place = it.place + r * P.tokens_tile + token;
      const bool live = token < P.tokens_tile && place < it.n;
      const int lim1 = place + 1, lim0 = A.window ? max(0, lim1 - A.window) : 0;
      const int p0 = it.place + r * P.tokens_tile;
      float e = kLowest;
      float l = 0.0f, l_rest = 0.0f;  // the sum of weights, and what its additions rounded off
      for (int i = 0; i < tiles; ++i, ++done) {
        const int key = (it.begin[r] + i) * kKeys;
        const bool anew = i > 0 && i % kPromptRun == 0;
        if (anew) {
          ok = wait(kPbO + buffer(r, done - 1), turn(done - 1), 12);
          if (!ok) break;
          ptx::tc_fence_after();
          run_add<D, false>(P.sums, to, e, i > kPromptRun);
        }
        ok = wait(kPbS + buffer(r, done), turn(done), 11);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t ts = tl + S::kColS + buffer(r, done) * kKeys;
        uint32_t sv[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) tmem_ld32(ts + c, sv + c);
        ptx::tmem_wait_ld();
        if (turned) {
#pragma unroll
          for (int x = 0; x < kKeys; ++x) sv[x] = __float_as_uint(__uint_as_float(sv[x]) * sign);
        }
        if (masked<kKeys>(P, p0, key)) {
#pragma unroll
          for (int x = 0; x < kKeys; ++x)
            if (key + x < lim0 || key + x >= lim1) sv[x] = 0xFF800000u;
        }
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < kKeys; x += 8)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            tops[y] = max3(tops[y], __uint_as_float(sv[x + 2 * y]), __uint_as_float(sv[x + 2 * y + 1]));
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * cs;
        if (__any_sync(0xffffffffu, top - e > kTop)) {  // the reference of some rows moves
          const float next = top - e > kTop ? top - kStart : e;
          const float f = ex2(e - next);
          e = next;
          l *= f, l_rest *= f;
          if (i > 0 && !anew) {
            ok = wait(kPbO + buffer(r, done - 1), turn(done - 1), 12);
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
        const ptx::f2 c2 = ptx::pk(cs, cs), e2 = ptx::pk(-e, -e);
        ptx::f2 tile_sum = ptx::pk(0.0f, 0.0f);
#pragma unroll
        for (int c = 0; c < kKeys; c += 32) {
          uint32_t w[16];
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            const ptx::f2 z = ptx::fma2(ptx::pk(__uint_as_float(sv[c + x]), __uint_as_float(sv[c + x + 1])), c2, e2);
            const float a = ex2(ptx::lo32(z)), b = ex2(ptx::hi32(z));
            w[x / 2] = pack2<TYPE>(a, b);
            if constexpr (TYPE == kF16) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[x / 2]));  // the weights as rounded
              tile_sum = ptx::add2(tile_sum, ptx::pk(f.x, f.y));
            } else {
              tile_sum = ptx::add2(tile_sum, ptx::pk(__uint_as_float(w[x / 2] << 16), __uint_as_float(w[x / 2] & 0xFFFF0000u)));
            }
          }
          ptx::tmem_st16(ts + c / 2, w);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(kPbP + buffer(r, done)));
        const float add = ptx::lo32(tile_sum) + ptx::hi32(tile_sum), next_l = l + add, kept = next_l - l;
        l_rest += (l - (next_l - kept)) + (add - kept);
        l = next_l;
      }
      if (!ok) break;
      // ---- the rows' results
      ok = wait(kPbO + buffer(r, done - 1), turn(done - 1), 13);
      if (!ok) break;
      ptx::tc_fence_after();
      if (tiles > kPromptRun) run_add<D, true>(P.sums, to, e, true);
      const float sum = l + l_rest, inv = 1.0f / sum;
      const size_t at = (static_cast<size_t>(it.first) + place) * A.heads + it.head + part;
      const bool store = live && XQ_IN(at, static_cast<size_t>(A.tokens) * A.heads, kChkPromptRow);
      const int to_row = store ? static_cast<int>(at) : -1;
      const uint32_t rows_out = base + kTiles * S::kQ + kStages * S::kStage, mine = rows_out + warp * 2048 + lane * 64;
      float odd[4] = {sum * 0.0f, 0.0f, 0.0f, 0.0f};  // NaN if anything is not finite
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t w[32];
        __syncwarp();
        tmem_ld32(to + c, w);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 32; ++x) odd[x & 3] = fmaf(__uint_as_float(w[x]), 0.0f, odd[x & 3]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = pack2<TYPE>(__uint_as_float(w[8 * x + 2 * i]) * inv, __uint_as_float(w[8 * x + 2 * i + 1]) * inv);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ((x ^ (lane >> 1 & 3)) << 4)), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]) : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r8 = 8 * i + (lane >> 2), row_to = __shfl_sync(0xffffffffu, to_row, r8);
          uint4 y;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                       : "r"(rows_out + warp * 2048 + r8 * 64 + (((lane & 3) ^ (r8 >> 1 & 3)) << 4))
                       : "memory");
          if (row_to >= 0) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.out) + static_cast<size_t>(row_to) * D + c + (lane & 3) * 8) = y;
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      bool meets = false;  // an element that was put to 0
      if (sh_odd[items & 1]) {
        const int kv = it.head / (A.heads / A.kv_heads);
#pragma unroll 1
        for (int j = it.begin[r]; j < it.end[r]; ++j)
          if (masked<kKeys>(P, it.place, j * kKeys) || (it.end[1] > 0 && masked<kKeys>(P, it.place + P.tokens_tile, j * kKeys)))
#pragma unroll 1
            for (int key = j * kKeys; key < min((j + 1) * kKeys, it.n); ++key) {
              bool odd_v = false;
              for (int x = lane; x < D; x += 32)
                odd_v |= !isfinite(load_elt<TYPE>(A.v, (static_cast<size_t>(it.first) + key) * A.v_stride + static_cast<size_t>(kv) * D + x));
              if (__any_sync(0xffffffffu, odd_v)) meets |= key >= lim0 && key < lim1;
            }
      }
      unsigned again = __ballot_sync(0xffffffffu, live && (meets || !(odd[0] + odd[1] + odd[2] + odd[3] == 0.0f && sum > 0.0f)));
      while (again) {
        const int src = __ffs(again) - 1;
        again &= again - 1;
        one_row<TYPE, D>(A, it.first, __shfl_sync(0xffffffffu, place, src), it.head + __shfl_sync(0xffffffffu, part, src), 0, D);
      }
      leave();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kMma) ptx::tmem_dealloc(tmem, S::kAlloc);
}

template <int TYPE, int D>
cudaError_t launch_tile(const PromptTileArgs& p, cudaStream_t s) {
  using S = PromptShape<D>;
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_shared(prompt_tile_kernel<TYPE, D>, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  prompt_tile_kernel<TYPE, D><<<prompt_tile_grid(p, S::kTiles), 32 * S::kWarps, S::kSmem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

template <int D>
cudaError_t PromptTileDim<D>::launch(PromptTileArgs& p, cudaStream_t s) {
  using S = PromptShape<D>;
  g_kv_launched.store(true, std::memory_order_relaxed);
  const PromptArgs& a = p.a;
  const bool bf16 = a.type == kBF16;
  const bool one = a.tokens == 1;
  if (!encode_tma_heads(&p.q, bf16, a.q, D, a.heads, a.tokens, one ? static_cast<long long>(a.heads) * D : a.q_stride, S::kBox, p.pack,
                        p.tokens_tile) ||
      !encode_tma_heads(&p.k, bf16, a.k, D, a.kv_heads, a.tokens, one ? static_cast<long long>(a.kv_heads) * D : a.k_stride, S::kBox, 1,
                        kKeys) ||
      !encode_tma_heads(&p.v, bf16, a.v, D, a.kv_heads, a.tokens, one ? static_cast<long long>(a.kv_heads) * D : a.v_stride, S::kBox, 1,
                        kKeys))
    return cudaErrorInvalidValue;
  return bf16 ? launch_tile<kBF16, D>(p, s) : launch_tile<kF16, D>(p, s);
}

template <int D>
cudaError_t PromptTileDim<D>::take_error(unsigned int* index, unsigned int* wait) {
  const cudaError_t e = take_record(g_prompt_error, index);
  return e != cudaSuccess ? e : take_record(g_prompt_wait, wait);
}
template <int D>
cudaError_t PromptTileDim<D>::take_check(unsigned int* code) {
  return take_check_word(code);
}

#endif  // XQ_PROMPT_TILE_IMPL

}  // namespace xq
