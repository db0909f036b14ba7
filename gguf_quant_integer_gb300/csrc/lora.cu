// Low-rank adapters of many requests beside shared projections.
//
// y[m] += scale[i] (x[m] A[i]^T) B[i]^T with the row's adapter i. A job is up to T rows of one adapter and projection, one
// cluster of 8 or 16 CTAs: each CTA multiplies its part of K (x against A, shared out among its warps), the CTAs add up their
// parts of t = x A^T [T][rank] through distributed shared memory in a fixed order, and each then adds t B^T to its part of y's
// columns. So one launch does both products, and t never leaves the SMs. Of large ranks a warp has 16 (or 32) and all of the
// CTA's K, before K is shared out too: rank 128 is one pass over x with no sums among the warps, where passes of 16 ranks, one
// behind the other, had 3500 clocks of latency each (4 rows, 4096 -> 2 x 14336: 33 us, now 23).
//
// Which rows make up a job is found in the kernel (count rows by adapter, number the jobs, collect the rows), as only the
// device knows the ids; all CTAs of a cluster find the same.
//
// Precision: both products run on the warp-level tensor cores in tf32, x and t as two numbers each (11 + 11 bits; hi is cut
// off, so that nothing overflows) and fp32 adapters too (without lo x lo); 16-bit adapters are exact. A tensor core's
// accumulator cuts off, towards 0, what an fp32 addition rounds, and all these errors have one sign: so sums leave it every 16
// elements of K and every 16 ranks (kept in it for K / 16, 4096 elements had 1.3e-6 of error; all of 256 ranks, with fp32
// adapters, 2.2e-6, now 0.4e-6 at any rank; every 8 would be 0.37e-6). y is added to in L2, in fp32, by one reduction a value.
//
// Infinities: one number of two is 0 where the other holds the value exactly, and 0 x infinity is NaN where the sum of products is an
// infinity. So what comes out of the tensor cores not finite is computed again in fp32, term by term (the test for it costs 1 row
// 0.15 us, 64 rows at q, k and v 0.25, 4099 rows nothing).
//
// T is 16 rows up to 2432 rows times projections, else 64 (32 beyond rank 128: shared memory): A and B are read once a job,
// so more rows save L2 traffic, and fewer start more clusters (352 rows of rank 128 to 2 x 14336: 55 us, 137 with 64 rows a
// job; 2854 rows of 25 adapters, 8960 -> 1536, rank 24: 72 us, above 110 with 16). Few jobs have clusters of 16, and as many
// clusters for a job's columns as fill the device, which all work out x A^T (1 row to 2 x 14336, rank 16: 6.0 us, 9.8 with 8
// CTAs a job). What bounds it: with few rows, a chain of memory round trips and instructions seen for the first time (one row
// 4096 -> 4096, rank 16: 5.3 us, x A^T, the exchange and y in like parts; 64 rows of 16 adapters at q, k and v: 11.7 us); with
// many, the warp-level tensor cores, 8 clocks a product of 16 x 8 x 8 on one of an SM's four sub-cores (4099 rows, rank 64, two
// projections 4096 -> 14336: 400 us, 371 with sums left in the tensor cores; 19.2 million products are 130 us at least, y's
// 0.94 GB 139 us); 777 mixed rows to 2 x 8960, rank 8: 39 us, 0.1 GB. Every CTA of every job reads all ids, so the search grows
// with rows x jobs (8 adapters, 1024 -> 1024, rank 16: 4099 rows 57 us, 131072 rows 8.5 ms). Tried and slower: y loaded and stored
// (at widths that are no multiple of 4, 1504 rows to 130 and 77 columns 38 us, 21 with single reductions), its lines prefetched
// into L2 (40 us for 39), 85 registers and three CTAs an SM for 16-row jobs (one row 7.6 us), 64 ranks a warp (spills), x and A
// two or three chunks ahead (352 rows above 60 and 76). With 128 registers a thread some are spilled: 16-bit adapters 40 bytes with
// 64 rows a job, 88 with 32, none with 16; fp32 ones 552, 216 and 24 (4099 rows, rank 64: 618 us, three products for two and no
// weights ahead).
#include <algorithm>
#include <utility>

#include "ops_common.cuh"

namespace xq {
namespace {

__device__ unsigned int g_lora_error;

constexpr int kThreads = 256, kWarps = kThreads / 32;
// The warps' parts of a pass's sums: [8 / MT][16 * MT][RB].
__host__ __device__ constexpr int sum_bytes(int rank_block) { return 8 * 16 * rank_block * 4; }
constexpr int kJobsGrid = 512;        // jobs of a projection with clusters of their own

struct LoraGrid {
  int jobs;       // at most, of a projection
  int first;      // index of the launch's projections
  int projections;
  int splits;  // clusters that share out a job's columns
  int rank_most;  // of the launch's projections
  int rows;       // T
};

// Row stride of t's pairs in bytes: 64 bytes beside whole 128-byte lines, so that two rows' quads share a load's banks.
__host__ __device__ constexpr int pair_stride(int rank) { return rank * 8 + (rank * 8 % 128 == 64 ? 0 : 64); }
__host__ __device__ constexpr int align16(int x) { return (x + 15) & ~15; }
// Shared memory: t's part [T][rank] fp32, then what follows one behind the other: row counts by adapter, the warps' partial
// sums, t as pairs.
__host__ __device__ constexpr int part_bytes(int rows, int rank) { return rows * rank * 4; }
inline int shared_bytes(int rows, int rank, int rank_block, int n) {
  return part_bytes(rows, rank) + std::max({sum_bytes(rank_block), rows * pair_stride(rank), align16(n * 4)});
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo to 22 bits: hi the upper 11 cut off (an infinity stays one, with lo = 0; what it meets see above), lo rounded.
__device__ __forceinline__ void split(float x, uint32_t* hi, uint32_t* lo) {
  *hi = __float_as_uint(x) & 0xFFFFE000u;
  const float h = __uint_as_float(*hi), rest = h == x ? 0.0f : x - h;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(*lo) : "f"(rest));
}

// Loads that are issued where they stand: a warp's loads go out together, before the products that wait for the first.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 load_floats(const float* p) {
  const uint4 v = load16(p);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// W consecutive weights (8, 4 or 2) as tf32 numbers: hi, and lo for fp32 ones.
template <int TYPE, int W>
struct Weights {
  uint32_t raw[TYPE == kF32 ? W : W / 2];
  __device__ __forceinline__ void load(const void* p, size_t at, bool there) {
    constexpr int kWords = TYPE == kF32 ? W : W / 2;
    const uint32_t* const f = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p) + at * (TYPE == kF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kWords; ++i) raw[i] = 0u;
    if (!there) return;
    if constexpr (kWords >= 4) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = load16(f + i);
        raw[i] = v.x, raw[i + 1] = v.y, raw[i + 2] = v.z, raw[i + 3] = v.w;
      }
    } else if constexpr (kWords == 2) {
      asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(raw[0]), "=r"(raw[1]) : "l"(f));
    } else {
      asm volatile("ld.global.b32 %0, [%1];" : "=r"(raw[0]) : "l"(f));
    }
  }
  // the i-th, i even, and the one after it
  __device__ __forceinline__ void get(int i, uint32_t (&hi)[2], uint32_t (&lo)[2]) const {
    if constexpr (TYPE == kF32) {
      split(__uint_as_float(raw[i]), &hi[0], &lo[0]);
      split(__uint_as_float(raw[i + 1]), &hi[1], &lo[1]);
    } else if constexpr (TYPE == kF16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&raw[i / 2]));
      hi[0] = __float_as_uint(f.x), hi[1] = __float_as_uint(f.y);
    } else {
      hi[0] = raw[i / 2] << 16, hi[1] = raw[i / 2] & 0xFFFF0000u;
    }
  }
};
// d += (ahi + alo) x (bhi + blo), small products first
template <int TYPE>
__device__ __forceinline__ void product(float (&d)[4], const uint32_t (&ahi)[4], const uint32_t (&alo)[4], const uint32_t (&bhi)[2],
                                        const uint32_t (&blo)[2]) {
  if constexpr (TYPE == kF32) mma_tf32(d, ahi, blo[0], blo[1]);
  mma_tf32(d, alo, bhi[0], bhi[1]);
  mma_tf32(d, ahi, bhi[0], bhi[1]);
}

__device__ __forceinline__ uint32_t smem_at(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t at, unsigned cta) {
  uint32_t d;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(at), "r"(cta));
  return d;
}
__device__ __forceinline__ float4 peer_load4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void peer_store4(uint32_t at, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// Place of rank r among the pairs: a thread's ranks are 8, 4 or 2 neighbours (what it loads of B at once), of which step s of
// a chunk takes two; the places of a step's four threads are neighbours.
__device__ __forceinline__ int pair_place(int r, int rank) {
  const int whole = rank & ~31, half = whole + (rank & 16);
  const int c0 = r < whole ? r & ~31 : r < half ? whole : half;
  const int per = r < whole ? 8 : r < half ? 4 : 2, i = r - c0, t = i / per, q = i - t * per;
  return c0 + (q >> 1) * 8 + t * 2 + (q & 1);
}

// A part of a row's product with a row of A, term by term.
template <int TYPE>
__device__ __forceinline__ float exact_part(const float* x, const void* w, size_t at, int n) {
  float s = 0.0f;
#pragma unroll 1
  for (int i = 0; i < n; ++i) s = fmaf(x[i], load_elt<TYPE>(w, at + i), s);
  return s;
}
// The same of t's pairs and a row of B.
template <int TYPE>
__device__ __forceinline__ float exact_column(const uint8_t* pairs, const void* b, size_t at, int rank) {
  float s = 0.0f;
#pragma unroll 1
  for (int r = 0; r < rank; ++r) {
    const float2 t = *reinterpret_cast<const float2*>(pairs + pair_place(r, rank) * 8);
    s = fmaf(t.x + t.y, load_elt<TYPE>(b, at + r), s);
  }
  return s;
}

struct JobShared {
  int rows[64];
  int adapter, chunk;
  int sums[kWarps];
};

// The ids of up to 8 x 32 rows from row m on (those before row `end`), a lane's in steps of 32.
struct Ids {
  int id[8];
  __device__ __forceinline__ void load(const int32_t* ids, int m, int end) {
#pragma unroll
    for (int i = 0; i < 8; ++i) id[i] = m + 32 * i + static_cast<int>(threadIdx.x & 31) < end ? ids[m + 32 * i + (threadIdx.x & 31)] : -1;
  }
};

// The j-th job of a projection with n adapters: its adapter, and its rows in sh.rows; returns how many, 0 if there is none.
// A warp has a run of the rows; up to 256 of them it reads once.
__device__ __noinline__ int find_job(const int32_t* ids, int M, int n, int T, int j, int* counts, JobShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = ((M + kThreads - 1) / kThreads) * 32, m0 = warp * run, m1 = min(M, m0 + run);
  Ids x;
  x.load(ids, m0, m1);
  for (int i = tid; i < n; i += kThreads) counts[i] = 0;
  if (tid == 0) sh.adapter = -1;
  __syncthreads();
  for (int m = m0; m < m1; m += 256) {
    if (m > m0) x.load(ids, m, m1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (m + 32 * i >= m1) break;
      const int id = x.id[i];
      if (id >= n) atomicCAS(&g_lora_error, 0u, kOpsBadAdapter);
      const unsigned same = __match_any_sync(0xffffffffu, id);
      if (id >= 0 && id < n && (same & ((1u << lane) - 1u)) == 0) atomicAdd(&counts[id], __popc(same));
    }
  }
  __syncthreads();
  // jobs are numbered by adapter: a thread's adapters are neighbours
  const int each = (n + kThreads - 1) / kThreads, i0 = tid * each, i1 = min(n, i0 + each);
  int jobs = 0;
  for (int i = i0; i < i1; ++i) jobs += (counts[i] + T - 1) / T;
  int before = jobs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) sh.sums[warp] = before;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += sh.sums[w];
  before -= jobs;
  if (j >= before && j < before + jobs) {
    int i = i0;
    for (; j >= before + (counts[i] + T - 1) / T; ++i) before += (counts[i] + T - 1) / T;
    sh.adapter = i;
    sh.chunk = j - before;
  }
  __syncthreads();
  const int adapter = sh.adapter;
  if (adapter < 0) return 0;
  const int lo = sh.chunk * T, have = min(T, counts[adapter] - lo);
  // the warps' numbers of its rows, then their places
  int mine = 0;
  for (int m = m0; m < m1; m += 256) {
    if (run > 256) x.load(ids, m, m1);
#pragma unroll
    for (int i = 0; i < 8; ++i) mine += __popc(__ballot_sync(0xffffffffu, x.id[i] == adapter));
  }
  if (lane == 0) sh.sums[warp] = mine;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += sh.sums[w];
  for (int m = m0; m < m1 && at < lo + have; m += 256) {
    if (run > 256) x.load(ids, m, m1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned all = __ballot_sync(0xffffffffu, x.id[i] == adapter);
      const int place = at + __popc(all & ((1u << lane) - 1u)) - lo;
      if (x.id[i] == adapter && place >= 0 && place < have) sh.rows[place] = m + 32 * i + lane;
      at += __popc(all);
    }
  }
  __syncthreads();
  return have;
}

// B's W * 4 ranks from r0 on, of a lane's column in each of four products: columns are dealt out so that the results' lane t
// has columns 4 t .. 4 t + 3 and 16 more than those.
template <int TYPE, int W>
__device__ __forceinline__ void load_columns(Weights<TYPE, W> (&w)[4], const AdapterProj& p, size_t b_row, int n0, int r0) {
  const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = n0 + (j >> 1) * 16 + (g >> 1) * 4 + (j & 1) * 2 + (g & 1);
    w[j].load(p.b, (b_row + col) * p.rank + r0 + (threadIdx.x & 3) * W, col < p.N);
  }
}
// t (pairs) x those.
template <int TYPE, int MH, int W>
__device__ __forceinline__ void expand(float (&acc)[MH][4][4], const Weights<TYPE, W> (&w)[4], int r0, const uint8_t* pairs, int stride, int tiles) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int kSteps = W / 2 < 2 ? W / 2 : 2;  // products of 8 ranks before a sum leaves the tensor cores
#pragma unroll
  for (int s0 = 0; s0 < W / 2; s0 += kSteps) {
    uint32_t bhi[kSteps][4][2], blo[kSteps][4][2];
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j].get(2 * (s0 + s), bhi[s][j], blo[s][j]);
#pragma unroll
    for (int m = 0; m < MH; ++m) {
      if (m >= tiles) break;
      float d[4][4] = {};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint8_t* const from = pairs + (m * 16 + g) * stride + (r0 + 8 * (s0 + s) + 2 * t) * 8;
        const uint4 a = *reinterpret_cast<const uint4*>(from), b = *reinterpret_cast<const uint4*>(from + 8 * stride);
        const uint32_t hi[4] = {a.x, b.x, a.z, b.z}, lo[4] = {a.y, b.y, a.w, b.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) product<TYPE>(d[j], hi, lo, bhi[s][j], blo[s][j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][j][i] += d[j][i];
    }
  }
}

// The same of up to 64 rows, by each warp for itself and without a barrier: jobs are numbered by their first rows.
__device__ __forceinline__ int find_job_64(const int32_t* ids, int M, int n, int T, int j, JobShared& sh) {
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  const int id0 = lane < M ? ids[lane] : -1, id1 = lane + 32 < M ? ids[lane + 32] : -1;
  if (max(id0, id1) >= n) atomicCAS(&g_lora_error, 0u, kOpsBadAdapter);
  // a row's place among its adapter's
  const int place0 = __popc(__match_any_sync(0xffffffffu, id0) & below);
  int place1 = 0;
  if (M > 32) {
    place1 = __popc(__match_any_sync(0xffffffffu, id1) & below);
#pragma unroll 4
    for (int i = 0; i < 32; ++i) place1 += __shfl_sync(0xffffffffu, id0, i) == id1;
  }
  unsigned first0 = __ballot_sync(0xffffffffu, id0 >= 0 && id0 < n && place0 % T == 0);
  unsigned first1 = __ballot_sync(0xffffffffu, id1 >= 0 && id1 < n && place1 % T == 0);
  for (int i = 0; i < j; ++i) {
    if (first0 != 0u)
      first0 &= first0 - 1;
    else
      first1 &= first1 - 1;
  }
  if ((first0 | first1) == 0u) return 0;
  const int lead = __ffs(first0 != 0u ? first0 : first1) - 1;
  const int lo = __shfl_sync(0xffffffffu, first0 != 0u ? place0 : place1, lead), id = __shfl_sync(0xffffffffu, first0 != 0u ? id0 : id1, lead);
  // all warps write the same
  if (id0 == id && place0 >= lo && place0 < lo + T) sh.rows[place0 - lo] = lane;
  if (id1 == id && place1 >= lo && place1 < lo + T) sh.rows[place1 - lo] = lane + 32;
  if (lane == 0) sh.adapter = id;
  const int all = __popc(__ballot_sync(0xffffffffu, id0 == id)) + __popc(__ballot_sync(0xffffffffu, id1 == id));
  __syncwarp();
  return min(T, all - lo);
}

// MT: row tiles of 16. RB: a warp's ranks in a pass over x (few for few rows: what matters there is how many instructions are
// seen for the first time). CS: CTAs of a cluster.
template <int TYPE, int MT, int RB, int CS>
__global__ void __launch_bounds__(kThreads, 2) lora_kernel(const __grid_constant__ LoraArgs A, const LoraGrid G) {
  constexpr int T = 16 * MT, kSplit = kWarps / MT, kRankBlock = RB, kCluster = CS;  // kSplit warps share out a CTA's part of K
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ JobShared sh;
  // the projections' jobs in turn: those that there are come before those that there may be
  const int cluster = blockIdx.x / kCluster / G.splits, clusters = gridDim.x / kCluster / G.splits / G.projections;
  const int share = blockIdx.x / kCluster % G.splits;
  const AdapterProj& p = A.p[G.first + cluster % G.projections];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int cta = blockIdx.x % kCluster;
  float* const part = reinterpret_cast<float*>(smem);
  uint8_t* const rest = smem + part_bytes(T, G.rank_most);
  const int rank = p.rank, K = p.K, N = p.N;
  for (int job = cluster / G.projections; job < G.jobs; job += clusters) {
    const int have = A.M <= 64 ? find_job_64(A.ids, A.M, p.n, T, job, sh) : find_job(A.ids, A.M, p.n, T, job, reinterpret_cast<int*>(rest), sh);
    if (have == 0) return;  // nor are there later ones; so for all of the cluster
    const int id = sh.adapter, tiles = (have + 15) / 16;
    const size_t b_row = static_cast<size_t>(id) * N;
    const int step = G.splits * kCluster * kWarps * 32;
    // the next 32 ranks' weights are loaded beside a block's products; no registers for it with 64 rows (442 us for 400)
    constexpr bool kAhead = TYPE != kF32 && MT < 4;
    Weights<TYPE, 8> w[4];
    int n0 = ((share * kCluster + cta) * kWarps + warp) * 32;
    if (MT == 1 && kAhead && rank >= 32 && n0 < N) load_columns(w, p, b_row, n0, 0);
    // ---- t's part from this CTA's K: warp (mt, ks) has 16 rows and a share of the 32-element chunks
    const int chunks = K / 32, mt = warp % MT, ks = warp / MT;
    const int c0 = chunks * cta / kCluster, c1 = chunks * (cta + 1) / kCluster;
    // large ranks: the warps share out the ranks first, then K
    int groups = 1;
    while (groups < kSplit && groups * kRankBlock < rank) groups *= 2;
    const int shares = kSplit / groups, part_k = ks / groups, wide_block = groups * kRankBlock;
    const int k0 = c0 + (c1 - c0) * part_k / shares, k1 = c0 + (c1 - c0) * (part_k + 1) / shares;
    const bool row0 = mt * 16 + g < have, row1 = mt * 16 + g + 8 < have;
    const float* const x0 = p.x + static_cast<size_t>(row0 ? sh.rows[mt * 16 + g] : 0) * K + t * 8;
    const float* const x1 = p.x + static_cast<size_t>(row1 ? sh.rows[mt * 16 + g + 8] : 0) * K + t * 8;
    float* const sums = reinterpret_cast<float*>(rest);  // [shares][T][wide_block]
    for (int block = 0; block < rank; block += wide_block) {
      const int rb = block + ks % groups * kRankBlock, nt = min(kRankBlock, rank - rb) / 8;
      float acc[kRankBlock / 8][4];
#pragma unroll
      for (int n = 0; n < kRankBlock / 8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
      if (mt < tiles && nt > 0) {
        const size_t a0 = (static_cast<size_t>(id) * rank + rb + g) * K + t * 8;
        float4 x[4];  // of the next chunk: two rows, 8 elements each
        auto load_x = [&](int c) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (row0 && c < k1) x[0] = load_floats(x0 + c * 32), x[1] = load_floats(x0 + c * 32 + 4);
          if (row1 && c < k1) x[2] = load_floats(x1 + c * 32), x[3] = load_floats(x1 + c * 32 + 4);
        };
        constexpr int kN = kRankBlock / 8;
        Weights<TYPE, 8> a_next[kN];
        auto load_a = [&](int c) {
#pragma unroll
          for (int n = 0; n < kN; ++n) a_next[n].load(p.a, a0 + static_cast<size_t>(n * 8) * K + c * 32, n < nt && c < k1);
        };
        load_x(k0);
        load_a(k0);
#pragma unroll 1
        for (int c = k0; c < k1; ++c) {
          const float xs[2][8] = {{x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w},
                                  {x[2].x, x[2].y, x[2].z, x[2].w, x[3].x, x[3].y, x[3].z, x[3].w}};
          Weights<TYPE, 8> aw[kN];
#pragma unroll
          for (int n = 0; n < kN; ++n) aw[n] = a_next[n];
          load_x(c + 1);
          load_a(c + 1);
          float d[kN][4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (s % 2 == 0) {
#pragma unroll
              for (int n = 0; n < kN; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.0f;
            }
            uint32_t hi[4], lo[4];
            split(xs[0][2 * s], &hi[0], &lo[0]);
            split(xs[1][2 * s], &hi[1], &lo[1]);
            split(xs[0][2 * s + 1], &hi[2], &lo[2]);
            split(xs[1][2 * s + 1], &hi[3], &lo[3]);
#pragma unroll
            for (int n = 0; n < kN; ++n) {
              if (n < nt) {
                uint32_t bhi[2], blo[2];
                aw[n].get(2 * s, bhi, blo);
                product<TYPE>(d[n], hi, lo, bhi, blo);
              }
            }
            if (s % 2 == 1) {
#pragma unroll
              for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][i] += d[n][i];
            }
          }
        }
        const int across = shares == 1 ? rank : wide_block;  // one share: it is the sum
        float* const row = shares == 1 ? part + (mt * 16 + g) * rank + rb : sums + (part_k * T + mt * 16 + g) * wide_block + rb - block;
#pragma unroll
        for (int n = 0; n < kRankBlock / 8; ++n) {
          if (n < nt) {
            float* const to = row + n * 8 + 2 * t;
            *reinterpret_cast<float2*>(to) = make_float2(acc[n][0], acc[n][1]);
            *reinterpret_cast<float2*>(to + 8 * across) = make_float2(acc[n][2], acc[n][3]);
          }
        }
        float odd = 0.0f;  // not finite if a sum is not
#pragma unroll
        for (int n = 0; n < kN; ++n) odd += (acc[n][0] + acc[n][1]) + (acc[n][2] + acc[n][3]);
        if (!(fabsf(odd) < INFINITY)) {
#pragma unroll 1
          for (int i = 0; i < 4 * nt; ++i) {
            const int r = i / 4 * 8 + 2 * t + (i & 1);
            float* const at = row + r + (i & 2) * 4 * across;
            if ((i & 2 ? row1 : row0) && !isfinite(*at))
              *at = exact_part<TYPE>((i & 2 ? x1 : x0) - t * 8 + k0 * 32, p.a, (static_cast<size_t>(id) * rank + rb + r) * K + k0 * 32, (k1 - k0) * 32);
          }
        }
      }
      if (shares == 1) continue;
      __syncthreads();
      // the warps' shares together, four ranks at a time
      const int quads = min(wide_block, rank - block) / 4;
      for (int i = tid; i < have * quads; i += kThreads) {
        const int row = i / quads, r = (i - row * quads) * 4;
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kSplit; ++w) {
          if (w >= shares) break;
          const float4 v = *reinterpret_cast<const float4*>(sums + (w * T + row) * wide_block + r);
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        *reinterpret_cast<float4*>(part + row * rank + block + r) = s;
      }
      __syncthreads();
    }
    cluster_sync();
    // ---- t: the parts of all CTAs in order. Few values: each CTA adds them all up (one barrier less: 64 rows 11.4 us for 11.7);
    // more: its share of them, which it hands to all (rank 128, 4 rows: 13000 clocks by all, 2500 this way)
    const float scale = p.scales ? p.scales[id] : 1.0f;
    const int quads = have * (rank / 4), stride = pair_stride(rank);  // groups of four ranks
    const bool alone = MT == 1 && quads <= 4096 / kCluster;
    for (int i = alone ? tid : cta * kThreads + tid; i < quads; i += (alone ? 1 : kCluster) * kThreads) {
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int c0 = 0; c0 < kCluster; c0 += 8) {
        float4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = peer_load4(peer(smem_at(part + i * 4), c0 + c));
#pragma unroll
        for (int c = 0; c < 8; ++c) s.x += v[c].x, s.y += v[c].y, s.z += v[c].z, s.w += v[c].w;
      }
      const int row = i / (rank / 4), r = (i - row * (rank / 4)) * 4;
      uint32_t h[4], l[4];
      split(s.x * scale, &h[0], &l[0]);
      split(s.y * scale, &h[1], &l[1]);
      split(s.z * scale, &h[2], &l[2]);
      split(s.w * scale, &h[3], &l[3]);
      // ranks 2k and 2k + 1 keep neighbouring places
      uint8_t *const to0 = rest + row * stride + pair_place(r, rank) * 8, *const to1 = rest + row * stride + pair_place(r + 2, rank) * 8;
      if (alone) {
        *reinterpret_cast<uint4*>(to0) = make_uint4(h[0], l[0], h[1], l[1]);
        *reinterpret_cast<uint4*>(to1) = make_uint4(h[2], l[2], h[3], l[3]);
      } else {
#pragma unroll 1
        for (int c = 0; c < kCluster; ++c) {
          peer_store4(peer(smem_at(to0), c), make_float4(__uint_as_float(h[0]), __uint_as_float(l[0]), __uint_as_float(h[1]), __uint_as_float(l[1])));
          peer_store4(peer(smem_at(to1), c), make_float4(__uint_as_float(h[2]), __uint_as_float(l[2]), __uint_as_float(h[3]), __uint_as_float(l[3])));
        }
      }
    }
    if (alone) {
      asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // this CTA has read the others' parts
      __syncthreads();
    } else {
      cluster_sync();
    }
    // ---- y: a warp has 32 columns, a lane 4 and 4 of them (two of each of four products). A value is added to y in L2, by the
    // only addition that it gets in the call: no loads to wait for.
    const bool wide = N % 4 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15) == 0;
    Weights<TYPE, 8> next[4];
    if (MT > 1 && kAhead && rank >= 32 && n0 < N) load_columns(w, p, b_row, n0, 0);
    for (; n0 < N; n0 += step) {
      float acc[MT][4][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j][0] = acc[m][j][1] = acc[m][j][2] = acc[m][j][3] = 0.0f;
      int r0 = 0;
#pragma unroll 1
      for (; r0 + 32 <= rank; r0 += 32) {
        if (kAhead) {
          const bool more = r0 + 64 <= rank;
          if (more || n0 + step < N) load_columns(next, p, b_row, more ? n0 : n0 + step, more ? r0 + 32 : 0);
        } else {
          load_columns(w, p, b_row, n0, r0);
        }
        expand<TYPE, MT, 8>(acc, w, r0, rest, stride, tiles);
        if (kAhead) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = next[j];
        }
      }
      if (rank & 16) {
        Weights<TYPE, 4> part_w[4];
        load_columns(part_w, p, b_row, n0, r0);
        expand<TYPE, MT, 4>(acc, part_w, r0, rest, stride, tiles);
        r0 += 16;
      }
      if (rank & 8) {
        Weights<TYPE, 2> part_w[4];
        load_columns(part_w, p, b_row, n0, r0);
        expand<TYPE, MT, 2>(acc, part_w, r0, rest, stride, tiles);
      }
      unsigned bad = 0u;  // a bit for the eight values of a row if they are not all finite
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (m >= tiles) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int place = m * 16 + h * 8 + g, row = place < have ? sh.rows[place] : -1;
          if (row < 0 || !XQ_IN(row, A.M, kChkLoraRow)) continue;
          float* const to = p.y + static_cast<size_t>(row) * N;
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) sum += acc[m][j][2 * h] + acc[m][j][2 * h + 1];
          if (!(fabsf(sum) < INFINITY)) {
            bad |= 1u << (m * 2 + h);
            continue;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int n = n0 + 16 * q + 4 * t;
            const float v[4] = {acc[m][2 * q][2 * h], acc[m][2 * q][2 * h + 1], acc[m][2 * q + 1][2 * h], acc[m][2 * q + 1][2 * h + 1]};
            if (wide && n + 4 <= N) {
              asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to + n), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n + i < N) asm volatile("red.global.add.f32 [%0], %1;" ::"l"(to + n + i), "f"(v[i]) : "memory");
            }
          }
        }
      }
      for (; bad != 0u; bad &= bad - 1u) {
        const int place = (__ffs(bad) - 1) * 8 + g, n = n0 + 4 * t;
#pragma unroll 1
        for (int c = n; c < min(n + 20, N); c += (c - n) == 3 ? 13 : 1)
          atomicAdd(p.y + static_cast<size_t>(sh.rows[place]) * N + c, exact_column<TYPE>(rest + place * stride, p.b, (b_row + c) * rank, rank));
      }
    }
    if (alone) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // its own are no longer read
    __syncthreads();  // of t and the rows, before the next job's
  }
}

template <int TYPE, int MT, int RB, int CS>
cudaError_t launch(const LoraArgs& a, const LoraGrid& g, int n_most, cudaStream_t s) {
  static std::atomic<unsigned long long> allowed{0}, wide{0};
  cudaError_t e = allow_shared(lora_kernel<TYPE, MT, RB, CS>, 200 * 1024, allowed);
  if (CS > 8 && e == cudaSuccess) {  // once a device, as allow_shared
    int dev = 0;
    e = cudaGetDevice(&dev);
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (e == cudaSuccess && !(wide.load(std::memory_order_relaxed) & bit)) {
      e = cudaFuncSetAttribute(lora_kernel<TYPE, MT, RB, CS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess) wide.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CS * std::min(g.jobs, kJobsGrid) * g.projections * g.splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = shared_bytes(16 * MT, g.rank_most, RB, n_most);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CS;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_kernel<TYPE, MT, RB, CS>, a, g);
}

template <int TYPE>
cudaError_t launch_type(const LoraArgs& a, LoraGrid g, int n_most, int columns_most, cudaStream_t s) {
  constexpr int kPlaces = 304;  // CTAs that are resident, two an SM
  const long long rows = static_cast<long long>(a.M) * g.projections;
  const int MT = rows < 2432 ? 1 : g.rank_most > 128 ? 2 : 4;
  g.rows = 16 * MT;
  g.jobs = std::max(1, std::min(a.M, n_most) + a.M / g.rows);
  g.splits = 1;
  if (MT == 4) return launch<TYPE, 4, 32, 8>(a, g, n_most, s);
  if (MT == 2) return launch<TYPE, 2, 32, 8>(a, g, n_most, s);
  // Few jobs: larger clusters, and several of them for a job's columns.
  const long long clusters = static_cast<long long>(std::min(g.jobs, kJobsGrid)) * g.projections;
  const bool wide = clusters * 16 <= kPlaces / 2;
  const int size = wide ? 16 : 8;  // a warp has 32 columns: 256 a CTA
  g.splits = static_cast<int>(std::max(1ll, std::min(kPlaces / (clusters * size), (columns_most + 256ll * size - 1) / (256 * size))));
  return wide ? launch<TYPE, 1, 16, 16>(a, g, n_most, s) : launch<TYPE, 1, 16, 8>(a, g, n_most, s);
}

}  // namespace

cudaError_t launch_lora(const LoraArgs& args, cudaStream_t s) {
  g_kv_launched.store(true, std::memory_order_relaxed);
  // projections of one type together
  LoraArgs a = args;
  for (int i = 1; i < a.n_proj; ++i)
    for (int k = i; k > 0 && a.p[k].type < a.p[k - 1].type; --k) std::swap(a.p[k], a.p[k - 1]);
  for (int i = 0; i < a.n_proj;) {
    LoraGrid g = {};
    int e = i, n_most = 0, columns_most = 0;
    g.first = i;
    for (; e < a.n_proj && a.p[e].type == a.p[i].type; ++e) {
      g.rank_most = std::max(g.rank_most, a.p[e].rank);
      n_most = std::max(n_most, a.p[e].n);
      columns_most = std::max(columns_most, a.p[e].N);
    }
    g.projections = e - i;
    const int type = a.p[i].type;
    const cudaError_t r = type == kF32   ? launch_type<kF32>(a, g, n_most, columns_most, s)
                          : type == kF16 ? launch_type<kF16>(a, g, n_most, columns_most, s)
                                         : launch_type<kBF16>(a, g, n_most, columns_most, s);
    if (r != cudaSuccess) return r;
    i = e;
  }
  return cudaSuccess;
}

cudaError_t take_lora_error(unsigned int* code) { return take_record(g_lora_error, code); }
cudaError_t take_lora_check(unsigned int* code) { return take_check_word(code); }

}  // namespace xq
