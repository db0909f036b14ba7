// What the KV cache kernels share: the cache as a kernel argument, element
// types, and the record of invalid indices.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "xq_check.cuh"

namespace xq {

// Element types of activations (the GGUF ids of the public header).
constexpr int kF32 = 0, kF16 = 1, kBF16 = 30;

__host__ __device__ constexpr int kv_elt_bytes(int type) { return type == kF32 ? 4 : 2; }

// The pools and their layout. A page: codes [heads][page][row_bytes], then
// fp16 scales [heads][page][dim / 32], from scale_off.
struct KvView {
  uint8_t* k;
  uint8_t* v;
  int n_pages, page_shift, heads, dim;
  int row_bytes;           // of one row's codes
  int scale_off;           // of the scales within a page
  long long page_bytes;    // pools pass 2^31 bytes: every page offset is 64-bit
};

// One attention call. Rows are the query rows of one KV head of one
// sequence: row r = i * group + j is query token i, query head h * group + j.
struct KvAttnArgs {
  KvView c;
  int type;
  int batch, n_q, q_heads, group, rows;
  const void* q;
  void* out;
  const int32_t* pages;
  int page_stride, max_pages;
  const int32_t* lens;
  float scale;
  int window;
  const int32_t* prefix_pages;
  int prefix_len;
};

enum KvRecord : unsigned { kKvBadSlot = 1, kKvBadPage = 2, kKvBadLen = 3 };

// Position of query token i of a sequence whose own pages hold n tokens, with
// `prefix` tokens before them: keys 0 .. pos are visible (none if pos < 0).
__host__ __device__ inline int kv_pos(int prefix, int n, int n_q, int i) { return prefix + n - n_q + i; }

cudaError_t launch_kv_write(const KvView& c, int bits, int x_type, const void* k, long long k_stride, const void* v,
                            long long v_stride, const int64_t* slots, int n_tokens, cudaStream_t s);
cudaError_t launch_kv_read(const KvView& c, int bits, const int64_t* slots, int n_tokens, int y_type, void* k, void* v,
                           cudaStream_t s);
cudaError_t launch_kv_attn(const KvAttnArgs& a, int bits, void* workspace, cudaStream_t s);
size_t kv_attn_workspace(const KvAttnArgs& a, int bits);

namespace {
// Whether a kernel of this translation unit was launched since the program began. Its records are read only then: a read
// takes 8 us and loads the unit's kernels, which callers who use no KV cache need not pay for.
std::atomic<bool> g_kv_launched{false};

// Allow a kernel `bytes` of dynamic shared memory on the current device. `done`: the devices that have it (one bit each, the
// first 64), of this kernel.
template <typename K>
inline cudaError_t allow_shared(K kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Read a record (a word in device memory), and clear it if it is set.
template <typename Word>
inline cudaError_t take_record(const Word& word, unsigned int* code) {
  *code = 0;
  if (!g_kv_launched.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaError_t e = cudaMemcpyFromSymbol(code, word, sizeof(*code));
  const unsigned int zero = 0;
  if (e == cudaSuccess && *code != 0) e = cudaMemcpyToSymbol(word, &zero, sizeof(zero));
  return e;
}
}  // namespace

// Read and clear the records of invalid indices (0: none) and the checked
// builds' words of the KV kernels.
cudaError_t take_kv_cache_error(unsigned int* code);
cudaError_t take_kv_attn_error(unsigned int* code);
cudaError_t take_kv_tile_error(unsigned int* index, unsigned int* wait);  // its invalid indices, its waits that ran out
cudaError_t take_kv_cache_check(unsigned int* code);
cudaError_t take_kv_attn_check(unsigned int* code);

}  // namespace xq
