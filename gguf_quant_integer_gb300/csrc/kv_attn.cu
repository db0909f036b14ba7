// Attention over the quantized KV cache: which kernels a call runs, and their
// workspace.
#include "kv_tile.cuh"

namespace xq {
namespace {

// Query rows of a CTA: n-tiles of 8 columns. fp32 takes two columns a row (its
// two fp16 numbers). So do 16-bit queries of at most 4 rows, which have the
// columns to spare: the weights' second numbers make them as exact as the
// result's type, and a lane has half the scores. More rows than one tile holds
// take two, more than two several row chunks, which read the same keys
// (through L2). dim 256 has registers for one tile.
struct Rows {
  bool exact;
  int np, nt;
};
Rows rows_for(const KvAttnArgs& a, int rows) {
  const bool exact = a.type == kF32;
  if (exact || rows <= 4) return {exact, 2, rows <= 4 || a.c.dim == 256 ? 1 : 2};
  return {exact, 1, rows <= 8 || a.c.dim == 256 ? 1 : 2};
}

// One pass of a call: every sequence's own pages, or the prefix for all rows.
struct Pass {
  int seqs, rows;   // rows of a pair
  long long keys;   // of a sequence, at most
};
Pass own_pass(const KvAttnArgs& a) { return {a.batch, a.rows, static_cast<long long>(a.max_pages) << a.c.page_shift}; }
Pass prefix_pass(const KvAttnArgs& a) { return {1, a.batch * a.rows, a.prefix_len}; }

// Whether a pass goes to the tcgen05 tiles, which are for 16-bit queries. They
// take some 20 us whatever the work, and then, from 64 rows on, a fraction of
// the split kernel's time for it. Both measured (tiles, split; 8 KV heads, dim
// 128, Q8_0, whole calls behind a prefix of that many keys, us):
//   bf16  256 rows x 2048 keys 32 and 32, x 8192 40 and 65, x 32768 69 and 196;
//         128 rows x 2048 24 and 23, x 8192 28 and 40, x 32768 48 and 106;
//         64 rows x 2048 24 and 20, x 8192 31 and 29, x 32768 59 and 62;
//         32 rows x 32768 57 and 41
//   fp16  256 rows x 2048 34 and 32, x 8192 45 and 65, x 32768 81 and 196;
//         128 rows x 2048 25 and 23, x 8192 31 and 40, x 32768 55 and 106;
//         64 rows x 8192 34 and 29, x 32768 65 and 62
// Where the rule is wrong: at 4.2 million (256 x 2048, 64 x 8192) the tiles are
// as fast or 7 % slower for bf16 and 7 to 16 % slower for fp16, and 64 fp16
// rows never gain. It counts the table's width, not the lengths, which are on
// the device.
bool tiled(const KvAttnArgs& a, const Pass& p) {
  if (a.type == kF32 || a.c.dim > 128 || p.rows < 64) return false;
  const long long reach = static_cast<long long>(a.window) + a.n_q;
  const long long seen = a.window > 0 && p.keys > reach ? reach : p.keys;
  return static_cast<double>(p.seqs) * p.rows * seen * a.c.heads >= 3e6;
}

// CTAs and rows of partial results (two a CTA): three resident CTAs an SM of
// 4 or 8 rows, two of up to 16; one of 128 or 256.
constexpr int kMaxCtas = 3 * kNumSMs;
constexpr size_t kSplitRows = 2 * kMaxCtas * 16;
constexpr size_t kTilePartRows = static_cast<size_t>(2) * kNumSMs * kTileChunk;

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

struct Layout {
  size_t record, part_el, part_o, pre_el, pre_o, total;
};
Layout layout(const KvAttnArgs& a) {
  Layout L;
  const bool tile = tiled(a, own_pass(a)) || (a.prefix_len > 0 && tiled(a, prefix_pass(a)));
  const size_t rows = tile ? kTilePartRows : kSplitRows;
  const size_t outs = a.prefix_len > 0 ? static_cast<size_t>(a.batch) * a.n_q * a.q_heads : 0;
  L.record = 0;
  L.part_el = L.record + kMaxCtas * sizeof(int4);
  L.part_o = L.part_el + rows * 8;
  L.pre_el = L.part_o + rows * a.c.dim * 4;
  L.pre_o = L.pre_el + round16(outs * 8);
  L.total = L.pre_o + outs * a.c.dim * 4;
  return L;
}

cudaError_t run(SplitArgs& p, const Pass& pass, const KvAttnArgs& a, int bits, cudaStream_t s) {
  p.seqs = pass.seqs;
  p.rows = pass.rows;
  const bool tile = tiled(a, pass);
  const Rows f = rows_for(a, p.rows);
  const int r = tile ? kTileChunk : f.nt * 8 / f.np;
  p.chunks = (p.rows + r - 1) / r;
  const long long units = (pass.keys + kAttnUnit - 1) / kAttnUnit;
  // Sequences too short for a second CTA to be worth a join: whole pairs.
  p.whole = units <= (p.store ? kAttnWholeOwn : kAttnWhole);
  // One a CTA where there are CTAs for all: that needs no lengths. Else stretches of equal work, not number (256 sequences
  // of up to 256 tokens, 8 KV heads: 29.4 us, not 32.0).
  p.counted = p.whole && static_cast<long long>(p.seqs) * p.c.heads * p.chunks <=
                             (tile ? 1 : f.nt == 2 || a.c.dim == 256 ? 2 : 3) * kNumSMs;
  p.head = tile ? kTileHead : f.nt == 2 ? kAttnHead2 : kAttnHead;
  p.units = p.seqs * ((units > 1 ? units : 1) + p.head) * p.c.heads * p.chunks;
  if (tile) {
    switch (a.c.dim) {
      case 64: return KvTileDim<64>::launch(p, bits, a.type == kF16, s);
      case 96: return KvTileDim<96>::launch(p, bits, a.type == kF16, s);
      default: return KvTileDim<128>::launch(p, bits, a.type == kF16, s);
    }
  }
  switch (a.c.dim) {
    case 64: return KvAttnDim<64>::launch(p, bits, f.exact, f.np, f.nt, s);
    case 96: return KvAttnDim<96>::launch(p, bits, f.exact, f.np, f.nt, s);
    case 128: return KvAttnDim<128>::launch(p, bits, f.exact, f.np, f.nt, s);
    default: return KvAttnDim<256>::launch(p, bits, f.exact, f.np, f.nt, s);
  }
}

}  // namespace

size_t kv_attn_workspace(const KvAttnArgs& a, int) { return layout(a).total; }

cudaError_t launch_kv_attn(const KvAttnArgs& a, int bits, void* workspace, cudaStream_t s) {
  const Layout L = layout(a);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  SplitArgs p = {};
  p.c = a.c;
  p.type = a.type;
  p.group = a.group;
  p.q_heads = a.q_heads;
  p.n_q = a.n_q;
  p.q = a.q;
  p.max_pages = a.max_pages;
  p.lens = a.lens;
  p.prefix_len = a.prefix_len;
  p.scale = a.scale;
  p.window = a.window;
  p.record = reinterpret_cast<int4*>(ws + L.record);
  p.part_el = reinterpret_cast<float*>(ws + L.part_el);
  p.part_o = reinterpret_cast<float*>(ws + L.part_o);
  p.pre_el = reinterpret_cast<float*>(ws + L.pre_el);
  p.pre_o = reinterpret_cast<float*>(ws + L.pre_o);
  p.out = a.out;
  p.pages = a.pages;
  p.page_stride = a.page_stride;
  p.store = a.prefix_len > 0;
  p.part_rows = static_cast<long long>((L.part_o - L.part_el) / 8);
  p.records = kMaxCtas;
  const cudaError_t e = run(p, own_pass(a), a, bits, s);
  if (e != cudaSuccess || a.prefix_len == 0) return e;
  // Then every row of the call against the prefix, which is read once. The
  // pass may start beside the first one where that leaves no parts (they would
  // share the workspace).
  p.store = false;
  p.merge = true;
  p.late = p.whole;
  p.flat = true;
  p.pages = a.prefix_pages;
  return run(p, prefix_pass(a), a, bits, s);
}

namespace {
typedef cudaError_t (*TakeFn)(unsigned int*);
// The first word recorded in any of the kernels' translation units; all are cleared.
template <size_t N>
cudaError_t take_all(const TakeFn (&fns)[N], unsigned int* code) {
  *code = 0;
  for (TakeFn f : fns) {
    unsigned int c = 0;
    const cudaError_t e = f(&c);
    if (e != cudaSuccess) return e;
    if (*code == 0) *code = c;
  }
  return cudaSuccess;
}
}  // namespace

cudaError_t take_kv_attn_error(unsigned int* code) {
  const TakeFn fns[4] = {KvAttnDim<64>::take_error, KvAttnDim<96>::take_error, KvAttnDim<128>::take_error,
                         KvAttnDim<256>::take_error};
  return take_all(fns, code);
}
cudaError_t take_kv_tile_error(unsigned int* index, unsigned int* wait) {
  typedef cudaError_t (*TakeTile)(unsigned int*, unsigned int*);
  const TakeTile fns[3] = {KvTileDim<64>::take_error, KvTileDim<96>::take_error, KvTileDim<128>::take_error};
  *index = *wait = 0;
  for (TakeTile f : fns) {
    unsigned int i = 0, w = 0;
    const cudaError_t e = f(&i, &w);
    if (e != cudaSuccess) return e;
    if (*index == 0) *index = i;
    if (*wait == 0) *wait = w;
  }
  return cudaSuccess;
}
cudaError_t take_kv_attn_check(unsigned int* code) {
  const TakeFn fns[7] = {KvAttnDim<64>::take_check, KvAttnDim<96>::take_check, KvAttnDim<128>::take_check, KvAttnDim<256>::take_check,
                         KvTileDim<64>::take_check, KvTileDim<96>::take_check, KvTileDim<128>::take_check};
  return take_all(fns, code);
}

}  // namespace xq
