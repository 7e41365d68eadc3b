// Index arithmetic of ragged batches over a paged 4-bit KV cache, shared by the
// kernels and by host code (plain C++ when compiled without nvcc).
//
// Every index that comes from device memory (row ranges, lengths, page
// numbers) is checked here before it is used as an address: a sequence whose
// rows do not lie in [0, T) has none, a page number outside the pool is -1.
#pragma once

#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define QOQ_HD __host__ __device__ __forceinline__
#else
#define QOQ_HD inline
#endif

namespace qoq {

// The query tokens of sequence b: rows q_start[b] .. + n of T (n = 0 for a
// range that is not one).
struct RowRange {
  int first, n;
};
QOQ_HD RowRange rows_of(const int* q_start, int b, int T) {
  const int a = q_start[b], e = q_start[b + 1];
  RowRange r;
  r.first = a;
  r.n = (a < 0 || e > T || e < a) ? 0 : e - a;
  return r;
}

// Tokens of a sequence that the cache can hold: seqlen clamped to
// [0, capacity].
QOQ_HD int clamp_len(int seqlen, int capacity) {
  return seqlen < 0 ? 0 : (seqlen > capacity ? capacity : seqlen);
}

// Position of the i-th of a sequence's n query tokens, the last of which is
// token seqlen - 1 (64 bits: seqlen is any int).
QOQ_HD long long position_of(int seqlen, int n, int i) {
  return static_cast<long long>(seqlen) - n + i;
}

// How many tokens a query at position pos sees of a sequence with len cached
// tokens: the ones at positions 0 .. pos.
QOQ_HD int visible(long long pos, int len) {
  return pos < 0 ? 0 : (pos + 1 < len ? static_cast<int>(pos + 1) : len);
}

// Number of the 16-token block (of one KV head) in the pool that holds block
// `blk` of a sequence, or -1 if its page is not one of the pool's.  ppb = 16-token
// blocks per page; blk < width * ppb.
QOQ_HD int pool_block(const int* table_row, int blk, int ppb, int pages, int Hkv, int hk) {
  const int idx = blk / ppb;
  const int pid = table_row[idx];
  if (pid < 0 || pid >= pages) return -1;
  return (pid * Hkv + hk) * ppb + (blk - idx * ppb);
}

// Slots of work for ragged row tiles: sequence b owns the tile slots
// [slot_base(b), slot_base(b + 1)), at least ceil(n * g / tile) of them, so that
// the sum over the batch is known without reading q_start: at most
// floor(T * g / tile) + B.
QOQ_HD int slot_base(int row_first, int b, int g, int tile) {
  return static_cast<int>(static_cast<long long>(row_first) * g / tile) + b;
}

}  // namespace qoq
