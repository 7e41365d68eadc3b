// How prompt chunks are cut into units of work: shared by the kernel that lists them,
// the prompt kernel and the merge.
#pragma once

#include "qoq_attn.cuh"
#include "qoq_device.cuh"
#include "qoq_paged.h"

namespace qoq {

constexpr int kSlotRows = 256;                  // rows of a slot
constexpr int kStepTokens = 128;
constexpr int kMinChunk = 8;                    // steps: a split's least length
constexpr int kMaxStagedSeqs = 1024;
constexpr int kSorted = 128;                    // slots up to which units go by length
constexpr int kPlanScratch = kSorted * 8 + kMaxStagedSeqs * 4;

// A unit of work: steps step0 .. step1 - 1 (of 128 tokens) for the slot of rows from
// row0 on of sequence b (-1: nothing) and KV head hk.
struct __align__(16) PromptUnit {
  int b, row0, hk;
  int whole;         // the slot is not split
  int step0, step1;
  int part;          // its number among the units of split slots
  int unused;
};

struct PromptPlan {
  PromptUnit* units;       // null: no prompt chunks
  int2* meta;              // per (slot, KV head): first part and parts (null: nothing splits)
  int grid, tiles, target, min_rows;
};

// Steps of slot `slot` (128-token steps that its last row sees), -1 for a slot
// without work here; b and the first row of it.
__device__ __forceinline__ int slot_steps(const PagedArgs& a, int slot, int min_rows,
                                          const int* starts, int& b, int& row0) {
  int lo = 0, hi = a.B;        // the last sequence whose slots start at or before this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (slot_base(starts[mid], mid, a.g, kSlotRows) <= slot) lo = mid;
    else hi = mid;
  }
  b = lo;
  const RowRange rr = rows_of(a.q_start, lo, a.T);
  const int R = rr.n * a.g;
  const long long first =
      static_cast<long long>(slot - slot_base(rr.first, lo, a.g, kSlotRows)) * kSlotRows;
  if (rr.n <= 0 || rr.n > a.max_q || R < min_rows || first < 0 || first >= R) return -1;
  row0 = static_cast<int>(first);
  const int last = (row0 + kSlotRows < R ? row0 + kSlotRows : R) - 1;
  const int len = clamp_len(a.seqlen[lo], a.width * a.page);
  return (visible(position_of(a.seqlen[lo], rr.n, last / a.g), len) + kStepTokens - 1) / kStepTokens;
}

// The list of units, by one CTA of kThreads; scratch: kPlanScratch bytes of shared
// memory.  Splits are equally long over the whole batch: the
// batch's steps over `target`, kMinChunk at least.  Units go by length where the slots
// are few (the CTAs that come last should be the shortest), else the last slots, which
// see most, come first.  meta: per (slot, KV head) its first part and their number, 0
// for a slot without work and 1 for a whole one.
template <int kThreads>
__device__ __forceinline__ void list_prompt_units(const PagedArgs& a, const PromptPlan& pp,
                                                  uint8_t* scratch) {
  __shared__ long long s_sum[kThreads / 32];
  __shared__ int2 s_scan[kThreads / 32];
  int2* s_len = reinterpret_cast<int2*>(scratch);
  int* s_starts = reinterpret_cast<int*>(s_len + kSorted);
  const int tiles = pp.tiles, min_rows = pp.min_rows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int* starts = a.q_start;
  if (a.B <= kMaxStagedSeqs) {
    for (int i = tid; i < a.B; i += kThreads) s_starts[i] = a.q_start[i];
    starts = s_starts;
  }
  __syncthreads();
  int b0 = 0, row0 = 0, n0 = -1;
  long long sum = 0;
  for (int s = tid; s < tiles; s += kThreads) {
    int b = 0, r = 0;
    const int n = slot_steps(a, tiles - 1 - s, min_rows, starts, b, r);
    if (s == tid) {
      n0 = n;
      b0 = b;
      row0 = r;
    }
    if (n > 0) sum += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) sum += s_sum[w];
  const long long want = (sum * a.Hkv + pp.target - 1) / pp.target;
  const int chunk = static_cast<int>(want < kMinChunk ? kMinChunk : want);
  const bool sorted = tiles <= kSorted;
  int base = 0, pbase = 0;
  for (int s0 = 0; s0 < tiles; s0 += kThreads) {
    const int s = s0 + tid;
    int n = n0, b = b0, r = row0;
    if (s0 > 0) n = s < tiles ? slot_steps(a, tiles - 1 - s, min_rows, starts, b, r) : -1;
    const int nsplit = n < 0 ? 0 : (n <= chunk ? 1 : (n + chunk - 1) / chunk);
    const int per = nsplit > 0 ? (n + nsplit - 1) / nsplit : 0;      // splits are equally long
    const int mine = nsplit * a.Hkv, parts = nsplit > 1 ? mine : 0;
    int incl = mine, pincl = parts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      const int pup = __shfl_up_sync(0xffffffffu, pincl, o);
      if (lane >= o) {
        incl += up;
        pincl += pup;
      }
    }
    if (lane == 31) s_scan[warp] = make_int2(incl, pincl);
    if (sorted)
      s_len[s] = make_int2(nsplit > 0 ? per : -1, mine);
    __syncthreads();
    int first = base + incl - mine, part = pbase + pincl - parts;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        first += s_scan[w].x;
        part += s_scan[w].y;
      }
      base += s_scan[w].x;
      pbase += s_scan[w].y;
    }
    if (sorted && mine > 0) {
      first = 0;
      for (int i = 0; i < tiles; ++i) {
        const int2 o = s_len[i];
        first += o.x > per || (o.x == per && i < tid) ? o.y : 0;
      }
    }
    if (s < tiles && pp.meta != nullptr)
      for (int hk = 0; hk < a.Hkv; ++hk)
        pp.meta[(tiles - 1 - s) * a.Hkv + hk] =
            make_int2(nsplit > 1 ? part + hk * nsplit : 0, nsplit);
    for (int i = 0; i < mine; ++i) {
      PromptUnit u;
      u.b = b;
      u.row0 = r;
      u.hk = i / nsplit;
      u.whole = nsplit == 1;
      u.step0 = (i - u.hk * nsplit) * per;
      u.step1 = u.step0 + per < n ? u.step0 + per : n;
      u.part = part + i;
      u.unused = 0;
      if (first + i < pp.grid) pp.units[first + i] = u;
    }
    __syncthreads();
  }
  for (int i = base + tid; i < pp.grid; i += kThreads) pp.units[i].b = -1;
}

}  // namespace qoq
