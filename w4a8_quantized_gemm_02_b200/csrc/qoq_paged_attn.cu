// Attention over a paged 4-bit KV cache: single tokens (decode) and the few
// query tokens of a sequence that is verified or extended by a handful.
//
// Rows.  The n query tokens of a sequence times the g = Hq / Hkv heads of a KV
// head are the rows of one problem: row r = i g + h.  Up to 16 rows run here,
// four to an MMA's eight columns; more go to the prompt kernel.
//
// Arithmetic.  The products run on the codes c, never on dequantized vectors.
// With k^ = s c + m:
//     q . k^_t = s_t (q . c_t) + m_t Q,    Q = sum_i q_i,
//     sum_t p_t v^_t = sum_t w_t (c_t - 8) + sum_t p_t (m_t + 8 s_t),  w_t = p_t s_t.
// Scores: 8-bit integer MMAs, exact in INT32, with the queries as 16-bit fixed
// point of their row (a column for the high and one for the low byte): a shift
// and two masks unpack eight codes.  That rounds a query value to 2^-16 of its
// row's largest, less than its own FP16 rounding for values within 32 times of
// it; a score moves by about 3e-5 of the size of k^ where |q| stays under 4.
// Outputs: FP16 MMAs, the weights as a high and a low FP16 column (22 bits from 2^-3
// up, where the largest of a row is at least 2^10; 2^-25 at the least, which is 2^-35 of
// it), the codes centred on 8, which keeps what the tensor cores' FP32 accumulation
// touches as small as v^ about its vector's middle: over 131000 tokens, sums of
// uncentred codes lost half the output's digits (5.5e-4 of it against 2.6e-4).
//
// The running reference (qoq_attn.cuh) only moves when a weight could pass FP16's
// range: one vote an iteration instead of a reduction, on the largest scale of a
// lane's four tokens; the weights themselves are looked at when that vote is carried.
//
// Work.  The batch's blocks of 16 tokens, in the order of sequences, KV heads and
// tokens, are cut into equal runs, one for each resident CTA, whatever the mix of
// lengths.  A run covers whole (sequence, KV head) pairs, whose outputs it writes,
// and at most one unfinished pair at either end, whose partial results a second
// kernel merges.
//
// Bound.  136 bytes a token and KV head, read once; the instructions that unpack
// them come close behind (see the figures at the kernel).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "qoq.h"
#include "qoq_attn.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"
#include "qoq_kv4.cuh"
#include "qoq_paged.h"
#include "qoq_prompt_plan.cuh"

namespace qoq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;                           // per warp: iterations in flight
constexpr int kBlockBytes = 1024 + 1024 + 128;       // K codes, V codes, scales of a block
constexpr int kStageBytes = 2 * kBlockBytes;         // an iteration is two blocks
constexpr int kMinBlocks = 16;                       // a run's least length
constexpr int kPairCost = 12;                        // a pair's beginning and end, in blocks
constexpr float kFixed = 32512.0f;                   // 127 * 256: a query row's largest value

// CTAs of the decode kernel on an SM, by its tiles of four rows.
constexpr int resident_ctas(int nt) { return nt == 1 ? 4 : (nt == 2 ? 3 : 2); }

__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes minus 8: 0x6400 | c is 1024 + c, 0x5400 | 16 c is 64 + c.
__device__ __forceinline__ uint32_t minus(uint32_t n, float k) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&n), __float2half2_rn(k));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void v_frag(uint32_t word, uint32_t (&a)[4]) {
  const uint32_t hi = word >> 8;
  a[0] = minus(and_or(word, 0x000f000fu, 0x64006400u), 1032.0f);
  a[1] = minus(and_or(word, 0x00f000f0u, 0x54005400u), 72.0f);
  a[2] = minus(and_or(hi, 0x000f000fu, 0x64006400u), 1032.0f);
  a[3] = minus(and_or(hi, 0x00f000f0u, 0x54005400u), 72.0f);
}

// 16-token blocks of sequence b for this kernel: 0 for an empty one that still
// has rows to write, -1 where it has no work here.
__device__ __forceinline__ int blocks_of(const PagedArgs& a, int b, int rows_max_here) {
  const RowRange rr = rows_of(a.q_start, b, a.T);
  if (rr.n <= 0 || rr.n > a.max_q || rr.n * a.g > rows_max_here) return -1;
  return (clamp_len(a.seqlen[b], a.width * a.page) + 15) >> 4;
}
// Its share of the work for one KV head: its blocks (an empty one counts as one)
// and kPairCost in front of them.
__device__ __forceinline__ int weight_of(int blocks) {
  return blocks < 0 ? 0 : kPairCost + (blocks == 0 ? 1 : blocks);
}

// Measured (32 / 8 heads; two cards): 64 sequences of 300 - 8100 tokens, 292 MB, 70 to 74 us
// with the merge (4.2 to 3.9 TB/s, 64 to 60% of the copy rate); two of 120000 - 131000, 265 MB,
// 61 to 64 us; 64 / 64 heads, 24 sequences of 1000 - 2047, 310 MB, 76 to 79 us.  (A reference
// that follows the scores alone: 1% less.)  Issue slots and the integer pipe are half used
// and DRAM a little more: what is left is latency between dependent instructions, at the 16
// warps an SM that the registers allow, the ring that runs dry at each pair's end, and the
// merge.  3 or 4 copy stages and an unrolled loop were no faster.
//
// Grid: `ctas` CTAs, one for each that is resident, and one more where there may be
// prompt chunks, which lists their units.
template <int NT>
__global__ void __launch_bounds__(kThreads, resident_ctas(NT))
paged_decode_kernel(const PagedArgs a, int ctas, const PromptPlan pp) {
  constexpr int kRows = 4 * NT;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long s_sum[kWarps], s_start;
  __shared__ int s_b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();
  if (static_cast<int>(blockIdx.x) == ctas) {
    static_assert(kPlanScratch <= kWarps * kStages * kStageBytes, "scratch");
    list_prompt_units<kThreads>(a, pp, smem);
    return;
  }

  // --- this CTA's run: [start, end) of the batch's `total` blocks ---
  // (counted with it: the sequences that have work, in the upper bits)
  auto share = [&](int b) {
    const int w = b < a.B ? weight_of(blocks_of(a, b, kRows)) : 0;
    return w ? (1LL << 40) + w : 0LL;
  };
  const long long mine = share(threadIdx.x);
  const int w0 = static_cast<int>(mine);
  long long sum = mine;
  for (int b = threadIdx.x + kThreads; b < a.B; b += kThreads) sum += share(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
  const int active = static_cast<int>(sum >> 40);
  sum &= (1LL << 40) - 1;
  const long long total = sum * a.Hkv;
  if (total == 0) return;
  // at least kPairCost + kMinBlocks, but no more than the mean pair: short ones have
  // a CTA each
  const long long mean = (sum + active - 1) / active;
  long long run = (total + ctas - 1) / ctas;
  const long long least = mean < kPairCost + kMinBlocks ? mean : kPairCost + kMinBlocks;
  if (run < least) run = least;
  const long long start = run * blockIdx.x;
  if (start >= total) return;
  const long long end = start + run < total ? start + run : total;
  // the sequence in which it starts, and that one's first block
  __syncthreads();
  long long base = 0;
  for (int b0 = 0; b0 < a.B && base <= start; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const int w = b0 == 0 ? w0 : static_cast<int>(share(b));
    long long incl = static_cast<long long>(w) * a.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    long long before = base;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += s_sum[i];
      base += s_sum[i];
    }
    const long long first = before + incl - static_cast<long long>(w) * a.Hkv;
    if (start >= first && start < before + incl) {
      s_b = b;
      s_start = first;
    }
    __syncthreads();
  }
  int b = s_b;
  long long seq0 = s_start;                // the run's position of sequence b's first block
  long long at = start;

  uint8_t* wring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_lo = smem_u32(wring) + 16 * chunk_slot(lane);
  const uint32_t ring_hi = smem_u32(wring) + 16 * chunk_slot(32 + lane);
  const uint32_t ring_sc = smem_u32(wring) + 2048 + 16 * lane;
  const uint8_t* k_lane = a.kc + 16 * lane;
  const uint8_t* v_lane = a.vc + 16 * lane;
  const uint8_t* s_lane = reinterpret_cast<const uint8_t*>(a.sc) + 16 * (lane & 7);
  const int ppb = a.page >> 4, g = a.g;
  const float scale2 = a.scale * 1.4426950408889634f;   // scores in log2 units

  while (at < end) {
    // --- the next pair: KV head hk of sequence b, and its blocks [c0, c1) ---
    const int nblk = blocks_of(a, b, kRows), weight = weight_of(nblk);
    if (at >= seq0 + static_cast<long long>(weight) * a.Hkv) {
      seq0 += static_cast<long long>(weight) * a.Hkv;
      ++b;
      continue;
    }
    const int into = static_cast<int>(at - seq0);
    const int hk = into / weight, from = into - hk * weight;
    const long long left = end - at;
    const int to = weight - from < left ? weight : from + static_cast<int>(left);
    at += to - from;
    const int c0 = from < kPairCost ? 0 : from - kPairCost, c1 = to - kPairCost;
    if (c1 <= 0) continue;      // the run ends before the pair's first block
    const bool whole = c0 == 0 && to == weight;
    const RowRange rr = rows_of(a.q_start, b, a.T);
    const int R = rr.n * g;
    const int seqlen = a.seqlen[b], Lb = clamp_len(seqlen, a.width * a.page);
    const int blk0 = c0 + 2 * warp, blk1 = c1 < nblk ? c1 : nblk;
    const int niter = blk0 < blk1 ? (blk1 - blk0 + 2 * kWarps - 1) / (2 * kWarps) : 0;
    const int* table_row = a.table + static_cast<size_t>(b) * a.width;

    // --- copies: the numbers of 16 iterations' block pairs are looked up at a
    // time, one block a lane; each copy instruction moves 512 contiguous bytes ---
    int window = -1;
    auto issue = [&](int it) {
      if (it < niter) {
        if ((it & 15) == 0) {
          const int blk = blk0 + (it + (lane >> 1)) * (2 * kWarps) + (lane & 1);
          window = blk < blk1 ? pool_block(table_row, blk, ppb, a.pages, a.Hkv, hk) : -1;
        }
        const uint32_t stage = (it & (kStages - 1)) * kStageBytes;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int blk = __shfl_sync(0xffffffffu, window, 2 * (it & 15) + i);
          if (blk >= 0) {
            const size_t off = static_cast<size_t>(static_cast<uint32_t>(blk)) * 1024u;
            const uint32_t lo = ring_lo + stage + i * kBlockBytes;
            const uint32_t hi = ring_hi + stage + i * kBlockBytes;
            cp_async16(lo, k_lane + off);
            cp_async16(hi, k_lane + off + 512);
            cp_async16(lo + 1024, v_lane + off);
            cp_async16(hi + 1024, v_lane + off + 512);
            if (lane < 8)
              cp_async16(ring_sc + stage + i * kBlockBytes,
                         s_lane + static_cast<size_t>(static_cast<uint32_t>(blk)) * 128u);
          }
        }
      }
      cp_async_commit();   // an empty group past the end keeps the counting uniform
    };
    static_assert((kStages & (kStages - 1)) == 0, "ring index");
#pragma unroll
    for (int it = 0; it < kStages - 1; ++it) issue(it);

    // --- queries as B fragments: column gid is row 4 nt + gid / 2, its high byte
    // (even) or low byte (odd); bytes are dimensions 2 tig + {0, 8, 1, 9} of words
    // 2 ks and 2 ks + 1, as the codes' ---
    uint32_t qb[NT][4][2];
    float qf[NT], qh[NT];    // of row 4 nt + tig: the fixed point's unit and Q, in score units
    int lim[NT];             // tokens it sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 4 * nt + (gid >> 1);
      const bool ok = r < R;
      const int qi = r / g;
      const __half* q = a.Q + static_cast<size_t>(rr.first + (ok ? qi : 0)) * a.ldq +
                        static_cast<size_t>(hk * g + (ok ? r - qi * g : 0)) * kHeadDim + 2 * tig;
      float2 f[4][4];
      float qs = 0.0f, top = 0.0f;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[ks][i] = ok ? __half22float2(*reinterpret_cast<const __half2*>(q + 32 * ks + 8 * i))
                        : make_float2(0.0f, 0.0f);
          qs += f[ks][i].x + f[ks][i].y;
          top = fmaxf(top, fmaxf(fabsf(f[ks][i].x), fabsf(f[ks][i].y)));
        }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        qs += __shfl_xor_sync(0xffffffffu, qs, o);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const float up = top > 0.0f ? kFixed / top : 0.0f;
      auto byte = [&](float v) {
        const int n = __float2int_rn(v * up);
        const int h = (n + 128) >> 8;
        return static_cast<uint32_t>((gid & 1) ? n - 256 * h : h) & 0xffu;
      };
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float2 p = f[ks][2 * w], o = f[ks][2 * w + 1];
          qb[nt][ks][w] = byte(p.x) | byte(o.x) << 8 | byte(p.y) << 16 | byte(o.y) << 24;
        }
      qf[nt] = __shfl_sync(0xffffffffu, top, 8 * tig) * (scale2 / kFixed);
      qh[nt] = __shfl_sync(0xffffffffu, qs, 8 * tig) * scale2;
      const int row = 4 * nt + tig;
      lim[nt] = row < R ? visible(position_of(seqlen, rr.n, row / g), Lb) : 0;
    }
    const int all_see = visible(position_of(seqlen, rr.n, 0), Lb);

    float acc[NT][8][4];     // dimensions 16 mt + gid and + 8, the weights' high and low parts
    float mrun[NT], lsum[NT], osum[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < 8; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[nt][mt][k] = 0.0f;
      mrun[nt] = -INFINITY;
      lsum[nt] = osum[nt] = 0.0f;
    }

    uint32_t absent = 0;    // of 16 iterations: the blocks whose page is not in the pool
    for (int it = 0; it < niter; ++it) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      // (the copies run less than 16 iterations ahead: at a multiple of 16 the
      // window is still the one of this iteration)
      if ((it & 15) == 0) absent = __ballot_sync(0xffffffffu, window < 0);
      issue(it + kStages - 1);
      const int blk = blk0 + it * (2 * kWarps);
      const uint32_t gone = (absent >> (2 * (it & 15))) & 3u;
      const uint8_t* stage = wring + (it & (kStages - 1)) * kStageBytes;

      auto step = [&](auto masked) {
        constexpr bool kMasked = decltype(masked)::value;
        // scores of tokens gid and gid + 8 of block i with row 4 nt + tig, in units of
        // the fixed point
        float s[2][NT][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* kp = stage + i * kBlockBytes;
          const uint4 k0 = *reinterpret_cast<const uint4*>(kp + 16 * chunk_slot(2 * lane));
          const uint4 k1 = *reinterpret_cast<const uint4*>(kp + 16 * chunk_slot(2 * lane + 1));
          const uint32_t wk[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
          int d[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) d[nt][k] = 0;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t a0 = wk[2 * ks] & 0x0f0f0f0fu, a1 = (wk[2 * ks] >> 4) & 0x0f0f0f0fu;
            const uint32_t a2 = wk[2 * ks + 1] & 0x0f0f0f0fu;
            const uint32_t a3 = (wk[2 * ks + 1] >> 4) & 0x0f0f0f0fu;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma_u8s8(d[nt], a0, a1, a2, a3, qb[nt][ks][0], qb[nt][ks][1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            s[i][nt][0] = __int2float_rn(256 * d[nt][0] + d[nt][1]);
            s[i][nt][1] = __int2float_rn(256 * d[nt][2] + d[nt][3]);
          }
        }
        float skt[2][2], mkt[2][2], svt[2][2], mvt[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint2 sq = *reinterpret_cast<const uint2*>(stage + i * kBlockBytes + 2048 +
                                                             64 * r + 8 * gid);
            const float2 k2 = __half22float2(*reinterpret_cast<const __half2*>(&sq.x));
            const float2 v2 = __half22float2(*reinterpret_cast<const __half2*>(&sq.y));
            skt[i][r] = k2.x;
            mkt[i][r] = k2.y;
            svt[i][r] = v2.x;
            mvt[i][r] = fmaf(8.0f, v2.x, v2.y);
          }
        auto hidden = [&](int i, int r, int nt) {
          return kMasked && ((blk + i) * 16 + gid + 8 * r >= lim[nt] || ((gone >> i) & 1u));
        };
        const float limit =
            kWeightTop - log2_scale(fmaxf(fmaxf(fabsf(svt[0][0]), fabsf(svt[0][1])),
                                          fmaxf(fabsf(svt[1][0]), fabsf(svt[1][1]))));
        bool raise = false;
        float x[2][NT][2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              // relative to the reference (-inf at first: the sum is then no number
              // below the threshold)
              float v = fmaf(skt[i][r] * qf[nt], s[i][nt][r], fmaf(mkt[i][r], qh[nt], -mrun[nt]));
              if (hidden(i, r, nt)) v = -INFINITY;
              x[i][nt][r] = v;
              raise |= !(v <= limit);
            }
        if (__any_sync(0xffffffffu, raise)) {
          float ls[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) ls[i][r] = log2_scale(svt[i][r]);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float y[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                y[i][r] = fmaf(skt[i][r] * qf[nt], s[i][nt][r], mkt[i][r] * qh[nt]);
                if (hidden(i, r, nt)) y[i][r] = -INFINITY;
              }
            // the largest weight's exponent, and the reference that it asks for
            float top = fmaxf(fmaxf(y[0][0] + ls[0][0], y[0][1] + ls[0][1]),
                              fmaxf(y[1][0] + ls[1][0], y[1][1] + ls[1][1]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = top - kWeightTop > mrun[nt] ? top - kWeightSet : mrun[nt];
            const float al = top == -INFINITY ? 1.0f : fast_exp2(mrun[nt] - top);
            mrun[nt] = top;
            lsum[nt] *= al;
            osum[nt] *= al;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
              for (int k = 0; k < 4; ++k) acc[nt][mt][k] *= al;
            const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              x[i][nt][0] = y[i][0] - ref;
              x[i][nt][1] = y[i][1] - ref;
            }
          }
        }
        uint32_t wb[2][NT][2];     // W^T as B fragments: k = tokens of block i
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float p = fast_exp2(x[i][nt][r]);
              lsum[nt] += p;
              // (a hidden token's scales may never have been written: its terms are
              // left out, not multiplied by 0)
              const bool in = !kMasked || x[i][nt][r] != -INFINITY;
              const float w = in ? p * svt[i][r] : 0.0f;
              if (in) osum[nt] = fmaf(p, mvt[i][r], osum[nt]);
              const float high = __half2float(__float2half_rn(w));
              wb[i][nt][r] = transpose8x8(pack_h2(high, w - high));
            }
        // O^T += (C_V - 8)^T W^T, dimensions 16 mt .. from word mt
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* vp = stage + i * kBlockBytes + 1024;
          const uint4 v0 = *reinterpret_cast<const uint4*>(vp + 16 * chunk_slot(2 * lane));
          const uint4 v1 = *reinterpret_cast<const uint4*>(vp + 16 * chunk_slot(2 * lane + 1));
          const uint32_t wv[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            uint32_t f[4];
            v_frag(wv[mt], f);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816(acc[nt][mt], f, wb[i][nt][0], wb[i][nt][1]);
          }
        }
      };
      if ((blk + 2) * 16 <= all_see && gone == 0u) step(std::false_type{});
      else step(std::true_type{});
      __syncwarp();           // every lane has read the stage before it is copied into again
    }
    cp_async_wait<0>();
    __syncthreads();   // the ring becomes the merge area

    // per warp and row: reference, sum, 128 outputs
    float* mrg = reinterpret_cast<float*>(smem);     // [warp][kRows][kPartFloats]
    static_assert(sizeof(float) * kRows * kPartFloats <= kStages * kStageBytes, "merge area");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float l = lsum[nt], o = osum[nt];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, d);
        o += __shfl_xor_sync(0xffffffffu, o, d);
      }
      // (a value that is not finite shows in o, whose finite terms cannot overflow: the row is NaN,
      // also where another warp's reference would leave this one's sums out)
      if (!isfinite(o)) l = NAN;
      float* row = mrg + (warp * kRows + 4 * nt + tig) * kPartFloats;
      if (gid == 0) {
        row[0] = part_reference(l, mrun[nt]);
        row[1] = l;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        row[4 + 16 * mt + gid] = acc[nt][mt][0] + acc[nt][mt][1] + o;
        row[4 + 16 * mt + gid + 8] = acc[nt][mt][2] + acc[nt][mt][3] + o;
      }
    }
    __syncthreads();
    if (threadIdx.x == 0 && c0 == 0 && a.meta != nullptr) {
      // the CTAs that hold the pair's first and last block
      const long long last = seq0 + static_cast<long long>(hk + 1) * weight - 1;
      a.meta[b * a.Hkv + hk] = make_int2(static_cast<int>(blockIdx.x), static_cast<int>(last / run));
    }
    // a warp a row at a time, four dimensions a lane
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 4 * nt + warp;
      if (r >= R) continue;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mrg[(w * kRows + r) * kPartFloats]);
      float den = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* row = mrg + (w * kRows + r) * kPartFloats;
        const float f = row[0] == -INFINITY ? 0.0f : fast_exp2(row[0] - M);
        if (f == 0.0f) continue;
        den += f * row[1];
        const float4 o = *reinterpret_cast<const float4*>(row + 4 + 4 * lane);
        v.x += f * o.x;
        v.y += f * o.y;
        v.z += f * o.z;
        v.w += f * o.w;
      }
      if (whole) {
        // (v is 0 where the row saw no token)
        const int qi = r / g;
        store_row4(a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + hk * g + (r - qi * g)) *
                               kHeadDim + 4 * lane, v, den == 0.0f ? 0.0f : __frcp_rn(den));
      } else {
        float* part = a.parts + (static_cast<size_t>(2 * blockIdx.x + (c0 == 0 ? 1 : 0)) * kRows +
                                 r) * kPartFloats;
        if (lane == 0) {
          part[0] = part_reference(den, M);
          part[1] = den;
        }
        *reinterpret_cast<float4*>(part + 4 + 4 * lane) = v;
      }
    }
    __syncthreads();   // the merge area becomes the ring again
  }
}

// A list of units where no decode kernel runs.
__global__ void __launch_bounds__(kThreads) prompt_plan_kernel(const PagedArgs a, const PromptPlan pp) {
  __shared__ __align__(16) uint8_t scratch[kPlanScratch];
  grid_dependency_wait();
  grid_launch_dependents();
  list_prompt_units<kThreads>(a, pp, scratch);
}

// Rows of a split slot from their partial results: kCombineRows rows a CTA (number `cta`),
// a warp a row at a time.
constexpr int kCombineRows = 32;
__device__ __forceinline__ void merge_slot(const PagedArgs& a, const PromptPlan& pp,
                                           const float* parts, int cta) {
  constexpr int kParts = kSlotRows / kCombineRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = cta / kParts;
  const int slot = pair / a.Hkv, hk = pair - slot * a.Hkv;
  const int2 mt = pp.meta[pair];
  if (mt.y <= 1) return;                   // no work, or not split
  int b = 0, row0 = 0;
  slot_steps(a, slot, pp.min_rows, a.q_start, b, row0);
  const RowRange rr = rows_of(a.q_start, b, a.T);
  for (int i = warp; i < kCombineRows; i += 8) {
    const int rs = (cta - pair * kParts) * kCombineRows + i;
    const int r = row0 + rs;
    if (r >= rr.n * a.g) return;
    const float* base = parts + (static_cast<size_t>(mt.x) * kSlotRows + rs) * kPartFloats;
    const size_t step = static_cast<size_t>(kSlotRows) * kPartFloats;
    float M = -INFINITY, den = 0.0f;
    float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int p0 = 0; p0 < mt.y; p0 += 4) {     // four parts at a time, loaded together
      float m[4], l[4];
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* pp = base + (p0 + i < mt.y ? p0 + i : p0) * step;
        m[i] = p0 + i < mt.y ? pp[0] : -INFINITY;
        l[i] = pp[1];
        v[i] = *reinterpret_cast<const float4*>(pp + 4 + 4 * lane);
      }
      const float top = fmaxf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), M);
      const float al = M == -INFINITY ? 0.0f : fast_exp2(M - top);
      M = top;
      den *= al;
      num.x *= al;
      num.y *= al;
      num.z *= al;
      num.w *= al;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float f = m[i] == -INFINITY ? 0.0f : fast_exp2(m[i] - top);
        if (f == 0.0f) continue;
        den += f * l[i];
        num.x += f * v[i].x;
        num.y += f * v[i].y;
        num.z += f * v[i].z;
        num.w += f * v[i].w;
      }
    }
    const int qi = r / a.g;
    store_row4(a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + hk * a.g + (r - qi * a.g)) *
                           kHeadDim + 4 * lane, num, den == 0.0f ? 0.0f : __frcp_rn(den));
  }
}

// The merge: CTAs up to `decode_ctas` take rows of the decode kernel's split pairs, W
// warps a row (a warp every W-th part, a lane four dimensions), the others rows of the
// prompt kernel's split slots.
template <int W>
__global__ void __launch_bounds__(256)
paged_combine_kernel(const PagedArgs a, int rows, int stride, int decode_ctas, const PromptPlan pp,
                     const float* prompt_parts) {
  __shared__ float4 red_num[8][32];
  __shared__ float2 red_md[8];
  grid_dependency_wait();
  grid_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= decode_ctas) {
    merge_slot(a, pp, prompt_parts, blockIdx.x - decode_ctas);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % W;
  const long long x = static_cast<long long>(blockIdx.x) * (8 / W) + warp / W;
  const int pair = static_cast<int>(x / rows), r = static_cast<int>(x - static_cast<long long>(pair) * rows);
  int n = 0;
  int2 mt = make_int2(0, 0);
  RowRange rr{0, 0};
  int b = 0, hk = 0;
  if (pair < a.B * a.Hkv) {
    b = pair / a.Hkv;
    hk = pair - b * a.Hkv;
    if (blocks_of(a, b, stride) >= 0) {
      rr = rows_of(a.q_start, b, a.T);
      if (r < rr.n * a.g) {
        mt = a.meta[pair];
        n = mt.y > mt.x ? mt.y - mt.x + 1 : 0;   // CTAs that hold a part of it
      }
    }
  }
  // the first part is at its CTA's end (place 2 x + 1), the others at their CTAs'
  // beginnings (places 2 (x + p))
  const float* base = a.parts + (static_cast<size_t>(2 * mt.x) * stride + r) * kPartFloats;
  const size_t step = static_cast<size_t>(stride) * kPartFloats;
  auto part = [&](int p) { return base + (p == 0 ? step : 2 * p * step); };
  float M = -INFINITY, den = 0.0f;
  float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p = lane; p < n; p += 32) M = fmaxf(M, part(p)[0]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll 4
  for (int p = sub; p < n; p += W) {
    const float* pp = part(p);
    const float m = pp[0];
    const float f = m == -INFINITY ? 0.0f : fast_exp2(m - M);
    const float4 v = *reinterpret_cast<const float4*>(pp + 4 + 4 * lane);
    den += f * pp[1];
    num.x += f * v.x;
    num.y += f * v.y;
    num.z += f * v.z;
    num.w += f * v.w;
  }
  if constexpr (W > 1) {
    red_num[warp][lane] = num;
    if (lane == 0) red_md[warp] = make_float2(M, den);
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float4 v = red_num[warp + w][lane];
      num.x += v.x;
      num.y += v.y;
      num.z += v.z;
      num.w += v.w;
      den += red_md[warp + w].y;
    }
  }
  if (n == 0) return;
  const int qi = r / a.g;
  store_row4(a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + hk * a.g + (r - qi * a.g)) *
                         kHeadDim + 4 * lane, num, den == 0.0f ? 0.0f : __frcp_rn(den));
}

template <int NT>
int launch_decode(const PagedArgs& a, const PagedPlan& p, const PromptPlan& pp, cudaStream_t s) {
  constexpr size_t smem = static_cast<size_t>(kWarps) * kStages * kStageBytes;
  static std::atomic<unsigned long long> ready{0};
  if (int st = opt_in_smem(reinterpret_cast<const void*>(paged_decode_kernel<NT>), smem, ready))
    return st;
  return launch_dependent(paged_decode_kernel<NT>,
                          dim3(static_cast<unsigned>(p.grid + (pp.units ? 1 : 0))), kThreads, smem,
                          s, a, p.grid, pp);
}

int launch_combine(const PagedArgs& a, const PagedPlan& p, const PromptPlan& pp,
                   const float* prompt_parts, cudaStream_t s) {
  const int rows = a.max_q * a.g < 4 * p.nt ? a.max_q * a.g : 4 * p.nt;
  const long long all = p.combine ? static_cast<long long>(a.B) * a.Hkv * rows : 0;
  const long long prompt = p.prompt && p.prompt_combine
                               ? static_cast<long long>(p.tiles) * a.Hkv * (kSlotRows / kCombineRows)
                               : 0;
  if (all + prompt == 0) return QOQ_OK;
  // few rows have many parts each: eight warps a row
  if (all <= 512)
    return launch_dependent(paged_combine_kernel<8>, dim3(static_cast<unsigned>(all + prompt)), 256,
                            0, s, a, rows, 4 * p.nt, static_cast<int>(all), pp, prompt_parts);
  const long long ctas = (all + 7) / 8;
  return launch_dependent(paged_combine_kernel<1>, dim3(static_cast<unsigned>(ctas + prompt)), 256, 0,
                          s, a, rows, 4 * p.nt, static_cast<int>(ctas), pp, prompt_parts);
}

}  // namespace

PagedPlan paged_plan(int T, int B, int Hq, int Hkv, int width, int page, int max_q) {
  PagedPlan p = {};
  const int g = Hq / Hkv;
  const long long pairs = static_cast<long long>(B) * Hkv;
  const long long most = static_cast<long long>(max_q) * g;     // rows of a sequence
  // tiles of four rows: for all sequences, or, where there are longer ones (prompt
  // chunks), for those with one query token
  p.nt = most <= 4 ? 1 : (most <= 8 ? 2 : (most <= 16 ? 4 : (g <= 4 ? 1 : (g <= 8 ? 2 : (g <= 16 ? 4 : 0)))));
  p.prompt = most > 4 * p.nt;
  const long long blocks = (static_cast<long long>(width) * page + 15) / 16;
  if (p.nt) {
    // a CTA for each that is resident, but no more than there can be blocks
    const int resident = resident_ctas(p.nt) * sm_count();
    p.grid = static_cast<int>(pairs * blocks < resident ? pairs * blocks : resident);
    p.combine = p.grid > 1;
    if (p.combine) {
      p.meta_off = p.take(static_cast<size_t>(pairs) * sizeof(int2));
      p.parts_off = p.take(static_cast<size_t>(2 * p.grid) * 4 * p.nt * kPartFloats * sizeof(float));
    }
  }
  if (p.prompt) plan_prompt(p, T, B, Hq, Hkv, width, page);
  return p;
}

}  // namespace qoq

using namespace qoq;

namespace {

int check_paged_attention(int T, int Hq, int Hkv, int d, int B, int width, int pages, int page,
                          int max_q) {
  if (Hq <= 0 || max_q <= 0) return QOQ_ERR_INVALID_ARG;
  if (int st = check_paged_shape(pages, Hkv, page, d)) return st;
  if (int st = check_batch(T, B, width, page)) return st;
  if (Hq % Hkv != 0) return QOQ_ERR_INVALID_ARG;
  if (Hq > 65535) return QOQ_ERR_UNSUPPORTED;
  // numbers of work units and of rows are 32-bit
  if (static_cast<long long>(B) * Hkv > (1 << 22) || static_cast<long long>(T) * Hq > (1LL << 30))
    return QOQ_ERR_UNSUPPORTED;
  // a sequence's place among its KV heads' blocks is 32-bit, the batch's sum of blocks has
  // 40 bits (a table may name a page many times, so the pool's size bounds neither)
  const long long blocks = static_cast<long long>(width) * (page / 16) + kPairCost + 1;
  if (blocks * Hkv > 0x7fffffffLL || blocks * B > (1LL << 40) - 1) return QOQ_ERR_UNSUPPORTED;
  return QOQ_OK;
}

}  // namespace

extern "C" size_t qoq_kv4_paged_attention_workspace_bytes(int T, int Hq, int Hkv, int d, int B,
                                                          int width, int page, int max_q) {
  if (check_paged_attention(T, Hq, Hkv, d, B, width, 1, page, max_q) || T == 0 || B == 0) return 0;
  return paged_plan(T, B, Hq, Hkv, width, page, max_q < T ? max_q : T).bytes;
}

extern "C" int qoq_kv4_paged_attention(const void* Q, size_t ldq, int T, int Hq, int Hkv, int d,
                                       const uint8_t* k_codes, const uint8_t* v_codes,
                                       const void* scales, const int* q_start, const int* seqlen,
                                       int B, const int* block_table, int width, int pages,
                                       int page, int max_q, float scale, void* out, void* ws,
                                       size_t ws_bytes, void* stream) {
  if (int st = check_paged_attention(T, Hq, Hkv, d, B, width, pages, page, max_q)) return st;
  if (ldq < static_cast<size_t>(Hq) * kHeadDim || ldq % 8 != 0) return QOQ_ERR_INVALID_ARG;
  if (!(fabsf(scale) <= 3.0e38f)) return QOQ_ERR_INVALID_ARG;      // infinite or NaN
  if (T == 0 || B == 0) return QOQ_OK;
  if (!Q || !k_codes || !v_codes || !scales || !q_start || !seqlen || !block_table || !out)
    return QOQ_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned16(scales) ||
      !aligned16(out) || !aligned4(q_start) || !aligned4(seqlen) || !aligned4(block_table))
    return QOQ_ERR_INVALID_ARG;
  if (max_q > T) max_q = T;
  const PagedPlan p = paged_plan(T, B, Hq, Hkv, width, page, max_q);
  if (p.bytes > 0 && (ws == nullptr || ws_bytes < p.bytes || !aligned16(ws)))
    return QOQ_ERR_WORKSPACE;
  if (int st = check_device()) return st;
  PagedArgs a;
  a.Q = static_cast<const __half*>(Q);
  a.ldq = ldq;
  a.kc = k_codes;
  a.vc = v_codes;
  a.sc = static_cast<const __half*>(scales);
  a.q_start = q_start;
  a.seqlen = seqlen;
  a.table = block_table;
  a.T = T; a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.g = Hq / Hkv;
  a.width = width; a.pages = pages; a.page = page; a.max_q = max_q;
  a.scale = scale;
  a.out = static_cast<__half*>(out);
  char* w = static_cast<char*>(ws);
  cudaStream_t s = as_stream(stream);
  PromptPlan pp = {};
  if (p.prompt) {
    pp.units = reinterpret_cast<PromptUnit*>(w + p.prompt_units_off);
    pp.meta = p.prompt_combine ? reinterpret_cast<int2*>(w + p.prompt_meta_off) : nullptr;
    pp.grid = p.prompt_grid;
    pp.tiles = p.tiles;
    pp.target = p.prompt_target;
    pp.min_rows = 4 * p.nt + 1;
  }
  a.meta = p.combine ? reinterpret_cast<int2*>(w + p.meta_off) : nullptr;
  a.parts = p.combine ? reinterpret_cast<float*>(w + p.parts_off) : nullptr;
  int st = QOQ_OK;
  if (p.nt == 1) st = launch_decode<1>(a, p, pp, s);
  else if (p.nt == 2) st = launch_decode<2>(a, p, pp, s);
  else if (p.nt == 4) st = launch_decode<4>(a, p, pp, s);
  else st = launch_dependent(prompt_plan_kernel, dim3(1), kThreads, 0, s, a, pp);
  if (st) return st;
  float* prompt_parts = nullptr;
  if (p.prompt) {
    PagedArgs b = a;
    prompt_parts = p.prompt_combine ? reinterpret_cast<float*>(w + p.prompt_parts_off) : nullptr;
    b.parts = prompt_parts;
    if (int e = launch_paged_prompt(b, p, pp.units, s)) return e;
  }
  return launch_combine(a, p, pp, prompt_parts, s);
}
