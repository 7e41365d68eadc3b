// Attention over a paged 4-bit KV cache for the sequences with more rows than
// the decode kernel takes: chunks of a prompt, on the tcgen05 tensor cores.
//
// Rows.  The n query tokens of a sequence times the g heads of a KV head are the
// rows r = i g + h of one problem; a CTA takes 256 consecutive ones (a slot) as
// two tiles of 128, and walks the tokens that they see, 128 at a time:
//     S = Q (c_K - 8)^T        x_t = s_K S_t + (m_K + 8 s_K) Q_sum
//     W = fp16(2^(x - ref) s_V)  O += W (c_V - 8),  o_off += p (m_V + 8 s_V).
// The codes enter both products as c - 8, exact FP16 numbers, so the rounding of
// W (2^-11 relative) is the only one besides the output's: rounding k^ and v^
// to FP16 instead would save the two scale products a score and cost two more
// errors of the output's own size.  Centred codes keep what the rounding of W
// touches as small as v^ about its vector's middle.  The reference (qoq_attn.cuh) keeps a
// row's largest W between 2^10 and 2^15.9; a half step is tested by its largest score and
// its largest value scale, and only where those could pass 2^15.9 by each token's.
//
// Warps.  Warpgroups 0 and 1 do the softmax of one tile each; warpgroup 2 turns codes
// into FP16 tiles; a thread of warpgroup 3 for each tile issues its MMAs (one thread for
// both had no time left: an issue takes it some 55 cycles, a commit 200).
// Tensor memory (512 columns) holds S and O of both tiles; W overwrites the scores it
// came from.  A step's softmax goes by halves of 64 tokens, so that O += W V of the
// first half runs beside the second half's softmax, and one tile's products beside the
// other's softmax.
//
// Layouts.  The cache's nibble order is the register layout of warp MMAs, so a
// lane of the producer holds, for one token, dimensions 16 w + 2 tig + {0, 1, 8,
// 9}, and for one dimension four tokens of a block.  Instead of shuffling, the
// tiles take that order: the K tile's k index is dimension position
// 32 tig + 4 w + 2 j1 + e (Q is stored the same way), and the columns of S, which
// are the k index of W V, are token position 8 tig + 4 block + 2 j1 + e of each 32
// (the rows of the K tile are stored at them).  Every store is 16 bytes.
//
// Splits.  One CTA of the kernel ahead looks the lengths over and lists the units of
// work: long sequences with few rows are split so that no CTA is left with a long one,
// and a last kernel merges.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>

#include <atomic>

#include "qoq.h"
#include "qoq_attn.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"
#include "qoq_kv4.cuh"
#include "qoq_paged.h"
#include "qoq_prompt_plan.cuh"

namespace qoq {

namespace {

// This file's part of the device error word (device code of different files
// shares no variables).
__device__ unsigned int g_prompt_error = 0;

constexpr int kThreads = 512;
constexpr int kTile = kStepTokens;              // rows of a tile, tokens of a step

// Shared memory: Q 2 tiles x 2 halves of 64 dimensions x [128 rows][128 bytes],
// K and V twice each, 2 halves x [128][128 bytes] (128-byte swizzle).
constexpr uint32_t kHalf = 16384;
constexpr uint32_t kQ = 0, kK = 4 * kHalf, kV = kK + 4 * kHalf;
constexpr uint32_t kSmemBytes = kV + 4 * kHalf + 1024;   // + alignment

struct Bars {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], c_full[2];
  uint64_t s_full[2][2], p_full[2][2];     // [tile][half step]
  uint64_t o_full;
};

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor: FP16 A and B, K-major, FP32 accumulator, 128 x n.
constexpr uint32_t idesc_f16(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(kTile >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]),
        "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]),
        "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
// Tensor memory by 16 lanes: thread (g, t) = (lane / 4, lane mod 4) of the warp gets, of
// every 8 columns, columns 2 t and 2 t + 1 of rows g (registers 4 k, 4 k + 1) and g + 8
// (4 k + 2, 4 k + 3).
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, float (&r)[32]) {
  uint32_t (&u)[32] = reinterpret_cast<uint32_t (&)[32]>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
        "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
        "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&r)[16]) {
  uint32_t (&u)[16] = reinterpret_cast<uint32_t (&)[16]>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
      "}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x32(uint32_t taddr, const float (&r)[16]) {
  const uint32_t (&u)[16] = reinterpret_cast<const uint32_t (&)[16]>(r);
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
      "};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
      "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
// 32 columns of 32 bits: of every 4 columns, column t of rows g (register 2 k) and
// g + 8 (2 k + 1).
__device__ __forceinline__ void tmem_st_16x32h(uint32_t taddr, const uint32_t (&u)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {"
      "%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16"
      "};" ::"r"(taddr),
      "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]),
      "r"(u[8]), "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15])
      : "memory");
}
// After the wait that completes loads: names a load's registers, so that no use of them
// moves above it.
template <int N>
__device__ __forceinline__ void keep(float (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}

// Two FP32 operations an instruction.
union F2 {
  float f[2];
  unsigned long long u;
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.u) : "l"(a.u), "l"(b.u), "l"(c.u));
  return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.u) : "l"(a.u), "l"(b.u));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ F2 pair2(float a, float b) {
  F2 d;
  d.f[0] = a;
  d.f[1] = b;
  return d;
}

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Column position of token 0 .. 31 (of its 32) in S.
__device__ __forceinline__ int column_of(int tok) {
  return 8 * ((tok & 7) >> 1) + 4 * (tok >> 4) + 2 * ((tok >> 3) & 1) + (tok & 1);
}

// Byte offset of 16-byte chunk `chunk` (0..15) of row `row` in a [2 halves][128
// rows][128 bytes] tile with the 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(int row, int chunk) {
  return (chunk >> 3) * kHalf + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// Nibbles n and n + 4 (counted from the lowest) of a word as FP16 numbers c - 8, n = 0, 1,
// 2 and 3: 0x6400 | c is 1024 + c, 0x5400 | 16 c is 64 + c, so one shift serves all four.
__device__ __forceinline__ void centred(uint32_t word, uint32_t (&d)[4]) {
  auto less = [](uint32_t n, float k) {
    const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&n), __float2half2_rn(k));
    return *reinterpret_cast<const uint32_t*>(&h);
  };
  const uint32_t high = word >> 8;
  d[0] = less(and_or(word, 0x000f000fu, 0x64006400u), 1032.0f);
  d[1] = less(and_or(word, 0x00f000f0u, 0x54005400u), 72.0f);
  d[2] = less(and_or(high, 0x000f000fu, 0x64006400u), 1032.0f);
  d[3] = less(and_or(high, 0x00f000f0u, 0x54005400u), 72.0f);
}

// Measured: a 4096-token prompt (32 / 8 heads) 219 to 222 us in all, 620 TFLOP/s of the two
// products over the pairs that the mask leaves (2.5% less time where the reference followed the
// scores alone);
// it is bound by the softmax warps, two on a scheduler: at 44% of the issue slots it is their
// chains' latency (read, scale, compare, exponential, pack, store, announce) that two warps do
// not cover.  The products would take half of a step, the exponentials 2/5.
__global__ void __launch_bounds__(kThreads, 1)
paged_prompt_kernel(const PagedArgs a, const PromptUnit* units) {
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_abort;
  __shared__ uint32_t s_absent[2][4];       // per step: bit per 16-token block and producer warp
  __shared__ float2 s_limit[2][2];          // per half step: what scores of its 2 x 32 tokens may
                                            // lie above the reference
  // The first token so far of each producer warp whose value has a scale or offset that is not
  // finite.  Such scales count as zero (a hidden token's weight 0 times them would be NaN), and
  // rows that see the token, which are the ones whose limit lies above it, become NaN at the end.
  __shared__ int s_odd[4];
  // scales of two steps, per column pair: (s_K, s_K', m_K, m_K') and (s_V, s_V', m_V, m_V')
  __shared__ float4 s_scale[2][2][kTile / 2];
  __shared__ float s_row[3][kSlotRows];     // Q sums; then l, offset sum and reference
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(smem);
  grid_dependency_wait();
  grid_launch_dependents();
  const PromptUnit u = units[blockIdx.x];
  if (u.b < 0) return;

  const RowRange rr = rows_of(a.q_start, u.b, a.T);
  const int g = a.g, R = rr.n * g;
  const int seqlen = a.seqlen[u.b], len = clamp_len(seqlen, a.width * a.page);
  const bool two = u.row0 + kTile < R;      // the second tile has rows
  const int steps = u.step1 - u.step0;
  if (steps <= 0) {
    // Rows that see no token (never split: a split has a step).  They are written from
    // here: below, rows leave by way of the memory that held Q, and only the products'
    // end tells that nobody writes or reads Q any more.
    const int rows = R - u.row0 < kSlotRows ? R - u.row0 : kSlotRows;
    for (int i = tid; i < rows * (kHeadDim / 8); i += kThreads) {
      const int r = u.row0 + i / (kHeadDim / 8), qi = r / g;
      __half* dst = a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + u.hk * g + (r - qi * g)) *
                                kHeadDim + 8 * (i & (kHeadDim / 8 - 1));
      *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  auto bar = [&](uint64_t& x) { return smem_u32(&x); };

  if (tid == 0) {
    s_abort = 0u;
    mbar_init(bar(bars.q_full), 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars.k_full[i]), 4);
      mbar_init(bar(bars.v_full[i]), 4);
      mbar_init(bar(bars.c_full[i]), 4);
      mbar_init(bar(bars.k_empty[i]), two ? 2 : 1);
      mbar_init(bar(bars.v_empty[i]), two ? 2 : 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(bar(bars.s_full[i][h]), 1);
        mbar_init(bar(bars.p_full[i][h]), 4);
      }
    }
    mbar_init(bar(bars.o_full), two ? 2 : 1);
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_u32(&s_tmem), 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s_tmem;
  auto wait = [&](uint64_t& x, uint32_t parity, uint32_t err) {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(&x), parity, &s_abort, &g_prompt_error,
                                             err)) != 0;
  };
  // (one arrival a warp: 128 in a row take longer than what they announce)
  auto arrive = [&](uint64_t& x) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&x));
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    regs_inc<168>();
    const int x = warp >> 2;         // tile
    // Q, four lanes a row and 8 rows a turn: lane part k has 32 dimensions, words w = 2k
    // and 2k + 1, whose four bytes (dimensions d, d + 1) at 16 w + 2 tig and
    // 16 w + 8 + 2 tig go to chunk 4 tig + k
    {
      const int k = lane & 3;
      uint4 v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = u.row0 + kTile * x + 32 * (warp & 3) + 8 * i + (lane >> 2), qi = r / g;
        const uint4* q = reinterpret_cast<const uint4*>(
            a.Q + static_cast<size_t>(rr.first + (r < R ? qi : 0)) * a.ldq +
            static_cast<size_t>(u.hk * g + (r < R ? r - qi * g : 0)) * kHeadDim + 32 * k);
#pragma unroll
        for (int c = 0; c < 4; ++c) v[i][c] = r < R ? q[c] : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 32 * (warp & 3) + 8 * i + (lane >> 2);
        const uint32_t d[16] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y,
                                v[i][1].z, v[i][1].w, v[i][2].x, v[i][2].y, v[i][2].z, v[i][2].w,
                                v[i][3].x, v[i][3].y, v[i][3].z, v[i][3].w};
        float qsum = 0.0f;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&d[c]));
          qsum += f.x + f.y;
        }
        qsum += __shfl_xor_sync(0xffffffffu, qsum, 1);
        qsum += __shfl_xor_sync(0xffffffffu, qsum, 2);
#pragma unroll
        for (int tig = 0; tig < 4; ++tig)
          sts16(s0 + kQ + x * 2 * kHalf + tile_at(row, 4 * tig + k),
                make_uint4(d[tig], d[4 + tig], d[8 + tig], d[12 + tig]));
        if (k == 0) s_row[0][kTile * x + row] = qsum;
      }
    }
    fence_proxy_async_smem();
    arrive(bars.q_full);

    // Scores are read 16 lanes at a time: thread (gr, t) has columns 2 t and 2 t + 1 of
    // every 8, of rows gr, gr + 8, gr + 16 and gr + 24 of its warp's 32.  A column's
    // scales then serve four rows: with a row a thread they came to 4096 cycles of
    // shared-memory reads a step, twice the products' time.
    const int gr = lane >> 2, t = lane & 3;
    int lim[4];
    F2 q2[4], ref2[4], l2[4], off2[4];
    bool seen[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ri = 32 * (warp & 3) + 8 * i + gr, rg = u.row0 + kTile * x + ri;
      lim[i] = rg < R ? visible(position_of(seqlen, rr.n, rg / g), len) : 0;
      const float qs = s_row[0][kTile * x + ri];
      q2[i] = pair2(qs, qs);
      ref2[i] = l2[i] = off2[i] = pair2(0.0f, 0.0f);     // ref: minus the reference
      seen[i] = false;
    }
    // the tokens that every row of the warp sees
    const int least = __reduce_min_sync(0xffffffffu, min(min(lim[0], lim[1]), min(lim[2], lim[3])));
    // token of column 8 k + 2 t + e in its step: first_token + 32 (k / 4) + 2 (k mod 4) + e
    const int first_token = 16 * (t >> 1) + 8 * (t & 1);
    const uint32_t t_s = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kTile * x;
    const uint32_t t_o = t_s + 2 * kTile, half16 = 16u << 16;
    bool ok = true;
    if (x == 0 || two) {
      uint32_t absent2 = 0;
      // (unrolled, the half is a constant: 216 -> 209 us at a 4096-token prompt; four times, or the
      // MMA loop too, is slower)
#pragma unroll 2
      for (int hs = 0; hs < 2 * steps; ++hs) {
        const int j = hs >> 1, hf = hs & 1;
        ok = wait(bars.s_full[x][hf], j & 1, kErrEpilogue) &&
             (hf == 1 || wait(bars.c_full[j & 1], (j >> 1) & 1, kErrEpilogue));
        if (!ok) break;
        tc_fence_after_sync();
        if (hf == 0) {
          absent2 = s_absent[j & 1][0] | s_absent[j & 1][1] | s_absent[j & 1][2] | s_absent[j & 1][3];
        }
        const uint32_t t_h = t_s + (kTile / 2) * hf;
        F2 s[4][8];          // row i, columns 8 k + 2 t and + 1
        {
          float r[2][32];    // rows gr and gr + 8, then gr + 16 and gr + 24
          tmem_ld_16x64(t_h, r[0]);
          tmem_ld_16x64(t_h + half16, r[1]);
          tmem_ld_wait();
          keep(r[0]);
          keep(r[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              s[i][k] = pair2(r[i >> 1][4 * k + 2 * (i & 1)], r[i >> 1][4 * k + 2 * (i & 1) + 1]);
        }
        const float4* sk = s_scale[j & 1][0] + 32 * hf + t;
        const float4* sv = s_scale[j & 1][1] + 32 * hf + t;
        // scores less the reference
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 kc = sk[4 * k];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s[i][k] = fma2(s[i][k], pair2(kc.x, kc.y), fma2(q2[i], pair2(kc.z, kc.w), ref2[i]));
        }
        const float2 lim2 = s_limit[j & 1][hf];
        const float limit = fminf(lim2.x, lim2.y);
        // tokens that a row does not see, or in no page
        const int seen_here = (u.step0 + j) * kTile + (kTile / 2) * hf;
        const uint32_t absent = (absent2 >> (4 * hf)) & 15u;
        if (least - seen_here < kTile / 2 || absent != 0u) {        // (the same for the warp)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rel = lim[i] - seen_here - first_token;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const bool gone = (absent >> (2 * (k >> 2) + (t >> 1))) & 1u;
              if (32 * (k >> 2) + 2 * (k & 3) >= rel || gone) s[i][k].f[0] = -INFINITY;
              if (32 * (k >> 2) + 2 * (k & 3) + 1 >= rel || gone) s[i][k].f[1] = -INFINITY;
            }
          }
        }
        bool raise = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
          for (int k = 0; k < 8; k += 2) {
            a0 = max3(a0, s[i][k].f[0], s[i][k].f[1]);
            a1 = max3(a1, s[i][k + 1].f[0], s[i][k + 1].f[1]);
          }
          // raise the reference: past the limit, or at the first token seen (a row's four
          // threads agree on it below, in the few half steps that need it)
          raise |= fmaxf(a0, a1) > (seen[i] ? limit : -INFINITY);
        }
        if (__any_sync(0xffffffffu, raise)) {
          // the largest weights' exponents
          float high[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 vc = sv[4 * k];
            const float l0 = log2_scale(vc.x), l1 = log2_scale(vc.y);
#pragma unroll
            for (int i = 0; i < 4; ++i) high[i] = max3(high[i], s[i][k].f[0] + l0, s[i][k].f[1] + l1);
          }
          float al[4];
          raise = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            high[i] = fmaxf(high[i], __shfl_xor_sync(0xffffffffu, high[i], 1));
            high[i] = fmaxf(high[i], __shfl_xor_sync(0xffffffffu, high[i], 2));
            const bool up_row = high[i] > (seen[i] ? kWeightTop : -INFINITY);
            const float up = up_row ? high[i] - kWeightSet : 0.0f;
            raise |= up_row;
            al[i] = seen[i] ? fast_exp2(-up) : 1.0f;
            seen[i] |= up_row;
            const F2 d2 = pair2(-up, -up), al2 = pair2(al[i], al[i]);
            ref2[i] = add2(ref2[i], d2);
            l2[i] = mul2(l2[i], al2);
            off2[i] = mul2(off2[i], al2);
#pragma unroll
            for (int k = 0; k < 8; ++k) s[i][k] = add2(s[i][k], d2);
          }
          if (hs > 0 && __any_sync(0xffffffffu, raise)) {
            // the last product into O: announced with the scores issued behind it (the one
            // before it came ahead of the scores here)
            ok = wait(bars.s_full[x][1 - hf], (j + hf) & 1, kErrEpilogue);
            if (!ok) break;
            tc_fence_after_sync();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll 1
              for (int c = 0; c < kTile; c += 32) {
                float o[16];
                tmem_ld_16x32(t_o + h * half16 + c, o);
                tmem_ld_wait();
                keep(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= al[2 * h + ((k >> 1) & 1)];
                tmem_st_16x32(t_o + h * half16 + c, o);
              }
            }
          }
        }
        // weights
        uint32_t w[2][16];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 vc = sv[4 * k];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const F2 p = pair2(fast_exp2(s[i][k].f[0]), fast_exp2(s[i][k].f[1]));
            l2[i] = add2(l2[i], p);
            off2[i] = fma2(p, pair2(vc.z, vc.w), off2[i]);
            const F2 d = mul2(p, pair2(vc.x, vc.y));
            w[i >> 1][2 * k + (i & 1)] = pack_h2(d.f[0], d.f[1]);
          }
        }
        tmem_st_16x32h(t_h, w[0]);
        tmem_st_16x32h(t_h + half16, w[1]);
        tmem_st_wait();
        tc_fence_before_sync();
        arrive(bars.p_full[x][hf]);
      }
      // the rows' sums, for the epilogue's row a thread
      const int odd = min(min(s_odd[0], s_odd[1]), min(s_odd[2], s_odd[3]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float li = l2[i].f[0] + l2[i].f[1], oi = off2[i].f[0] + off2[i].f[1];
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          li += __shfl_xor_sync(0xffffffffu, li, d);
          oi += __shfl_xor_sync(0xffffffffu, oi, d);
        }
        // (a query with an infinity has scores of +-inf or NaN: inf - inf in every softmax, also
        // where all of them are -inf, which a hidden token's score is as well)
        if (odd < lim[i] || (lim[i] > 0 && !isfinite(q2[i].f[0]))) li = NAN;
        if (t == 0) {
          const int ri = kTile * x + 32 * (warp & 3) + 8 * i + gr;
          s_row[0][ri] = li;
          s_row[1][ri] = oi;
          s_row[2][ri] = -ref2[i].f[0];
        }
      }
      __syncwarp();        // (a warp reads the rows it wrote)
      const float l = s_row[0][tid], off = s_row[1][tid], mref = s_row[2][tid];
      if (ok) ok = wait(bars.o_full, 0, kErrEpilogue);
      if (ok) {
        tc_fence_after_sync();
        const bool whole = u.whole;
        // (a row that saw no token has l = 0)
        const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
        const int rows0 = u.row0 + kTile * x + 32 * (warp & 3);      // the warp's first row
        const int left = R - rows0 < 32 ? R - rows0 : 32;
        // A row a thread comes out of tensor memory; rows leave by way of the warp's 16 KB
        // of shared memory (the products are done with it), 16 bytes a lane along a row.
        // Chunk c of row r lies at c ^ (r & 7).
        const uint32_t mine = s0 + warp * 16384 + lane * 512;
#pragma unroll 1
        for (int c = 0; c < kTile; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, o);
          tmem_ld_wait();
          keep(o);
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = l == 0.0f ? 0.0f : o[k + i] + off;
            if (whole) {
              sts16(mine + ((((c + k) >> 3) ^ (lane & 7)) << 4),
                    make_uint4(pack_h2(v[0] * inv, v[1] * inv), pack_h2(v[2] * inv, v[3] * inv),
                               pack_h2(v[4] * inv, v[5] * inv), pack_h2(v[6] * inv, v[7] * inv)));
            } else {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                sts16(mine + (((((c + k) >> 2) + i) ^ (lane & 7)) << 4),
                      make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                 __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])));
            }
          }
        }
        __syncwarp();
        const uint32_t from = s0 + warp * 16384;
        if (whole) {
#pragma unroll 4
          for (int i = lane >> 4; i < left; i += 2) {
            const int qi = (rows0 + i) / g, c = lane & 15;
            __half* dst = a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + u.hk * g +
                                   (rows0 + i - qi * g)) * kHeadDim + 8 * c;
            *reinterpret_cast<uint4*>(dst) = lds16(from + i * 512 + ((c ^ (i & 7)) << 4));
          }
        } else {
          float* part = a.parts + (static_cast<size_t>(u.part) * kSlotRows + kTile * x +
                                   32 * (warp & 3)) * kPartFloats;
          if (lane < left) {
            part[lane * kPartFloats] = part_reference(l, mref);
            part[lane * kPartFloats + 1] = l;
          }
#pragma unroll 4
          for (int i = 0; i < left; ++i)
            *reinterpret_cast<uint4*>(part + i * kPartFloats + 4 + 4 * lane) =
                lds16(from + i * 512 + ((lane ^ (i & 7)) << 4));
        }
      }
    }
  } else if (warp < 12) {
    // --------------------------------------------------------------- producer
    regs_dec<96>();
    const int pw = warp - 8, gid = lane >> 2, tig = lane & 3;
    const int nblk = (len + 15) >> 4, ppb = a.page >> 4;
    const int* table_row = a.table + static_cast<size_t>(u.b) * a.width;
    const float scale2 = a.scale * 1.4426950408889634f;
    // of the next step: 32 bytes of K and of V of two blocks, one token's scales
    uint4 k4[2][2], v4[2][2];
    uint2 s4;
    uint32_t gone = 0;
    int first_odd = INT_MAX;
    auto fetch = [&](int step) {
      gone = 0;
      s4 = make_uint2(0u, 0u);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int blk = 8 * step + 2 * pw + i;
        const int at = blk < nblk ? pool_block(table_row, blk, ppb, a.pages, a.Hkv, u.hk) : -1;
        if (at >= 0) {
          // (K: the half of the run that goes to the lane's half of the tile
          // first, so that eight lanes store to eight different 16-byte columns)
          const uint4* kp = reinterpret_cast<const uint4*>(a.kc + static_cast<size_t>(at) * 1024) +
                            2 * lane;
          const uint4* vp = reinterpret_cast<const uint4*>(a.vc + static_cast<size_t>(at) * 1024) +
                            2 * lane;
          k4[i][0] = kp[tig >> 1];
          k4[i][1] = kp[1 - (tig >> 1)];
          v4[i][0] = vp[0];
          v4[i][1] = vp[1];
          if ((lane >> 4) == i)
            s4 = *reinterpret_cast<const uint2*>(a.sc + static_cast<size_t>(at) * 64 +
                                                 4 * (lane & 15));
        } else {
          k4[i][0] = k4[i][1] = v4[i][0] = v4[i][1] = make_uint4(0u, 0u, 0u, 0u);
          if (blk < nblk) gone |= 1u << (2 * pw + i);
        }
      }
    };
    fetch(u.step0);
    for (int j = 0; j < steps; ++j) {
      const int st = j & 1, use = j >> 1;
      if (use > 0 && !wait(bars.k_empty[st], (use - 1) & 1, kErrProducer)) break;
      // K tile: row column_of(token), chunks 4 tig + k of words 2k, 2k + 1
      const uint32_t kt = s0 + kK + st * 2 * kHalf;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 q4 = k4[i][k >> 1];
          const int kk = (k & 1) + 2 * ((k >> 1) ^ (tig >> 1));
          uint32_t c0[4], c1[4];
          centred((k & 1) ? q4.z : q4.x, c0);
          centred((k & 1) ? q4.w : q4.y, c1);
#pragma unroll
          for (int j0 = 0; j0 < 2; ++j0)
            sts16(kt + tile_at(32 * pw + column_of(16 * i + gid + 8 * j0), 4 * tig + kk),
                  make_uint4(c0[j0], c0[j0 + 2], c1[j0], c1[j0 + 2]));
        }
      }
      fence_proxy_async_smem();
      arrive(bars.k_full[st]);

      if (use > 0 && !wait(bars.v_empty[st], (use - 1) & 1, kErrProducer)) break;
      {
        const int tok = (u.step0 + j) * kTile + 32 * pw + lane;
        const float2 fk = __half22float2(*reinterpret_cast<const __half2*>(&s4.x));
        const float2 fv = __half22float2(*reinterpret_cast<const __half2*>(&s4.y));
        // (a slot past the length may hold anything: its scales count as zero)
        const bool in = tok < len, odd = in && !(isfinite(fv.x) && isfinite(fv.y));
        const int c = 32 * pw + column_of(lane);
        float* ks = reinterpret_cast<float*>(&s_scale[st][0][c >> 1]) + (c & 1);
        float* vs = reinterpret_cast<float*>(&s_scale[st][1][c >> 1]) + (c & 1);
        ks[0] = in ? fk.x * scale2 : 0.0f;
        ks[2] = in ? fmaf(8.0f, fk.x, fk.y) * scale2 : 0.0f;
        const float sv = in && !odd ? fv.x : 0.0f;
        vs[0] = sv;
        vs[2] = in && !odd ? fmaf(8.0f, fv.x, fv.y) : 0.0f;
        first_odd = min(first_odd, __reduce_min_sync(0xffffffffu, odd ? tok : INT_MAX));
        const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(sv)));
        if (lane == 0) {
          s_absent[st][pw] = gone;
          s_odd[pw] = first_odd;
          reinterpret_cast<float*>(s_limit[st])[pw] = kWeightTop - log2_scale(__uint_as_float(top));
        }
      }
      arrive(bars.c_full[st]);
      // V tile: row dimension, chunk of tokens 32 pw + 8 tig ..
      const uint32_t vt = s0 + kV + st * 2 * kHalf;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const uint4 a4 = v4[0][w >> 2], b4 = v4[1][w >> 2];
        const uint32_t wa = (w & 3) == 0 ? a4.x : (w & 3) == 1 ? a4.y : (w & 3) == 2 ? a4.z : a4.w;
        const uint32_t wb = (w & 3) == 0 ? b4.x : (w & 3) == 1 ? b4.y : (w & 3) == 2 ? b4.z : b4.w;
        uint32_t ca[4], cb[4];
        centred(wa, ca);
        centred(wb, cb);
#pragma unroll
        for (int j0 = 0; j0 < 2; ++j0)
          sts16(vt + tile_at(16 * w + gid + 8 * j0, 4 * pw + tig),
                make_uint4(ca[j0], ca[j0 + 2], cb[j0], cb[j0 + 2]));
      }
      fence_proxy_async_smem();
      arrive(bars.v_full[st]);
      if (j + 1 < steps) fetch(u.step0 + j + 1);
    }
  } else {
    regs_dec<80>();
    const uint32_t x = warp - 12;          // the tile
    if (lane == 0 && (x == 0 || (x == 1 && two))) {
      // ------------------------------------------------------------------ MMA
      auto pass = [&](uint64_t& b, uint32_t parity) {
        return mbar_wait(smem_u32(&b), parity, &s_abort, &g_prompt_error, kErrMma);
      };
      // (descriptors differ in their low word only: an address in units of 16 bytes)
      const uint64_t dq = smem_desc_sw128(s0 + kQ + x * 2 * kHalf);
      const uint64_t dk = smem_desc_sw128(s0 + kK), dv = smem_desc_sw128(s0 + kV);
      const uint32_t t_s = tmem + kTile * x, t_o = t_s + 2 * kTile;
      // scores of half a step: 64 rows of the K tile
      auto scores = [&](int st, int hf) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t at = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
          mma_f16_ss(t_s + (kTile / 2) * hf, dq + at,
                     dk + ((st * 2 * kHalf + hf * (kHalf / 2)) >> 4) + at, idesc_f16(kTile / 2),
                     ks > 0);
        }
      };
      bool ok = pass(bars.q_full, 0) && pass(bars.k_full[0], 0);
      if (ok) {
        tc_fence_after_sync();
        for (int h = 0; h < 2; ++h) {
          scores(0, h);
          mma_commit(bar(bars.s_full[x][h]));
        }
        mma_commit(bar(bars.k_empty[0]));
      }
      for (int hs = 0; ok && hs < 2 * steps; ++hs) {
        const int j = hs >> 1, hf = hs & 1, st = j & 1, next = st ^ 1;
        ok = pass(bars.p_full[x][hf], j & 1) && (hf == 1 || pass(bars.v_full[st], (j >> 1) & 1));
        if (!ok) break;
        tc_fence_after_sync();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_f16_ts(t_o, t_s + (kTile / 2) * hf + 8 * ks,
                     dv + ((st * 2 * kHalf + hf * kHalf + ks * 32) >> 4), idesc_f16(kTile),
                     hs > 0 || ks > 0);
        if (hf == 1) mma_commit(bar(bars.v_empty[st]));
        if (j + 1 < steps) {
          // the same half of the next step's scores, over the weights just multiplied: they
          // are there when the softmax of the other half is done
          if (hf == 0) {
            ok = pass(bars.k_full[next], ((j + 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after_sync();
          }
          scores(next, hf);
        }
        mma_commit(bar(bars.s_full[x][hf]));
        if (hf == 1 && j + 1 < steps) mma_commit(bar(bars.k_empty[next]));
      }
      if (ok) mma_commit(bar(bars.o_full));
    }
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// Once per device: opt in to the shared memory, and check the registers.  The
// kernel's warpgroups split 4 x 128 a thread among them (168, 168, 96, 80); a
// launch with fewer would wait for registers that never come free.
int prepare_prompt_kernel() {
  static std::atomic<unsigned long long> ready{0};
  return opt_in_smem(reinterpret_cast<const void*>(paged_prompt_kernel), kSmemBytes, ready, 128);
}

}  // namespace

void plan_prompt(PagedPlan& p, int T, int B, int Hq, int Hkv, int width, int page) {
  const int g = Hq / Hkv;
  p.tiles = slot_base(T, B, g, kSlotRows);
  p.prompt_target = sm_count();
  const long long pairs = static_cast<long long>(p.tiles) * Hkv;
  const long long steps = (static_cast<long long>(width) * page + kTile - 1) / kTile;
  const long long most_splits = (steps + kMinChunk - 1) / kMinChunk;
  // (split slots have over `chunk` >= steps * Hkv / target steps each, so fewer than
  // n / chunk + 1 < 2 n / chunk units, and the batch at most 2 target of them)
  const long long units = p.prompt_target + pairs, all = pairs * most_splits;
  p.prompt_grid = static_cast<int>(units < all ? units : all);
  p.prompt_units_off = p.take(static_cast<size_t>(p.prompt_grid) * sizeof(PromptUnit));
  if (most_splits > 1) {
    const long long split = 2LL * p.prompt_target;
    const long long parts = split < p.prompt_grid ? split : p.prompt_grid;
    p.prompt_combine = true;
    p.prompt_meta_off = p.take(static_cast<size_t>(pairs) * sizeof(int2));
    p.prompt_parts_off =
        p.take(static_cast<size_t>(parts) * kSlotRows * kPartFloats * sizeof(float));
  }
}

int launch_paged_prompt(const PagedArgs& a, const PagedPlan& p, const PromptUnit* units,
                        cudaStream_t s) {
  if (int st = prepare_prompt_kernel()) return st;
  return launch_dependent(paged_prompt_kernel, dim3(static_cast<unsigned>(p.prompt_grid)), kThreads,
                          kSmemBytes, s, a, units);
}

int prompt_device_error(unsigned int* value, int clear) {
  unsigned int v = 0;
  const unsigned int zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_prompt_error, sizeof(v)) != cudaSuccess ||
      (clear && v && cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(zero)) != cudaSuccess)) {
    cudaGetLastError();
    return QOQ_ERR_CUDA;
  }
  *value |= v;
  return QOQ_OK;
}

}  // namespace qoq
