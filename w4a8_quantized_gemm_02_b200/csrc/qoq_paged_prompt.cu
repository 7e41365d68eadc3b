// Attention over a paged 4-bit KV cache for the sequences with more rows than
// the decode kernel takes: chunks of a prompt, on the tcgen05 tensor cores.
//
// Rows.  The n query tokens of a sequence times the g heads of a KV head are the
// rows r = i g + h of one problem; a CTA takes 256 consecutive ones (a slot) as
// two tiles of 128, and walks the tokens that they see, 128 at a time:
//     S = Q (c_K - 8)^T        x_t = s_K S_t + (m_K + 8 s_K) Q_sum
//     W = fp16(2^(x - max) s_V)  O += W (c_V - 8),  o_off += p (m_V + 8 s_V).
// The codes enter both products as c - 8, exact FP16 numbers, so the rounding of
// W (2^-11 relative) is the only one besides the output's: rounding k^ and v^
// to FP16 instead would save the two scale products a score and cost two more
// errors of the output's own size.  Centred codes keep what the rounding of W
// touches as small as v^ about its vector's middle.
//
// Warps.  Warpgroups 0 and 1 hold a row a thread of one tile each (softmax);
// warpgroup 2 turns codes into FP16 tiles; one thread of warpgroup 3 issues the
// MMAs: for each tile in turn O += W V and then the next S, so one tile's
// products run while the other's softmax does.  W overwrites S in tensor memory
// (512 columns: S and O of both tiles).
//
// Layouts.  The cache's nibble order is the register layout of warp MMAs, so a
// lane of the producer holds, for one token, dimensions 16 w + 2 tig + {0, 1, 8,
// 9}, and for one dimension four tokens of a block.  Instead of shuffling, the
// tiles take that order: the K tile's k index is dimension position
// 32 tig + 4 w + 2 j1 + e (Q is stored the same way), and the columns of S, which
// are the k index of W V, are token position 8 tig + 4 block + 2 j1 + e of each 32
// (the rows of the K tile are stored at them).  Every store is 16 bytes.
//
// Splits.  All CTAs agree on the tokens a unit walks, from the lengths: long
// sequences with few rows are split so that no CTA is left with a long one, and
// a second kernel merges.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

#include "qoq.h"
#include "qoq_attn.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"
#include "qoq_kv4.cuh"
#include "qoq_paged.h"

namespace qoq {

namespace {

// This file's part of the device error word (device code of different files
// shares no variables).
__device__ unsigned int g_prompt_error = 0;

constexpr int kThreads = 512;
constexpr int kSlotRows = 256;
constexpr int kTile = 128;                      // rows of a tile, tokens of a step
constexpr int kMinChunk = 8;                    // steps: a split's least length
constexpr float kRaise = 2.9f;                  // 2^2.9 * 131008 / 15 is an FP16 number
constexpr int kMaxStagedSeqs = 2048;

// Shared memory: Q 2 tiles x 2 halves of 64 dimensions x [128 rows][128 bytes],
// K and V twice each, 2 halves x [128][128 bytes] (128-byte swizzle), then the
// scales of two steps: per column pair (s_K, s_K', m_K, m_K') and (s_V, s_V', m_V, m_V').
constexpr uint32_t kHalf = 16384;
constexpr uint32_t kQ = 0, kK = 4 * kHalf, kV = kK + 4 * kHalf, kScales = kV + 4 * kHalf;
constexpr uint32_t kScaleStage = 2 * 64 * 16;
constexpr uint32_t kSmemBytes = kScales + 2 * kScaleStage + 1024;   // + alignment

struct Bars {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], c_full[2], s_full[2], p_full[2],
      o_full;
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
// Instruction descriptor: FP16 A and B, K-major, FP32 accumulator, 128 x 128.
constexpr uint32_t kIdesc = (1u << 4) | (static_cast<uint32_t>(kTile >> 3) << 17) |
                            (static_cast<uint32_t>(kTile >> 4) << 24);

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
// The wait that completes loads, naming their registers so that no use moves
// above it.
__device__ __forceinline__ void tmem_ld_done(float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]),
                 "+r"(u[6]), "+r"(u[7]), "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]),
                 "+r"(u[12]), "+r"(u[13]), "+r"(u[14]), "+r"(u[15]), "+r"(u[16]), "+r"(u[17]),
                 "+r"(u[18]), "+r"(u[19]), "+r"(u[20]), "+r"(u[21]), "+r"(u[22]), "+r"(u[23]),
                 "+r"(u[24]), "+r"(u[25]), "+r"(u[26]), "+r"(u[27])
               :
               : "memory");
  asm volatile("" : "+r"(u[28]), "+r"(u[29]), "+r"(u[30]), "+r"(u[31])::"memory");
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

// Token (within its 32) at column position q of S, and back.
__host__ __device__ constexpr int token_at(int q) {
  return 16 * ((q >> 2) & 1) + 2 * (q >> 3) + (q & 1) + 8 * ((q >> 1) & 1);
}
__device__ __forceinline__ int column_of(int tok) {    // tok: 0 .. 31
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
__device__ __forceinline__ float4 lds16(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at));
  return v;
}

// Nibbles 4 s and 4 s + 16 of a word as FP16 numbers c - 8 (0x6400 | c is
// 1024 + c).
__device__ __forceinline__ uint32_t centred(uint32_t word, int s) {
  const uint32_t n = and_or(word >> s, 0x000f000fu, 0x64006400u);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&n), __float2half2_rn(1032.0f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct Unit {
  int b;             // sequence, -1: nothing to do
  int part;          // number of this unit among those of split slots
  int row0;          // first row r of the slot in its sequence
  int hk, split, nsplit;
  int slot;
  int step0, step1;  // steps of 128 tokens
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
  return (visible(position_of(a.seqlen[lo], rr.n, last / a.g), len) + kTile - 1) / kTile;
}

// The unit of this CTA: splits of equal length over the whole batch, the last
// slots (which see most) first.
__device__ __forceinline__ Unit find_unit(const PagedArgs& a, int tiles, int target, int min_rows,
                                          uint8_t* scratch) {
  __shared__ long long s_sum[kThreads / 32];
  __shared__ int2 s_scan[kThreads / 32];
  __shared__ int s_unit[7];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int* starts = a.q_start;
  if (a.B <= kMaxStagedSeqs) {
    int* staged = reinterpret_cast<int*>(scratch);
    for (int i = tid; i < a.B; i += kThreads) staged[i] = a.q_start[i];
    starts = staged;
  }
  if (tid == 0) s_unit[0] = -1;
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
  const long long want = (sum * a.Hkv + target - 1) / target;
  const int chunk = static_cast<int>(want < kMinChunk ? kMinChunk : want);
  int base = 0, pbase = 0;
  for (int s0 = 0; s0 < tiles && base <= static_cast<int>(blockIdx.x); s0 += kThreads) {
    const int s = s0 + tid;
    int n = n0, b = b0, r = row0;
    if (s0 > 0) n = s < tiles ? slot_steps(a, tiles - 1 - s, min_rows, starts, b, r) : -1;
    const int nsplit = n < 0 ? 0 : (n <= chunk ? 1 : (n + chunk - 1) / chunk);
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
    __syncthreads();
    int before = base, pbefore = pbase;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        before += s_scan[w].x;
        pbefore += s_scan[w].y;
      }
      base += s_scan[w].x;
      pbase += s_scan[w].y;
    }
    const int off = static_cast<int>(blockIdx.x) - (before + incl - mine);
    if (off >= 0 && off < mine) {
      s_unit[0] = b;
      s_unit[1] = r;
      s_unit[2] = off;
      s_unit[3] = nsplit;
      s_unit[4] = tiles - 1 - s;
      s_unit[5] = n;
      s_unit[6] = pbefore + pincl - parts + off;
    }
    __syncthreads();
  }
  Unit u;
  u.b = s_unit[0];
  if (u.b < 0) return u;
  u.row0 = s_unit[1];
  u.nsplit = s_unit[3];
  u.hk = s_unit[2] / u.nsplit;
  u.split = s_unit[2] - u.hk * u.nsplit;
  u.slot = s_unit[4];
  u.part = s_unit[6];
  // splits of one slot are equally long
  const int per = (s_unit[5] + u.nsplit - 1) / u.nsplit;
  u.step0 = u.split * per;
  u.step1 = u.step0 + per < s_unit[5] ? u.step0 + per : s_unit[5];
  return u;
}

__global__ void __launch_bounds__(kThreads, 1)
paged_prompt_kernel(const PagedArgs a, int tiles, int target, int min_rows) {
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ volatile uint32_t s_abort;
  __shared__ uint32_t s_absent[2][4];       // per step: bit per 16-token block and producer warp
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s0 = smem_u32(smem);
  grid_dependency_wait();
  grid_launch_dependents();
  const Unit u = find_unit(a, tiles, target, min_rows, smem);
  if (u.b < 0) return;

  const RowRange rr = rows_of(a.q_start, u.b, a.T);
  const int g = a.g, R = rr.n * g;
  const int seqlen = a.seqlen[u.b], len = clamp_len(seqlen, a.width * a.page);
  const bool two = u.row0 + kTile < R;      // the second tile has rows
  const int steps = u.step1 - u.step0;
  auto bar = [&](uint64_t& x) { return smem_u32(&x); };

  if (tid == 0) {
    s_abort = 0u;
    mbar_init(bar(bars.q_full), 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(bars.k_full[i]), 128);
      mbar_init(bar(bars.v_full[i]), 128);
      mbar_init(bar(bars.c_full[i]), 128);
      mbar_init(bar(bars.k_empty[i]), 1);
      mbar_init(bar(bars.v_empty[i]), 1);
      mbar_init(bar(bars.s_full[i]), 1);
      mbar_init(bar(bars.p_full[i]), 128);
    }
    mbar_init(bar(bars.o_full), 1);
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
    return mbar_wait(smem_u32(&x), parity, &s_abort, &g_prompt_error, err);
  };

  if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    regs_inc<192>();
    const int x = warp >> 2, row = 32 * (warp & 3) + lane;       // tile and row of it
    const int r = u.row0 + kTile * x + row;
    const int qi = r / g;
    const bool mine = r < R;
    const __half* q = a.Q + static_cast<size_t>(rr.first + (mine ? qi : 0)) * a.ldq +
                      static_cast<size_t>(u.hk * g + (mine ? r - qi * g : 0)) * kHeadDim;
    float qsum = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // 32 dimensions, words w = 2k and 2k + 1: four bytes (dimensions d, d + 1) at
      // 16 w + 2 tig and 16 w + 8 + 2 tig go to chunk 4 tig + k
      uint32_t d[2][8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = mine ? *reinterpret_cast<const uint4*>(q + 32 * k + 8 * i)
                             : make_uint4(0u, 0u, 0u, 0u);
        d[i >> 1][4 * (i & 1) + 0] = v.x;
        d[i >> 1][4 * (i & 1) + 1] = v.y;
        d[i >> 1][4 * (i & 1) + 2] = v.z;
        d[i >> 1][4 * (i & 1) + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&d[i >> 3][i & 7]));
        qsum += f.x + f.y;
      }
#pragma unroll
      for (int tig = 0; tig < 4; ++tig)
        sts16(s0 + kQ + x * 2 * kHalf + tile_at(row, 4 * tig + k),
              make_uint4(d[0][tig], d[0][4 + tig], d[1][tig], d[1][4 + tig]));
    }
    fence_proxy_async_smem();
    mbar_arrive(bar(bars.q_full));

    const int lim = mine ? visible(position_of(seqlen, rr.n, qi), len) : 0;
    float mref = 0.0f, l = 0.0f, off = 0.0f;
    const F2 q2 = pair2(qsum, qsum);
    const uint32_t t_s = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kTile * x;
    const uint32_t t_o = t_s + 2 * kTile;
    bool ok = true;
    if (x == 0 || two) {
      for (int j = 0; j < steps; ++j) {
        ok = wait(bars.s_full[x], j & 1, kErrEpilogue) &&
             wait(bars.c_full[j & 1], (j >> 1) & 1, kErrEpilogue);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        float s[kTile];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, s + 32 * c);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_done(s + 32 * c);
        const uint32_t sc = s0 + kScales + (j & 1) * kScaleStage;
        // x - mref
        const F2 ref = pair2(-mref, -mref);
#pragma unroll
        for (int c = 0; c < kTile; c += 2) {
          const float4 kc = lds16(sc + 8 * c);
          const F2 v = fma2(pair2(s[c], s[c + 1]), pair2(kc.x, kc.y),
                            fma2(q2, pair2(kc.z, kc.w), ref));
          s[c] = v.f[0];
          s[c + 1] = v.f[1];
        }
        // tokens that the row does not see, or in no page
        const int rel = lim - (u.step0 + j) * kTile;
        const uint32_t absent = s_absent[j & 1][0] | s_absent[j & 1][1] | s_absent[j & 1][2] |
                                s_absent[j & 1][3];
        if (__any_sync(0xffffffffu, rel < kTile || absent != 0u)) {
#pragma unroll
          for (int c = 0; c < kTile; ++c) {
            const int tok = 32 * (c >> 5) + token_at(c & 31);
            if (tok >= rel || ((absent >> (tok >> 4)) & 1u)) s[c] = -INFINITY;
          }
        }
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kTile; c += 2) top[(c >> 1) & 3] = max3(top[(c >> 1) & 3], s[c], s[c + 1]);
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // raise the reference: past the threshold, or at the first token seen
        const bool raise = high > kRaise || (l == 0.0f && high > -INFINITY);
        if (__any_sync(0xffffffffu, raise)) {
          const float up = raise ? high : 0.0f;
          mref += up;
          const float al = l == 0.0f ? 1.0f : fast_exp2(-up);
          l *= al;
          off *= al;
          const F2 d2 = pair2(-up, -up), al2 = pair2(al, al);
#pragma unroll
          for (int c = 0; c < kTile; c += 2) {
            const F2 v = add2(pair2(s[c], s[c + 1]), d2);
            s[c] = v.f[0];
            s[c + 1] = v.f[1];
          }
          if (j > 0) {
            // (the products that wrote O are complete: this step's S came after
            // them)
#pragma unroll 1
            for (int c = 0; c < kTile; c += 32) {
              float o[32];
              tmem_ld32(t_o + c, o);
              tmem_ld_done(o);
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const F2 v = mul2(pair2(o[k], o[k + 1]), al2);
                o[k] = v.f[0];
                o[k + 1] = v.f[1];
              }
              tmem_st_32x32b_x32(t_o + c, *reinterpret_cast<const uint32_t(*)[32]>(o));
            }
          }
        }
        // weights
        F2 l2[2] = {pair2(0.0f, 0.0f), pair2(0.0f, 0.0f)};
        F2 o2[2] = {pair2(0.0f, 0.0f), pair2(0.0f, 0.0f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int c = 64 * h + 2 * k;
            const float4 vc = lds16(sc + 1024 + 8 * c);
            const F2 p = pair2(fast_exp2(s[c]), fast_exp2(s[c + 1]));
            l2[k & 1] = add2(l2[k & 1], p);
            o2[k & 1] = fma2(p, pair2(vc.z, vc.w), o2[k & 1]);
            const F2 v = mul2(p, pair2(vc.x, vc.y));
            w[k] = pack_h2(v.f[0], v.f[1]);
          }
          tmem_st_32x32b_x32(t_s + 32 * h, w);
        }
        l2[0] = add2(l2[0], l2[1]);
        o2[0] = add2(o2[0], o2[1]);
        l += l2[0].f[0] + l2[0].f[1];
        off += o2[0].f[0] + o2[0].f[1];
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(bar(bars.p_full[x]));
      }
      if (steps > 0 && ok) ok = wait(bars.o_full, 0, kErrEpilogue);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after_sync();
        const bool whole = u.nsplit == 1;
        // (a row that saw no token has l = 0; its O is zero or was not written)
        const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
        float* part = nullptr;
        __half* dst = nullptr;
        if (whole)
          dst = a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + u.hk * g + (r - qi * g)) *
                            kHeadDim;
        else
          part = a.parts + (static_cast<size_t>(u.part) * kSlotRows + kTile * x + row) *
                               kPartFloats;
        if (!whole && mine) {
          part[0] = l == 0.0f ? -INFINITY : mref;
          part[1] = l;
        }
#pragma unroll 1
        for (int c = 0; c < kTile; c += 32) {
          float o[32];
          if (steps > 0) {
            tmem_ld32(t_o + c, o);
            tmem_ld_done(o);
          }
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = l == 0.0f ? 0.0f : o[k + i] + off;
            if (mine) {
              if (whole) {
                store_row8(dst + c + k, v, inv);
              } else {
                *reinterpret_cast<float4*>(part + 4 + c + k) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4*>(part + 8 + c + k) = make_float4(v[4], v[5], v[6], v[7]);
              }
            }
          }
        }
      }
    }
    if (tid == 0 && u.split == 0 && a.meta != nullptr)
      a.meta[u.slot * a.Hkv + u.hk] = make_int2(u.part, u.nsplit);
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
    if (steps > 0) fetch(u.step0);
    for (int j = 0; j < steps; ++j) {
      const int st = j & 1, use = j >> 1;
      if (use > 0 && !wait(bars.k_empty[st], (use - 1) & 1, kErrProducer)) break;
      // K tile: row column_of(token), chunks 4 tig + k of words 2k, 2k + 1
      const uint32_t kt = s0 + kK + st * 2 * kHalf;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j0 = 0; j0 < 2; ++j0) {
          const int row = 32 * pw + column_of(16 * i + gid + 8 * j0);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 q4 = k4[i][k >> 1];
            const uint32_t w0 = (k & 1) ? q4.z : q4.x, w1 = (k & 1) ? q4.w : q4.y;
            const int kk = (k & 1) + 2 * ((k >> 1) ^ (tig >> 1));
            sts16(kt + tile_at(row, 4 * tig + kk),
                  make_uint4(centred(w0, 4 * j0), centred(w0, 4 * j0 + 8), centred(w1, 4 * j0),
                             centred(w1, 4 * j0 + 8)));
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(bars.k_full[st]));

      if (use > 0 && !wait(bars.v_empty[st], (use - 1) & 1, kErrProducer)) break;
      {
        const int tok = (u.step0 + j) * kTile + 32 * pw + lane;
        const float2 fk = __half22float2(*reinterpret_cast<const __half2*>(&s4.x));
        const float2 fv = __half22float2(*reinterpret_cast<const __half2*>(&s4.y));
        // (a slot past the length may hold anything: its scales count as zero)
        const bool in = tok < len;
        const int c = 32 * pw + column_of(lane);
        const uint32_t at = s0 + kScales + st * kScaleStage + 16 * (c >> 1) + 4 * (c & 1);
        auto put = [&](uint32_t d, float v) {
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + d), "f"(in ? v : 0.0f) : "memory");
        };
        put(0, fk.x * scale2);
        put(8, fmaf(8.0f, fk.x, fk.y) * scale2);
        put(1024, fv.x);
        put(1024 + 8, fmaf(8.0f, fv.x, fv.y));
        if (lane == 0) s_absent[st][pw] = gone;
      }
      mbar_arrive(bar(bars.c_full[st]));
      // V tile: row dimension, chunk of tokens 32 pw + 8 tig ..
      const uint32_t vt = s0 + kV + st * 2 * kHalf;
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const uint4 a4 = v4[0][w >> 2], b4 = v4[1][w >> 2];
        const uint32_t wa = (w & 3) == 0 ? a4.x : (w & 3) == 1 ? a4.y : (w & 3) == 2 ? a4.z : a4.w;
        const uint32_t wb = (w & 3) == 0 ? b4.x : (w & 3) == 1 ? b4.y : (w & 3) == 2 ? b4.z : b4.w;
#pragma unroll
        for (int j0 = 0; j0 < 2; ++j0)
          sts16(vt + tile_at(16 * w + gid + 8 * j0, 4 * pw + tig),
                make_uint4(centred(wa, 4 * j0), centred(wa, 4 * j0 + 8), centred(wb, 4 * j0),
                           centred(wb, 4 * j0 + 8)));
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(bars.v_full[st]));
      if (j + 1 < steps) fetch(u.step0 + j + 1);
    }
  } else {
    regs_dec<32>();
    if (warp == 12 && lane == 0 && steps > 0) {
      // ------------------------------------------------------------------ MMA
      const uint32_t tiles_here = two ? 2 : 1;
      auto scores = [&](uint32_t x, int st) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t at = (ks >> 2) * kHalf + (ks & 3) * 32;
          mma_f16_ss(tmem + kTile * x, smem_desc_sw128(s0 + kQ + x * 2 * kHalf + at),
                     smem_desc_sw128(s0 + kK + st * 2 * kHalf + at), kIdesc, ks > 0);
        }
        mma_commit(bar(bars.s_full[x]));
      };
      bool ok = wait(bars.q_full, 0, kErrMma) && wait(bars.k_full[0], 0, kErrMma);
      if (ok) {
        tc_fence_after_sync();
        for (uint32_t x = 0; x < tiles_here; ++x) scores(x, 0);
        mma_commit(bar(bars.k_empty[0]));
      }
      for (int j = 0; j < steps && ok; ++j) {
        const int st = j & 1, next = (j + 1) & 1;
        for (uint32_t x = 0; x < tiles_here && ok; ++x) {
          ok = wait(bars.p_full[x], j & 1, kErrMma);
          if (ok && x == 0) ok = wait(bars.v_full[st], (j >> 1) & 1, kErrMma);
          if (!ok) break;
          tc_fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_f16_ts(tmem + 2 * kTile + kTile * x, tmem + kTile * x + 8 * ks,
                       smem_desc_sw128(s0 + kV + st * 2 * kHalf + (ks >> 2) * kHalf + (ks & 3) * 32),
                       kIdesc, j > 0 || ks > 0);
          if (j + 1 < steps) {
            if (x == 0) ok = wait(bars.k_full[next], ((j + 1) >> 1) & 1, kErrMma);
            if (!ok) break;
            tc_fence_after_sync();
            scores(x, next);
          }
        }
        if (!ok) break;
        mma_commit(bar(bars.v_empty[st]));
        if (j + 1 < steps) mma_commit(bar(bars.k_empty[next]));
        else mma_commit(bar(bars.o_full));
      }
    }
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

// Rows of the split slots from their partial results: kCombineRows rows a CTA, a warp a
// row at a time.
constexpr int kCombineRows = 32;
__global__ void __launch_bounds__(256)
paged_prompt_combine_kernel(const PagedArgs a, int tiles, int min_rows) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int kParts = kSlotRows / kCombineRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x / kParts;
  const int slot = pair / a.Hkv, hk = pair - slot * a.Hkv;
  int b = 0, row0 = 0;
  if (slot_steps(a, slot, min_rows, a.q_start, b, row0) <= kMinChunk) return;   // not split
  const int2 mt = a.meta[pair];
  if (mt.y <= 1) return;
  const RowRange rr = rows_of(a.q_start, b, a.T);
  for (int i = warp; i < kCombineRows; i += 8) {
    const int rs = (blockIdx.x - pair * kParts) * kCombineRows + i;
    const int r = row0 + rs;
    if (r >= rr.n * a.g) return;
    const float* base = a.parts + (static_cast<size_t>(mt.x) * kSlotRows + rs) * kPartFloats;
    const size_t step = static_cast<size_t>(kSlotRows) * kPartFloats;
    float M = -INFINITY;
    for (int p = lane; p < mt.y; p += 32) M = fmaxf(M, base[p * step]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float den = 0.0f;
    float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int p = 0; p < mt.y; ++p) {
      const float* pp = base + p * step;
      const float m = pp[0];
      const float f = m == -INFINITY ? 0.0f : fast_exp2(m - M);
      const float4 v = *reinterpret_cast<const float4*>(pp + 4 + 4 * lane);
      den += f * pp[1];
      num.x += f * v.x;
      num.y += f * v.y;
      num.z += f * v.z;
      num.w += f * v.w;
    }
    const int qi = r / a.g;
    store_row4(a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + hk * a.g + (r - qi * a.g)) *
                           kHeadDim + 4 * lane, num, den == 0.0f ? 0.0f : __frcp_rn(den));
  }
}

// Once per device: opt in to the shared memory, and check the registers.  The
// kernel's warpgroups split 4 x 128 a thread among them (192, 192, 96, 32); a
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
  if (most_splits > 1) {
    const long long split = 2LL * p.prompt_target;
    const long long parts = split < p.prompt_grid ? split : p.prompt_grid;
    p.prompt_combine = true;
    p.prompt_meta_off = p.take(static_cast<size_t>(pairs) * sizeof(int2));
    p.prompt_parts_off =
        p.take(static_cast<size_t>(parts) * kSlotRows * kPartFloats * sizeof(float));
  }
}

int launch_paged_prompt(const PagedArgs& a, const PagedPlan& p, int min_rows, cudaStream_t s) {
  if (int st = prepare_prompt_kernel()) return st;
  if (int st = launch_dependent(paged_prompt_kernel, dim3(static_cast<unsigned>(p.prompt_grid)),
                                kThreads, kSmemBytes, s, a, p.tiles, p.prompt_target, min_rows))
    return st;
  if (!p.prompt_combine) return QOQ_OK;
  const long long ctas = static_cast<long long>(p.tiles) * a.Hkv * (kSlotRows / kCombineRows);
  return launch_dependent(paged_prompt_combine_kernel, dim3(static_cast<unsigned>(ctas)), 256, 0, s,
                          a, p.tiles, min_rows);
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
