// Attention over a paged 4-bit KV cache: single tokens (decode) and the few
// query tokens of a sequence that is verified or extended by a handful.
//
// Row tile.  The n query tokens of a sequence times the g = Hq / Hkv heads of a
// KV head are the rows of one problem: row r = i g + h.  Up to 16 rows run
// here; more go to the prompt kernel.
//
// Arithmetic.  With k^ = s q + m the products never leave the codes c (the
// cache's UINT4 values, exact as FP16 subnormals c 2^-24):
//     q . k^_t = s_t (q . c_t) + m_t Q,    Q = sum_i q_i,
//     sum_t p_t v^_t = sum_t w_t c_t + sum_t p_t m_t,    w_t = p_t s_t.
// The weights enter the tensor cores as w~ = fp16(w), half an FP16 step (2^-12)
// off.  Codes lie around 8, so that error times 8 would dominate where values
// cancel; with
//     sum w c = sum w~ (c - 8) + 8 sum w + (error: sum (w - w~)(c - 8))
// the products stay on c, and each weight adds 8 (w - w~) to its row's FP32
// offset sum: what is left is 2^-12 of values centred on their vector's middle,
// no more than rounding v^ itself would cost.
//
// The running maximum is only raised when a score passes it by 2.9 (in log2
// units): one vote a block instead of a reduction.  2^2.9 = 7.46 times the
// largest scale of a finite FP16 vector, 131008 / 15, is still an FP16 number.
//
// Bound.  136 bytes a token and KV head, read once; the instructions of the
// unpacking and of the softmax come close behind (see the figures at the
// kernel).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "qoq.h"
#include "qoq_attn.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"
#include "qoq_kv4.cuh"
#include "qoq_paged.h"

namespace qoq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;                           // per warp: blocks of 16 tokens in flight
constexpr int kStageBytes = 1024 + 1024 + 128;       // K codes, V codes, scales of a block
constexpr int kMinBlocks = 32;                       // a split's least length: 8 blocks a warp
constexpr float kRaise = 2.9f;
// Codes are FP16 subnormals: c 2^-24 on rows 0..7 of the 16-row operand, c 2^-20
// on rows 8..15 (masked out of bits 4..7 without a shift).
constexpr float kRowScale0 = 16777216.0f, kRowScale1 = 1048576.0f;

__device__ __forceinline__ void a_frag(uint32_t word, uint32_t (&a)[4]) {
  const uint32_t hi = word >> 8;
  a[0] = word & 0x000f000fu;
  a[1] = word & 0x00f000f0u;
  a[2] = hi & 0x000f000fu;
  a[3] = hi & 0x00f000f0u;
}

// 16-token blocks of sequence b for this kernel: 0 for an empty one that still
// has rows to write, -1 where it has no work here.
__device__ __forceinline__ int blocks_of(const PagedArgs& a, int b, int rows_max_here) {
  const RowRange rr = rows_of(a.q_start, b, a.T);
  if (rr.n <= 0 || rr.n > a.max_q || rr.n * a.g > rows_max_here) return -1;
  return (clamp_len(a.seqlen[b], a.width * a.page) + 15) >> 4;
}

// Grid: `target` + B * Hkv CTAs at most; every one finds its work from the
// lengths.  All CTAs agree on the split length `chunk` = the batch's blocks over
// `target`, so splits are equally long whatever the mix of lengths, and a
// sequence has as many as it needs.  Unit u is split u - base of a (sequence, KV
// head) pair; warp w takes every fourth block of it.
template <int NT>
__global__ void __launch_bounds__(kThreads)
paged_decode_kernel(const PagedArgs a, int target) {
  __shared__ __align__(16) uint8_t smem[kWarps * kStages * kStageBytes];
  __shared__ long long s_sum[kWarps];
  __shared__ int2 s_scan[kWarps];
  __shared__ int s_unit[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  grid_dependency_wait();
  grid_launch_dependents();

  // --- the unit of this CTA ---
  const int u = blockIdx.x;
  long long sum = 0;
  const int n0 = static_cast<int>(threadIdx.x) < a.B ? blocks_of(a, threadIdx.x, 8 * NT) : -1;
  if (n0 > 0) sum = n0;
  for (int b = threadIdx.x + kThreads; b < a.B; b += kThreads) {
    const int n = blocks_of(a, b, 8 * NT);
    if (n > 0) sum += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  if (threadIdx.x == 0) s_unit[0] = -1;
  __syncthreads();
  sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
  long long want = (sum * a.Hkv + target - 1) / target;
  want = (want + kWarps - 1) / kWarps * kWarps;
  const int chunk = static_cast<int>(want < kMinBlocks ? kMinBlocks : want);
  int base = 0, pbase = 0;
  for (int b0 = 0; b0 < a.B && base <= u; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const int n = b0 == 0 ? n0 : (b < a.B ? blocks_of(a, b, 8 * NT) : -1);
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
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        before += s_scan[w].x;
        pbefore += s_scan[w].y;
      }
      base += s_scan[w].x;
      pbase += s_scan[w].y;
    }
    const int off = u - (before + incl - mine);
    if (off >= 0 && off < mine) {
      s_unit[0] = b;
      s_unit[1] = off;
      s_unit[2] = nsplit;
      s_unit[3] = pbefore + pincl - parts + off;    // its number among the split ones
    }
    __syncthreads();
  }
  const int b = s_unit[0];
  if (b < 0) return;
  const int nsplit = s_unit[2];
  const int hk = s_unit[1] / nsplit, split = s_unit[1] - hk * nsplit;
  const RowRange rr = rows_of(a.q_start, b, a.T);
  const int g = a.g, R = rr.n * g;
  const int Lb = clamp_len(a.seqlen[b], a.width * a.page);
  const int nblk = (Lb + 15) >> 4;
  const int ppb = a.page >> 4;
  const int blk0 = split * chunk + warp;
  const int blk1 = (split + 1) * chunk < nblk ? (split + 1) * chunk : nblk;
  const int niter = blk0 < blk1 ? (blk1 - blk0 + kWarps - 1) / kWarps : 0;
  const int* table_row = a.table + static_cast<size_t>(b) * a.width;

  // --- copies: the numbers of 32 iterations' blocks are looked up at a time, one
  // a lane; each copy instruction moves 512 contiguous bytes ---
  uint8_t* wring = smem + warp * kStages * kStageBytes;
  const uint32_t ring0 = smem_u32(wring);
  const uint32_t s_lo = 16 * chunk_slot(lane), s_hi = 16 * chunk_slot(32 + lane);
  int window = -1;
  auto issue = [&](int it) {
    if (it < niter) {
      if ((it & 31) == 0) {
        const int blk = blk0 + (it + lane) * kWarps;
        window = blk < blk1 ? pool_block(table_row, blk, ppb, a.pages, a.Hkv, hk) : -1;
      }
      const int blk = __shfl_sync(0xffffffffu, window, it & 31);
      if (blk >= 0) {
        const uint32_t dst = ring0 + (it % kStages) * kStageBytes;
        const uint8_t* kp = a.kc + static_cast<size_t>(blk) * 1024 + 16 * lane;
        const uint8_t* vp = a.vc + static_cast<size_t>(blk) * 1024 + 16 * lane;
        cp_async16(dst + s_lo, kp);
        cp_async16(dst + s_hi, kp + 512);
        cp_async16(dst + 1024 + s_lo, vp);
        cp_async16(dst + 1024 + s_hi, vp + 512);
        if (lane < 8)
          cp_async16(dst + 2048 + 16 * lane,
                     reinterpret_cast<const uint8_t*>(a.sc) + static_cast<size_t>(blk) * 128 +
                         16 * lane);
      }
    }
    cp_async_commit();   // an empty group past the end keeps the counting uniform
  };
#pragma unroll
  for (int it = 0; it < kStages - 1; ++it) issue(it);

  // --- Q^T as B fragments (k = dimensions, n = row 8 nt + gid) and the sums Q of
  // the rows 8 nt + 2 tig + c of this lane's accumulators ---
  uint32_t qb[NT][8][2];
  float qh[NT][2];
  int lim[NT][2];          // tokens a row sees
  const float scale2 = a.scale * 1.4426950408889634f;   // scores in log2 units
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + gid;
    const bool ok = r < R;
    const int qi = r / g;
    const __half* q = a.Q + static_cast<size_t>(rr.first + (ok ? qi : 0)) * a.ldq +
                      static_cast<size_t>(hk * g + (ok ? r - qi * g : 0)) * kHeadDim;
    float qs = 0.0f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const int d0 = 16 * ks + 2 * tig;
      qb[nt][ks][0] = ok ? *reinterpret_cast<const uint32_t*>(q + d0) : 0u;
      qb[nt][ks][1] = ok ? *reinterpret_cast<const uint32_t*>(q + d0 + 8) : 0u;
      const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&qb[nt][ks][0]));
      const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&qb[nt][ks][1]));
      qs += (f0.x + f0.y) + (f1.x + f1.y);
    }
    qs += __shfl_xor_sync(0xffffffffu, qs, 1);
    qs += __shfl_xor_sync(0xffffffffu, qs, 2);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      qh[nt][c] = __shfl_sync(0xffffffffu, qs, 8 * tig + 4 * c) * scale2;
      const int row = 8 * nt + 2 * tig + c;
      lim[nt][c] = row < R ? visible(position_of(a.seqlen[b], rr.n, row / g), Lb) : 0;
    }
  }
  const int all_see = visible(position_of(a.seqlen[b], rr.n, 0), Lb);

  float acc[NT][8][4];
  float mrun[NT][2], lsum[NT][2], osum[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < 8; ++mt)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[nt][mt][k] = 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      mrun[nt][c] = -INFINITY;
      lsum[nt][c] = osum[nt][c] = 0.0f;
    }
  }

  uint32_t absent = 0;    // of 32 iterations: the blocks whose page is not in the pool
  for (int it = 0; it < niter; ++it) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    // (the copies run less than 32 iterations ahead: at a multiple of 32 the
    // window is still the one of this iteration)
    if ((it & 31) == 0) absent = __ballot_sync(0xffffffffu, window < 0);
    const int blk = blk0 + it * kWarps;
    const uint8_t* stage = wring + (it % kStages) * kStageBytes;
    const uint4 kq0 = *reinterpret_cast<const uint4*>(stage + 16 * chunk_slot(2 * lane));
    const uint4 kq1 = *reinterpret_cast<const uint4*>(stage + 16 * chunk_slot(2 * lane + 1));
    const uint4 vq0 = *reinterpret_cast<const uint4*>(stage + 1024 + 16 * chunk_slot(2 * lane));
    const uint4 vq1 = *reinterpret_cast<const uint4*>(stage + 1024 + 16 * chunk_slot(2 * lane + 1));
    const uint2 sq[2] = {*reinterpret_cast<const uint2*>(stage + 2048 + 8 * gid),
                         *reinterpret_cast<const uint2*>(stage + 2048 + 64 + 8 * gid)};
    __syncwarp();           // every lane has read the stage before it is copied into again
    issue(it + kStages - 1);
    if ((absent >> (it & 31)) & 1u) continue;

    auto step = [&](auto masked) {
      constexpr bool kMasked = decltype(masked)::value;
      const uint32_t wk[8] = {kq0.x, kq0.y, kq0.z, kq0.w, kq1.x, kq1.y, kq1.z, kq1.w};
      const uint32_t wv[8] = {vq0.x, vq0.y, vq0.z, vq0.w, vq1.x, vq1.y, vq1.z, vq1.w};
      // S^T = C_K Q^T: rows tokens gid and gid + 8, columns rows 2 tig and + 1
      float s[NT][4], s2[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[nt][k] = s2[nt][k] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < 8; ks += 2) {
        uint32_t f0[4], f1[4];
        a_frag(wk[ks], f0);
        a_frag(wk[ks + 1], f1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(s[nt], f0, qb[nt][ks][0], qb[nt][ks][1]);
          mma_16816(s2[nt], f1, qb[nt][ks + 1][0], qb[nt][ks + 1][1]);
        }
      }
      float skt[2], mkt[2], svt[2], mvt[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 k2 = __half22float2(*reinterpret_cast<const __half2*>(&sq[r].x));
        const float2 v2 = __half22float2(*reinterpret_cast<const __half2*>(&sq[r].y));
        skt[r] = k2.x * ((r ? kRowScale1 : kRowScale0) * scale2);
        mkt[r] = k2.y;
        svt[r] = v2.x;
        mvt[r] = v2.y;
      }
      bool raise = false;
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = k >> 1, c = k & 1;
          s[nt][k] += s2[nt][k];
          // relative to the running maximum (-inf at first: the sum is then no
          // number below the threshold)
          float v = fmaf(skt[r], s[nt][k], fmaf(mkt[r], qh[nt][c], -mrun[nt][c]));
          if (kMasked && blk * 16 + gid + 8 * r >= lim[nt][c]) v = -INFINITY;
          x[nt][k] = v;
          raise |= !(v <= kRaise);
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float y[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              y[r] = fmaf(skt[r], s[nt][2 * r + c], mkt[r] * qh[nt][c]);
              if (kMasked && blk * 16 + gid + 8 * r >= lim[nt][c]) y[r] = -INFINITY;
            }
            float top = fmaxf(y[0], y[1]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            top = fmaxf(top, mrun[nt][c]);
            const float al = top == -INFINITY ? 1.0f : fast_exp2(mrun[nt][c] - top);
            mrun[nt][c] = top;
            lsum[nt][c] *= al;
            osum[nt][c] *= al;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              acc[nt][mt][c] *= al;
              acc[nt][mt][2 + c] *= al;
            }
            const float ref = top == -INFINITY ? 0.0f : top;
            x[nt][c] = y[0] - ref;
            x[nt][2 + c] = y[1] - ref;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float wt[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = k >> 1, c = k & 1;
          const float p = fast_exp2(x[nt][k]);
          lsum[nt][c] += p;
          // (a masked token's scales may never have been written: its terms are
          // left out, not multiplied by 0)
          const bool in = !kMasked || x[nt][k] != -INFINITY;
          wt[k] = in ? p * svt[r] : 0.0f;
          osum[nt][c] += in ? p * mvt[r] : 0.0f;
        }
        const uint32_t top = pack_h2(wt[0], wt[1]), bot = pack_h2(wt[2], wt[3]);
        const float2 ft = __half22float2(*reinterpret_cast<const __half2*>(&top));
        const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&bot));
        osum[nt][0] = fmaf(8.0f, (wt[0] - ft.x) + (wt[2] - fb.x), osum[nt][0]);
        osum[nt][1] = fmaf(8.0f, (wt[1] - ft.y) + (wt[3] - fb.y), osum[nt][1]);
        const uint32_t b0 = transpose8x8(top), b1 = transpose8x8(bot);
        // O^T += C_V^T W^T, dimensions 16 mt .. from word mt
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          uint32_t f[4];
          a_frag(wv[mt], f);
          mma_16816(acc[nt][mt], f, b0, b1);
        }
      }
    };
    if (blk * 16 + 16 <= all_see) step(std::false_type{});
    else step(std::true_type{});
  }
  cp_async_wait<0>();
  __syncthreads();   // the ring becomes the merge area

  // per warp and row: max, sum, 128 outputs
  float* mrg = reinterpret_cast<float*>(smem);     // [warp][8 NT][kPartFloats]
  static_assert(sizeof(float) * kWarps * 8 * NT * kPartFloats <= sizeof(smem), "merge area");
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = lsum[nt][c], o = osum[nt][c];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, d);
        o += __shfl_xor_sync(0xffffffffu, o, d);
      }
      float* row = mrg + (warp * 8 * NT + 8 * nt + 2 * tig + c) * kPartFloats;
      if (gid == 0) {
        row[0] = mrun[nt][c];
        row[1] = l;
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        row[4 + 16 * mt + gid] = fmaf(acc[nt][mt][c], kRowScale0, o);
        row[4 + 16 * mt + gid + 8] = fmaf(acc[nt][mt][2 + c], kRowScale1, o);
      }
    }
  __syncthreads();
  const int pair = b * a.Hkv + hk;
  if (threadIdx.x == 0 && split == 0 && a.meta != nullptr)
    a.meta[pair] = make_int2(s_unit[3], nsplit);
  // 16 threads a row, 8 dimensions each
  const int d0 = 8 * (threadIdx.x & 15);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + (threadIdx.x >> 4);
    if (r >= R) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, mrg[(w * 8 * NT + r) * kPartFloats]);
    float den = 0.0f, v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* row = mrg + (w * 8 * NT + r) * kPartFloats;
      const float f = row[0] == -INFINITY ? 0.0f : fast_exp2(row[0] - M);
      if (f == 0.0f) continue;
      den += f * row[1];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += f * row[4 + d0 + k];
    }
    if (nsplit == 1) {
      const int qi = r / g;
      const float inv = den > 0.0f ? __frcp_rn(den) : 0.0f;
      if (!(den > 0.0f) && den == den)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      store_row8(a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + hk * g + (r - qi * g)) *
                             kHeadDim + d0, v, den == den ? inv : den);
    } else {
      float* part = a.parts + (static_cast<size_t>(s_unit[3]) * (8 * NT) + r) * kPartFloats;
      if ((threadIdx.x & 15) == 0) {
        part[0] = M;
        part[1] = den;
      }
      *reinterpret_cast<float4*>(part + 4 + d0) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(part + 8 + d0) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
}

// The rows of the split sequences from their partial results, W warps a row:
// a warp takes every W-th split, a lane four dimensions.
template <int W>
__global__ void __launch_bounds__(256) paged_combine_kernel(const PagedArgs a, int rows, int stride) {
  __shared__ float4 red_num[8][32];
  __shared__ float2 red_md[8];
  grid_dependency_wait();
  grid_launch_dependents();
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
        n = mt.y > 1 ? mt.y : 0;
      }
    }
  }
  const float* base = a.parts + (static_cast<size_t>(mt.x) * stride + r) * kPartFloats;
  const size_t step = static_cast<size_t>(stride) * kPartFloats;
  float M = -INFINITY, den = 0.0f;
  float4 num = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int p = lane; p < n; p += 32) M = fmaxf(M, base[p * step]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll 4
  for (int p = sub; p < n; p += W) {
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
  const float inv = den == 0.0f ? 0.0f : __frcp_rn(den);
  const int qi = r / a.g;
  __half2 o[2] = {__floats2half2_rn(num.x * inv, num.y * inv),
                  __floats2half2_rn(num.z * inv, num.w * inv)};
  *reinterpret_cast<uint2*>(a.out + (static_cast<size_t>(rr.first + qi) * a.Hq + hk * a.g +
                                     (r - qi * a.g)) * kHeadDim + 4 * lane) =
      *reinterpret_cast<const uint2*>(o);
}

template <int NT>
int launch_decode(const PagedArgs& a, const PagedPlan& p, cudaStream_t s) {
  if (int st = launch_dependent(paged_decode_kernel<NT>, dim3(static_cast<unsigned>(p.grid)),
                                kThreads, 0, s, a, p.target))
    return st;
  if (!p.combine) return QOQ_OK;
  const int rows = a.max_q * a.g < 8 * NT ? a.max_q * a.g : 8 * NT;
  const long long all = static_cast<long long>(a.B) * a.Hkv * rows;
  // few rows have many splits each: eight warps a row
  if (all <= 512)
    return launch_dependent(paged_combine_kernel<8>, dim3(static_cast<unsigned>(all)), 256, 0, s, a,
                            rows, 8 * NT);
  return launch_dependent(paged_combine_kernel<1>, dim3(static_cast<unsigned>((all + 7) / 8)), 256,
                          0, s, a, rows, 8 * NT);
}

}  // namespace

PagedPlan paged_plan(int T, int B, int Hq, int Hkv, int width, int page, int max_q) {
  PagedPlan p = {};
  const int g = Hq / Hkv;
  const long long pairs = static_cast<long long>(B) * Hkv;
  const long long most = static_cast<long long>(max_q) * g;     // rows of a sequence
  p.nt = most <= 8 || g <= 8 ? 1 : (g <= 16 ? 2 : 0);
  if (most > 8 && most <= 16) p.nt = 2;
  p.prompt = most > 8 * p.nt;
  const long long blocks = (static_cast<long long>(width) * page + 15) / 16;
  if (p.nt) {
    const long long most_splits = (blocks + kMinBlocks - 1) / kMinBlocks;
    p.target = 8 * sm_count();
    const long long a = p.target + pairs, b = pairs * most_splits;
    p.grid = static_cast<int>(a < b ? a : b);
    p.combine = most_splits > 1;
    if (p.combine) {
      // A sequence is split where its length n is over chunk >= blocks * Hkv / target
      // (all in blocks), into fewer than n / chunk + 1 < 2 n / chunk: at most 2 target
      // units of the batch leave partial results.
      const long long split = 2LL * p.target;
      const long long parts = split < p.grid ? split : p.grid;
      p.meta_off = p.take(static_cast<size_t>(pairs) * sizeof(int2));
      p.parts_off = p.take(static_cast<size_t>(parts) * 8 * p.nt * kPartFloats * sizeof(float));
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
  if (p.nt) {
    a.meta = p.combine ? reinterpret_cast<int2*>(w + p.meta_off) : nullptr;
    a.parts = p.combine ? reinterpret_cast<float*>(w + p.parts_off) : nullptr;
    const int st = p.nt == 1 ? launch_decode<1>(a, p, s) : launch_decode<2>(a, p, s);
    if (st) return st;
  }
  if (p.prompt) {
    a.meta = p.prompt_combine ? reinterpret_cast<int2*>(w + p.prompt_meta_off) : nullptr;
    a.parts = p.prompt_combine ? reinterpret_cast<float*>(w + p.prompt_parts_off) : nullptr;
    return launch_paged_prompt(a, p, 8 * p.nt + 1, s);
  }
  return QOQ_OK;
}
