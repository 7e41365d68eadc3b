// Appending the rows of a fused QKV projection to a paged 4-bit KV cache, with
// the position rotation (RoPE) applied on the way.
//
// Row r, the i-th of the n query tokens of its sequence, has position
// p = seqlen - n + i.  The pairs of the rotated part of every query and key
// head turn by p * inv_freq[j] radians:
//     (x0, x1) -> factor * (x0 cos - x1 sin, x1 cos + x0 sin),
// pair j being the dimensions (j, j + rot/2) or (2j, 2j + 1).  Queries are
// rounded to FP16 and returned; keys are rounded to binary32 and then FP16, and
// keys and values quantized per (token, head) vector as kv4_quantize does.
//
// Precision.  A key beside a code's border moves by a whole step (1/15 of its
// vector's range) if its rotation is off in the last bit, so angles and keys
// are rotated in binary64.  The angle is reduced in turns: with 1/(2 pi) as a
// pair of doubles, h + l = inv_freq / (2 pi) to about 2^-100, p h is split by an
// FMA into its rounded value and the rest, and the fraction of a turn goes to
// sincospi: the error is about 2^-53 turns for any 32-bit position.  Queries cross no
// such border: their angles are reduced the same way, and in prompts (by blocks) their
// products are binary32, 2^-21 of the pair's size beside the FP16 rounding; binary64 would
// take more conversions a pair than it has arithmetic.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qoq.h"
#include "qoq_device.cuh"
#include "qoq_internal.h"
#include "qoq_kv4.cuh"
#include "qoq_paged.h"

namespace qoq {
namespace {

// Rows a sequence, on average, from which a call goes by blocks.  64 sequences of 12
// rows (32 / 8 heads) take 16.6 us either way, of 6 rows 14.5 us by blocks and 12.3 by
// rows, of 24 rows 20.7 and 28.8.
constexpr int kBlockRows = 16;

struct AppendArgs {
  const __half* qkv;
  size_t ld;                  // elements between rows
  int T, Hq, Hkv, B;
  const int* q_start;
  const int* seqlen;
  const int* table;
  int width, pages, page;
  const double* inv_freq;     // rot / 2 of them
  int rot;                    // rotated dimensions of a head (0: none)
  int interleaved;
  double factor;
  __half* q_out;
  uint8_t* kc;
  uint8_t* vc;
  __half* sc;
  __half* k_hat;              // optional: the values the cache then holds
  __half* v_hat;
};

// The fraction of a turn in p * f radians.
__device__ __forceinline__ double rope_turn(long long p, double f) {
  const double kInvTau = 0.15915494309189535, kInvTauLow = -9.839338337591243e-18;
  const double h = f * kInvTau;
  const double l = fma(f, kInvTau, -h) + f * kInvTauLow;
  const double pd = static_cast<double>(p);
  const double t = pd * h;
  return (t - rint(t)) + (fma(pd, h, -t) + pd * l);
}
// factor * (cos, sin) of p * f radians.
__device__ __forceinline__ double2 rope_cos_sin(long long p, double f, double factor) {
  double s, c;
  sincospi(2.0 * rope_turn(p, f), &s, &c);
  return make_double2(c * factor, s * factor);
}
__device__ __forceinline__ float2 rope_cos_sin_f(long long p, double f, float factor) {
  float s, c;
  sincospif(static_cast<float>(2.0 * rope_turn(p, f)), &s, &c);
  return make_float2(c * factor, s * factor);
}

__device__ __forceinline__ void load8(const __half* p, __half (&x)[8]) {
  *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void store8(__half* p, const __half (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(x);
}

// Scale, offset and codes of a vector of 128 spread over 8 lanes, 16 values a
// lane: the arithmetic of kv4_params / kv4_code.
__device__ __forceinline__ Quant4 kv4_params16(const float (&x)[16]) {
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int u = 1; u < 16; ++u) {
    mn = fminf(mn, x[u]);
    mx = fmaxf(mx, x[u]);
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  Quant4 r;
  r.s = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.0f));
  r.sf = __half2float(r.s);
  r.mn = mn;
  r.m = mn == 0.0f ? __float2half_rn(0.0f) : __float2half_rn(mn);
  return r;
}

// Codes of 16 values (a byte each) without a division: t = x - mn, and with
// u = fma(t, 1 / s, 1.5 * 2^23) the integer q0 that u holds in its low bits.  The
// remainder e = t - q0 s tells whether the binary32 quotient that kv4_code rounds
// can round to another integer: it is within 2^-20 of t / s (quotients under 16),
// so not while |e| < s (1/2 - 2^-18).  The few vectors with a value nearer to a
// border divide.  (16 divisions a lane took most of the time of a prompt's append.)
// u: the codes as 1.5 * 2^23 + code.
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
__device__ __forceinline__ void kv4_codes16(const float (&x)[16], const Quant4& p, float (&u)[16],
                                            uint32_t (&c)[4]) {
  const float r = p.sf > 0.0f ? __frcp_rn(p.sf) : 0.0f;
  const float edge = p.sf > 0.0f ? p.sf * (0.5f - 3.814697265625e-06f) : INFINITY;
  bool near = false;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float t = __fsub_rn(x[k], p.mn);
    u[k] = __fmaf_rn(t, r, kMagic);
    near |= !(fabsf(__fmaf_rn(-(u[k] - kMagic), p.sf, t)) < edge);
    u[k] = fminf(u[k], kMagic + 15.0f);
  }
  if (near) {
#pragma unroll
    for (int k = 0; k < 16; ++k) u[k] = kMagic + static_cast<float>(kv4_code(x[k], p));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = __byte_perm(__byte_perm(__float_as_uint(u[4 * k]), __float_as_uint(u[4 * k + 1]), 0x0040),
                       __byte_perm(__float_as_uint(u[4 * k + 2]), __float_as_uint(u[4 * k + 3]), 0x0040),
                       0x5410);
}
__device__ __forceinline__ int code_of(const uint32_t (&c)[4], int k) {
  return static_cast<int>((c[k >> 2] >> (8 * (k & 3))) & 15u);
}

// Replace the nibbles under `mask` of *word by those of `bits`.  The exclusive
// or changes no other nibble, so tokens of one word may be written at the same
// time by different threads.
__device__ __forceinline__ void put_nibbles(uint32_t* word, uint32_t bits, uint32_t mask) {
  const uint32_t diff = (*word ^ bits) & mask;
  if (diff) atomicXor(word, diff);
}

// Two kernels: by rows, for decode steps, where a row's block of 16 cache slots
// holds no other row; by blocks, for prompts, whose words are put together in
// shared memory and stored whole.  By rows a prompt's words take an atomic for
// each of their tokens: 8300 rows (32 / 8 heads) in 98 us against 51 by blocks;
// by blocks a decode step would leave 15 of 16 threads without a token.

// Measured: one row 4.4 us a call, 96 rows (64 / 8 heads) 7.1 us, both of them mostly the
// launch; 6751 prompt rows (32 / 8 heads, values returned, 173 MB) 49 us, 54% of the copy
// rate, by the latency between a head's loads, its arithmetic and the barrier.

// Grid (T, ceil((Hq + 2 Hkv) / 32)), 256 threads.  Eight lanes take one vector
// (a query, key or value head of the row), lane i its dimensions 16i .. 16i+15,
// which are word i of the runs that hold the token.
__global__ void __launch_bounds__(256) append_rows_kernel(const AppendArgs a) {
  __shared__ double2 cs[kHeadDim / 2];
  const int row = blockIdx.x, tid = threadIdx.x;
  const int vec = blockIdx.y * 32 + (tid >> 3), i = tid & 7;
  grid_dependency_wait();
  grid_launch_dependents();
  // the sequence of the row: the last one that starts at or before it
  int b = -1;
  for (int at = 0; at < a.B; at += 256) {
    const int c = at + tid;
    b += __syncthreads_count(c < a.B && a.q_start[c < a.B ? c : 0] <= row);
  }
  if (b < 0) return;
  const RowRange rr = rows_of(a.q_start, b, a.T);
  if (row < rr.first || row >= rr.first + rr.n) return;   // behind the last sequence
  const long long pos = position_of(a.seqlen[b], rr.n, row - rr.first);
  if (tid < (a.rot >> 1)) cs[tid] = rope_cos_sin(pos, a.inv_freq[tid], a.factor);
  __syncthreads();

  const int heads = a.Hq + 2 * a.Hkv;
  const bool mine = vec < heads;
  const __half* src = a.qkv + static_cast<size_t>(row) * a.ld + static_cast<size_t>(vec) * kHeadDim;
  __half x[2][8];
  if (mine) {
    load8(src + 16 * i, x[0]);
    load8(src + 16 * i + 8, x[1]);
  } else {
#pragma unroll
    for (int u = 0; u < 16; ++u) x[u >> 3][u & 7] = __float2half_rn(0.0f);
  }
  if (mine && vec < a.Hq + a.Hkv) {
    const int half_rot = a.rot >> 1;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int d0 = 16 * i + 8 * q;
      if (d0 >= a.rot) continue;
      if (a.interleaved) {
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
          const double2 w = cs[(d0 + u) >> 1];
          const double x0 = __half2float(x[q][u]), x1 = __half2float(x[q][u + 1]);
          x[q][u] = __float2half_rn(static_cast<float>(x0 * w.x - x1 * w.y));
          x[q][u + 1] = __float2half_rn(static_cast<float>(x1 * w.x + x0 * w.y));
        }
      } else {
        const bool low = d0 < half_rot;
        __half o[8];
        load8(src + (low ? d0 + half_rot : d0 - half_rot), o);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const double2 w = cs[(low ? d0 : d0 - half_rot) + u];
          const double xs = __half2float(x[q][u]), os = __half2float(o[u]);
          x[q][u] = __float2half_rn(static_cast<float>(xs * w.x + (low ? -os : os) * w.y));
        }
      }
    }
  }
  if (mine && vec < a.Hq) {
    __half* dst = a.q_out + (static_cast<size_t>(row) * a.Hq + vec) * kHeadDim + 16 * i;
    store8(dst, x[0]);
    store8(dst + 8, x[1]);
  }
  // keys and values (the shuffles need whole warps: eight-lane groups without a
  // vector quantize zeros)
  if (blockIdx.y * 32 + 32 <= a.Hq) return;
  float f[16];
#pragma unroll
  for (int u = 0; u < 16; ++u) f[u] = __half2float(x[u >> 3][u & 7]);
  const Quant4 p = kv4_params16(f);
  if (!mine || vec < a.Hq) return;
  const bool is_v = vec >= a.Hq + a.Hkv;
  const int hk = vec - a.Hq - (is_v ? a.Hkv : 0);
  uint32_t c[4];
  float u16[16];
  kv4_codes16(f, p, u16, c);
  __half* hat = is_v ? a.v_hat : a.k_hat;
  if (hat) {
    const float m = __half2float(p.m);
    hat += (static_cast<size_t>(row) * a.Hkv + hk) * kHeadDim + 16 * i;
#pragma unroll
    for (int u = 0; u < 16; ++u)
      x[u >> 3][u & 7] = __float2half_rn(fmaf(u16[u] - kMagic, p.sf, m));
    store8(hat, x[0]);
    store8(hat + 8, x[1]);
  }
  const int ppb = a.page >> 4;
  if (pos < 0 || pos >= static_cast<long long>(a.width) * a.page) return;   // no slot
  const int blk = pool_block(a.table + static_cast<size_t>(b) * a.width, static_cast<int>(pos >> 4),
                             ppb, a.pages, a.Hkv, hk);
  if (blk < 0) return;
  const int t = static_cast<int>(pos & 15);
  if (i == 0)
    *reinterpret_cast<__half2*>(a.sc + static_cast<size_t>(blk) * 64 + 4 * t + (is_v ? 2 : 0)) =
        __halves2half2(p.s, p.m);
  if (!is_v) {
    // token t: gid = t & 7, nibbles j0 = t >> 3; dimension 16 i + 2 tig + e + 8 j1
    uint32_t* w = reinterpret_cast<uint32_t*>(a.kc + static_cast<size_t>(blk) * 1024) +
                  (t & 7) * 32 + i;
    const int sh = (t >> 3) * 4;
#pragma unroll
    for (int tig = 0; tig < 4; ++tig) {
      uint32_t bits = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int j1 = 0; j1 < 2; ++j1)
          bits |= static_cast<uint32_t>(code_of(c, 2 * tig + e + 8 * j1)) << (16 * e + 8 * j1);
      put_nibbles(w + tig * 8, bits << sh, 0x0f0f0f0fu << sh);
    }
  } else {
    // token t: tig = (t & 7) >> 1, e = t & 1, j1 = t >> 3; dimension
    // 16 i + gid + 8 j0
    uint32_t* w = reinterpret_cast<uint32_t*>(a.vc + static_cast<size_t>(blk) * 1024) +
                  ((t & 7) >> 1) * 8 + i;
    const int sh = 16 * (t & 1) + 8 * (t >> 3);
#pragma unroll
    for (int gid = 0; gid < 8; ++gid) {
      const uint32_t bits = static_cast<uint32_t>(code_of(c, gid) | (code_of(c, gid + 8) << 4));
      put_nibbles(w + gid * 32, bits << sh, 0xffu << sh);
    }
  }
}

// By blocks: grid slots x (KV head groups + query head groups), the groups of a slot
// next to each other (the KV groups' arithmetic then runs beside the query groups'
// copies), 256 threads.  A slot is one block of 16 positions of one sequence: sequence b owns the slots from
// q_start[b] / 16 + 2 b on, enough for its rows however they lie in blocks.  Thread
// (half, token, i) keeps its token's rotation for its 16 dimensions (8 pairs) over
// all heads.  Of the KV groups, half 0 takes keys and half 1 values.
__device__ __forceinline__ int block_slot(int first, int b) { return (first >> 4) + 2 * b; }

__global__ void __launch_bounds__(256, 4)
append_blocks_kernel(const AppendArgs a, int groups, int kv_groups, int kv_per, int q_per) {
  __shared__ uint8_t s_code[2][2][16][kHeadDim];       // [turn][K, V][token][dimension]
  __shared__ double2 s_cs[8][128];                     // [pair of 8][8 token + i]: rotations
  float2 (*s_csf)[128] = reinterpret_cast<float2 (*)[128]>(s_cs);
  const int tid = threadIdx.x, half = tid >> 7, tok = (tid >> 3) & 15, i = tid & 7;
  grid_dependency_wait();
  grid_launch_dependents();
  const int slot = blockIdx.x / groups, group = blockIdx.x - slot * groups;
  int b = -1;      // the last sequence whose slots start at or before this one
  for (int at = 0; at < a.B; at += 256) {
    const int c = at + tid;
    b += __syncthreads_count(c < a.B && block_slot(a.q_start[c < a.B ? c : 0], c) <= slot);
  }
  if (b < 0) return;
  const RowRange rr = rows_of(a.q_start, b, a.T);
  const long long pos0 = position_of(a.seqlen[b], rr.n, 0);
  const long long blk = (pos0 >> 4) + (slot - block_slot(rr.first, b));
  const int lo = static_cast<int>(blk * 16 < pos0 ? pos0 - blk * 16 : 0);     // tokens of the
  const long long left = pos0 + rr.n - blk * 16;                              // block: lo .. hi - 1
  const int hi = left < 16 ? static_cast<int>(left) : 16;
  if (rr.n == 0 || hi <= lo) return;
  const bool mine = tok >= lo && tok < hi;
  const long long pos = blk * 16 + tok;
  const int row = rr.first + (mine ? static_cast<int>(pos - pos0) : 0);
  const __half* src = a.qkv + static_cast<size_t>(row) * a.ld;

  // the thread's two chunks of 8 dimensions, rotated against each other (half
  // layout) or each in itself
  const int pairs8 = a.rot >> 4;               // groups of 8 pairs
  const bool turns = i < pairs8;
  int d0 = 16 * i, d1 = 16 * i + 8;
  if (!a.interleaved && turns) {
    d0 = 8 * i;
    d1 = (a.rot >> 1) + 8 * i;
  }

  // the block's rotations, spread over the threads
  const bool queries = group >= kv_groups;
  for (int k = tid; k < 8 * a.rot; k += 256) {         // 16 tokens x rot / 2 pairs
    const int t = k / (a.rot >> 1), j = k - t * (a.rot >> 1);
    if (t < lo || t >= hi) continue;
    if (queries)
      s_csf[j & 7][8 * t + (j >> 3)] =
          rope_cos_sin_f(blk * 16 + t, a.inv_freq[j], static_cast<float>(a.factor));
    else
      s_cs[j & 7][8 * t + (j >> 3)] = rope_cos_sin(blk * 16 + t, a.inv_freq[j], a.factor);
  }
  if (queries) {
    // ---------------------------------------------------------------- queries
    __syncthreads();
    const int h0 = (group - kv_groups) * q_per;
    const int h1 = h0 + q_per < a.Hq ? h0 + q_per : a.Hq;
    if (!mine) return;
    float2 w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) w[u] = turns ? s_csf[u][tid & 127] : make_float2(1.0f, 0.0f);
#pragma unroll 4
    for (int h = h0 + half; h < h1; h += 2) {
      __half x0[8], x1[8];
      load8(src + static_cast<size_t>(h) * kHeadDim + d0, x0);
      load8(src + static_cast<size_t>(h) * kHeadDim + d1, x1);
      if (turns) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          __half& p = a.interleaved ? (u < 4 ? x0 : x1)[(2 * u) & 7] : x0[u];
          __half& q = a.interleaved ? (u < 4 ? x0 : x1)[(2 * u + 1) & 7] : x1[u];
          const float y0 = __half2float(p), y1 = __half2float(q);
          p = __float2half_rn(fmaf(y0, w[u].x, -(y1 * w[u].y)));
          q = __float2half_rn(fmaf(y1, w[u].x, y0 * w[u].y));
        }
      }
      __half* dst = a.q_out + (static_cast<size_t>(row) * a.Hq + h) * kHeadDim;
      store8(dst + d0, x0);
      store8(dst + d1, x1);
    }
    return;
  }
  // ------------------------------------------------------------ keys and values
  const int h0 = group * kv_per;
  const int h1 = h0 + kv_per < a.Hkv ? h0 + kv_per : a.Hkv;
  if (half == 1) {
    d0 = 16 * i;
    d1 = 16 * i + 8;
  }
  const bool held = blk >= 0 && blk < ((static_cast<long long>(a.width) * a.page) >> 4);
  // the block of head h0 in the pool; the next heads' follow
  const int ppb = a.page >> 4;
  const int at0 = held ? pool_block(a.table + static_cast<size_t>(b) * a.width,
                                    static_cast<int>(blk), ppb, a.pages, a.Hkv, h0) : -1;
  const __half* kv = src + static_cast<size_t>(a.Hq + half * a.Hkv) * kHeadDim;
  // tokens of the block that this call writes, a bit each
  const uint32_t cover = (0xffffu >> (16 - hi)) & (0xffffu << lo);
  uint4 n0 = make_uint4(0u, 0u, 0u, 0u), n1 = n0;
  auto fetch = [&](int h) {
    if (mine && h < h1) {
      n0 = *reinterpret_cast<const uint4*>(kv + static_cast<size_t>(h) * kHeadDim + d0);
      n1 = *reinterpret_cast<const uint4*>(kv + static_cast<size_t>(h) * kHeadDim + d1);
    }
  };
  fetch(h0);
  __syncthreads();       // the rotations
  for (int h = h0; h < h1; ++h) {
    __half x0[8], x1[8];
    *reinterpret_cast<uint4*>(x0) = n0;
    *reinterpret_cast<uint4*>(x1) = n1;
    fetch(h + 1);
    if (half == 0 && turns && mine) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        __half& p = a.interleaved ? (u < 4 ? x0 : x1)[(2 * u) & 7] : x0[u];
        __half& q = a.interleaved ? (u < 4 ? x0 : x1)[(2 * u + 1) & 7] : x1[u];
        const double y0 = __half2float(p), y1 = __half2float(q);
        const double2 w = s_cs[u][tid];
        p = __float2half_rn(static_cast<float>(y0 * w.x - y1 * w.y));
        q = __float2half_rn(static_cast<float>(y1 * w.x + y0 * w.y));
      }
    }
    float f[16];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      f[u] = __half2float(x0[u]);
      f[8 + u] = __half2float(x1[u]);
    }
    const Quant4 p = kv4_params16(f);
    uint32_t c[4];                           // a byte a code
    float u16[16];
    kv4_codes16(f, p, u16, c);
    __half* hat = half ? a.v_hat : a.k_hat;
    if (hat && mine) {
      const float m = __half2float(p.m);
      hat += (static_cast<size_t>(row) * a.Hkv + h) * kHeadDim;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        x0[u] = __float2half_rn(fmaf(u16[u] - kMagic, p.sf, m));
        x1[u] = __float2half_rn(fmaf(u16[8 + u] - kMagic, p.sf, m));
      }
      store8(hat + d0, x0);
      store8(hat + d1, x1);
    }
    if (at0 < 0) continue;                   // (the same for the whole CTA)
    const int at = at0 + (h - h0) * ppb;
    uint8_t (*code)[16][kHeadDim] = s_code[(h - h0) & 1];
    *reinterpret_cast<uint2*>(&code[half][tok][d0]) = make_uint2(c[0], c[1]);
    *reinterpret_cast<uint2*>(&code[half][tok][d1]) = make_uint2(c[2], c[3]);
    if (i == 0 && mine)
      *reinterpret_cast<__half2*>(a.sc + static_cast<size_t>(at) * 64 + 4 * tok + 2 * half) =
          __halves2half2(p.s, p.m);
    __syncthreads();     // (the other turn's codes are read until the next one)
    // word w of run (gid, tig): gid the warp
    const int word = tid & 7, tig = (tid >> 3) & 3, gid = tid >> 5;
    uint32_t kw = 0, vw = 0;
#pragma unroll
    for (int j0 = 0; j0 < 2; ++j0)
#pragma unroll
      for (int j1 = 0; j1 < 2; ++j1) {
        // K: two dimensions (e) of one token
        const uint32_t two = *reinterpret_cast<const uint16_t*>(
            &code[0][gid + 8 * j0][16 * word + 2 * tig + 8 * j1]);
        kw |= __byte_perm(two, 0u, 0x4140) << (4 * j0 + 8 * j1);
        // V: two tokens (e) of one dimension
        const int d = 16 * word + gid + 8 * j0;
        const uint32_t e0 = code[1][2 * tig + 8 * j1][d], e1 = code[1][2 * tig + 1 + 8 * j1][d];
        vw |= (e0 | (e1 << 16)) << (4 * j0 + 8 * j1);
      }
    uint32_t* kd = reinterpret_cast<uint32_t*>(a.kc + static_cast<size_t>(at) * 1024) + tid;
    uint32_t* vd = reinterpret_cast<uint32_t*>(a.vc + static_cast<size_t>(at) * 1024) + tid;
    if (cover == 0xffffu) {
      *kd = kw;
      *vd = vw;
    } else {
      uint32_t km = 0, vm = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if ((cover >> (gid + 8 * j)) & 1u) km |= 0x0f0f0f0fu << (4 * j);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if ((cover >> (2 * tig + e + 8 * j)) & 1u) vm |= 0xffu << (16 * e + 8 * j);
      }
      if (km) put_nibbles(kd, kw, km);
      if (vm) put_nibbles(vd, vw, vm);
    }
  }
}

}  // namespace

int check_paged_shape(int pages, int Hkv, int page, int d) {
  if (pages <= 0 || Hkv <= 0 || page <= 0) return QOQ_ERR_INVALID_ARG;
  if (d != kHeadDim || page % 16 != 0) return QOQ_ERR_UNSUPPORTED;
  if (Hkv > 65535) return QOQ_ERR_UNSUPPORTED;
  // block numbers of 16 tokens are 32-bit
  if (static_cast<long long>(Hkv) * (page / 16) > 0x7fffffffLL / pages) return QOQ_ERR_UNSUPPORTED;
  return QOQ_OK;
}

int check_batch(int T, int B, int width, int page) {
  if (T < 0 || B < 0 || width <= 0) return QOQ_ERR_INVALID_ARG;
  // tokens are 32-bit numbers, also those of a tile that begins at a sequence's last one
  if (width > (0x7fffffff - 4095) / page) return QOQ_ERR_UNSUPPORTED;
  return QOQ_OK;
}

}  // namespace qoq

using namespace qoq;

extern "C" int qoq_kv4_paged_bytes(int pages, int Hkv, int page, int d, size_t* k_bytes,
                                   size_t* v_bytes, size_t* scale_bytes) {
  if (int st = check_paged_shape(pages, Hkv, page, d)) return st;
  const size_t blocks = static_cast<size_t>(pages) * Hkv * (page / 16);
  if (k_bytes) *k_bytes = blocks * 1024;
  if (v_bytes) *v_bytes = blocks * 1024;
  if (scale_bytes) *scale_bytes = blocks * 128;
  return QOQ_OK;
}

extern "C" int qoq_kv4_paged_append(const void* qkv, size_t ld, int T, int Hq, int Hkv, int d,
                                    const int* q_start, const int* seqlen, int B,
                                    const int* block_table, int width, int pages, int page,
                                    const double* inv_freq, int rot, int interleaved,
                                    double rope_factor, void* q_out, uint8_t* k_codes,
                                    uint8_t* v_codes, void* scales, void* k_values,
                                    void* v_values, void* stream) {
  if (Hq <= 0) return QOQ_ERR_INVALID_ARG;
  if (int st = check_paged_shape(pages, Hkv, page, d)) return st;
  if (int st = check_batch(T, B, width, page)) return st;
  if (Hq > 65535) return QOQ_ERR_UNSUPPORTED;
  if (rot < 0 || rot > kHeadDim || (rot > 0 && !inv_freq)) return QOQ_ERR_INVALID_ARG;
  if (rot % 16 != 0) return QOQ_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return QOQ_ERR_INVALID_ARG;
  if (ld < (static_cast<size_t>(Hq) + 2 * static_cast<size_t>(Hkv)) * kHeadDim || ld % 8 != 0)
    return QOQ_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return QOQ_OK;
  if (!qkv || !q_start || !seqlen || !block_table || !q_out || !k_codes || !v_codes || !scales)
    return QOQ_ERR_INVALID_ARG;
  if (!k_values != !v_values) return QOQ_ERR_INVALID_ARG;
  if (!aligned16(qkv) || !aligned16(q_out) || !aligned16(k_codes) || !aligned16(v_codes) ||
      !aligned16(scales) || !aligned16(k_values) || !aligned16(v_values) ||
      (reinterpret_cast<uintptr_t>(inv_freq) & 7u) || !aligned4(q_start) || !aligned4(seqlen) ||
      !aligned4(block_table))
    return QOQ_ERR_INVALID_ARG;
  if (int st = check_device()) return st;
  AppendArgs a;
  a.qkv = static_cast<const __half*>(qkv);
  a.ld = ld;
  a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.B = B;
  a.q_start = q_start; a.seqlen = seqlen; a.table = block_table;
  a.width = width; a.pages = pages; a.page = page;
  a.inv_freq = inv_freq; a.rot = rot; a.interleaved = interleaved; a.factor = rope_factor;
  a.q_out = static_cast<__half*>(q_out);
  a.kc = k_codes; a.vc = v_codes; a.sc = static_cast<__half*>(scales);
  a.k_hat = static_cast<__half*>(k_values); a.v_hat = static_cast<__half*>(v_values);
  if (T >= static_cast<long long>(kBlockRows) * B) {
    // heads to a CTA: enough CTAs for every SM to hold some, and few enough that the
    // angles of a block are not computed for every head
    const int slots = T / 16 + 2 * B;
    const long long room = 6LL * sm_count();
    int kv_per = static_cast<int>(static_cast<long long>(slots) * Hkv / room);
    kv_per = kv_per < 1 ? 1 : (kv_per > 4 ? 4 : kv_per);
    const int q_per = 8 * kv_per;
    const int kv_groups = (Hkv + kv_per - 1) / kv_per;
    const int all = kv_groups + (Hq + q_per - 1) / q_per;
    const long long ctas = static_cast<long long>(slots) * all;
    if (ctas <= 0x7fffffffLL)
      return launch_dependent(append_blocks_kernel, dim3(static_cast<unsigned>(ctas)), 256, 0,
                              as_stream(stream), a, all, kv_groups, kv_per, q_per);
  }
  const unsigned groups = static_cast<unsigned>((Hq + 2 * Hkv + 31) / 32);
  return launch_dependent(append_rows_kernel, dim3(static_cast<unsigned>(T), groups), 256, 0,
                          as_stream(stream), a);
}
