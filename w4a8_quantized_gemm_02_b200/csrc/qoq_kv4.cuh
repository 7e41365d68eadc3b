// What the kernels over the 4-bit KV cache share: the cache format (see the
// public header), its quantizer, and the warp-level tensor-core pieces.
#pragma once

#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

namespace qoq {

constexpr int kHeadDim = 128;
// A partial result of an attention split, per row: max, sum, two unused words,
// 128 outputs (the outputs start 16-byte aligned).
constexpr int kPartFloats = 4 + kHeadDim;

struct Quant4 {
  __half s, m;
  float sf, mn;
};

// Scale and offset of the warp's vector from each lane's four values.
__device__ __forceinline__ Quant4 kv4_params(const float (&x)[4]) {
  float mn = fminf(fminf(x[0], x[1]), fminf(x[2], x[3]));
  float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  Quant4 r;
  r.s = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.0f));
  r.sf = __half2float(r.s);
  r.mn = mn;
  r.m = mn == 0.0f ? __float2half_rn(0.0f) : __float2half_rn(mn);   // exact: mn is an FP16 value
  return r;
}

__device__ __forceinline__ int kv4_code(float x, const Quant4& p) {
  if (!(p.sf > 0.0f)) return 0;
  const int c = __float2int_rn(__fdiv_rn(__fsub_rn(x, p.mn), p.sf));
  return c < 0 ? 0 : (c > 15 ? 15 : c);
}

// Nibble positions of a block's codes: the (token, dimension) of word w
// (0..7) of run r (0..31), nibble p, for K and for V.
__device__ __forceinline__ void k_slot(int r, int w, int p, int& tok, int& dim) {
  const int gid = r >> 2, tig = r & 3, j = p & 3, e = p >> 2;
  tok = gid + 8 * (j & 1);
  dim = 16 * w + 2 * tig + e + 8 * (j >> 1);
}
__device__ __forceinline__ void v_slot(int r, int w, int p, int& tok, int& dim) {
  const int gid = r >> 2, tig = r & 3, j = p & 3, e = p >> 2;
  tok = 2 * tig + e + 8 * (j >> 1);
  dim = 16 * w + gid + 8 * (j & 1);
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// (x & m) | o in one operation.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t o) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(x), "r"(m), "r"(o));
  return d;
}

// 8x8 transpose of 16-bit elements across the warp: lane 4 r + c holds row r,
// columns 2c and 2c + 1, before and after.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 2^x by the SFU's approximation (relative error ~2^-22, far inside the
// attention's tolerance); 2^-inf = 0.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Slot of the 16-byte chunk c of a block of codes in shared memory: lane l
// reads chunks 2l and 2l + 1 (its run) without bank conflicts.
__device__ __forceinline__ int chunk_slot(int c) { return c ^ ((c >> 3) & 1); }

}  // namespace qoq
