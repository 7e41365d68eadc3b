// What the paged attention kernels share: arguments, the launch plan and the
// output store.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "qoq_internal.h"

namespace qoq {

struct PagedArgs {
  const __half* Q;          // T rows of Hq heads, ldq elements apart
  size_t ldq;
  const uint8_t* kc;
  const uint8_t* vc;
  const __half* sc;
  const int* q_start;       // B + 1
  const int* seqlen;        // B
  const int* table;         // B x width page numbers
  int T, B, Hq, Hkv, g, width, pages, page, max_q;
  float scale;
  __half* out;              // T x Hq x 128
  int2* meta;               // decode: per (sequence, KV head), its first and last CTA;
                            // prompt: per (slot, KV head), its first part and their number
  float* parts;             // partial results, kPartFloats a row
};

// A sequence with at most 4 nt rows (query tokens x g) runs in the decode
// kernel, a longer one in the prompt kernel.
struct PagedPlan {
  int nt;                   // four-row tiles of the decode kernel: 1, 2, 4, or 0 (not launched)
  int grid;                 // its CTAs
  bool combine;             // a (sequence, KV head) pair may lie in several of them
  bool prompt;              // sequences with more rows may be there
  int tiles;                // prompt: row slots of the batch
  int prompt_target, prompt_grid;
  bool prompt_combine;
  size_t meta_off, parts_off, prompt_units_off, prompt_meta_off, prompt_parts_off, bytes;
  size_t take(size_t n) {   // the workspace's next n bytes
    const size_t off = bytes;
    bytes += (n + 255) / 256 * 256;
    return off;
  }
};
PagedPlan paged_plan(int T, int B, int Hq, int Hkv, int width, int page, int max_q);
void plan_prompt(PagedPlan& p, int T, int B, int Hq, int Hkv, int width, int page);

struct PromptUnit;
int launch_paged_prompt(const PagedArgs& a, const PagedPlan& p, const PromptUnit* units,
                        cudaStream_t s);

// A row's running reference.  Token t has the probability p = 2^(x_t - ref) and enters the
// product with V as the FP16 weight w = p s_V; sums of p stay in FP32, so the reference is
// free to keep the weights, not the probabilities, in FP16's range: the largest w of a row
// is never above 2^kWeightTop, and a reference that is set puts it at 2^kWeightSet.  From
// there down to 2^-14 weights have all their bits, and what is lost below is 2^-35 of the
// largest: values may be of any size, and a row may have nearly all its weight on one token
// and thousands of others 2^-20 below.  (A reference at the largest score lost them: of values of
// size 1e-3, 4096 tokens, all but one 12 powers of two below it, 6.5% of the output in the
// prompt kernel and 0.26% in the single-token kernel; now FP16's rounding alone, 2.1e-4.)
// Probabilities reach 2^(kWeightTop + 24) where s_V is FP16's smallest or 0, far inside FP32.
constexpr float kWeightTop = 15.9f;      // 61147: FP16 ends at 65504
constexpr float kWeightSet = 10.0f;      // a rise by 5.9 then needs no new reference
// log2 of a value scale's size for that: of 0 and NaN the smallest scale's, of infinity the
// largest's.  (Scales that append writes are not negative; a caller's own may be.)
__device__ __forceinline__ float log2_scale(float s) {
  return __log2f(fminf(fmaxf(fabsf(s), 5.9604645e-08f), 65504.0f));
}

// The reference that a partial result with the sum l is merged by: -inf for one without
// tokens, which is left out, and NaN for one that is NaN, which no merge may leave out (its
// factor is then NaN; fmaxf passes over it).
__device__ __forceinline__ float part_reference(float l, float ref) {
  return l == 0.0f ? -INFINITY : (l != l ? l : ref);
}

// 4 or 8 outputs times `f`, rounded to FP16.
__device__ __forceinline__ void store_row4(__half* dst, float4 v, float f) {
  const __half2 o[2] = {__floats2half2_rn(v.x * f, v.y * f), __floats2half2_rn(v.z * f, v.w * f)};
  *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(o);
}
__device__ __forceinline__ void store_row8(__half* dst, const float (&v)[8], float f) {
  __half2 o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = __floats2half2_rn(v[2 * k] * f, v[2 * k + 1] * f);
  *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
}

}  // namespace qoq
