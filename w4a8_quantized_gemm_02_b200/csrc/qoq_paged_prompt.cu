// Attention over a paged 4-bit KV cache for the sequences with more rows than
// the decode kernel takes: chunks of a prompt.  A warp takes one row (query
// token and head) and walks the tokens that it sees.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "qoq.h"
#include "qoq_attn.cuh"
#include "qoq_device.cuh"
#include "qoq_internal.h"
#include "qoq_kv4.cuh"
#include "qoq_paged.h"

namespace qoq {
namespace {

__global__ void __launch_bounds__(256) paged_rows_kernel(const PagedArgs a, int min_rows) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  const long long x = static_cast<long long>(blockIdx.x) * 8 + warp;
  const int row = static_cast<int>(x / a.Hq), h = static_cast<int>(x - static_cast<long long>(row) * a.Hq);
  if (row >= a.T) return;
  int lo = 0, hi = a.B;      // the last sequence that starts at or before the row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= row) lo = mid;
    else hi = mid;
  }
  const int b = lo;
  const RowRange rr = rows_of(a.q_start, b, a.T);
  if (row < rr.first || row >= rr.first + rr.n) return;
  if (rr.n > a.max_q || rr.n * a.g < min_rows) return;
  const int hk = h / a.g;
  const int n = visible(position_of(a.seqlen[b], rr.n, row - rr.first),
                        clamp_len(a.seqlen[b], a.width * a.page));
  const int w = lane >> 2, tig = lane & 3;
  const __half* q = a.Q + row * a.ldq + static_cast<size_t>(h) * kHeadDim + 16 * w + 2 * tig;
  const float q0 = __half2float(q[0]), q1 = __half2float(q[1]), q2 = __half2float(q[8]),
              q3 = __half2float(q[9]);
  const float scale2 = a.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int t = 0; t < n; ++t) {
    const int blk = pool_block(a.table + static_cast<size_t>(b) * a.width, t >> 4, a.page >> 4,
                               a.pages, a.Hkv, hk);
    if (blk < 0) continue;
    const int j = (t >> 3) & 1, gid = t & 7, tt = (t & 7) >> 1, e = t & 1;
    const __half* sc = a.sc + static_cast<size_t>(blk) * 64 + 4 * (t & 15);
    const uint32_t kw = reinterpret_cast<const uint32_t*>(
        a.kc + static_cast<size_t>(blk) * 1024)[(gid * 4 + tig) * 8 + w] >> (4 * j);
    const uint32_t* vw = reinterpret_cast<const uint32_t*>(a.vc + static_cast<size_t>(blk) * 1024) +
                         (2 * tig * 4 + tt) * 8 + w;
    const uint32_t v0 = vw[0] >> (16 * e + 8 * j), v1 = vw[32] >> (16 * e + 8 * j);
    const float sk = __half2float(sc[0]), mk = __half2float(sc[1]);
    const float sv = __half2float(sc[2]), mv = __half2float(sc[3]);
    float s = q0 * fmaf(static_cast<float>(kw & 15), sk, mk) +
              q1 * fmaf(static_cast<float>((kw >> 16) & 15), sk, mk) +
              q2 * fmaf(static_cast<float>((kw >> 8) & 15), sk, mk) +
              q3 * fmaf(static_cast<float>((kw >> 24) & 15), sk, mk);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= scale2;
    const float top = fmaxf(m, s);
    const float al = fast_exp2(m - top), p = fast_exp2(s - top);
    m = top;
    l = fmaf(l, al, p);
    o[0] = fmaf(o[0], al, p * fmaf(static_cast<float>(v0 & 15), sv, mv));
    o[1] = fmaf(o[1], al, p * fmaf(static_cast<float>((v0 >> 4) & 15), sv, mv));
    o[2] = fmaf(o[2], al, p * fmaf(static_cast<float>(v1 & 15), sv, mv));
    o[3] = fmaf(o[3], al, p * fmaf(static_cast<float>((v1 >> 4) & 15), sv, mv));
  }
  const float inv = l == 0.0f ? 0.0f : __frcp_rn(l);
  // dimensions 16 w + 2 tig + {0, 8, 1, 9}
  __half* dst = a.out + (static_cast<size_t>(row) * a.Hq + h) * kHeadDim + 16 * w + 2 * tig;
  dst[0] = __float2half_rn(o[0] * inv);
  dst[8] = __float2half_rn(o[1] * inv);
  dst[1] = __float2half_rn(o[2] * inv);
  dst[9] = __float2half_rn(o[3] * inv);
}

}  // namespace

int launch_paged_prompt(const PagedArgs& a, const PagedPlan&, int min_rows, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.T) * a.Hq;
  return launch_dependent(paged_rows_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), 256, 0, s,
                          a, min_rows);
}

}  // namespace qoq
