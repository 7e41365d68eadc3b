// Low-rank adapters of many requests beside a shared projection:
//     out[t] = fp16(Y[t] + scaling[a] * B_a (A_a x_t)),   a = ids[t].
//
// Two kernels.  "shrink": h[t] = A_a x_t, R values a row, K long: a CTA takes 32
// rows, finds the distinct adapters among them and multiplies each adapter's
// rows (gathered) with a slice of K; slices leave FP32 partial sums.  "expand":
// a CTA takes 16 or 64 rows and 256 columns, adds the slices up in order, and
// accumulates over its distinct adapters with the other adapters' rows set to
// zero, so that every output is formed once, from Y and the whole sum.
//
// Both multiply on mma.sync m16n8k16 (FP16, FP32 sums): the work is a few
// operations a byte, so what counts is that adapters and rows stream from
// memory; operands go from global memory to registers without shared memory.
// The k order within 32 is permuted the same way in both operands, so that each
// lane loads 16 contiguous bytes of a row for two MMAs.
//
// Rounding.  h is kept in FP32; for the second product it is scaled by a power
// of two to its row's largest value and split in two FP16 numbers (2^-22 of that
// value is lost), so the output's own rounding is the only one that shows.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qoq.h"
#include "qoq_device.cuh"
#include "qoq_internal.h"
#include "qoq_kv4.cuh"

namespace qoq {
namespace {

constexpr int kShrinkRows = 32;
constexpr int kShrinkWarps = 4;
constexpr int kExpandWarps = 8;
constexpr int kExpandCols = 32 * kExpandWarps;
constexpr int kMaxRank = 128;

struct LoraArgs {
  const __half* X;        // T x K
  const __half* A;        // n x R x K
  const __half* Bm;       // n x N x R
  const int* ids;         // T
  const float* scaling;   // n
  const __half* Y;        // T x N
  __half* out;            // T x N
  float* h;               // [slices][T][R]
  int T, K, N, R, n, slices, k_slice;
};

__device__ __forceinline__ uint4 load16(const __half* p, bool ok) {
  return ok ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
}

// h of `rows` (this lane's row of each 8-row tile) for ranks 0 .. 16 MT - 1 over
// the k-steps of this warp, reduced over the CTA's warps and stored.
template <int MT, int NT>
__device__ __forceinline__ void shrink_tile(const LoraArgs& a, int adapter, const int (&row)[NT],
                                            int count, int row0, uint32_t group, int k0, int k1,
                                            float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const __half* ar = a.A + (static_cast<size_t>(adapter) * a.R + gid) * a.K + 8 * tig;
  float acc[MT][NT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[mt][nt][k] = 0.0f;
#pragma unroll 2
  for (int k = k0 + 32 * warp; k < k1; k += 32 * kShrinkWarps) {
    uint4 x[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      x[nt] = load16(a.X + static_cast<size_t>(row[nt] < 0 ? 0 : row[nt]) * a.K + k + 8 * tig,
                     row[nt] >= 0);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const uint4 w0 = load16(ar + static_cast<size_t>(16 * mt) * a.K + k, 16 * mt + gid < a.R);
      const uint4 w1 =
          load16(ar + static_cast<size_t>(16 * mt + 8) * a.K + k, 16 * mt + 8 + gid < a.R);
      const uint32_t f0[4] = {w0.x, w1.x, w0.y, w1.y}, f1[4] = {w0.z, w1.z, w0.w, w1.w};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_16816(acc[mt][nt], f0, x[nt].x, x[nt].y);
        mma_16816(acc[mt][nt], f1, x[nt].z, x[nt].w);
      }
    }
  }
  // warps 2, 3 -> 0, 1, then 1 -> 0, always in this order
  constexpr int kTile = MT * NT * 4;
#pragma unroll
  for (int half = kShrinkWarps / 2; half > 0; half >>= 1) {
    __syncthreads();
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int i = 0; i < kTile; ++i)
        red[((warp - half) * kTile + i) * 32 + lane] = acc[i / (4 * NT)][(i / 4) % NT][i % 4];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int i = 0; i < kTile; ++i)
        acc[i / (4 * NT)][(i / 4) % NT][i % 4] += red[(warp * kTile + i) * 32 + lane];
    }
  }
  if (warp != 0) return;
  float* h = a.h + static_cast<size_t>(blockIdx.z) * a.T * a.R;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int q = 8 * nt + 2 * tig + c;      // the q-th row of the adapter
      if (q >= count) continue;
      const int t = row0 + static_cast<int>(__fns(group, 0, q + 1));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int rank = 16 * mt + 8 * r + gid;
          if (rank < a.R) h[static_cast<size_t>(t) * a.R + rank] = acc[mt][nt][2 * r + c];
        }
    }
}

// Grid (row tiles, adapter slots, K slices).
template <int MT>
__global__ void __launch_bounds__(32 * kShrinkWarps) lora_shrink_kernel(const LoraArgs a) {
  __shared__ float red[(kShrinkWarps / 2) * MT * 4 * 4 * 32];
  const int lane = threadIdx.x & 31, gid = lane >> 2;
  grid_dependency_wait();
  grid_launch_dependents();
  const int row0 = blockIdx.x * kShrinkRows;
  const int mine = row0 + lane;
  int id = mine < a.T ? a.ids[mine] : -1;
  if (id < 0 || id >= a.n) id = -1;
  const uint32_t same = __match_any_sync(0xffffffffu, id);
  uint32_t leaders = __ballot_sync(0xffffffffu, id >= 0 && (same & ((1u << lane) - 1u)) == 0u);
  const int k0 = blockIdx.z * a.k_slice;
  const int k1 = k0 + a.k_slice < a.K ? k0 + a.k_slice : a.K;
  for (int slot = 0; leaders != 0u; ++slot) {
    const int first = __ffs(leaders) - 1;
    leaders &= leaders - 1u;
    if (slot % gridDim.y != blockIdx.y) continue;
    const int adapter = __shfl_sync(0xffffffffu, id, first);
    const uint32_t group = __shfl_sync(0xffffffffu, same, first);
    const int count = __popc(group);
    if (count <= 8) {
      int row[1];
      row[0] = gid < count ? row0 + static_cast<int>(__fns(group, 0, gid + 1)) : -1;
      shrink_tile<MT, 1>(a, adapter, row, count, row0, group, k0, k1, red);
    } else {
      int row[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
        row[nt] = 8 * nt + gid < count ? row0 + static_cast<int>(__fns(group, 0, 8 * nt + gid + 1))
                                       : -1;
      shrink_tile<MT, 4>(a, adapter, row, count, row0, group, k0, k1, red);
    }
  }
}

// Grid (ceil(N / 256), row tiles of TM): warp w takes columns 32 w .. of the
// CTA's 256 and all TM rows.
template <int TM>
__global__ void __launch_bounds__(32 * kExpandWarps) lora_expand_kernel(const LoraArgs a) {
  extern __shared__ __align__(16) __half hs[];     // [TM][2][pitch]: high and low parts
  __shared__ int s_id[TM];
  __shared__ int s_lead[TM];
  __shared__ int s_leads;
  __shared__ float s_factor[TM];
  constexpr int MT = TM / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int Rp = (a.R + 31) & ~31, pitch = Rp + 8;
  const int row0 = blockIdx.y * TM;
  const int n0 = blockIdx.x * kExpandCols + 32 * warp;
  grid_dependency_wait();
  if (threadIdx.x < TM) {
    const int t = row0 + threadIdx.x;
    const int id = t < a.T ? a.ids[t] : -1;
    s_id[threadIdx.x] = id >= 0 && id < a.n ? id : -1;
  }
  __syncthreads();
  if (warp == 0) {
    int found = 0;
    for (int r0 = 0; r0 < TM; r0 += 32) {
      const int r = r0 + lane;
      const int id = r < TM ? s_id[r] : -1;
      bool lead = id >= 0;
      for (int e = 0; e < r && lead; ++e) lead = s_id[e] != id;
      const uint32_t m = __ballot_sync(0xffffffffu, lead);
      if (lead) s_lead[found + __popc(m & ((1u << lane) - 1u))] = id;
      found += __popc(m);
    }
    if (lane == 0) s_leads = found;
  }
  // h: the slices added in order, a warp a row, a lane every 32nd rank
  for (int r = warp; r < TM; r += kExpandWarps) {
    const int id = s_id[r];
    float v[kMaxRank / 32];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kMaxRank / 32; ++i) {
      const int rank = 32 * i + lane;
      float s = 0.0f;
      if (id >= 0 && rank < a.R) {
        const float* p = a.h + static_cast<size_t>(row0 + r) * a.R + rank;
        for (int z = 0; z < a.slices; ++z) s += p[static_cast<size_t>(z) * a.T * a.R];
      }
      v[i] = s;
      top = fmaxf(top, fabsf(s));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    int e = 0;
    if (top > 0.0f && top < INFINITY) frexpf(top, &e);
#pragma unroll
    for (int i = 0; i < kMaxRank / 32; ++i) {
      const int rank = 32 * i + lane;
      if (rank < Rp) {
        const float s = ldexpf(v[i], -e);
        const __half hi = __float2half_rn(s);
        hs[(2 * r) * pitch + rank] = hi;
        hs[(2 * r + 1) * pitch + rank] = __float2half_rn(s - __half2float(hi));
      }
    }
    if (lane == 0) s_factor[r] = id >= 0 ? ldexpf(a.scaling[id], e) : 0.0f;
  }
  __syncthreads();
  if (n0 >= a.N) return;

  float acc[MT][4][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[mt][j][k] = 0.0f;
  int rid[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    rid[mt][0] = s_id[16 * mt + gid];
    rid[mt][1] = s_id[16 * mt + 8 + gid];
  }
  // column gid of MMA j is column 8 (gid >> 1) + 2 j + (gid & 1) of the warp's 32:
  // a lane's outputs are then 8 contiguous columns
  const int leads = s_leads, chunks = Rp / 32;
  const int ncol = n0 + 8 * (gid >> 1) + (gid & 1);
#pragma unroll 2
  for (int it = 0; it < leads * chunks; ++it) {
    const int adapter = s_lead[it / chunks], r0 = 32 * (it % chunks);
    uint4 b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      b[j] = load16(a.Bm + (static_cast<size_t>(adapter) * a.N + ncol + 2 * j) * a.R + r0 + 8 * tig,
                    r0 + 8 * tig < a.R);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const bool in0 = rid[mt][0] == adapter, in1 = rid[mt][1] == adapter;
      if (!__any_sync(0xffffffffu, in0 || in1)) continue;
      const __half* p0 = hs + (2 * (16 * mt + gid)) * pitch + r0 + 8 * tig;
      const __half* p1 = p0 + 16 * pitch;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const uint4 u0 = load16(p0 + part * pitch, in0), u1 = load16(p1 + part * pitch, in1);
        const uint32_t f0[4] = {u0.x, u1.x, u0.y, u1.y}, f1[4] = {u0.z, u1.z, u0.w, u1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma_16816(acc[mt][j], f0, b[j].x, b[j].y);
          mma_16816(acc[mt][j], f1, b[j].z, b[j].w);
        }
      }
    }
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = 16 * mt + 8 * q + gid, t = row0 + r;
      if (t >= a.T) continue;
      const size_t at = static_cast<size_t>(t) * a.N + n0 + 8 * tig;
      uint4 y = *reinterpret_cast<const uint4*>(a.Y + at);
      __half2* y2 = reinterpret_cast<__half2*>(&y);
      const float f = s_factor[r];
      if (rid[mt][q] >= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = __half22float2(y2[j]);
          y2[j] = __floats2half2_rn(fmaf(f, acc[mt][j][2 * q], v.x),
                                    fmaf(f, acc[mt][j][2 * q + 1], v.y));
        }
      }
      *reinterpret_cast<uint4*>(a.out + at) = y;
    }
}

struct LoraPlan {
  int tiles, slots, slices, k_slice;
  size_t bytes;
};

// Slices of K: about four CTAs an SM in all, each at least 256 long, at most 16.
LoraPlan lora_plan(int T, int K, int R, int n) {
  LoraPlan p;
  const int sms = sm_count();
  p.tiles = (T + kShrinkRows - 1) / kShrinkRows;
  p.slots = n < kShrinkRows ? n : kShrinkRows;
  if (p.slots > T) p.slots = T;
  const int room = 2 * sms / p.tiles;
  if (p.slots > room) p.slots = room < 1 ? 1 : room;
  const int units = p.tiles * p.slots;
  int s = (4 * sms + units - 1) / units;
  if (s > K / 256) s = K / 256;
  if (s > 16) s = 16;
  if (s < 1) s = 1;
  p.k_slice = ((K + s - 1) / s + 127) / 128 * 128;
  p.slices = (K + p.k_slice - 1) / p.k_slice;
  p.bytes = static_cast<size_t>(p.slices) * T * R * sizeof(float);
  return p;
}

int check_lora(int T, int K, int N, int R, int n) {
  if (T < 0 || K <= 0 || N <= 0 || R <= 0 || n <= 0) return QOQ_ERR_INVALID_ARG;
  if (N % kTileN != 0 || K % kTileK != 0) return QOQ_ERR_INVALID_ARG;
  if (K > kMaxK || R % 8 != 0 || R > kMaxRank || T > (1 << 20)) return QOQ_ERR_UNSUPPORTED;
  return QOQ_OK;
}

template <int TM>
int launch_expand(const LoraArgs& a, cudaStream_t s) {
  const int pitch = ((a.R + 31) & ~31) + 8;
  const size_t smem = static_cast<size_t>(TM) * 2 * pitch * sizeof(__half);   // 34 KB at most
  return launch_dependent(lora_expand_kernel<TM>,
                          dim3(static_cast<unsigned>((a.N + kExpandCols - 1) / kExpandCols),
                               static_cast<unsigned>((a.T + TM - 1) / TM)),
                          32 * kExpandWarps, smem, s, a);
}

}  // namespace
}  // namespace qoq

using namespace qoq;

extern "C" size_t qoq_lora_workspace_bytes(int T, int K, int N, int R, int n) {
  if (check_lora(T, K, N, R, n) || T == 0) return 0;
  return lora_plan(T, K, R, n).bytes;
}

extern "C" int qoq_lora_add(const void* Y, const void* X, int T, int K, int N, const void* A,
                            const void* B, int R, int n, const int* ids, const float* scaling,
                            void* out, void* ws, size_t ws_bytes, void* stream) {
  if (int st = check_lora(T, K, N, R, n)) return st;
  if (T == 0) return QOQ_OK;
  if (!Y || !X || !A || !B || !ids || !scaling || !out) return QOQ_ERR_INVALID_ARG;
  if (!aligned16(Y) || !aligned16(X) || !aligned16(A) || !aligned16(B) || !aligned16(out) ||
      !aligned4(ids) || !aligned4(scaling))
    return QOQ_ERR_INVALID_ARG;
  const LoraPlan p = lora_plan(T, K, R, n);
  if (ws == nullptr || ws_bytes < p.bytes || !aligned16(ws)) return QOQ_ERR_WORKSPACE;
  if (int st = check_device()) return st;
  LoraArgs a;
  a.X = static_cast<const __half*>(X);
  a.A = static_cast<const __half*>(A);
  a.Bm = static_cast<const __half*>(B);
  a.ids = ids;
  a.scaling = scaling;
  a.Y = static_cast<const __half*>(Y);
  a.out = static_cast<__half*>(out);
  a.h = static_cast<float*>(ws);
  a.T = T; a.K = K; a.N = N; a.R = R; a.n = n;
  a.slices = p.slices;
  a.k_slice = p.k_slice;
  cudaStream_t s = as_stream(stream);
  const dim3 grid(static_cast<unsigned>(p.tiles), static_cast<unsigned>(p.slots),
                  static_cast<unsigned>(p.slices));
  constexpr unsigned threads = 32 * kShrinkWarps;
  int st;
  if (R <= 16) st = launch_dependent(lora_shrink_kernel<1>, grid, threads, 0, s, a);
  else if (R <= 32) st = launch_dependent(lora_shrink_kernel<2>, grid, threads, 0, s, a);
  else if (R <= 64) st = launch_dependent(lora_shrink_kernel<4>, grid, threads, 0, s, a);
  else st = launch_dependent(lora_shrink_kernel<8>, grid, threads, 0, s, a);
  if (st) return st;
  return T <= 512 ? launch_expand<16>(a, s) : launch_expand<64>(a, s);
}
