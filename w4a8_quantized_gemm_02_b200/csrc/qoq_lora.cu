// Low-rank adapters of many requests beside a shared projection:
//     out[t] = fp16(Y[t] + scaling[a] * B_a (A_a x_t)),   a = ids[t].
//
// Units.  Rows are taken by adapter, wherever they stand: within chunks of 4096
// rows, the rows of one adapter are cut into units of up to 64, so that a unit
// reads its adapter once, for a decode batch of all different requests as for runs
// of a prompt.  Every CTA finds its unit from the ids itself (a histogram in shared
// memory, then a scan for the unit's adapter); no row moves.
//
// Two kernels.  "shrink": h = A_a x, K split over a cluster of up to eight CTAs
// whose partial sums are added in a fixed order through distributed shared memory;
// "expand": y += scaling B_a h, 32 rows by 32 columns a warp, every output formed
// once.  Both multiply on mma.sync m16n8k16 (FP16, FP32 sums): a few operations a
// byte, so what counts is that adapters and rows stream from memory (cp.async
// stages in the first, all of a CTA's loads in flight at once in the second).
//
// Rounding.  h is summed in FP32, scaled by a power of two to its row's largest
// value and handed on as two FP16 numbers (2^-22 of that value is lost), so the
// output's own rounding is the only one that shows.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "qoq.h"
#include "qoq_device.cuh"
#include "qoq_internal.h"
#include "qoq_kv4.cuh"

namespace qoq {
namespace {

constexpr int kUnitRows = 64;
constexpr int kChunkRows = 4096;         // rows within which units are formed
constexpr int kMaxAdapters = 4096;
constexpr int kMaxRank = 128;
constexpr int kShrinkThreads = 256;
constexpr int kShrinkWarps = kShrinkThreads / 32;
constexpr int kStepK = 64;               // K of a copy stage
constexpr int kMaxCluster = 8;
constexpr int kExpandThreads = 128;
constexpr int kExpandCols = 128;         // columns of a CTA at a time
constexpr int kExpandRows = 32;

// What shrink leaves for expand: the units' rows, and per row a factor and the high
// and low FP16 parts of h (Rp = R rounded up to 32 of each).
struct UnitRows {
  int adapter;      // -1: rows without one
  int count;
  int rows[kUnitRows];
};

struct LoraArgs {
  const __half* X;        // T x K
  const __half* A;        // n x R x K
  const __half* Bm;       // n x N x R
  const int* ids;         // T
  const float* scaling;   // n
  const __half* Y;        // T x N
  __half* out;            // T x N
  UnitRows* units;        // [chunks][per_chunk]
  float* factor;          // [T]
  __half* h;              // [T][2][Rp]
  int T, K, N, R, n;
  int per_chunk;          // unit slots of a chunk
  int k_slice;            // K of a CTA of the cluster
};

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ float4 ld_cluster16(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// Unit `u` of the chunk of rows [row0, row1): its adapter and rows.  hist: shared
// memory for n + 1 counts (the last for rows without an adapter) and the chunk's ids.
__device__ __forceinline__ void find_unit(const LoraArgs& a, int row0, int row1, int u, int* hist,
                                          UnitRows& unit) {
  __shared__ int s_warp[kShrinkThreads / 32], s_adapter, s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto id_of = [&](int r) {
    const int id = a.ids[r];
    return id < 0 || id >= a.n ? a.n : id;
  };
  if (row1 - row0 <= 32) {
    // a few rows: a unit for each of their adapters, in the order of their first rows
    if (warp == 0) {
      const int id = lane < row1 - row0 ? id_of(row0 + lane) : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, id);
      uint32_t first = __ballot_sync(0xffffffffu, id >= 0 && (same & ((1u << lane) - 1u)) == 0u);
      for (int i = 0; i < u; ++i) first &= first - 1u;
      const int at = first ? __ffs(first) - 1 : 0;
      const uint32_t rows = first ? __shfl_sync(0xffffffffu, same, at) : 0u;
      const int adapter = __shfl_sync(0xffffffffu, id, at);
      if ((rows >> lane) & 1u) unit.rows[__popc(rows & ((1u << lane) - 1u))] = row0 + lane;
      if (lane == 0) {
        unit.adapter = adapter == a.n ? -1 : adapter;
        unit.count = __popc(rows);
      }
    }
    __syncthreads();
    return;
  }
  int* ids = hist + a.n + 1;
  for (int r0 = row0; r0 < row1; r0 += 8 * kShrinkThreads) {
    int v[8];                       // (loads together: their latency is most of this)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + i * kShrinkThreads + tid;
      v[i] = r < row1 ? id_of(r) : 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + i * kShrinkThreads + tid;
      if (r < row1) ids[r - row0] = v[i];
    }
  }
  for (int i = tid; i <= a.n; i += kShrinkThreads) hist[i] = 0;
  if (tid == 0) {
    s_adapter = -1;
    unit.count = 0;
    unit.adapter = -1;
  }
  __syncthreads();
  for (int r0 = row0 + 32 * warp; r0 < row1; r0 += kShrinkThreads) {
    const int id = r0 + lane < row1 ? ids[r0 - row0 + lane] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, id);    // (runs: one add for all)
    if (id >= 0 && (same & ((1u << lane) - 1u)) == 0u) atomicAdd(&hist[id], __popc(same));
  }
  __syncthreads();
  // the adapter whose units hold number u
  int base = 0;
  for (int i0 = 0; i0 <= a.n && base <= u; i0 += kShrinkThreads) {
    const int i = i0 + tid;
    const int mine = i <= a.n ? (hist[i] + kUnitRows - 1) / kUnitRows : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int before = base;
#pragma unroll
    for (int w = 0; w < kShrinkThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      base += s_warp[w];
    }
    const int first = before + incl - mine;
    if (u >= first && u < first + mine) {
      s_adapter = i;
      s_first = (u - first) * kUnitRows;
    }
    __syncthreads();
  }
  const int adapter = s_adapter;
  if (adapter < 0) return;
  // its rows number s_first .. + 63, in their order
  const int lo = s_first;
  int seen = 0;
  for (int r0 = row0; r0 < row1 && seen < lo + kUnitRows; r0 += kShrinkThreads) {
    const int r = r0 + tid;
    const bool is = r < row1 && ids[r - row0] == adapter;
    const uint32_t m = __ballot_sync(0xffffffffu, is);
    if (lane == 0) s_warp[warp] = __popc(m);
    __syncthreads();
    int at = seen + __popc(m & ((1u << lane) - 1u));
#pragma unroll
    for (int w = 0; w < kShrinkThreads / 32; ++w) {
      if (w < warp) at += s_warp[w];
      seen += s_warp[w];
    }
    if (is && at >= lo && at < lo + kUnitRows) unit.rows[at - lo] = r;
    __syncthreads();
  }
  if (tid == 0) {
    unit.adapter = adapter == a.n ? -1 : adapter;
    unit.count = seen - lo < kUnitRows ? seen - lo : kUnitRows;
  }
  __syncthreads();
}

// Stages a CTA keeps: as many as 64 KB hold (three CTAs an SM), 4 to 6.
constexpr int stage_bytes(int mt) { return (16 * mt + kUnitRows) * kStepK * 2; }
constexpr int stages_of(int mt) {
  const int s = 65536 / stage_bytes(mt);
  return s > 6 ? 6 : (s < 4 ? 4 : s);
}
// ... and then the warps' partial sums, [128][16 MT + 4] floats, in the same place.
constexpr size_t shrink_smem(int mt) {
  const size_t ring = static_cast<size_t>(stages_of(mt)) * stage_bytes(mt);
  const size_t sums = static_cast<size_t>(2 * kUnitRows) * (16 * mt + 4) * sizeof(float);
  const size_t hist = static_cast<size_t>(kMaxAdapters + 1 + kChunkRows) * sizeof(int);
  const size_t most = ring > sums ? ring : sums;
  return most > hist ? most : hist;
}

// Measured, both kernels: one row of rank 16 (4096 x 6144) 7.6 us; 48 rows over 64 adapters
// of rank 32 (8192 x 24576, 77 MB) 29.3 us; 2500 rows of rank 64 (14336 x 4096, 122 MB)
// 62.5 us, 38 of them here, where the latency of ldmatrix and the barrier of each step of
// 64 K take more time than the copies.
//
// Grid: units x cluster size (S).  MT: tiles of 16 ranks.
template <int MT>
__global__ void __launch_bounds__(kShrinkThreads) lora_shrink_kernel(const LoraArgs a, int S) {
  constexpr int kStage = stage_bytes(MT), kStages = stages_of(MT);
  constexpr int kPitch = 16 * MT + 4;      // floats a row of partial sums
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ UnitRows unit;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = blockIdx.x / S, rank = blockIdx.x - slot * S;
  grid_dependency_wait();
  grid_launch_dependents();
  const int chunk = slot / a.per_chunk, u = slot - chunk * a.per_chunk;
  const int row0 = chunk * kChunkRows;
  const int row1 = row0 + kChunkRows < a.T ? row0 + kChunkRows : a.T;
  find_unit(a, row0, row1, u, reinterpret_cast<int*>(smem), unit);
  const int count = unit.count, adapter = unit.adapter;
  if (rank == 0) {
    UnitRows& d = a.units[slot];
    if (tid < count) d.rows[tid] = unit.rows[tid];
    if (tid == 0) {
      d.adapter = adapter;
      d.count = count;
    }
  }
  if (count == 0 || adapter < 0) return;   // (the whole cluster)

  const float scaling = a.scaling[adapter];
  const uint32_t s0 = smem_u32(smem);
  const int k0 = rank * a.k_slice;
  const int k1 = k0 + a.k_slice < a.K ? k0 + a.k_slice : a.K;
  const int steps = k0 < k1 ? (k1 - k0) / kStepK : 0;
  // rows that no copy writes but the products read: ranks past R, and tokens past the
  // unit's up to a multiple of 16
  const int r_pad = 16 * MT - a.R, t_pad = (16 - (count & 15)) & 15;
  for (int i = tid; i < kStages * (r_pad + t_pad) * 8; i += kShrinkThreads) {
    const int c = i & 7, p = (i >> 3) % (r_pad + t_pad), st = (i >> 3) / (r_pad + t_pad);
    const int r = p < r_pad ? a.R + p : 16 * MT + count + (p - r_pad);
    *reinterpret_cast<uint4*>(smem + st * kStage + r * 128 + 16 * c) = make_uint4(0u, 0u, 0u, 0u);
  }
  // a stage: 16 MT rows of A and 64 rows of X, 128 bytes each, the 16-byte chunk c of
  // row r at c ^ (r & 7); thread (cr, cc) copies chunk cc of every 32nd row
  const int cc = tid & 7, cr = tid >> 3;
  const uint32_t to = s0 + cr * 128 + ((cc ^ (cr & 7)) << 4);
  const __half* A = a.A + (static_cast<size_t>(adapter) * a.R + cr) * a.K + k0 + 8 * cc;
  const size_t a_step = static_cast<size_t>(32) * a.K;
  const __half* X[kUnitRows / 32];
#pragma unroll
  for (int i = 0; i < kUnitRows / 32; ++i)
    X[i] = cr + 32 * i < count
               ? a.X + static_cast<size_t>(unit.rows[cr + 32 * i]) * a.K + k0 + 8 * cc : nullptr;
  int put = 0;                             // the stage of the next copies
  auto issue = [&](int j) {
    if (j < steps) {
      const uint32_t st = to + put * kStage;
      const int k = j * kStepK;
#pragma unroll
      for (int i = 0; i < (MT + 1) / 2; ++i)
        if (cr + 32 * i < a.R) cp_async16(st + i * 4096, A + i * a_step + k);
#pragma unroll
      for (int i = 0; i < kUnitRows / 32; ++i)
        if (X[i] != nullptr) cp_async16(st + MT * 2048 + i * 4096, X[i] + k);
    }
    cp_async_commit();
    put = put + 1 == kStages ? 0 : put + 1;
  };
#pragma unroll
  for (int j = 0; j < kStages - 1; ++j) issue(j);

  // warp w: tokens 16 (w % 4) .. of the unit, all ranks, half w / 4 of every step's K;
  // or, for up to 16 rows (`few`), the first four warps a quarter of K for all of them
  const bool few = count <= 16;
  const int token0 = few ? 0 : 16 * (warp & 3);
  const int ks0 = few ? warp : 2 * (warp >> 2), ks1 = few ? warp + 1 : ks0 + 2;
  const bool busy = few ? warp < 4 : token0 < count;
  float acc[MT][2][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[mt][nt][k] = 0.0f;
  // X: tokens (lane & 7) + 8 (lane >> 4), k half (lane >> 3) & 1; A: ranks lane & 15, k
  // half lane >> 4
  const uint32_t x_at = (16 * MT + token0 + (lane & 7) + 8 * (lane >> 4)) * 128;
  const uint32_t a_at = (lane & 15) * 128;
  const int xh = (lane >> 3) & 1, ah = lane >> 4, sw = lane & 7;
  auto chunk_at = [&](int c) { return static_cast<uint32_t>((c ^ sw) << 4); };
  int get = 0;
  for (int j = 0; j < steps; ++j) {
    cp_async_wait<kStages - 2>();
    __syncthreads();                       // everybody's copies of step j, and reads of j - 1
    issue(j + kStages - 1);
    const uint32_t st = s0 + get * kStage;
    get = get + 1 == kStages ? 0 : get + 1;
    if (!busy) continue;
#pragma unroll 2
    for (int ks = ks0; ks < ks1; ++ks) {
      uint32_t x[4], f[MT][4];
      ldmatrix4(x, st + x_at + chunk_at(2 * ks + xh));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) ldmatrix4(f[mt], st + a_at + mt * 2048 + chunk_at(2 * ks + ah));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma_16816(acc[mt][0], f[mt], x[0], x[1]);
        mma_16816(acc[mt][1], f[mt], x[2], x[3]);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  // the warps' partial sums, a row a token, then the CTA's in the first rows
  float* sums = reinterpret_cast<float*>(smem);
  const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        sums[(16 * warp + 8 * nt + 2 * tig + (k & 1)) * kPitch + 16 * mt + gid + 8 * (k >> 1)] =
            acc[mt][nt][k];
  __syncthreads();
  if (few) {
    for (int i = tid; i < 16 * kPitch; i += kShrinkThreads) {
      float v = sums[i];
#pragma unroll
      for (int w = 1; w < 4; ++w) v += sums[16 * w * kPitch + i];
      sums[i] = v;
    }
  } else {
    for (int i = tid; i < kUnitRows * kPitch; i += kShrinkThreads) sums[i] += sums[kUnitRows * kPitch + i];
  }
  cluster_sync_all();
  // CTA `rank` finishes the unit's rows rank, rank + S, ...: 32 lanes a row, four
  // ranks a lane, the cluster's sums added in order
  const int Rp = (a.R + 31) & ~31;
  for (int r = rank + S * warp; r < count; r += S * kShrinkWarps) {
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (4 * lane < a.R) {
      const uint32_t at = s0 + (r * kPitch + 4 * lane) * 4;
      float4 p[kMaxCluster];
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q)      // all in flight before the first is added
        p[q] = q < S ? ld_cluster16(map_to_rank(at, q)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        v.x += p[q].x;
        v.y += p[q].y;
        v.z += p[q].z;
        v.w += p[q].w;
      }
    }
    float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // 2^e over the largest value (e at least -100: smaller rows keep their place)
    int e = static_cast<int>((__float_as_uint(top) >> 23) & 255u) - 126;
    e = e < -100 ? -100 : (e > 126 ? 126 : e);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const float h4[4] = {v.x * down, v.y * down, v.z * down, v.w * down};
    __half hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi[i] = __float2half_rn(h4[i]);
      // (an infinite value has no low part: inf - inf would make NaN of it)
      lo[i] = __float2half_rn(isinf(h4[i]) ? 0.0f : h4[i] - __half2float(hi[i]));
    }
    const int row = unit.rows[r];
    __half* h = a.h + static_cast<size_t>(row) * 2 * Rp;
    if (4 * lane < Rp) {
      *reinterpret_cast<uint2*>(h + 4 * lane) = *reinterpret_cast<const uint2*>(hi);
      *reinterpret_cast<uint2*>(h + Rp + 4 * lane) = *reinterpret_cast<const uint2*>(lo);
    }
    if (lane == 0)
      a.factor[row] = scaling * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  }
  cluster_sync_all();    // no CTA leaves while its sums are read
}

__device__ __forceinline__ uint4 load16(const __half* p, bool ok) {
  return ok ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
}

// MT tiles of 16 rows (from the unit's row first) by the warp's 32 columns n0 .. of
// every 128 up to c1.
template <int RC, int MT>
__device__ __forceinline__ void expand_rows(const LoraArgs& a, const UnitRows& u, int first,
                                            int count, int n0, int c1) {
  // the rows' h stays in registers over the columns where it fits
  constexpr bool kHold = RC * MT <= 2;
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  const int Rp = (a.R + 31) & ~31;
  int row[MT][2];
  float f[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = first + 16 * mt + 8 * q + gid;
      row[mt][q] = r < count ? u.rows[r] : -1;
    }
  // A fragments: rows gid and gid + 8, 8 ranks from 32 c + 8 tig on
  auto load_h = [&](int mt, int c, int part, int q) {
    return load16(a.h + (static_cast<size_t>(row[mt][q] < 0 ? 0 : row[mt][q]) * 2 + part) * Rp +
                      32 * c + 8 * tig, row[mt][q] >= 0);
  };
  uint4 h[kHold ? RC : 1][MT][2][2];
  if constexpr (kHold) {
#pragma unroll
    for (int c = 0; c < RC; ++c)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[c][mt][i >> 1][i & 1] = load_h(mt, c, i >> 1, i & 1);
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int q = 0; q < 2; ++q) f[mt][q] = row[mt][q] >= 0 ? a.factor[row[mt][q]] : 0.0f;
  // column gid of MMA j is column 8 (gid >> 1) + 2 j + (gid & 1) of the warp's 32: a
  // lane's outputs are then 8 contiguous columns.  The k order within 32 is permuted
  // the same way in both operands: a lane loads 16 contiguous bytes for two MMAs.
  const __half* b0 = a.Bm + (static_cast<size_t>(u.adapter) * a.N + n0 + 8 * (gid >> 1) + (gid & 1)) *
                                a.R + 8 * tig;
  for (; n0 < c1; n0 += kExpandCols, b0 += static_cast<size_t>(kExpandCols) * a.R) {
    uint4 b[RC][4];
#pragma unroll
    for (int c = 0; c < RC; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        b[c][j] = load16(b0 + static_cast<size_t>(2 * j) * a.R + 32 * c, 32 * c + 8 * tig < a.R);
    uint4 y[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        y[mt][q] = load16(a.Y + static_cast<size_t>(row[mt][q] < 0 ? 0 : row[mt][q]) * a.N + n0 +
                              8 * tig, row[mt][q] >= 0);
    float acc[MT][4][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[mt][j][k] = 0.0f;
#pragma unroll
    for (int c = 0; c < RC; ++c) {
      if (32 * c >= a.R) break;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint4 u0 = kHold ? h[kHold ? c : 0][mt][part][0] : load_h(mt, c, part, 0);
          const uint4 u1 = kHold ? h[kHold ? c : 0][mt][part][1] : load_h(mt, c, part, 1);
          const uint32_t f0[4] = {u0.x, u1.x, u0.y, u1.y}, f1[4] = {u0.z, u1.z, u0.w, u1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mma_16816(acc[mt][j], f0, b[c][j].x, b[c][j].y);
            mma_16816(acc[mt][j], f1, b[c][j].z, b[c][j].w);
          }
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (row[mt][q] < 0) continue;
        __half2* y2 = reinterpret_cast<__half2*>(&y[mt][q]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 v = __half22float2(y2[j]);
          y2[j] = __floats2half2_rn(fmaf(f[mt][q], acc[mt][j][2 * q], v.x),
                                    fmaf(f[mt][q], acc[mt][j][2 * q + 1], v.y));
        }
        *reinterpret_cast<uint4*>(a.out + static_cast<size_t>(row[mt][q]) * a.N + n0 + 8 * tig) =
            y[mt][q];
      }
  }
}

// Grid: units (x 2 where they may have over 32 rows) x column groups (of `per` times 128
// columns).  RC: 32-rank steps.  Four CTAs an SM where they fit without spills (up to rank
// 32, five spilled: 1500 rows of rank 32, 8192 x 8192, took both kernels 38 us against 31).
template <int RC>
__global__ void __launch_bounds__(kExpandThreads, RC <= 2 ? 4 : 3)
lora_expand_kernel(const LoraArgs a, int halves, int groups, int per) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  const int part = blockIdx.x / groups;
  const int first = (part & (halves - 1)) * kExpandRows;
  const UnitRows& u = a.units[part / halves];
  const int count = u.count;
  if (first >= count) return;
  const int c0 = (blockIdx.x - part * groups) * per * kExpandCols + 32 * warp;
  const int c1 = c0 + per * kExpandCols < a.N ? c0 + per * kExpandCols : a.N;
  if (u.adapter < 0 && a.out == a.Y) return;
  if (u.adapter < 0) {
    const int last = first + kExpandRows < count ? first + kExpandRows : count;
    for (int n0 = c0; n0 < c1; n0 += kExpandCols)
      for (int r = first + (lane >> 2); r < last; r += 8) {
        const size_t at = static_cast<size_t>(u.rows[r]) * a.N + n0 + 8 * (lane & 3);
        *reinterpret_cast<uint4*>(a.out + at) = *reinterpret_cast<const uint4*>(a.Y + at);
      }
    return;
  }
  if (count - first <= 16) expand_rows<RC, 1>(a, u, first, count, c0, c1);
  else expand_rows<RC, 2>(a, u, first, count, c0, c1);
}

struct LoraPlan {
  int chunks, per_chunk, cluster, k_slice;
  size_t units_off, factor_off, h_off, bytes;
};

LoraPlan lora_plan(int T, int K, int R, int n) {
  LoraPlan p;
  const int rows = T < kChunkRows ? T : kChunkRows;
  p.chunks = (T + kChunkRows - 1) / kChunkRows;
  // every unit has a row, and all but one of an adapter's are full
  const int by_adapter = rows / kUnitRows + n + 1;
  p.per_chunk = rows < by_adapter ? rows : by_adapter;
  p.cluster = kMaxCluster;
  while (p.cluster > 1 && K / p.cluster < kStepK) p.cluster >>= 1;
  p.k_slice = ((K + p.cluster - 1) / p.cluster + kStepK - 1) / kStepK * kStepK;
  const size_t units = static_cast<size_t>(p.chunks) * p.per_chunk;
  const size_t Rp = static_cast<size_t>((R + 31) & ~31);
  auto round = [](size_t b) { return (b + 255) / 256 * 256; };
  p.units_off = 0;
  p.factor_off = round(units * sizeof(UnitRows));
  p.h_off = p.factor_off + round(static_cast<size_t>(T) * sizeof(float));
  p.bytes = p.h_off + static_cast<size_t>(T) * 2 * Rp * sizeof(__half);
  return p;
}

int check_lora(int T, int K, int N, int R, int n) {
  if (T < 0 || K <= 0 || N <= 0 || R <= 0 || n <= 0) return QOQ_ERR_INVALID_ARG;
  if (N % kTileN != 0 || K % kTileK != 0) return QOQ_ERR_INVALID_ARG;
  if (K > kMaxK || R % 8 != 0 || R > kMaxRank || n > kMaxAdapters || T > (1 << 20))
    return QOQ_ERR_UNSUPPORTED;
  return QOQ_OK;
}

template <int MT>
int launch_shrink(const LoraArgs& a, const LoraPlan& p, cudaStream_t s) {
  static std::atomic<unsigned long long> ready{0};
  if (int st = opt_in_smem(reinterpret_cast<const void*>(lora_shrink_kernel<MT>), shrink_smem(MT),
                           ready))
    return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.cluster * p.chunks * p.per_chunk), 1, 1);
  cfg.blockDim = dim3(kShrinkThreads, 1, 1);
  cfg.dynamicSmemBytes = shrink_smem(MT);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, lora_shrink_kernel<MT>, a, p.cluster) != cudaSuccess) {
    cudaGetLastError();
    return QOQ_ERR_CUDA;
  }
  return QOQ_OK;
}

template <int RC>
int launch_expand(const LoraArgs& a, const LoraPlan& p, cudaStream_t s) {
  // columns to a CTA: about eight CTAs an SM over all units' slots
  const int halves = a.T > kExpandRows ? 2 : 1;
  const long long units = static_cast<long long>(p.chunks) * p.per_chunk * halves;
  const int blocks = a.N / kExpandCols;
  long long per = units * blocks / (8LL * sm_count());
  per = per < 1 ? 1 : (per > 8 ? 8 : per);
  const int groups = static_cast<int>((blocks + per - 1) / per);
  return launch_dependent(lora_expand_kernel<RC>, dim3(static_cast<unsigned>(units * groups)),
                          kExpandThreads, 0, s, a, halves, groups, static_cast<int>(per));
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
  if (2LL * p.chunks * p.per_chunk * (N / kExpandCols) > 0x7fffffffLL)
    return QOQ_ERR_UNSUPPORTED;   // the grid
  if (ws == nullptr || ws_bytes < p.bytes || !aligned16(ws)) return QOQ_ERR_WORKSPACE;
  if (int st = check_device()) return st;
  char* w = static_cast<char*>(ws);
  LoraArgs a;
  a.X = static_cast<const __half*>(X);
  a.A = static_cast<const __half*>(A);
  a.Bm = static_cast<const __half*>(B);
  a.ids = ids;
  a.scaling = scaling;
  a.Y = static_cast<const __half*>(Y);
  a.out = static_cast<__half*>(out);
  a.units = reinterpret_cast<UnitRows*>(w + p.units_off);
  a.factor = reinterpret_cast<float*>(w + p.factor_off);
  a.h = reinterpret_cast<__half*>(w + p.h_off);
  a.T = T; a.K = K; a.N = N; a.R = R; a.n = n;
  a.per_chunk = p.per_chunk;
  a.k_slice = p.k_slice;
  cudaStream_t s = as_stream(stream);
  int st;
  if (R <= 16) st = launch_shrink<1>(a, p, s);
  else if (R <= 32) st = launch_shrink<2>(a, p, s);
  else if (R <= 64) st = launch_shrink<4>(a, p, s);
  else st = launch_shrink<8>(a, p, s);
  if (st) return st;
  if (R <= 32) return launch_expand<1>(a, p, s);
  if (R <= 64) return launch_expand<2>(a, p, s);
  return launch_expand<4>(a, p, s);
}
