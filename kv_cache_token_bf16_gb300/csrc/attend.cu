// Attention of a batch over a shared prefix and its own pages.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max)
// over the rows a query sees, in one pass over K and V with a running maximum
// and sum; logits are kept in base 2 (scale * log2 e), so p = 2^(x - m).
//
// attend_kernel: persistent, one CTA of eight warps per SM. All the batch's
// rows of K and V, prefix and pages alike, are cut into steps of 128 rows that
// are laid end to end, and every CTA takes an equal share of them whatever the
// sequences' lengths are: the lengths live on the device, so the shares are
// found there, by one block scan over the batch. Warp w takes rows
// 16 w .. 16 w + 15 of every step and works alone, with its own running
// maximum, sum and output and its own ring of TMA boxes (16 rows x 128
// elements of K and of V, 8 KB); the eight results meet only where the CTA
// leaves a unit. A 16-row box never crosses a page. Bound: HBM; a warp has up
// to kStages - 1 boxes in flight (128 KB an SM) while it computes on another,
// and the tensor cores (m16n8k16, queries as rows, one or two tiles of 16)
// need about a quarter of the time its box needs from memory.
//
// attend_join_kernel: a warp per output row merges the partial results of the
// row's units, in the order of their slots.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "attend.h"
#include "attend.cuh"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "rotary.h"
#include "tcgen05.cuh"

namespace evict {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kBoxTokens = 16;
constexpr int kBoxBytes = kBoxTokens * kHeadDim * 2;       // of K or of V
constexpr int kStages = 3;
constexpr int kRingBytes = kWarps * kStages * 2 * kBoxBytes;
constexpr int kQPitch = kHeadDim * 2 + 16;                 // bytes: ldmatrix rows on different banks

// Columns of the warps' results that are merged at a time, and the dynamic shared memory, for
// `tiles` tiles of 16 query rows: the ring, the queries and the merge's buffers.
__host__ __device__ constexpr int merge_cols(int tiles) { return tiles == 1 ? 32 : 16; }
constexpr int few_smem(int tiles) {
  return kRingBytes + 1024 + 16 * tiles * kQPitch + kWarps * 16 * tiles * (merge_cols(tiles) + 4) * 4 +
         kWarps * 16 * tiles * 8;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 in, fp32 sums
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
struct FewShared {
  uint64_t full[kWarps][kStages];
  ScanShared scan;
  int fail;
};

// Last row that row r of the tile sees (-1: none; rows behind the unit's last see none).
template <int kRows>
__device__ __forceinline__ int last_row(const AttendParams& p, const StreamSet& set, const Cursor<kRows>& c, int r) {
  const int t = (c.tile * kRows + r) / p.group;
  if (c.s < set.prefixes) return c.st.pre - 1;
  return t < c.st.n ? c.st.len - c.st.n + t : -1;
}

template <int kTiles>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kRows = 16 * kTiles;
  constexpr int kCols = merge_cols(kTiles);
  if (!p.late_wait) pdl_wait();
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ FewShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* ring = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* qs = ring + kRingBytes;
  float* red = reinterpret_cast<float*>(qs + kRows * kQPitch);          // [warp][row][kCols + 4]
  float2* red_ml = reinterpret_cast<float2*>(red + kWarps * kRows * (kCols + 4));
  const StreamSet& set = p.set;

  if (tid < kWarps * kStages) tc::mbar_init(&sh.full[tid / kStages][tid % kStages], 1);
  if (tid == 0) sh.fail = 0;
  Cursor<kRows> cur;
  const int count = find_share<kRows, kThreads>(p, set, sh.scan, cur);

  // Does this warp have rows to read at this step? (its box begins inside what the tile sees)
  auto active = [&](const Cursor<kRows>& c) {
    const int row0 = c.step * kStepTokens + kBoxTokens * warp;
    return c.s < set.prefixes ? row0 < c.st.pre : row0 <= c.st.reach(p, c.tile);
  };

  // --- the ring: boxes are requested in the order in which they are used ---
  const uint32_t my_ring = tc::smem_u32(ring) + warp * kStages * 2 * kBoxBytes;
  Cursor<kRows> ahead = cur;
  int ahead_left = count, page = 0;
  // advance `ahead` to the next box of this warp and look its page up
  auto seek = [&] {
    while (ahead_left > 0 && !active(ahead)) {
      ahead.next(p, set);
      --ahead_left;
    }
    if (ahead_left > 0 && ahead.s >= set.prefixes && lane == 0)
      page = p.table[(long long)(ahead.s - set.prefixes) * p.table_stride +
                     ((ahead.step * kStepTokens + kBoxTokens * warp) >> p.page_shift)];
  };
  auto request = [&](int stage) {
    if (ahead_left <= 0) return;
    if (lane == 0) {
      uint64_t* bar = &sh.full[warp][stage];
      const uint32_t dst = my_ring + stage * 2 * kBoxBytes;
      const int row = ahead.step * kStepTokens + kBoxTokens * warp;
      tc::mbar_arrive_expect_tx(bar, 2 * kBoxBytes);
      if (ahead.s < set.prefixes) {
        tma_load_5d(dst, &p.tm_pk, 0, row, 0, ahead.h, ahead.s, bar);
        tma_load_5d(dst + kBoxBytes, &p.tm_pv, 0, row, 0, ahead.h, ahead.s, bar);
      } else {
        const bool in_pool = page >= 0 && page < p.n_pages;
        if (!in_pool) raise_device_error(p.err, kDevBadIndex);
        const int at = in_pool ? page : p.n_pages;                 // outside: the box is zeros
        const int y = row & ((1 << p.page_shift) - 1);
        tma_load_5d(dst, &p.tm_k, 0, y, 0, ahead.h, at, bar);
        tma_load_5d(dst + kBoxBytes, &p.tm_v, 0, y, 0, ahead.h, at, bar);
      }
    }
    ahead.next(p, set);
    --ahead_left;
    seek();
  };
  int waited = 0, requested = 0;
  seek();
  for (int i = 0; i < kStages - 1; ++i)
    if (ahead_left > 0) request(requested++ % kStages);

  bool dead = false;
  uint32_t q[kTiles][8][4];
  float o[kTiles][16][4], mx[kTiles][2], sum[kTiles][2];
  int last[kTiles][2], low = 0;                   // each row's last visible row; the tile's lowest
  bool fresh = true;

  for (int i = 0; i < count; ++i) {
    if (fresh) {                                  // a new unit: its queries
      fresh = false;
      for (int e = tid; e < kRows * 16; e += kThreads) {
        const int r = e >> 4, c = e & 15;
        const QueryRow qr = query_row(p, set, cur, r);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (qr.real)
          x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (long long)qr.b * p.qb +
                                              (long long)qr.hq * p.qh + (long long)qr.t * p.qm + c * 8);
        *reinterpret_cast<uint4*>(qs + r * kQPitch + c * 16) = x;
      }
      __syncthreads();
      low = last_row(p, set, cur, 0);
#pragma unroll
      for (int x = 0; x < kTiles; ++x) {
#pragma unroll
        for (int s = 0; s < 8; ++s)
          ldsm4(tc::smem_u32(qs) + (16 * x + (lane & 15)) * kQPitch + s * 32 + (lane >> 4) * 16, q[x][s]);
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[x][j][k] = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mx[x][k] = -INFINITY;
          sum[x][k] = 0.f;
          last[x][k] = last_row(p, set, cur, 16 * x + (lane >> 2) + 8 * k);
        }
      }
    }

    if (active(cur)) {
      const int stage = waited % kStages;
      // the next box goes where the last one was: every lane has read it
      __syncwarp();
      if (ahead_left > 0 && !dead) request(requested++ % kStages);
      if (!dead) {
        const bool ok = wait_phase(&sh.full[warp][stage], (uint32_t)((waited / kStages) & 1), &sh.fail, p.err);
        if (!__all_sync(0xffffffffu, ok)) {
          // copies in flight must land before this CTA may end
          for (int w = waited; w < requested; ++w)
            drain_phase(&sh.full[warp][w % kStages], (uint32_t)((w / kStages) & 1), p.err);
          dead = true;
        }
      }
      ++waited;
      if (!dead) {
        const uint32_t kb = my_ring + stage * 2 * kBoxBytes, vb = kb + kBoxBytes;
        const int row0 = cur.step * kStepTokens + kBoxTokens * warp;
        const bool full = row0 + kBoxTokens - 1 <= low;            // every query sees every row
        float z[kTiles][2][4];
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) z[x][j][k] = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          uint32_t k4[4];
          ldsm4(kb + tc::sw128_offset((lane & 7) + ((lane >> 4) << 3), 2 * s + ((lane >> 3) & 1), kBoxTokens), k4);
#pragma unroll
          for (int x = 0; x < kTiles; ++x) {
            mma16816(z[x][0], q[x][s], k4[0], k4[1]);
            mma16816(z[x][1], q[x][s], k4[2], k4[3]);
          }
        }
        uint32_t hi[kTiles][4], lo[kTiles][4];
#pragma unroll
        for (int x = 0; x < kTiles; ++x) {
          float rm[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float v = z[x][j][k] * p.scale2;
              if (!full && row0 + 8 * j + 2 * (lane & 3) + (k & 1) > last[x][k >> 1]) v = -INFINITY;
              z[x][j][k] = v;
              rm[k >> 1] = fmaxf(rm[k >> 1], v);
            }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            rm[k] = fmaxf(rm[k], __shfl_xor_sync(0xffffffffu, rm[k], 1));
            rm[k] = fmaxf(rm[k], __shfl_xor_sync(0xffffffffu, rm[k], 2));
          }
          const bool up = rm[0] > mx[x][0] || rm[1] > mx[x][1];
          if (__any_sync(0xffffffffu, up)) {
            float f[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float nm = fmaxf(mx[x][k], rm[k]);
              f[k] = weight_of(mx[x][k], nm);
              mx[x][k] = nm;
              sum[x][k] *= f[k];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              o[x][j][0] *= f[0];
              o[x][j][1] *= f[0];
              o[x][j][2] *= f[1];
              o[x][j][3] *= f[1];
            }
          }
          const float m0 = base_of(mx[x][0]), m1 = base_of(mx[x][1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int k = 0; k < 4; ++k) z[x][j][k] = ex2(z[x][j][k] - (k < 2 ? m0 : m1));
            sum[x][0] += z[x][j][0] + z[x][j][1];
            sum[x][1] += z[x][j][2] + z[x][j][3];
            // weights as bf16 pairs hi + lo: 16 bits of each, so that their rounding does not
            // add to the output's own (the tensor cores wait for memory here anyway)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float a = z[x][j][2 * k], b = z[x][j][2 * k + 1];
              const uint32_t h2 = pack_bf16(a, b);
              hi[x][2 * j + k] = h2;
              lo[x][2 * j + k] = pack_bf16(a - __uint_as_float(h2 << 16), b - __uint_as_float(h2 & 0xffff0000u));
            }
          }
        }
        // V of rows behind the stream's end may hold anything: zeros in its place
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
        if (!full) {
          const int r0 = row0 + 2 * (lane & 3), end = cur.s < set.prefixes ? cur.st.pre : cur.st.len;
          auto mask = [&](int r) { return (r < end ? 0xffffu : 0u) | (r + 1 < end ? 0xffff0000u : 0u); };
          keep0 = mask(r0);
          keep1 = mask(r0 + 8);
        }
        const int vrow = lane & 15, vchunk = lane >> 4;
        uint32_t bad = 0;                         // tokens of the box whose V holds an infinity or NaN
        if (!full && p.m > 1 && cur.s >= set.prefixes) {
          // A query that does not see such a row gives it weight 0, but 0 * infinity is not 0: the
          // products leave these rows out, and the queries that see them take them afterwards.
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint32_t v4[4];
            ldsm4_t(vb + tc::sw128_offset(vrow, 2 * j + vchunk, kBoxTokens), v4);
            const uint32_t odd0 = nonfinite2(v4[0] & keep0) | nonfinite2(v4[2] & keep0);
            const uint32_t odd1 = nonfinite2(v4[1] & keep1) | nonfinite2(v4[3] & keep1);
            bad |= (odd0 | odd1 << 8) << (2 * (lane & 3));
          }
          bad = __reduce_or_sync(0xffffffffu, bad);
          if (bad) {
            auto drop = [&](uint32_t two) { return (two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u); };
            keep0 &= ~drop(bad >> (2 * (lane & 3)));
            keep1 &= ~drop(bad >> (2 * (lane & 3) + 8));
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t v4[4];
          ldsm4_t(vb + tc::sw128_offset(vrow, 2 * j + vchunk, kBoxTokens), v4);
          if (!full) v4[0] &= keep0, v4[1] &= keep1, v4[2] &= keep0, v4[3] &= keep1;
#pragma unroll
          for (int x = 0; x < kTiles; ++x) {
            mma16816(o[x][2 * j], hi[x], v4[0], v4[1]);
            mma16816(o[x][2 * j + 1], hi[x], v4[2], v4[3]);
            mma16816(o[x][2 * j], lo[x], v4[0], v4[1]);
            mma16816(o[x][2 * j + 1], lo[x], v4[2], v4[3]);
          }
        }
        if (bad) {
#pragma unroll
          for (int k = 0; k < kBoxTokens; ++k) {
            if (!(bad >> k & 1)) continue;
            const int from = (lane & 28) | ((k & 7) >> 1);
#pragma unroll
            for (int x = 0; x < kTiles; ++x) {
              const float w0 = __shfl_sync(0xffffffffu, z[x][k >> 3][k & 1], from);
              const float w1 = __shfl_sync(0xffffffffu, z[x][k >> 3][2 + (k & 1)], from);
              const bool s0 = row0 + k <= last[x][0], s1 = row0 + k <= last[x][1];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                uint32_t v;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v)
                             : "r"(vb + tc::sw128_offset(k, j, kBoxTokens) + 4 * (lane & 3)) : "memory");
                const float v0 = __uint_as_float(v << 16), v1 = __uint_as_float(v & 0xffff0000u);
                if (s0) o[x][j][0] += w0 * v0, o[x][j][1] += w0 * v1;
                if (s1) o[x][j][2] += w1 * v0, o[x][j][3] += w1 * v1;
              }
            }
          }
        }
      }
    }

    // --- the CTA leaves the unit: the warps' results meet ---
    if (cur.step == cur.steps - 1 || i == count - 1) {
      const long long slot = cur.unit + blockIdx.x;
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float t = sum[x][k];
          t += __shfl_xor_sync(0xffffffffu, t, 1);
          t += __shfl_xor_sync(0xffffffffu, t, 2);
          if ((lane & 3) == 0) red_ml[warp * kRows + 16 * x + (lane >> 2) + 8 * k] = make_float2(mx[x][k], t);
        }
      __syncthreads();
      float f[kTiles][2];
#pragma unroll
      for (int x = 0; x < kTiles; ++x)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float top = -INFINITY;
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_ml[w * kRows + 16 * x + (lane >> 2) + 8 * k].x);
          f[x][k] = weight_of(mx[x][k], top);
        }
      if (tid < kRows) {
        float top = -INFINITY, t = 0.f;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, red_ml[w * kRows + tid].x);
        for (int w = 0; w < kWarps; ++w) t += red_ml[w * kRows + tid].y * weight_of(red_ml[w * kRows + tid].x, top);
        set.part_ml[slot * kRows + tid] = make_float2(top, t);
      }
#pragma unroll
      for (int c = 0; c < kHeadDim / kCols; ++c) {
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
#pragma unroll
          for (int j = 0; j < kCols / 8; ++j) {
            const float* v = o[x][c * (kCols / 8) + j];
            float* d = red + (warp * kRows + 16 * x + (lane >> 2)) * (kCols + 4) + 8 * j + 2 * (lane & 3);
            *reinterpret_cast<float2*>(d) = make_float2(v[0] * f[x][0], v[1] * f[x][0]);
            *reinterpret_cast<float2*>(d + 8 * (kCols + 4)) = make_float2(v[2] * f[x][1], v[3] * f[x][1]);
          }
        __syncthreads();
#pragma unroll
        for (int e = tid; e < kRows * kCols / 2; e += kThreads) {
          const int r = e / (kCols / 2), cc = 2 * (e % (kCols / 2));
          float2 a = make_float2(0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 y = *reinterpret_cast<const float2*>(red + (w * kRows + r) * (kCols + 4) + cc);
            a.x += y.x;
            a.y += y.y;
          }
          *reinterpret_cast<float2*>(set.part_o + (slot * kRows + r) * kHeadDim + c * kCols + cc) = a;
        }
        __syncthreads();
      }
      fresh = true;
    }
    cur.next(p, set);
  }
  if (p.late_wait) pdl_wait();
}

// Partial results of one output row in one unit: `count` slots from `slot` on, row `row` of each;
// `twice`: rows row and row + 128 (the wide kernel's two groups took turns).
struct Parts {
  const float2* ml;
  const float* o;
  long long slot;
  int count, rows, row, twice;
  __device__ long long at(int k) const {
    return twice ? (slot + (k >> 1)) * rows + row + (k & 1) * 128 : (slot + k) * rows + row;
  }
  __device__ int parts() const { return count << twice; }
};

// Row r of stream s and head h.
template <int kRows>
__device__ __forceinline__ Parts find_parts(const AttendParams& p, const StreamSet& set, int s, int h, long long r) {
  Stream<kRows> st;
  st.load(p, set, s);
  const int tile = (int)(r / kRows);
  const int steps = st.steps(p, set, tile);
  if (steps == 0) return Parts{nullptr, nullptr, 0, 0, kRows, 0, 0};
  const long long total = set.step_base[set.prefixes + set.own];
  const long long ctas = total < set.ctas ? total : set.ctas;
  long long g = set.step_base[s] + (long long)h * st.head_work(p, set);
  if (st.len == 0) g += (long long)tile * steps;
  else
    for (int i = 0; i < tile; ++i) g += st.steps(p, set, i);
  const int c0 = (int)(((g + 1) * ctas - 1) / total), c1 = (int)(((g + steps) * ctas - 1) / total);
  const bool twice = kRows == kWideRows && (long long)st.n * p.group - (long long)tile * kRows <= 128;
  return Parts{set.part_ml, set.part_o, set.unit_base[s] + (long long)h * st.tiles + tile + c0, c1 - c0 + 1, kRows,
               (int)(r % kRows), twice};
}

constexpr int kJoinWarps = 8;

// A warp merges the parts of one output row, in their order, and writes it.
__device__ __forceinline__ void join_row(const AttendParams& p, const Parts* parts, int np, int b, int t, int hq, bool sees) {
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  for (int x = 0; x < np; ++x)
    for (int k = lane; k < parts[x].parts(); k += 32) top = fmaxf(top, parts[x].ml[parts[x].at(k)].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int x = 0; x < np; ++x) {
    const int n = parts[x].parts();
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const long long at = parts[x].at(k);
      const float2 ml = parts[x].ml[at];
      const float4 v = reinterpret_cast<const float4*>(parts[x].o + at * kHeadDim)[lane];
      const float w = weight_of(ml.x, top);
      sum += ml.y * w;
      acc.x += v.x * w;
      acc.y += v.y * w;
      acc.z += v.z * w;
      acc.w += v.w * w;
    }
  }
  const float inv = sees ? 1.f / sum : 0.f;       // a query that sees no row: zeros
  uint2 y = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (long long)b * p.ob + (long long)hq * p.oh +
                            (long long)t * p.om + 4 * lane) = y;
  if (p.lse && lane == 0)
    p.lse[((long long)b * p.hq + hq) * p.m + t] = sees ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Every output row: the parts of its prefix unit and of its own.
template <int kRows>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  const long long row = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row >= (long long)p.batch * p.hq * p.m) return;
  const int t = (int)(row % p.m), hq = (int)(row / p.m % p.hq), b = (int)(row / p.m / p.hq);
  const Seq q = sequence(p, b, !p.pages && t == 0 && hq == 0 && (threadIdx.x & 31) == 0);
  if (t >= q.n) return;
  const int h = hq / p.group, g = hq - h * p.group;
  Parts parts[2];
  int np = 0;
  if (p.fan) {
    const int s = b / p.fan;
    const long long r = (long long)(tokens_before(p, b) - tokens_before(p, s * p.fan) + t) * p.group + g;
    if (p.wide.prefixes) parts[np++] = find_parts<kWideRows>(p, p.wide, s, h, r);
    else parts[np++] = find_parts<kRows>(p, p.set, s, h, r);
  }
  if (q.len - q.n + t >= 0 && q.len > 0) {
    const long long r = (long long)t * p.group + g;
    if (p.wide.own) parts[np++] = find_parts<kWideRows>(p, p.wide, p.wide.prefixes + b, h, r);
    else parts[np++] = find_parts<kRows>(p, p.set, p.set.prefixes + b, h, r);
  }
  join_row(p, parts, np, b, t, hq, np > 0);
}

// Joint units: only those that two or more CTAs share have parts to merge. Block (c, y) takes 32 rows of
// the unit that CTA c + 1 begins inside, where that is the first CTA to begin inside it.
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_split_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  const StreamSet& set = p.wide;
  const int streams = set.prefixes + set.own;
  const long long total = set.step_base[streams];
  const long long ctas = total < set.ctas ? total : set.ctas;
  const int c = blockIdx.x + 1;
  if (c >= ctas) return;
  const long long begin = total * c / ctas;
  int lo = 0, hi = streams;                       // the last stream that begins at or before this step
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (set.step_base[mid] <= begin) lo = mid;
    else hi = mid;
  }
  Cursor<kWideRows> cur;
  cur.s = lo;
  cur.st.load(p, set, lo);
  const long long per_head = cur.st.head_work(p, set);
  long long r = begin - set.step_base[lo];
  cur.h = (int)(r / per_head);
  r -= cur.h * per_head;
  for (cur.tile = 0;; ++cur.tile) {
    cur.steps = cur.st.steps(p, set, cur.tile);
    if (r < cur.steps) break;
    r -= cur.steps;
  }
  if (r == 0) return;                             // CTA c begins with the unit
  const long long first = begin - r;              // the unit's first step
  if (c > 1 && total * (c - 1) / ctas > first) return;
  const int c1 = (int)(((first + cur.steps) * ctas - 1) / total);
  const Parts part = {set.part_ml, set.part_o, set.unit_base[lo] + (long long)cur.h * cur.st.tiles + cur.tile + c - 1,
                      c1 - (c - 1) + 1, kWideRows, 0, 0};
  for (int i = threadIdx.x >> 5; i < 32; i += kJoinWarps) {
    Parts one = part;
    one.row = blockIdx.y * 32 + i;
    const QueryRow q = query_row(p, set, cur, one.row);
    if (!q.real) continue;
    join_row(p, &one, 1, q.b, q.t, q.hq, cur.st.pre > 0 || cur.st.len - cur.st.n + q.t >= 0);
  }
}

// Boxes of `rows_box` rows of `halves` halves of 64 elements, each row 128 bytes, 128-byte swizzle.
bool encode_boxes(CUtensorMap* tm, const void* base, int rows, int heads, long long head_stride, int planes,
                  long long plane_stride, int rows_box, int halves) {
  const cuuint64_t dims[5] = {64, (cuuint64_t)rows, 2, (cuuint64_t)heads, (cuuint64_t)planes};
  const cuuint64_t strides[4] = {(cuuint64_t)kHeadDim * 2, 128, (cuuint64_t)head_stride * 2, (cuuint64_t)plane_stride * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)rows_box, (cuuint32_t)halves, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return encode_tiled()(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool multiple(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Query rows from which the wide kernel takes a unit, and above which a sequence fills one.
constexpr int kWideFrom = 33, kJointFrom = 128;

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  int few_tiles;            // query tiles of 16 rows of a unit of the few-row kernel
  StreamSet few, wide;      // counts, and offsets into the workspace in place of pointers
  size_t bytes;
  bool runs(const StreamSet& s) const { return s.prefixes + s.own > 0; }
};

// Room for a kernel's streams and partial results; sets the set's pointers (from a null base).
void lay_out(StreamSet& s, long long units, int rows, size_t& off) {
  const long long streams = s.prefixes + s.own, slots = units + s.ctas;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round256(bytes);
    return at;
  };
  if (!streams) return;
  s.step_base = reinterpret_cast<long long*>(take((size_t)(streams + 1) * 8));
  s.unit_base = reinterpret_cast<long long*>(take((size_t)streams * 8));
  s.part_ml = reinterpret_cast<float2*>(take((size_t)slots * rows * sizeof(float2)));
  s.part_o = reinterpret_cast<float*>(take((size_t)slots * rows * kHeadDim * sizeof(float)));
}
template <typename T>
void rebase(T*& x, char* base) { x = reinterpret_cast<T*>(base + reinterpret_cast<size_t>(x)); }
void rebase(StreamSet& s, char* base) {
  rebase(s.step_base, base);
  rebase(s.unit_base, base);
  rebase(s.part_ml, base);
  rebase(s.part_o, base);
}

constexpr size_t kWorkHead = 256;                 // an error word, for callers without one

// Sizes alone decide: lens and n_new are the device's.
int make_plan(const evict_attention* a, Plan* out) {
  if (!a) return fail(EVICT_EINVAL, "the arguments are NULL");
  if (a->batch < 0 || a->m < 0) return fail(EVICT_EINVAL, "batch and m must be >= 0 (got %d, %d)", a->batch, a->m);
  if (a->n_q_heads < 1 || a->n_kv_heads < 1 || a->n_q_heads % a->n_kv_heads)
    return fail(EVICT_EINVAL, "n_q_heads (%d) must be a multiple of n_kv_heads (%d)", a->n_q_heads, a->n_kv_heads);
  if (a->batch > EVICT_MAX_ATTEND_BATCH)
    return fail(EVICT_ELIMIT, "batch %d is above %d", a->batch, EVICT_MAX_ATTEND_BATCH);
  if ((long long)a->batch * a->m >= (1ll << 31) || (long long)a->batch * a->m * a->n_q_heads >= (1ll << 31))
    return fail(EVICT_ELIMIT, "batch * n_q_heads * m is 2^31 or more");
  if (a->n_prefix < 0 || a->n_prefix > (1 << 30)) return fail(EVICT_EINVAL, "n_prefix must be in [0, 2^30]");
  if (a->n_prefix > 0 && (a->prefix_batch < 1 || a->batch % a->prefix_batch))
    return fail(EVICT_EINVAL, "prefix_batch (%d) must divide batch (%d)", a->prefix_batch, a->batch);
  Plan& P = *out;
  P = Plan();
  if (a->batch == 0 || a->m == 0) return EVICT_OK;
  const int group = a->n_q_heads / a->n_kv_heads;
  const bool pre = a->n_prefix > 0;
  int dev = 0, ctas = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&ctas, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "looking up the device");
  P.few.ctas = P.wide.ctas = ctas;

  // Which kernel takes a unit goes by its query rows, the wide one from kWideFrom on. Sequences of
  // more than kJointFrom rows fill a wide unit by themselves: their units take the prefix along
  // (no partial results to merge); below that, rows of several sequences share the prefix's units.
  const long long own_rows = (long long)a->m * group, pre_rows = pre ? own_rows * (a->batch / a->prefix_batch) : 0;
  if (own_rows > kJointFrom && (pre || a->pages)) {
    P.wide.joint = 1;
    P.wide.own = a->batch;
  } else {
    if (pre) (pre_rows >= kWideFrom ? P.wide : P.few).prefixes = a->prefix_batch;
    if (a->pages) (own_rows >= kWideFrom ? P.wide : P.few).own = a->batch;
  }
  const long long few_rows = std::max(P.few.prefixes ? pre_rows : 0, P.few.own ? own_rows : 0);
  // One tile of 16 query rows where that holds every row; two (each box of K and V then serves
  // twice the rows) otherwise.
  P.few_tiles = few_rows <= 16 ? 1 : 2;
  auto units = [&](const StreamSet& s, int rows) {
    return (s.prefixes * ((pre_rows + rows - 1) / rows) + s.own * ((own_rows + rows - 1) / rows)) * a->n_kv_heads;
  };
  size_t off = kWorkHead + round256((size_t)(a->batch + 1) * sizeof(int));
  lay_out(P.few, units(P.few, 16 * P.few_tiles), 16 * P.few_tiles, off);
  lay_out(P.wide, units(P.wide, kWideRows), kWideRows, off);
  P.bytes = off;
  return EVICT_OK;
}

int check_rows(const evict_rows& x, int heads, const char* name) {
  if (!x.data) return fail(EVICT_EINVAL, "%s must not be NULL", name);
  if (x.heads != heads) return fail(EVICT_EINVAL, "%s has %d heads, not %d", name, x.heads, heads);
  if (!multiple(x.data, 16) || x.stride_b % 8 || x.stride_h % 8 || x.stride_m % 8)
    return fail(EVICT_EINVAL, "%s: addresses and strides must be multiples of 16 bytes", name);
  return EVICT_OK;
}

}  // namespace
}  // namespace evict

using namespace evict;

extern "C" int evict_shared_attention_workspace(const evict_attention* a, size_t* bytes) {
  if (!bytes) return fail(EVICT_EINVAL, "bytes is NULL");
  Plan plan;
  const int rc = make_plan(a, &plan);
  if (rc) return rc;
  *bytes = plan.bytes;
  return EVICT_OK;
}

extern "C" int evict_shared_attention(const evict_attention* a) {
  if (!a) return fail(EVICT_EINVAL, "the arguments are NULL");
  int rc;
  if (a->pages) {
    if ((rc = check_pages(a->pages))) return rc;
    if (a->pages->dtype != EVICT_BF16) return fail(EVICT_EINVAL, "attention reads bf16 pages only");
    if (a->pages->n_kv_heads != a->n_kv_heads)
      return fail(EVICT_EINVAL, "the pages hold %d KV heads, the call %d", a->pages->n_kv_heads, a->n_kv_heads);
  }
  if (!std::isfinite(a->scale)) return fail(EVICT_EINVAL, "scale must be finite");
  if (!multiple(a->n_new, 4) || !multiple(a->lse, 4) || !multiple(a->error, 4))
    return fail(EVICT_EINVAL, "n_new, lse and error must be 4-byte aligned");
  if (a->n_prefix > 0) {
    if (!a->prefix_k || !a->prefix_v) return fail(EVICT_EINVAL, "prefix_k and prefix_v must not be NULL");
    if (!multiple(a->prefix_k, 16) || !multiple(a->prefix_v, 16) || a->prefix_stride_b % 8 || a->prefix_stride_h % 8 ||
        a->prefix_stride_b < 0 || a->prefix_stride_h < 0)
      return fail(EVICT_EINVAL, "the prefix must be 16-byte aligned, with strides that are multiples of 8");
  }
  if (a->batch > 0 && a->m > 0)
    if ((rc = check_rows(a->q, a->n_q_heads, "q")) || (rc = check_rows(a->out, a->n_q_heads, "out"))) return rc;
  Plan plan;
  if ((rc = make_plan(a, &plan))) return rc;
  if (a->batch == 0 || a->m == 0) return EVICT_OK;
  if (!a->workspace || !multiple(a->workspace, 256)) return fail(EVICT_EINVAL, "workspace must be 256-byte aligned");
  if (a->workspace_bytes < plan.bytes)
    return fail(EVICT_EINVAL, "workspace has %zu bytes, the call needs %zu", a->workspace_bytes, plan.bytes);
  if (!encode_tiled()) return fail(EVICT_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");

  AttendParams P;
  memset(&P, 0, sizeof(P));
  char* ws = static_cast<char*>(a->workspace);
  P.err = a->error ? a->error : reinterpret_cast<int*>(ws);
  P.tok_base = reinterpret_cast<int*>(ws + kWorkHead);
  rebase(plan.few, ws);
  rebase(plan.wide, ws);
  P.q = a->q.data;
  P.qb = a->q.stride_b, P.qh = a->q.stride_h, P.qm = a->q.stride_m;
  P.out = a->out.data;
  P.ob = a->out.stride_b, P.oh = a->out.stride_h, P.om = a->out.stride_m;
  P.lse = a->lse;
  P.batch = a->batch, P.m = a->m, P.hq = a->n_q_heads, P.hkv = a->n_kv_heads;
  P.group = a->n_q_heads / a->n_kv_heads;
  if (a->n_prefix > 0) {
    P.prefix_batch = a->prefix_batch;
    P.fan = a->batch / a->prefix_batch;
    P.n_prefix = a->n_prefix;
  }
  P.scale2 = (a->scale == 0.f ? 0.08838834764831845f : a->scale) * kLog2e;
  P.n_new = a->n_new;
  const evict_pages* g = a->pages;
  if (g) {
    P.pages = 1;
    P.table = g->table;
    P.table_stride = g->table_stride ? g->table_stride : g->table_width;
    P.table_width = g->table_width;
    P.page_shift = __builtin_ctz((unsigned)g->page_size);
    P.n_pages = g->n_pages;
    P.lens = g->lens;
    P.page_k = g->k;
    P.page_v = g->v;
    P.page_stride = g->page_stride ? g->page_stride : (long long)g->n_kv_heads * g->page_size * kHeadDim;
  }
  // The boxes of one of the kernels: 16 whole rows, or up to 128 rows of one half.
  auto encode = [&](bool wide, const StreamSet& s) {
    if (s.prefixes || (s.joint && P.fan)) {
      // a dimension of extent 1 is never stepped over, but its stride still has to be one the encoder takes
      const long long hs = P.hkv > 1 ? a->prefix_stride_h : (long long)P.n_prefix * kHeadDim;
      const long long bs = P.prefix_batch > 1 ? a->prefix_stride_b : P.hkv * hs;
      for (int v = 0; v < 2; ++v)
        if (!encode_boxes(v ? &P.tm_pv : &P.tm_pk, v ? a->prefix_v : a->prefix_k, P.n_prefix, P.hkv, hs, P.prefix_batch, bs,
                          wide ? kStepTokens : kBoxTokens, wide ? 1 : 2))
          return fail(EVICT_EINVAL, "the prefix has sizes or strides beyond a tensor map's");
    }
    if (s.own && g) {
      P.box_rows = std::min(g->page_size, kStepTokens);
      for (int v = 0; v < 2; ++v)
        if (!encode_boxes(v ? &P.tm_v : &P.tm_k, v ? g->v : g->k, g->page_size, P.hkv, (long long)g->page_size * kHeadDim,
                          g->n_pages, P.page_stride, wide ? P.box_rows : kBoxTokens, wide ? 1 : 2))
          return fail(EVICT_EINVAL, "the pages have sizes or strides beyond a tensor map's");
    }
    return (int)EVICT_OK;
  };
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  cudaError_t e = cudaSuccess;
  const bool few = plan.runs(plan.few), wide = plan.runs(plan.wide);
  if (wide) {
    if ((rc = encode(true, plan.wide))) return rc;
    P.set = plan.wide;
    if ((e = prepare_wide()) != cudaSuccess || (e = launch_wide(P, few, st)) != cudaSuccess)
      return cuda_fail(e, "wide attention kernel launch");
    g_launches.fetch_add(1);
    P.late_wait = 1;                              // the few-row kernel needs nothing of the wide one's
  }
  P.set = plan.few;
  P.wide = plan.wide;
  if (few) {
    if ((rc = encode(false, plan.few))) return rc;
    auto go = [&](auto kernel, int tiles) {
      const cudaError_t x = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem(tiles));
      return x != cudaSuccess ? x : launch_pdl(kernel, dim3(plan.few.ctas), dim3(kThreads), few_smem(tiles), st, nullptr, P);
    };
    e = plan.few_tiles == 1 ? go(attend_kernel<1>, 1) : go(attend_kernel<2>, 2);
    if (e != cudaSuccess) return cuda_fail(e, "attention kernel launch");
    g_launches.fetch_add(1);
  }
  if (plan.wide.joint) {
    if (plan.wide.ctas > 1)
      e = launch_pdl(attend_join_split_kernel, dim3(plan.wide.ctas - 1, kWideRows / 32), dim3(kJoinWarps * 32), 0, st, nullptr, P);
  } else {
    const long long rows = (long long)a->batch * a->n_q_heads * a->m;
    const dim3 grid((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), block(kJoinWarps * 32);
    e = plan.few_tiles == 1 ? launch_pdl(attend_join_kernel<16>, grid, block, 0, st, nullptr, P)
                            : launch_pdl(attend_join_kernel<32>, grid, block, 0, st, nullptr, P);
  }
  g_launches.fetch_add(1);
  return e == cudaSuccess ? EVICT_OK : cuda_fail(e, "attention kernel launch");
}
