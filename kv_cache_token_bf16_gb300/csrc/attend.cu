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
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* tmap, int x, int y, int z, int w, int v,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(tc::smem_u32(bar))
      : "memory");
}
// Bit 0: the lower bf16 of the pair is an infinity or NaN; bit 1: the upper.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) {
  return ((x & 0x7f80u) == 0x7f80u ? 1u : 0u) | ((x & 0x7f800000u) == 0x7f800000u ? 2u : 0u);
}

// Where a weight meets no finite maximum (no row seen yet, or every logit -inf or NaN) the
// exponent is taken against 0, so that masked rows stay 0 and NaN stays NaN.
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float weight_of(float m, float to) { return m == to ? 1.f : ex2(m - base_of(to)); }

// New rows and visible rows of a sequence.
struct Seq {
  int n, len;                        // new tokens; rows, the new ones included
};
__device__ __forceinline__ Seq sequence(const AttendParams& p, int b, bool report) {
  int n = p.n_new ? p.n_new[b] : p.m;
  bool odd = n < 0 || n > p.m;
  n = n < 0 ? 0 : n > p.m ? p.m : n;
  int len = p.own ? p.lens[b] : 0;
  const int room = p.own ? p.table_width << p.page_shift : 0;
  odd = odd || len < 0 || len > room;
  len = len < 0 ? 0 : len > room ? room : len;
  if (odd && report) raise_device_error(p.err, kDevBadIndex);
  return {n, len};
}

// Stream s: row tiles of a unit and steps of a row tile.
template <int kRows>
struct Stream {
  int tiles, steps, n, len;
  __device__ void load(const AttendParams& p, int s, bool report = false) {
    if (s < p.prefixes) {
      n = p.m;
      len = p.n_prefix;
      tiles = p.prefix_tiles;
    } else {
      const Seq q = sequence(p, s - p.prefixes, report);
      n = q.n;
      len = q.len;
      tiles = (n * p.group + kRows - 1) / kRows;
    }
    steps = (len + kStepTokens - 1) / kStepTokens;
    if (tiles == 0 || steps == 0) tiles = steps = 0;
  }
  __device__ long long work(const AttendParams& p) const { return (long long)tiles * steps * p.hkv; }
};

// Position in the line of steps.
template <int kRows>
struct Cursor {
  int s, h, tile, step;
  Stream<kRows> st;
  __device__ void next(const AttendParams& p, int streams) {
    if (++step < st.steps) return;
    step = 0;
    if (++tile < st.tiles) return;
    tile = 0;
    if (++h < p.hkv) return;
    h = 0;
    do {
      if (++s >= streams) return;
      st.load(p, s);
    } while (st.steps == 0);
  }
};

// Rows of this tile see own rows up to `last`: row r of the unit is token r / group.
template <int kRows>
__device__ __forceinline__ int last_row(const AttendParams& p, const Cursor<kRows>& c, int r) {
  if (c.s < p.prefixes) return p.n_prefix - 1;
  const int t = r / p.group;
  return t < c.st.n ? c.st.len - c.st.n + t : -1;
}

struct FewShared {
  uint64_t full[kWarps][kStages];
  long long begin, total;
  int s;
  long long rest, unit;
  long long sums[kWarps], usums[kWarps];
  int fail;
};

template <int kTiles>
__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kRows = 16 * kTiles;
  constexpr int kCols = merge_cols(kTiles);
  pdl_wait();
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ FewShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* ring = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* qs = ring + kRingBytes;
  float* red = reinterpret_cast<float*>(qs + kRows * kQPitch);          // [warp][row][kCols + 4]
  float2* red_ml = reinterpret_cast<float2*>(red + kWarps * kRows * (kCols + 4));
  const int streams = p.prefixes + (p.own ? p.batch : 0);

  if (tid < kWarps * kStages) tc::mbar_init(&sh.full[tid / kStages][tid % kStages], 1);
  if (tid == 0) sh.fail = 0;

  // --- this CTA's share: a block scan over the streams' steps and units ---
  {
    const int per = (streams + kThreads - 1) / kThreads;
    const int s0 = min(tid * per, streams), s1 = min(s0 + per, streams);
    long long steps = 0, units = 0;
    Stream<kRows> st;
    for (int s = s0; s < s1; ++s) {
      st.load(p, s, blockIdx.x == 0);
      steps += st.work(p);
      units += (long long)st.tiles * p.hkv;
    }
    long long a = steps, u = units;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, u, d);
      if (lane >= d) a += x, u += y;
    }
    if (lane == 31) sh.sums[warp] = a, sh.usums[warp] = u;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) a += sh.sums[w], u += sh.usums[w];
      total += sh.sums[w];
    }
    a -= steps;
    u -= units;
    const long long ctas = total < p.ctas ? total : p.ctas;
    const long long mine = ctas ? total * blockIdx.x / ctas : 0;
    if (blockIdx.x == 0) {                        // where the join finds every stream
      long long x = a, y = u;
      for (int s = s0; s < s1; ++s) {
        st.load(p, s);
        p.step_base[s] = x;
        p.unit_base[s] = y;
        x += st.work(p);
        y += (long long)st.tiles * p.hkv;
      }
      if (tid == kThreads - 1) p.step_base[streams] = total;
    }
    if (tid == 0) sh.total = total;
    if (blockIdx.x < ctas && mine >= a && mine < a + steps) {
      int s = s0;
      for (; s < s1; ++s) {
        st.load(p, s);
        if (mine < a + st.work(p)) break;
        a += st.work(p);
        u += (long long)st.tiles * p.hkv;
      }
      sh.s = s;
      sh.rest = mine - a;
      sh.unit = u;
      sh.begin = mine;
    }
    __syncthreads();
    if (blockIdx.x >= ctas) return;
  }
  const long long ctas = sh.total < p.ctas ? sh.total : p.ctas;
  const int count = (int)(sh.total * (blockIdx.x + 1) / ctas - sh.begin);    // steps of this CTA

  Cursor<kRows> cur;
  cur.s = sh.s;
  cur.st.load(p, cur.s);
  {
    const long long per_head = (long long)cur.st.tiles * cur.st.steps;
    cur.h = (int)(sh.rest / per_head);
    const int r = (int)(sh.rest - cur.h * per_head);
    cur.tile = r / cur.st.steps;
    cur.step = r - cur.tile * cur.st.steps;
  }
  long long unit = sh.unit + (long long)cur.h * cur.st.tiles + cur.tile;

  // Does this warp have rows to read at this step? (its box begins inside the stream, and the
  // tile's last token sees its first row)
  auto active = [&](const Cursor<kRows>& c) {
    const int row0 = c.step * kStepTokens + kBoxTokens * warp;
    if (row0 >= c.st.len) return false;
    if (c.s < p.prefixes) return true;
    const int t = min((kRows * (c.tile + 1) - 1) / p.group, c.st.n - 1);
    return row0 <= c.st.len - c.st.n + t;
  };

  // --- the ring: boxes are requested in the order in which they are used ---
  const uint32_t my_ring = tc::smem_u32(ring) + warp * kStages * 2 * kBoxBytes;
  Cursor<kRows> ahead = cur;
  int ahead_left = count, page = 0;
  // advance `ahead` to the next box of this warp and look its page up
  auto seek = [&] {
    while (ahead_left > 0 && !active(ahead)) {
      ahead.next(p, streams);
      --ahead_left;
    }
    if (ahead_left > 0 && ahead.s >= p.prefixes && lane == 0)
      page = p.table[(long long)(ahead.s - p.prefixes) * p.table_stride +
                     ((ahead.step * kStepTokens + kBoxTokens * warp) >> p.page_shift)];
  };
  auto request = [&](int stage) {
    if (ahead_left <= 0) return;
    if (lane == 0) {
      uint64_t* bar = &sh.full[warp][stage];
      const uint32_t dst = my_ring + stage * 2 * kBoxBytes;
      const int row = ahead.step * kStepTokens + kBoxTokens * warp;
      tc::mbar_arrive_expect_tx(bar, 2 * kBoxBytes);
      if (ahead.s < p.prefixes) {
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
    ahead.next(p, streams);
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
        const int r = e >> 4, c = e & 15, ur = cur.tile * kRows + r;
        const bool pre = cur.s < p.prefixes;
        const int per_seq = p.m * p.group;
        const int b = pre ? cur.s * p.fan + ur / per_seq : cur.s - p.prefixes;
        const int rr = pre ? ur % per_seq : ur;
        const int t = rr / p.group, hq = cur.h * p.group + rr % p.group;
        const bool real = pre ? ur < p.fan * per_seq : t < cur.st.n;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (real)
          x = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (long long)b * p.qb +
                                              (long long)hq * p.qh + (long long)t * p.qm + c * 8);
        *reinterpret_cast<uint4*>(qs + r * kQPitch + c * 16) = x;
      }
      __syncthreads();
      low = cur.s < p.prefixes ? p.n_prefix - 1 : last_row(p, cur, cur.tile * kRows);
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
          last[x][k] = last_row(p, cur, cur.tile * kRows + 16 * x + (lane >> 2) + 8 * k);
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
          const int r0 = row0 + 2 * (lane & 3);
          auto mask = [&](int r) { return (r < cur.st.len ? 0xffffu : 0u) | (r + 1 < cur.st.len ? 0xffff0000u : 0u); };
          keep0 = mask(r0);
          keep1 = mask(r0 + 8);
        }
        const int vrow = lane & 15, vchunk = lane >> 4;
        uint32_t bad = 0;                         // tokens of the box whose V holds an infinity or NaN
        if (!full && p.m > 1 && cur.s >= p.prefixes) {
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
    if (cur.step == cur.st.steps - 1 || i == count - 1) {
      const long long slot = unit + blockIdx.x;
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
        p.part_ml[slot * kRows + tid] = make_float2(top, t);
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
          *reinterpret_cast<float2*>(p.part_o + (slot * kRows + r) * kHeadDim + c * kCols + cc) = a;
        }
        __syncthreads();
      }
      fresh = true;
      ++unit;
    }
    cur.next(p, streams);
  }
}

// Partial results of one output row: `count` slots from `first`, row `row` of each.
struct Parts {
  long long first;
  int count, row;
};

template <int kRows>
__device__ __forceinline__ Parts find_parts(const AttendParams& p, long long total, long long ctas, int s, int h,
                                            int tiles, int steps, int r) {
  const int tile = r / kRows;
  const long long g = p.step_base[s] + ((long long)h * tiles + tile) * steps;
  const int c0 = (int)(((g + 1) * ctas - 1) / total), c1 = (int)(((g + steps) * ctas - 1) / total);
  return {p.unit_base[s] + (long long)h * tiles + tile + c0, c1 - c0 + 1, r % kRows};
}

constexpr int kJoinWarps = 8;

template <int kRows>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (row >= (long long)p.batch * p.hq * p.m) return;
  const int t = (int)(row % p.m), hq = (int)(row / p.m % p.hq), b = (int)(row / p.m / p.hq);
  const Seq q = sequence(p, b, !p.own && t == 0 && hq == 0 && lane == 0);
  if (t >= q.n) return;
  const int h = hq / p.group, g = hq - h * p.group;
  const int streams = p.prefixes + (p.own ? p.batch : 0);
  const long long total = p.step_base[streams];
  const long long ctas = total < p.ctas ? total : p.ctas;
  Parts parts[2];
  int np = 0;
  if (p.prefixes) {
    const int s = b / p.fan, steps = (p.n_prefix + kStepTokens - 1) / kStepTokens;
    parts[np++] = find_parts<kRows>(p, total, ctas, s, h, p.prefix_tiles, steps,
                                    ((b - s * p.fan) * p.m + t) * p.group + g);
  }
  const bool sees_own = q.len - q.n + t >= 0 && q.len > 0;
  if (sees_own) {
    const int tiles = (q.n * p.group + kRows - 1) / kRows, steps = (q.len + kStepTokens - 1) / kStepTokens;
    parts[np++] = find_parts<kRows>(p, total, ctas, p.prefixes + b, h, tiles, steps, t * p.group + g);
  }
  float top = -INFINITY;
  for (int x = 0; x < np; ++x)
    for (int k = lane; k < parts[x].count; k += 32)
      top = fmaxf(top, p.part_ml[(parts[x].first + k) * kRows + parts[x].row].x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int x = 0; x < np; ++x) {
#pragma unroll 4
    for (int k = 0; k < parts[x].count; ++k) {
      const long long at = (parts[x].first + k) * kRows + parts[x].row;
      const float2 ml = p.part_ml[at];
      const float4 v = reinterpret_cast<const float4*>(p.part_o + at * kHeadDim)[lane];
      const float w = weight_of(ml.x, top);
      sum += ml.y * w;
      acc.x += v.x * w;
      acc.y += v.y * w;
      acc.z += v.z * w;
      acc.w += v.w * w;
    }
  }
  const float inv = np ? 1.f / sum : 0.f;         // a query that sees no row: zeros
  uint2 y = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (long long)b * p.ob + (long long)hq * p.oh +
                            (long long)t * p.om + 4 * lane) = y;
  if (p.lse && lane == 0) p.lse[row] = np ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Boxes of 16 rows: two halves of 64 elements, each row 128 bytes, 128-byte swizzle.
bool encode_boxes(CUtensorMap* tm, const void* base, int rows, int heads, long long head_stride, int planes,
                  long long plane_stride) {
  const cuuint64_t dims[5] = {64, (cuuint64_t)rows, 2, (cuuint64_t)heads, (cuuint64_t)planes};
  const cuuint64_t strides[4] = {(cuuint64_t)kHeadDim * 2, 128, (cuuint64_t)head_stride * 2, (cuuint64_t)plane_stride * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)kBoxTokens, 2, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return encode_tiled()(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool multiple(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  int tiles;                // query tiles of 16 rows a unit
  int prefixes, prefix_tiles, streams, ctas;
  long long slots;
  size_t off_unit, off_ml, off_o, bytes;
};

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
  const int group = a->n_q_heads / a->n_kv_heads;
  const bool pre = a->n_prefix > 0;
  Plan& P = *out;
  P.bytes = 0;
  if (a->batch == 0 || a->m == 0) return EVICT_OK;
  P.prefixes = pre ? a->prefix_batch : 0;
  const long long fan = pre ? a->batch / a->prefix_batch : 0;
  const long long most = std::max(pre ? fan * a->m * group : 0, a->pages ? (long long)a->m * group : 0);
  // One tile of 16 query rows where that holds every row; two (each box of K and V then serves
  // twice the rows) otherwise.
  P.tiles = most <= 16 ? 1 : 2;
  const int rows = 16 * P.tiles;
  P.prefix_tiles = pre ? (int)((fan * a->m * group + rows - 1) / rows) : 0;
  P.streams = P.prefixes + (a->pages ? a->batch : 0);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&P.ctas, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "looking up the device");
  const long long own_tiles = a->pages ? ((long long)a->m * group + rows - 1) / rows : 0;
  P.slots = ((long long)P.prefixes * P.prefix_tiles + (a->pages ? a->batch : 0) * own_tiles) * a->n_kv_heads + P.ctas;
  P.off_unit = 256 + round256((size_t)(P.streams + 1) * 8);
  P.off_ml = P.off_unit + round256((size_t)P.streams * 8 + 8);
  P.off_o = P.off_ml + round256((size_t)P.slots * rows * sizeof(float2));
  P.bytes = P.off_o + (size_t)P.slots * rows * kHeadDim * sizeof(float);
  return EVICT_OK;
}

int check_rows(const evict_rows& x, int heads, const char* name) {
  if (!x.data) return fail(EVICT_EINVAL, "%s must not be NULL", name);
  if (x.heads != heads) return fail(EVICT_EINVAL, "%s has %d heads, not %d", name, x.heads, heads);
  if (!multiple(x.data, 16) || x.stride_b % 8 || x.stride_h % 8 || x.stride_m % 8)
    return fail(EVICT_EINVAL, "%s: addresses and strides must be multiples of 16 bytes", name);
  return EVICT_OK;
}

template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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
  P.step_base = reinterpret_cast<long long*>(ws + 256);
  P.unit_base = reinterpret_cast<long long*>(ws + plan.off_unit);
  P.part_ml = reinterpret_cast<float2*>(ws + plan.off_ml);
  P.part_o = reinterpret_cast<float*>(ws + plan.off_o);
  P.q = a->q.data;
  P.qb = a->q.stride_b, P.qh = a->q.stride_h, P.qm = a->q.stride_m;
  P.out = a->out.data;
  P.ob = a->out.stride_b, P.oh = a->out.stride_h, P.om = a->out.stride_m;
  P.lse = a->lse;
  P.batch = a->batch, P.m = a->m, P.hq = a->n_q_heads, P.hkv = a->n_kv_heads;
  P.group = a->n_q_heads / a->n_kv_heads;
  P.prefixes = plan.prefixes;
  P.fan = plan.prefixes ? a->batch / plan.prefixes : 1;
  P.n_prefix = plan.prefixes ? a->n_prefix : 0;
  P.prefix_tiles = plan.prefix_tiles;
  P.scale2 = (a->scale == 0.f ? 0.08838834764831845f : a->scale) * kLog2e;
  P.n_new = a->n_new;
  P.ctas = plan.ctas;
  if (plan.prefixes) {
    // a dimension of extent 1 is never stepped over, but its stride still has to be one the encoder takes
    const long long hs = a->n_kv_heads > 1 ? a->prefix_stride_h : (long long)a->n_prefix * kHeadDim;
    const long long bs = plan.prefixes > 1 ? a->prefix_stride_b : (long long)a->n_kv_heads * hs;
    if (!encode_boxes(&P.tm_pk, a->prefix_k, a->n_prefix, a->n_kv_heads, hs, plan.prefixes, bs) ||
        !encode_boxes(&P.tm_pv, a->prefix_v, a->n_prefix, a->n_kv_heads, hs, plan.prefixes, bs))
      return fail(EVICT_EINVAL, "the prefix has sizes or strides beyond a tensor map's");
  }
  if (a->pages) {
    const evict_pages* g = a->pages;
    const long long ps = g->page_stride ? g->page_stride : (long long)g->n_kv_heads * g->page_size * kHeadDim;
    const long long hs = (long long)g->page_size * kHeadDim;
    if (!encode_boxes(&P.tm_k, g->k, g->page_size, g->n_kv_heads, hs, g->n_pages, ps) ||
        !encode_boxes(&P.tm_v, g->v, g->page_size, g->n_kv_heads, hs, g->n_pages, ps))
      return fail(EVICT_EINVAL, "the pages have sizes or strides beyond a tensor map's");
    P.own = 1;
    P.table = g->table;
    P.table_stride = g->table_stride ? g->table_stride : g->table_width;
    P.table_width = g->table_width;
    P.page_shift = __builtin_ctz((unsigned)g->page_size);
    P.n_pages = g->n_pages;
    P.lens = g->lens;
  }
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  cudaError_t e;
  const long long out_rows = (long long)a->batch * a->n_q_heads * a->m;
  const dim3 join((unsigned)((out_rows + kJoinWarps - 1) / kJoinWarps));
  if (plan.tiles == 1) {
    if ((e = allow_smem(attend_kernel<1>, few_smem(1))) != cudaSuccess) return cuda_fail(e, "attention kernel attribute");
    e = launch_pdl(attend_kernel<1>, dim3(plan.ctas), dim3(kThreads), few_smem(1), st, nullptr, P);
    if (e == cudaSuccess) e = launch_pdl(attend_join_kernel<16>, join, dim3(kJoinWarps * 32), 0, st, nullptr, P);
  } else {
    if ((e = allow_smem(attend_kernel<2>, few_smem(2))) != cudaSuccess) return cuda_fail(e, "attention kernel attribute");
    e = launch_pdl(attend_kernel<2>, dim3(plan.ctas), dim3(kThreads), few_smem(2), st, nullptr, P);
    if (e == cudaSuccess) e = launch_pdl(attend_join_kernel<32>, join, dim3(kJoinWarps * 32), 0, st, nullptr, P);
  }
  g_launches.fetch_add(2);
  return e == cudaSuccess ? EVICT_OK : cuda_fail(e, "attention kernel launch");
}
