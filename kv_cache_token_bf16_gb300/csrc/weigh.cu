// The weights that a step's queries put on the kept rows of a cache, added to the rows' scores:
//   score_j += sum over the sequences of a kept prefix, their tokens and the group's query heads of
//              exp(scale q.k_j - lse).
//
// Few queries (weigh_kernel): a warp takes 32 keys, straight from memory to the registers of m16n8k16 products (their
// rows; a lane's 16-byte pieces of a row stand for the product's columns in another order, the same for the queries),
// and goes through the queries eight at a time, which come from L1 and L2. A key's sum lies in four lanes. Keys are
// read once: what bounds it is HBM, 4.2 of 6.8 TB/s for one token of 32 caches of 512 rows (32 / 8 heads; 7.9 to 8.6
// us). Where there are fewer warps of keys than the GPU has room for, the queries are dealt out to up to eight warps for
// the same keys. 320 queries over 16384 rows were bound by these products (65 us).
// Many (weigh_wide_kernel): the large products of the tensor cores, bound by HBM up to about a hundred queries and by
// the exponentials behind that: 8 heads' 16384 rows by 64 queries 10.9 us (3.1 TB/s), by 320 22.2, by 1024 52 (0.66
// PFLOP/s; their exponentials, at 32 a clock and SM, are 14 us). The rest is the launch and the laying out of the
// queries, some 3 us once a chunk, in which nothing else runs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "api_internal.h"
#include "attend.h"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "prompt.cuh"
#include "prompt.h"
#include "tmem.cuh"

namespace evict {
namespace {

constexpr int kWarps = 8, kKeys = 32, kQueries = 8;
constexpr int kScan = kWarps * 32;                // query rows that are looked through at once

struct WeighParams {
  const void* k;                     // [batch][heads][cap][128]
  float* score;                      // [batch][heads][cap]
  int cap, rows, heads;              // rows: kept
  const void* q;
  long long qb, qh, qm;              // element strides
  const float* lse;                  // [sequences][hq][m]
  const int32_t* n_new;
  int fan, m, hq, group, seqs;       // fan: sequences of a cache's batch row
  int queries;                       // fan * m * group
  int split;                         // warps that share the queries of the same keys
  Divisor by_heads, by_per, by_group;   // per = m * group: query rows of a sequence
  float scale2;
  int* err;
};

// -lse in base 2, and what its rounding left out as a factor of the weights: 2^(x + neg) rest. (A large weight's relative
// error is the exponent's, and a log-sum-exp of 11 has 2^-20 of one in base 2: a step's few queries add up no others.)
struct Lse {
  float neg, rest;
};
__device__ __forceinline__ Lse base2(float l) {
  const float neg = -l * kLog2e, lo = fmaf(-l, kLog2e, -neg) - l * kLog2eRest;
  return {neg, fabsf(lo) < 1e-3f ? fmaf(lo, 0.69314718f, 1.f) : 1.f};
}

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A tile's queries as a lane holds them: its pieces of one row, and the row's log-sum-exp (base 2, negative;
// -inf: the query does not count).
struct Queries {
  uint4 x[4];
  Lse lse;
};

__global__ void __launch_bounds__(kWarps * 32, 2) weigh_kernel(const __grid_constant__ WeighParams p) {
  __shared__ float sums[kWarps][kKeys];
  __shared__ long long at[kScan];                 // of the queries that count: where their rows lie in q,
  __shared__ int lse_at[kScan];                   // and their log-sum-exps
  __shared__ int counts[kWarps];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % p.split;
  const int unit = blockIdx.y, b = p.by_heads.div(unit), h = unit - b * p.heads;
  const int row0 = (blockIdx.x * (kWarps / p.split) + warp / p.split) * kKeys;
  const int n = lane >> 2, t = lane & 3;          // row of a fragment, and which pieces of it
  const __nv_bfloat16* keys = static_cast<const __nv_bfloat16*>(p.k) + (long long)unit * p.cap * kHeadDim;
  uint4 a[4][4];                                  // key n + 8 i, elements 32 j + 8 t ..
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + n + 8 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a[i][j] = row < p.rows ? reinterpret_cast<const uint4*>(keys + (long long)row * kHeadDim)[4 * j + t]
                             : make_uint4(0, 0, 0, 0);
  }
  float sum[4] = {0.f, 0.f, 0.f, 0.f};            // of keys row0 + n + 8 i
#pragma unroll 1
  for (int c0 = 0; c0 < p.queries; c0 += kScan) {
    // a thread's query row: sequence, token, head of the group
    const int c = c0 + threadIdx.x, f = p.by_per.div(c), in = c - f * p.m * p.group, tok = p.by_group.div(in);
    const int seq = b * p.fan + f, hq = h * p.group + in - tok * p.group;
    const bool counts_here = c < p.queries && (!p.n_new || tok < p.n_new[seq]);
    const uint32_t mine = __ballot_sync(0xffffffffu, counts_here);
    if (c0) __syncthreads();                      // the last ones are worked off
    if (lane == 0) counts[warp] = __popc(mine);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i == warp) before = total;
      total += counts[i];
    }
    if (counts_here) {
      const int i = before + __popc(mine & ((1u << lane) - 1));
      at[i] = seq * p.qb + hq * p.qh + tok * p.qm;
      lse_at[i] = (seq * p.hq + hq) * p.m + tok;
    }
    __syncthreads();
    if (row0 >= p.rows) continue;
    auto load = [&](int r0) {
      Queries q;
      const int r = r0 + n;
#pragma unroll
      for (int j = 0; j < 4; ++j) q.x[j] = make_uint4(0, 0, 0, 0);
      q.lse = {-INFINITY, 1.f};
      if (r < total) {
        const float l = p.lse[lse_at[r]];
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) q.x[j] = row[4 * j + t];
        q.lse = base2(l);
        if (l == -INFINITY) q.lse.neg = l;
      }
      return q;
    };
    Queries next = load(part * kQueries);
#pragma unroll 1
    for (int r0 = part * kQueries; r0 < total; r0 += p.split * kQueries) {
      const Queries q = next;
      next = load(r0 + p.split * kQueries);
      float d[2][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 &u = a[2 * i][j], &v = a[2 * i + 1][j];
          mma(d[i], u.x, v.x, u.y, v.y, q.x[j].x, q.x[j].y);
          mma(d[i], u.z, v.z, u.w, v.w, q.x[j].z, q.x[j].w);
        }
      // columns 2 t and 2 t + 1 are the queries of lanes 8 t and 8 t + 4
      const float n0 = __shfl_sync(0xffffffffu, q.lse.neg, 8 * t), n1 = __shfl_sync(0xffffffffu, q.lse.neg, 8 * t + 4);
      const float f0 = __shfl_sync(0xffffffffu, q.lse.rest, 8 * t), f1 = __shfl_sync(0xffffffffu, q.lse.rest, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float w0 = n0 == -INFINITY ? 0.f : ex2(fmaf(d[i][2 * k], p.scale2, n0));
          const float w1 = n1 == -INFINITY ? 0.f : ex2(fmaf(d[i][2 * k + 1], p.scale2, n1));
          sum[2 * i + k] += fmaf(w0, f0, w1 * f1);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
  }
  if (t == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][n + 8 * i] = sum[i];
  }
  if (p.split > 1) __syncthreads();
  else __syncwarp();
  const int row = row0 + lane;
  if (part == 0 && row < p.rows) {
    float all = sums[warp][lane];
    for (int i = 1; i < p.split; ++i) all += sums[warp + i][lane];
    p.score[(long long)unit * p.cap + row] += all;
  }
  if (p.n_new && p.err && blockIdx.x == 0 && h == 0)
    for (int f = threadIdx.x; f < p.fan; f += blockDim.x) {
      const int c = p.n_new[b * p.fan + f];
      if (c < 0 || c > p.m) raise_device_error(p.err, kDevBadIndex);
    }
}

// Many queries: the tensor cores' large products, in 128 keys by 128 queries, D[key, query] in tensor memory. A CTA
// takes an equal share of the key tiles. Of a unit's queries it lays up to kChunk that count into shared memory
// once, behind each other, and goes through its tiles of the unit by them; a warp sums 32 keys of every other tile over
// 64 queries of each product. (Of every tile over 32, so that what it does once a product counts twice: 14.6 us instead
// of 13.4 for some 190 queries over 8 heads' 16384 rows.)
constexpr int kTile = 128, kTileBytes = kTile * kHeadDim * 2;
constexpr int kChunk = 256, kKeyRing = 4, kBuffers = 4;
constexpr int kSumWarps = 16, kIssueWarp = 16, kCopyWarp = 17, kWideThreads = 576;

struct WideShared {
  uint64_t k_full[kKeyRing], k_empty[kKeyRing], s_full[kBuffers], s_empty[kBuffers], done;
  uint64_t sums_full[4][2], sums_empty[4][2];     // of a quarter of the keys, of every other tile
  uint32_t tmem_base;
  int fail, next;                                 // next: first query row behind the chunk's
  int counts[kSumWarps];
  long long at[kChunk];                           // where the chunk's query rows lie in q,
  alignas(16) float neg[kChunk], rest[kChunk];    // and their log-sum-exps
  float sums[2][kTile];
};
constexpr int kWideSmem = (kKeyRing + kChunk / kTile) * kTileBytes + (int)sizeof(WideShared);
static_assert(kWideSmem <= 227 * 1024);

struct WideParams {
  WeighParams w;
  CUtensorMap k_map;
  int tiles;                                      // of a unit
  long long all;                                  // of all
  Divisor by_tiles;
};

// The next query rows from c0 on that count, at most kChunk, to shared memory; their number. By all threads.
__device__ int lay_queries(const WeighParams& p, WideShared& sh, uint32_t rows, int b, int h, int c0) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = c0 + tid;
  bool counts_here = false;
  long long at = 0;
  float l = 0.f;
  if (warp < kSumWarps && c < p.queries) {
    const int f = p.by_per.div(c), in = c - f * p.m * p.group, tok = p.by_group.div(in);
    const int seq = b * p.fan + f, hq = h * p.group + in - tok * p.group;
    const int news = p.n_new ? p.n_new[seq] : p.m;
    l = p.lse[((long long)seq * p.hq + hq) * p.m + tok];
    // (no weights of a query that saw nothing, or with all of them elsewhere)
    counts_here = tok < news && fabsf(l) != INFINITY;
    at = seq * p.qb + hq * p.qh + tok * p.qm;
  }
  const uint32_t mine = __ballot_sync(0xffffffffu, counts_here);
  if (lane == 0 && warp < kSumWarps) sh.counts[warp] = __popc(mine);
  if (tid == 0) sh.next = c0 + kSumWarps * 32;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kSumWarps; ++i) {
    if (i == warp) before = total;
    total += sh.counts[i];
  }
  if (counts_here) {
    const int i = before + __popc(mine & ((1u << lane) - 1));
    if (i < kChunk) {
      sh.at[i] = at;
      const Lse x = base2(l);
      sh.neg[i] = x.neg;
      sh.rest[i] = x.rest;
      if (i == kChunk - 1) sh.next = c + 1;
    }
  }
  // (none once a wait has given up: no thread is between these barriers and a wait)
  total = *(volatile int*)&sh.fail ? 0 : min(total, kChunk);
  __syncthreads();
  // 128-byte halves of the rows, their 16-byte pieces in the order of a 128-byte swizzle
#pragma unroll 4
  for (int i = tid; i < total * 16; i += kWideThreads) {
    const int r = i >> 4, piece = i & 15;
    const uint32_t to = rows + (r / kTile) * kTileBytes + (piece >> 3) * (kTileBytes / 2) + (r % kTile) * 128 +
                        (((piece & 7) ^ (r & 7)) << 4);
    const void* from = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + sh.at[r]) + piece;
    tc::cp_async16(to, from, 16);
  }
  tc::cp_async_wait_all();
  tc::fence_proxy_async_smem();
  __syncthreads();
  return total;
}

// Tiles first .. last - 1 of the unit's keys into the ring, by one thread. `used` counts the ring's tiles.
__device__ __forceinline__ bool copy_tiles(const WideParams& p, WideShared& sh, uint32_t ring, int b, int h, int first, int last,
                                           int& used) {
#pragma unroll 1
  for (int t = first; t < last; ++t, ++used) {
    const int i = used % kKeyRing;
    if (!wait_for(&sh.k_empty[i], ((used / kKeyRing) & 1) ^ 1, &sh.fail)) return false;
    tc::mbar_arrive_expect_tx(&sh.k_full[i], kTileBytes);
    for (int j = 0; j < 2; ++j)
      tma_load_4d(ring + i * kTileBytes + j * (kTileBytes / 2), &p.k_map, j * 64, t * kTile, h, b, &sh.k_full[i]);
  }
  return true;
}

__global__ void __launch_bounds__(kWideThreads, 1) weigh_wide_kernel(const __grid_constant__ WideParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t smem = tc::smem_u32(smem_raw), queries = smem + kKeyRing * kTileBytes;
  WideShared& sh = *reinterpret_cast<WideShared*>(smem_raw + (kKeyRing + kChunk / kTile) * kTileBytes);
  const WeighParams& w = p.w;
  if (smem & 1023) {                              // not as declared: no tile could be right
    if (threadIdx.x == 0) raise_device_error(w.err, kDevBadIndex);
    return;
  }
  const int tid = threadIdx.x, warp = uni(tid >> 5), lane = tid & 31;
  if (warp == 0) tc::tmem_alloc(&sh.tmem_base, kBuffers * kTile);
  if (tid == 32) {
    for (int i = 0; i < kKeyRing; ++i) {
      tc::mbar_init(&sh.k_full[i], 1);
      tc::mbar_init(&sh.k_empty[i], 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      tc::mbar_init(&sh.s_full[i], 1);
      tc::mbar_init(&sh.s_empty[i], kSumWarps / 2);
    }
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(&sh.sums_full[i >> 1][i & 1], 1);
      tc::mbar_init(&sh.sums_empty[i >> 1][i & 1], 1);
    }
    tc::mbar_init(&sh.done, 1);
    sh.fail = 0;
  }
  if (warp == kCopyWarp && lane == 0) tc::tma_prefetch_desc(&p.k_map);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = uni(sh.tmem_base);
  pdl_wait();
  const uint64_t kd = tc::sw128_desc(smem), qd = tc::sw128_desc(queries);
  const uint32_t hi = (uint32_t)(kd >> 32), k_lo = (uint32_t)kd, q_lo = (uint32_t)qd;
  const int quarter = warp & 3, half = (warp >> 2) & 1, set = warp >> 3;
  const int end = (int)(p.all * (blockIdx.x + 1) / gridDim.x);
  int tiles = 0, steps = 0;                       // done by this warp's role: places in the rings
  bool ok = true;
#pragma unroll 1
  for (int t0 = (int)(p.all * blockIdx.x / gridDim.x); t0 < end;) {
    const int unit = uni(p.by_tiles.div(t0)), b = uni(w.by_heads.div(unit)), h = unit - b * w.heads;
    const int first = t0 - unit * p.tiles, last = min(p.tiles, end - unit * p.tiles);
    t0 = unit * p.tiles + last;
#pragma unroll 1
    for (int c0 = 0; c0 < w.queries;) {
      // keys on their way meanwhile
      const int ahead = min(first + kKeyRing, last);
      if (warp == kCopyWarp && lane == 0 && ok) ok = copy_tiles(p, sh, smem, b, h, first, ahead, tiles);
      __syncwarp();
      const int total = uni(lay_queries(w, sh, queries, b, h, c0));
      c0 = uni(sh.next);
      const int blocks = (total + kTile - 1) / kTile;
      if (total == 0) {                           // no use for them
        if (warp == kIssueWarp)
          for (int t = first; ok && t < ahead; ++t, ++tiles) {
            if (!(ok = warp_wait(&sh.k_full[tiles % kKeyRing], (tiles / kKeyRing) & 1, &sh.fail))) break;
            if (lane == 0) tc::mbar_arrive(&sh.k_empty[tiles % kKeyRing]);
          }
      } else if (warp == kCopyWarp) {
        if (lane == 0 && ok) ok = copy_tiles(p, sh, smem, b, h, ahead, last, tiles);
        __syncwarp();
      } else if (warp == kIssueWarp) {
#pragma unroll 1
        for (int t = first; ok && t < last; ++t, ++tiles) {
          const int i = uni(tiles % kKeyRing);
          if (!(ok = warp_wait(&sh.k_full[i], (tiles / kKeyRing) & 1, &sh.fail))) break;
#pragma unroll 1
          for (int j = 0; j < blocks; ++j, ++steps) {
            const int buf = uni(steps % kBuffers);
            if (!(ok = warp_wait(&sh.s_empty[buf], ((steps / kBuffers) & 1) ^ 1, &sh.fail))) break;
            tc::fence_after_sync();
            tm::warp_mma_rows(tmem + buf * kTile, tm::desc_of(k_lo + ((i * kTileBytes) >> 4), hi),
                              tm::desc_of(q_lo + ((j * kTileBytes) >> 4), hi),
                              tc::idesc_bf16_f32(kTile, (min(kTile, total - j * kTile) + 15) & ~15));
            tm::warp_mma_commit(&sh.s_full[buf]);
          }
          if (!ok) break;
          tm::warp_mma_commit(&sh.k_empty[i]);
        }
      } else {
        const int key = quarter * 32 + lane;
        const uint64_t sc2 = pack_f32x2(w.scale2, w.scale2);
#pragma unroll 1
        for (int t = first; t < last; ++t, ++tiles) {
          if ((tiles & 1) != set) {
            steps += blocks;
            continue;
          }
          const int row = t * kTile + key;
          float* to = w.score + (long long)unit * w.cap + row;
          float was = 0.f;
          if (half == 0 && row < w.rows) was = *to;
          uint64_t acc[2] = {0ull, 0ull};
#pragma unroll 1
          for (int j = 0; j < blocks; ++j, ++steps) {
            const int buf = steps % kBuffers, columns = total - j * kTile - half * 64;
            // (a wait that gives up leaves `fail`)
            wait_for(&sh.s_full[buf], (steps / kBuffers) & 1, &sh.fail);
            __syncwarp();
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
              float x[32];
              if (columns > c) {
                tm::load32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * kTile + half * 64 + c, x);
                tm::wait32(x);
              }
              if (c || columns <= 32) {           // the last that is read
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sh.s_empty[buf]);
              }
              const int c0 = j * kTile + half * 64 + c;
              const float4 *neg = reinterpret_cast<const float4*>(&sh.neg[c0]), *rest = reinterpret_cast<const float4*>(&sh.rest[c0]);
              if (columns >= c + 32) {
#pragma unroll
                for (int q = 0; q < 32; q += 4) {
                  const float4 n = neg[q / 4], f = rest[q / 4];
                  acc[0] = fma_f32x2(ex2_f32x2(fma_f32x2(pack_f32x2(x[q], x[q + 1]), sc2, pack_f32x2(n.x, n.y))), pack_f32x2(f.x, f.y), acc[0]);
                  acc[1] = fma_f32x2(ex2_f32x2(fma_f32x2(pack_f32x2(x[q + 2], x[q + 3]), sc2, pack_f32x2(n.z, n.w))), pack_f32x2(f.z, f.w), acc[1]);
                }
              } else if (columns > c) {           // (what lies behind them may be anything)
#pragma unroll
                for (int q = 0; q < 32; q += 2) {
                  const float e = ex2(fmaf(x[q], w.scale2, sh.neg[c0 + q])) * sh.rest[c0 + q];
                  const float f = ex2(fmaf(x[q + 1], w.scale2, sh.neg[c0 + q + 1])) * sh.rest[c0 + q + 1];
                  acc[0] = add_f32x2(acc[0], pack_f32x2(c + q < columns ? e : 0.f, c + q + 1 < columns ? f : 0.f));
                }
              }
              if (columns <= 32) break;
            }
          }
          float lo, up;
          split_f32x2(add_f32x2(acc[0], acc[1]), lo, up);
          float sum = lo + up;
          // a key's two sums meet in the warp of the first half
          const int parity = (tiles >> 1) & 1;
          if (half) {
            wait_for(&sh.sums_empty[quarter][set], parity ^ 1, &sh.fail);
            sh.sums[set][key] = sum;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.sums_full[quarter][set]);
          } else {
            wait_for(&sh.sums_full[quarter][set], parity, &sh.fail);
            sum += sh.sums[set][key];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.sums_empty[quarter][set]);
            if (row < w.rows && !*(volatile int*)&sh.fail) *to = was + sum;
          }
        }
      }
      __syncthreads();                            // the queries' rows are read
    }
  }
  // every product and copy issued must end before tensor and shared memory are released
  if (warp == kIssueWarp) {
    tm::warp_mma_commit(&sh.done);
    drain_phase(&sh.done, 0, w.err);
  } else if (warp == kCopyWarp && lane == 0) {
#pragma unroll 1
    for (int i = 0; i < kKeyRing && i < tiles; ++i) drain_phase(&sh.k_full[i], ((tiles - 1 - i) / kKeyRing) & 1, w.err);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, kBuffers * kTile);
  if (tid == 0 && sh.fail) raise_device_error(w.err, kDevWaitTimeout);
  if (w.n_new && w.err && blockIdx.x == 0)
    for (int f = tid; f < w.seqs; f += kWideThreads)
      if (w.n_new[f] < 0 || w.n_new[f] > w.m) raise_device_error(w.err, kDevBadIndex);
}

// The rows of a block behind the kept ones, with their positions and given scores: a warp per row.
constexpr int kAppendWarps = 8;
__global__ void __launch_bounds__(kAppendWarps * 32) append_given_kernel(const __grid_constant__ GroupParams P) {
  pdl_wait();
  const Shape& s = P.s;
  const LayerPtrs& L = P.L[0];
  const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31, bh = blockIdx.y;
  if (t >= s.m) return;
  const size_t from = (size_t)bh * s.m + t, to = (size_t)bh * s.cap + s.k + t;
  constexpr int kPieces = kHeadDim * 2 / 16;      // of K, and of V
  const bool value = lane >= kPieces;
  const uint4* src = static_cast<const uint4*>(value ? L.v_in : L.k_in) + from * kPieces;
  uint4* dst = static_cast<uint4*>(value ? L.vst : L.kst) + to * kPieces;
  dst[lane & (kPieces - 1)] = src[lane & (kPieces - 1)];
  if (lane == 0) {
    L.score_st[to] = L.new_score[(size_t)bh * s.new_stride + t];
    L.pos_st[to] = L.pos_in ? L.pos_in[(size_t)(bh / s.heads) * s.m + t] : (int32_t)(s.offset + t);
  }
}

// The wide kernel's dynamic shared memory, allowed once for each device.
cudaError_t allow_smem(int dev) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(weigh_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

bool multiple(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

cudaError_t launch_append_given(const GroupParams& P, cudaStream_t st) {
  return launch_pdl(append_given_kernel, dim3((P.s.m + kAppendWarps - 1) / kAppendWarps, P.s.batch * P.s.heads),
                    dim3(kAppendWarps * 32), 0, st, nullptr, P);
}

}  // namespace evict

using namespace evict;

extern "C" int evict_weigh(evict_handle* h, const evict_rows* q, int batch, int m, const float* lse, const int32_t* n_new,
                           float scale, void* stream) {
  if (!h || !q) return fail(EVICT_EINVAL, "handle and q must not be NULL");
  if (h->cfg.method != EVICT_ATTENTION) return fail(EVICT_EINVAL, "only scores that are accumulated attention weights can be added to");
  if (batch < 0 || m < 0) return fail(EVICT_EINVAL, "batch and m must be >= 0 (got %d, %d)", batch, m);
  if (batch % h->cfg.batch) return fail(EVICT_EINVAL, "batch (%d) must be a multiple of the cache's (%d)", batch, h->cfg.batch);
  if (q->heads < 1 || q->heads % h->cfg.n_kv_heads)
    return fail(EVICT_EINVAL, "q's heads (%d) must be a multiple of the cache's (%d)", q->heads, h->cfg.n_kv_heads);
  if (!good_scale(scale)) return fail(EVICT_EINVAL, "scale must be finite and below 2^127");
  if (!multiple(lse, 4) || !multiple(n_new, 4)) return fail(EVICT_EINVAL, "lse and n_new must be 4-byte aligned");
  if ((long long)batch * m >= (1ll << 30) || (long long)batch * m * q->heads >= (1ll << 30))
    return fail(EVICT_ELIMIT, "batch * heads * m is 2^30 or more");
  if (batch == 0 || m == 0 || h->n_kept == 0) return EVICT_OK;
  if (!q->data || !lse) return fail(EVICT_EINVAL, "q and lse must not be NULL");
  if (!multiple(q->data, 16) || q->stride_b % 8 || q->stride_h % 8 || q->stride_m % 8)
    return fail(EVICT_EINVAL, "q: addresses and strides must be multiples of 16 bytes");
  WeighParams p = {};
  p.k = h->kst;
  p.score = h->score_st;
  p.cap = h->cap;
  p.rows = h->n_kept;
  p.heads = h->cfg.n_kv_heads;
  p.q = q->data;
  p.qb = q->stride_b, p.qh = q->stride_h, p.qm = q->stride_m;
  p.lse = lse;
  p.n_new = n_new;
  p.fan = batch / h->cfg.batch;
  p.seqs = batch;
  p.m = m;
  p.hq = q->heads;
  p.group = q->heads / p.heads;
  p.queries = p.fan * m * p.group;
  p.by_heads = Divisor(p.heads);
  p.by_per = Divisor(m * p.group);
  p.by_group = Divisor(p.group);
  p.scale2 = scale_base2(scale);
  p.err = h->err;
  int dev, sms;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "looking up the device");
  if (dev != h->dev) return fail(EVICT_EINVAL, "the cache is on device %d, the current device is %d", h->dev, dev);
  const int units = h->cfg.batch * p.heads;
  if (const unsigned long long id = capture_of(static_cast<cudaStream_t>(stream))) h->captured = id;
  // Key tiles for every SM and enough products for the wide kernel's start to pay (8 heads; us, narrow and wide):
  // 1024 tiles by 16 queries 9.0 and 10.0, by 32 11.5 and 10.1; 512 by 32 7.4 and 8.3, by 64 9.9 and 9.1; 2048 by 16
  // 20.3 and 19.8; but 16 tiles by 3584 queries 31 and 64, which the narrow kernel deals out.
  const int key_tiles = (p.rows + kTile - 1) / kTile;
  const long long tiles = (long long)units * key_tiles;
  if (tiles >= sms && p.queries >= 16 && tiles * p.queries >= 32768) {
    WideParams wide = {};
    wide.w = p;
    wide.tiles = key_tiles;
    wide.all = tiles;
    wide.by_tiles = Divisor(wide.tiles);
    const evict_rows keys = {h->kst, (int64_t)p.heads * p.cap * kHeadDim, (int64_t)p.cap * kHeadDim, kHeadDim, p.heads};
    if (!encode_tiled()) return fail(EVICT_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const int rc = encode_heads(&wide.k_map, keys, h->cfg.batch, p.rows, 1, kTile, false, "the kept rows");
    if (rc) return rc;
    if ((e = allow_smem(dev)) != cudaSuccess) return cuda_fail(e, "the weigh kernel's shared memory");
    e = launch_pdl(weigh_wide_kernel, dim3(sms), dim3(kWideThreads), kWideSmem,
                   static_cast<cudaStream_t>(stream), nullptr, wide);
    if (e != cudaSuccess) return cuda_fail(e, "weigh kernel launch");
    g_launches.fetch_add(1);
    return EVICT_OK;
  }
  // warps for the same keys: as many as there is room for, while each has a tile of queries
  const long long key_warps = (long long)units * ((p.rows + kKeys - 1) / kKeys);
  p.split = 1;
  while (p.split < kWarps && key_warps * p.split < 2ll * kWarps * sms && p.split * kQueries < p.queries) p.split *= 2;
  const int keys_cta = kKeys * (kWarps / p.split);
  e = launch_pdl(weigh_kernel, dim3((p.rows + keys_cta - 1) / keys_cta, units), dim3(kWarps * 32), 0,
                 static_cast<cudaStream_t>(stream), nullptr, p);
  if (e != cudaSuccess) return cuda_fail(e, "weigh kernel launch");
  g_launches.fetch_add(1);
  return EVICT_OK;
}
