// The weights that a prompt's attention put on each key: w_j = sum over the group's query heads and the
// queries t that see key j (t >= j; with `last` only a sequence's last ones) of exp(scale q_t.k_j - lse_t).
//
// A unit is a (sequence, KV head, block of 256 keys), a step 128 of its queries: 128 tokens of one head, or
// fewer tokens of several heads where few tokens of a sequence count. The logits are taken transposed,
// S^T = K Q^T, keys along the rows of tensor memory: a thread then holds one key and sums along its row, and
// no sum crosses threads but that of the row's two halves at a unit's end. K is held (two buffers of two
// 128-row tiles, the next unit's is fetched meanwhile), Q streams through a ring of three 32 KB tiles, and so
// do its log-sum-exps through shared memory, negated, in base 2 and with a bit for each that is -infinity: those
// queries are masked, whatever their logits are. Two accumulators for each of the two key tiles (512 columns):
// products run while the sixteen summing warps exponentiate the step before. Warps 16 and 17 issue the products of one key
// tile each (of both by one warp they take some 300 clocks of 1,100 from the summing warps beside it) and take
// turns, so that the one's waits run beside the other's products (8192 tokens, 28 / 4 heads: 183 us, without 190, on one
// GPU); warp 18 goes through the schedule and fetches (TMA), warp 19 loads the log-sum-exps.
//
// What bounds it: a step is 1,024 clocks of the tensor cores and as many of exponentials (at 32 a clock and SM) and
// takes some 1,750: tensor memory holds no more than the four accumulators, whose products come one after the other,
// 512 clocks each. 8192 tokens with 28 / 4 heads 183 to 197 us (1.22 to 1.31 PFLOP/s of 1.90); 24 sequences of up to
// 1021 tokens with 32 / 8 heads 68 us, of which 23 would be the products of what queries see: tiles at the diagonal, and their masks;
// windows of 64 tokens of 8 x 8192 41 us, 3.3 TB/s.
// Tried and taken back: K in tensor memory (214 us), 64 columns at a time (190 -> 196), chunks of a masked step that no
// query or every one sees left out or unmasked (packed no gain, 8192 tokens 200).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "api_internal.h"
#include "common.cuh"
#include "launch.h"
#include "prompt.cuh"
#include "prompt.h"
#include "tmem.cuh"

namespace evict {
namespace {

constexpr int kTile = 128, kTileBytes = kTile * kHeadDim * 2;
constexpr int kKeys = 2 * kTile;                  // keys of a unit
constexpr int kRing = 3, kUnits = 2;
constexpr int kSumWarps = 16;
constexpr int kReaders = kSumWarps + 3;           // warps that read a unit: summing, issuing, loading log-sum-exps
constexpr int kMmaWarp = 16, kTmaWarp = 18, kThreads = 640;
constexpr int kEntry = 3, kMinSteps = 4;
// Units of few steps go uncut (too short to share), and all where every SM has this many: then nothing is joined, and
// CTAs take units as they come to them, in an order in which the long ones are early. (us, uncut and cut: windows of 64
// tokens, 8192, 28 / 4 heads, 10 and 13; of 256, 4000, 32 / 8 heads, 14 and 18; units of 32 steps, 446 tokens, 16 / 2
// heads, 35 and 13. Of many steps, 64 sequences of up to 1021 tokens, 32 / 8 heads, 14 units an SM, 131 and 145; 24,
// 32 / 16 heads, 7 an SM, 69 and 80; 32 / 8 heads, 3.5 an SM, 68 and 75, in the sequences' order 77; 8 of up to 4000,
// 2.5 an SM, 99 and 93.)
constexpr int kWholeSteps = 8, kWholeRounds = 3;

// The first query that counts for the keys from key0 on.
__device__ __forceinline__ int first_query(int last, int key0, int len) { return max(key0, last ? len - last : 0); }

struct Steps {
  int heads_of, last, tokens;                     // heads (rounded up to whole steps' worth) over heads of a step; tokens of one
  __device__ __forceinline__ explicit Steps(const PromptParams& p)
      : heads_of(p.head_steps), last(p.last), tokens(p.half) {}
  __device__ __forceinline__ int operator()(int key0, int len) const {
    return heads_of * ((len - first_query(last, key0, len) + tokens - 1) / tokens);
  }
};

// A CTA's part of a unit, as every warp sees it.
struct alignas(16) Unit {
  int plane, row0, h;                             // the sequence's plane and first row; KV head
  int key0, keys;                                 // first key; keys
  int first, len;                                 // first query that counts; the sequence's length
  int from, to, tiles;                            // steps of the part; tiles of tokens
  int kind;                                       // 0: there is none
};
constexpr int kPart = 1, kWhole = 2;              // kinds

struct WeightsShared {
  uint64_t unit_full[kUnits], unit_empty[kUnits], k_full[2], k_empty[2], q_full[kRing], q_empty[kRing];
  uint64_t s_full[2][2], s_empty[2][2], lse_full[kRing], lse_empty[kRing], done[2];   // buffer, key tile
  uint64_t turn[2];                               // of the issuing warps
  uint32_t tmem_base;
  int fail;
  Unit units[kUnits];
  union {
    alignas(16) float neg_lse2[kRing][kTile];
    PromptScan scan;                              // before the first of them
  };
  float sums[kKeys];
  alignas(16) uint32_t none[kRing][kTile / 32];   // columns of a step whose log-sum-exp is -infinity
};
// All of it is dynamic: seven tiles and this fill the 227 KB.
constexpr int kSmem = (4 + kRing) * kTileBytes + (int)sizeof(WeightsShared);
static_assert(kSmem <= 227 * 1024);

// What a step works on: column c is query tok0 + c % tokens of head g0 + c / tokens of the group; it counts
// where the token is below tok0 + n and the head one of the group's.
struct Step {
  int hs, tile;                                   // heads_of's, tile
  int g0, tok0, n;
  __device__ __forceinline__ Step(const PromptParams& p, const Unit& u) {
    hs = u.from / u.tiles;
    tile = u.from - hs * u.tiles;
    place(p, u);
  }
  __device__ __forceinline__ void place(const PromptParams& p, const Unit& u) {
    g0 = hs * p.step_heads;
    tok0 = u.first + tile * p.half;
    n = min(p.half, u.len - tok0);
  }
  __device__ __forceinline__ void next(const PromptParams& p, const Unit& u) {
    tok0 += p.half;
    if (++tile == u.tiles) {
      tile = 0;
      ++hs;
      g0 += p.step_heads;
      tok0 = u.first;
    }
    n = min(p.half, u.len - tok0);
  }
  // some query of the step sees a key of tile kt
  __device__ __forceinline__ bool sees(const Unit& u, int kt) const {
    return kt * kTile < u.keys && tok0 + n > u.key0 + kt * kTile;
  }
  // columns up to the last one that counts
  __device__ __forceinline__ int columns(const PromptParams& p) const {
    return (min(p.step_heads, p.group - g0) - 1) * p.half + n;
  }
  __device__ __forceinline__ bool full(const PromptParams& p) const { return n == p.half && g0 + p.step_heads <= p.group; }
};

template <int kCount>
struct Ring {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == kCount) i = 0, parity ^= 1;
  }
};

// The i-th unit of the CTA, by a whole warp; kind 0 behind the last one, and where a wait gave up.
__device__ __forceinline__ Unit read_unit(WeightsShared& sh, int i) {
  Unit u = {};
  if (warp_wait(&sh.unit_full[i % kUnits], (i / kUnits) & 1, &sh.fail)) u = sh.units[i % kUnits];
  u.plane = uni(u.plane), u.row0 = uni(u.row0), u.h = uni(u.h), u.key0 = uni(u.key0), u.keys = uni(u.keys);
  u.first = uni(u.first), u.len = uni(u.len), u.from = uni(u.from), u.to = uni(u.to), u.tiles = uni(u.tiles);
  u.kind = uni(u.kind);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&sh.unit_empty[i % kUnits]);
  return u;
}

// The schedule and the copies, by one thread.
__device__ void producer(const PromptParams& p, WeightsShared& sh, PromptCursor c, uint32_t kbuf, uint32_t ring) {
  const Steps steps(p);
  Ring<2> k;
  Ring<kRing> q;
  int used_k = 0, used_q = 0;
  bool ok = true, any = true;                     // any: there is a unit at hand
  auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = wait_for(bar, parity, &sh.fail); };
  for (int unit = 0;; ++unit) {
    if (!wait(&sh.unit_empty[unit % kUnits], ((unit / kUnits) & 1) ^ 1)) break;
    Unit u = {};
    if (any) {
      u.plane = c.k.at.plane;
      u.row0 = c.k.at.row0;
      u.h = c.h;
      u.key0 = c.k.tile * kKeys;
      u.keys = min(kKeys, c.k.at.len - u.key0);
      u.len = c.k.at.len;
      u.first = first_query(p.last, u.key0, u.len);
      u.from = c.from;
      u.to = c.to;
      u.tiles = (u.len - u.first + p.half - 1) / p.half;
      u.kind = c.to - c.from == c.k.steps ? kWhole : kPart;
    }
    sh.units[unit % kUnits] = u;
    tc::mbar_arrive(&sh.unit_full[unit % kUnits]);
    if (!any) break;
    const int tiles = u.keys > kTile ? 2 : 1;
    if (!wait(&sh.k_empty[k.i], k.parity ^ 1)) break;
    tc::mbar_arrive_expect_tx(&sh.k_full[k.i], tiles * kTileBytes);
    for (int j = 0; j < 2 * tiles; ++j)
      tma_load_4d(kbuf + k.i * 2 * kTileBytes + j * (kTileBytes / 2), &p.k_map, (j & 1) * 64, u.row0 + u.key0 + (j >> 1) * kTile,
                  u.h, u.plane, &sh.k_full[k.i]);
    k.next();
    ++used_k;
    Step s(p, u);
#pragma unroll 1
    for (int i = u.from; i < u.to; ++i, s.next(p, u)) {
      if (!wait(&sh.q_empty[q.i], q.parity ^ 1)) break;
      tc::mbar_arrive_expect_tx(&sh.q_full[q.i], kTileBytes);
      for (int hf = 0; hf < 2; ++hf)
        tma_load_4d(ring + q.i * kTileBytes + hf * (kTileBytes / 2), &p.q_map, hf * 64, u.row0 + s.tok0, u.h * p.group + s.g0,
                    u.plane, &sh.q_full[q.i]);
      q.next();
      ++used_q;
    }
    if (!ok) break;
    any = next_unit(p.work, c, steps);
  }
  // every copy issued must land before the CTA may release its shared memory
#pragma unroll 1
  for (int i = 0; i < 2 && i < used_k; ++i) drain_phase(&sh.k_full[i], ((used_k - 1 - i) / 2) & 1, p.work.err);
#pragma unroll 1
  for (int i = 0; i < kRing && i < used_q; ++i) drain_phase(&sh.q_full[i], ((used_q - 1 - i) / kRing) & 1, p.work.err);
}

// The steps' log-sum-exps to shared memory, four of a step by each lane. All four are on their way before any is looked
// at: one after the other, as they came out with more arithmetic in the loop, everything waits for them (8192 tokens 299
// us instead of 183). Those of the next step fetched ahead gained nothing.
__device__ void lse_loader(const PromptParams& p, WeightsShared& sh) {
  const int lane = threadIdx.x & 31;
  Ring<kRing> r;
#pragma unroll 1
  for (int unit = 0;; ++unit) {
    const Unit u = read_unit(sh, unit);
    if (!u.kind) return;
    Step s(p, u);
#pragma unroll 1
    for (int i = u.from; i < u.to; ++i, s.next(p, u)) {
      float l[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = 32 * j + lane, g = s.g0 + (col >> p.half_shift), t = col & (p.half - 1);
        l[j] = -INFINITY;
        if (t < s.n && g < p.group) l[j] = p.lse[((long long)u.plane * p.hq + u.h * p.group + g) * p.work.m + u.row0 + s.tok0 + t];
      }
      if (!warp_wait(&sh.lse_empty[r.i], r.parity ^ 1, &sh.fail)) return;
      // no weights of a query that saw nothing; log2 e in two parts, as all weights would lean to where its rounding does
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool none = l[j] == -INFINITY;
        sh.neg_lse2[r.i][32 * j + lane] = none ? l[j] : fmaf(-l[j], kLog2e, -l[j] * kLog2eRest);
        const uint32_t of = __ballot_sync(0xffffffffu, none);
        if (lane == 0) sh.none[r.i][j] = of;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.lse_full[r.i]);
      r.next();
    }
  }
}

// The products of key tile kt, by a converged warp. (It waits for a step's log-sum-exps, too: who sees the logits
// sees those.)
__device__ void mma_issuer(const PromptParams& p, WeightsShared& sh, int kt, uint32_t tmem, uint32_t kbuf, uint32_t ring) {
  const uint64_t kd = tc::sw128_desc(kbuf), qd = tc::sw128_desc(ring);
  const uint32_t hi = (uint32_t)(kd >> 32), k_lo = (uint32_t)kd, q_lo = (uint32_t)qd;
  Ring<2> k, s_buf;
  uint32_t turns = 0;
  Ring<kRing> q;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = ok && warp_wait(bar, parity, &sh.fail); };
#pragma unroll 1
  for (int unit = 0; ok; ++unit) {
    const Unit u = read_unit(sh, unit);
    if (!u.kind || !wait(&sh.k_full[k.i], k.parity)) break;
    Step s(p, u);
#pragma unroll 1
    for (int i = u.from; i < u.to; ++i, s.next(p, u)) {
      if (!wait(&sh.q_full[q.i], q.parity) || !wait(&sh.lse_full[q.i], q.parity) || !wait(&sh.s_empty[s_buf.i][kt], s_buf.parity ^ 1)) break;
      // the two take turns, each with its waits behind it: the tensor cores have the one's products while the other waits
      if ((kt || turns) && !wait(&sh.turn[kt], (turns - 1 + kt) & 1)) break;
      ++turns;
      tc::fence_after_sync();
      if (s.sees(u, kt))
        tm::warp_mma_rows(tmem + (2 * s_buf.i + kt) * kTile, tm::desc_of(k_lo + (((2 * k.i + kt) * kTileBytes) >> 4), hi),
                          tm::desc_of(q_lo + ((q.i * kTileBytes) >> 4), hi), tc::idesc_bf16_f32(kTile, (s.columns(p) + 15) & ~15));
      if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&sh.turn[kt ^ 1]);
      tm::warp_mma_commit(&sh.s_full[s_buf.i][kt]);
      tm::warp_mma_commit(&sh.q_empty[q.i]);
      q.next();
      s_buf.next();
    }
    if (!ok) break;
    tm::warp_mma_commit(&sh.k_empty[k.i]);
    k.next();
  }
  // every MMA must finish before tensor and shared memory are released
  tm::warp_mma_commit(&sh.done[kt]);
  drain_phase(&sh.done[kt], 0, p.work.err);
}

// A barrier of `threads` threads; whether x holds for all of them.
__device__ __forceinline__ bool named_and(uint32_t id, uint32_t threads, bool x) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(all)
      : "r"(x ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return all != 0;
}

// Bits lo .. hi - 1 of 32, cut to them.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t below = hi >= 32 ? ~0u : hi > 0 ? (1u << hi) - 1u : 0u;
  return lo >= 32 ? 0u : lo > 0 ? below & ~((1u << lo) - 1u) : below;
}
// Of columns c0 .. c0 + 31 of a step with `columns`: those whose query counts and sees a key that `before` tokens of
// the step do not see.
__device__ __forceinline__ uint32_t seen_columns(const PromptParams& p, const Step& s, int c0, int columns, int before) {
  const int t0 = c0 & (p.half - 1);
  uint32_t m = bit_range(before - t0, s.n - t0);
  if (p.half == 16) m = (m & 0xffffu) * 0x10001u;
  return m & bit_range(0, columns - c0);
}

// A summing warp: 32 keys of tile kt, a thread each, and every other step (so that the four warps of an SM's
// quarter are at different places: one's waits and loads run beside the others' exponentials).
__device__ void sum_warp(const PromptParams& p, WeightsShared& sh, uint32_t tmem, int warp) {
  const int lane = threadIdx.x & 31;
  const int kt = (warp >> 2) & 1, buf = warp >> 3, key = kt * kTile + (warp & 3) * 32 + lane;
  const uint32_t s_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (2 * buf + kt) * kTile;
  const uint64_t sc2 = pack_f32x2(p.scale2, p.scale2);
  Ring<2> s_buf;
  Ring<kRing> r;
#pragma unroll 1
  for (int unit = 0;; ++unit) {
    // Warps w and w + 8 meet at a unit's end, so they go on, or leave, together: where a wait has given up somewhere, one
    // of them may have come before the unit was there, the other after. (And the sums of the unit before are read.)
    const Unit u = read_unit(sh, unit);
    if (!named_and(1 + (warp & 7), 64, u.kind != 0)) break;
    Step s(p, u);
    float sum = 0.f;
#pragma unroll 1
    for (int i = u.from; i < u.to; ++i, s.next(p, u)) {
      if (s_buf.i == buf) {
        // (no vote: a wait that gives up leaves `fail`, which is looked at once a unit)
        wait_for(&sh.s_full[buf][kt], s_buf.parity, &sh.fail);
        __syncwarp();
        tc::fence_after_sync();
        const int columns = s.sees(u, kt) ? s.columns(p) : 0;
        const int before = u.key0 + key - s.tok0;                  // tokens that do not see this key
        const uint32_t* none = sh.none[r.i];
        const uint4 nones = *reinterpret_cast<const uint4*>(none);
        const bool masked = !s.full(p) || u.key0 + kt * kTile + kTile - 1 > s.tok0 || (nones.x | nones.y | nones.z | nones.w);
        uint64_t acc[2] = {0ull, 0ull};
#pragma unroll 1
        for (int c0 = 0; c0 < columns; c0 += 32) {
          const float4* l2 = reinterpret_cast<const float4*>(&sh.neg_lse2[r.i][c0]);
          float x[32];
          tm::load32(s_at + c0, x);
          tm::wait32(x);
          if (c0 + 32 >= columns) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.s_empty[buf][kt]);
          }
          if (!masked) {
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 l = l2[j / 4];
              acc[0] = add_f32x2(acc[0], ex2_f32x2(fma_f32x2(pack_f32x2(x[j], x[j + 1]), sc2, pack_f32x2(l.x, l.y))));
              acc[1] = add_f32x2(acc[1], ex2_f32x2(fma_f32x2(pack_f32x2(x[j + 2], x[j + 3]), sc2, pack_f32x2(l.z, l.w))));
            }
          } else {
            // (log-sum-exps of columns that do not count are -infinity, but their logits may be anything)
            const uint32_t m = seen_columns(p, s, c0, columns, before) & ~none[c0 / 32];
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 l = l2[j / 4];
              float e[4];
              split_f32x2(ex2_f32x2(fma_f32x2(pack_f32x2(x[j], x[j + 1]), sc2, pack_f32x2(l.x, l.y))), e[0], e[1]);
              split_f32x2(ex2_f32x2(fma_f32x2(pack_f32x2(x[j + 2], x[j + 3]), sc2, pack_f32x2(l.z, l.w))), e[2], e[3]);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!(m & (1u << (j + k)))) e[k] = 0.f;
              acc[0] = add_f32x2(acc[0], pack_f32x2(e[0], e[1]));
              acc[1] = add_f32x2(acc[1], pack_f32x2(e[2], e[3]));
            }
          }
        }
        float a, b;
        split_f32x2(add_f32x2(acc[0], acc[1]), a, b);
        sum += a + b;
        __syncwarp();
        if (lane == 0) {
          if (columns == 0) tc::mbar_arrive(&sh.s_empty[buf][kt]);
          tc::mbar_arrive(&sh.lse_empty[r.i]);
        }
      }
      s_buf.next();
      r.next();
    }
    // a key's two sums meet: warp w + 8's go to warp w
    if (buf) sh.sums[key] = sum;
    if (!named_and(1 + (warp & 7), 64, !*(volatile int*)&sh.fail)) break;
    if (!buf) {
      sum += sh.sums[key];
      if (u.kind == kWhole) {
        if (key < u.keys) p.weights[((long long)u.plane * p.work.hkv + u.h) * p.work.m + u.row0 + u.key0 + key] = sum;
      } else {
        p.part[(size_t)(2 * blockIdx.x + (u.from == 0 ? 1 : 0)) * kKeys + key] = sum;
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) prompt_weights_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t smem = tc::smem_u32(smem_raw);
  WeightsShared& sh = *reinterpret_cast<WeightsShared*>(smem_raw + (4 + kRing) * kTileBytes);
  if (smem & 1023) {                              // not as declared: no tile could be right
    if (threadIdx.x == 0) raise_device_error(p.work.err, kDevBadIndex);
    return;
  }
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (warp == 0) tc::tmem_alloc(&sh.tmem_base, 4 * kTile);
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.k_full[i], 1);
      tc::mbar_init(&sh.k_empty[i], 2);           // both issuers
      tc::mbar_init(&sh.done[i], 1);
      tc::mbar_init(&sh.turn[i], 1);
      for (int kt = 0; kt < 2; ++kt) {
        tc::mbar_init(&sh.s_full[i][kt], 1);
        tc::mbar_init(&sh.s_empty[i][kt], kSumWarps / 4);
      }
    }
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(&sh.q_full[i], 1);
      tc::mbar_init(&sh.q_empty[i], 2);
      tc::mbar_init(&sh.lse_full[i], 1);
      tc::mbar_init(&sh.lse_empty[i], kSumWarps / 2);
    }
    for (int i = 0; i < kUnits; ++i) {
      tc::mbar_init(&sh.unit_full[i], 1);
      tc::mbar_init(&sh.unit_empty[i], kReaders);
    }
    sh.fail = 0;
  }
  if (warp == kTmaWarp && lane == 0) {
    tc::tma_prefetch_desc(&p.q_map);
    tc::tma_prefetch_desc(&p.k_map);
  }
  pdl_wait();
  PromptCursor c;
  const bool any = first_unit<kThreads>(p.work, sh.scan, reinterpret_cast<int*>(smem_raw), c, Steps(p));
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0), ring = smem + 4 * kTileBytes;
  if (any) {
    if (warp < kSumWarps) {
      sum_warp(p, sh, tmem, warp);
    } else if (warp < kTmaWarp) {
      mma_issuer(p, sh, warp - kMmaWarp, tmem, smem, ring);
    } else if (warp == kTmaWarp) {
      if (lane == 0) producer(p, sh, c, smem, ring);
      __syncwarp();
    } else {
      lse_loader(p, sh);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, 4 * kTile);
  if (tid == 0 && sh.fail) raise_device_error(p.work.err, kDevWaitTimeout);
}

// Keys of units that two or more CTAs share: their parts' sums, in the shares' order.
__global__ void __launch_bounds__(kKeys) prompt_weights_join_kernel(const __grid_constant__ PromptParams p) {
  pdl_wait();
  SplitUnit u;
  if (!split_unit(p.work, blockIdx.x + 1, u)) return;
  const int key = threadIdx.x, at = u.tile * kKeys + key;
  if (at >= u.at.len) return;
  float sum = 0.f;
#pragma unroll 4
  for (int i = u.c0; i <= u.c1; ++i) sum += p.part[(size_t)(2 * i + (i == u.c0 ? 1 : 0)) * kKeys + key];
  p.weights[((long long)u.at.plane * p.work.hkv + u.h) * p.work.m + u.at.row0 + at] = sum;
}

// The kernel's dynamic shared memory, allowed once for each device.
cudaError_t allow_smem(int dev) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(prompt_weights_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

// Tokens of a step: 128 of one head, but 64, 32 or 16 of several where no more of a sequence count. (A window of 64
// tokens of 8 x 8192 with 32 / 8 heads: steps of one head leave half of them empty.)
int step_tokens(const evict_prompt* a) {
  const int group = a->q.heads / a->k.heads;
  int tokens = kTile;
  while (tokens > 16 && a->last > 0 && a->last <= tokens / 2 && 2 * tokens > kTile / group) tokens /= 2;
  return tokens;
}

int make_plan(const evict_prompt* a, PromptPlan* plan) {
  const int group = a->q.heads / a->k.heads, tokens = step_tokens(a), heads = kTile / tokens, head_steps = (group + heads - 1) / heads;
  const long long most = (long long)head_steps * (((long long)(a->last > 0 ? std::min(a->last, a->m) : a->m) + tokens - 1) / tokens);
  const int rc = plan_prompt(a, kKeys, most, kEntry, kMinSteps, most <= kWholeSteps ? 0 : kWholeRounds, 0, 2 * kKeys * sizeof(float), false, plan);
  PromptParams& p = plan->p;
  p.last = a->last;
  p.half = tokens;
  p.half_shift = __builtin_ctz((unsigned)tokens);
  p.step_heads = heads;
  p.head_steps = head_steps;
  return rc;
}

}  // namespace
}  // namespace evict

using namespace evict;

extern "C" int evict_prompt_weights_workspace(const evict_prompt* a, size_t* bytes) {
  if (!bytes) return fail(EVICT_EINVAL, "bytes is NULL");
  PromptPlan plan;
  int rc;
  if ((rc = check_prompt_sizes(a))) return rc;
  evict_prompt all = *a;                          // a window needs no more
  all.last = 0;
  if ((rc = make_plan(&all, &plan))) return rc;
  *bytes = plan.bytes;
  return EVICT_OK;
}

extern "C" int evict_prompt_weights(const evict_prompt* a) {
  int rc;
  if ((rc = check_prompt(a, false))) return rc;
  if (a->batch == 0 || a->m == 0 || (a->starts && a->n_seqs == 0)) return EVICT_OK;
  PromptPlan plan;
  if ((rc = make_plan(a, &plan)) || (rc = bind_prompt(a, &plan))) return rc;
  PromptParams& p = plan.p;
  if ((rc = encode_heads(&p.q_map, a->q, a->batch, a->m, p.step_heads, p.half, false, "q")) ||
      (rc = encode_heads(&p.k_map, a->k, a->batch, a->m, 1, kTile, false, "k")))
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  cudaError_t e = allow_smem(plan.dev);
  if (e != cudaSuccess) return cuda_fail(e, "prompt weights kernel attribute");
  const int ctas = p.work.whole ? std::min(plan.sms, p.work.blocks * p.work.hkv) : plan.sms;
  if ((rc = begin_prompt(p.work, st))) return rc;
  if ((e = launch_pdl(prompt_weights_kernel, dim3(ctas), dim3(kThreads), kSmem, st, nullptr, p)) != cudaSuccess)
    return cuda_fail(e, "prompt weights kernel launch");
  g_launches.fetch_add(1);
  if (!p.work.whole && ctas > 1) {
    if ((e = launch_pdl(prompt_weights_join_kernel, dim3(ctas - 1), dim3(kKeys), 0, st, nullptr, p)) != cudaSuccess)
      return cuda_fail(e, "prompt weights join kernel launch");
    g_launches.fetch_add(1);
  }
  return EVICT_OK;
}
