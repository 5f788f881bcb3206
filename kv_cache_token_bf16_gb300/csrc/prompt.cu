// Attention of whole prompts with themselves, causal, query heads in groups, sequences packed behind
// each other or in a batch.
//
//   o_t = sum_{j <= t} p_j v_j / sum_{j <= t} p_j,  p_j = exp(scale q_t.k_j - max)
// in one pass over K and V; logits are kept in base 2 (scale * log2 e), so p = 2^(x - ref).
//
// A unit is a (sequence, KV head, tile of tokens): the tokens' query rows of the whole group, token by
// token, fill two tiles of 128 rows, so that K and V are read once for all of the group's heads and few
// rows at the diagonal go unseen. Warps 0-3 and 4-7 are two softmax groups, a thread per query row, each
// with its own 128 x 128 logits and 128 x 128 output accumulator in tensor memory (512 columns in all);
// warps 8 and 9 issue the tensor cores' work of one group each, in halves of 64 rows of K and V:
//     S = Q K^T -> P = 2^(S scale - ref) as bf16 over S (softmax group) -> O += P V.
// While the group exponentiates one half, the logits of the other are made, of the next unit as well.
// Warp 10 fetches (TMA): K and V through a ring of five 32 KB tiles of 128 rows, the queries of the next
// unit as soon as the last product that reads a tile is through. Warp 11 clears rows of V that only some
// of the unit's queries see, or none (see scrub).
//
// What bounds it: a half step of both groups is 1,280 clocks of the tensor cores (logits in halves of 64 columns take
// 48 clocks a product instead of 32) and takes 1,450; beginning and leaving a unit takes 5,300, of which 3,000 are the
// stores of its 64 KB. 8192 tokens with 28 / 4 heads 333 to 352 us (1.37 to 1.44 PFLOP/s of 1.90); 4 x 2048 with 40 / 8
// 148 to 156 us (1.10 to 1.16); 24 sequences of up to 1021 tokens with 32 / 8 116 us (0.77), 45 tokens 8.2 us.
// Tried and taken back: logits of 128 columns at once (518 us for the 8192 tokens; a lone thread issued the products
// then, and was what bound it, so this says nothing of them with the warps that issue now), masked and unmasked
// exponentials apart (10-20 % more on short prompts: instruction cache), the second group a step behind the first (no
// gain), rows stored 128 bytes by four lanes (packed 124 instead of 129 at the time, but short prompts
// 9.0 instead of 8.7 and the batch as before), results stored by a warpgroup of its own while the groups go on (8192
// tokens 333 instead of 337, packed 120 instead of 116, 64 sequences of up to 512 100 instead of 91), a ring of four
// tiles (3-6 % more).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "common.cuh"
#include "launch.h"
#include "prompt.cuh"
#include "prompt.h"
#include "rotary.h"
#include "tmem.cuh"

namespace evict {
namespace {

constexpr int kTile = 128, kHalf = 64;
constexpr int kTileBytes = kTile * kHeadDim * 2;
constexpr int kRows = 2 * kTile;                  // query rows of a unit
constexpr int kRing = 5;
constexpr int kSmem = 1024 + (2 + kRing) * kTileBytes;
constexpr int kMmaWarp = 8, kTmaWarp = 10, kThreads = 384;   // warp 11 scrubs
constexpr int kUnits = 8;                         // units that warps are apart at most
constexpr int kReaders = 11;                      // warps that read a unit: softmax, issuers, scrubbing
constexpr int kBadWords = kRows / 32;             // rows of V behind the unit's first token, a bit each
constexpr int kPartly = 4;                        // barriers of tiles to scrub, in turn: the ring holds at most three
constexpr float kMoveAbove = 4096.f;              // sum of 32 weights that makes the reference move
constexpr int kEntry = 2, kMinSteps = 4;
// Units that go uncut are taken as CTAs come to them where every SM has more than two (a kernel of its own sets their
// count to 0): dealt out by their number, 24 sequences of up to 1021 tokens took 130 us instead of 117, 4 x 2048 171
// instead of 150, 3 sequences of up to 2000 71 instead of 56.
// Units go uncut in planes of this many rows (too short to share), and where there is one for every SM: then nothing is
// joined. (us, uncut and cut, of one sequence: 1021 tokens, 16 / 2 heads, 20 and 26; 1500, 26 and 30; 2000, 8 / 1 heads,
// 33 and 29; 4000, 8 / 1 heads, 0.8 units an SM, 57 and 46; 2900, 16 / 2 heads, 1.2 an SM, 44 and 51; 2000, 28 / 4 heads,
// 1.5 an SM, 34 and 48; 8192, 28 / 4 heads, 6 an SM, 343 and 352. 24 of up to 1021 tokens, 32 / 8 heads, 12 an SM, 117
// and 135; 4 x 2048, 40 / 8 heads, 9 an SM, 150 and 168.)
constexpr int kWholeRows = 1536, kWholeRounds = 1, kTakenRounds = 2;
// Weights' units of so many sequences are put in order: each block looks through all of them.
constexpr int kOrderedSeqs = 256;

struct Steps {
  int tile;
  __device__ __forceinline__ int operator()(int tok0, int len) const { return (min(tok0 + tile, len) + kTile - 1) / kTile; }
};

// A CTA's part of a unit, as every warp sees it. (The fetching warp alone goes through the schedule: one
// warp's code for it, and nothing of it between a product and the next.)
struct alignas(16) Unit {
  int plane, row0, h;                             // the sequence's plane and first row; KV head
  int tok0, reach;                                // first token; last one
  int from;                                       // first step of the part
  int n0, n1;                                     // steps of the two groups, from there on: n1 >= n0, or 0
  int kind;                                       // 0: there is none
  __device__ __forceinline__ int n(int w) const { return w ? n1 : n0; }
  __device__ __forceinline__ int steps() const { return max(n0, n1); }
  // the step's rows of V hold some that not every query of the unit sees
  __device__ __forceinline__ bool partly(int step) const { return step * kTile + kTile - 1 > tok0; }
};
constexpr int kPart = 1, kWhole = 2;              // kinds

struct AttentionShared {
  uint64_t unit_full[kUnits], unit_empty[kUnits];
  uint64_t q_full[2], q_empty[2], kv_full[kRing], kv_empty[kRing], partly_full[kPartly], scrubbed[kPartly];
  uint64_t s_full[2][2], p_full[2][2], o_full[2][2], done[2];   // group, half of the step
  uint32_t tmem_base;
  int fail;
  Unit units[kUnits];
  uint32_t bad[kUnits][kBadWords];                // rows of V that were cleared
  PromptScan scan;
};

struct Slot {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == kRing) i = 0, parity ^= 1;
  }
  __device__ __forceinline__ void step() {
    next();
    next();
  }
};

// The i-th unit of the CTA, by a whole warp; kind 0 behind the last one, and where a wait gave up.
__device__ __forceinline__ Unit read_unit(AttentionShared& sh, int i) {
  Unit u = {};
  if (warp_wait(&sh.unit_full[i % kUnits], (i / kUnits) & 1, &sh.fail)) u = sh.units[i % kUnits];
  u.plane = uni(u.plane), u.row0 = uni(u.row0), u.h = uni(u.h);
  u.tok0 = uni(u.tok0), u.reach = uni(u.reach), u.from = uni(u.from);
  u.n0 = uni(u.n0), u.n1 = uni(u.n1), u.kind = uni(u.kind);
  return u;
}
__device__ __forceinline__ void let_go(AttentionShared& sh, int i) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&sh.unit_empty[i % kUnits]);
}

// The schedule and the copies, by one thread.
__device__ void producer(const PromptParams& p, AttentionShared& sh, PromptCursor c, uint32_t qbuf, uint32_t ring) {
  const Steps steps{p.work.tile};
  Slot slot;
  int used = 0, turns0 = 0, turns1 = 0, partly = 0, unit = 0;
  bool ok = true, any = true;                     // any: there is a unit at hand
  auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = wait_for(bar, parity, &sh.fail); };
  for (;; ++unit) {
    if (!wait(&sh.unit_empty[unit % kUnits], ((unit / kUnits) & 1) ^ 1)) break;
    Unit u = {};
    if (any) {
      u.plane = c.k.at.plane;
      u.row0 = c.k.at.row0;
      u.h = c.h;
      u.tok0 = c.k.tile * p.work.tile;
      u.reach = min(u.tok0 + p.work.tile, c.k.at.len) - 1;
      u.from = c.from;
      const int first_reach = min(u.tok0 + p.half - 1, u.reach);  // of the first group's tokens
      u.n0 = max(min(c.to, first_reach / kTile + 1) - c.from, 0);
      u.n1 = first_reach < u.reach ? c.to - c.from : 0;
      u.kind = c.to - c.from == c.k.steps ? kWhole : kPart;
    }
    sh.units[unit % kUnits] = u;
    tc::mbar_arrive(&sh.unit_full[unit % kUnits]);
    if (!any) break;
#pragma unroll 1
    for (int j = 0; j < 2 * u.steps(); ++j) {     // K and V of a step; the queries behind the first K
      if (j == 1) {
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          if (u.n(w) == 0) continue;
          const int turn = w ? turns1 : turns0;
          if (!wait(&sh.q_empty[w], (turn & 1) ^ 1)) break;
          if (w) ++turns1;
          else ++turns0;
          tc::mbar_arrive_expect_tx(&sh.q_full[w], 2 * p.half * p.group * 128);
          for (int hf = 0; hf < 2; ++hf)
            tma_load_4d(qbuf + w * kTileBytes + hf * (kTileBytes / 2), &p.q_map, hf * 64, u.h * p.group,
                        u.row0 + u.tok0 + w * p.half, u.plane, &sh.q_full[w]);
        }
        if (!ok) break;
      }
      if (!wait(&sh.kv_empty[slot.i], slot.parity ^ 1)) break;
      const int step = u.from + j / 2;
      uint64_t* bar = &sh.kv_full[slot.i];
      if ((j & 1) && u.partly(step)) {
        // a tile to be scrubbed lands on a barrier of the scrubbing warp's, and its slot counts as full at once
        tc::mbar_arrive(bar);
        bar = &sh.partly_full[partly++ % kPartly];
      }
      tc::mbar_arrive_expect_tx(bar, kTileBytes);
      for (int hf = 0; hf < 2; ++hf)
        tma_load_4d(ring + slot.i * kTileBytes + hf * (kTileBytes / 2), j & 1 ? &p.v_map : &p.k_map, hf * 64,
                    u.row0 + step * kTile, u.h, u.plane, bar);
      slot.next();
      ++used;
    }
    if (!ok) break;
    any = next_unit(p.work, c, steps);
  }
  // every copy issued must land before the CTA may release its shared memory
#pragma unroll 1
  for (int i = 0; i < kRing && i < used; ++i) drain_phase(&sh.kv_full[i], ((used - 1 - i) / kRing) & 1, p.work.err);
#pragma unroll 1
  for (int i = 0; i < kPartly && i < partly; ++i) drain_phase(&sh.partly_full[i], ((partly - 1 - i) / kPartly) & 1, p.work.err);
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    const int turns = w ? turns1 : turns0;
    if (turns) drain_phase(&sh.q_full[w], (turns - 1) & 1, p.work.err);
  }
}

// Rows of V that a query does not see meet a weight of 0, but 0 * infinity is not 0. Rows behind the unit's
// last token (another sequence's, or none) are cleared; rows between its first and last token are cleared
// where they hold infinities or NaN, and marked: the queries that do see them add them at the unit's end.
__device__ void scrub(const PromptParams& p, AttentionShared& sh, uint32_t ring) {
  const int lane = threadIdx.x & 31;
  Slot slot;
  uint32_t count = 0;
#pragma unroll 1
  for (int unit = 0;; ++unit) {
    const Unit u = read_unit(sh, unit);
    if (!u.kind) return;
    uint32_t* bad = sh.bad[unit % kUnits];
    if (lane < kBadWords) bad[lane] = 0;
    __syncwarp();
    // a wait for the unit's last tiles lasts as long as its steps do: of 2^20 tokens 8192 steps, some 13 ms
    const uint32_t most = kPolls * (1 + (uint32_t)u.steps() / 4096);
#pragma unroll 1
    for (int step = u.from; step < u.from + u.steps(); ++step) {
      slot.next();                                // the step's V
      if (u.partly(step)) {
        if (!warp_wait(&sh.partly_full[count % kPartly], (count / kPartly) & 1, &sh.fail, most)) return;
#pragma unroll 1
        for (int r = lane; r < kTile; r += 32) {
          const uint32_t at = ring + slot.i * kTileBytes + r * 128;
          const int tok = step * kTile + r;
          bool blank = tok > u.reach;
          if (!blank && tok > u.tok0) {
            uint32_t seen = 0;                    // x * 0 is 0, or NaN where x is not finite
#pragma unroll 4
            for (int j = 0; j < 16; ++j) {
              uint4 x;
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                           : "r"(at + (j >> 3) * (kTileBytes / 2) + ((j + r) & 7) * 16) : "memory");
              asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(seen) : "r"(x.x), "r"(0u));
              asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(seen) : "r"(x.y), "r"(0u));
              asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(seen) : "r"(x.z), "r"(0u));
              asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(seen) : "r"(x.w), "r"(0u));
            }
            blank = nonfinite2(seen) != 0;
            if (blank) atomicOr(&bad[(tok - u.tok0 - 1) >> 5], 1u << ((tok - u.tok0 - 1) & 31));
          }
          if (blank) {
#pragma unroll 1
            for (int j = 0; j < 16; ++j)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};"
                           ::"r"(at + (j >> 3) * (kTileBytes / 2) + ((j + r) & 7) * 16), "r"(0u) : "memory");
            tc::fence_proxy_async_smem();
          }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.scrubbed[count % kPartly]);
        ++count;
      }
      slot.next();
    }
    let_go(sh, unit);
  }
}

// The tensor cores' work of group w, by a converged warp of its own. They take it in order, so the logits
// of half step j + 2 may be issued over the weights of half step j behind their product with V.
__device__ void mma_issuer(const PromptParams& p, AttentionShared& sh, int w, uint32_t tmem, uint32_t qbuf, uint32_t ring) {
  const uint64_t qd = tc::sw128_desc(qbuf + w * kTileBytes), vd = tc::sw128_desc_mn(ring, kTileBytes / 2, 1024);
  const uint32_t k_lo = (uint32_t)tc::sw128_desc(ring), v_lo = (uint32_t)vd;
  const uint32_t qk_hi = (uint32_t)(qd >> 32), v_hi = (uint32_t)(vd >> 32);
  const uint32_t s_at = tmem + w * kTile, o_at = s_at + 2 * kTile;
  constexpr uint32_t s_idesc = tc::idesc_bf16_f32(kTile, kHalf), o_idesc = tc::idesc_bf16_f32(kTile, kTile) | (1u << 16);
  uint32_t q_parity = 0, p_parity = 0, scrubs = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = ok && warp_wait(bar, parity, &sh.fail); };
  auto test = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, test_phase(bar, parity)) != 0; };
  // The logits of half step j of n, K in `slot`.
  auto logits = [&](const Slot& slot, int j, int n) {
    const int h = j & 1;
    tc::fence_after_sync();
    tm::warp_mma_rows(s_at + h * kHalf, qd, tm::desc_of(k_lo + ((slot.i * kTileBytes + h * (kHalf * 128)) >> 4), qk_hi), s_idesc);
    tm::warp_mma_commit(&sh.s_full[w][h]);
    if (h) tm::warp_mma_commit(&sh.kv_empty[slot.i]);
    if (j + 1 == n) tm::warp_mma_commit(&sh.q_empty[w]);
  };
  Slot k;                                         // K of the step whose logits come next (in the unit at hand)
  Unit u = read_unit(sh, 0);
  int lead = 0;                                   // half steps of the unit whose logits are issued beforehand
#pragma unroll 1
  for (int unit = 0; u.kind && ok; ++unit) {
    const int n = 2 * u.n(w);
    Slot v = k, first = k;                        // V's step; the next unit's first K
#pragma unroll 1
    for (int i = 0; i < u.steps(); ++i) first.step();
    Unit next = {};
    bool known = false;                           // the next unit
    int ahead = 0;                                // half steps of it whose logits are issued
#pragma unroll 1
    for (int j = lead; j < 2 && j < n && ok; ++j) {
      if (j == 0 && wait(&sh.q_full[w], q_parity)) q_parity ^= 1;
      if (wait(&sh.kv_full[k.i], k.parity)) logits(k, j, n);
    }
    if (n > 0) k.step();
#pragma unroll 1
    for (int j = 0; j < n && ok; ++j) {
      const int h = j & 1;
      if (h == 0) {
        v.next();
        if (!wait(&sh.kv_full[v.i], v.parity)) break;
        if (u.partly(u.from + j / 2)) {
          if (!wait(&sh.scrubbed[scrubs % kPartly], (scrubs / kPartly) & 1)) break;
          ++scrubs;
        }
      }
      if (!wait(&sh.p_full[w][h], p_parity)) break;
      tc::fence_after_sync();
      tm::warp_mma_weights(o_at, s_at + h * kHalf, tm::desc_of(v_lo + ((v.i * kTileBytes + h * (kHalf * 128)) >> 4), v_hi), o_idesc,
                           j > 0 ? 1u : 0u);
      tm::warp_mma_commit(&sh.o_full[w][h]);
      if (h) {
        tm::warp_mma_commit(&sh.kv_empty[v.i]);
        p_parity ^= 1;
        v.next();
      }
      if (j + 2 < n) {
        if (!wait(&sh.kv_full[k.i], k.parity)) break;
        logits(k, j + 2, n);
        if (h) k.step();
      } else {
        // the next unit's first logits, where that is no wait for the products to come
        if (!known && test(&sh.unit_full[(unit + 1) % kUnits], ((unit + 1) / kUnits) & 1)) {
          next = read_unit(sh, unit + 1);
          known = true;
        }
        if (known && next.n(w) > 0 && ahead == j + 2 - n && test(&sh.kv_full[first.i], first.parity) &&
            (ahead > 0 || test(&sh.q_full[w], q_parity))) {
          if (ahead == 0) q_parity ^= 1;
          logits(first, ahead++, 2 * next.n(w));
        }
      }
    }
    // both groups let go of every tile, of those of steps as well that the other group alone has
    Slot rest = v;
#pragma unroll 1
    for (int i = n; i < 2 * u.steps() && ok; ++i, rest.next()) {
      wait(&sh.kv_full[rest.i], rest.parity);
      if ((i & 1) && u.partly(u.from + i / 2)) {
        wait(&sh.scrubbed[scrubs % kPartly], (scrubs / kPartly) & 1);
        ++scrubs;
      }
      if (ok && (threadIdx.x & 31) == 0) tc::mbar_arrive(&sh.kv_empty[rest.i]);
    }
    if (!ok) break;
    let_go(sh, unit);
    u = known ? next : read_unit(sh, unit + 1);
    lead = ahead;
    k = first;
  }
  // every MMA must finish before tensor and shared memory are released
  tm::warp_mma_commit(&sh.done[w]);
  drain_phase(&sh.done[w], 0, p.work.err);
}

// The reference of a row's exponents moved: its O (where there is one) and the half step's weights so far
// (`columns` of them) follow by the factor f, those weights with a second rounding to bf16. (Whole numbers as references
// would spare them that, but round the largest weight, which is 1 otherwise: outputs were 0.0022 off instead of 0.0017
// for prompts of up to 45 tokens, and 0.0023 instead of 0.0022 for 8192; with the maximum first and whole steps from
// there on 0.0017 and 0.0023.) Whole warp; rare after a unit's first step.
__device__ __noinline__ void move_reference(uint32_t p_at, int columns, uint32_t o_at, float f) {
  tm::wait_stores();
  uint32_t x[16];
#pragma unroll 1
  for (int c = 0; c < columns; c += 16) {
    tm::load16(p_at + c, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = pack_bf16(__uint_as_float(x[k] << 16) * f, __uint_as_float(x[k] & 0xffff0000u) * f);
    tm::store16(p_at + c, x);
  }
#pragma unroll 1
  for (int c = 0; o_at && c < kHeadDim; c += 16) {
    tm::load16(o_at + c, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
    tm::store16(o_at + c, x);
  }
}

// A row's result of one part of a unit, and where it goes.
struct RowResult {
  Unit u;
  int n, unit;                                    // steps of this row's group; units before
  float ref, sum;
};

// Thread `row` of group w leaves its row of O, as it is when the group's products are through.
__device__ __forceinline__ void leave_row(const PromptParams& p, AttentionShared& sh, const RowResult& r, int w, int row, uint32_t o_at) {
  const int tl = p.by_group.div(row), token = r.u.tok0 + w * p.half + tl, hq = r.u.h * p.group + row - tl * p.group;
  const bool real = tl < p.half && token <= r.u.reach;
  const uint32_t* bad = sh.bad[r.unit % kUnits];
  uint32_t any_bad = 0;
  if (r.n > 0 && r.u.partly(r.u.from + r.n - 1))
    for (int k = 0; k < kBadWords; ++k) any_bad |= bad[k];
  const bool whole = r.u.kind == kWhole;
  const size_t part_row = (size_t)(2 * blockIdx.x + (r.u.from == 0 ? 1 : 0)) * kRows + w * kTile + row;
  const float inv = 1.f / r.sum;
  const long long out_row = (long long)r.u.row0 + token;
#pragma unroll 1
  for (int h = 0; h < 4; ++h) {
    float o[32];
    if (r.n > 0) {
      tc::tmem_ld32(o_at + 32 * h, o);
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = 0.f;
    }
    if (any_bad && real) {
      // rare: the rows that were cleared, for the queries that see them, where this part's steps hold them
#pragma unroll 1
      for (int k = 0; k < kRows; ++k) {
        const int tok = r.u.tok0 + 1 + k;
        if (!((bad[k >> 5] >> (k & 31)) & 1) || tok > token) continue;
        const int step = tok / kTile - r.u.from;
        if (step < 0 || step >= r.n) continue;
        const long long at = (long long)r.u.row0 + tok;
        const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(p.k) + r.u.plane * p.kb + r.u.h * p.kh + at * p.km;
        const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(p.v) + r.u.plane * p.vb + r.u.h * p.vh + at * p.vm + 32 * h;
        const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + r.u.plane * p.qb + hq * p.qh + out_row * p.qm;
        float z = 0.f;
#pragma unroll 1
        for (int d = 0; d < kHeadDim; ++d) z += __bfloat162float(qr[d]) * __bfloat162float(kr[d]);
        const float wt = ex2(z * p.scale2 - base_of(r.ref));
#pragma unroll
        for (int d = 0; d < 32; ++d) o[d] += wt * __bfloat162float(vr[d]);
      }
    }
    if (!real) continue;
    if (whole) {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + r.u.plane * p.ob + hq * p.oh + out_row * p.om + 32 * h;
      uint32_t y[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) y[k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
      if (p.out_sectors) {
        tm::store_sector(dst, y);
        tm::store_sector(dst + 16, y + 8);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          reinterpret_cast<uint4*>(dst)[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
      }
    } else {
      float* dst = p.part + part_row * kHeadDim + 32 * h;
#pragma unroll
      for (int k = 0; k < 4; ++k) tm::store_sector(dst + 8 * k, reinterpret_cast<const uint32_t*>(o) + 8 * k);
    }
  }
  if (!real) return;
  if (!whole) {
    p.part_ml[part_row] = make_float2(r.ref, r.sum);
  } else if (p.lse) {
    p.lse[((long long)r.u.plane * p.hq + hq) * p.work.m + out_row] = (r.ref + log2f(r.sum)) * 0.6931471805599453f;
  }
}

// One softmax group: thread `row` of group w.
__device__ void softmax_group(const PromptParams& p, AttentionShared& sh, int w, int row, uint32_t tmem) {
  const uint32_t lanes = (uint32_t)(row & ~31) << 16;
  const uint32_t s_at = tmem + lanes + (uint32_t)(w * kTile), o_at = s_at + 2 * kTile;
  const float scale = p.scale2, hidden = scale < 0.f ? INFINITY : -INFINITY;   // a logit that gives -infinity
  const int tl = p.by_group.div(row) + w * p.half;                // the row's token in the unit
  const bool has = tl < (w + 1) * p.half;
  uint32_t turn = 0;                              // steps so far
  // (no vote: a wait that gives up leaves `fail`, which is looked at once a unit)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    wait_for(bar, parity, &sh.fail);
    __syncwarp();
    tc::fence_after_sync();
  };
  // The products with V before half h of this step.
  auto wait_products = [&](int h) {
    wait(&sh.o_full[w][0], (h == 0 ? turn + 1 : turn) & 1);
    wait(&sh.o_full[w][1], (turn + 1) & 1);
  };
#pragma unroll 1
  for (int unit = 0;; ++unit) {
    const Unit u = read_unit(sh, unit);
    if (!u.kind) break;
    const int n = u.n(w), token = u.tok0 + tl;
    const bool real = has && token <= u.reach;
    float ref = real ? -INFINITY : 0.f;           // rows without a query never wait for a maximum
    float sum = 0.f;
#pragma unroll 1
    for (int j = 0; j < 2 * n; ++j) {
      const int h = j & 1;
      const uint32_t at = s_at + h * kHalf;
      const int seen = token - u.from * kTile - j * kHalf;        // columns 0 .. seen
      const bool masked = u.from * kTile + j * kHalf + kHalf - 1 > u.tok0 + w * p.half;   // some row does not see them all
      wait(&sh.s_full[w][h], turn & 1);
      // 32 columns at a time; the next ones are on their way while these are at work
      float x[2][32];
      auto chunk = [&](int ch, float(&y)[32], float(&next)[32]) {
        tm::wait32(y);
        if (ch == 0) tm::load32(at + 32, next);
        if (masked) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (32 * ch + k > seen) y[k] = hidden;
        }
        const uint64_t sc2 = pack_f32x2(scale, scale);
        uint32_t pk[16];
        float got;
#pragma unroll 1
        for (bool again = false;; again = true) {
          // weights against the reference, packed, and their sum
          const float nb = -base_of(ref);
          const uint64_t nb2 = pack_f32x2(nb, nb);
          uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const uint64_t e = ex2_f32x2(fma_f32x2(pack_f32x2(y[k], y[k + 1]), sc2, nb2));
            acc[(k >> 1) & 1] = add_f32x2(acc[(k >> 1) & 1], e);
            float e0, e1;
            split_f32x2(e, e0, e1);
            pk[k >> 1] = pack_bf16(e0, e1);
          }
          float a0, a1;
          split_f32x2(add_f32x2(acc[0], acc[1]), a0, a1);
          got = a0 + a1;
          // no reference yet, or a sum that says that it has fallen far behind the maximum (NaN as well)
          if (again || !__any_sync(0xffffffffu, real && (ref == -INFINITY || !(got < kMoveAbove)))) break;
          if (ch == 0) tm::wait32(next);          // no call while a load is on its way to registers
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 32; k += 2) top = fmax3(top, y[k] * scale, y[k + 1] * scale);
          const float to = real ? fmaxf(ref, top) : ref, f = weight_of(ref, to);
          ref = to;
          sum *= f;
          if (j > 0) wait_products(h);            // O follows once the products before this half step are through
          move_reference(at, 16 * ch, j > 0 ? o_at : 0, f);
        }
        sum += got;
        tm::store16(at + 16 * ch, pk);            // over columns that are in registers by now
      };
      tm::load32(at, x[0]);
      chunk(0, x[0], x[1]);
      chunk(1, x[1], x[0]);
      tm::wait_stores();
      tc::fence_before_sync();
      __syncwarp();
      if ((row & 31) == 0) tc::mbar_arrive(&sh.p_full[w][h]);     // a warp's 32 arrivals would go one by one
      turn += h;
    }
    if (n > 0) wait_products(0);
    if (__any_sync(0xffffffffu, *(volatile int*)&sh.fail)) break;
    leave_row(p, sh, RowResult{u, n, unit, ref, sum}, w, row, o_at);
    let_go(sh, unit);
    tc::fence_before_sync();                      // O is read: the next unit's first product follows our weights
  }
}

__global__ void __launch_bounds__(kThreads, 1) prompt_attention_kernel(const __grid_constant__ PromptParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ AttentionShared sh;
  const uint32_t smem = (tc::smem_u32(smem_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (warp == 0) tc::tmem_alloc(&sh.tmem_base, 4 * kTile);
  if (tid == 32) {
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(&sh.q_full[w], 1);
      tc::mbar_init(&sh.q_empty[w], 1);
      for (int h = 0; h < 2; ++h) {
        tc::mbar_init(&sh.s_full[w][h], 1);
        tc::mbar_init(&sh.p_full[w][h], kTile / 32);
        tc::mbar_init(&sh.o_full[w][h], 1);
      }
      tc::mbar_init(&sh.done[w], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(&sh.kv_full[i], 1);
      tc::mbar_init(&sh.kv_empty[i], 2);          // both groups' issuers
    }
    for (int i = 0; i < kPartly; ++i) {
      tc::mbar_init(&sh.partly_full[i], 1);
      tc::mbar_init(&sh.scrubbed[i], 1);
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
    tc::tma_prefetch_desc(&p.v_map);
  }
  pdl_wait();
  PromptCursor c;
  const bool any = first_unit<kThreads>(p.work, sh.scan, reinterpret_cast<int*>(smem_raw + (smem - tc::smem_u32(smem_raw))), c, Steps{p.work.tile});
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0), ring = smem + 2 * kTileBytes;
  if (any) {
    if (warp < kMmaWarp) {
      softmax_group(p, sh, warp >> 2, tid & (kTile - 1), tmem);
    } else if (warp < kTmaWarp) {
      mma_issuer(p, sh, warp - kMmaWarp, tmem, smem, ring);
    } else if (warp == kTmaWarp) {
      if (lane == 0) producer(p, sh, c, smem, ring);
      __syncwarp();
    } else {
      scrub(p, sh, ring);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, 4 * kTile);
  if (tid == 0 && sh.fail) raise_device_error(p.work.err, kDevWaitTimeout);
}

__global__ void prompt_begin_kernel(int* taken) {
  pdl_wait();
  if (threadIdx.x == 0) *taken = 0;
}

// Rows of units that two or more CTAs share: a warp merges its rows' parts, in the shares' order, four rows at a
// time, whose loads are on their way together.
constexpr int kJoinWarps = 8, kJoinSplit = 4, kJoinRows = 4;
static_assert(kRows % (kJoinRows * kJoinWarps * kJoinSplit) == 0);
__global__ void __launch_bounds__(kJoinWarps * 32) prompt_join_kernel(const __grid_constant__ PromptParams p) {
  pdl_wait();
  SplitUnit u;
  if (!split_unit(p.work, blockIdx.x + 1, u)) return;
  const int lane = threadIdx.x & 31, warp = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
#pragma unroll 1
  for (int row0 = warp * kJoinRows; row0 < kRows; row0 += kJoinWarps * kJoinSplit * kJoinRows) {
    float top[kJoinRows], sum[kJoinRows];
    float4 acc[kJoinRows];
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) top[r] = -INFINITY, sum[r] = 0.f, acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i = u.c0; i <= u.c1; ++i) {
      const size_t at = (size_t)(2 * i + (i == u.c0 ? 1 : 0)) * kRows + row0;
      float2 ml[kJoinRows];
      float4 v[kJoinRows];
#pragma unroll
      for (int r = 0; r < kJoinRows; ++r) {       // (of rows without a query whatever lies there)
        ml[r] = p.part_ml[at + r];
        v[r] = reinterpret_cast<const float4*>(p.part + (at + r) * kHeadDim)[lane];
      }
#pragma unroll
      for (int r = 0; r < kJoinRows; ++r) {
        const float to = fmaxf(top[r], ml[r].x), f = weight_of(top[r], to), wt = weight_of(ml[r].x, to);
        top[r] = to;
        sum[r] = sum[r] * f + ml[r].y * wt;
        acc[r].x = acc[r].x * f + v[r].x * wt;
        acc[r].y = acc[r].y * f + v[r].y * wt;
        acc[r].z = acc[r].z * f + v[r].z * wt;
        acc[r].w = acc[r].w * f + v[r].w * wt;
      }
    }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) {
      const int row = row0 + r, w = row / kTile, tl = p.by_group.div(row - w * kTile), g = row - w * kTile - tl * p.group;
      const int token = u.tile * p.work.tile + w * p.half + tl;
      if (tl >= p.half || token >= u.at.len) continue;
      const float inv = 1.f / sum[r];
      const int hq = u.h * p.group + g;
      const long long out_row = (long long)u.at.row0 + token;
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + u.at.plane * p.ob + hq * p.oh + out_row * p.om + 4 * lane) =
          make_uint2(pack_bf16(acc[r].x * inv, acc[r].y * inv), pack_bf16(acc[r].z * inv, acc[r].w * inv));
      if (p.lse && lane == 0)
        p.lse[((long long)u.at.plane * p.hq + hq) * p.work.m + out_row] = (top[r] + log2f(sum[r])) * 0.6931471805599453f;
    }
  }
}

bool multiple(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

int check_tensor(const evict_rows& x, int batch, int m, int heads, bool output, const char* name) {
  if (!x.data) return fail(EVICT_EINVAL, "%s must not be NULL", name);
  if (x.heads != heads) return fail(EVICT_EINVAL, "%s has %d heads, not %d", name, x.heads, heads);
  if (!multiple(x.data, 16) || x.stride_b % 8 || x.stride_h % 8 || x.stride_m % 8)
    return fail(EVICT_EINVAL, "%s: addresses and strides must be multiples of 16 bytes", name);
  if (x.stride_b < 0 || x.stride_h < 0 || x.stride_m < 0) return fail(EVICT_EINVAL, "%s: strides must not be negative", name);
  if ((batch > 1 && !x.stride_b) || (heads > 1 && !x.stride_h) || (m > 1 && !x.stride_m))
    return fail(EVICT_EINVAL, "%s is expanded (a stride of 0): give every row a place of its own", name);
  if (output && rows_overlap(x, batch, m)) return fail(EVICT_EINVAL, "%s: rows lie on top of each other", name);
  return EVICT_OK;
}

// The kernel's dynamic shared memory, allowed once for each device.
cudaError_t allow_smem(int dev) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(prompt_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

int make_plan(const evict_prompt* a, PromptPlan* plan) {
  const int group = a->q.heads / a->k.heads, half = kTile / group, tile = 2 * half;
  const int rc = plan_prompt(a, tile, ((long long)a->m + kTile - 1) / kTile, kEntry, kMinSteps,
                             a->m <= kWholeRows ? 0 : kWholeRounds, 2 * kRows * sizeof(float2), 2 * (size_t)kRows * kHeadDim * sizeof(float), true, plan);
  plan->p.half = half;
  return rc;
}

}  // namespace

int check_prompt_sizes(const evict_prompt* a) {
  if (!a) return fail(EVICT_EINVAL, "the arguments are NULL");
  if (a->batch < 0 || a->m < 0) return fail(EVICT_EINVAL, "batch and m must be >= 0 (got %d, %d)", a->batch, a->m);
  if (a->q.heads < 1 || a->k.heads < 1 || a->q.heads % a->k.heads)
    return fail(EVICT_EINVAL, "q's heads (%d) must be a multiple of k's (%d)", a->q.heads, a->k.heads);
  if (a->q.heads / a->k.heads > EVICT_MAX_PROMPT_GROUP)
    return fail(EVICT_ELIMIT, "%d query heads for a KV head are more than %d", a->q.heads / a->k.heads, EVICT_MAX_PROMPT_GROUP);
  if (a->starts && (a->batch != 1 || a->n_seqs < 0))
    return fail(EVICT_EINVAL, "packed sequences lie in a batch of 1 (got %d), and n_seqs must be >= 0 (got %d)", a->batch, a->n_seqs);
  if (a->starts && a->n_seqs > EVICT_MAX_PROMPT_SEQS)
    return fail(EVICT_ELIMIT, "%d sequences are more than %d", a->n_seqs, EVICT_MAX_PROMPT_SEQS);
  if ((long long)a->batch * a->m >= (1ll << 30) || (long long)a->batch * a->m * a->q.heads >= (1ll << 30))
    return fail(EVICT_ELIMIT, "batch * heads * m is 2^30 or more");
  return EVICT_OK;
}

int check_prompt(const evict_prompt* a, bool attention) {
  if (const int rc = check_prompt_sizes(a)) return rc;
  if (!good_scale(a->scale)) return fail(EVICT_EINVAL, "scale must be finite and below 2^127");
  if (!multiple(a->starts, 4) || !multiple(a->lse, 4) || !multiple(a->weights, 4) || !multiple(a->error, 4))
    return fail(EVICT_EINVAL, "starts, lse, weights and error must be 4-byte aligned");
  if (a->batch == 0 || a->m == 0) return EVICT_OK;
  int rc;
  if ((rc = check_tensor(a->q, a->batch, a->m, a->q.heads, false, "q")) ||
      (rc = check_tensor(a->k, a->batch, a->m, a->k.heads, false, "k")))
    return rc;
  if (!attention) {
    if (!a->lse || !a->weights) return fail(EVICT_EINVAL, "lse and weights must not be NULL");
    if (a->last < 0) return fail(EVICT_EINVAL, "last must be >= 0 (got %d)", a->last);
    const size_t tokens = (size_t)a->batch * a->m;
    if (overlap(a->weights, tokens * a->k.heads * 4, a->lse, tokens * a->q.heads * 4))
      return fail(EVICT_EINVAL, "weights must not overlap lse: it is read while results are written");
    if (a->weights == a->q.data || a->weights == a->k.data)
      return fail(EVICT_EINVAL, "weights must not be q or k: they are read while results are written");
    return EVICT_OK;
  }
  if ((rc = check_tensor(a->v, a->batch, a->m, a->k.heads, false, "v")) ||
      (rc = check_tensor(a->out, a->batch, a->m, a->q.heads, true, "out")))
    return rc;
  if (a->out.data == a->q.data || a->out.data == a->k.data || a->out.data == a->v.data)
    return fail(EVICT_EINVAL, "out must not be q, k or v: they are read while results are written");
  return EVICT_OK;
}

// Sizes alone decide: the sequences' lengths are the device's.
int plan_prompt(const evict_prompt* a, int tile, long long most_steps, int entry, int min_steps, int whole_rounds,
                size_t part_ml, size_t part, bool longest_last, PromptPlan* out) {
  PromptPlan& P = *out;
  P = PromptPlan();
  PromptParams& p = P.p;
  PromptWork& w = p.work;
  p.hq = a->q.heads;
  p.group = a->q.heads / a->k.heads;
  p.by_group = Divisor(p.group);
  w.starts = a->starts;
  w.seqs = a->starts ? a->n_seqs : a->batch;
  w.m = a->m;
  w.hkv = a->k.heads;
  w.tile = tile;
  w.entry = entry;
  w.min_steps = min_steps;
  w.longest_last = longest_last;
  const int seq_blocks = (a->m + tile - 1) / tile;
  const long long blocks = a->starts ? (long long)a->m / tile + a->n_seqs : (long long)a->batch * seq_blocks;
  if (blocks * w.hkv >= (1ll << 30)) return fail(EVICT_ELIMIT, "sequences and KV heads make 2^30 units of work or more");
  w.blocks = (int)blocks;
  w.by_hkv = Divisor(w.hkv);
  w.by_tile = Divisor(tile);
  w.by_seq_blocks = Divisor(seq_blocks);
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&P.sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "looking up the device");
  P.dev = dev;
  w.whole = blocks * w.hkv >= (long long)whole_rounds * P.sms;
  // Steps are added up only where units are cut: the plane has few blocks then, and is short.
  if (!w.whole && (double)blocks * w.hkv * (double)(most_steps + entry) >= 2147483648.0)
    return fail(EVICT_ELIMIT, "the sequences are too long for one call");
  size_t off = 256;                               // an error word, for callers without one
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round256(bytes);
    return at;
  };
  w.total = reinterpret_cast<int*>(take(3 * sizeof(int)));
  w.taken = w.whole && blocks * w.hkv > kTakenRounds * P.sms ? w.total + 2 : nullptr;
  w.begin = reinterpret_cast<PromptBegin*>(take(P.sms * sizeof(PromptBegin)));
  w.block_base = reinterpret_cast<int*>(take(((size_t)w.seqs + 1) * sizeof(int)));
  if (w.starts && w.seqs <= kOrderedSeqs && !longest_last) {
    int* order = reinterpret_cast<int*>(take(blocks * sizeof(int)));   // (taken or not: `last` does not change the bytes)
    if (w.taken) w.order = order;
  }
  p.part_ml = reinterpret_cast<float2*>(take(w.whole ? 0 : P.sms * part_ml));
  p.part = reinterpret_cast<float*>(take(w.whole ? 0 : P.sms * part));
  P.bytes = off;
  return EVICT_OK;
}

int bind_prompt(const evict_prompt* a, PromptPlan* plan) {
  if (!a->workspace || !multiple(a->workspace, 256)) return fail(EVICT_EINVAL, "workspace must be 256-byte aligned");
  if (a->workspace_bytes < plan->bytes)
    return fail(EVICT_EINVAL, "workspace has %zu bytes, the call needs %zu", a->workspace_bytes, plan->bytes);
  if (!encode_tiled()) return fail(EVICT_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");
  char* base = static_cast<char*>(a->workspace);
  PromptParams& p = plan->p;
  auto rebase = [&](auto*& x) { x = reinterpret_cast<std::remove_reference_t<decltype(x)>>(base + reinterpret_cast<size_t>(x)); };
  rebase(p.work.total);
  rebase(p.work.begin);
  if (p.work.taken) p.work.taken = p.work.total + 2;
  rebase(p.work.block_base);
  if (p.work.order) rebase(p.work.order);
  rebase(p.part_ml);
  rebase(p.part);
  p.work.err = a->error ? a->error : reinterpret_cast<int*>(base);
  p.lse = a->lse;
  p.weights = a->weights;
  p.scale2 = scale_base2(a->scale);
  return EVICT_OK;
}

int begin_prompt(const PromptWork& w, cudaStream_t st) {
  if (!w.taken) return EVICT_OK;
  const cudaError_t e = launch_pdl(prompt_begin_kernel, dim3(1), dim3(32), 0, st, nullptr, w.taken);
  if (e != cudaSuccess) return cuda_fail(e, "prompt begin kernel launch");
  g_launches.fetch_add(1);
  return EVICT_OK;
}

int encode_heads(CUtensorMap* map, const evict_rows& x, int batch, int m, int heads_box, int rows_box, bool heads_first,
                 const char* name) {
  // a dimension of extent 1 is never stepped over, but its stride still has to be one the encoder takes
  const cuuint64_t hs = (x.heads > 1 ? x.stride_h : kHeadDim) * 2, ms = (m > 1 ? x.stride_m : kHeadDim) * 2,
                   bs = (batch > 1 ? x.stride_b : kHeadDim) * 2;
  const cuuint64_t hn = (cuuint64_t)x.heads, mn = (cuuint64_t)m;
  const cuuint64_t dims[4] = {kHeadDim, heads_first ? hn : mn, heads_first ? mn : hn, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {heads_first ? hs : ms, heads_first ? ms : hs, bs};
  const cuuint32_t hb = (cuuint32_t)heads_box, mb = (cuuint32_t)rows_box;
  const cuuint32_t box[4] = {64, heads_first ? hb : mb, heads_first ? mb : hb, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  if (encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, x.data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return fail(EVICT_EINVAL, "%s has sizes or strides beyond a tensor map's", name);
  return EVICT_OK;
}

}  // namespace evict

using namespace evict;

extern "C" int evict_prompt_attention_workspace(const evict_prompt* a, size_t* bytes) {
  if (!bytes) return fail(EVICT_EINVAL, "bytes is NULL");
  PromptPlan plan;
  int rc;
  if ((rc = check_prompt_sizes(a)) || (rc = make_plan(a, &plan))) return rc;
  *bytes = plan.bytes;
  return EVICT_OK;
}

extern "C" int evict_prompt_attention(const evict_prompt* a) {
  int rc;
  if ((rc = check_prompt(a, true))) return rc;
  if (a->batch == 0 || a->m == 0 || (a->starts && a->n_seqs == 0)) return EVICT_OK;
  PromptPlan plan;
  if ((rc = make_plan(a, &plan)) || (rc = bind_prompt(a, &plan))) return rc;
  PromptParams& p = plan.p;
  p.q = a->q.data, p.qb = a->q.stride_b, p.qh = a->q.stride_h, p.qm = a->q.stride_m;
  p.k = a->k.data, p.kb = a->k.stride_b, p.kh = a->k.stride_h, p.km = a->k.stride_m;
  p.v = a->v.data, p.vb = a->v.stride_b, p.vh = a->v.stride_h, p.vm = a->v.stride_m;
  p.out = a->out.data, p.ob = a->out.stride_b, p.oh = a->out.stride_h, p.om = a->out.stride_m;
  p.out_sectors = multiple(a->out.data, 32) && a->out.stride_b % 16 == 0 && a->out.stride_h % 16 == 0 && a->out.stride_m % 16 == 0;
  if ((rc = encode_heads(&p.q_map, a->q, a->batch, a->m, p.group, p.half, true, "q")) ||
      (rc = encode_heads(&p.k_map, a->k, a->batch, a->m, 1, kTile, false, "k")) ||
      (rc = encode_heads(&p.v_map, a->v, a->batch, a->m, 1, kTile, false, "v")))
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  cudaError_t e = allow_smem(plan.dev);
  if (e != cudaSuccess) return cuda_fail(e, "prompt attention kernel attribute");
  const int ctas = p.work.whole ? std::min(plan.sms, p.work.blocks * p.work.hkv) : plan.sms;
  if ((rc = begin_prompt(p.work, st))) return rc;
  if ((e = launch_pdl(prompt_attention_kernel, dim3(ctas), dim3(kThreads), kSmem, st, nullptr, p)) != cudaSuccess)
    return cuda_fail(e, "prompt attention kernel launch");
  g_launches.fetch_add(1);
  if (!p.work.whole && ctas > 1) {
    if ((e = launch_pdl(prompt_join_kernel, dim3(ctas - 1, kJoinSplit), dim3(kJoinWarps * 32), 0, st, nullptr, p)) != cudaSuccess)
      return cuda_fail(e, "prompt join kernel launch");
    g_launches.fetch_add(1);
  }
  return EVICT_OK;
}
