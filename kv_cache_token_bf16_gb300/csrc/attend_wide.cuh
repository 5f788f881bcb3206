// Attention of many query rows over a shared prefix or a sequence's rows (see attend.cu): tcgen05
// tensor cores.
//
// A CTA works with eleven of its warps on its share. A unit is a
// (stream, KV head, tile of 256 query rows); K and V stream through a ring of
// five 32 KB tiles of 128 rows (TMA, warp 10). Warps 0-3 and 4-7 are two
// softmax groups, a thread per query row, each with its own 128 x 128 logits
// and 128 x 128 output accumulator in tensor memory (512 columns in all);
// warps 8 and 9 issue their MMAs. A group's work on a step goes in two halves
// of 64 rows of K and V:
//     S = Q K^T (MMA) -> P = 2^(S scale - ref) as bf16 over S in tensor memory
//     (softmax group) -> O += P V (MMA, P read from tensor memory).
// While the tensor cores work on one half the group exponentiates the other,
// and the other group's halves come between. A unit of more than 128 rows
// gives each group 128 rows and both groups every step; a smaller one gives
// both the same rows and every other step each (two partial results).
//
// The exponent's reference is a row's maximum over the first 32 columns that it
// sees, and stays there: later columns are taken against it without a maximum
// of their own while the sum of 32 of their weights is below 2^12, and it moves
// to the running maximum (with a read and write of O in tensor memory) where
// that is passed. Weights, sums and O are relative to it and floating, so the
// result does not depend on where it stands, but for roundings: the weight of the
// maximum itself is 1, and bf16 holds that. (A whole number for a reference would
// let the at most 32 bf16 weights of a half step that move with it go unrounded, and
// round the largest weights in place of them: an error of 0.0023-0.0024 where this
// has 0.0020-0.0022, relative to the result in the 2-norm.) Weights enter the product
// with V as bf16 (half a step: 2^-8 of a weight at most), at twice the rate of
// the split that the few-row kernel uses; their roundings are independent, so
// the output's error grows from one rounding to the root of two.
//
// Measured: 8 sequences of up to 509 questions behind 4,096 rows (32 query
// heads, 141 GFLOP) 160 us, 0.88 PFLOP/s; a step of 256 query rows takes 3,400
// clocks, 2,048 of them the products' at the tensor cores' rate. What bounds
// it there: the first product reads Q from shared memory, 64 clocks for an
// instruction whatever its width, so halves of 64 columns cost it twice, 3,072
// in all. Steps of whole 128 columns cost 2,048 there but leave the tensor
// cores waiting for the softmax: 179 us, and with only the second product in
// halves 190. Half the exponentials, or none of the row sums, change nothing.
// Around the steps: 10,000 clocks to the first logits (schedule, queries, K),
// 10,000 between two units.
#pragma once

#include <cuda_bf16.h>

#include "attend.cuh"

namespace evict {
namespace {

constexpr int kTile = 128, kHalf = 64;
constexpr int kTileBytes = kTile * kHeadDim * 2;
constexpr int kRing = 5;
constexpr int kWideSmem = (2 + kRing) * kTileBytes;
constexpr int kMmaWarp = 8, kTmaWarp = 10;
constexpr int kBadWords = 9;                      // 257 tokens and more
constexpr int kBadSets = 4;                       // of a group's segments in turn (see softmax_group)
constexpr float kMoveAbove = 4096.f;              // sum of 32 weights that makes the reference move

struct WideShared {
  uint64_t kv_full[kRing], kv_empty[kRing];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2], done[2];   // group, half of the step
  uint32_t tmem_base;
  int fail;
  uint32_t bad[2][kBadSets][kBadWords];           // of either group: rows of V that it found blanked
  uint32_t blanked[kRing][kTile / 32];            // of the tile of V in a slot: rows that either group blanked
};

using WideCursor = Cursor<kWideRows, kWideTokens>;

// The part of a unit that this CTA takes.
struct Segment {
  int steps;                                      // from the cursor's on
  int pre_steps;                                  // of the unit
  bool two, alt;                                  // both groups on every step; or taking turns
  __device__ __forceinline__ Segment(const AttendParams& p, const WideCursor& c, int left) {
    steps = min(c.k.steps - c.step, left);
    pre_steps = (c.k.pre + kWideTokens - 1) / kWideTokens;
    two = c.k.n * p.group - c.k.tile * kWideRows > kTile;
    alt = !two && !p.wide.joint;
  }
  __device__ __forceinline__ bool has(int w, int i) const { return two || (alt ? (i & 1) == w : w == 0); }
  __device__ __forceinline__ int jobs(int w) const { return two ? steps : alt ? (steps + 1 - w) / 2 : w == 0 ? steps : 0; }
};

// The unit's first query sees own rows before this one; from here to the last query's, rows with
// infinities or NaN in V are marked (at most 256 tokens).
__device__ __forceinline__ int first_marked(const AttendParams& p, const WideCursor& c) {
  return c.k.len - c.k.n + p.by_group.div(c.k.tile * kWideRows) + 1;
}

// A position in the ring of K and V tiles, and the parity of the phase that fills it.
struct Slot {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == kRing) i = 0, parity ^= 1;
  }
};

__device__ void producer(const AttendParams& p, WideShared& sh, WideCursor c, int count, uint32_t ring) {
  const WorkSet& set = p.wide;
  const int lane = threadIdx.x & 31, blocks = set.blocks();
  const int box = p.box_rows, boxes = box ? kTile / box : 0;
  Slot slot;
  int used = 0;
  bool ok = true;
  while (ok && count > 0) {
    const Segment g(p, c, count);
    const int plane = c.k.s < set.prefixes ? c.k.s : p.fan ? p.by_fan.div(c.k.s - set.prefixes) : 0;
    const int32_t* table = p.table + (long long)(c.k.s - set.prefixes) * p.table_stride;
    for (int i = 0; i < g.steps && ok; ++i) {
      const int step = c.step + i;
      const bool pre = step < g.pre_steps;
      const int row0 = (pre ? step : step - g.pre_steps) * kWideTokens, row = row0 + lane * box;   // this lane's page
      int page = p.n_pages;                       // outside the pool: zeros
      if (!pre && lane < boxes && row < c.k.len) {
        page = table[row >> p.page_shift];
        if (page < 0 || page >= p.n_pages) {
          raise_device_error(p.err, kDevBadIndex);
          page = p.n_pages;
        }
      }
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        ok = wait_phase(&sh.kv_empty[slot.i], slot.parity ^ 1, &sh.fail, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint64_t* bar = &sh.kv_full[slot.i];
        const uint32_t dst = ring + slot.i * kTileBytes;
        // both groups are done with the slot's last tile, and see these zeros once they see the next
        if (kv && lane < kTile / 32) sh.blanked[slot.i][lane] = 0;
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, kTileBytes);
        __syncwarp();
        if (pre) {
          if (lane < 2)
            tma_load_5d(dst + lane * (kTileBytes / 2), &p.wide_pre[kv], 0, row0, lane, c.h, plane, bar);
        } else if (lane < boxes) {
          for (int hf = 0; hf < 2; ++hf)
            tma_load_5d(dst + hf * (kTileBytes / 2) + lane * box * 128, &p.wide_own[kv], 0,
                        row & ((1 << p.page_shift) - 1), hf, c.h, page, bar);
        }
        slot.next();
        ++used;
      }
    }
    count -= g.steps;
    if (count == 0) break;
    c.next_unit(p, set, blocks);
    c.settle(count);
  }
  // every copy issued must land before the CTA may release its shared memory
  for (int i = 0; i < kRing && i < used; ++i) drain_phase(&sh.kv_full[i], ((used - 1 - i) / kRing) & 1, p.err);
}

// Bounds a thread's polling (the clock is read rarely).
struct Watch {
  uint32_t polls = 0;
  uint64_t t0 = 0;
  __device__ __forceinline__ bool go_on(WideShared& sh, int* err) {
    if ((++polls & 1023) != 0) return true;
    if (*(volatile int*)&sh.fail) return false;
    const uint64_t t = tc::global_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 <= kWaitLimitNs) return true;
    *(volatile int*)&sh.fail = 1;
    raise_device_error(err, kDevWaitTimeout);
    return false;
  }
};
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) { return (uint64_t)lo | ((uint64_t)hi << 32); }

// Half a step's S = Q K^T, both K-major; q and k: the tiles' descriptors' low words (their steps
// differ in the start address alone, which does not carry over).
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t q, uint32_t k, uint32_t hi) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, kHalf);
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const uint32_t off = (uint32_t)((s >> 2) * kTile * 128 + (s & 3) * 32) >> 4;
    tc::mma_bf16(d, desc_of(q + off, hi), desc_of(k + off, hi), idesc, s > 0 ? 1u : 0u);
  }
}
// O (+)= P V of half a step: P in tensor memory (two weights a column), V with its rows as the
// product's depth (MN-major). 16 rows of V are 2048 bytes of each half of its columns.
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t pt, uint32_t v, uint32_t hi, bool accumulate) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, kTile) | (1u << 16);
#pragma unroll
  for (int s = 0; s < kHalf / 16; ++s) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(pt + s * 8), "l"(desc_of(v + s * 128, hi)), "r"(idesc), "r"(accumulate || s > 0 ? 1u : 0u)
        : "memory");
  }
}

// The MMAs of group w, issued by one warp of its own. S of half step j + 2 goes where the weights of
// half step j lay: behind their product with V, MMAs run in order. What is there first is done first:
// the next K, the weights of the next product, the other group's tiles (let go of).
__device__ void mma_issuer(const AttendParams& p, WideShared& sh, WideCursor c, int count, int w, uint32_t tmem,
                           uint32_t qbuf, uint32_t ring) {
  const WorkSet& set = p.wide;
  const int blocks = set.blocks();
  const uint64_t qk = tc::sw128_desc(qbuf + w * kTileBytes), pv = tc::sw128_desc_mn(ring, kTileBytes / 2, 1024);
  const uint32_t q_lo = (uint32_t)qk, k_lo = (uint32_t)tc::sw128_desc(ring), qk_hi = (uint32_t)(qk >> 32);
  const uint32_t v_lo = (uint32_t)pv, v_hi = (uint32_t)(pv >> 32);
  const uint32_t s_at = tmem + w * kTile, o_at = s_at + 2 * kTile;
  uint32_t p_parity = 0, q_parity = 0;
  Slot slot;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = wait_phase(bar, parity, &sh.fail, p.err); };
  // Tiles of the other group's steps. Both groups let go of every tile: were its user alone to do
  // it, the other might look for a phase of its barrier that has long been over.
  auto release = [&](int tiles) {
#pragma unroll 1
    for (; tiles > 0 && wait(&sh.kv_full[slot.i], slot.parity); --tiles, slot.next()) tc::mbar_arrive(&sh.kv_empty[slot.i]);
  };
  while (ok && count > 0) {
    const Segment g(p, c, count);
    const int n = 2 * g.jobs(w);                  // half steps
    if (n > 0) {
      if (!wait(&sh.q_full[w], q_parity)) break;
      q_parity ^= 1;
    }
    Slot v, v_next;                               // V of the product's step, of the last S's
    int jq = 0, jp = 0;                           // half steps whose S, whose product were issued
    int pass = g.alt && w == 1 && n > 0 ? 2 : 0;  // tiles of the other group before the next K
    int at = pass / 2;                            // steps passed
    Watch watch;
#pragma unroll 1
    while (jp < n) {
      if (pass > 0) {
        if (tc::mbar_try_wait(&sh.kv_full[slot.i], slot.parity)) {
          tc::mbar_arrive(&sh.kv_empty[slot.i]);
          slot.next();
          --pass;
        }
      } else if (jq < n && jq < jp + 2 && tc::mbar_try_wait(&sh.kv_full[slot.i], slot.parity)) {
        const int h = jq & 1;
        tc::fence_after_sync();
        issue_qk(s_at + h * kHalf, q_lo, k_lo + ((slot.i * kTileBytes + h * (kHalf * 128)) >> 4), qk_hi);
        tc::mma_commit(&sh.s_full[w][h]);
        if (h == 0) {
          v_next = slot;
          v_next.next();
        } else {
          tc::mma_commit(&sh.kv_empty[slot.i]);
          slot.next();
          slot.next();
          ++at;
          if (g.alt && jq + 1 < n) pass = 2, ++at;
        }
        ++jq;
      }
      if (jp < jq) {
        const int h = jp & 1;
        if (h == 0) v = v_next;
        if (tc::mbar_try_wait(&sh.p_full[w][h], p_parity) && tc::mbar_try_wait(&sh.kv_full[v.i], v.parity)) {
          tc::fence_after_sync();
          issue_pv(o_at, s_at + h * kHalf, v_lo + ((v.i * kTileBytes + h * (kHalf * 128)) >> 4), v_hi, jp > 0);
          tc::mma_commit(&sh.o_full[w][h]);
          if (h) {
            tc::mma_commit(&sh.kv_empty[v.i]);
            p_parity ^= 1;
          }
          ++jp;
          watch = Watch();
        }
      }
      if (!(ok = watch.go_on(sh, p.err))) break;
    }
    if (ok) release(2 * (g.steps - at));
    count -= g.steps;
    if (count == 0 || !ok) break;
    c.next_unit(p, set, blocks);
    c.settle(count);
  }
  // every MMA must finish before tensor and shared memory are released
  tc::mma_commit(&sh.done[w]);
  drain_phase(&sh.done[w], 0, p.err);
}

// 32 columns of this thread's row. The load runs on; nothing may use the registers before wait32,
// which has them as operands to that end.
__device__ __forceinline__ void load32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void wait32(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :: "memory");
}
__device__ __forceinline__ void store16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 32 bytes to global memory, 32-byte aligned: a whole sector from each thread
__device__ __forceinline__ void store_sector(void* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
// 16 columns, complete on return
__device__ __forceinline__ void load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
}
__device__ __forceinline__ void wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The reference of a row's exponents moved: its O (where there is one) and the step's weights so
// far (`columns` of them) follow by the factor f. Whole warp; rare after a unit's first step.
__device__ __noinline__ void move_reference(uint32_t s_at, int columns, uint32_t o_at, float f) {
  wait_stores();
  uint32_t x[16];
  for (int c = 0; c < columns; c += 16) {
    load16(s_at + c, x);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = pack_bf16(__uint_as_float(x[k] << 16) * f, __uint_as_float(x[k] & 0xffff0000u) * f);
    store16(s_at + c, x);
  }
  if (o_at) {
    for (int c = 0; c < kHeadDim; c += 16) {
      load16(o_at + c, x);
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * f);
      store16(o_at + c, x);
    }
  }
}

// One softmax group: thread `row` of group w.
__device__ void softmax_group(const AttendParams& p, WideShared& sh, WideCursor c, int count, int w, int row, uint32_t tmem,
                              unsigned char* qbuf, uint32_t ring) {
  const WorkSet& set = p.wide;
  const int warp = row >> 5, blocks = set.blocks();
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t s_at = tmem + lanes + (uint32_t)(w * kTile), o_at = s_at + 2 * kTile;
  const uint32_t flip = p.scale2 < 0.f ? 0x80008000u : 0u;   // a negative scale: of -Q, so that maxima stay maxima
  const float scale = fabsf(p.scale2);
  unsigned char* q_mine = qbuf + w * kTileBytes;

  // this row's query into the group's tile
  auto load_query = [&](const WideCursor& cu, const Segment& g) {
    const QueryRow q = query_row<kWideRows>(p, set, cu.k, g.two ? w * kTile + row : row);
    // A group without a job in this part announces nothing (it could announce twice before the
    // MMA warp has looked once).
    if (g.jobs(w) == 0) return q;
    // two rows of the warp at a time, half a warp on each: whole lines of global memory
    const long long mine = q.real ? (long long)q.b * p.qb + (long long)(cu.h * p.group + q.g) * p.qh + (long long)q.t * p.qm : -1;
    const int half = (row >> 4) & 1, chunk = row & 15;
    uint4 x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const long long from = __shfl_sync(0xffffffffu, mine, 2 * i + half);
      x[i] = make_uint4(0, 0, 0, 0);
      if (from >= 0) x[i] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + from)[chunk];
    }
    // row 2 i + half: its chunk's place is that of row `half` moved on, but for the swizzle
    unsigned char* to = q_mine + 32 * warp * 128 + (chunk >> 3) * (kTileBytes / 2) + half * 128;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i].x ^= flip, x[i].y ^= flip, x[i].z ^= flip, x[i].w ^= flip;
      *reinterpret_cast<uint4*>(to + 2 * i * 128 + (((chunk & 7) ^ ((2 * i + half) & 7)) << 4)) = x[i];
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if ((row & 31) == 0) tc::mbar_arrive(&sh.q_full[w]);
    return q;
  };

  // A step's rows of V that no query of the unit sees may hold anything, and so may rows that some
  // queries do not see: both meet weights of 0, but 0 * infinity is not 0. This thread looks at the
  // tile's row `row` and writes zeros over it in the first case and, where it holds infinities or
  // NaN, in the second, with a mark for the group's queries that do see it. Both groups may do so with
  // the same tile, and each writes all of a row's zeros itself before its own product. A group may
  // find a row that the other one has begun to clear, finite by then: the row's bit in `blanked` is
  // there before the zeros are, so who reads a zero of the other's reads its bit afterwards.
  auto blank_rows = [&](int slot, int own0, int first, uint32_t* bad) {
    const uint32_t at = ring + slot * kTileBytes + row * 128;
    const int tok = own0 + row;
    bool blank = tok > c.k.reach;
    if (!blank && tok >= first && tok >= 0) {
#pragma unroll 1
      for (int j = 0; j < 16 && !blank; ++j) {
        uint4 x;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(at + (j >> 3) * (kTileBytes / 2) + ((j + row) & 7) * 16) : "memory");
        blank = nonfinite2(x.x) | nonfinite2(x.y) | nonfinite2(x.z) | nonfinite2(x.w);
      }
      const uint32_t bit = 1u << (row & 31);
      uint32_t* const blanked = &sh.blanked[slot][row >> 5];
      __threadfence_block();
      if (!blank) blank = *(volatile uint32_t*)blanked & bit;
      if (blank) {
        atomicOr(blanked, bit);
        atomicOr(&bad[(tok - first) >> 5], 1u << ((tok - first) & 31));
        __threadfence_block();
      }
    }
    if (blank) {
#pragma unroll 1
      for (int j = 0; j < 16; ++j)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + (j >> 3) * (kTileBytes / 2) + ((j + row) & 7) * 16),
                     "r"(0u) : "memory");
      tc::fence_proxy_async_smem();
    }
  };

  uint32_t s_parity = 0;                          // of the step at hand
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool there = wait_phase(bar, parity, &sh.fail, p.err);
    ok = __all_sync(0xffffffffu, there) && ok;
    tc::fence_after_sync();
    return ok;
  };
  // The products with V before half h of this step. (Two are in flight at most: one barrier for both could be
  // a phase further than the one that is waited for.)
  auto wait_products = [&](int h) {
    wait(&sh.o_full[w][0], h == 0 ? s_parity ^ 1 : s_parity);
    wait(&sh.o_full[w][1], s_parity ^ 1);
  };
  Segment g(p, c, count);
  QueryRow q = {};
  int limit = -1;                                 // last own row that this query sees
  float ref = -INFINITY, sum = 0.f;
  bool marks = false;                             // the segment holds rows that may have been marked
  // The segments in which this group has a job, counted: segment i's marks are in set i % kBadSets. Its
  // first warp clears the set of segment i + 2 as it begins segment i. It has then seen the products of
  // segment i - 1, so every warp has left segment i - 2 and its marks, which lay there; and none marks
  // in segment i + 2 before all four warps have announced its queries.
  int turn = -1;
  Slot slot;                                      // of the segment's first tile
  for (int segment = -1;; ++segment) {            // -1: only the first unit's queries
    // The next unit's queries: this group's last S is in registers, so its tile is free.
    const WideCursor at = c;
    const Segment part = g;
    const QueryRow mine = q;
    if (segment >= 0) {
      count -= part.steps;
      if (count > 0) {
        c.next_unit(p, set, blocks);
        c.settle(count);
      }
    }
    const bool more = count > 0;
    if (more) {
      g = Segment(p, c, count);
      q = load_query(c, g);
    }
    if (segment >= 0) {
      const int jobs = part.jobs(w);
      if (jobs > 0) wait_products(0);
      if (!ok) break;
      const bool whole = set.joint && part.steps == at.k.steps;     // no other part, no other unit for these rows
      const bool write = mine.real && (part.two || part.alt || w == 0);
      // groups that take turns leave a row each, half a slot apart (kTile where both have all steps)
      const size_t prow = set.joint ? (size_t)(2 * blockIdx.x + (at.step == 0 ? 1 : 0)) * kWideRows + w * kTile + row
                                    : set.slot_row(at.unit, blockIdx.x) + w * (set.rows_of(at.unit) >> 1) + row;
      const bool sees = at.k.pre > 0 || limit >= 0;
      const int hq = at.h * p.group + mine.g;
      const float inv = sees ? 1.f / sum : 0.f;
      uint32_t any_bad = 0;
      const int first = first_marked(p, at);
      const uint32_t* bad = sh.bad[w][turn & (kBadSets - 1)];   // (marks: the group had a job)
      if (marks)
        for (int k = 0; k < kBadWords; ++k) any_bad |= bad[k];
#pragma unroll 1
      for (int h = 0; h < 4; ++h) {
        float o[32];
        if (jobs > 0) {
          tc::tmem_ld32(o_at + 32 * h, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        if (any_bad && write) {
          // rare: the rows that were blanked, for the queries that see them, where the steps of this
          // part (of this group) hold them
#pragma unroll 1
          for (int k = 0; k < 32 * kBadWords; ++k) {
            const int tok = first + k;
            if (!((bad[k >> 5] >> (k & 31)) & 1) || tok < 0 || tok > limit) continue;
            const int step = part.pre_steps + tok / kWideTokens - at.step;
            if (step < 0 || step >= part.steps || !part.has(w, step)) continue;
            const int page = p.table[(long long)(at.k.s - set.prefixes) * p.table_stride + (tok >> p.page_shift)];
            const long long e = (long long)page * p.page_stride +
                                (((long long)at.h << p.page_shift) + (tok & ((1 << p.page_shift) - 1))) * kHeadDim;
            const __nv_bfloat16* kr = static_cast<const __nv_bfloat16*>(p.page_k) + e;
            const __nv_bfloat16* vr = static_cast<const __nv_bfloat16*>(p.page_v) + e + 32 * h;
            const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + (long long)mine.b * p.qb +
                                      (long long)hq * p.qh + (long long)mine.t * p.qm;
            float z = 0.f;
#pragma unroll 1
            for (int d = 0; d < kHeadDim; ++d) z += __bfloat162float(qr[d]) * __bfloat162float(kr[d]);
            const float wt = ex2(z * p.scale2 - base_of(ref));
#pragma unroll
            for (int d = 0; d < 32; ++d) o[d] += wt * __bfloat162float(vr[d]);
          }
        }
        if (!write) continue;
        if (whole) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + (long long)mine.b * p.ob + (long long)hq * p.oh +
                               (long long)mine.t * p.om + 32 * h;
          uint32_t y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
          if (p.out_sectors) {
            store_sector(dst, y);
            store_sector(dst + 16, y + 8);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              reinterpret_cast<uint4*>(dst)[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
          }
        } else {
          float* dst = set.part_o + prow * kHeadDim + 32 * h;
#pragma unroll
          for (int k = 0; k < 4; ++k) store_sector(dst + 8 * k, reinterpret_cast<const uint32_t*>(o) + 8 * k);
        }
      }
      if (write) {
        if (!whole) {
          set.part_ml[prow] = make_float2(ref, sum);
        } else if (p.lse) {
          p.lse[((long long)mine.b * p.hq + hq) * p.m + mine.t] =
              sees ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
        }
      }
    }
    if (!more) break;

    limit = q.real ? c.k.len - c.k.n + q.t : -1;
    ref = q.real ? -INFINITY : 0.f;               // rows without a query never wait for a maximum
    sum = 0.f;
    marks = false;
    bool begun = false;
    const int first = p.m > 1 && c.k.reach >= 0 ? first_marked(p, c) : 1 << 30;
    if (g.jobs(w) > 0) {
      ++turn;
      if (row < kBadWords) sh.bad[w][(turn + 2) & (kBadSets - 1)][row] = 0;
    }
    uint32_t* bad = sh.bad[w][turn & (kBadSets - 1)];
#pragma unroll 1
    for (int i = 0; i < g.steps; ++i) {
      slot.next();                                // the step's V
      const int v_slot = slot.i;
      const uint32_t v_parity = slot.parity;
      slot.next();
      if (!g.has(w, i)) continue;
      const int own0 = (c.step + i - g.pre_steps) * kWideTokens;
      const int seen = own0 < 0 ? c.k.pre - 1 - (c.step + i) * kWideTokens : limit - own0;   // columns 0 .. seen
      const bool masked = __any_sync(0xffffffffu, seen < kTile - 1);
      // 32 columns at a time; the next ones of the half step are on their way while these are at work
      float x[2][32];
      auto chunk = [&](uint32_t at, int ch, int from, float(&y)[32], float(&next)[32]) {
        wait32(y);
        if (ch == 0) load32(at + 32, next);
        if (masked) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (from + k > seen) y[k] = -INFINITY;
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
          if (again || !__any_sync(0xffffffffu, ref == -INFINITY || !(got < kMoveAbove))) break;
          if (ch == 0) wait32(next);              // no call while a load is on its way to registers
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < 32; k += 2) top = fmax3(top, y[k], y[k + 1]);
          const float to = fmaxf(ref, top * scale), f = weight_of(ref, to);
          ref = to;
          sum *= f;
          // O follows once the products before this half step are through
          if (begun) wait_products(from / kHalf);
          move_reference(at, 16 * ch, begun ? o_at : 0, f);
        }
        sum += got;
        store16(at + 16 * ch, pk);                // over columns that are in registers by now
      };
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = s_at + h * kHalf;
        if (!wait(&sh.s_full[w][h], s_parity)) break;
        load32(at, x[0]);
        chunk(at, 0, h * kHalf, x[0], x[1]);
        chunk(at, 1, h * kHalf + 32, x[1], x[0]);
        if (h == 0 && own0 >= 0 && (own0 + kTile - 1 > c.k.reach || own0 + kTile > first)) {
          if (!wait(&sh.kv_full[v_slot], v_parity)) break;
          blank_rows(v_slot, own0, first, bad);
          marks = marks || own0 + kTile > first;
        }
        wait_stores();
        tc::fence_before_sync();
        __syncwarp();
        if ((row & 31) == 0) tc::mbar_arrive(&sh.p_full[w][h]);   // a warp's 32 arrivals would go one by one
        begun = true;
      }
      if (!ok) break;
      s_parity ^= 1;
    }
    if (!ok) break;
  }
}

// Before the totals are known: tensor memory, barriers. The whole CTA.
__device__ __forceinline__ void wide_setup(WideShared& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == 0) tc::tmem_alloc(&sh.tmem_base, 4 * kTile);
  if (warp == 1 && lane < kRing) {
    tc::mbar_init(&sh.kv_full[lane], 1);
    tc::mbar_init(&sh.kv_empty[lane], 2);         // both groups' MMA warps
  }
  if (warp == 2 && lane < 2) {
    tc::mbar_init(&sh.q_full[lane], kTile / 32);
    for (int h = 0; h < 2; ++h) {
      tc::mbar_init(&sh.s_full[lane][h], 1);
      tc::mbar_init(&sh.p_full[lane][h], kTile / 32);
      tc::mbar_init(&sh.o_full[lane][h], 1);
    }
    tc::mbar_init(&sh.done[lane], 1);
  }
  if (warp > 3) {
    for (int i = tid - 128; i < 2 * kBadSets * kBadWords; i += blockDim.x - 128) (&sh.bad[0][0][0])[i] = 0;
    if (tid == 128) sh.fail = 0;
  }
}
__device__ __forceinline__ void wide_teardown(const WideShared& sh) {
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (threadIdx.x < 32) tc::tmem_dealloc(sh.tmem_base, 4 * kTile);
}

// The wide kernel's part of a CTA: `count` steps from where its share begins.
__device__ __forceinline__ void wide_rows(const AttendParams& p, WideShared& sh, const ScanShared& scan, int count,
                                          unsigned char* qbuf) {
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t q_at = tc::smem_u32(qbuf), ring = q_at + 2 * kTileBytes, tmem = sh.tmem_base;
  WideCursor c = place<kWideRows, kWideTokens>(p, p.wide, scan.e[0], scan.rest[0]);
  c.settle(count);
  if (warp == kTmaWarp) {
    producer(p, sh, c, count, ring);
  } else if (warp >= kMmaWarp && warp < kTmaWarp) {
    if ((tid & 31) == 0) mma_issuer(p, sh, c, count, warp - kMmaWarp, tmem, q_at, ring);
    __syncwarp();
  } else if (warp < kMmaWarp) {
    softmax_group(p, sh, c, count, warp >> 2, tid & (kTile - 1), tmem, qbuf, ring);
  }
}

}  // namespace
}  // namespace evict
