// Attention of many query rows over a shared prefix or a sequence's rows
// (see attend.cu for the operator and the other kernels): tcgen05 tensor cores.
//
// attend_wide_kernel: persistent, one CTA of eleven warps per SM. A unit is a
// (stream, KV head, tile of 256 query rows); K and V stream through a ring of
// five 32 KB tiles of 128 rows (TMA). Warps 0-3 and 4-7 are two softmax
// groups, a thread per query row, each with its own 128 x 128 logits and
// 128 x 128 output accumulator in tensor memory (512 columns in all); warp 8
// issues the MMAs, warp 9 the TMA loads. A "job" is one group's work on one
// step:
//     S = Q K^T (MMA) -> P = 2^(S scale - ref) as bf16 over S in tensor memory
//     (softmax group) -> O += P V (MMA, P read from tensor memory).
// The tensor cores work on one group's job while the other group exponentiates.
// A unit of more than 128 rows gives each group 128 rows and both groups every
// step; a smaller one gives both the same rows and every other step each (two
// partial results).
//
// The exponent's reference is the running maximum where it was last moved: it
// moves only when a row's maximum passes it by more than 2^32, which costs the
// group a read and write of its O in tensor memory (in practice only a unit's
// first step moves it). Weights, sums and O are relative to it and floating, so
// the result does not depend on where it stands. Weights enter the product
// with V as bf16 (half a step: 2^-9 of a weight), at twice the rate of the
// split that the few-row kernel uses; their roundings are independent, so the
// output's error grows from one rounding to the root of two.
//
// Bound: the tensor cores (2 x 512 clocks a job) with many rows, HBM with few.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attend.cuh"
#include "attend.h"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "tcgen05.cuh"

namespace evict {
namespace {

constexpr int kTile = 128;
constexpr int kTileBytes = kTile * kHeadDim * 2;
constexpr int kRing = 5;
constexpr int kWideThreads = 11 * 32;
constexpr int kWideSmem = (2 + kRing) * kTileBytes + 1024;
constexpr int kMmaWarp = 8, kTmaWarp = 10;
constexpr int kBadWords = 9;                      // 257 tokens and more
constexpr float kRefSlack = 32.f;                 // log2 of the largest weight

struct WideShared {
  uint64_t kv_full[kRing], kv_empty[kRing];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], done[2];
  uint32_t tmem_base;
  int fail;
  uint32_t bad[2][2][kBadWords];                  // [group][segment parity]
  ScanShared scan;
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
    alt = !two && !p.set.joint;
  }
  __device__ __forceinline__ bool has(int w, int i) const { return two || (alt ? (i & 1) == w : w == 0); }
  __device__ __forceinline__ int jobs(int w) const { return two ? steps : alt ? (steps + 1 - w) / 2 : w == 0 ? steps : 0; }
};

// The unit's first query sees own rows before this one; from here to the last query's, rows with
// infinities or NaN in V are marked (at most 256 tokens).
__device__ __forceinline__ int first_marked(const AttendParams& p, const WideCursor& c) {
  return c.k.len - c.k.n + (c.k.tile * kWideRows) / p.group + 1;
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
  const WorkSet& set = p.set;
  const int lane = threadIdx.x & 31, blocks = set.blocks();
  const int box = p.box_rows, boxes = box ? kTile / box : 0;
  Slot slot;
  int used = 0;
  bool ok = true;
  while (ok) {
    const Segment g(p, c, count);
    const int plane = c.k.s < set.prefixes ? c.k.s : p.fan ? (c.k.s - set.prefixes) / p.fan : 0;
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
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, kTileBytes);
        __syncwarp();
        if (pre) {
          if (lane < 2)
            tma_load_5d(dst + lane * (kTileBytes / 2), kv ? &p.tm_pv : &p.tm_pk, 0, row0, lane, c.h, plane, bar);
        } else if (lane < boxes) {
          for (int hf = 0; hf < 2; ++hf)
            tma_load_5d(dst + hf * (kTileBytes / 2) + lane * box * 128, kv ? &p.tm_v : &p.tm_k, 0,
                        row & ((1 << p.page_shift) - 1), hf, c.h, page, bar);
        }
        slot.next();
        ++used;
      }
    }
    count -= g.steps;
    if (count == 0) break;
    c.next_unit(p, set, blocks);
  }
  // every copy issued must land before the CTA may release its shared memory
  for (int i = 0; i < kRing && i < used; ++i) drain_phase(&sh.kv_full[i], ((used - 1 - i) / kRing) & 1, p.err);
}

__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) { return (uint64_t)lo | ((uint64_t)hi << 32); }

// S = Q K^T, both K-major; q and k: the tiles' descriptors' low words (their steps differ in the
// start address alone, which does not carry over).
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t q, uint32_t k, uint32_t hi) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, kTile);
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const uint32_t off = (uint32_t)((s >> 2) * kTile * 128 + (s & 3) * 32) >> 4;
    tc::mma_bf16(d, desc_of(q + off, hi), desc_of(k + off, hi), idesc, s > 0 ? 1u : 0u);
  }
}
// O (+)= P V: P in tensor memory (two weights a column), V with its rows as the product's
// depth (MN-major). 16 rows of V are 2048 bytes of each half.
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t pt, uint32_t v, uint32_t hi, bool accumulate) {
  constexpr uint32_t idesc = tc::idesc_bf16_f32(kTile, kTile) | (1u << 16);
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(pt + s * 8), "l"(desc_of(v + s * 128, hi)), "r"(idesc), "r"(accumulate || s > 0 ? 1u : 0u)
        : "memory");
  }
}

// The MMAs of group w, issued by one warp of its own: S = Q K^T of a step as soon as the product
// with V of the step before has been issued (it reads the weights that lie where S goes; MMAs run
// in order), then, with the group's weights, that step's product with V.
__device__ void mma_issuer(const AttendParams& p, WideShared& sh, WideCursor c, int count, int w, uint32_t tmem,
                           uint32_t qbuf, uint32_t ring) {
  const WorkSet& set = p.set;
  const int lane = threadIdx.x & 31, blocks = set.blocks();
  const uint64_t qk = tc::sw128_desc(qbuf + w * kTileBytes), pv = tc::sw128_desc_mn(ring, kTileBytes / 2, 1024);
  const uint32_t q_lo = (uint32_t)qk, k_lo = (uint32_t)tc::sw128_desc(ring), qk_hi = (uint32_t)(qk >> 32);
  const uint32_t v_lo = (uint32_t)pv, v_hi = (uint32_t)(pv >> 32);
  const uint32_t s_at = tmem + w * kTile, o_at = s_at + 2 * kTile;
  uint32_t p_parity = 0, q_parity = 0;
  Slot slot;
  int segment = 0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    ok = wait_phase(bar, parity, &sh.fail, p.err);
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  while (ok) {
    const Segment g(p, c, count);
    const int jobs = g.jobs(w);
    if (jobs > 0) {
      if (!wait(&sh.q_full[w], q_parity)) break;
      q_parity ^= 1;
    }
    int done = 0;
#pragma unroll 1
    for (int i = 0; i < g.steps; ++i) {
      if (!g.has(w, i)) {                         // the other group's step: this one lets go of its tiles
#pragma unroll 1
        for (int kv = 0; kv < 2 && wait(&sh.kv_full[slot.i], slot.parity); ++kv, slot.next())
          if (lane == 0) tc::mbar_arrive(&sh.kv_empty[slot.i]);
        if (!ok) break;
        continue;
      }
      if (!wait(&sh.kv_full[slot.i], slot.parity)) break;
      tc::fence_after_sync();
      if (lane == 0) {
        issue_qk(s_at, q_lo, k_lo + slot.i * (kTileBytes >> 4), qk_hi);
        tc::mma_commit(&sh.s_full[w]);
        tc::mma_commit(&sh.kv_empty[slot.i]);
      }
      __syncwarp();
      slot.next();
      if (!wait(&sh.kv_full[slot.i], slot.parity)) break;
      const int own0 = (c.step + i - g.pre_steps) * kWideTokens;           // < 0: rows of the prefix
      if (own0 >= 0) {
        // rows that no query of the unit sees, and rows with infinities or NaN that some queries do
        // not see, meet weights of 0: zeros in their place (both groups' warps write the same zeros)
        const uint32_t at = ring + slot.i * kTileBytes + ((lane >> 3) & 1) * (kTileBytes / 2) + (lane & 7) * 16;
        auto blank = [&](int r) {
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + r * 128), "r"(0u) : "memory");
        };
        bool wrote = false;
#pragma unroll 1
        for (int r = max(0, c.k.reach + 1 - own0) + (lane >> 4); r < kTile; r += 2) blank(r), wrote = true;
        const int mark0 = p.m > 1 && c.k.reach >= 0 ? first_marked(p, c) - own0 : kTile;
        if (mark0 < kTile) {
          const uint32_t* bad = sh.bad[w][segment & 1];
          uint32_t any = 0;
          for (int k = 0; k < kBadWords; ++k) any |= bad[k];
          if (any) {
            wrote = true;
#pragma unroll 1
            for (int k = max(0, -mark0); k < 32 * kBadWords && mark0 + k < kTile; ++k)
              if ((bad[k >> 5] >> (k & 31)) & 1) blank(mark0 + k);
          }
        }
        if (__any_sync(0xffffffffu, wrote)) tc::fence_proxy_async_smem();
        __syncwarp();
      }
      if (!wait(&sh.p_full[w], p_parity)) break;
      p_parity ^= 1;
      tc::fence_after_sync();
      ++done;
      if (lane == 0) {
        issue_pv(o_at, s_at, v_lo + slot.i * (kTileBytes >> 4), v_hi, done > 1);
        tc::mma_commit(&sh.kv_empty[slot.i]);
        if (done == jobs) tc::mma_commit(&sh.o_full[w]);
      }
      __syncwarp();
      slot.next();
    }
    ++segment;
    count -= g.steps;
    if (count == 0) break;
    c.next_unit(p, set, blocks);
  }
  // every MMA must finish before tensor and shared memory are released
  if (lane == 0) {
    tc::mma_commit(&sh.done[w]);
    drain_phase(&sh.done[w], 0, p.err);
  }
  __syncwarp();
}

// 64 columns of this thread's row; the load and its wait are one statement, so that nothing uses
// the registers before the data is there.
__device__ __forceinline__ void load64(uint32_t taddr, float* v) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void store32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One softmax group: thread `row` of group w.
__device__ void softmax_group(const AttendParams& p, WideShared& sh, WideCursor c, int count, int w, int row, uint32_t tmem,
                              unsigned char* qbuf) {
  const WorkSet& set = p.set;
  const int warp = row >> 5, blocks = set.blocks();
  const uint32_t lanes = (uint32_t)(32 * warp) << 16;
  const uint32_t s_at = tmem + lanes + (uint32_t)(w * kTile), o_at = s_at + 2 * kTile;
  const uint32_t flip = p.scale2 < 0.f ? 0x80008000u : 0u;   // a negative scale: of -Q, so that maxima stay maxima
  const float scale = fabsf(p.scale2);
  unsigned char* q_mine = qbuf + w * kTileBytes;

  // this row's query into the group's tile, and which rows with infinities or NaN in V some
  // queries of the unit do not see
  auto load_query = [&](const WideCursor& cu, const Segment& g, int segment) {
    const QueryRow q = query_row<kWideRows>(p, set, cu.k, g.two ? w * kTile + row : row);
    // A group without a job in this part announces nothing (it could announce twice before the
    // MMA warp has looked once).
    if (g.jobs(w) == 0) return q;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (long long)q.b * p.qb +
                                                      (long long)(cu.h * p.group + q.g) * p.qh + (long long)q.t * p.qm);
    uint4 x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = q.real ? src[j] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      x[j].x ^= flip, x[j].y ^= flip, x[j].z ^= flip, x[j].w ^= flip;
      *reinterpret_cast<uint4*>(q_mine + tc::sw128_offset(row, j, kTile)) = x[j];
    }
    if (p.m > 1 && cu.k.reach >= 0) {
      const int first = first_marked(p, cu);
      uint32_t* bad = sh.bad[w][segment & 1];
      if (row < kBadWords) bad[row] = 0;
      tc::named_sync(1 + w, kTile);
      const int32_t* table = p.table + (long long)(cu.k.s - set.prefixes) * p.table_stride;
#pragma unroll 1
      for (int e = row; e < 16 * (cu.k.reach + 1 - first); e += kTile) {
        const int tok = first + (e >> 4);
        if (tok < 0) continue;
        const int page = table[tok >> p.page_shift];
        if (page < 0 || page >= p.n_pages) continue;
        const uint4 v = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.page_v) +
                                                       (long long)page * p.page_stride +
                                                       (((long long)cu.h << p.page_shift) +
                                                        (tok & ((1 << p.page_shift) - 1))) * kHeadDim)[e & 15];
        if (nonfinite2(v.x) | nonfinite2(v.y) | nonfinite2(v.z) | nonfinite2(v.w))
          atomicOr(&bad[(tok - first) >> 5], 1u << ((tok - first) & 31));
      }
    }
    tc::fence_proxy_async_smem();
    tc::mbar_arrive(&sh.q_full[w]);
    return q;
  };

  uint32_t s_parity = 0, o_parity = 0;
  int segment = 0;
  bool ok = true;
  Segment g(p, c, count);
  QueryRow q = load_query(c, g, 0);
  for (;;) {
    const int jobs = g.jobs(w);
    const int limit = q.real ? c.k.len - c.k.n + q.t : -1;       // last own row that this query sees
    float ref = -INFINITY, sum = 0.f;
    bool begun = false;
#pragma unroll 1
    for (int i = 0; i < g.steps && ok; ++i) {
      if (!g.has(w, i)) continue;
      ok = wait_phase(&sh.s_full[w], s_parity, &sh.fail, p.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      s_parity ^= 1;
      tc::fence_after_sync();
      const int own0 = (c.step + i - g.pre_steps) * kWideTokens;
      const int seen = own0 < 0 ? c.k.pre - 1 - (c.step + i) * kWideTokens : limit - own0;   // columns 0 .. seen
      const bool masked = __any_sync(0xffffffffu, seen < kTile - 1);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {      // 64 columns at a time: their registers are few enough
        float v[64];
        load64(s_at + 64 * half, v);
        if (masked) {
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (64 * half + k > seen) v[k] = -INFINITY;
        }
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmax3(v[j], v[j + 4], v[j + 8]);
#pragma unroll
        for (int k = 12; k < 60; k += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = fmax3(mx[j], v[k + j], v[k + 4 + j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], v[60 + j]);
        const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * scale;
        if (__any_sync(0xffffffffu, top > ref + kRefSlack)) {         // also from no reference to the first
          const float to = fmaxf(ref, top), f = weight_of(ref, to);
          ref = to;
          sum *= f;
          if (begun) {
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
              float o[32];
              tc::tmem_ld32(o_at + 32 * h, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= f;
              store32(o_at + 32 * h, reinterpret_cast<const uint32_t*>(o));
            }
          }
          if (half == 1) {                        // the first half's weights, too
            float o[32];
            wait_stores();
            tc::tmem_ld32(s_at, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t x = __float_as_uint(o[k]);
              o[k] = __uint_as_float(pack_bf16(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f));
            }
            store32(s_at, reinterpret_cast<const uint32_t*>(o));
          }
        }
        const float base = base_of(ref);
        const uint64_t sc2 = pack_f32x2(scale, scale), nb2 = pack_f32x2(-base, -base);
        uint64_t acc[2] = {0ull, 0ull};
        uint32_t pk[32];
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          const uint64_t e = ex2_f32x2(fma_f32x2(pack_f32x2(v[k], v[k + 1]), sc2, nb2));
          acc[(k >> 1) & 1] = add_f32x2(acc[(k >> 1) & 1], e);
          float a, b;
          split_f32x2(e, a, b);
          pk[k >> 1] = pack_bf16(a, b);
        }
        // over columns that are in registers by now: half 0 over 0 .. 31, half 1 over 32 .. 63
        store32(s_at + 32 * half, pk);
        float a0, a1;
        split_f32x2(add_f32x2(acc[0], acc[1]), a0, a1);
        sum += a0 + a1;
      }
      begun = true;
      wait_stores();
      tc::fence_before_sync();
      tc::mbar_arrive(&sh.p_full[w]);
    }
    // the next unit's queries: this group's last S is in registers, so its tile is free
    const WideCursor at = c;
    const Segment part = g;
    const QueryRow mine = q;
    count -= g.steps;
    if (count > 0 && ok) {
      c.next_unit(p, set, blocks);
      g = Segment(p, c, count);
      q = load_query(c, g, segment + 1);
    }
    if (ok && jobs > 0) {
      ok = wait_phase(&sh.o_full[w], o_parity, &sh.fail, p.err);
      ok = __all_sync(0xffffffffu, ok);
      o_parity ^= 1;
    }
    if (!ok) break;
    tc::fence_after_sync();
    const bool whole = set.joint && part.steps == at.k.steps;     // no other part, no other unit for these rows
    const bool write = mine.real && (part.two || part.alt || w == 0);
    const size_t prow = (size_t)(at.unit + blockIdx.x) * kWideRows + w * kTile + row;
    const bool sees = at.k.pre > 0 || limit >= 0;
    const int hq = at.h * p.group + mine.g;
    const float inv = sees ? 1.f / sum : 0.f;
    uint32_t any_bad = 0;
    const int first = first_marked(p, at);
    const uint32_t* bad = sh.bad[w][segment & 1];
    if (p.m > 1 && at.k.reach >= 0 && jobs > 0)
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
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (long long)mine.b * p.ob +
                                              (long long)hq * p.oh + (long long)mine.t * p.om + 32 * h);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          dst[k] = make_uint4(pack_bf16(o[8 * k] * inv, o[8 * k + 1] * inv), pack_bf16(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                              pack_bf16(o[8 * k + 4] * inv, o[8 * k + 5] * inv), pack_bf16(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
      } else {
        float4* dst = reinterpret_cast<float4*>(set.part_o + prow * kHeadDim + 32 * h);
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
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
    ++segment;
    if (count == 0) break;
  }
}

__global__ void __launch_bounds__(kWideThreads, 1) attend_wide_kernel(const __grid_constant__ AttendParams p, int early) {
  pdl_wait();
  // what comes next may start on an SM as soon as this kernel leaves it
  if (early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ WideShared sh;
  const int tid = threadIdx.x, warp = tid >> 5;
  unsigned char* qbuf = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const uint32_t q_at = tc::smem_u32(qbuf), ring = q_at + 2 * kTileBytes;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(&sh.kv_full[i], 1);
      tc::mbar_init(&sh.kv_empty[i], 2);          // both groups' MMA warps
    }
    for (int w = 0; w < 2; ++w) {
      tc::mbar_init(&sh.q_full[w], kTile);
      tc::mbar_init(&sh.s_full[w], 1);
      tc::mbar_init(&sh.p_full[w], kTile);
      tc::mbar_init(&sh.o_full[w], 1);
      tc::mbar_init(&sh.done[w], 1);
    }
    sh.fail = 0;
  }
  const Shares shares = find_shares<kWideRows, kWideTokens, kWideThreads, 1>(p, p.set, sh.scan);
  if ((int)blockIdx.x >= shares.count) return;
  const int count = shares.begin(blockIdx.x + 1) - shares.begin(blockIdx.x);
  const WideCursor c = place<kWideRows, kWideTokens>(p, p.set, sh.scan.e[0], sh.scan.rest[0]);
  if (warp == 0) tc::tmem_alloc(&sh.tmem_base, 4 * kTile);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem_base;
  if (warp == kTmaWarp) producer(p, sh, c, count, ring);
  else if (warp >= kMmaWarp) mma_issuer(p, sh, c, count, warp - kMmaWarp, tmem, q_at, ring);
  else softmax_group(p, sh, c, count, warp >> 2, tid & (kTile - 1), tmem, qbuf);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, 4 * kTile);
}

}  // namespace

cudaError_t prepare_wide() {
  return cudaFuncSetAttribute(attend_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem);
}

// early: the next kernel in the stream waits for this one by itself (late_wait).
cudaError_t launch_wide(const AttendParams& p, int ctas, bool early, cudaStream_t st) {
  return launch_pdl(attend_wide_kernel, dim3(ctas), dim3(kWideThreads), kWideSmem, st, nullptr, p, early ? 1 : 0);
}

}  // namespace evict
