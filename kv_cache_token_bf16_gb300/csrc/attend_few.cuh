// Attention of up to 16 query rows over a shared prefix or a sequence's rows (see attend.cu): warps
// that work by themselves, on m16n8k16 products.
//
// A warp takes an equal share of the boxes of 16 rows of K and V that all such units read, whatever
// the sequences' lengths are, with its own ring of TMA boxes (16 rows of K and of V, 8 KB; a box
// never crosses a page), its own running maximum, sum and output, and no barrier, so that one warp's
// start or end of a unit hides behind the others' rows. Queries are the products' rows. Bound: HBM;
// a warp has one box in flight while it computes on another (96 KB an SM).
//
// Measured: 16 sequences of 16,384 own rows with 4 query rows a KV head (1.07 GB) 174 us, 6.2 TB/s;
// 32 sequences of 4,096 rows 95 us, 5.7; of 1,024 rows 33 us, 4.0: 11 us of a call are its start and
// the join. The split of the weights into hi + lo costs no time there and keeps the output's error
// that of one rounding (each weight within 2^-15).
#pragma once

#include <cuda_bf16.h>

#include "attend.cuh"

namespace evict {
namespace {

constexpr int kBoxBytes = kBoxTokens * kHeadDim * 2;       // of K or of V

constexpr int kRows = kFewRows;
constexpr int kWarps = 12;
constexpr int kStages = 2;                        // boxes of a warp's ring
constexpr int kFewSmem = kWarps * kStages * 2 * kBoxBytes;

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
  int fail;
};

__device__ __forceinline__ void few_setup(FewShared& sh) {
  const int tid = threadIdx.x;
  if (tid < kWarps * kStages) tc::mbar_init(&sh.full[tid / kStages][tid % kStages], 1);
  if (tid == 0) sh.fail = 0;
}

// The few-row kernel's part of a CTA: a share for each of its warps; ring0: 1024-byte aligned.
__device__ __forceinline__ void few_rows(const AttendParams& p, FewShared& sh, const ScanShared& scan, const Place& at,
                                         uint32_t ring0) {
  using Cur = Cursor<kRows, kBoxTokens>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = ring0 + warp * kStages * 2 * kBoxBytes;
  const WorkSet& set = p.few;
  const int blocks = set.blocks();
  const Shares& shares = at.shares;
  const int share = at.first + warp * at.stride;
  if (share < shares.count) {
    int left = shares.begin(share + 1) - shares.begin(share);
    Cur cur = place<kRows, kBoxTokens>(p, set, scan.e[warp], scan.rest[warp]);
    cur.settle(left);

    // --- the ring: boxes are requested in the order in which they are used ---
    Cur ahead = cur;
    int ahead_left = left, page = 0;
    auto look_up = [&] {                          // the page of the next box to request
      if (lane == 0 && ahead_left > 0 && ahead.k.s >= set.prefixes)
        page = p.table[(long long)(ahead.k.s - set.prefixes) * p.table_stride + ((ahead.step * kBoxTokens) >> p.page_shift)];
    };
    auto request = [&](int stage) {
      if (lane == 0) {
        uint64_t* bar = &sh.full[warp][stage];
        const uint32_t dst = ring + stage * 2 * kBoxBytes;
        int row = ahead.step * kBoxTokens, plane = ahead.k.s;
        const bool pre = ahead.k.s < set.prefixes;
        if (!pre) {
          if (page < 0 || page >= p.n_pages) {
            raise_device_error(p.err, kDevBadIndex);
            page = p.n_pages;                     // outside the pool: the box is zeros
          }
          plane = page;
          row &= (1 << p.page_shift) - 1;
        }
        tc::mbar_arrive_expect_tx(bar, 2 * kBoxBytes);
        tma_load_5d(dst, pre ? &p.few_pre[0] : &p.few_own[0], 0, row, 0, ahead.h, plane, bar);
        tma_load_5d(dst + kBoxBytes, pre ? &p.few_pre[1] : &p.few_own[1], 0, row, 0, ahead.h, plane, bar);
      }
      if (--ahead_left > 0 && ++ahead.step == ahead.k.steps) {
        ahead.next_unit(p, set, blocks);
        ahead.settle(ahead_left);
      }
      look_up();
    };
    look_up();
    int requested = 0, flying = 0;                // the stage that the next request takes; boxes in the ring

    // addresses of this lane's rows for ldmatrix: 16-byte chunk j of a row sits at j ^ (row % 8), so a
    // chunk's address is the lane's own xor 16 j (and 2 KB on for the second half)
    const uint32_t k_at = tc::sw128_offset((lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1, kBoxTokens);
    const uint32_t v_at = kBoxBytes + tc::sw128_offset(lane & 15, lane >> 4, kBoxTokens);
    int stage = 0;
    uint32_t parity = 0;
    bool dead = false;

    while (left > 0) {
      const int boxes = min(cur.k.steps - cur.step, left);
      const bool own = cur.k.s >= set.prefixes;
      // this lane's queries (rows lane / 4 and 8 on) and the last row each sees
      uint32_t q[8][4];
      float o[16][4], mx[2], sum[2];
      int last[2], low = 0;

#pragma unroll 1
      for (int i = 0; i < boxes; ++i) {
        __syncwarp();                             // every lane has read the box that the next one replaces
        // a unit's queries pass through a stage before the last box is requested
#pragma unroll 1
        for (int room = i == 0 ? kStages - 1 : kStages; room <= kStages; ++room) {
#pragma unroll 1
          while (flying < room && ahead_left > 0 && !dead) {
            request(requested);
            requested = requested == kStages - 1 ? 0 : requested + 1;
            ++flying;
          }
          if (room == kStages) break;
          const uint32_t at = ring + requested * 2 * kBoxBytes;
          // two rows at a time, half a warp on each; lanes l and l + 16 know where row l is
          const QueryRow r = query_row<kRows>(p, set, cur.k, lane & 15);
          const long long mine =
              r.real ? (long long)r.b * p.qb + (long long)(cur.h * p.group + r.g) * p.qh + (long long)r.t * p.qm : -1;
          uint4 x[kRows / 2];
#pragma unroll
          for (int e = 0; e < kRows / 2; ++e) {
            const long long from = __shfl_sync(0xffffffffu, mine, 2 * e + (lane >> 4));
            x[e] = make_uint4(0, 0, 0, 0);
            if (from >= 0) x[e] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + from)[lane & 15];
          }
#pragma unroll
          for (int e = 0; e < kRows / 2; ++e)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};"
                         ::"r"(at + tc::sw128_offset(2 * e + (lane >> 4), lane & 15, kRows)),
                         "r"(x[e].x), "r"(x[e].y), "r"(x[e].z), "r"(x[e].w) : "memory");
          __syncwarp();
          const uint32_t q_at = at + tc::sw128_offset(lane & 15, lane >> 4, kRows);
#pragma unroll
          for (int s = 0; s < 8; ++s) ldsm4((q_at ^ ((s & 3) * 32)) + (s >> 2) * (kRows * 128), q[s]);
          tc::fence_proxy_async_smem();           // the stage's next content comes by TMA
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = p.by_group.div(cur.k.tile * kRows + (lane >> 2) + 8 * k);
            last[k] = !own ? cur.k.pre - 1 : t < cur.k.n ? cur.k.len - cur.k.n + t : -1;
            mx[k] = -INFINITY;
            sum[k] = 0.f;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
          low = __shfl_sync(0xffffffffu, last[0], 0);              // the first row's: the lowest
          __syncwarp();
        }
        if (!dead) {
          const bool ok = wait_phase(&sh.full[warp][stage], parity, &sh.fail, p.err);
          if (!__all_sync(0xffffffffu, ok)) {
            // the copies in flight must land before this CTA may end
            for (int w = 0, s = stage; w < flying; ++w) {
              drain_phase(&sh.full[warp][s], s >= stage ? parity : parity ^ 1, p.err);
              s = s == kStages - 1 ? 0 : s + 1;
            }
            dead = true;
          }
        }
        const uint32_t kb = ring + stage * 2 * kBoxBytes;
        if (++stage == kStages) stage = 0, parity ^= 1;
        --flying;
        const int row0 = (cur.step + i) * kBoxTokens;
        if (dead) continue;

        const bool full = row0 + kBoxTokens - 1 <= low;            // every query sees every row
        float z[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[j][k] = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          uint32_t k4[4];
          ldsm4(((kb + k_at) ^ ((s & 3) * 32)) + (s >> 2) * (kBoxTokens * 128), k4);
          mma16816(z[0], q[s], k4[0], k4[1]);
          mma16816(z[1], q[s], k4[2], k4[3]);
        }
        float rm[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v = z[j][k] * p.scale2;
            if (!full && row0 + 8 * j + 2 * (lane & 3) + (k & 1) > last[k >> 1]) v = -INFINITY;
            z[j][k] = v;
            rm[k >> 1] = fmaxf(rm[k >> 1], v);
          }
        // the running maximum moves only when a logit passes it
        if (__any_sync(0xffffffffu, rm[0] > mx[0] || rm[1] > mx[1])) {
          float f[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            rm[k] = fmaxf(rm[k], __shfl_xor_sync(0xffffffffu, rm[k], 1));
            rm[k] = fmaxf(rm[k], __shfl_xor_sync(0xffffffffu, rm[k], 2));
            const float nm = fmaxf(mx[k], rm[k]);
            f[k] = weight_of(mx[k], nm);
            mx[k] = nm;
            sum[k] *= f[k];
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j][0] *= f[0];
            o[j][1] *= f[0];
            o[j][2] *= f[1];
            o[j][3] *= f[1];
          }
        }
        const float m0 = base_of(mx[0]), m1 = base_of(mx[1]);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int k = 0; k < 4; ++k) z[j][k] = ex2(z[j][k] - (k < 2 ? m0 : m1));
          sum[0] += z[j][0] + z[j][1];
          sum[1] += z[j][2] + z[j][3];
          // weights as bf16 pairs hi + lo, within 2^-15 of each, so that their rounding does not add to the
          // output's own (the tensor cores wait for memory here anyway). Both meet a V that may be infinite:
          // hi is cut off, not rounded, so that lo is not negative, and lo is 0 only where the weight is
          // (otherwise 2^-133 at least, bf16's least).
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float a = z[j][2 * k], b = z[j][2 * k + 1];
            const uint32_t h2 = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
            hi[2 * j + k] = h2;
            lo[2 * j + k] = __vmaxu2(pack_bf16(a - __uint_as_float(h2 << 16), b - __uint_as_float(h2 & 0xffff0000u)),
                                     __vminu2(h2, 0x00010001u));
          }
        }
        // V of rows behind the stream's end may hold anything: zeros in its place
        uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu, bad = 0;
        if (!full) {
          const int r0 = row0 + 2 * (lane & 3), end = own ? cur.k.len : cur.k.pre;
          auto mask = [&](int r) { return (r < end ? 0xffffu : 0u) | (r + 1 < end ? 0xffff0000u : 0u); };
          keep0 = mask(r0);
          keep1 = mask(r0 + 8);
          if (p.m > 1 && own) {
            // A query that does not see a row gives it weight 0, but 0 * infinity is not 0: the
            // products leave rows with infinities or NaN out (`bad`), and the queries that see them
            // take them afterwards.
#pragma unroll 1
            for (int j = 0; j < 8; ++j) {
              uint32_t v4[4];
              ldsm4_t(((kb + v_at) ^ ((j & 3) * 32)) + (j >> 2) * (kBoxTokens * 128), v4);
              const uint32_t odd0 = nonfinite2(v4[0] & keep0) | nonfinite2(v4[2] & keep0);
              const uint32_t odd1 = nonfinite2(v4[1] & keep1) | nonfinite2(v4[3] & keep1);
              bad |= (odd0 | odd1 << 8) << (2 * (lane & 3));
            }
            bad = __reduce_or_sync(0xffffffffu, bad);
            auto drop = [&](uint32_t two) { return (two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u); };
            keep0 &= ~drop(bad >> (2 * (lane & 3)));
            keep1 &= ~drop(bad >> (2 * (lane & 3) + 8));
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t v4[4];
          ldsm4_t(((kb + v_at) ^ ((j & 3) * 32)) + (j >> 2) * (kBoxTokens * 128), v4);
          if (!full) v4[0] &= keep0, v4[1] &= keep1, v4[2] &= keep0, v4[3] &= keep1;
          mma16816(o[2 * j], hi, v4[0], v4[1]);
          mma16816(o[2 * j + 1], hi, v4[2], v4[3]);
          mma16816(o[2 * j], lo, v4[0], v4[1]);
          mma16816(o[2 * j + 1], lo, v4[2], v4[3]);
        }
#pragma unroll 1
        for (; bad; bad &= bad - 1) {             // rare
          const int k = __ffs(bad) - 1, from = (lane & 28) | ((k & 7) >> 1);
          const float a0 = k & 1 ? z[0][1] : z[0][0], a1 = k & 1 ? z[1][1] : z[1][0];
          const float b0 = k & 1 ? z[0][3] : z[0][2], b1 = k & 1 ? z[1][3] : z[1][2];
          const float w0 = __shfl_sync(0xffffffffu, k & 8 ? a1 : a0, from);
          const float w1 = __shfl_sync(0xffffffffu, k & 8 ? b1 : b0, from);
          const bool s0 = row0 + k <= last[0], s1 = row0 + k <= last[1];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint32_t v;
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v)
                         : "r"(kb + kBoxBytes + tc::sw128_offset(k, j, kBoxTokens) + 4 * (lane & 3)) : "memory");
            const float v0 = __uint_as_float(v << 16), v1 = __uint_as_float(v & 0xffff0000u);
            if (s0) o[j][0] += w0 * v0, o[j][1] += w0 * v1;
            if (s1) o[j][2] += w1 * v0, o[j][3] += w1 * v1;
          }
        }
      }

      // --- the share leaves the unit: its part of the result ---
      const size_t slot = set.slot_row(cur.unit, share);
      const int rows = min(kRows, cur.k.n * p.group - cur.k.tile * kRows);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float t = sum[k];
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        const int r = (lane >> 2) + 8 * k;
        if (r < rows) {
          if ((lane & 3) == 0) set.part_ml[slot + r] = make_float2(mx[k], t);
          float2* dst = reinterpret_cast<float2*>(set.part_o + (slot + r) * kHeadDim) + (lane & 3);
#pragma unroll
          for (int j = 0; j < 16; ++j) dst[4 * j] = make_float2(o[j][2 * k], o[j][2 * k + 1]);
        }
      }
      left -= boxes;
      if (left > 0) {
        cur.next_unit(p, set, blocks);
        cur.settle(left);
      }
    }
  }
}

}  // namespace
}  // namespace evict
