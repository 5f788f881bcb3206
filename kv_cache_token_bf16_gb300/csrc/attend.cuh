// Device side of the attention kernels' schedule: streams, units, steps and
// the share of them that a CTA takes (see attend.h).
#pragma once

#include "attend.h"
#include "common.cuh"
#include "pipeline.cuh"
#include "tcgen05.cuh"

namespace evict {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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

// New rows and rows of a sequence, with what lies outside their bounds cut off (and reported).
struct Seq {
  int n, len;                        // new tokens; own rows, the new ones included
};
__device__ __forceinline__ Seq sequence(const AttendParams& p, int b, bool report) {
  int n = p.n_new ? p.n_new[b] : p.m;
  bool odd = n < 0 || n > p.m;
  n = n < 0 ? 0 : n > p.m ? p.m : n;
  int len = p.pages ? p.lens[b] : 0;
  const int room = p.pages ? p.table_width << p.page_shift : 0;
  odd = odd || len < 0 || len > room;
  len = len < 0 ? 0 : len > room ? room : len;
  if (odd && report) raise_device_error(p.err, kDevBadIndex);
  return {n, len};
}
// New tokens of the sequences before b. Padding is left out of a prefix's query rows.
__device__ __forceinline__ int tokens_before(const AttendParams& p, int b) {
  return p.n_new ? p.tok_base[b] : b * p.m;
}

template <int kRows>
struct Stream {
  int n, pre, len, tiles;            // query tokens, prefix rows, own rows, row tiles
  __device__ void load(const AttendParams& p, const StreamSet& set, int s, bool report = false) {
    if (s < set.prefixes) {
      n = tokens_before(p, (s + 1) * p.fan) - tokens_before(p, s * p.fan);
      pre = p.n_prefix;
      len = 0;
    } else {
      const Seq q = sequence(p, s - set.prefixes, report);
      n = q.n;
      len = q.len;
      pre = set.joint ? p.n_prefix : 0;
    }
    tiles = (int)(((long long)n * p.group + kRows - 1) / kRows);
  }
  __device__ int pre_steps() const { return (pre + kStepTokens - 1) / kStepTokens; }
  // Last own row that the tile's last token sees (-1: none).
  __device__ int reach(const AttendParams& p, int tile) const {
    if (len == 0) return -1;
    const long long t = ((long long)kRows * (tile + 1) - 1) / p.group;
    const int v = len - n + (int)(t < n - 1 ? t : n - 1);
    return v < -1 ? -1 : v;
  }
  __device__ int steps(const AttendParams& p, const StreamSet& set, int tile) const {
    const int k = pre_steps() + (reach(p, tile) + kStepTokens) / kStepTokens;
    return set.joint && k == 0 ? 1 : k;            // joint units write their rows themselves: all need a step
  }
  __device__ long long head_work(const AttendParams& p, const StreamSet& set) const {
    if (len == 0) return (long long)tiles * steps(p, set, 0);
    long long w = 0;
    for (int i = 0; i < tiles; ++i) w += steps(p, set, i);
    return w;
  }
};

// A position in the line of steps.
template <int kRows>
struct Cursor {
  int s, h, tile, step, steps;       // steps of the unit
  long long unit;
  Stream<kRows> st;
  __device__ void next(const AttendParams& p, const StreamSet& set) {
    if (++step < steps) return;
    step = 0;
    do {
      ++unit;
      if (++tile >= st.tiles) {
        tile = 0;
        if (++h >= p.hkv) {
          h = 0;
          do {
            if (++s >= set.prefixes + set.own) return;
            st.load(p, set, s);
          } while (st.tiles == 0);
        }
      }
      steps = st.steps(p, set, tile);
    } while (steps == 0);
  }
};

struct ScanShared {
  long long a[32], u[32];
  long long begin, rest, unit, total;
  int s;
};

// Exclusive sums of (a, u) over the block's threads, and the total of a.
template <int kThreads>
__device__ __forceinline__ void block_scan(long long& a, long long& u, long long& total, ScanShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long a0 = a, u0 = u;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, u, d);
    if (lane >= d) a += x, u += y;
  }
  if (lane == 31) sh.a[warp] = a, sh.u[warp] = u;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) a += sh.a[w], u += sh.u[w];
    total += sh.a[w];
  }
  a -= a0;
  u -= u0;
  __syncthreads();
}

// This CTA's share of the steps, found from the lengths on the device: `count` steps from `cur`.
// All threads call it; CTA 0 leaves the streams' first steps and units for the join.
template <int kRows, int kThreads>
__device__ __forceinline__ int find_share(const AttendParams& p, const StreamSet& set, ScanShared& sh,
                                          Cursor<kRows>& cur) {
  const int tid = threadIdx.x;
  long long a, u, total;
  if (p.n_new && p.fan) {
    // every CTA writes the same sums, and reads back its own
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    a = 0;
    u = 0;
    for (int b = b0; b < b1; ++b) a += sequence(p, b, false).n;
    block_scan<kThreads>(a, u, total, sh);
    for (int b = b0; b < b1; ++b) {
      p.tok_base[b] = (int)a;
      a += sequence(p, b, false).n;
    }
    if (tid == 0) p.tok_base[p.batch] = (int)total;
    __syncthreads();
  }
  const int streams = set.prefixes + set.own;
  const int per = (streams + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, streams), s1 = min(s0 + per, streams);
  Stream<kRows> st;
  a = 0;
  u = 0;
  for (int s = s0; s < s1; ++s) {
    st.load(p, set, s, blockIdx.x == 0);
    a += st.head_work(p, set) * p.hkv;
    u += (long long)st.tiles * p.hkv;
  }
  const long long mine_work = a;
  block_scan<kThreads>(a, u, total, sh);
  const long long ctas = total < set.ctas ? total : set.ctas;
  const long long begin = ctas ? total * blockIdx.x / ctas : 0;
  if (blockIdx.x == 0) {
    long long x = a, y = u;
    for (int s = s0; s < s1; ++s) {
      st.load(p, set, s);
      set.step_base[s] = x;
      set.unit_base[s] = y;
      x += st.head_work(p, set) * p.hkv;
      y += (long long)st.tiles * p.hkv;
    }
    if (tid == 0) set.step_base[streams] = total;
  }
  if (blockIdx.x < ctas && begin >= a && begin < a + mine_work) {
    int s = s0;
    for (; s < s1; ++s) {
      st.load(p, set, s);
      const long long w = st.head_work(p, set) * p.hkv;
      if (begin < a + w) break;
      a += w;
      u += (long long)st.tiles * p.hkv;
    }
    sh.s = s;
    sh.rest = begin - a;
    sh.unit = u;
    sh.begin = begin;
  }
  __syncthreads();
  if (blockIdx.x >= ctas) return 0;
  cur.s = sh.s;
  cur.st.load(p, set, cur.s);
  const long long per_head = cur.st.head_work(p, set);
  cur.h = (int)(sh.rest / per_head);
  long long r = sh.rest - cur.h * per_head;
  cur.tile = 0;
  for (;; ++cur.tile) {
    cur.steps = cur.st.steps(p, set, cur.tile);
    if (r < cur.steps) break;
    r -= cur.steps;
  }
  cur.step = (int)r;
  cur.unit = sh.unit + (long long)cur.h * cur.st.tiles + cur.tile;
  return (int)(total * (blockIdx.x + 1) / ctas - sh.begin);
}

// A query row of a unit.
struct QueryRow {
  int b, t, hq;
  bool real;
};
template <int kRows>
__device__ __forceinline__ QueryRow query_row(const AttendParams& p, const StreamSet& set, const Cursor<kRows>& c, int r) {
  const long long ur = (long long)c.tile * kRows + r;
  const int tok = (int)(ur / p.group);
  QueryRow q;
  q.hq = c.h * p.group + (int)(ur - (long long)tok * p.group);
  q.real = tok < c.st.n;
  q.b = c.s - set.prefixes;
  q.t = tok;
  if (c.s < set.prefixes) {
    const int b0 = c.s * p.fan;
    if (!p.n_new) {
      q.b = b0 + tok / p.m;
      q.t = tok % p.m;
    } else {
      int lo = b0, hi = b0 + p.fan;               // the last sequence that begins at or before the token
      const int at = tokens_before(p, b0) + tok;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.tok_base[mid] <= at) lo = mid;
        else hi = mid;
      }
      q.b = lo;
      q.t = at - p.tok_base[lo];
    }
  }
  return q;
}

}  // namespace evict
