// Device side of the attention kernels' schedule: blocks, units, steps and the
// share of them that a warp or CTA takes (see attend.h). Counts of steps and
// rows fit 31 bits (the host refuses calls that might pass them).
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
// The first lanes of a warp fetch the maps that this launch uses.
__device__ __forceinline__ void prefetch_maps(const AttendParams& p, int lane) {
  if (lane < 2 && p.few.prefixes) tc::tma_prefetch_desc(&p.few_pre[lane]);
  if (lane < 2 && p.few.seqs && p.pages) tc::tma_prefetch_desc(&p.few_own[lane]);
  if (lane < 2 && p.fan && (p.wide.prefixes || p.wide.joint)) tc::tma_prefetch_desc(&p.wide_pre[lane]);
  if (lane < 2 && p.wide.seqs && p.pages) tc::tma_prefetch_desc(&p.wide_own[lane]);
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
  int len = p.pages ? p.lens[b] : 0;
  const int room = p.pages ? p.table_width << p.page_shift : 0;
  const int n1 = min(max(n, 0), p.m), len1 = min(max(len, 0), room);
  if (report && (n1 != n || len1 != len)) raise_device_error(p.err, kDevBadIndex);
  return {n1, len1};
}
// New tokens of the sequences before b. Padding is left out of a prefix's query rows.
__device__ __forceinline__ int tokens_before(const AttendParams& p, int b) {
  return p.n_new ? p.tok_base[b] : b * p.m;
}

// A block: a tile of query rows of a stream.
struct Block {
  int s, tile;                       // prefix, or prefixes + sequence
  int n, len;                        // query tokens of the stream; own rows
  int pre;                           // prefix rows
  int reach;                         // last own row that the tile's last token sees (-1: none)
  int steps;                         // of each of its units
};
template <int kRows, int kTokens>
__device__ __forceinline__ void load_block(const AttendParams& p, const WorkSet& set, int e, Block& k,
                                           bool report = false) {
  const int pe = set.prefixes * set.prefix_tiles;
  if (e < pe) {
    k.s = set.by_prefix_tiles.div(e);
    k.tile = e - k.s * set.prefix_tiles;
    k.n = tokens_before(p, (k.s + 1) * p.fan) - tokens_before(p, k.s * p.fan);
    k.len = 0;
    k.pre = p.n_prefix;
  } else {
    const int b = set.by_seq_tiles.div(e - pe);
    k.s = set.prefixes + b;
    k.tile = e - pe - b * set.seq_tiles;
    const Seq q = sequence(p, b, report && k.tile == 0);
    k.n = q.n;
    k.len = q.len;
    k.pre = set.joint ? p.n_prefix : 0;
  }
  k.reach = -1;
  k.steps = 0;
  if (kRows * k.tile < k.n * p.group) {
    if (k.len > 0) {
      const int t = p.by_group.div(kRows * (k.tile + 1) - 1);
      k.reach = max(-1, k.len - k.n + min(t, k.n - 1));
    }
    k.steps = (k.pre + kTokens - 1) / kTokens + (k.reach + kTokens) / kTokens;
    if (set.joint) k.steps = max(k.steps, 1);     // joint units write their rows themselves: all need a step
  }
}

// Steps of a block's units, entries included.
__device__ __forceinline__ int work_of(const AttendParams& p, const WorkSet& set, const Block& k) {
  return k.steps ? (k.steps + set.entry) * p.hkv : 0;
}

// A position in the line of steps.
template <int kRows, int kTokens>
struct Cursor {
  int e, h, step, unit;              // step < 0: in the unit's entry
  Block k;
  // past the entry, as far as the share's `left` steps reach
  __device__ __forceinline__ void settle(int& left) {
    if (step >= 0) return;
    const int pay = min(left, -step);
    step += pay;
    left -= pay;
  }
  // on to the next unit
  __device__ __forceinline__ void next_unit(const AttendParams& p, const WorkSet& set, int blocks) {
    step = -set.entry;
    ++unit;
    if (++h < p.hkv) return;
    h = 0;
#pragma unroll 1
    for (;;) {
      if (++e >= blocks) return;
      load_block<kRows, kTokens>(p, set, e, k);
      if (k.steps) break;
      unit += p.hkv;
    }
  }
};

// Equal shares of `total` steps: the first `extra` have one step more.
struct Shares {
  int count = 0, each = 0, extra = 0;
  Shares() = default;
  __device__ __forceinline__ Shares(int total, int shares) : count(shares) {
    each = count ? total / count : 0;
    extra = total - each * count;
  }
  // as the kernel that took them left it
  __device__ __forceinline__ explicit Shares(const WorkSet& set) {
    const int* end = set.base + set.blocks();
    *this = Shares(end[0], end[1]);
  }
  __device__ __forceinline__ int begin(int i) const { return i * each + min(i, extra); }
  __device__ __forceinline__ int of(int g) const {                 // the share that holds step g
    const int cut = extra * (each + 1);
    return g < cut ? g / (each + 1) : extra + (g - cut) / each;
  }
};

// SMs of the wide units, with `wide` steps beside the few-row units' `few`: so many that both end
// together, start + a / w = b / (sms - w) with the two kinds' work a and b and the time by which a
// wide CTA's start is longer.
__device__ __forceinline__ int wide_sms(const AttendParams& p, int wide, int few) {
  if (few == 0 || wide == 0) return wide ? p.sms : 0;
  const float a = (float)wide * (float)p.wide.cost, b = (float)few * (float)p.few.cost, n = (float)p.sms;
  const float h = a + b - kWideStart * n;
  const float w = (sqrtf(h * h + 4.f * kWideStart * a * n) - h) / (2.f * kWideStart);
  return min(min(p.sms - 1, max(1, wide / p.wide.min_steps)), max(1, (int)(w + 0.5f)));
}

constexpr int kMaxWarps = 12;
struct ScanShared {
  int a[kMaxWarps], b[kMaxWarps];
  int e[kMaxWarps], rest[kMaxWarps];              // where the shares of this CTA begin
};

// Sums of a and b over the threads before this one, and their totals. Between two calls is a barrier.
template <int kThreads>
__device__ __forceinline__ void block_scan(int& a, int& b, int& total, int& total_b, ScanShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a, y = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) x += u, y += v;
  }
  if (lane == 31) sh.a[warp] = x, sh.b[warp] = y;
  __syncthreads();
  // every warp scans the warps' sums
  constexpr int kCount = kThreads / 32;
  int u = lane < kCount ? sh.a[lane] : 0, v = lane < kCount ? sh.b[lane] : 0;
#pragma unroll
  for (int d = 1; d < kCount; d <<= 1) {
    const int s = __shfl_up_sync(0xffffffffu, u, d), t = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) u += s, v += t;
  }
  total = __shfl_sync(0xffffffffu, u, kCount - 1);
  total_b = __shfl_sync(0xffffffffu, v, kCount - 1);
  const int before = __shfl_sync(0xffffffffu, u, max(warp - 1, 0)), before_b = __shfl_sync(0xffffffffu, v, max(warp - 1, 0));
  a = x - a + (warp ? before : 0);
  b = y - b + (warp ? before_b : 0);
}

// What a CTA works on: for wide units one share, otherwise one for each of its warps, `stride` apart
// (where there are fewer shares than warps, every SM has some).
struct Place {
  bool wide;
  int first, stride;
  Shares shares;
};

// The blocks e0 .. e1 - 1 of a set, whose steps before are `a`: their first steps for the join (`leave`), and
// where the CTA's shares begin that begin in them.
template <int kRows, int kTokens>
__device__ __forceinline__ void find_starts(const AttendParams& p, const WorkSet& set, const Place& at, int per, int e0,
                                            int e1, int a, int work, bool leave, ScanShared& sh) {
#pragma unroll 1
  for (int e = e0; e < e1; ++e) {
    int w = work;
    if (per > 1) {
      Block k;
      load_block<kRows, kTokens>(p, set, e, k);
      w = work_of(p, set, k);
    }
    if (leave) set.base[e] = a;
#pragma unroll 1
    for (int i = 0; i < set.workers && w > 0; ++i) {
      const int share = at.first + i * at.stride;
      if (share >= at.shares.count) break;
      const int g = at.shares.begin(share);
      if (g >= a && g < a + w) {
        sh.e[i] = e;
        sh.rest[i] = g - a;
        if (set.workers == 1) set.start[at.first] = make_int2(e, g - a);
      }
    }
    a += w;
  }
}

// The kind of units and the shares of this CTA, found from the lengths on the device (sh.e, sh.rest;
// all threads call it). The first CTA of either kind leaves the blocks' first steps for the join.
template <int kThreads, int kWarps>
__device__ __forceinline__ Place find_place(const AttendParams& p, ScanShared& sh) {
  const int tid = threadIdx.x;
  int total_w, total_f;
  if (p.n_new && (p.few.prefixes || p.wide.prefixes)) {
    // every CTA writes the same sums, and reads back its own
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    int a = 0, none = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) a += sequence(p, b, false).n;
    block_scan<kThreads>(a, none, total_w, total_f, sh);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      p.tok_base[b] = a;
      a += sequence(p, b, false).n;
    }
    if (tid == 0) p.tok_base[p.batch] = total_w;
    __syncthreads();
  }
  const int bw = p.wide.blocks(), bf = p.few.blocks();
  const int pw = (bw + kThreads - 1) / kThreads, pf = (bf + kThreads - 1) / kThreads;
  const int w0 = min(tid * pw, bw), w1 = min(w0 + pw, bw), f0 = min(tid * pf, bf), f1 = min(f0 + pf, bf);
  int work_w = 0, work_f = 0;
#pragma unroll 1
  for (int e = w0; e < w1; ++e) {
    Block k;
    load_block<kWideRows, kWideTokens>(p, p.wide, e, k, blockIdx.x == 0);
    work_w += work_of(p, p.wide, k);
  }
#pragma unroll 1
  for (int e = f0; e < f1; ++e) {
    Block k;
    load_block<kFewRows, kBoxTokens>(p, p.few, e, k, blockIdx.x == 0);
    work_f += work_of(p, p.few, k);
  }
  int a = work_w, f = work_f;
  block_scan<kThreads>(a, f, total_w, total_f, sh);
  const int ctas = wide_sms(p, total_w, total_f);
  Place at;
  at.wide = (int)blockIdx.x < ctas;
  at.first = at.wide ? blockIdx.x : blockIdx.x - ctas;
  at.stride = p.sms - ctas;
  const int total = at.wide ? total_w : total_f, most = at.wide ? ctas : (p.sms - ctas) * kWarps;
  const int least = at.wide ? p.wide.min_steps : p.few.min_steps;
  at.shares = Shares(total, total == 0 ? 0 : max(1, min(most, total / least)));
  const bool leave = at.first == 0;
  if (at.wide) find_starts<kWideRows, kWideTokens>(p, p.wide, at, pw, w0, w1, a, work_w, leave, sh);
  else find_starts<kFewRows, kBoxTokens>(p, p.few, at, pf, f0, f1, f, work_f, leave, sh);
  if (leave && tid == 0) {
    const WorkSet& set = at.wide ? p.wide : p.few;
    set.base[set.blocks()] = total;
    set.base[set.blocks() + 1] = at.shares.count;
  }
  if (blockIdx.x == 0 && tid == 0 && total_w == 0 && bw > 0) p.wide.base[bw] = p.wide.base[bw + 1] = 0;
  __syncthreads();
  return at;
}

template <int kRows, int kTokens>
__device__ __forceinline__ Cursor<kRows, kTokens> place(const AttendParams& p, const WorkSet& set, int e, int rest) {
  Cursor<kRows, kTokens> c;
  c.e = e;
  load_block<kRows, kTokens>(p, set, e, c.k);
  c.h = rest / (c.k.steps + set.entry);
  c.step = rest - c.h * (c.k.steps + set.entry) - set.entry;
  c.unit = e * p.hkv + c.h;
  return c;
}

// A query row of a block: row r is token r / group of the stream, head r % group of the KV head's.
struct QueryRow {
  int b, t, g;
  bool real;
};
template <int kRows>
__device__ __forceinline__ QueryRow query_row(const AttendParams& p, const WorkSet& set, const Block& k, int r) {
  const int ur = k.tile * kRows + r;
  const int tok = p.by_group.div(ur);
  QueryRow q;
  q.g = ur - tok * p.group;
  q.real = tok < k.n;
  q.b = k.s - set.prefixes;
  q.t = tok;
  if (k.s < set.prefixes) {
    const int b0 = k.s * p.fan;
    if (!p.n_new) {
      const int i = p.by_m.div(tok);
      q.b = b0 + i;
      q.t = tok - i * p.m;
    } else {
      int lo = b0, hi = b0 + p.fan;               // the last sequence that begins at or before the token
      const int at = p.tok_base[b0] + tok;
#pragma unroll 1
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
