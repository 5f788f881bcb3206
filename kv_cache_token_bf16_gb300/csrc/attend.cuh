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
__device__ __forceinline__ void prefetch_maps(const AttendParams& p, const WorkSet& set, int lane) {
  if (lane < 2 && p.pages && set.seqs) tc::tma_prefetch_desc(lane == 0 ? &p.tm_k : &p.tm_v);
  if (lane >= 2 && lane < 4 && p.fan && (set.prefixes || set.joint)) tc::tma_prefetch_desc(lane == 2 ? &p.tm_pk : &p.tm_pv);
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

// A position in the line of steps.
template <int kRows, int kTokens>
struct Cursor {
  int e, h, step, unit;
  Block k;
  // on to the next unit
  __device__ __forceinline__ void next_unit(const AttendParams& p, const WorkSet& set, int blocks) {
    step = 0;
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

// SMs of a kernel with `mine` steps beside one with `other` steps, of sms in all.
__device__ __forceinline__ int sms_of(const WorkSet& set, int mine, const WorkSet& rest, int other, int sms) {
  if (other == 0 || mine == 0) return sms;
  const float a = (float)mine * (float)set.cost, b = (float)other * (float)rest.cost;
  // the wide kernel's number is computed alike on both sides, and the few-row kernel has what is left
  const bool wide = set.workers == 1;
  const float w = wide ? a : b;
  const int n = min(sms - 1, max(1, (int)((float)sms * (w / (a + b)) + 0.5f)));
  return wide ? n : sms - n;
}

constexpr int kMaxWarps = 12;
struct ScanShared {
  int a[kMaxWarps], b[kMaxWarps];
  int e[kMaxWarps], rest[kMaxWarps];              // where the shares of this CTA begin
};

// Exclusive sum of `a` over the block's threads, and the totals of a and b.
template <int kThreads>
__device__ __forceinline__ int block_scan(int a, int b, int& total, int& total_b, ScanShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  b = __reduce_add_sync(0xffffffffu, b);
  if (lane == 31) sh.a[warp] = x, sh.b[warp] = b;
  __syncthreads();
  total = total_b = 0;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) x += sh.a[w];
    total += sh.a[w];
    total_b += sh.b[w];
  }
  __syncthreads();
  return x - a;
}

// Where the shares first .. first + kPer - 1 of this CTA begin, found from the lengths on the
// device (sh.e, sh.rest; all threads call it). `rest`: the other kernel's work (blocks of kRestRows
// rows, steps of kRestTokens). CTA 0 leaves the blocks' first steps for the join.
template <int kRows, int kTokens, int kRestRows, int kRestTokens, int kThreads, int kPer>
__device__ __forceinline__ Shares find_shares(const AttendParams& p, const WorkSet& set, const WorkSet& rest,
                                              ScanShared& sh) {
  const int tid = threadIdx.x;
  int total, total_rest;
  if (p.n_new && (set.prefixes || rest.prefixes)) {
    // every CTA writes the same sums, and reads back its own
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    int a = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) a += sequence(p, b, false).n;
    a = block_scan<kThreads>(a, 0, total, total_rest, sh);
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      p.tok_base[b] = a;
      a += sequence(p, b, false).n;
    }
    if (tid == 0) p.tok_base[p.batch] = total;
    __syncthreads();
  }
  const int blocks = set.blocks();
  const int per = (blocks + kThreads - 1) / kThreads;
  const int e0 = min(tid * per, blocks), e1 = min(e0 + per, blocks);
  Block k;
  int other = 0;
#pragma unroll 1
  for (int e = tid; e < rest.blocks(); e += kThreads) {
    load_block<kRestRows, kRestTokens>(p, rest, e, k);
    other += k.steps * p.hkv;
  }
  int work = 0, a = 0, lo = 0, hi = 0;
  Shares shares;
  const int first = blockIdx.x * kPer;
  // two passes over this thread's blocks: their sum, then (with the sums before) what begins in them
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1) {
      a = block_scan<kThreads>(work, other, total, total_rest, sh);
      const int most = sms_of(set, total, rest, total_rest, p.sms) * kPer;
      shares = Shares(total, total == 0 ? 0 : max(1, min(most, total / set.min_steps)));
      lo = shares.begin(min(first, shares.count));
      hi = shares.begin(min(first + kPer, shares.count));
      if (blockIdx.x != 0 && (a >= hi || a + work <= lo)) break;
    }
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      if (pass == 0 || per > 1) load_block<kRows, kTokens>(p, set, e, k, blockIdx.x == 0 && pass == 0);
      const int w = k.steps * p.hkv;
      if (pass == 0) {
        work += w;
        continue;
      }
      if (blockIdx.x == 0) set.base[e] = a;
#pragma unroll 1
      for (int i = 0; i < kPer && first + i < shares.count; ++i) {
        const int g = shares.begin(first + i);
        if (g >= a && g < a + w) {
          sh.e[i] = e;
          sh.rest[i] = g - a;
          if (set.start) set.start[first + i] = make_int2(e, g - a);
        }
      }
      a += w;
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    set.base[blocks] = total;
    set.base[blocks + 1] = shares.count;
  }
  __syncthreads();
  return shares;
}

template <int kRows, int kTokens>
__device__ __forceinline__ Cursor<kRows, kTokens> place(const AttendParams& p, const WorkSet& set, int e, int rest) {
  Cursor<kRows, kTokens> c;
  c.e = e;
  load_block<kRows, kTokens>(p, set, e, c.k);
  c.h = rest / c.k.steps;
  c.step = rest - c.h * c.k.steps;
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
