// Device side of the prompts' schedule: blocks, units, steps and the share of
// them that a CTA takes (see prompt.h). The sequences' lengths are the device's.
// Counts of units fit 30 bits, and of cut units' steps 31 (the host refuses calls that might pass them).
#pragma once

#include "attend.cuh"
#include "common.cuh"
#include "pipeline.cuh"
#include "prompt.h"
#include "tcgen05.cuh"

namespace evict {

// Tokens of a sequence: rows row0 .. row0 + len - 1 of a plane.
struct Span {
  int plane, row0, len;
};

struct PromptBlock {
  int s, tile;                       // sequence, block of it
  Span at;
  int steps;                         // of each of its units
};

// Where packed sequences begin, and the blocks of those before each: in memory, or in shared memory.
struct Tables {
  const int32_t* starts;
  const int* base;
};

// Block e (below the blocks' number), where sequences are packed the last that begins at or before it.
// Steps(first token, length) are the kernel's.
template <typename Steps>
__device__ __forceinline__ PromptBlock block_of(const PromptWork& w, const Tables& t, int e, Steps steps) {
  PromptBlock k;
  if (!w.starts) {
    k.s = w.by_seq_blocks.div(e);
    k.tile = e - k.s * (int)w.by_seq_blocks.by;
    k.at = {k.s, 0, w.m};
  } else {
    int lo = 0, hi = w.seqs;
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (t.base[mid] <= e) lo = mid;
      else hi = mid;
    }
    k.s = lo;
    k.tile = e - t.base[lo];
    const int row0 = t.starts[lo];
    k.at = {0, row0, t.starts[lo + 1] - row0};
  }
  k.steps = steps(k.tile * w.tile, k.at.len);
  return k;
}

constexpr int kMaxPromptWarps = 20;
struct PromptScan {
  int sum[kMaxPromptWarps];
  int e, rest;
  PromptBlock k;
};

// Sum of x over the threads before this one; its total. Between two calls is a barrier.
template <int kThreads>
__device__ __forceinline__ int prompt_scan(int x, int& total, PromptScan& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int y = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) y += u;
  }
  if (lane == 31) sh.sum[warp] = y;
  __syncthreads();
  constexpr int kCount = kThreads / 32;
  int u = lane < kCount ? sh.sum[lane] : 0;
#pragma unroll
  for (int d = 1; d < kCount; d <<= 1) {
    const int s = __shfl_up_sync(0xffffffffu, u, d);
    if (lane >= d) u += s;
  }
  total = __shfl_sync(0xffffffffu, u, kCount - 1);
  return y - x + (warp ? __shfl_sync(0xffffffffu, u, warp - 1) : 0);
}

// Sequences whose tables fit the shared memory that the tiles have not come to yet.
constexpr int kScratchSeqs = 4096;

// The blocks' number, 0 where the sequences are not one behind the other inside the plane: then the call
// writes nothing but the error. All threads. Every CTA leaves the same block_base, and reads back its own.
template <int kThreads>
__device__ __forceinline__ int count_blocks(const PromptWork& w, PromptScan& sh, int* scratch, Tables& t) {
  t = {w.starts, w.block_base};
  if (!w.starts) return w.blocks;
  const int tid = threadIdx.x, per = (w.seqs + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, w.seqs), s1 = min(s0 + per, w.seqs);
  int* bases = nullptr;
  if (w.seqs <= kScratchSeqs) {                   // the searches below are in them
#pragma unroll 1
    for (int s = tid; s <= w.seqs; s += kThreads) scratch[s] = w.starts[s];
    bases = scratch + kScratchSeqs + 1;
    t = {scratch, bases};
    __syncthreads();
  }
  int bad = 0, mine = 0;
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    const int a = t.starts[s], b = t.starts[s + 1];
    if (a < 0 || b < a || b > w.m) bad = 1;
    else mine += w.by_tile.div(b - a + w.tile - 1);
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && tid == 0) raise_device_error(w.err, kDevBadIndex);
    return 0;
  }
  int total, base = prompt_scan<kThreads>(mine, total, sh);
#pragma unroll 1
  for (int s = s0; s < s1; ++s) {
    w.block_base[s] = base;
    if (bases) bases[s] = base;
    base += w.by_tile.div(t.starts[s + 1] - t.starts[s] + w.tile - 1);
  }
  __syncthreads();
  return total;
}

// A CTA's way through its units.
struct PromptCursor {
  PromptBlock k;
  int blocks;
  int e, h;
  int from, to;                      // steps of the unit that are this CTA's
  int left;                          // of the share, from `from` on
  int round;                         // whole: units before
};

// Whole units: the CTA's unit of this turn; negative where there is none. The longest units come first. Either a CTA
// takes the next one when it comes to it (who takes which changes no result), or every other round goes the other way
// round the CTAs, so that their sums are nearly equal.
__device__ __forceinline__ int whole_unit(const PromptWork& w, int units, int round) {
  int rank = round * (int)gridDim.x + (round & 1 ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
  if (w.taken && round > 0) rank = (int)gridDim.x + atomicAdd(w.taken, 1);
  return rank >= units ? -1 : w.longest_last ? units - 1 - rank : rank;
}

// The steps of the unit at hand behind `step` (negative: in its entry); false where the share ends before.
__device__ __forceinline__ bool settle(PromptCursor& c, int step) {
  if (step < 0) {
    const int pay = min(c.left, -step);
    step += pay;
    c.left -= pay;
  }
  if (c.left <= 0) return false;
  c.from = step;
  c.to = min(c.k.steps, step + c.left);
  return true;
}

// Block of a whole unit.
__device__ __forceinline__ int whole_block(const PromptWork& w, int unit) {
  const int e = w.by_hkv.div(unit);
  return w.order ? w.order[e] : e;
}

// Blocks by their number in their sequence, all sequences' first ones first: where a sequence's first blocks have the
// most steps, long units then come early and the last ones taken are short. All threads.
template <int kThreads, typename Steps>
__device__ __forceinline__ void order_blocks(const PromptWork& w, const Tables& t, int blocks, Steps steps) {
#pragma unroll 1
  for (int e = threadIdx.x; e < blocks; e += kThreads) {
    const PromptBlock k = block_of(w, t, e, steps);
    int at = 0;                                   // blocks before: of lower number, and of the same one
    int base = 0;
#pragma unroll 4
    for (int s = 0; s < w.seqs; ++s) {
      const int next = s + 1 < w.seqs ? t.base[s + 1] : blocks, n = next - base;
      at += min(n, k.tile) + (s < k.s && n > k.tile);
      base = next;
    }
    w.order[at] = e;
  }
  __syncthreads();
}

// On to the next unit; false at the share's end. (Blocks are looked up at few places, and uncut units without the search
// for a share: at a kernel's start its code comes from memory, some 6,000 clocks for 25 KB of it.)
template <typename Steps>
__device__ __forceinline__ bool next_unit(const PromptWork& w, PromptCursor& c, Steps steps) {
  int e = c.e;
  if (w.whole) {
    const int unit = whole_unit(w, c.blocks * w.hkv, ++c.round);
    if (unit < 0) return false;
    e = whole_block(w, unit);
    c.h = unit - w.by_hkv.div(unit) * w.hkv;
  } else {
    c.left -= c.to - c.from;
    if (c.left <= 0) return false;
    if (++c.h == w.hkv) c.h = 0, ++e;
  }
  if (e != c.e) {
    c.e = e;
    c.k = block_of(w, Tables{w.starts, w.block_base}, e, steps);
  }
  if (!w.whole) return settle(c, -w.entry);
  c.from = 0;
  c.to = c.k.steps;
  return true;
}

// Where this CTA's share begins; false where it has none. All threads call it, and a barrier comes before the first
// copy to `scratch` (2 kScratchSeqs + 1 words). The shares are left for the join.
template <int kThreads, typename Steps>
__device__ __forceinline__ bool first_unit(const PromptWork& w, PromptScan& sh, int* scratch, PromptCursor& c, Steps steps) {
  Tables t;
  c.blocks = count_blocks<kThreads>(w, sh, scratch, t);
  tc::fence_proxy_async_smem();                   // of `scratch`, for the copies to come
  if (w.whole) {
    if (w.order) order_blocks<kThreads>(w, t, c.blocks, steps);
    const int unit = whole_unit(w, c.blocks * w.hkv, 0);
    if (unit < 0) return false;                   // the whole CTA, here and below
    c.round = 0;
    c.e = whole_block(w, unit);
    c.h = unit - w.by_hkv.div(unit) * w.hkv;
    c.k = block_of(w, t, c.e, steps);
    c.from = 0;
    c.to = c.k.steps;
    return true;
  }
  const int tid = threadIdx.x, per = (c.blocks + kThreads - 1) / kThreads;
  const int e0 = min(tid * per, c.blocks), e1 = min(e0 + per, c.blocks);
  Shares shares;
  int base = 0, g0 = 0;
  // the sums of the steps; then the block where the share begins
#pragma unroll 1
  for (int find = 0; find < 2; ++find) {
    if (find) {
      if ((int)blockIdx.x >= shares.count) return false;
      g0 = shares.begin(blockIdx.x);
    }
    int at = base;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      const PromptBlock k = block_of(w, t, e, steps);
      const int of_block = (k.steps + w.entry) * w.hkv;
      if (find && g0 >= at && g0 < at + of_block) {
        sh.e = e;
        sh.rest = g0 - at;
        sh.k = k;
      }
      at += of_block;
    }
    if (!find) {
      int total;
      base = prompt_scan<kThreads>(at, total, sh);
      shares = Shares(total, total ? max(1, min((int)gridDim.x, total / w.min_steps)) : 0);
      if (blockIdx.x == 0 && tid == 0) {
        w.total[0] = total;
        w.total[1] = shares.count;
      }
    }
  }
  __syncthreads();
  c.e = sh.e;
  c.k = sh.k;
  const int unit = c.k.steps + w.entry;
  c.h = sh.rest / unit;
  c.left = shares.begin(blockIdx.x + 1) - g0;
  const int step = sh.rest - c.h * unit - w.entry;
  if (tid == 0) {                                 // what the join needs to know
    int4* at = reinterpret_cast<int4*>(w.begin + blockIdx.x);
    at[0] = make_int4(c.k.at.plane, c.k.at.row0, c.k.at.len, c.k.tile);
    at[1] = make_int4(c.h, step, c.k.steps, 0);
  }
  return settle(c, step);            // false: the share lies in one unit's entry
}

// A unit that two or more CTAs share, found where a share begins inside it: the first such share's
// block does the work. Its parts: slot 2 c0 + 1, then 2 c of the following shares up to c1.
struct SplitUnit {
  Span at;
  int tile, h, c0, c1;
};
__device__ __forceinline__ bool split_unit(const PromptWork& w, int c, SplitUnit& u) {
  const int4* from = reinterpret_cast<const int4*>(w.begin + c);
  const int4 a = from[0], b = from[1];            // beside the next, whether there is such a share or not
  const Shares shares(w.total[0], w.total[1]);
  if (c >= shares.count) return false;
  if (b.y <= 0) return false;                     // the share begins with the unit, or in its entry
  const int first = shares.begin(c) - b.y;
  u.at = {a.x, a.y, a.z};
  u.tile = a.w;
  u.h = b.x;
  u.c0 = shares.of(first);
  u.c1 = shares.of(first + b.z - 1);
  return u.c0 == c - 1;
}

// Waits at many places, so little code: polls that sleep in hardware, a bounded number of them. The kernel's end
// reports one that gave up.
constexpr uint32_t kPolls = 100000;               // of a wait, each of up to 20 us
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* fail, uint32_t most = kPolls) {
  if (tc::mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (uint32_t polls = 0; !tc::mbar_try_wait_sleep(bar, parity, kWaitSleepNs);)
    if (++polls == most || *fail) {
      *fail = 1;
      return false;
    }
  return true;
}
// A warp's wait; the same for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* fail, uint32_t most = kPolls) {
  return __all_sync(0xffffffffu, wait_for(bar, parity, fail, most));
}
// One lane's value for the warp, which the compiler then knows to be the same: what follows from it stays in uniform
// registers, where products take their operands from. (A lone thread's, or what might differ, is moved there one by
// one: 128 x 64 x 16 products then take 65 clocks instead of 48; a document of 8192 tokens 395 us instead of 369.)
__device__ __forceinline__ int uni(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Whether a phase is over, without a wait.
__device__ __forceinline__ bool test_phase(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(tc::smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(bar))
      : "memory");
}

}  // namespace evict
