// The weights that a prompt's attention put on each key: w_j = sum over the group's query heads and the
// queries t that see key j (t >= j; with `last` only a sequence's last ones) of exp(scale q_t.k_j - lse_t).
//
// A unit is a (sequence, KV head, block of 256 keys), a step 128 tokens' queries of one head. The logits
// are taken transposed, S^T = K Q^T, keys along the rows of tensor memory: a thread then holds one key and
// sums along its row, and no sum crosses threads but that of the row's two halves at a unit's end. K is
// held (two buffers of two 128-row tiles, the next unit's is fetched meanwhile), Q streams through a ring
// of three 32 KB tiles, and so do its log-sum-exps through shared memory, negated, in base 2 and with
// -infinity for queries that do not count, whose weights are then 0. Two accumulators for each of the two key tiles
// (512 columns): products run while the sixteen summing warps exponentiate the step before.
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
constexpr int kRing = 3, kLseRing = 3;
constexpr int kSumWarps = 16;
constexpr int kMmaWarp = 16, kTmaWarp = 17, kThreads = 608;   // warp 18 loads the log-sum-exps
constexpr int kEntry = 2, kMinSteps = 8;
constexpr int kWholeRows = 1024;

struct WeightsShared {
  uint64_t k_full[2], k_empty[2], q_full[kRing], q_empty[kRing], s_full[2], s_empty[2];
  uint64_t lse_full[kLseRing], lse_empty[kLseRing], done;
  uint32_t tmem_base;
  int fail;
  alignas(16) float neg_lse2[kLseRing][kTile];
  float sums[kKeys];
  PromptScan scan;
};
// All of it is dynamic: seven tiles and this fill the 227 KB.
constexpr int kSmem = (4 + kRing) * kTileBytes + (int)sizeof(WeightsShared);
static_assert(kSmem <= 227 * 1024);

// The first query that counts for the keys from key0 on.
__device__ __forceinline__ int first_query(int last, int key0, int len) { return max(key0, last ? len - last : 0); }

struct Steps {
  int group, last;
  __device__ __forceinline__ int operator()(int key0, int len) const {
    return group * ((len - first_query(last, key0, len) + kTile - 1) / kTile);
  }
};

// What a step works on: queries tok0 .. tok0 + n - 1 of head g, all of which count.
struct Unit {
  int key0, keys, first, tiles;
  __device__ __forceinline__ Unit(const PromptParams& p, const PromptCursor& c) {
    key0 = c.k.tile * kKeys;
    keys = min(kKeys, c.k.at.len - key0);
    first = first_query(p.last, key0, c.k.at.len);
    tiles = (c.k.at.len - first + kTile - 1) / kTile;
  }
};
struct Step {
  int g, tile;                                    // head of the group, tile of 128 queries
  int tok0, n;
  __device__ __forceinline__ Step(const Unit& u, const PromptCursor& c) {
    g = c.from / u.tiles;
    tile = c.from - g * u.tiles;
    place(u, c);
  }
  __device__ __forceinline__ void place(const Unit& u, const PromptCursor& c) {
    tok0 = u.first + tile * kTile;
    n = min(kTile, c.k.at.len - tok0);
  }
  __device__ __forceinline__ void next(const Unit& u, const PromptCursor& c) {
    if (++tile == u.tiles) tile = 0, ++g;
    place(u, c);
  }
  // some query of the step sees a key of tile kt
  __device__ __forceinline__ bool sees(const Unit& u, int kt) const {
    return kt * kTile < u.keys && tok0 + n > u.key0 + kt * kTile;
  }
};

template <int kCount>
struct Ring {
  int i = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++i == kCount) i = 0, parity ^= 1;
  }
};

__device__ void producer(const PromptParams& p, WeightsShared& sh, PromptCursor c, uint32_t kbuf, uint32_t ring) {
  const Steps steps{p.group, p.last};
  Ring<2> k;
  Ring<kRing> q;
  int used_k = 0, used_q = 0;
  bool ok = true;
  do {
    const Unit u(p, c);
    const int tiles = u.keys > kTile ? 2 : 1;
    if (!(ok = wait_phase(&sh.k_empty[k.i], k.parity ^ 1, &sh.fail, p.work.err))) break;
    tc::mbar_arrive_expect_tx(&sh.k_full[k.i], tiles * kTileBytes);
    for (int j = 0; j < 2 * tiles; ++j)
      tma_load_4d(kbuf + k.i * 2 * kTileBytes + j * (kTileBytes / 2), &p.k_map, (j & 1) * 64,
                  c.k.at.row0 + u.key0 + (j >> 1) * kTile, c.h, c.k.at.plane, &sh.k_full[k.i]);
    k.next();
    ++used_k;
    Step s(u, c);
    for (int i = c.from; i < c.to; ++i, s.next(u, c)) {
      if (!(ok = wait_phase(&sh.q_empty[q.i], q.parity ^ 1, &sh.fail, p.work.err))) break;
      tc::mbar_arrive_expect_tx(&sh.q_full[q.i], kTileBytes);
      for (int hf = 0; hf < 2; ++hf)
        tma_load_4d(ring + q.i * kTileBytes + hf * (kTileBytes / 2), &p.q_map, hf * 64, c.k.at.row0 + s.tok0,
                    c.h * p.group + s.g, c.k.at.plane, &sh.q_full[q.i]);
      q.next();
      ++used_q;
    }
  } while (ok && next_unit(p.work, c, steps));
  // every copy issued must land before the CTA may release its shared memory
  for (int i = 0; i < 2 && i < used_k; ++i) drain_phase(&sh.k_full[i], ((used_k - 1 - i) / 2) & 1, p.work.err);
  for (int i = 0; i < kRing && i < used_q; ++i) drain_phase(&sh.q_full[i], ((used_q - 1 - i) / kRing) & 1, p.work.err);
}

// The steps' log-sum-exps to shared memory, four of a step by each lane.
__device__ void lse_loader(const PromptParams& p, WeightsShared& sh, PromptCursor c) {
  const Steps steps{p.group, p.last};
  const int lane = threadIdx.x & 31;
  Ring<kLseRing> r;
  bool ok = true;
  do {
    const Unit u(p, c);
    Step s(u, c);
    for (int i = c.from; i < c.to; ++i, s.next(u, c)) {
      const float* from = p.lse + ((long long)c.k.at.plane * p.hq + c.h * p.group + s.g) * p.work.m + c.k.at.row0 + s.tok0;
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 32 * j + lane;
        const float l = t < s.n ? from[t] : -INFINITY;
        x[j] = l == -INFINITY ? l : -l * kLog2e;                   // no weights of a query that saw nothing
      }
      ok = wait_phase(&sh.lse_empty[r.i], r.parity ^ 1, &sh.fail, p.work.err);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) sh.neg_lse2[r.i][32 * j + lane] = x[j];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.lse_full[r.i]);
      r.next();
    }
  } while (ok && next_unit(p.work, c, steps));
}

__device__ void mma_issuer(const PromptParams& p, WeightsShared& sh, PromptCursor c, uint32_t tmem, uint32_t kbuf,
                           uint32_t ring) {
  const Steps steps{p.group, p.last};
  const uint64_t kd = tc::sw128_desc(kbuf), qd = tc::sw128_desc(ring);
  const uint32_t hi = (uint32_t)(kd >> 32), k_lo = (uint32_t)kd, q_lo = (uint32_t)qd;
  Ring<2> k, s_buf;
  Ring<kRing> q;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return ok = __all_sync(0xffffffffu, wait_phase(bar, parity, &sh.fail, p.work.err));
  };
  do {
    const Unit u(p, c);
    if (!wait(&sh.k_full[k.i], k.parity)) break;
    Step s(u, c);
    for (int i = c.from; i < c.to; ++i, s.next(u, c)) {
      if (!wait(&sh.q_full[q.i], q.parity) || !wait(&sh.s_empty[s_buf.i], s_buf.parity ^ 1)) break;
      tc::fence_after_sync();
      const uint32_t idesc = tc::idesc_bf16_f32(kTile, (s.n + 15) & ~15);
#pragma unroll 1
      for (int kt = 0; kt < 2; ++kt) {
        if (!s.sees(u, kt)) continue;
        tm::warp_mma_rows(tmem + (2 * s_buf.i + kt) * kTile, tm::desc_of(k_lo + (((2 * k.i + kt) * kTileBytes) >> 4), hi),
                          tm::desc_of(q_lo + ((q.i * kTileBytes) >> 4), hi), idesc);
      }
      tm::warp_mma_commit(&sh.s_full[s_buf.i]);
      tm::warp_mma_commit(&sh.q_empty[q.i]);
      if (i + 1 == c.to) tm::warp_mma_commit(&sh.k_empty[k.i]);
      q.next();
      s_buf.next();
    }
    if (!ok) break;
    k.next();
  } while (next_unit(p.work, c, steps));
  // every MMA must finish before tensor and shared memory are released
  tm::warp_mma_commit(&sh.done);
  drain_phase(&sh.done, 0, p.work.err);
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

// A summing warp: 32 keys of tile kt, a thread each, and half of a step's queries.
__device__ void sum_warp(const PromptParams& p, WeightsShared& sh, PromptCursor c, uint32_t tmem) {
  const Steps steps{p.group, p.last};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kt = (warp >> 2) & 1, half = warp >> 3, key = kt * kTile + (warp & 3) * 32 + lane;
  const uint32_t s_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kt * kTile + half * 64;
  const uint64_t sc2 = pack_f32x2(p.scale2, p.scale2);
  Ring<2> s_buf;
  Ring<kLseRing> r;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool there = wait_phase(bar, parity, &sh.fail, p.work.err);
    ok = __all_sync(0xffffffffu, there) && ok;
    return ok;
  };
  do {
    const Unit u(p, c);
    Step s(u, c);
    float sum = 0.f;
#pragma unroll 1
    for (int i = c.from; i < c.to; ++i, s.next(u, c)) {
      if (!wait(&sh.lse_full[r.i], r.parity) || !wait(&sh.s_full[s_buf.i], s_buf.parity)) break;
      tc::fence_after_sync();
      const int columns = s.sees(u, kt) ? s.n - 64 * half : 0;   // of this warp's 64
      if (columns > 0) {
        const uint32_t at = s_at + s_buf.i * 2 * kTile;
        const int before = u.key0 + key - s.tok0 - 64 * half;    // columns that do not see this key
        const bool masked = columns < 64 || __any_sync(0xffffffffu, before > 0);
        const float4* l2 = reinterpret_cast<const float4*>(&sh.neg_lse2[r.i][64 * half]);
        float x[64];
        tm::load64(at, x);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.s_empty[s_buf.i]);
        auto add = [&](auto with_mask) {
          uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
          for (int j = 0; j < 64; j += 4) {
            const float4 l = l2[j / 4];
            uint64_t e0 = ex2_f32x2(fma_f32x2(pack_f32x2(x[j], x[j + 1]), sc2, pack_f32x2(l.x, l.y)));
            uint64_t e1 = ex2_f32x2(fma_f32x2(pack_f32x2(x[j + 2], x[j + 3]), sc2, pack_f32x2(l.z, l.w)));
            if constexpr (decltype(with_mask)::value) {
              float a, b;
              split_f32x2(e0, a, b);
              e0 = pack_f32x2(j >= before && j < columns ? a : 0.f, j + 1 >= before && j + 1 < columns ? b : 0.f);
              split_f32x2(e1, a, b);
              e1 = pack_f32x2(j + 2 >= before && j + 2 < columns ? a : 0.f, j + 3 >= before && j + 3 < columns ? b : 0.f);
            }
            acc[0] = add_f32x2(acc[0], e0);
            acc[1] = add_f32x2(acc[1], e1);
          }
          float a, b;
          split_f32x2(add_f32x2(acc[0], acc[1]), a, b);
          sum += a + b;
        };
        if (masked) add(std::true_type{});
        else add(std::false_type{});
        __syncwarp();
      } else if (lane == 0) {
        tc::mbar_arrive(&sh.s_empty[s_buf.i]);
      }
      if (lane == 0) tc::mbar_arrive(&sh.lse_empty[r.i]);
      s_buf.next();
      r.next();
    }
    // the halves of a key's sum meet: warp w + 8's go to warp w. Both leave together where either has given up.
    if (half) sh.sums[key] = sum;
    if (!named_and(1 + (warp & 7), 64, ok)) break;
    if (!half) {
      sum += sh.sums[key];
      if (c.to - c.from == c.k.steps) {
        if (key < u.keys)
          p.weights[((long long)c.k.at.plane * p.work.hkv + c.h) * p.work.m + c.k.at.row0 + u.key0 + key] = sum;
      } else {
        p.part[(size_t)(2 * blockIdx.x + (c.from == 0 ? 1 : 0)) * kKeys + key] = sum;
      }
    }
    tc::named_sync(1 + (warp & 7), 64);
  } while (next_unit(p.work, c, steps));
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
      tc::mbar_init(&sh.k_empty[i], 1);
      tc::mbar_init(&sh.s_full[i], 1);
      tc::mbar_init(&sh.s_empty[i], kSumWarps);
    }
    for (int i = 0; i < kRing; ++i) {
      tc::mbar_init(&sh.q_full[i], 1);
      tc::mbar_init(&sh.q_empty[i], 1);
    }
    for (int i = 0; i < kLseRing; ++i) {
      tc::mbar_init(&sh.lse_full[i], 1);
      tc::mbar_init(&sh.lse_empty[i], kSumWarps);
    }
    tc::mbar_init(&sh.done, 1);
    sh.fail = 0;
  }
  if (warp == kTmaWarp && lane == 0) {
    tc::tma_prefetch_desc(&p.q_map);
    tc::tma_prefetch_desc(&p.k_map);
  }
  pdl_wait();
  PromptCursor c;
  const bool any = first_unit<kThreads>(p.work, sh.scan, c, Steps{p.group, p.last});
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0), ring = smem + 4 * kTileBytes;
  if (any) {
    if (warp < kSumWarps) {
      sum_warp(p, sh, c, tmem);
    } else if (warp == kMmaWarp) {
      mma_issuer(p, sh, c, tmem, smem, ring);
    } else if (warp == kTmaWarp) {
      if (lane == 0) producer(p, sh, c, smem, ring);
      __syncwarp();
    } else {
      lse_loader(p, sh, c);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, 4 * kTile);
}

// Keys of units that two or more CTAs share: their parts' sums, in the shares' order.
__global__ void __launch_bounds__(kKeys) prompt_weights_join_kernel(const __grid_constant__ PromptParams p) {
  pdl_wait();
  SplitUnit u;
  if (!split_unit(p.work, blockIdx.x + 1, u, Steps{p.group, p.last})) return;
  const int key = threadIdx.x, at = u.k.tile * kKeys + key;
  if (at >= u.k.at.len) return;
  float sum = 0.f;
#pragma unroll 4
  for (int i = u.c0; i <= u.c1; ++i) sum += p.part[(size_t)(2 * i + (i == u.c0 ? 1 : 0)) * kKeys + key];
  p.weights[((long long)u.k.at.plane * p.work.hkv + u.h) * p.work.m + u.k.at.row0 + at] = sum;
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

int make_plan(const evict_prompt* a, PromptPlan* plan) {
  const long long most = (long long)(a->q.heads / a->k.heads) * (((long long)a->m + kTile - 1) / kTile);
  const int rc = plan_prompt(a, kKeys, most, kEntry, kMinSteps, kWholeRows, 0, 2 * kKeys * sizeof(float), plan);
  plan->p.last = a->last;
  return rc;
}

}  // namespace
}  // namespace evict

using namespace evict;

extern "C" int evict_prompt_weights_workspace(const evict_prompt* a, size_t* bytes) {
  if (!bytes) return fail(EVICT_EINVAL, "bytes is NULL");
  PromptPlan plan;
  int rc;
  if ((rc = check_prompt_sizes(a)) || (rc = make_plan(a, &plan))) return rc;
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
  if ((rc = encode_heads(&p.q_map, a->q, a->batch, a->m, 1, kTile, false, "q")) ||
      (rc = encode_heads(&p.k_map, a->k, a->batch, a->m, 1, kTile, false, "k")))
    return rc;
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  cudaError_t e = allow_smem(plan.dev);
  if (e != cudaSuccess) return cuda_fail(e, "prompt weights kernel attribute");
  const int ctas = p.work.whole ? std::min(plan.sms, p.work.blocks * p.work.hkv) : plan.sms;
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
