// The weights that a step's queries put on the kept rows of a cache, added to the rows' scores:
//   score_j += sum over the sequences of a kept prefix, their tokens and the group's query heads of
//              exp(scale q.k_j - lse).
//
// A warp takes 32 keys, straight from memory to the registers of m16n8k16 products (their rows; a lane's
// 16-byte pieces of a row stand for the product's columns in another order, the same for the queries), and
// goes through the queries eight at a time, which come from L1 and L2. A key's sum lies in four lanes.
// Keys are read once: what bounds few queries is HBM or L2, many queries the products. Where there are
// fewer warps of keys than the GPU has room for, the queries are dealt out to up to eight warps for the same keys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "api_internal.h"
#include "attend.h"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"

namespace evict {
namespace {

constexpr int kWarps = 8, kKeys = 32, kQueries = 8;
constexpr int kScan = kWarps * 32;                // query rows that are looked through at once

struct WeighParams {
  const void* k;                     // [batch][heads][cap][128]
  float* score;                      // [batch][heads][cap]
  int cap, rows, heads;              // rows: kept
  const void* q;
  long long qb, qh, qm;              // element strides
  const float* lse;                  // [sequences][hq][m]
  const int32_t* n_new;
  int fan, m, hq, group;             // sequences of a cache's batch row
  int queries;                       // fan * m * group
  int split;                         // warps that share the queries of the same keys
  Divisor by_heads, by_per, by_group;   // per = m * group: query rows of a sequence
  float scale2;
  int* err;
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A tile's queries as a lane holds them: its pieces of one row, and the row's log-sum-exp (base 2, negative;
// -inf: the query does not count).
struct Queries {
  uint4 x[4];
  float neg;
};

__global__ void __launch_bounds__(kWarps * 32, 2) weigh_kernel(const __grid_constant__ WeighParams p) {
  __shared__ float sums[kWarps][kKeys];
  __shared__ long long at[kScan];                 // of the queries that count: where their rows lie in q,
  __shared__ int lse_at[kScan];                   // and their log-sum-exps
  __shared__ int counts[kWarps];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % p.split;
  const int unit = blockIdx.y, b = p.by_heads.div(unit), h = unit - b * p.heads;
  const int row0 = (blockIdx.x * (kWarps / p.split) + warp / p.split) * kKeys;
  const int n = lane >> 2, t = lane & 3;          // row of a fragment, and which pieces of it
  const __nv_bfloat16* keys = static_cast<const __nv_bfloat16*>(p.k) + (long long)unit * p.cap * kHeadDim;
  uint4 a[4][4];                                  // key n + 8 i, elements 32 j + 8 t ..
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + n + 8 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a[i][j] = row < p.rows ? reinterpret_cast<const uint4*>(keys + (long long)row * kHeadDim)[4 * j + t]
                             : make_uint4(0, 0, 0, 0);
  }
  float sum[4] = {0.f, 0.f, 0.f, 0.f};            // of keys row0 + n + 8 i
#pragma unroll 1
  for (int c0 = 0; c0 < p.queries; c0 += kScan) {
    // a thread's query row: sequence, token, head of the group
    const int c = c0 + threadIdx.x, f = p.by_per.div(c), in = c - f * p.m * p.group, tok = p.by_group.div(in);
    const int seq = b * p.fan + f, hq = h * p.group + in - tok * p.group;
    const bool counts_here = c < p.queries && (!p.n_new || tok < p.n_new[seq]);
    const uint32_t mine = __ballot_sync(0xffffffffu, counts_here);
    if (c0) __syncthreads();                      // the last ones are worked off
    if (lane == 0) counts[warp] = __popc(mine);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i == warp) before = total;
      total += counts[i];
    }
    if (counts_here) {
      const int i = before + __popc(mine & ((1u << lane) - 1));
      at[i] = seq * p.qb + hq * p.qh + tok * p.qm;
      lse_at[i] = (seq * p.hq + hq) * p.m + tok;
    }
    __syncthreads();
    if (row0 >= p.rows) continue;
    auto load = [&](int r0) {
      Queries q;
      const int r = r0 + n;
#pragma unroll
      for (int j = 0; j < 4; ++j) q.x[j] = make_uint4(0, 0, 0, 0);
      q.neg = -INFINITY;
      if (r < total) {
        const float l = p.lse[lse_at[r]];
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) q.x[j] = row[4 * j + t];
        q.neg = l == -INFINITY ? l : -l * kLog2e;
      }
      return q;
    };
    Queries next = load(part * kQueries);
#pragma unroll 1
    for (int r0 = part * kQueries; r0 < total; r0 += p.split * kQueries) {
      const Queries q = next;
      next = load(r0 + p.split * kQueries);
      float d[2][4] = {};
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 &u = a[2 * i][j], &v = a[2 * i + 1][j];
          mma(d[i], u.x, v.x, u.y, v.y, q.x[j].x, q.x[j].y);
          mma(d[i], u.z, v.z, u.w, v.w, q.x[j].z, q.x[j].w);
        }
      // columns 2 t and 2 t + 1 are the queries of lanes 8 t and 8 t + 4
      const float n0 = __shfl_sync(0xffffffffu, q.neg, 8 * t), n1 = __shfl_sync(0xffffffffu, q.neg, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float w0 = n0 == -INFINITY ? 0.f : ex2(fmaf(d[i][2 * k], p.scale2, n0));
          const float w1 = n1 == -INFINITY ? 0.f : ex2(fmaf(d[i][2 * k + 1], p.scale2, n1));
          sum[2 * i + k] += w0 + w1;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
  }
  if (t == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][n + 8 * i] = sum[i];
  }
  if (p.split > 1) __syncthreads();
  else __syncwarp();
  const int row = row0 + lane;
  if (part == 0 && row < p.rows) {
    float all = sums[warp][lane];
    for (int i = 1; i < p.split; ++i) all += sums[warp + i][lane];
    p.score[(long long)unit * p.cap + row] += all;
  }
  if (p.n_new && p.err && blockIdx.x == 0 && h == 0)
    for (int f = threadIdx.x; f < p.fan; f += blockDim.x) {
      const int c = p.n_new[b * p.fan + f];
      if (c < 0 || c > p.m) raise_device_error(p.err, kDevBadIndex);
    }
}

// The rows of a block behind the kept ones, with their positions and given scores: a warp per row.
constexpr int kAppendWarps = 8;
__global__ void __launch_bounds__(kAppendWarps * 32) append_given_kernel(const __grid_constant__ GroupParams P) {
  pdl_wait();
  const Shape& s = P.s;
  const LayerPtrs& L = P.L[0];
  const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31, bh = blockIdx.y;
  if (t >= s.m) return;
  const size_t from = (size_t)bh * s.m + t, to = (size_t)bh * s.cap + s.k + t;
  constexpr int kPieces = kHeadDim * 2 / 16;      // of K, and of V
  const bool value = lane >= kPieces;
  const uint4* src = static_cast<const uint4*>(value ? L.v_in : L.k_in) + from * kPieces;
  uint4* dst = static_cast<uint4*>(value ? L.vst : L.kst) + to * kPieces;
  dst[lane & (kPieces - 1)] = src[lane & (kPieces - 1)];
  if (lane == 0) {
    L.score_st[to] = L.new_score[(size_t)bh * s.new_stride + t];
    L.pos_st[to] = L.pos_in ? L.pos_in[(size_t)(bh / s.heads) * s.m + t] : (int32_t)(s.offset + t);
  }
}

bool multiple(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

cudaError_t launch_append_given(const GroupParams& P, cudaStream_t st) {
  return launch_pdl(append_given_kernel, dim3((P.s.m + kAppendWarps - 1) / kAppendWarps, P.s.batch * P.s.heads),
                    dim3(kAppendWarps * 32), 0, st, nullptr, P);
}

}  // namespace evict

using namespace evict;

extern "C" int evict_weigh(evict_handle* h, const evict_rows* q, int batch, int m, const float* lse, const int32_t* n_new,
                           float scale, void* stream) {
  if (!h || !q) return fail(EVICT_EINVAL, "handle and q must not be NULL");
  if (h->cfg.method != EVICT_ATTENTION) return fail(EVICT_EINVAL, "only scores that are accumulated attention weights can be added to");
  if (batch < 0 || m < 0) return fail(EVICT_EINVAL, "batch and m must be >= 0 (got %d, %d)", batch, m);
  if (batch % h->cfg.batch) return fail(EVICT_EINVAL, "batch (%d) must be a multiple of the cache's (%d)", batch, h->cfg.batch);
  if (q->heads < 1 || q->heads % h->cfg.n_kv_heads)
    return fail(EVICT_EINVAL, "q's heads (%d) must be a multiple of the cache's (%d)", q->heads, h->cfg.n_kv_heads);
  if (!std::isfinite(scale)) return fail(EVICT_EINVAL, "scale must be finite");
  if (!multiple(lse, 4) || !multiple(n_new, 4)) return fail(EVICT_EINVAL, "lse and n_new must be 4-byte aligned");
  if ((long long)batch * m >= (1ll << 30) || (long long)batch * m * q->heads >= (1ll << 30))
    return fail(EVICT_ELIMIT, "batch * heads * m is 2^30 or more");
  if (batch == 0 || m == 0 || h->n_kept == 0) return EVICT_OK;
  if (!q->data || !lse) return fail(EVICT_EINVAL, "q and lse must not be NULL");
  if (!multiple(q->data, 16) || q->stride_b % 8 || q->stride_h % 8 || q->stride_m % 8)
    return fail(EVICT_EINVAL, "q: addresses and strides must be multiples of 16 bytes");
  WeighParams p = {};
  p.k = h->kst;
  p.score = h->score_st;
  p.cap = h->cap;
  p.rows = h->n_kept;
  p.heads = h->cfg.n_kv_heads;
  p.q = q->data;
  p.qb = q->stride_b, p.qh = q->stride_h, p.qm = q->stride_m;
  p.lse = lse;
  p.n_new = n_new;
  p.fan = batch / h->cfg.batch;
  p.m = m;
  p.hq = q->heads;
  p.group = q->heads / p.heads;
  p.queries = p.fan * m * p.group;
  p.by_heads = Divisor(p.heads);
  p.by_per = Divisor(m * p.group);
  p.by_group = Divisor(p.group);
  p.scale2 = (scale == 0.f ? 0.08838834764831845f : scale) * kLog2e;
  p.err = h->err;
  int dev, sms;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "looking up the device");
  // warps for the same keys: as many as there is room for, while each has a tile of queries
  const int units = h->cfg.batch * p.heads;
  const long long key_warps = (long long)units * ((p.rows + kKeys - 1) / kKeys);
  p.split = 1;
  while (p.split < kWarps && key_warps * p.split < 2ll * kWarps * sms && p.split * kQueries < p.queries) p.split *= 2;
  const int keys_cta = kKeys * (kWarps / p.split);
  if (const unsigned long long id = capture_of(static_cast<cudaStream_t>(stream))) h->captured = id;
  e = launch_pdl(weigh_kernel, dim3((p.rows + keys_cta - 1) / keys_cta, units), dim3(kWarps * 32), 0,
                 static_cast<cudaStream_t>(stream), nullptr, p);
  if (e != cudaSuccess) return cuda_fail(e, "weigh kernel launch");
  g_launches.fetch_add(1);
  return EVICT_OK;
}
