// Attention of a batch over a shared prefix and its own pages.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max)
// over the rows a query sees, in one pass over K and V with a running maximum
// and sum; logits are kept in base 2 (scale * log2 e), so p = 2^(x - m).
//
// attend_kernel: persistent, one CTA per SM. Units of up to 16 query rows go to
// CTAs that work as attend_few.cuh says, units of more to CTAs that work as
// attend_wide.cuh says, side by side. The lengths live on the device, so the
// SMs that each kind gets, and the shares of its CTAs, are found there: every
// CTA sums the work of all units, by one block scan.
//
// attend_join_kernel: a warp per output row merges the partial results of the
// row's units, in the order of their slots.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "api_internal.h"
#include "attend.h"
#include "attend.cuh"
#include "attend_few.cuh"
#include "attend_wide.cuh"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "rotary.h"
#include "tcgen05.cuh"

namespace evict {
namespace {

constexpr int kThreads = kWarps * 32;
constexpr int kSmem = 1024 + (kFewSmem > kWideSmem ? kFewSmem : kWideSmem);

__global__ void __launch_bounds__(kThreads, 1) attend_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  __shared__ FewShared few;
  __shared__ WideShared wide;
  __shared__ ScanShared scan;
  unsigned char* smem = reinterpret_cast<unsigned char*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  const bool may_wide = p.wide.blocks() > 0;
  if (p.few.blocks() > 0) few_setup(few);
  if (may_wide) wide_setup(wide);
  if (threadIdx.x >= kThreads - 32) prefetch_maps(p, threadIdx.x & 31);
  pdl_wait();
  const Place at = find_place<kThreads, kWarps>(p, scan);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (at.wide) {
    if (at.first < at.shares.count)
      wide_rows(p, wide, scan, at.shares.begin(at.first + 1) - at.shares.begin(at.first), smem);
  } else {
    few_rows(p, few, scan, at, tc::smem_u32(smem));
  }
  if (may_wide) wide_teardown(wide);
}

// Partial results of one output row in one unit: `count` of them, the first at row `first`, the others
// `step` rows apart behind it, and all but the first `back` rows before that. `twice`: each is two, half a
// slot apart (the wide kernel's two groups took turns).
struct Parts {
  const float2* ml;
  const float* o;
  long long first;
  int count, step, back, twice;
  __device__ size_t at(int k) const {
    const int i = k >> twice;
    return first + (long long)i * step - (i ? back : 0) + (twice ? (k & 1) * (step >> 1) : 0);
  }
  __device__ int parts() const { return count << twice; }
};

// Row r of block e and head h; twice: see Parts.
__device__ __forceinline__ Parts find_parts(const AttendParams& p, const WorkSet& set, int e, int h, int r, int twice) {
  const int g0 = set.base[e], per = p.by_hkv.div(set.base[e + 1] - g0), steps = per - set.entry;
  const Shares shares(set);
  const int g = g0 + h * per + set.entry;
  const int c0 = shares.of(g), c1 = shares.of(g + steps - 1), unit = e * p.hkv + h;
  return Parts{set.part_ml, set.part_o, set.slot_row(unit, c0) + r, c1 - c0 + 1, set.rows_of(unit), 0, twice};
}

constexpr int kJoinWarps = 8;

// One output row's running merge: lane l holds columns 4 l .. 4 l + 3.
struct Merge {
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float2 ml, float4 v) {
    const float to = fmaxf(top, ml.x), f = weight_of(top, to), w = weight_of(ml.x, to);
    top = to;
    sum = sum * f + ml.y * w;
    acc.x = acc.x * f + v.x * w;
    acc.y = acc.y * f + v.y * w;
    acc.z = acc.z * f + v.z * w;
    acc.w = acc.w * f + v.w * w;
  }
  // parts first, first + step, ... in this order, four of them in flight
  __device__ __forceinline__ void add_parts(const Parts& x, int first, int step) {
    const int lane = threadIdx.x & 31, n = x.parts();
#pragma unroll 1
    for (int k = first; k < n; k += 4 * step) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k + i * step < n) {
          const size_t at = x.at(k + i * step);
          ml[i] = x.ml[at];
          v[i] = reinterpret_cast<const float4*>(x.o + at * kHeadDim)[lane];
        }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k + i * step < n) add(ml[i], v[i]);
    }
  }
  __device__ __forceinline__ void write(const AttendParams& p, int b, int t, int hq, bool sees) const {
    const int lane = threadIdx.x & 31;
    const float inv = sees ? 1.f / sum : 0.f;     // a query that sees no row: zeros
    const uint2 y = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + (long long)b * p.ob + (long long)hq * p.oh +
                              (long long)t * p.om + 4 * lane) = y;
    if (p.lse && lane == 0)
      p.lse[((long long)b * p.hq + hq) * p.m + t] = sees ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  }
};

// Every output row: the parts of its prefix unit and of its own. kSplit warps share a row's parts
// (few rows have many parts each, and one warp would wait for memory part after part) and their
// results meet in shared memory, in the order of the warps.
template <int kSplit>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) attend_join_kernel(const __grid_constant__ AttendParams p) {
  __shared__ float4 acc[kJoinWarps][32];
  __shared__ float2 ml[kJoinWarps];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % kSplit;
  const int row = blockIdx.x * (kJoinWarps / kSplit) + warp / kSplit;
  const bool in = row < p.batch * p.hq * p.m;
  const int bh = in ? p.by_m.div(row) : 0, t = row - bh * p.m, b = p.by_hq.div(bh), hq = bh - b * p.hq;
  const Seq q = sequence(p, b, in && !p.pages && t == 0 && hq == 0 && lane == 0 && part == 0);
  const bool real = in && t < q.n;
  Merge m;
  bool sees = false;
  if (real) {
    const int h = p.by_group.div(hq), g = hq - h * p.group;
#pragma unroll 1
    for (int part_of = 0; part_of < 2; ++part_of) {                // the prefix's rows, its own
      int r = t * p.group + g, all = q.n * p.group, s = b;
      if (part_of == 0) {
        if (!p.fan) continue;
        s = p.by_fan.div(b);
        const int before = tokens_before(p, s * p.fan);
        r += (tokens_before(p, b) - before) * p.group;
        all = (tokens_before(p, (s + 1) * p.fan) - before) * p.group;
      } else if (q.len - q.n + t < 0 || q.len == 0) {
        continue;
      }
      const bool wide = part_of == 0 ? p.wide.prefixes > 0 : p.wide.seqs > 0;
      const WorkSet& set = wide ? p.wide : p.few;
      const int rows = wide ? kWideRows : kRows, tile = wide ? r / kWideRows : r / kRows;
      const int e = part_of == 0 ? s * set.prefix_tiles + tile : set.prefixes * set.prefix_tiles + s * set.seq_tiles + tile;
      m.add_parts(find_parts(p, set, e, h, r - tile * rows, wide && all - tile * rows <= kWideRows / 2), part, kSplit);
      sees = true;
    }
  }
  if constexpr (kSplit > 1) {
    if (part > 0) {
      acc[warp][lane] = m.acc;
      if (lane == 0) ml[warp] = make_float2(m.top, m.sum);
    }
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int i = 1; i < kSplit; ++i) m.add(ml[warp + i], acc[warp + i][lane]);
  }
  if (real) m.write(p, b, t, hq, sees);
}

// Joint units: only those that two or more CTAs share have parts to merge. Block (c, y) takes eight
// rows of the unit that share c + 1 begins inside, where that is the first share to begin inside it.
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_split_kernel(const __grid_constant__ AttendParams p) {
  pdl_wait();
  const WorkSet& set = p.wide;
  const Shares shares(set);
  const int c = blockIdx.x + 1;
  if (c >= shares.count) return;
  const int2 at = set.start[c];
  Block k;
  load_block<kWideRows, kWideTokens>(p, set, at.x, k);
  const int per = k.steps + set.entry, h = at.y / per, r = at.y - h * per - set.entry;
  if (r <= 0) return;                             // the share begins with the unit
  const int first = shares.begin(c) - r;          // the unit's first step
  if (c > 1 && shares.begin(c - 1) > first) return;
  const int c1 = shares.of(first + k.steps - 1), row = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  const QueryRow q = query_row<kWideRows>(p, set, k, row);
  if (!q.real) return;
  Merge m;
  m.add_parts(Parts{set.part_ml, set.part_o, (long long)(2 * (c - 1) + 1) * kWideRows + row, c1 - (c - 1) + 1, 2 * kWideRows,
                    kWideRows, 0}, 0, 1);
  m.write(p, q.b, q.t, h * p.group + q.g, k.pre > 0 || k.len - k.n + q.t >= 0);
}

// Boxes of `rows_box` rows of `halves` halves of 64 elements, each row 128 bytes, 128-byte swizzle.
bool encode_boxes(CUtensorMap* tm, const void* base, int rows, int heads, long long head_stride, int planes,
                  long long plane_stride, int rows_box, int halves) {
  const cuuint64_t dims[5] = {64, (cuuint64_t)rows, 2, (cuuint64_t)heads, (cuuint64_t)planes};
  const cuuint64_t strides[4] = {(cuuint64_t)kHeadDim * 2, 128, (cuuint64_t)head_stride * 2, (cuuint64_t)plane_stride * 2};
  const cuuint32_t box[5] = {64, (cuuint32_t)rows_box, (cuuint32_t)halves, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return encode_tiled()(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool multiple(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Which kernel takes which units. Times are of whole calls with 32 query and 8 KV heads.
//
// A prefix is the few-row kernel's where its queries fill at most two tiles of 16 rows and reading it
// for each tile is little work: then the start counts, and the wide kernel's is longer. One tile (16
// rows) over 1,024 / 2,048 / 4,096 / 16,384 rows: 12.1 / 14.0 / 17.6 / 28.3 us, wide 15.2 / 15.8 /
// 16.2 / 22.0; two tiles (32 rows) over 512 / 1,024 / 2,048: 11.5 / 12.8 / 15.3, wide 15.3 / 15.4 / 16.2.
constexpr int kFewTiles = 2, kFewPrefix = 2048;
// Own rows are the few-row kernel's up to two tiles: 32 sequences of 1,024 rows with 20 / 32 query
// rows each 42 / 45 us, wide 50 / 52; with 40 / 64 rows 56 / 89 us, wide 54 / 57.
constexpr int kOwnWideFrom = kFewTiles * kRows + 1;
// Sequences of more query rows than these take the prefix along in units of their own (joint: no
// partial results to merge) where the prefix is short or they fill tiles of 256 rows by three
// quarters; otherwise the sequences' rows share the prefix's tiles. 16 sequences behind 1,024 rows,
// 160 / 320 rows each: joint 46 / 73 us, else 49 / 102; behind 16,384 rows, 160 / 208 / 320 / 512
// rows each: joint 227 / 232 / 431 / 439, else 183 / 248 / 352 / 598.
constexpr int kJointFrom = 128, kJointPrefix = 2048;

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  int dev, sms;
  WorkSet few, wide;        // counts, and offsets into the workspace in place of pointers
  size_t bytes;
};

// Room for a kernel's blocks and partial results of units of up to pre_rows and own_rows rows; sets the
// set's pointers (from a null base). Wide units of up to half a tile's rows are two groups' that take
// turns, and leave two rows for each of theirs.
void lay_out(WorkSet& s, bool wide, int kv_heads, int pre_rows, int own_rows, size_t& off) {
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += round256(bytes);
    return at;
  };
  if (s.blocks() == 0) return;
  auto rows_of = [&](int rows) {
    return !wide ? std::min(rows, kFewRows) : rows > kWideRows / 2 ? kWideRows : 2 * rows;
  };
  s.pre_units = s.prefixes * s.prefix_tiles * kv_heads;
  s.pre_rows = rows_of(pre_rows);
  s.own_rows = rows_of(own_rows);
  size_t rows = 0;                                // of all slots
  if (s.joint) {
    rows = 2 * (size_t)s.max_shares * kWideRows;
  } else {
    if (s.prefixes) rows = ((size_t)s.pre_units + s.max_shares) * s.pre_rows;
    s.own_at = (long long)rows;
    if (s.seqs) rows += ((size_t)s.seqs * s.seq_tiles * kv_heads + s.max_shares) * s.own_rows;
  }
  s.base = reinterpret_cast<int*>(take((size_t)(s.blocks() + 2) * sizeof(int)));
  s.start = reinterpret_cast<int2*>(take((size_t)s.max_shares * sizeof(int2)));
  s.part_ml = reinterpret_cast<float2*>(take(rows * sizeof(float2)));
  s.part_o = reinterpret_cast<float*>(take(rows * kHeadDim * sizeof(float)));
}
template <typename T>
void rebase(T*& x, char* base) { x = reinterpret_cast<T*>(base + reinterpret_cast<size_t>(x)); }
void rebase(WorkSet& s, char* base) {
  rebase(s.base, base);
  rebase(s.start, base);
  rebase(s.part_ml, base);
  rebase(s.part_o, base);
}

constexpr size_t kWorkHead = 256;                 // an error word, for callers without one
// Boxes (steps) that a share has at least: fewer would leave more partial results to merge than rows to
// read. A step of 4 sequences behind 1,024 rows 11.8 us with two boxes, 12.2 with one, 13.4 with four;
// 16 sequences behind 2,048 rows 16.8 us with three steps, 18.1 with one and 19.9 with six.
constexpr int kFewMinBoxes = 2;
constexpr int kWideMinSteps = 3;
// Clocks of an SM, side by side, for a box of 16 rows, and for a step of 128 rows with two groups of
// query rows at it, or with the groups taking turns. Fitted to when the two kinds end: 128 sequences
// behind 16,384 rows take 75 us (with kWideCostTwo 4,000 80, with 4,700 79), 32 sequences' draft tokens
// behind 8,192 rows 41 (43, 42); four answers to each of eight prompts 32 (with kWideCostAlt 2,400 37,
// with 2,800 35), a decode step of 32 sequences 27 (27, 26).
constexpr int kFewCost = 300, kWideCostTwo = 4400, kWideCostAlt = 2600;
// What a unit's start costs beside: a warp or CTA fetches its queries and leaves the last unit's results.
// (Counted as nothing: 16 sequences behind 2,048 rows 19.4 us instead of 16.8, 256 new rows of each of
// eight sequences 60.7 instead of 57.3.)
constexpr int kFewEntry = 2, kWideEntry = 3;

int check_sizes(const evict_attention* a) {
  if (!a) return fail(EVICT_EINVAL, "the arguments are NULL");
  if (a->batch < 0 || a->m < 0) return fail(EVICT_EINVAL, "batch and m must be >= 0 (got %d, %d)", a->batch, a->m);
  if (a->n_q_heads < 1 || a->n_kv_heads < 1 || a->n_q_heads % a->n_kv_heads)
    return fail(EVICT_EINVAL, "n_q_heads (%d) must be a multiple of n_kv_heads (%d)", a->n_q_heads, a->n_kv_heads);
  if (a->batch > EVICT_MAX_ATTEND_BATCH)
    return fail(EVICT_ELIMIT, "batch %d is above %d", a->batch, EVICT_MAX_ATTEND_BATCH);
  if ((long long)a->batch * a->m >= (1ll << 30) || (long long)a->batch * a->m * a->n_q_heads >= (1ll << 30))
    return fail(EVICT_ELIMIT, "batch * n_q_heads * m is 2^30 or more");
  if (a->n_prefix < 0 || a->n_prefix > (1 << 30)) return fail(EVICT_EINVAL, "n_prefix must be in [0, 2^30]");
  if (a->n_prefix > 0 && (a->prefix_batch < 1 || a->batch % a->prefix_batch))
    return fail(EVICT_EINVAL, "prefix_batch (%d) must divide batch (%d)", a->prefix_batch, a->batch);
  return EVICT_OK;
}

// Sizes alone decide: lens and n_new are the device's.
int make_plan(const evict_attention* a, Plan* out) {
  if (const int rc = check_sizes(a)) return rc;
  Plan& P = *out;
  P = Plan();
  if (a->batch == 0 || a->m == 0) return EVICT_OK;
  const int group = a->n_q_heads / a->n_kv_heads;
  const bool pre = a->n_prefix > 0;

  const int own_rows = a->m * group, pre_rows = pre ? own_rows * (a->batch / a->prefix_batch) : 0;
  const int wide_tiles = (own_rows + kWideRows - 1) / kWideRows, few_tiles = (pre_rows + kRows - 1) / kRows;
  if (own_rows > kJointFrom && (pre || a->pages) &&
      (a->n_prefix <= kJointPrefix || 4ll * own_rows > 3ll * kWideRows * wide_tiles)) {
    P.wide.joint = 1;
    P.wide.seqs = a->batch;
  } else {
    const bool few = few_tiles <= kFewTiles && (long long)few_tiles * a->n_prefix * a->prefix_batch <= kFewPrefix;
    if (pre) (few ? P.few : P.wide).prefixes = a->prefix_batch;
    if (a->pages) (own_rows >= kOwnWideFrom ? P.wide : P.few).seqs = a->batch;
  }
  const long long seq_tokens = a->pages ? (long long)a->pages->table_width * a->pages->page_size : 0;
  auto tiles = [&](WorkSet& s, int rows, int tokens) {
    s.prefix_tiles = (pre_rows + rows - 1) / rows;
    s.seq_tiles = (own_rows + rows - 1) / rows;
    s.by_prefix_tiles = Divisor(s.prefix_tiles);
    s.by_seq_tiles = Divisor(s.seq_tiles);
    const long long pre_steps = (a->n_prefix + tokens - 1) / tokens, seq_steps = (seq_tokens + tokens - 1) / tokens + 1;
    const long long work = ((long long)s.prefixes * s.prefix_tiles * pre_steps +
                            (long long)s.seqs * s.seq_tiles * (seq_steps + (s.joint ? pre_steps : 0)) + 4ll * s.blocks()) * a->n_kv_heads;
    return work < (1ll << 31) && ((long long)s.blocks() + 1) * a->n_kv_heads < (1ll << 30);
  };
  if (!tiles(P.few, kRows, kBoxTokens) || !tiles(P.wide, kWideRows, kWideTokens))
    return fail(EVICT_ELIMIT, "the batch's heads and rows (to the tables' width) are too many for one call");
  cudaError_t e = cudaGetDevice(&P.dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&P.sms, cudaDevAttrMultiProcessorCount, P.dev);
  if (e != cudaSuccess) return cuda_fail(e, "looking up the device");
  P.few.workers = kWarps;
  P.few.max_shares = P.sms * kWarps;
  P.few.min_steps = kFewMinBoxes;
  P.few.cost = kFewCost;
  P.few.entry = kFewEntry;
  P.wide.workers = 1;
  P.wide.max_shares = P.sms;
  P.wide.min_steps = kWideMinSteps;
  P.wide.cost = (P.wide.prefixes ? pre_rows : own_rows) > 128 ? kWideCostTwo : kWideCostAlt;
  P.wide.entry = kWideEntry;
  size_t off = kWorkHead + round256((size_t)(a->batch + 1) * sizeof(int));
  lay_out(P.few, false, a->n_kv_heads, pre_rows, own_rows, off);
  lay_out(P.wide, true, a->n_kv_heads, pre_rows, own_rows, off);
  P.bytes = off;
  return EVICT_OK;
}

int check_rows(const evict_rows& x, int heads, const char* name) {
  if (!x.data) return fail(EVICT_EINVAL, "%s must not be NULL", name);
  if (x.heads != heads) return fail(EVICT_EINVAL, "%s has %d heads, not %d", name, x.heads, heads);
  if (!multiple(x.data, 16) || x.stride_b % 8 || x.stride_h % 8 || x.stride_m % 8)
    return fail(EVICT_EINVAL, "%s: addresses and strides must be multiples of 16 bytes", name);
  if (x.stride_b < 0 || x.stride_h < 0 || x.stride_m < 0) return fail(EVICT_EINVAL, "%s: strides must not be negative", name);
  return EVICT_OK;
}

// The kernel's dynamic shared memory, allowed once for each device.
cudaError_t allow_smem(int dev) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(attend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

}  // namespace
}  // namespace evict

using namespace evict;

extern "C" int evict_shared_attention_workspace(const evict_attention* a, size_t* bytes) {
  if (!bytes) return fail(EVICT_EINVAL, "bytes is NULL");
  Plan plan;
  const int rc = make_plan(a, &plan);
  if (rc) return rc;
  *bytes = plan.bytes;
  return EVICT_OK;
}

extern "C" int evict_shared_attention(const evict_attention* a) {
  if (!a) return fail(EVICT_EINVAL, "the arguments are NULL");
  int rc;
  if (a->pages) {
    if ((rc = check_pages(a->pages))) return rc;
    if (a->pages->dtype != EVICT_BF16) return fail(EVICT_EINVAL, "attention reads bf16 pages only");
    if (a->pages->n_kv_heads != a->n_kv_heads)
      return fail(EVICT_EINVAL, "the pages hold %d KV heads, the call %d", a->pages->n_kv_heads, a->n_kv_heads);
  }
  if (!std::isfinite(a->scale)) return fail(EVICT_EINVAL, "scale must be finite");
  if (!multiple(a->n_new, 4) || !multiple(a->lse, 4) || !multiple(a->error, 4))
    return fail(EVICT_EINVAL, "n_new, lse and error must be 4-byte aligned");
  if (a->n_prefix > 0) {
    if (!a->prefix_k || !a->prefix_v) return fail(EVICT_EINVAL, "prefix_k and prefix_v must not be NULL");
    if (!multiple(a->prefix_k, 16) || !multiple(a->prefix_v, 16) || a->prefix_stride_b % 8 || a->prefix_stride_h % 8 ||
        a->prefix_stride_b < 0 || a->prefix_stride_h < 0)
      return fail(EVICT_EINVAL, "the prefix must be 16-byte aligned, with strides that are multiples of 8");
    if ((a->prefix_batch > 1 && a->prefix_stride_b == 0) || (a->n_kv_heads > 1 && a->prefix_stride_h == 0))
      return fail(EVICT_EINVAL, "prefixes or KV heads in one place (stride 0): say prefix_batch or n_kv_heads 1");
  }
  if (a->batch > 0 && a->m > 0)
    if ((rc = check_rows(a->q, a->n_q_heads, "q")) || (rc = check_rows(a->out, a->n_q_heads, "out"))) return rc;
  if ((rc = check_sizes(a))) return rc;
  if (a->batch > 0 && a->m > 0) {
    if (a->out.data == a->q.data) return fail(EVICT_EINVAL, "out must not be q: queries are read while results are written");
    if (rows_overlap(a->out, a->batch, a->m)) return fail(EVICT_EINVAL, "out: rows lie on top of each other");
  }
  Plan plan;
  if ((rc = make_plan(a, &plan))) return rc;
  if (a->batch == 0 || a->m == 0) return EVICT_OK;
  if (!a->workspace || !multiple(a->workspace, 256)) return fail(EVICT_EINVAL, "workspace must be 256-byte aligned");
  if (a->workspace_bytes < plan.bytes)
    return fail(EVICT_EINVAL, "workspace has %zu bytes, the call needs %zu", a->workspace_bytes, plan.bytes);
  if (!encode_tiled()) return fail(EVICT_ECUDA, "cuTensorMapEncodeTiled is not available from the driver");

  AttendParams P;
  memset(&P, 0, sizeof(P));
  char* ws = static_cast<char*>(a->workspace);
  P.err = a->error ? a->error : reinterpret_cast<int*>(ws);
  P.tok_base = reinterpret_cast<int*>(ws + kWorkHead);
  rebase(plan.few, ws);
  rebase(plan.wide, ws);
  P.q = a->q.data;
  P.qb = a->q.stride_b, P.qh = a->q.stride_h, P.qm = a->q.stride_m;
  P.out = a->out.data;
  P.ob = a->out.stride_b, P.oh = a->out.stride_h, P.om = a->out.stride_m;
  P.out_sectors = multiple(a->out.data, 32) && a->out.stride_b % 16 == 0 && a->out.stride_h % 16 == 0 && a->out.stride_m % 16 == 0;
  P.lse = a->lse;
  P.batch = a->batch, P.m = a->m, P.hq = a->n_q_heads, P.hkv = a->n_kv_heads;
  P.group = a->n_q_heads / a->n_kv_heads;
  if (a->n_prefix > 0) {
    P.prefix_batch = a->prefix_batch;
    P.fan = a->batch / a->prefix_batch;
    P.n_prefix = a->n_prefix;
  }
  P.by_m = Divisor(P.m);
  P.by_hq = Divisor(P.hq);
  P.by_hkv = Divisor(P.hkv);
  P.by_group = Divisor(P.group);
  P.by_fan = Divisor(P.fan);
  P.scale2 = (a->scale == 0.f ? 0.08838834764831845f : a->scale) * kLog2e;
  P.n_new = a->n_new;
  const evict_pages* g = a->pages;
  if (g) {
    P.pages = 1;
    P.table = g->table;
    P.table_stride = g->table_stride ? g->table_stride : g->table_width;
    P.table_width = g->table_width;
    P.page_shift = __builtin_ctz((unsigned)g->page_size);
    P.n_pages = g->n_pages;
    P.lens = g->lens;
    P.page_k = g->k;
    P.page_v = g->v;
    P.page_stride = g->page_stride ? g->page_stride : (long long)g->n_kv_heads * g->page_size * kHeadDim;
  }
  // The two kinds' boxes: 16 whole rows, or up to 128 rows of one half.
  auto encode = [&](bool wide, const WorkSet& s, CUtensorMap (&pre)[2], CUtensorMap (&own)[2]) {
    if (s.prefixes || (s.joint && P.fan)) {
      // a dimension of extent 1 is never stepped over, but its stride still has to be one the encoder takes
      const long long hs = P.hkv > 1 ? a->prefix_stride_h : (long long)P.n_prefix * kHeadDim;
      const long long bs = P.prefix_batch > 1 ? a->prefix_stride_b : P.hkv * hs;
      for (int v = 0; v < 2; ++v)
        if (!encode_boxes(&pre[v], v ? a->prefix_v : a->prefix_k, P.n_prefix, P.hkv, hs, P.prefix_batch, bs,
                          wide ? kWideTokens : kBoxTokens, wide ? 1 : 2))
          return fail(EVICT_EINVAL, "the prefix has sizes or strides beyond a tensor map's");
    }
    if (s.seqs && g) {
      P.box_rows = std::min(g->page_size, kWideTokens);
      for (int v = 0; v < 2; ++v)
        if (!encode_boxes(&own[v], v ? g->v : g->k, g->page_size, P.hkv, (long long)g->page_size * kHeadDim, g->n_pages,
                          P.page_stride, wide ? P.box_rows : kBoxTokens, wide ? 1 : 2))
          return fail(EVICT_EINVAL, "the pages have sizes or strides beyond a tensor map's");
    }
    return (int)EVICT_OK;
  };
  P.few = plan.few;
  P.wide = plan.wide;
  P.sms = plan.sms;
  // a stream is of one kind, so either kind's maps have a place of their own
  if ((rc = encode(false, P.few, P.few_pre, P.few_own)) || (rc = encode(true, P.wide, P.wide_pre, P.wide_own))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(a->stream);
  cudaError_t e = allow_smem(plan.dev);
  if (e != cudaSuccess) return cuda_fail(e, "attention kernel attribute");
  if (P.few.blocks() + P.wide.blocks() > 0) {
    if ((e = launch_pdl(attend_kernel, dim3(plan.sms), dim3(kThreads), kSmem, st, nullptr, P)) != cudaSuccess)
      return cuda_fail(e, "attention kernel launch");
    g_launches.fetch_add(1);
  }
  if (plan.wide.joint) {
    if (plan.sms > 1)
      e = launch_pdl(attend_join_split_kernel, dim3(plan.sms - 1, kWideRows / kJoinWarps), dim3(kJoinWarps * 32), 0, st, nullptr, P);
  } else {
    // four warps a row while the rows are few (4 sequences x 12 heads 11.8 us, with one 15.3; 48 x 32 heads
    // 34.5 us with one, with four 39.1)
    const int rows = a->batch * a->n_q_heads * a->m, split = rows <= plan.sms * kJoinWarps ? 4 : 1;
    const dim3 grid((rows * split + kJoinWarps - 1) / kJoinWarps), block(kJoinWarps * 32);
    e = split == 4 ? launch_pdl(attend_join_kernel<4>, grid, block, 0, st, nullptr, P)
                   : launch_pdl(attend_join_kernel<1>, grid, block, 0, st, nullptr, P);
  }
  g_launches.fetch_add(1);
  return e == cudaSuccess ? EVICT_OK : cuda_fail(e, "attention kernel launch");
}
