// Position rotation of query and key rows, and the append of a batch's own
// rows to pages with the rotation applied on the way.
//
// Pair i of a row turns by a = pos[axis(i)] * w_i:
//     (x, y) -> s (x cos a - y sin a, x sin a + y cos a).
//
// Angles. In fp32 a product pos * w loses the angle itself at far positions
// (position 10^5 at w = 1: an error of 0.004 radians). The tables hold
// F_i = frac(w_i / 2 pi) * 2^64 instead, so the low 64 bits of pos * F_i are
// the angle's fraction of a turn, off by at most |pos| / 2 units of 2^-64
// turns; whole turns fall off the top of the integer. Its upper 32 bits, read
// as a signed number, times 2^-31 are the angle in half turns in [-1, 1). In fp32
// whole quarters are taken off before it is rounded: within 0.42 steps of 2^-24
// radians of the angle (1.6 without).
//
// Bound: HBM, every row read once and written once. A block of 128 threads
// owns two tokens (one where they are few): each thread makes the sine and
// cosine of one angle, and they meet in shared memory. Eight threads then take
// a row (sixteen in fp32, so that they read 16-byte pieces side by side), each
// thread 8 pairs (4), and go from head to head with them in registers, in
// packed fp32 pairs. The first heads' loads leave before the angles and the
// page table are looked at: the rows' addresses need neither.
//
// Measured: 8,192 tokens of 32 bf16 heads 22.8 us (134 MB, 5.9 TB/s); 4 x 1,023
// tokens of 40 fp32 heads 27.1 us (168 MB, 6.2 TB/s); prompts of up to 2,048
// tokens of 48 heads, 219 MB, into pages 37.9 us (5.8 TB/s; 43.9 where blocks of
// padding made their angles, too, and pages were looked up behind them). With
// 256 threads and 4 tokens a block the first two took 24.3 and 28.0, with the
// loads after the angles and eight threads of an fp32 row 28 and 50.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "api_internal.h"
#include "common.cuh"
#include "launch.h"
#include "pipeline.cuh"
#include "rotary.h"

namespace evict {
namespace {

constexpr int kRowThreads = 128;
constexpr int kTokens = 2;                        // tokens of a block, at most
constexpr int kMaxTensors = 3;

struct RowTensor {
  const void* src;
  void* dst;                         // null: the pages (k or v)
  long long sb, sh, sm, db, dh, dm;  // element strides
  int begin, end;                    // its heads, counted through all tensors
  int rotate;
};

struct RowsParams {
  RotaryTable rot;                   // half = 0: nothing is rotated
  RowTensor t[kMaxTensors];
  int n_tensors, heads;
  unsigned tokens;                   // batch * m
  int per_block;                     // tokens of a block: 1 or kTokens
  int batch, m;
  const int32_t* pos;
  long long pos_base;
  int transpose;
  // pages
  char* pages[2];                    // K, V of tensors 0 and 1 where their dst is null
  long long page_stride;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* n_new;
  long long table_stride;
  int table_width, page_shift, n_pages, kv_heads;
  int* err;
};

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// The angles' sines and cosines, of `turn` as a signed fraction of 2^31 half turns. bf16 results have
// 8 bits: the special-function unit's, absolutely within 2^-21 on [-pi, pi], are far more than enough.
template <typename T>
__device__ __forceinline__ void sine_cosine(int32_t turn, float& s, float& c) {
  if constexpr (sizeof(T) == 2) {
    const float a = (float)turn * 1.4629180792671596e-9f;            // pi 2^-31
    s = __sinf(a);
    c = __cosf(a);
  } else {
    // off to the nearest quarter turn in integers first: what is left has at most 30 bits, of which fp32
    // drops five in place of seven
    const uint32_t quarters = ((uint32_t)turn + (1u << 29)) >> 30;
    float rs, rc;
    sincospif((float)(int32_t)((uint32_t)turn - (quarters << 30)) * 0x1p-31f, &rs, &rc);
    s = quarters & 1 ? rc : rs;
    c = quarters & 1 ? rs : rc;
    if (quarters & 2) s = -s;
    if ((quarters + 1) & 2) c = -c;
  }
}

// 16 bytes of a row as fp32 pairs.
template <typename T>
struct Piece {
  uint4 raw;
  __device__ __forceinline__ uint64_t get(int i) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t x = i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w;
      return (uint64_t)(x << 16) | (uint64_t)(x & 0xffff0000u) << 32;
    } else {
      return i ? (uint64_t)raw.z | (uint64_t)raw.w << 32 : (uint64_t)raw.x | (uint64_t)raw.y << 32;
    }
  }
  __device__ __forceinline__ void set(int i, uint64_t v) {
    float lo, hi;
    split_f32x2(v, lo, hi);
    if constexpr (sizeof(T) == 2) {
      uint32_t r;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
      (i == 0 ? raw.x : i == 1 ? raw.y : i == 2 ? raw.z : raw.w) = r;
    } else if (i) {
      raw.z = __float_as_uint(lo), raw.w = __float_as_uint(hi);
    } else {
      raw.x = __float_as_uint(lo), raw.y = __float_as_uint(hi);
    }
  }
};

// (x, y) of an adjacent pair -> (y, x)
__device__ __forceinline__ uint64_t swap_f32x2(uint64_t v) { return v << 32 | v >> 32; }

// kVec: 16-byte pieces (rows and strides aligned, rotary_dim a multiple of 16, so that every
// thread's 16 elements are rotated or copied as a whole); else an element at a time.
template <typename T, bool kVec, bool kPaged>
__global__ void __launch_bounds__(kRowThreads, 8) rows_kernel(const __grid_constant__ RowsParams p) {
  constexpr int kUnit = 16 / (int)sizeof(T);       // pairs of a thread
  constexpr int kLanes = kHeadDim / 2 / kUnit;     // threads of a row
  constexpr int kRows = kRowThreads / kLanes;      // rows that a block works on at a time
  constexpr int kAhead = sizeof(T) == 4 ? 2 : kPaged ? 3 : 4;   // heads of a thread in flight
  __shared__ __align__(16) float cosine[kTokens][kHeadDim / 2], sine[kTokens][kHeadDim / 2];
  pdl_wait();
  const int half = p.rot.half;
  const int u = threadIdx.x % kLanes, groups = kRows / p.per_block;
  const int own = threadIdx.x / kLanes / groups, group = threadIdx.x / kLanes - own * groups;   // token, row of its heads
  const unsigned tok = blockIdx.x * p.per_block + own;
  const int b = (int)(tok / (unsigned)p.m), t = (int)(tok - (unsigned)b * p.m);
  int n = p.m, len = 0;
  if constexpr (kPaged) {
    if (tok < p.tokens) {
      len = p.lens[b];
      if (p.n_new) {
        n = p.n_new[b];
        if ((n < 0 || n > p.m) && u == 0 && group == 0 && t == 0 && p.err) raise_device_error(p.err, kDevBadIndex);
        n = n < 0 ? 0 : n > p.m ? p.m : n;
      }
    }
  }
  const bool live = tok < p.tokens && t < n;
  if constexpr (kPaged)
    if (p.n_new && !__syncthreads_or(live)) return;            // padding

  const bool turns = kUnit * u < half;             // kVec: all of its pairs turn, or none
  // this thread's elements: at `ea` and `eb`, kUnit each
  const int ea = turns && !p.rot.adjacent ? kUnit * u : 2 * kUnit * u;
  const int eb = turns && !p.rot.adjacent ? half + kUnit * u : 2 * kUnit * u + kUnit;
  auto tensor_of = [&](int h) { return (p.n_tensors > 1 && h >= p.t[0].end) + (p.n_tensors > 2 && h >= p.t[1].end); };
  auto source = [&](int h) {
    const RowTensor& x = p.t[tensor_of(h)];
    return static_cast<const T*>(x.src) + (long long)b * x.sb + (long long)(h - x.begin) * x.sh + (long long)t * x.sm;
  };
  Piece<T> lo[kAhead], hi[kAhead];
  auto pull = [&](int first) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int h = first + j * groups;
      if (h < p.heads) {
        const T* src = source(h);
        lo[j].raw = *reinterpret_cast<const uint4*>(src + ea);
        hi[j].raw = *reinterpret_cast<const uint4*>(src + eb);
      }
    }
  };
  if constexpr (kVec)
    if (live) pull(group);
  // The token's page, its row there: looked up while the angles are made. (fp32's take sincospif's
  // registers: 12.7 us behind them, 13.6 before, for 59 MB.)
  int page = -1, row = 0;
  if constexpr (kPaged && sizeof(T) == 2) {
    if (live) {
      const int j = len - n + t;
      row = j & ((1 << p.page_shift) - 1);
      if (j >= 0 && (j >> p.page_shift) < p.table_width)
        page = p.table[(long long)b * p.table_stride + (j >> p.page_shift)];
    }
  }

  // the angles
  if ((int)threadIdx.x < p.per_block * (kHeadDim / 2)) {
    const int i = threadIdx.x / (kHeadDim / 2), f = threadIdx.x % (kHeadDim / 2);
    const unsigned at = blockIdx.x * p.per_block + i;
    float s = 0.f, c = 1.f;
    if (f < half && at < p.tokens) {
      const int ab = (int)(at / (unsigned)p.m), a = (int)(at - (unsigned)ab * p.m);
      long long ps = p.pos_base + a;
      if (p.pos) {
        ps = p.pos[((long long)p.rot.axis[f] * p.batch + ab) * p.m + a];
      } else if (kPaged) {
        const int k = p.n_new ? min(max(p.n_new[ab], 0), p.m) : p.m;
        ps = p.pos_base + (p.lens[ab] - k + a);
      }
      const int32_t turn = (int32_t)(uint32_t)(((uint64_t)ps * p.rot.freq[f]) >> 32);
      sine_cosine<T>(turn, s, c);
      c *= p.rot.scale;
      s *= p.transpose ? -p.rot.scale : p.rot.scale;
    }
    cosine[i][f] = c;
    sine[i][f] = s;
  }
  if constexpr (kPaged && sizeof(T) == 4) {
    if (live) {
      const int j = len - n + t;
      row = j & ((1 << p.page_shift) - 1);
      if (j >= 0 && (j >> p.page_shift) < p.table_width)
        page = p.table[(long long)b * p.table_stride + (j >> p.page_shift)];
    }
  }
  bool stored = true;                              // the token's page row exists
  long long at = 0;                                // its element offset in the pool (head 0)
  if constexpr (kPaged) {
    if (live) {
      stored = page >= 0 && page < p.n_pages;
      if (!stored && u == 0 && group == 0 && p.err) raise_device_error(p.err, kDevBadIndex);
      if (stored) at = (long long)page * p.page_stride + (long long)row * kHeadDim;
    }
  }
  auto target = [&](int h) -> T* {                 // null: nowhere
    const int w = tensor_of(h);
    const RowTensor& x = p.t[w];
    if (kPaged && !x.dst)
      return stored ? reinterpret_cast<T*>(p.pages[w]) + at + ((long long)(h - x.begin) * kHeadDim << p.page_shift)
                    : nullptr;
    return static_cast<T*>(x.dst) + (long long)b * x.db + (long long)(h - x.begin) * x.dh + (long long)t * x.dm;
  };
  __syncthreads();
  if (!live) return;
  // cosines and sines of pairs (2 i, 2 i + 1) of the thread's
  uint64_t co[kUnit / 2], si[kUnit / 2];
#pragma unroll
  for (int i = 0; i < kUnit / 2; i += 2) {
    const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(&cosine[own][kUnit * u + 2 * i]);
    const ulonglong2 s = *reinterpret_cast<const ulonglong2*>(&sine[own][kUnit * u + 2 * i]);
    co[i] = c.x, co[i + 1] = c.y;
    si[i] = s.x, si[i + 1] = s.y;
  }

  if constexpr (kVec) {
    for (int first = group;;) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int h = first + j * groups;
        if (h >= p.heads) break;
        if (turns && p.t[tensor_of(h)].rotate) {
          if (!p.rot.adjacent) {
#pragma unroll
            for (int i = 0; i < kUnit / 2; ++i) {
              const uint64_t x = lo[j].get(i), y = hi[j].get(i);
              lo[j].set(i, sub_f32x2(mul_f32x2(x, co[i]), mul_f32x2(y, si[i])));
              hi[j].set(i, fma_f32x2(x, si[i], mul_f32x2(y, co[i])));
            }
          } else {
            // pair i is an element pair of lo (the first half of the pairs) or of hi: (x c - y s, x s + y c)
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
              Piece<T>& e = i < kUnit / 2 ? lo[j] : hi[j];
              float c0, c1, s0, s1;
              split_f32x2(co[i / 2], c0, c1);
              split_f32x2(si[i / 2], s0, s1);
              const float c = i & 1 ? c1 : c0, s = i & 1 ? s1 : s0;
              const uint64_t v = e.get(i % (kUnit / 2));
              e.set(i % (kUnit / 2), fma_f32x2(swap_f32x2(v), pack_f32x2(-s, s), mul_f32x2(v, pack_f32x2(c, c))));
            }
          }
        }
        if (T* dst = target(h)) {
          *reinterpret_cast<uint4*>(dst + ea) = lo[j].raw;
          *reinterpret_cast<uint4*>(dst + eb) = hi[j].raw;
        }
      }
      first += kAhead * groups;
      if (first >= p.heads) break;
      pull(first);
    }
  } else {
#pragma unroll 1
    for (int h = group; h < p.heads; h += groups) {
      const T* src = source(h);
      T* dst = target(h);
      if (!dst) continue;
      const bool rotate = p.t[tensor_of(h)].rotate;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        const int f = kUnit * u + i;
        const bool rotates = f < half;
        const int i0 = rotates && !p.rot.adjacent ? f : 2 * f;
        const int i1 = rotates && !p.rot.adjacent ? f + half : 2 * f + 1;
        const T x0 = src[i0], x1 = src[i1];
        if (rotates && rotate) {
          float c0, c1, s0, s1;
          split_f32x2(co[i / 2], c0, c1);
          split_f32x2(si[i / 2], s0, s1);
          const float a = widen(x0), y = widen(x1), c = i & 1 ? c1 : c0, s = i & 1 ? s1 : s0;
          dst[i0] = narrow<T>(a * c - y * s);
          dst[i1] = narrow<T>(a * s + y * c);
        } else {
          dst[i0] = x0;
          dst[i1] = x1;
        }
      }
    }
  }
}

bool multiple(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Address and strides of a tensor, in bytes, are multiples of `bytes`.
bool rows_aligned(const evict_rows& x, int elem, size_t bytes) {
  const long long n = (long long)(bytes / elem);
  return multiple(x.data, bytes) && x.stride_b % n == 0 && x.stride_h % n == 0 && x.stride_m % n == 0;
}

int check_tensor(const evict_rows* x, int elem, const char* name) {
  if (!x || !x->data) return fail(EVICT_EINVAL, "%s must not be NULL", name);
  if (x->heads < 1) return fail(EVICT_EINVAL, "%s has %d heads", name, x->heads);
  if (!multiple(x->data, elem)) return fail(EVICT_EINVAL, "%s must be aligned to its elements", name);
  return EVICT_OK;
}

int check_output(const evict_rows* x, const evict_rows* in, int elem, const char* name) {
  if (const int rc = check_tensor(x, elem, name)) return rc;
  if (x->heads != in->heads) return fail(EVICT_EINVAL, "%s has %d heads, its input %d", name, x->heads, in->heads);
  if (x->data == in->data && (x->stride_b != in->stride_b || x->stride_h != in->stride_h || x->stride_m != in->stride_m))
    return fail(EVICT_EINVAL, "an output in place must have its input's strides");
  return EVICT_OK;
}

int check_common(int dtype, int batch, int m, const int32_t* pos) {
  if (dtype != EVICT_BF16 && dtype != EVICT_FP32) return fail(EVICT_EINVAL, "unknown dtype %d", dtype);
  if (batch < 0 || m < 0) return fail(EVICT_EINVAL, "batch and m must be >= 0 (got %d, %d)", batch, m);
  if (!multiple(pos, 4)) return fail(EVICT_EINVAL, "pos must be 4-byte aligned");
  return EVICT_OK;
}

void set_tensor(RowsParams& P, const evict_rows& x, const evict_rows* out, bool rotate) {
  RowTensor& t = P.t[P.n_tensors++];
  t.src = x.data;
  t.sb = x.stride_b, t.sh = x.stride_h, t.sm = x.stride_m;
  t.dst = out ? out->data : nullptr;
  if (out) t.db = out->stride_b, t.dh = out->stride_h, t.dm = out->stride_m;
  t.begin = P.heads;
  P.heads += x.heads;
  t.end = P.heads;
  t.rotate = rotate;
}

// Rows of all tensors, whose heads have been checked one by one: no product or sum here passes 2^63.
int check_size(int batch, int m, const evict_rows& a, const evict_rows* b, const evict_rows* c) {
  const long long tokens = (long long)batch * m, heads = (long long)a.heads + (b ? b->heads : 0) + (c ? c->heads : 0);
  if (tokens >= (1ll << 31) || heads >= (1ll << 31) || tokens * heads >= (1ll << 31))
    return fail(EVICT_ELIMIT, "batch * m * heads (%lld tokens of %lld heads): 2^31 rows or more", tokens, heads);
  return EVICT_OK;
}

int run_rows(RowsParams& P, bool vec, bool paged, int dtype, cudaStream_t st) {
  const long long tokens = (long long)P.batch * P.m;
  P.tokens = (unsigned)tokens;
  // A block a token while that is no more than two blocks an SM: a decode step of 32 sequences takes 3.2 us so, and
  // 4.8 with kTokens. With many tokens the other way round: 8,192 tokens 26.0 us with one and 22.8 with kTokens.
  P.per_block = tokens <= 2 * 152 ? 1 : kTokens;
  const dim3 grid((P.tokens + P.per_block - 1) / P.per_block);
  cudaError_t e;
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kRowThreads), 0, st, nullptr, P); };
  if (dtype == EVICT_BF16) {
    if (paged) e = vec ? go(rows_kernel<__nv_bfloat16, true, true>) : go(rows_kernel<__nv_bfloat16, false, true>);
    else e = vec ? go(rows_kernel<__nv_bfloat16, true, false>) : go(rows_kernel<__nv_bfloat16, false, false>);
  } else {
    if (paged) e = vec ? go(rows_kernel<float, true, true>) : go(rows_kernel<float, false, true>);
    else e = vec ? go(rows_kernel<float, true, false>) : go(rows_kernel<float, false, false>);
  }
  g_launches.fetch_add(1);
  return e == cudaSuccess ? EVICT_OK : cuda_fail(e, paged ? "append kernel launch" : "rotation kernel launch");
}

}  // namespace

bool rows_overlap(const evict_rows& x, int batch, int m) {
  struct Dim {
    long long n, s;
  };
  const Dim axes[3] = {{batch, x.stride_b}, {x.heads, x.stride_h}, {m, x.stride_m}};
  auto size = [](long long v) { return v < 0 ? -(__int128)v : (__int128)v; };
  Dim d[3];
  int dims = 0;
  for (const Dim& e : axes) {                     // axes to step over, by the size of their strides
    if (e.n <= 1) continue;
    if (e.s == 0) return true;
    int at = dims++;
    for (; at > 0 && size(e.s) < size(d[at - 1].s); --at) d[at] = d[at - 1];
    d[at] = e;
  }
  // ordinary layouts: each stride steps over all that the smaller ones reach
  __int128 reach = kHeadDim;
  bool nested = true;
  for (int i = 0; i < dims; ++i) {
    nested = nested && size(d[i].s) >= reach;
    reach += size(d[i].s) * (d[i].n - 1);
  }
  if (nested) return false;
  // others: two rows lie i, j, k steps apart, with less than a row between them. i and j go through the
  // shorter axes (of 2^31 rows at most some 2^21 pairs), k is what brings the third nearest.
  for (int i = dims; i < 3; ++i) d[i] = Dim{1, 1};
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.n < b.n; });
  for (long long i = 0; i < d[0].n; ++i)
    for (long long j = i ? 1 - d[1].n : 0; j < d[1].n; ++j) {
      const __int128 at = (__int128)i * d[0].s + (__int128)j * d[1].s;
      const __int128 near = -at / d[2].s;
      for (__int128 k = near - 1; k <= near + 1; ++k)
        if (k < d[2].n && -k < d[2].n && (i || j || k) && at + k * d[2].s < kHeadDim && at + k * d[2].s > -kHeadDim)
          return true;
    }
  return false;
}

int check_pages(const evict_pages* g) {
  if (!g) return fail(EVICT_EINVAL, "pages is NULL");
  if (g->dtype != EVICT_BF16 && g->dtype != EVICT_FP32) return fail(EVICT_EINVAL, "unknown dtype %d", g->dtype);
  if (g->n_pages < 1 || g->n_kv_heads < 1 || g->table_width < 1)
    return fail(EVICT_EINVAL, "n_pages, n_kv_heads and table_width must be >= 1");
  const int s = g->page_size;
  if (s != 16 && s != 32 && s != 64 && s != 128 && s != 256)
    return fail(EVICT_EINVAL, "page_size must be 16, 32, 64, 128 or 256 (got %d)", s);
  if ((long long)g->table_width * s > (1ll << 30))
    return fail(EVICT_ELIMIT, "table_width * page_size = %lld rows are above 2^30", (long long)g->table_width * s);
  if (!g->k || !g->v || !g->table || !g->lens) return fail(EVICT_EINVAL, "pages' k, v, table and lens must not be NULL");
  if (!multiple(g->k, 16) || !multiple(g->v, 16)) return fail(EVICT_EINVAL, "pages must be 16-byte aligned");
  if (!multiple(g->table, 4) || !multiple(g->lens, 4) || !multiple(g->error, 4))
    return fail(EVICT_EINVAL, "table, lens and error must be 4-byte aligned");
  const long long dense = (long long)g->n_kv_heads * s * kHeadDim;
  if (g->page_stride && (g->page_stride % 8 || g->page_stride < dense))
    return fail(EVICT_EINVAL, "page_stride must be a multiple of 8 and hold n_kv_heads * page_size rows");
  if (g->table_stride && g->table_stride < g->table_width) return fail(EVICT_EINVAL, "table_stride is below table_width");
  return EVICT_OK;
}

}  // namespace evict

using namespace evict;

extern "C" int evict_rotary_init(const evict_rotary_config* c, evict_rotary** out) {
  if (!out) return fail(EVICT_EINVAL, "out is NULL");
  *out = nullptr;
  if (!c || !c->inv_freq) return fail(EVICT_EINVAL, "config and inv_freq must not be NULL");
  if (c->rotary_dim < 2 || c->rotary_dim > kHeadDim || c->rotary_dim % 2)
    return fail(EVICT_EINVAL, "rotary_dim must be even and in [2, %d] (got %d)", kHeadDim, c->rotary_dim);
  if (c->adjacent != 0 && c->adjacent != 1) return fail(EVICT_EINVAL, "adjacent must be 0 or 1");
  if (c->n_axes < 1 || c->n_axes > 4) return fail(EVICT_EINVAL, "n_axes must be in [1, 4] (got %d)", c->n_axes);
  if (!std::isfinite(c->scale)) return fail(EVICT_EINVAL, "scale must be finite");
  RotaryTable t;
  memset(&t, 0, sizeof(t));
  t.half = c->rotary_dim / 2;
  t.adjacent = c->adjacent;
  t.n_axes = c->n_axes;
  t.scale = c->scale;
  // 1 / (2 pi) to 106 bits, so that a turn's fraction keeps its 64
  const double hi = 0x1.45f306dc9c883p-3, lo = -9.839338337591243e-18;
  for (int i = 0; i < t.half; ++i) {
    const double w = c->inv_freq[i];
    if (!std::isfinite(w) || std::fabs(w) > 65536.0)
      return fail(EVICT_EINVAL, "inv_freq must be finite and at most 65536 in magnitude");
    if (c->axis && c->axis[i] >= c->n_axes) return fail(EVICT_EINVAL, "axis %d of %d", (int)c->axis[i], c->n_axes);
    t.axis[i] = c->axis ? c->axis[i] : 0;
    const double prod = w * hi, rest = std::fma(w, hi, -prod) + w * lo;
    double frac = prod - std::floor(prod);
    if (frac >= 1.0) frac = 0.0;                  // a tiny negative product rounds up to a whole turn
    t.freq[i] = (uint64_t)std::ldexp(frac, 64) + (uint64_t)(int64_t)std::llrint(std::ldexp(rest, 64));
  }
  evict_rotary* r = new (std::nothrow) evict_rotary;
  if (!r) return fail(EVICT_EINVAL, "out of host memory");
  r->t = t;
  *out = r;
  return EVICT_OK;
}

extern "C" void evict_rotary_destroy(evict_rotary* r) { delete r; }

extern "C" int evict_rotate(const evict_rotary* r, int dtype, int batch, int m, const int32_t* pos, int64_t pos_base,
                            int transpose, const evict_rows* x, const evict_rows* out, int n_tensors, void* stream) {
  if (!r) return fail(EVICT_EINVAL, "the rotation is NULL");
  int rc = check_common(dtype, batch, m, pos);
  if (rc) return rc;
  if (transpose != 0 && transpose != 1) return fail(EVICT_EINVAL, "transpose must be 0 or 1");
  if (n_tensors < 1 || n_tensors > 2 || !x || !out) return fail(EVICT_EINVAL, "need 1 or 2 tensors (got %d)", n_tensors);
  if (batch == 0 || m == 0) return EVICT_OK;
  const int elem = dtype == EVICT_BF16 ? 2 : 4;
  for (int i = 0; i < n_tensors; ++i)
    if ((rc = check_tensor(&x[i], elem, "x")) || (rc = check_output(&out[i], &x[i], elem, "out"))) return rc;
  if ((rc = check_size(batch, m, x[0], n_tensors > 1 ? &x[1] : nullptr, nullptr))) return rc;
  RowsParams P;
  memset(&P, 0, sizeof(P));
  P.rot = r->t;
  bool vec = r->t.half % 8 == 0;
  for (int i = 0; i < n_tensors; ++i) {
    if (rows_overlap(out[i], batch, m)) return fail(EVICT_EINVAL, "out: rows lie on top of each other");
    vec = vec && rows_aligned(x[i], elem, 16) && rows_aligned(out[i], elem, 16);
    set_tensor(P, x[i], &out[i], true);
  }
  P.batch = batch;
  P.m = m;
  P.pos = pos;
  P.pos_base = pos_base;
  P.transpose = transpose;
  return run_rows(P, vec, false, dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int evict_paged_append(const evict_pages* g, int batch, int m, const int32_t* n_new, const evict_rotary* r,
                                  const int32_t* pos, int64_t pos_base, const evict_rows* k, const evict_rows* v,
                                  const evict_rows* q, const evict_rows* q_out, void* stream) {
  int rc = check_pages(g);
  if (rc) return rc;
  if ((rc = check_common(g->dtype, batch, m, pos))) return rc;
  if (!multiple(n_new, 4)) return fail(EVICT_EINVAL, "n_new must be 4-byte aligned");
  if (!!q != !!q_out) return fail(EVICT_EINVAL, "q and q_out go together");
  if (batch == 0 || m == 0) return EVICT_OK;
  const int elem = g->dtype == EVICT_BF16 ? 2 : 4;
  if ((rc = check_tensor(k, elem, "k")) || (rc = check_tensor(v, elem, "v"))) return rc;
  if (k->heads != g->n_kv_heads || v->heads != g->n_kv_heads)
    return fail(EVICT_EINVAL, "k and v have %d and %d heads, the pages %d", k->heads, v->heads, g->n_kv_heads);
  if (q) {
    if ((rc = check_tensor(q, elem, "q")) || (rc = check_output(q_out, q, elem, "q_out"))) return rc;
  }
  if ((rc = check_size(batch, m, *k, v, q))) return rc;
  if (q && rows_overlap(*q_out, batch, m)) return fail(EVICT_EINVAL, "q_out: rows lie on top of each other");
  RowsParams P;
  memset(&P, 0, sizeof(P));
  if (r) P.rot = r->t;
  bool vec = P.rot.half % 8 == 0 && rows_aligned(*k, elem, 16) && rows_aligned(*v, elem, 16);
  set_tensor(P, *k, nullptr, r != nullptr);
  set_tensor(P, *v, nullptr, false);
  if (q) {
    vec = vec && rows_aligned(*q, elem, 16) && rows_aligned(*q_out, elem, 16);
    set_tensor(P, *q, q_out, r != nullptr);
  }
  P.batch = batch;
  P.m = m;
  P.pos = pos;
  P.pos_base = pos_base;
  P.pages[0] = static_cast<char*>(g->k);
  P.pages[1] = static_cast<char*>(g->v);
  P.page_stride = g->page_stride ? g->page_stride : (long long)g->n_kv_heads * g->page_size * kHeadDim;
  P.table = g->table;
  P.table_stride = g->table_stride ? g->table_stride : g->table_width;
  P.table_width = g->table_width;
  P.page_shift = __builtin_ctz((unsigned)g->page_size);
  P.n_pages = g->n_pages;
  P.lens = g->lens;
  P.n_new = n_new;
  P.err = g->error;
  return run_rows(P, vec, true, g->dtype, static_cast<cudaStream_t>(stream));
}

extern "C" int evict_pages_status(int32_t* error, void* stream) {
  if (!error || !multiple(error, 4)) return fail(EVICT_EINVAL, "error must be a device word");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, error, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "reading the pages' error word");
  if (word == kDevOk) return EVICT_OK;
  e = cudaMemsetAsync(error, 0, sizeof(int), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the pages' error word");
  return fail(EVICT_EDEVICE, "a kernel reported %s",
              word == kDevWaitTimeout ? "a bounded wait that gave up" :
              word == kDevBadIndex ? "an index outside its bounds (table, lens or n_new)" : "an error");
}
