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
// as a signed number, times 2^-31 are the angle in half turns in [-1, 1),
// which sincospif takes without a range reduction of its own.
//
// Bound: HBM, every row read once and written once. A group of 8 threads owns
// one token: thread u holds pairs [8 u, 8 u + 8), whose sines and cosines it
// computes once and uses for every head of its slice (~250 instructions, as
// many as the rotation of four or five heads). A token's heads are cut into
// as many slices as fill the GPU's resident threads once, so that a decode
// step of a few tokens still spreads over the SMs and a long prompt pays for
// its angles once in 4 to 8 heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <new>

#include "api_internal.h"
#include "common.cuh"
#include "launch.h"
#include "rotary.h"

namespace evict {
namespace {

constexpr int kRowThreads = 256;
constexpr int kUnit = 8;                          // pairs of a thread
constexpr int kLanes = kHeadDim / 2 / kUnit;      // threads of a row
constexpr int kGroups = kRowThreads / kLanes;     // tokens' slices of a block
constexpr int kMaxTensors = 3;

struct RowTensor {
  const void* src;
  void* dst;                         // null: the pages (k or v)
  long long sb, sh, sm, db, dh, dm;  // element strides
  int end;                           // heads of this and the earlier tensors
  int rotate;
};

struct RowsParams {
  RotaryTable rot;                   // half = 0: nothing is rotated
  RowTensor t[kMaxTensors];
  int n_tensors, heads, per_slice, slices;
  int batch, m;
  long long groups;
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

// 16 elements of a row as raw 16-byte pieces: 8 from `lo`, 8 from `hi`.
template <typename T>
struct Piece {
  static constexpr int kVecs = kUnit * (int)sizeof(T) / 16;
  uint4 lo[kVecs], hi[kVecs];
  __device__ __forceinline__ void load(const T* a, const T* b) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) lo[i] = reinterpret_cast<const uint4*>(a)[i];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) hi[i] = reinterpret_cast<const uint4*>(b)[i];
  }
  __device__ __forceinline__ void store(T* a, T* b) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4*>(a)[i] = lo[i];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4*>(b)[i] = hi[i];
  }
  __device__ __forceinline__ void values(float (&x)[2 * kUnit]) const {
    if constexpr (sizeof(T) == 2) {
      float a[kUnit], b[kUnit];
      bf16x8_to_f32(lo[0], a);
      bf16x8_to_f32(hi[0], b);
#pragma unroll
      for (int i = 0; i < kUnit; ++i) x[i] = a[i], x[kUnit + i] = b[i];
    } else {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const uint4 a = lo[i], b = hi[i];
        x[4 * i] = __uint_as_float(a.x), x[4 * i + 1] = __uint_as_float(a.y);
        x[4 * i + 2] = __uint_as_float(a.z), x[4 * i + 3] = __uint_as_float(a.w);
        x[kUnit + 4 * i] = __uint_as_float(b.x), x[kUnit + 4 * i + 1] = __uint_as_float(b.y);
        x[kUnit + 4 * i + 2] = __uint_as_float(b.z), x[kUnit + 4 * i + 3] = __uint_as_float(b.w);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&x)[2 * kUnit]) {
    if constexpr (sizeof(T) == 2) {
      auto two = [](float a, float b) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
      };
      lo[0] = make_uint4(two(x[0], x[1]), two(x[2], x[3]), two(x[4], x[5]), two(x[6], x[7]));
      hi[0] = make_uint4(two(x[8], x[9]), two(x[10], x[11]), two(x[12], x[13]), two(x[14], x[15]));
    } else {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        lo[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                           __float_as_uint(x[4 * i + 3]));
        hi[i] = make_uint4(__float_as_uint(x[kUnit + 4 * i]), __float_as_uint(x[kUnit + 4 * i + 1]),
                           __float_as_uint(x[kUnit + 4 * i + 2]), __float_as_uint(x[kUnit + 4 * i + 3]));
      }
    }
  }
};

// kVec: 16-byte pieces (rows and strides aligned, rotary_dim a multiple of 16, so that every
// thread's 16 elements are rotated or copied as a whole); else an element at a time.
template <typename T, bool kVec, bool kPaged>
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowsParams p) {
  pdl_wait();
  const long long g = (long long)blockIdx.x * kGroups + threadIdx.x / kLanes;
  if (g >= p.groups) return;
  const int u = threadIdx.x % kLanes;
  const unsigned tok = (unsigned)(g / p.slices);
  const int slice = (int)(g - (long long)tok * p.slices);
  const int b = (int)(tok / (unsigned)p.m), t = (int)(tok - (unsigned)b * p.m);

  bool stored = true;                              // the token's page row exists
  long long at = 0, index = t;                     // its element offset in the pool (head 0)
  if constexpr (kPaged) {
    int n = p.n_new ? p.n_new[b] : p.m;
    const bool odd = n < 0 || n > p.m;
    n = n < 0 ? 0 : n > p.m ? p.m : n;
    if (odd && u == 0 && t == 0 && p.err) raise_device_error(p.err, kDevBadIndex);
    if (t >= n) return;
    const int j = p.lens[b] - n + t;
    index = j;
    int page = -1;
    if (j >= 0 && (j >> p.page_shift) < p.table_width)
      page = p.table[(long long)b * p.table_stride + (j >> p.page_shift)];
    stored = page >= 0 && page < p.n_pages;
    if (!stored && u == 0 && p.err) raise_device_error(p.err, kDevBadIndex);
    if (stored) at = (long long)page * p.page_stride + (long long)(j & ((1 << p.page_shift) - 1)) * kHeadDim;
  }

  // this thread's 16 elements: at `ea` and `eb`, 8 each (kVec)
  const int half = p.rot.half;
  const bool turns = kUnit * u < half;             // kVec: all of its pairs turn, or none
  const int ea = turns && !p.rot.adjacent ? kUnit * u : 2 * kUnit * u;
  const int eb = turns && !p.rot.adjacent ? half + kUnit * u : 2 * kUnit * u + kUnit;

  auto source = [&](const RowTensor& x, int h) {
    return static_cast<const T*>(x.src) + (long long)b * x.sb + (long long)h * x.sh + (long long)t * x.sm;
  };
  auto target = [&](const RowTensor& x, int which, int h) -> T* {
    if (kPaged && !x.dst)
      return stored ? reinterpret_cast<T*>(p.pages[which]) + at + ((long long)h << p.page_shift) * kHeadDim : nullptr;
    return static_cast<T*>(x.dst) + (long long)b * x.db + (long long)h * x.dh + (long long)t * x.dm;
  };
  auto which_of = [&](int hv) { return hv < p.t[0].end ? 0 : hv < p.t[1].end ? 1 : 2; };
  const int h0 = slice * p.per_slice;
  const int h1 = h0 + p.per_slice < p.heads ? h0 + p.per_slice : p.heads;

  float co[kUnit], si[kUnit];
  auto angles = [&] {
#pragma unroll
    for (int i = 0; i < kUnit; ++i) co[i] = 1.f, si[i] = 0.f;
    if (!turns) return;
    long long one = 0;
    if (!p.pos) one = p.pos_base + index;
    else if (p.rot.n_axes == 1) one = p.pos[(long long)b * p.m + t];
#pragma unroll
    for (int i = 0; i < kUnit; ++i) {
      const int f = kUnit * u + i;
      if (f >= half) continue;
      long long ps = one;
      if (p.pos && p.rot.n_axes > 1) ps = p.pos[((long long)p.rot.axis[f] * p.batch + b) * p.m + t];
      const int32_t turn = (int32_t)(uint32_t)(((uint64_t)ps * p.rot.freq[f]) >> 32);
      float s, c;
      sincospif((float)turn * 0x1p-31f, &s, &c);
      co[i] = c * p.rot.scale;
      si[i] = p.transpose ? -s * p.rot.scale : s * p.rot.scale;
    }
  };

  if constexpr (kVec) {
    constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;   // heads in flight: 128 bytes of loads a thread
    Piece<T> x[kBatch];
    auto load = [&](int hv0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int hv = hv0 + k;
        if (hv >= h1) break;
        const int w = which_of(hv);
        const T* s = source(p.t[w], hv - (w ? p.t[w - 1].end : 0));
        x[k].load(s + ea, s + eb);
      }
    };
    load(h0);
    angles();
    for (int hv0 = h0; hv0 < h1; hv0 += kBatch) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int hv = hv0 + k;
        if (hv >= h1) break;
        const int w = which_of(hv);
        T* d = target(p.t[w], w, hv - (w ? p.t[w - 1].end : 0));
        if (turns && p.t[w].rotate) {
          float e[2 * kUnit], y[2 * kUnit];
          x[k].values(e);
          if (p.rot.adjacent) {
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
              y[2 * i] = e[2 * i] * co[i] - e[2 * i + 1] * si[i];
              y[2 * i + 1] = e[2 * i] * si[i] + e[2 * i + 1] * co[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < kUnit; ++i) {
              y[i] = e[i] * co[i] - e[kUnit + i] * si[i];
              y[kUnit + i] = e[i] * si[i] + e[kUnit + i] * co[i];
            }
          }
          x[k].set(y);
        }
        if (d) x[k].store(d + ea, d + eb);
      }
      if (hv0 + kBatch < h1) load(hv0 + kBatch);
    }
  } else {
    angles();
    for (int hv = h0; hv < h1; ++hv) {
      const int w = which_of(hv), h = hv - (w ? p.t[w - 1].end : 0);
      const T* s = source(p.t[w], h);
      T* d = target(p.t[w], w, h);
      if (!d) continue;
#pragma unroll
      for (int i = 0; i < kUnit; ++i) {
        const int f = kUnit * u + i;
        const bool turn = f < half && p.t[w].rotate;
        const int i0 = f < half && !p.rot.adjacent ? f : 2 * f;
        const int i1 = f < half && !p.rot.adjacent ? f + half : 2 * f + 1;
        const T x0 = s[i0], x1 = s[i1];
        if (turn) {
          const float a = widen(x0), c = widen(x1);
          d[i0] = narrow<T>(a * co[i] - c * si[i]);
          d[i1] = narrow<T>(a * si[i] + c * co[i]);
        } else {
          d[i0] = x0;
          d[i1] = x1;
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
  P.heads += x.heads;
  t.end = P.heads;
  t.rotate = rotate;
}

// One wave of resident threads: a token's heads in as few slices as give every SM its 2048 threads.
int run_rows(RowsParams& P, bool vec, bool paged, int dtype, cudaStream_t st) {
  for (int i = P.n_tensors; i < kMaxTensors; ++i) P.t[i].end = P.heads;
  const long long tokens = (long long)P.batch * P.m;
  if (tokens * P.heads >= (1ll << 31))
    return fail(EVICT_ELIMIT, "batch * m * heads = %lld rows are 2^31 or more", tokens * P.heads);
  constexpr long long kResident = 152ll * 2048 / kLanes;
  long long per = (tokens * P.heads + kResident - 1) / kResident;
  P.per_slice = (int)(per < 1 ? 1 : per > P.heads ? P.heads : per);
  P.slices = (P.heads + P.per_slice - 1) / P.per_slice;
  P.groups = tokens * P.slices;
  const dim3 grid((unsigned)((P.groups + kGroups - 1) / kGroups));
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
  RowsParams P;
  memset(&P, 0, sizeof(P));
  P.rot = r->t;
  bool vec = r->t.half % kUnit == 0;
  for (int i = 0; i < n_tensors; ++i) {
    if ((rc = check_tensor(&x[i], elem, "x")) || (rc = check_tensor(&out[i], elem, "out"))) return rc;
    if (x[i].heads != out[i].heads)
      return fail(EVICT_EINVAL, "tensor %d has %d heads and its output %d", i, x[i].heads, out[i].heads);
    if (x[i].data == out[i].data && (x[i].stride_b != out[i].stride_b || x[i].stride_h != out[i].stride_h ||
                                     x[i].stride_m != out[i].stride_m))
      return fail(EVICT_EINVAL, "an output in place must have its input's strides");
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
  RowsParams P;
  memset(&P, 0, sizeof(P));
  if (r) P.rot = r->t;
  bool vec = P.rot.half % kUnit == 0 && rows_aligned(*k, elem, 16) && rows_aligned(*v, elem, 16);
  set_tensor(P, *k, nullptr, r != nullptr);
  set_tensor(P, *v, nullptr, false);
  if (q) {
    if ((rc = check_tensor(q, elem, "q")) || (rc = check_tensor(q_out, elem, "q_out"))) return rc;
    if (q->heads != q_out->heads) return fail(EVICT_EINVAL, "q has %d heads and q_out %d", q->heads, q_out->heads);
    if (q->data == q_out->data &&
        (q->stride_b != q_out->stride_b || q->stride_h != q_out->stride_h || q->stride_m != q_out->stride_m))
      return fail(EVICT_EINVAL, "an output in place must have its input's strides");
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
