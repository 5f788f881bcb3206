// Launch parameters and workspace layout of the shared-prefix attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/evict.h"

namespace evict {

constexpr int kBoxTokens = 16;       // rows of K and V that a warp of the few-row kernel takes at a time
constexpr int kWideTokens = 128;     // rows that a CTA of the wide kernel takes at a time
constexpr int kFewRows = 16;         // query rows of a unit of the few-row kernel (one MMA tile)
constexpr float kWideStart = 8000.f; // clocks by which the wide kernel's start is longer
constexpr int kWideRows = 256;       // query rows of a unit of the wide kernel (two MMA tiles)

// Quotient by a divisor that the host knows, for dividends below 2^31: a multiplication and a shift.
struct Divisor {
  uint32_t by, mul, one, shift;
  Divisor() = default;
  __host__ explicit Divisor(int d) : by(d), mul(0), one(0), shift(0) {
    if (d == 1) {
      one = ~0u;
    } else if (d > 1) {
      while ((2u << shift) < by) ++shift;         // ceil(log2 d) - 1
      mul = (uint32_t)(((1ull << (32 + shift)) + by - 1) / by);
    }
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, mul) + ((uint32_t)n & one)) >> shift); }
#endif
};

// The work of one kernel. A block is a tile of query rows of one stream; the
// streams are the prefixes (all query rows of their sequences), then the
// sequences (their own pages; `joint`: behind the prefix as well). A unit is a
// block and a KV head, and its work the rows of K and V that the tile sees, in
// steps of 16 (few-row kernel) or 128 (wide kernel) rows, behind `entry` more
// for its start. The steps of all units, in the order of blocks and heads, are
// laid end to end and cut into equal contiguous shares, one for every warp
// (few-row kernel) or CTA (wide).
// Where a call has work for both kernels, they run side by side on different SMs, as many as their
// work asks for.
// What a share holds of a unit leaves one partial result, in slot unit +
// share: from one part to the next either of them goes up, so slots are unique.
// A slot has the rows that the largest unit of its kind fills; prefixes' slots
// come first, then the sequences' own, counted anew. Joint units leave one only
// where a share ends or begins inside a unit: slot 2 share for the part of a unit
// that began before, 2 share + 1 for one that begins there.
struct WorkSet {
  int prefixes, prefix_tiles;        // streams of prefixes, blocks of one
  int seqs, seq_tiles;               // streams of sequences: 0 or the batch; blocks of one
  int joint;                         // a sequence's stream begins with its prefix
  int workers, min_steps;            // shares that a CTA takes (its warps, or itself); steps of a share at least
  int entry;                         // steps that the start of a unit counts as
  int cost;                          // of a step: clocks of an SM, roughly
  int max_shares;                    // workers of every SM
  Divisor by_prefix_tiles, by_seq_tiles;
  int* base;                         // [blocks + 2] first step of every block, their total, the shares' number
  int2* start;                       // [shares] block and step in it where every share begins
  int pre_units, pre_rows, own_rows; // units of prefixes; rows of their slots, and of the others'
  long long own_at;                  // first row of the others' slots
  float2* part_ml;                   // [rows of all slots] running maximum (base 2) and sum
  float* part_o;                     // [rows of all slots][128]
  __host__ __device__ int blocks() const { return prefixes * prefix_tiles + seqs * seq_tiles; }
#ifdef __CUDACC__
  __device__ __forceinline__ int rows_of(int unit) const { return unit < pre_units ? pre_rows : own_rows; }
  // First row of the slot of what `share` holds of a unit (not joint).
  __device__ __forceinline__ long long slot_row(int unit, int share) const {
    return unit < pre_units ? (long long)(unit + share) * pre_rows : own_at + (long long)(unit - pre_units + share) * own_rows;
  }
#endif
};

struct AttendParams {
  // K and V: the prefix [prefix_batch][n_kv_heads][n_prefix][128], the pages
  // [n_pages][n_kv_heads][page_size][128]
  CUtensorMap few_pre[2], few_own[2], wide_pre[2], wide_own[2];
  WorkSet few, wide;                 // of the two kernels
  int sms;
  const void* q;
  void* out;
  float* lse;
  long long qb, qh, qm, ob, oh, om;  // element strides
  int batch, m, hq, hkv, group;      // group = query heads of a KV head
  int prefix_batch, fan;             // prefixes, and sequences of one (fan = 0: no prefix)
  Divisor by_m, by_hq, by_hkv, by_group, by_fan;
  int n_prefix;
  int pages;                         // the sequences have own rows
  const int32_t* table;
  const int32_t* lens;
  const int32_t* n_new;
  long long table_stride;
  int table_width, page_shift, n_pages;
  const void* page_k;                // (the wide kernel's rare path)
  const void* page_v;
  long long page_stride;
  int box_rows;                      // rows of a box of the pages (wide kernel)
  int out_sectors;                   // every row of out begins on a multiple of 32 bytes
  float scale2;                      // log2(e) * scale
  int* tok_base;                     // [batch + 1] new tokens of the sequences before (with n_new)
  int* err;
};

}  // namespace evict
