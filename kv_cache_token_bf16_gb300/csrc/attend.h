// Launch parameters and workspace layout of the shared-prefix attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/evict.h"

namespace evict {

constexpr int kStepTokens = 128;     // rows of K and V that a CTA takes at a time ("step")

// Streams: one per prefix, then one per sequence (its own pages). A stream's
// work is, for every KV head and tile of query rows, its rows in steps; the
// steps of all streams are laid end to end and every CTA takes an equal
// contiguous share. A unit is one (stream, head, row tile). The part of a unit
// that one CTA takes leaves one partial result in slot unit + CTA: from one
// part to the next either the unit or the CTA goes up, so slots are unique.
struct AttendParams {
  CUtensorMap tm_pk, tm_pv;          // prefix [prefix_batch][n_kv_heads][n_prefix][128]
  CUtensorMap tm_k, tm_v;            // pages [n_pages][n_kv_heads][page_size][128]
  const void* q;
  void* out;
  float* lse;
  long long qb, qh, qm, ob, oh, om;  // element strides
  int batch, m, hq, hkv, group;      // group = query heads of a KV head
  int prefixes, fan;                 // sequences of a prefix
  int n_prefix;
  int prefix_tiles;                  // row tiles of a prefix unit (0: no prefix)
  int own;                           // there are pages
  const int32_t* table;
  const int32_t* lens;
  const int32_t* n_new;
  long long table_stride;
  int table_width, page_shift, n_pages;
  float scale2;                      // log2(e) * scale
  int ctas;
  int* err;
  long long* step_base;              // [streams + 1] first step of every stream, then their total
  long long* unit_base;              // [streams] first unit
  float2* part_ml;                   // [slots][tile rows] running maximum (base 2) and sum
  float* part_o;                     // [slots][tile rows][128]
};

}  // namespace evict
