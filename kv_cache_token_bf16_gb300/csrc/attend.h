// Launch parameters and workspace layout of the shared-prefix attention.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/evict.h"

namespace evict {

constexpr int kStepTokens = 128;     // rows of K and V that a CTA takes at a time ("step")
constexpr int kWideRows = 256;       // query rows of a unit of the wide kernel (two MMA tiles)

// The work of one kernel. Streams: one per prefix (all query rows of its
// sequences), then one per sequence (its own pages; `joint`: behind the prefix
// as well). A unit is one (stream, KV head, tile of query rows); its work is
// the rows of K and V that the tile sees, in steps. The steps of all units are
// laid end to end and every CTA takes an equal contiguous share. The part of a
// unit that one CTA takes leaves one partial result in slot unit + CTA: from
// one part to the next either the unit or the CTA goes up, so slots are unique.
struct StreamSet {
  int prefixes;                      // streams of prefixes
  int own;                           // streams of sequences: 0 or the batch
  int joint;                         // a sequence's stream begins with its prefix
  int ctas;
  long long* step_base;              // [streams + 1] first step of every stream, then their total
  long long* unit_base;              // [streams] first unit
  float2* part_ml;                   // [slots][tile rows] running maximum (base 2) and sum
  float* part_o;                     // [slots][tile rows][128]
};

struct AttendParams {
  CUtensorMap tm_pk, tm_pv;          // prefix [prefix_batch][n_kv_heads][n_prefix][128]
  CUtensorMap tm_k, tm_v;            // pages [n_pages][n_kv_heads][page_size][128]
  StreamSet set;                     // of this launch (the join: of the few-row kernel)
  StreamSet wide;                    // the join: of the wide kernel
  const void* q;
  void* out;
  float* lse;
  long long qb, qh, qm, ob, oh, om;  // element strides
  int batch, m, hq, hkv, group;      // group = query heads of a KV head
  int prefix_batch, fan;             // prefixes, and sequences of one (fan = 0: no prefix)
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
  int box_rows;                      // rows of a box of the pages
  float scale2;                      // log2(e) * scale
  int* tok_base;                     // [batch + 1] new tokens of the sequences before (with n_new)
  int late_wait;                     // this kernel may start before its predecessor has ended
  int* err;
};

int wide_smem();
cudaError_t prepare_wide();
cudaError_t launch_wide(const AttendParams& p, bool early, cudaStream_t st);

}  // namespace evict
