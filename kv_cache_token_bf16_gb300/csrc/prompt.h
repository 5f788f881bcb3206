// Launch parameters of the prompts' kernels: attention (prompt.cu), weights of keys (weights.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "../../include/evict.h"
#include "attend.h"

namespace evict {

// Where a share begins: the block's plane, its sequence's first row and length, the block; KV head, step, steps.
struct alignas(16) PromptBegin {
  int of[8];
};

// The work of one call. A block is `tile` tokens of one sequence; a unit is a
// block and a KV head, and its work a number of steps that the kernel knows,
// behind `entry` more for its start. The blocks' units, in the order of blocks
// and heads, are laid end to end and cut into equal contiguous shares, one for
// a CTA. `whole`: units are not cut, but dealt out to the CTAs, or taken as CTAs come to them.
struct PromptWork {
  const int32_t* starts;             // [seqs + 1] first rows of the sequences of one plane; or NULL: a plane each
  int seqs, m;                       // sequences; rows of a plane
  int hkv;
  int tile;                          // tokens of a block
  int blocks;                        // at most
  int entry, min_steps;              // steps that a unit's start counts as; of a share at least
  int whole, longest_last;           // longest_last: of a sequence's blocks the last has the most steps
  Divisor by_hkv, by_tile, by_seq_blocks;
  int* block_base;                   // [seqs + 1] blocks of the sequences before (packed)
  PromptBegin* begin;                // [CTAs]
  int* total;                        // [3] steps of all units, the shares' number; units taken
  int* taken;                        // whole: units taken beyond the CTAs' first ones; or NULL
  int* order;                        // [blocks] whole: the blocks in the order in which units are taken; or NULL
  int* err;
};

constexpr float kLog2eRest = 1.92596299e-8f;       // log2 e beyond its fp32 value

// scale * log2 e (0: 1 / sqrt(128)), a little more. The tensor cores cut each of a logit's eight partial sums toward
// zero: logits of 10 .. 20 of random rows lost 0.9e-7 of themselves in the mean, of a row with itself 1.4e-7 .. 2.3e-7,
// and sums of weights add that up. 2^-23 makes up for it: a prompt's weights of keys (8192 tokens, 28 heads) were
// 1.6e-6 off and are 0.05e-6 .. 1.0e-6 by their values, an fp32 product's 0.5e-6 .. 1.4e-6 (with 2^-22 2.1e-6 .. 3.5e-6).
inline float scale_base2(float scale) {
  return (float)((scale == 0.f ? 0.08838834764831845 : (double)scale) * 1.4426950408889634 * (1.0 + 0x1p-23));
}

// Whether that is a number (NaN is not below anything).
inline bool good_scale(float scale) { return std::fabs(scale) < 0x1p127f; }

struct PromptParams {
  CUtensorMap q_map, k_map, v_map;
  PromptWork work;
  const void* q;                     // (the attention's rare path)
  const void* k;
  const void* v;
  void* out;
  float* lse;
  float* weights;
  long long qb, qh, qm, kb, kh, km, vb, vh, vm, ob, oh, om;   // element strides
  int hq, group;                     // group = query heads of a KV head
  Divisor by_group;
  int half;                          // attention: tokens of a tile of 128 query rows; weights: tokens of a step
  int out_sectors;                   // every row of out begins on a multiple of 32 bytes
  int last;                          // weights: the last queries of a sequence that count
  int half_shift;                    // weights: log2 half
  int step_heads, head_steps;        // weights: heads of a step, steps that the group's heads take
  float scale2;                      // log2(e) * scale
  float2* part_ml;                   // attention: [2 CTAs][256] maximum (base 2) and sum
  float* part;                       // attention: [2 CTAs][256][128] outputs; weights: [2 CTAs][256] sums
};

// The checks of a call's sizes, and of its pointers as well (prompt.cu).
int check_prompt_sizes(const evict_prompt* a);
int check_prompt(const evict_prompt* a, bool attention);
// The schedule and the workspace, with offsets in place of pointers until bind_prompt.
struct PromptPlan {
  int dev, sms;
  PromptParams p;
  size_t bytes;
};
// tile, entry, min_steps, longest_last: as above; most_steps: of a unit; whole_rounds: where there are so many units for
// every SM, they are not cut; part_ml, part: bytes of a CTA's partial results.
int plan_prompt(const evict_prompt* a, int tile, long long most_steps, int entry, int min_steps, int whole_rounds,
                size_t part_ml, size_t part, bool longest_last, PromptPlan* out);
int bind_prompt(const evict_prompt* a, PromptPlan* plan);
// No units taken yet, before the kernel that takes them.
int begin_prompt(const PromptWork& w, cudaStream_t st);
// Boxes of heads_box heads of rows_box rows of 64 elements, 128-byte swizzle: a row's heads one behind the other
// (heads_first; coordinates element, head, row, plane), or a head's rows (element, row, head, plane).
int encode_heads(CUtensorMap* map, const evict_rows& x, int batch, int m, int heads_box, int rows_box, bool heads_first,
                 const char* name);

}  // namespace evict
