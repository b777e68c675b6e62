// Work items of the packed prompt attention, shared by its planner (api_serving.cu) and kernel.
#pragma once
#include "skv_internal.h"

namespace skv {

// One item: query tiles A and B (up to 128 tokens of one head each) over key tiles
// [tile_begin, tile_end) of 128 keys of one sequence, whose keys are rows kv0 .. kv0 + kv_len.  Row i
// of a tile sees the sequence's first min(kv_len, limit + i) keys when causal, else all of them.
// part_row < 0: results go to o / lse; else token t (0-based from q0a) goes to partial row
// part_row + t * part_stride.
struct PromptItem {
  int32_t q0a, q0b, na, nb, ha, hb, limit_a, limit_b;
  int32_t kv0, kv_len, tile_begin, tile_end, part_row, part_stride, causal, pad;
};
static_assert(sizeof(PromptItem) == 64, "prompt item is 16 int32 words");
constexpr int kPromptTile = 128;

int launch_prompt_attn(const skv_prompt_params& p, const PromptItem* items, const int32_t* cta_indptr, int num_ctas,
                       cudaStream_t s);

}  // namespace skv
