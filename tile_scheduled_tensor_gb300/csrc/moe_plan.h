// What moe.cu and moe_score.cu share: the scored kernels' instances, which a scored plan brings along, so
// that the unit of the other calls needs none of them.
#pragma once
#include "tstgemm.h"

// Instances for `vpl` logits per lane, rows read in whole packs (vec) or not, 8 or 32 (whole packs never)
// warps a block.
struct TstScoreKernels {
  const void* (*rows)(bool bf16, int vpl, bool vec, int warps);
  const void* (*grad)(bool bf16, int vpl, bool vec);
};

// moe_plan_create (score null) and moe_plan_create_scored
tst_status tst_moe_create(tst_moe_plan** out, int64_t max_tokens, int32_t experts, int32_t top_k, const tst_moe_options* opts,
                          const tst_moe_score_options* score, const TstScoreKernels* kernels);
