// Internal interface of routing by scores, with a bias and groups (route.hip).
#pragma once

#include "hq_internal.h"

namespace hq {

struct RouteArgs {
  const void* logits;  // [t][E]
  const float* bias;   // [E], or null
  int32_t* ids;        // [t][topk]
  float* w;
  int logit_type;      // 0 fp32, 1 bf16, 2 fp16
  int t, E, topk;      // E <= 1024, topk <= 64
  int softmax;         // scores: softmax of the row, or the sigmoid of each logit
  int groups, group_topk, group_best;  // groups <= 64, each of E / groups experts
  int renorm;
  float scale;
};

int launch_route_experts(const RouteArgs& a, void* stream);

}  // namespace hq
