// moe_few.cuh -- the routing a mixture-of-experts call leaves on the device for its products.
#pragma once

#include "common.cuh"

namespace fp8gemm {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxExperts = 512;

// A pair p = token * k + choice.  Device memory, rewritten by every call.
struct MoeRoute {
  float* weight;  // [T k]
  int* pairs;     // [E][T]: the pairs that chose expert e, ascending
  int* count;     // [E]
  int* expert;    // the chosen experts, ascending
  int* active;    // how many
};

}  // namespace fp8gemm
