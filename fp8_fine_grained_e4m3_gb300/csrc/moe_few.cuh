// moe_few.cuh -- limits of the few-token mixture-of-experts layer.
#pragma once

namespace fp8gemm {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxExperts = 512;

}  // namespace fp8gemm
