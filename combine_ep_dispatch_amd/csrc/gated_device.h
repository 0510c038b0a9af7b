// The gated block's arithmetic, on results in registers.
#pragma once

#include "expert_device.h"

namespace epx {

// 1 / (1 + exp(-a)) from the hardware's exp2 and reciprocal, each within one
// unit in the last place: the argument's rounding makes it |a| 2^-24 of the value
// at most.  exp(-a) past the largest float is infinite and the result 0.
__device__ __forceinline__ float fast_sigmoid(float a) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(a * -1.44269504f));
}

// The routing weight of receive row r: its slot's probability, 1 in the shared
// slot or without probabilities.  slot: where its gradient goes in [T, K], -1: nowhere.
__device__ __forceinline__ float row_weight(const BlockArgs& a, int64_t r, int64_t& slot) {
    const int32_t t = a.src_info[2 * r], k = a.src_info[2 * r + 1];
    slot = t >= 0 && t < a.T && k >= 0 && k < a.K ? (int64_t)t * a.K + k : -1;
    return a.probs != nullptr && slot >= 0 ? a.probs[slot] : 1.0f;
}

}  // namespace epx
