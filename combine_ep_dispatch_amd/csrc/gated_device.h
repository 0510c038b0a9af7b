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

// The routing weights of COUNT receive rows of this lane, row(n) each: the slots'
// probabilities, 1 in the shared slot or without probabilities.  slot: where their
// gradients go in [T, K], -1: nowhere.  All loads go out together, twice: one row's
// after the other's they took 16 000 of an epilogue's 25 000 cycles.
template <int COUNT, typename Row>
__device__ __forceinline__ void row_weights(const BlockArgs& a, Row row, float (&w)[COUNT], int32_t (&slot)[COUNT]) {
    v2u src[COUNT];
#pragma unroll
    for (int n = 0; n < COUNT; ++n) src[n] = *reinterpret_cast<const v2u*>(a.src_info + 2 * row(n));
#pragma unroll
    for (int n = 0; n < COUNT; ++n) {
        const int32_t t = (int32_t)src[n].x, k = (int32_t)src[n].y;
        slot[n] = t >= 0 && t < a.T && k >= 0 && k < a.K ? t * a.K + k : -1;
        w[n] = 1.0f;
    }
    if (a.probs == nullptr) return;
#pragma unroll
    for (int n = 0; n < COUNT; ++n) w[n] = a.probs[max(slot[n], 0)];
#pragma unroll
    for (int n = 0; n < COUNT; ++n) w[n] = slot[n] >= 0 ? w[n] : 1.0f;
}

}  // namespace epx
