// Gated activation on the receive rows with the routing weights applied, and
// its gradients (NeMo AutoModel fused_a2a page, HybridEPDispatch.forward: the
// experts get their rows' probabilities):
//   act[r]     = w silu(a) b            h[r] = (a | b), silu(a) = a s, s = 1 / (1 + exp(-a))
//   grad_a     = w g b s (1 + a (1 - s)),   grad_b = w g a s,   grad_w = <g, a s b>
//
// One wave per slot: row r = token_row[t, k], weight probs[t, k], so only
// rows that a kept slot owns are touched.  Bound by HBM: 3 inter values of a
// row read and written forward, 5 backward.
#include "epx_device.h"

namespace epx {
namespace {

constexpr int kSwThreads = 256;
constexpr int kSwWaves = kSwThreads / kWave;

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float sigmoid(float a) { return 1.0f / (1.0f + expf(-a)); }

// Slots [s0, s1), one wave each.
template <bool BWD>
__global__ __launch_bounds__(kSwThreads) void k_swiglu(SwigluArgs a, int64_t s0, int64_t s1) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t slot = s0 + (int64_t)blockIdx.x * kSwWaves + uniform((int32_t)(threadIdx.x / kWave));
    if (slot >= s1) return;
    const int32_t t = (int32_t)(slot / a.Kp), k = (int32_t)(slot - (int64_t)t * a.Kp);
    const int32_t row = a.token_row[slot];
    const int64_t at = (int64_t)t * a.K + k;
    if (row < 0 || row >= a.R) {  // masked, dropped, or outside the buffer
        if (BWD && a.grad_probs != nullptr && k < a.K && lane == 0) a.grad_probs[at] = 0.0f;
        return;
    }
    const float w = a.probs != nullptr && k < a.K ? a.probs[at] : 1.0f;
    const int32_t Iv = a.I / 8;
    const v4u* ha = reinterpret_cast<const v4u*>(a.h) + (int64_t)row * 2 * Iv;
    const v4u* hb = ha + Iv;
    const v4u* ga = reinterpret_cast<const v4u*>(a.grad_act) + (int64_t)row * Iv;
    v4u* out = reinterpret_cast<v4u*>(a.out) + (int64_t)row * (BWD ? 2 * Iv : Iv);
    float sum = 0.0f;
    for (int32_t v = lane; v < Iv; v += kWave) {
        const v4u va = ha[v], vb = hb[v];
        v4u o0, o1, vg = {0, 0, 0, 0};
        if (BWD) vg = ga[v];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float r0[2], r1[2];
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                const float x = hi ? bf16_hi(va[j]) : bf16_lo(va[j]);
                const float b = hi ? bf16_hi(vb[j]) : bf16_lo(vb[j]);
                const float s = sigmoid(x);
                const float silu = x * s;
                if (BWD) {
                    const float g = hi ? bf16_hi(vg[j]) : bf16_lo(vg[j]);
                    sum += g * (silu * b);
                    const float wg = w * g;
                    r0[hi] = wg * b * (s * (1.0f + x * (1.0f - s)));
                    r1[hi] = wg * silu;
                } else {
                    r0[hi] = w * (silu * b);
                }
            }
            o0[j] = pack_bf16x2(r0[0], r0[1]);
            if (BWD) o1[j] = pack_bf16x2(r1[0], r1[1]);
        }
        __builtin_nontemporal_store(o0, out + v);
        if (BWD) __builtin_nontemporal_store(o1, out + Iv + v);
    }
    if (BWD && a.grad_probs != nullptr && k < a.K) {
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
        if (lane == 0) a.grad_probs[at] = sum;
    }
}

template <bool BWD>
hipError_t swiglu(const SwigluArgs& a, hipStream_t stream) {
    const int64_t slots = (int64_t)a.T * a.Kp;
    constexpr int64_t chunk = 0xFFFFFFFFll / kSwThreads * kSwWaves;  // one grid's work-items
    for (int64_t s0 = 0; s0 < slots; s0 += chunk) {
        const int64_t n = slots - s0 < chunk ? slots - s0 : chunk;
        hipLaunchKernelGGL(k_swiglu<BWD>, dim3((unsigned)((n + kSwWaves - 1) / kSwWaves)), dim3(kSwThreads), 0, stream,
                           a, s0, s0 + n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t stream) { return swiglu<false>(a, stream); }

hipError_t launch_swiglu_bwd(const SwigluArgs& a, hipStream_t stream) { return swiglu<true>(a, stream); }

}  // namespace epx
