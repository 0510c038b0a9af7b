// Gated activation on the receive rows with the routing weights applied, and
// its gradients (NeMo AutoModel fused_a2a page, HybridEPDispatch.forward: the
// experts get their rows' probabilities):
//   act[r]     = w silu(a) b            h[r] = (a | b), silu(a) = a s, s = 1 / (1 + exp(-a))
//   grad_a     = w g b s (1 + a (1 - s)),   grad_b = w g a s,   grad_w = <g, a s b>
//
// Rows are found through token_row, so only those that a kept slot owns are
// touched.  Bound by HBM: 3 inter values of a row read and written forward, 5
// backward.  35 700 rows of 2048: 84 us forward (5.2 TB/s), 140 backward (5.2);
// a copy of 1 GiB reaches 5.2.  128 rows (a decode step): 4.5 us.
#include "epx_device.h"

namespace epx {
namespace {

constexpr int kSwThreads = 256;
constexpr int kSwWaves = kSwThreads / kWave;

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float sigmoid(float a) { return 1.0f / (1.0f + expf(-a)); }

// The lane's 8 values of act, or of both halves of grad_h (and its share of
// the weight's gradient).
__device__ __forceinline__ v4u forward8(v4u va, v4u vb, float w) {
    v4u o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float r[2];
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
            const float x = hi ? bf16_hi(va[j]) : bf16_lo(va[j]);
            const float b = hi ? bf16_hi(vb[j]) : bf16_lo(vb[j]);
            r[hi] = w * (x * sigmoid(x) * b);
        }
        o[j] = pack_bf16x2(r[0], r[1]);
    }
    return o;
}

__device__ __forceinline__ void backward8(v4u va, v4u vb, v4u vg, float w, v4u& oa, v4u& ob, float& sum) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float ra[2], rb[2];
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
            const float x = hi ? bf16_hi(va[j]) : bf16_lo(va[j]);
            const float b = hi ? bf16_hi(vb[j]) : bf16_lo(vb[j]);
            const float g = hi ? bf16_hi(vg[j]) : bf16_lo(vg[j]);
            const float s = sigmoid(x), silu = x * s, wg = w * g;
            sum += g * (silu * b);
            ra[hi] = wg * b * (s * (1.0f + x * (1.0f - s)));
            rb[hi] = wg * silu;
        }
        oa[j] = pack_bf16x2(ra[0], ra[1]);
        ob[j] = pack_bf16x2(rb[0], rb[1]);
    }
}

// Forward: one wave per slot.
__global__ __launch_bounds__(kSwThreads) void k_swiglu(SwigluArgs a, int64_t s0, int64_t s1) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t slot = s0 + (int64_t)blockIdx.x * kSwWaves + uniform((int32_t)(threadIdx.x / kWave));
    if (slot >= s1) return;
    const int32_t t = (int32_t)(slot / a.Kp), k = (int32_t)(slot - (int64_t)t * a.Kp);
    const int32_t row = a.token_row[slot];
    const float w = a.probs != nullptr && k < a.K ? a.probs[(int64_t)t * a.K + k] : 1.0f;
    if (row < 0 || row >= a.R) return;  // masked, dropped, or outside the buffer
    const int32_t Iv = a.I / 8;
    const v4u* h = reinterpret_cast<const v4u*>(a.h) + (int64_t)row * 2 * Iv;
    v4u* out = reinterpret_cast<v4u*>(a.out) + (int64_t)row * Iv;
    constexpr int kBatch = 4;  // pieces whose loads are in flight together (2: 87 instead of 84 us at 35 700 rows of 2048)
    for (int32_t v0 = lane; v0 < Iv; v0 += kBatch * kWave) {
        v4u va[kBatch], vb[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int32_t v = min(v0 + i * kWave, Iv - 1);
            va[i] = __builtin_nontemporal_load(h + v);
            vb[i] = __builtin_nontemporal_load(h + Iv + v);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int32_t v = v0 + i * kWave;
            if (v >= Iv) break;
            __builtin_nontemporal_store(forward8(va[i], vb[i], w), out + v);
        }
    }
}

// Backward: one wave per slot, which sums the weight's gradient along the row
// (each lane its values in order, then a fixed tree over the lanes).
__global__ __launch_bounds__(kSwThreads) void k_swiglu_bwd(SwigluArgs a, int64_t s0, int64_t s1) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t slot = s0 + (int64_t)blockIdx.x * kSwWaves + uniform((int32_t)(threadIdx.x / kWave));
    if (slot >= s1) return;
    const int32_t t = (int32_t)(slot / a.Kp), k = (int32_t)(slot - (int64_t)t * a.Kp);
    const int32_t row = a.token_row[slot];
    const int64_t at = (int64_t)t * a.K + k;
    const float w = a.probs != nullptr && k < a.K ? a.probs[at] : 1.0f;
    const bool wanted = a.grad_probs != nullptr && k < a.K;
    if (row < 0 || row >= a.R) {  // masked, dropped, or outside the buffer
        if (wanted && lane == 0) a.grad_probs[at] = 0.0f;
        return;
    }
    const int32_t Iv = a.I / 8;
    const v4u* h = reinterpret_cast<const v4u*>(a.h) + (int64_t)row * 2 * Iv;
    const v4u* ga = reinterpret_cast<const v4u*>(a.grad_act) + (int64_t)row * Iv;
    v4u* out = reinterpret_cast<v4u*>(a.out) + (int64_t)row * 2 * Iv;
    float sum = 0.0f;
    constexpr int kBatch = 4;  // as above
    for (int32_t v0 = lane; v0 < Iv; v0 += kBatch * kWave) {
        v4u va[kBatch], vb[kBatch], vg[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int32_t v = min(v0 + i * kWave, Iv - 1);
            va[i] = __builtin_nontemporal_load(h + v);
            vb[i] = __builtin_nontemporal_load(h + Iv + v);
            vg[i] = __builtin_nontemporal_load(ga + v);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int32_t v = v0 + i * kWave;
            if (v >= Iv) break;
            v4u oa, ob;
            backward8(va[i], vb[i], vg[i], w, oa, ob, sum);
            __builtin_nontemporal_store(oa, out + v);
            __builtin_nontemporal_store(ob, out + Iv + v);
        }
    }
    if (wanted) {
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o, kWave);
        if (lane == 0) a.grad_probs[at] = sum;
    }
}

// One wave per slot, in launches that fit one grid's work-items.
template <typename Kernel>
hipError_t by_slots(Kernel kernel, const SwigluArgs& a, hipStream_t stream) {
    const int64_t slots = (int64_t)a.T * a.Kp;
    constexpr int64_t chunk = 0xFFFFFFFFll / kSwThreads * kSwWaves;
    for (int64_t s0 = 0; s0 < slots; s0 += chunk) {
        const int64_t n = slots - s0 < chunk ? slots - s0 : chunk;
        hipLaunchKernelGGL(kernel, dim3((unsigned)((n + kSwWaves - 1) / kSwWaves)), dim3(kSwThreads), 0, stream, a, s0,
                           s0 + n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_swiglu(const SwigluArgs& a, hipStream_t stream) { return by_slots(k_swiglu, a, stream); }

hipError_t launch_swiglu_bwd(const SwigluArgs& a, hipStream_t stream) { return by_slots(k_swiglu_bwd, a, stream); }

}  // namespace epx
