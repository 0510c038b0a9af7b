// Router of the expert layer: the top-k experts and weights of every token
// from its logits, and the gradient of the weights with respect to the
// logits (NeMo AutoModel token_dispatcher page, TokenDispatcherConfig.
// moe_router_dtype: fp32 routing weights; fused_a2a page,
// HybridEPDispatch.forward: topk_idx with -1 for unused slots).
//
// One wave per token; lane l holds experts l, l + 64, ...
#include "epx_device.h"

namespace epx {
namespace {

constexpr int kTopkThreads = 256;
constexpr int kTopkWaves = kTopkThreads / kWave;

template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

__device__ __forceinline__ float load_logit(const TopkArgs& a, int64_t i) {
    if (a.bf16) return bf16_lo(static_cast<const uint16_t*>(a.logits)[i]);
    return static_cast<const float*>(a.logits)[i];
}

// VPL: experts of a lane.
template <int VPL>
__global__ __launch_bounds__(kTopkThreads) void k_route(TopkArgs a) {
    __shared__ double s_key[kTopkWaves][VPL * kWave];
    const int w = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int32_t t = uniform((int32_t)(blockIdx.x * kTopkWaves + w));
    if (t >= a.T) return;  // no barrier below: each wave uses its own part of s_key
    const int64_t row = (int64_t)t * a.E;
    if (a.mask != nullptr && a.mask[t] == 0) {
        if (lane < a.K) {
            a.ids[(int64_t)t * a.K + lane] = -1;
            a.probs[(int64_t)t * a.K + lane] = 0.0f;
        }
        return;
    }
    float z[VPL];
    double key[VPL];
    float zmax = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int32_t e = i * kWave + lane;
        z[i] = e < a.E ? load_logit(a, row + e) : -INFINITY;
        zmax = fmaxf(zmax, z[i]);
    }
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) zmax = fmaxf(zmax, __shfl_xor(zmax, o, kWave));
    double total = 1.0;
    if (!a.sigmoid) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i * kWave + lane < a.E) sum += exp((double)z[i] - (double)zmax);
        total = wave_sum(sum);
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int32_t e = i * kWave + lane;
        key[i] = z[i];
        if (a.bias != nullptr && e < a.E) {
            const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)z[i])) : exp((double)z[i] - (double)zmax) / total;
            key[i] = s + (double)a.bias[e];
        }
        if (!(z[i] > -INFINITY) || e >= a.E) key[i] = -INFINITY;
    }
    if (a.groups > 1) {
        const int per = a.E / a.groups;
#pragma unroll
        for (int i = 0; i < VPL; ++i) s_key[w][i * kWave + lane] = key[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        double gkey = -INFINITY;
        if (lane < a.groups) {
            double b0 = -INFINITY, b1 = -INFINITY;
            for (int j = 0; j < per; ++j) {
                const double k = s_key[w][lane * per + j];
                b1 = k > b0 ? b0 : (k > b1 ? k : b1);
                b0 = k > b0 ? k : b0;
            }
            gkey = a.bias != nullptr && per > 1 ? b0 + b1 : b0;
        }
        int before = 0;  // groups that come before this one
        for (int g = 0; g < a.groups; ++g) {
            const double other = __shfl(gkey, g, kWave);
            before += other > gkey || (other == gkey && g < lane);
        }
        const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && before < a.top_groups);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int32_t e = i * kWave + lane;
            if (e >= a.E || !((kept >> (e / per)) & 1)) key[i] = -INFINITY;
        }
    }
    int32_t my_id = -1;
    float my_s = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        double best = -INFINITY;
        int32_t at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i * kWave + lane;
            }
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) {
            const double ob = __shfl_xor(best, o, kWave);
            const int32_t oa = __shfl_xor(at, o, kWave);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
            }
        }
        if (!(best > -INFINITY)) break;  // no expert left to choose
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (at == i * kWave + lane) {
                key[i] = -INFINITY;
                s = z[i];
            }
        s = __shfl(s, at & (kWave - 1), kWave);
        s = a.sigmoid ? 1.0f / (1.0f + expf(-s)) : expf(s - zmax) / (float)total;
        if (lane == k) {
            my_id = at;
            my_s = s;
        }
    }
    float p = my_s;
    if (a.normalize) p = my_s / (wave_sum(my_s) + 1e-20f);
    if (lane < a.K) {
        a.ids[(int64_t)t * a.K + lane] = my_id;
        a.probs[(int64_t)t * a.K + lane] = a.scale * p;
    }
}

__global__ __launch_bounds__(kTopkThreads) void k_route_bwd(TopkArgs a) {
    const int w = threadIdx.x / kWave, lane = threadIdx.x & (kWave - 1);
    const int32_t t = uniform((int32_t)(blockIdx.x * kTopkWaves + w));
    if (t >= a.T) return;
    const int64_t row = (int64_t)t * a.E;
    int32_t id = lane < a.K ? a.ids[(int64_t)t * a.K + lane] : -1;
    if (id < 0 || id >= a.E) id = -1;
    const bool any = __builtin_amdgcn_ballot_w64(id >= 0) != 0;
    const float g = id >= 0 ? a.grad_probs[(int64_t)t * a.K + lane] : 0.0f;
    const float zk = id >= 0 ? load_logit(a, row + id) : 0.0f;
    float zmax = 0.0f, total = 1.0f;
    if (!a.sigmoid && any) {
        zmax = -INFINITY;
        for (int32_t e = lane; e < a.E; e += kWave) zmax = fmaxf(zmax, load_logit(a, row + e));
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) zmax = fmaxf(zmax, __shfl_xor(zmax, o, kWave));
        total = 0.0f;
        for (int32_t e = lane; e < a.E; e += kWave) total += expf(load_logit(a, row + e) - zmax);
        total = wave_sum(total);
    }
    float q = 0.0f;
    if (id >= 0) q = a.sigmoid ? 1.0f / (1.0f + expf(-zk)) : expf(zk - zmax) / total;
    float gq = a.scale * g;
    if (a.normalize) {
        const float Q = wave_sum(q) + 1e-20f;
        gq = a.scale * (g - wave_sum(g * q) / Q) / Q;
    }
    if (id < 0) gq = 0.0f;
    const float dot = wave_sum(gq * q);
    const float own = a.sigmoid ? gq * q * (1.0f / (1.0f + expf(zk))) : gq;
    for (int32_t e0 = 0; e0 < a.E; e0 += kWave) {
        const int32_t e = e0 + lane;
        float sum = 0.0f;  // of the slots that chose e
        for (int k = 0; k < a.K; ++k) {
            const float o = __shfl(own, k, kWave);
            sum += __shfl(id, k, kWave) == e ? o : 0.0f;
        }
        float gz = sum;
        if (!a.sigmoid && any && e < a.E) gz = expf(load_logit(a, row + e) - zmax) / total * (sum - dot);
        if (e >= a.E) continue;
        if (a.bf16)
            static_cast<uint16_t*>(a.grad_logits)[row + e] = (uint16_t)f32_to_bf16(gz);
        else
            static_cast<float*>(a.grad_logits)[row + e] = gz;
    }
}

template <int VPL>
hipError_t route(const TopkArgs& a, hipStream_t stream) {
    const unsigned blocks = (unsigned)((a.T + kTopkWaves - 1) / kTopkWaves);
    hipLaunchKernelGGL(k_route<VPL>, dim3(blocks), dim3(kTopkThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const TopkArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const int vpl = (a.E + kWave - 1) / kWave;
    if (vpl <= 1) return route<1>(a, stream);
    if (vpl <= 2) return route<2>(a, stream);
    if (vpl <= 4) return route<4>(a, stream);
    if (vpl <= 8) return route<8>(a, stream);
    if (vpl <= 16) return route<16>(a, stream);
    return route<32>(a, stream);
}

hipError_t launch_route_bwd(const TopkArgs& a, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    const unsigned blocks = (unsigned)((a.T + kTopkWaves - 1) / kTopkWaves);
    hipLaunchKernelGGL(k_route_bwd, dim3(blocks), dim3(kTopkThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace epx
