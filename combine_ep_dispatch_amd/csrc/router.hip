// Router of the expert layer: the top-k experts and weights of every token
// from its logits, and the gradient of the weights with respect to the
// logits (NeMo AutoModel token_dispatcher page, TokenDispatcherConfig.
// moe_router_dtype: fp32 routing weights; fused_a2a page,
// HybridEPDispatch.forward: topk_idx with -1 for unused slots).
//
// One wave per token; lane l holds experts [l VPL, (l + 1) VPL).  (Up to 256
// experts and 16 slots four tokens share a wave: the gradient, and the choice
// where there is neither bias nor groups; see the narrow forms.)  Keys are
// 32-bit integers that order like the floats they stand for, so that the
// largest of a wave is six cross-lane maxima; the K experts are taken one by
// one.
//
// Without a bias a key is the logit, and the order is exact.  With one it is
// score + bias, whose fp32 value is off by a few roundings (key_error below):
// where other keys lie closer to the largest than that, these few are compared
// in 64 bits, where groups' keys do, the groups are ranked in 64 bits, and where
// many experts' do, the token is chosen again from 64-bit keys.  So is every token
// where the groups do not fill whole lanes (E other than 64 VPL, or a number of
// groups that is no power of two), without a bias too.
//
// What bounds it: a few tokens, the launch and K dependent choices (16 tokens
// of 256 experts, 4 of 8 groups, top-8: 6.9 us); many, instructions, for a
// token's logits are read once (4096 tokens: 13.0 us forward, 5.5 backward, of
// 1.7 us of bytes; in 64-bit keys 160 experts in 8 groups 16 us, 240 in 4 20;
// 65 536 tokens of 64, four a wave: 12.3 us forward and 10.8 backward, 43 with
// a wave each, 119 with 64-bit keys throughout).
#include "epx_device.h"

namespace epx {
namespace {

constexpr int kTopkThreads = 256;
constexpr int kTopkWaves = kTopkThreads / kWave;

constexpr int kMaxClose = 8;  // keys too close to tell that are settled one by one

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// DPP controls for a reduction over the wave: row shifts by 1, 2, 4 and 8
// lanes, then the last lane of a row into the next rows.  Lane 63 has it all.
template <typename F>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t identity, F f) {
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)identity, (int)v, 0x111, 0xf, 0xf, false));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)identity, (int)v, 0x112, 0xf, 0xf, false));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)identity, (int)v, 0x114, 0xf, 0xf, false));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)identity, (int)v, 0x118, 0xf, 0xf, false));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)identity, (int)v, 0x142, 0xa, 0xf, false));
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)identity, (int)v, 0x143, 0xc, 0xf, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float wave_sum(float v) {
    return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// Floats as integers of the same order, from 1 on (0: no candidate); NaN has none.
__device__ __forceinline__ uint32_t ordered(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);  // -0 and +0 are one value
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ float lane_value(float v, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

template <bool BF16>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
    if constexpr (BF16) return bf16_lo(static_cast<const uint16_t*>(p)[i]);
    return static_cast<const float*>(p)[i];
}

// The lane's VPL logits; -infinity past the last expert.  Rows of 64 VPL
// experts are read as vectors.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_logits(const TopkArgs& a, int64_t row, int lane, float (&z)[VPL]) {
    if (VPL % 4 == 0 && a.E == VPL * kWave) {
#pragma unroll
        for (int i = 0; i < VPL / 4 * 4; i += 4) {
            const int64_t at = row + lane * VPL + i;
            if constexpr (BF16) {
                const v2u v = *reinterpret_cast<const v2u*>(static_cast<const uint16_t*>(a.logits) + at);
                z[i] = bf16_lo(v.x), z[i + 1] = bf16_hi(v.x), z[i + 2] = bf16_lo(v.y), z[i + 3] = bf16_hi(v.y);
            } else {
                const v4u v = *reinterpret_cast<const v4u*>(static_cast<const float*>(a.logits) + at);
#pragma unroll
                for (int j = 0; j < 4; ++j) z[i + j] = __uint_as_float(v[j]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int32_t e = lane * VPL + i;
        z[i] = e < a.E ? logit<BF16>(a.logits, row + e) : -INFINITY;
    }
}

// A bound on how far an fp32 key with a bias is from the 64-bit one.  Sigmoid:
// exp2 of a rounded argument, 1 + e, the reciprocal, the sum with the bias:
// each at most 2^-24 of a value of at most 1, or of the key.  Softmax: exp's
// argument is rounded relative to its size d (d exp(-d) < 0.4), the sum over
// the experts and the division by it: fewer than 40 + VPL such roundings.
__device__ __forceinline__ float key_error(const TopkArgs& a, float largest, int vpl) {
    return ((a.sigmoid ? 6.0f : 42.0f + vpl) + largest) * 1.1920929e-7f;  // 2^-23
}

// The two largest of two sorted pairs.
template <typename T>
__device__ __forceinline__ void merge(T& b0, T& b1, T o0, T o1) {
    const T lo = b0 < o0 ? b0 : o0, hi = b1 < o1 ? o1 : b1;
    b0 = b0 < o0 ? o0 : b0;
    b1 = lo < hi ? hi : lo;
}

// Largest (with a bias: sum of the two largest) key of every group, in all
// lanes that hold the group's experts; per: lanes of a group.  Only where
// every lane's experts belong to one group.
template <int VPL>
__device__ __forceinline__ float group_key(const float (&key)[VPL], int per, bool two) {
    float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        b1 = fmaxf(b1, fminf(b0, key[i]));
        b0 = fmaxf(b0, key[i]);
    }
    auto across = [&](int ctrl_is, float v) {
        const int u = __float_as_int(v);
        switch (ctrl_is) {
            case 1: return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0xB1, 0xf, 0xf, false));   // lane ^ 1
            case 2: return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0x4E, 0xf, 0xf, false));   // lane ^ 2
            case 4: return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0x141, 0xf, 0xf, false));  // 7 - lane of 8
            case 8: return __int_as_float(__builtin_amdgcn_update_dpp(u, u, 0x140, 0xf, 0xf, false));  // 15 - lane of 16
            default: return __shfl_xor(v, ctrl_is, kWave);
        }
    };
#define EPX_MERGE(n)                                         \
    if (per > n) {                                           \
        const float o0 = across(n, b0), o1 = across(n, b1);  \
        merge(b0, b1, o0, o1);                               \
    }
    EPX_MERGE(1) EPX_MERGE(2) EPX_MERGE(4) EPX_MERGE(8) EPX_MERGE(16) EPX_MERGE(32)
#undef EPX_MERGE
    return two ? b0 + b1 : b0;
}

// The 64-bit key of an expert with logit z; total: sum of exp(z - zmax) in 64 bits.
__device__ __forceinline__ double exact_key(const TopkArgs& a, float z, float zmax, double total, int32_t e) {
    const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)z)) : exp((double)z - (double)zmax) / total;
    return s + (double)a.bias[e];
}

template <int VPL>
__device__ __forceinline__ double exact_total(const TopkArgs& a, const float (&z)[VPL], float zmax, int lane) {
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (lane * VPL + i < a.E) total += exp((double)z[i] - (double)zmax);
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) total += __shfl_xor(total, o, kWave);
    return total;
}

// How many groups come before the lane's, from 64-bit keys; lanes: of a group.
template <int VPL>
__device__ __forceinline__ int exact_group_rank(const TopkArgs& a, const float (&z)[VPL], float zmax, int lane, int lanes) {
    const double total = a.sigmoid ? 1.0 : exact_total<VPL>(a, z, zmax, lane);
    double b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
        if (z[i] > -INFINITY) merge(b0, b1, exact_key(a, z[i], zmax, total, lane * VPL + i), (double)-INFINITY);
    for (int o = 1; o < lanes; o *= 2) {
        const double o0 = __shfl_xor(b0, o, kWave), o1 = __shfl_xor(b1, o, kWave);
        merge(b0, b1, o0, o1);
    }
    const double mine = lanes * VPL > 1 ? b0 + b1 : b0;
    int before = 0;
    for (int g = 0; g < a.groups; ++g) {
        const double other = __shfl(mine, g * lanes, kWave);
        before += other > mine || (other == mine && g < lane / lanes);
    }
    return before;
}

// The choice in full: keys of 64 bits where there is a bias, groups of any
// size.  Lane k gets the k-th expert (-1: none) and its logit.
template <int VPL>
__device__ __forceinline__ void choose_exactly(const TopkArgs& a, bool biased, const float (&z)[VPL], float zmax, int lane,
                                               double* s_key, int32_t& my_id, float& my_z) {
    double key[VPL];
    const double total = biased && !a.sigmoid ? exact_total<VPL>(a, z, zmax, lane) : 1.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int32_t e = lane * VPL + i;
        key[i] = z[i];
        if (biased && e < a.E) key[i] = exact_key(a, z[i], zmax, total, e);
        if (!(z[i] > -INFINITY) || e >= a.E) key[i] = -INFINITY;
    }
    if (a.groups > 1) {
        const int per = a.E / a.groups;
#pragma unroll
        for (int i = 0; i < VPL; ++i) s_key[lane * VPL + i] = key[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        double gkey = -INFINITY;
        if (lane < a.groups) {
            double b0 = -INFINITY, b1 = -INFINITY;
            for (int j = 0; j < per; ++j) {
                const double k = s_key[lane * per + j];
                merge(b0, b1, k, (double)-INFINITY);
            }
            gkey = biased && per > 1 ? b0 + b1 : b0;
        }
        int before = 0;  // groups that come before this one
        for (int g = 0; g < a.groups; ++g) {
            const double other = __shfl(gkey, g, kWave);
            before += other > gkey || (other == gkey && g < lane);
        }
        const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && before < a.top_groups);
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            const int32_t e = lane * VPL + i;
            if (e >= a.E || !((kept >> (e / per)) & 1)) key[i] = -INFINITY;
        }
    }
    my_id = -1;
    for (int k = 0; k < a.K; ++k) {
        double best = -INFINITY;
        int32_t at = 0x7FFFFFFF;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane * VPL + i;
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
        float zk = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (at == lane * VPL + i) {
                key[i] = -INFINITY;
                zk = z[i];
            }
        zk = __shfl(zk, at / VPL, kWave);
        if (lane == k) {
            my_id = at;
            my_z = zk;
        }
    }
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(kTopkThreads) void k_route(TopkArgs a) {
    __shared__ double s_key[kTopkWaves][VPL * kWave];
    const int w = uniform((int32_t)(threadIdx.x / kWave)), lane = threadIdx.x & (kWave - 1);
    const int32_t t = (int32_t)(blockIdx.x * kTopkWaves) + w;
    if (t >= a.T) return;  // no barrier below: each wave uses its own part of s_key
    const int64_t slot = (int64_t)t * a.K + lane;
    if (a.mask != nullptr && a.mask[t] == 0) {
        if (lane < a.K) {
            a.ids[slot] = -1;
            a.probs[slot] = 0.0f;
        }
        return;
    }
    float z[VPL];
    load_logits<VPL, BF16>(a, (int64_t)t * a.E, lane, z);
    float zmax = -INFINITY, total = 1.0f;
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) zmax = fmaxf(zmax, z[i]);
        zmax = unordered(wave_max(ordered(zmax)));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum += expf(z[i] - zmax);
        total = wave_sum(sum);
    }
    // Softmax over a NaN or +infinity leaves no scores to add a bias to (its sum is
    // NaN): the choice goes by the logits then, and the weights show the NaN.
    const bool biased = a.bias != nullptr && total == total;
    // keys, in fp32; unavailable experts have -infinity
    float key[VPL];
    float largest = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        key[i] = z[i];
        if (biased) {
            const int32_t e = lane * VPL + i;
            const float s = a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z[i]))
                                      : expf(z[i] - zmax) / total;
            key[i] = s + (e < a.E ? a.bias[e] : 0.0f);
            largest = fmaxf(largest, fabsf(key[i]));
        }
        if (!(z[i] > -INFINITY)) key[i] = -INFINITY;
    }
    float off = 0.0f;
    if (biased) off = 2.0f * key_error(a, __uint_as_float(wave_max(__float_as_uint(largest))), VPL);

    // Groups whose experts fill whole lanes here; the others in full.
    const int per = a.E / a.groups;  // experts of a group
    bool sure = a.groups == 1 || (a.E == VPL * kWave && per % VPL == 0 &&
                                  (a.groups & (a.groups - 1)) == 0);
    if (sure && a.groups > 1) {
        const int lanes = per / VPL;
        const float gkey = group_key<VPL>(key, lanes, biased && per > 1);
        int before = 0, maybe = 0;  // groups that come before this one, for sure and at most
        for (int g = 0; g < a.groups; ++g) {
            const float other = lane_value(gkey, g * lanes);
            const bool mine = lane / lanes == g;
            if (biased) {
                before += other > gkey + 2.0f * off;
                maybe += !mine && !(other < gkey - 2.0f * off);
            } else {
                before += other > gkey || (other == gkey && g < lane / lanes);
            }
        }
        if (!biased) maybe = before;
        if (__builtin_amdgcn_ballot_w64(before < a.top_groups && maybe >= a.top_groups) != 0)
            before = exact_group_rank<VPL>(a, z, zmax, lane, lanes);
        if (before >= a.top_groups)
#pragma unroll
            for (int i = 0; i < VPL; ++i) key[i] = -INFINITY;
    }
    int32_t my_id = -1;
    float my_z = 0.0f;
    if (sure) {
        uint32_t u[VPL];
#pragma unroll
        for (int i = 0; i < VPL; ++i) u[i] = key[i] > -INFINITY ? ordered(key[i]) : 0u;
        double exact = 0.0;  // softmax's sum in 64 bits, once it is needed
        for (int k = 0; k < a.K; ++k) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) m = m < u[i] ? u[i] : m;
            uint32_t best = wave_max(m);
            if (best == 0) break;  // no expert left to choose
            int32_t chosen = -1;
            if (biased) {
                const uint32_t near = ordered(unordered(best) - off);
                int close = 0;
#pragma unroll
                for (int i = 0; i < VPL; ++i) close += __builtin_popcountll(__builtin_amdgcn_ballot_w64(u[i] >= near));
                if (close > kMaxClose) {
                    sure = false;
                    break;
                }
                if (close > 1) {  // the largest of these in 64 bits
                    if (!a.sigmoid && exact == 0.0) exact = exact_total<VPL>(a, z, zmax, lane);
                    double top = -INFINITY;
#pragma unroll
                    for (int i = 0; i < VPL; ++i) {
                        uint64_t left = __builtin_amdgcn_ballot_w64(u[i] >= near);
                        if (left == 0) continue;
                        const double mine = u[i] >= near ? exact_key(a, z[i], zmax, exact, lane * VPL + i) : 0.0;
                        for (; left != 0; left &= left - 1) {
                            const int from = __builtin_ctzll(left);
                            const uint64_t bits = __builtin_bit_cast(uint64_t, mine);
                            const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)bits, from);
                            const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(bits >> 32), from);
                            const double other = __builtin_bit_cast(double, hi << 32 | lo);
                            const int32_t e = from * VPL + i;
                            if (other > top || (other == top && e < chosen)) {
                                top = other;
                                chosen = e;
                            }
                        }
                    }
                }
            }
            int at = 0;
            int from;
            if (chosen >= 0) {
                from = chosen / VPL;
                at = chosen - from * VPL;
            } else {
#pragma unroll
                for (int i = VPL - 1; i >= 0; --i)
                    if (u[i] == best) at = i;
                from = __builtin_ctzll(__builtin_amdgcn_ballot_w64(m == best));
                at = __builtin_amdgcn_readlane(at, from);
            }
            float zk = z[0];
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (i == at) zk = z[i];
                if (i == at && lane == from) u[i] = 0;
            }
            zk = lane_value(zk, from);
            if (lane == k) {
                my_id = from * VPL + at;
                my_z = zk;
            }
        }
    }
    if (!sure) choose_exactly<VPL>(a, biased, z, zmax, lane, s_key[w], my_id, my_z);
    float q = 0.0f;
    if (my_id >= 0) q = a.sigmoid ? 1.0f / (1.0f + expf(-my_z)) : expf(my_z - zmax) / total;
    float p = q;
    if (a.normalize) p = q / (wave_sum(q) + 1e-20f);
    if (lane < a.K) {
        a.ids[slot] = my_id;
        a.probs[slot] = a.scale * p;
    }
}

// The lane's VPL gradients of a row that `lanes` lanes hold.
template <int VPL, bool BF16>
__device__ __forceinline__ void store_gradient(const TopkArgs& a, int64_t row, int lane, int lanes, const float (&gz)[VPL]) {
    if (VPL % 4 == 0 && a.E == VPL * lanes) {
#pragma unroll
        for (int i = 0; i < VPL / 4 * 4; i += 4) {
            const int64_t at = row + lane * VPL + i;
            if constexpr (BF16) {
                const v2u v = {pack_bf16x2(gz[i], gz[i + 1]), pack_bf16x2(gz[i + 2], gz[i + 3])};
                *reinterpret_cast<v2u*>(static_cast<uint16_t*>(a.grad_logits) + at) = v;
            } else {
                const v4u v = {__float_as_uint(gz[i]), __float_as_uint(gz[i + 1]), __float_as_uint(gz[i + 2]),
                               __float_as_uint(gz[i + 3])};
                *reinterpret_cast<v4u*>(static_cast<float*>(a.grad_logits) + at) = v;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int32_t e = lane * VPL + i;
        if (e >= a.E) continue;
        if constexpr (BF16)
            static_cast<uint16_t*>(a.grad_logits)[row + e] = (uint16_t)f32_to_bf16(gz[i]);
        else
            static_cast<float*>(a.grad_logits)[row + e] = gz[i];
    }
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(kTopkThreads) void k_route_bwd(TopkArgs a) {
    const int w = uniform((int32_t)(threadIdx.x / kWave)), lane = threadIdx.x & (kWave - 1);
    const int32_t t = (int32_t)(blockIdx.x * kTopkWaves) + w;
    if (t >= a.T) return;
    const int64_t row = (int64_t)t * a.E;
    int32_t id = -1;
    float g = 0.0f, zk = 0.0f, z[VPL];
    if (lane < a.K) {
        id = a.ids[(int64_t)t * a.K + lane];
        g = a.grad_probs[(int64_t)t * a.K + lane];
    }
    if (!a.sigmoid) load_logits<VPL, BF16>(a, row, lane, z);
    if (id < 0 || id >= a.E) {
        id = -1;
        g = 0.0f;
    } else {
        zk = logit<BF16>(a.logits, row + id);
    }
    const bool any = __builtin_amdgcn_ballot_w64(id >= 0) != 0;
    float zmax = 0.0f, total = 1.0f;
    if (!a.sigmoid) {
        zmax = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) zmax = fmaxf(zmax, z[i]);
        zmax = unordered(wave_max(ordered(zmax)));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            z[i] = expf(z[i] - zmax);
            sum += z[i];
        }
        total = wave_sum(sum);
    }
    float q = 0.0f;
    if (id >= 0) q = a.sigmoid ? 1.0f / (1.0f + expf(-zk)) : expf(zk - zmax) / total;
    // g_k - sum_j g_j q_j / Q as (sum_j (g_k - g_j) q_j + 1e-20 g_k) / Q: weights
    // of nearly equal gradients, or a token's only one, cancel exactly.
    float gq = a.scale * g, dot = 0.0f;
    if (a.normalize) {
        const float Q = wave_sum(q) + 1e-20f, gq_sum = wave_sum(g * q);
        float diff = 1e-20f * g;
        for (int j = 0; j < a.K; ++j) diff += (g - lane_value(g, j)) * lane_value(q, j);
        gq = a.scale * diff / Q / Q;
        dot = a.scale * 1e-20f * gq_sum / Q / Q;  // sum_k gq_k q_k: the differences cancel in pairs
    }
    if (id < 0) gq = 0.0f;
    if (!a.normalize) dot = wave_sum(gq * q);
    const float own = a.sigmoid ? gq * q * (1.0f / (1.0f + expf(zk))) : gq;
    float gz[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) gz[i] = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        const int32_t e = __builtin_amdgcn_readlane(id, k);
        const float o = lane_value(own, k);
#pragma unroll
        for (int i = 0; i < VPL; ++i) gz[i] += e == lane * VPL + i ? o : 0.0f;
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) gz[i] = any ? z[i] / total * (gz[i] - dot) : 0.0f;
    }
    store_gradient<VPL, BF16>(a, row, lane, kWave, gz);
}

// Narrow forms, four tokens a wave: a token has the 16 lanes of a DPP row, lane
// l of them experts [l VPL, (l + 1) VPL), so that each cross-lane step serves
// four tokens.  For at most 16 slots, and forward only where the logits are the
// keys (no bias, no groups).  65 536 tokens of 64 experts: forward 13.0 us
// (25.6 with a wave per token), backward 10.4 (19.0).
constexpr int kRowLanes = 16;
constexpr int kNarrowTokens = kTopkWaves * kWave / kRowLanes;  // of a workgroup

template <typename F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, F f) {
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xf, 0xf, false));   // lane ^ 1
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xf, 0xf, false));   // lane ^ 2
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x141, 0xf, 0xf, false));  // 7 - lane of 8
    v = f(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x140, 0xf, 0xf, false));  // 15 - lane of 16
    return v;
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
    return row_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
__device__ __forceinline__ float row_sum(float v) {
    return __uint_as_float(row_reduce(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// As load_logits and its store, for 16 lanes a row.
template <int VPL, bool BF16>
__device__ __forceinline__ void load_row(const TopkArgs& a, int64_t row, int l, bool on, float (&z)[VPL]) {
    if (VPL % 4 == 0 && a.E == VPL * kRowLanes) {
#pragma unroll
        for (int i = 0; i < VPL / 4 * 4; i += 4) {
            const int64_t at = on ? row + l * VPL + i : 0;
            if constexpr (BF16) {
                const v2u v = *reinterpret_cast<const v2u*>(static_cast<const uint16_t*>(a.logits) + at);
                z[i] = bf16_lo(v.x), z[i + 1] = bf16_hi(v.x), z[i + 2] = bf16_lo(v.y), z[i + 3] = bf16_hi(v.y);
            } else {
                const v4u v = *reinterpret_cast<const v4u*>(static_cast<const float*>(a.logits) + at);
#pragma unroll
                for (int j = 0; j < 4; ++j) z[i + j] = __uint_as_float(v[j]);
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const int32_t e = l * VPL + i;
        z[i] = on && e < a.E ? logit<BF16>(a.logits, row + e) : -INFINITY;
    }
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(kTopkThreads) void k_route_narrow(TopkArgs a) {
    __shared__ int32_t s_id[kNarrowTokens][kRowLanes];
    __shared__ float s_z[kNarrowTokens][kRowLanes];
    const int lane = threadIdx.x & (kWave - 1), l = lane % kRowLanes, mine = threadIdx.x / kRowLanes;
    const int32_t t = (int32_t)(blockIdx.x * kNarrowTokens) + mine;
    const bool in = t < a.T, on = in && (a.mask == nullptr || a.mask[t] != 0);
    float z[VPL];
    load_row<VPL, BF16>(a, (int64_t)t * a.E, l, on, z);
    float zmax = -INFINITY, total = 1.0f;
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) zmax = fmaxf(zmax, z[i]);
        zmax = unordered(row_max(ordered(zmax)));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum += expf(z[i] - zmax);
        total = row_sum(sum);
    }
    uint32_t u[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) u[i] = on && z[i] > -INFINITY ? ordered(z[i]) : 0u;
    s_id[mine][l] = -1;  // each row writes and reads its own line of these, in program order
    for (int k = 0; k < a.K; ++k) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) m = m < u[i] ? u[i] : m;
        const uint32_t best = row_max(m);
        if (__builtin_amdgcn_ballot_w64(best != 0) == 0) break;  // no token has an expert left to choose
        const uint32_t at_best = (uint32_t)(__builtin_amdgcn_ballot_w64(m == best && best != 0) >> (lane & 48)) & 0xFFFFu;
        if (best != 0 && l == __builtin_ctz(at_best | 0x10000u)) {  // the lowest lane that holds it, and its lowest
            int at = 0;
#pragma unroll
            for (int i = VPL - 1; i >= 0; --i)
                if (u[i] == best) at = i;
#pragma unroll
            for (int i = 0; i < VPL; ++i)
                if (i == at) u[i] = 0;
            s_id[mine][k] = l * VPL + at;
            s_z[mine][k] = unordered(best);  // the key is the logit
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int32_t id = s_id[mine][l];
    float q = 0.0f;
    if (id >= 0) {
        const float zk = s_z[mine][l];
        q = a.sigmoid ? 1.0f / (1.0f + expf(-zk)) : expf(zk - zmax) / total;
    }
    float p = q;
    if (a.normalize) p = q / (row_sum(q) + 1e-20f);
    if (in && l < a.K) {
        a.ids[(int64_t)t * a.K + l] = id;
        a.probs[(int64_t)t * a.K + l] = a.scale * p;
    }
}

template <int VPL, bool BF16>
__global__ __launch_bounds__(kTopkThreads) void k_route_bwd_narrow(TopkArgs a) {
    __shared__ int32_t s_id[kNarrowTokens][kRowLanes];
    __shared__ float s_own[kNarrowTokens][kRowLanes], s_g[kNarrowTokens][kRowLanes], s_q[kNarrowTokens][kRowLanes];
    const int l = threadIdx.x % kRowLanes, mine = threadIdx.x / kRowLanes;
    const int32_t t = (int32_t)(blockIdx.x * kNarrowTokens) + mine;
    const bool in = t < a.T;
    const int64_t row = (int64_t)t * a.E;
    int32_t id = -1;
    float g = 0.0f, zk = 0.0f, z[VPL];
    if (in && l < a.K) {
        id = a.ids[(int64_t)t * a.K + l];
        g = a.grad_probs[(int64_t)t * a.K + l];
    }
    if (!a.sigmoid) load_row<VPL, BF16>(a, row, l, in, z);
    if (id < 0 || id >= a.E) {
        id = -1;
        g = 0.0f;
    } else {
        zk = logit<BF16>(a.logits, row + id);
    }
    const bool any = row_max(id >= 0) != 0;
    float zmax = 0.0f, total = 1.0f;
    if (!a.sigmoid) {
        zmax = -INFINITY;
#pragma unroll
        for (int i = 0; i < VPL; ++i) zmax = fmaxf(zmax, z[i]);
        zmax = unordered(row_max(ordered(zmax)));
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
            z[i] = expf(z[i] - zmax);
            sum += z[i];
        }
        total = row_sum(sum);
    }
    float q = 0.0f;
    if (id >= 0) q = a.sigmoid ? 1.0f / (1.0f + expf(-zk)) : expf(zk - zmax) / total;
    float gq = a.scale * g, dot = 0.0f;  // as in k_route_bwd
    if (a.normalize) {
        const float Q = row_sum(q) + 1e-20f, gq_sum = row_sum(g * q);
        s_g[mine][l] = g;
        s_q[mine][l] = q;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float diff = 1e-20f * g;
        for (int j = 0; j < a.K; ++j) diff += (g - s_g[mine][j]) * s_q[mine][j];
        gq = a.scale * diff / Q / Q;
        dot = a.scale * 1e-20f * gq_sum / Q / Q;
    }
    if (id < 0) gq = 0.0f;
    if (!a.normalize) dot = row_sum(gq * q);
    s_id[mine][l] = id;
    s_own[mine][l] = a.sigmoid ? gq * q * (1.0f / (1.0f + expf(zk))) : gq;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    float gz[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) gz[i] = 0.0f;
    for (int k = 0; k < a.K; ++k) {
        const int32_t e = s_id[mine][k];
        const float o = s_own[mine][k];
#pragma unroll
        for (int i = 0; i < VPL; ++i) gz[i] += e == l * VPL + i ? o : 0.0f;
    }
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) gz[i] = any ? z[i] / total * (gz[i] - dot) : 0.0f;
    }
    if (!in) return;
    store_gradient<VPL, BF16>(a, row, l, kRowLanes, gz);
}

template <int VPL>
hipError_t route(const TopkArgs& a, bool bwd, hipStream_t stream) {
    const dim3 blocks((unsigned)((a.T + kTopkWaves - 1) / kTopkWaves)), threads(kTopkThreads);
    if (bwd && a.bf16)
        hipLaunchKernelGGL((k_route_bwd<VPL, true>), blocks, threads, 0, stream, a);
    else if (bwd)
        hipLaunchKernelGGL((k_route_bwd<VPL, false>), blocks, threads, 0, stream, a);
    else if (a.bf16)
        hipLaunchKernelGGL((k_route<VPL, true>), blocks, threads, 0, stream, a);
    else
        hipLaunchKernelGGL((k_route<VPL, false>), blocks, threads, 0, stream, a);
    return hipGetLastError();
}

template <int VPL>
hipError_t narrow(const TopkArgs& a, bool bwd, hipStream_t stream) {
    const dim3 blocks((unsigned)((a.T + kNarrowTokens - 1) / kNarrowTokens)), threads(kTopkThreads);
    if (bwd && a.bf16)
        hipLaunchKernelGGL((k_route_bwd_narrow<VPL, true>), blocks, threads, 0, stream, a);
    else if (bwd)
        hipLaunchKernelGGL((k_route_bwd_narrow<VPL, false>), blocks, threads, 0, stream, a);
    else if (a.bf16)
        hipLaunchKernelGGL((k_route_narrow<VPL, true>), blocks, threads, 0, stream, a);
    else
        hipLaunchKernelGGL((k_route_narrow<VPL, false>), blocks, threads, 0, stream, a);
    return hipGetLastError();
}

hipError_t by_experts(const TopkArgs& a, bool bwd, hipStream_t stream) {
    if (a.T == 0) return hipSuccess;
    if (a.K <= kRowLanes && a.E <= 16 * kRowLanes && (bwd || (a.bias == nullptr && a.groups == 1))) {
        if (a.E <= kRowLanes) return narrow<1>(a, bwd, stream);
        if (a.E <= 2 * kRowLanes) return narrow<2>(a, bwd, stream);
        if (a.E <= 4 * kRowLanes) return narrow<4>(a, bwd, stream);
        if (a.E <= 8 * kRowLanes) return narrow<8>(a, bwd, stream);
        return narrow<16>(a, bwd, stream);
    }
    const int vpl = (a.E + kWave - 1) / kWave;
    if (vpl <= 1) return route<1>(a, bwd, stream);
    if (vpl <= 2) return route<2>(a, bwd, stream);
    if (vpl <= 4) return route<4>(a, bwd, stream);
    if (vpl <= 8) return route<8>(a, bwd, stream);
    if (vpl <= 16) return route<16>(a, bwd, stream);
    return route<32>(a, bwd, stream);
}

}  // namespace

hipError_t launch_route(const TopkArgs& a, hipStream_t stream) { return by_experts(a, false, stream); }

hipError_t launch_route_bwd(const TopkArgs& a, hipStream_t stream) { return by_experts(a, true, stream); }

}  // namespace epx
