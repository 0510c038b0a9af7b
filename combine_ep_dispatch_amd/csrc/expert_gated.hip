// The experts' gated block in one kernel, bf16 weights (gate rows, then up rows):
//   g = x[r] . w[e, i, :],  u = x[r] . w[e, I + i, :]
//   act[r, i] = w_r silu(g) u,   silu(g) = g s,   s = 1 / (1 + exp(-g))
// and its backward pass, which makes g and u again from x and w:
//   grad_h[r, i] = w_r ga u s (1 + g (1 - s)),   grad_h[r, I + i] = w_r ga g s
//   grad_probs[t, k] = sum_i ga silu(g) u
// g and u are not rounded between the product and the activation.  Low-rank
// adapters, if any, add to g and u before it.
//
// Against the product and the activation apart, the rows' 2 I values of h are neither
// written nor read.  The backward pass makes g and u again, which costs a product more
// but keeps nothing of 2 I values a row from one pass to the next: forward and backward
// the two calls take 1280 us where this takes 1570 (64 experts of 2048 x 1416, 49 152 rows).
// grad_h is rounded to bf16, the type that the products behind it multiply: their
// gradients are then off by 0.0023 of their norm, 0.0017 with grad_h in 32 bits.
//
// 32 experts of 4096 x 7168 (2 I x in): 128 rows 311 us, bound by reading 1.88 GB of
// weights (6.0 TB/s); 32 768 rows 1490 to 1610 us, 1190 to 1290 TFLOP/s, where one
// library product of as many operations reaches 1590.  Of a tile's time 89 % are its
// 112 steps, each 2290 cycles of which 2048 are matrix instructions; 3400 cycles find
// the tile, 2000 wait for its first step, 14 500 are the epilogue.  The backward
// epilogue takes 33 700: 64 experts of 2048 x 1416, 49 152 rows, forward and gradients
// 1560 us with the two products behind it.  There rows of 2832 bytes straddle the
// 128-byte lines of memory: 22 steps take 88 000 cycles instead of 55 700.
#include "expert_loop.h"
#include "gated_device.h"

namespace epx {
namespace {

template <int KF, int KN>
__device__ __forceinline__ void adapters_of(const BlockArgs& a, const LoopTile& t, int32_t c0, int32_t wn, f32x4 (&acc)[KF][KN]) {
    const int i = threadIdx.x % 16;
    add_adapters<KF, KN>(a, t.first, t.rows, wn, [&](int f, int32_t ad, int32_t c) {
        const int32_t col = c0 + f / 2 * 16 + i;  // of act
        const int64_t expert = (int64_t)ad * (a.e.E + a.e.shared) + t.expert;
        if (col >= a.I) return bf16x8{};
        return *reinterpret_cast<const bf16x8*>(a.l.b + (expert * a.e.on + f % 2 * a.I + col) * a.l.rank + c * 8);
    }, acc);
}

// BACKWARD: grad_h and the weights' gradients from grad_act (and act again, if wanted).
template <bool BACKWARD, bool LORA>
__global__ __launch_bounds__(kLoopThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_gated(BlockArgs a, int32_t ftiles) {
    __shared__ __align__(1024) uint16_t lds[kLoopLds / 2];
    const int lane = threadIdx.x & (kWave - 1), i = lane % 16, q = lane / 16;
    const int32_t I = a.I, in = a.e.in;
    GatedOperand fo;
    fo.init(in);
    auto start_f = [&](GatedOperand& op, const LoopTile& t) {
        const int32_t c0 = t.ft * (kTileF / 2);
        const bool on = t.expert >= 0;
        op.start(on ? a.e.w + ((int64_t)t.expert * a.e.on + c0) * in : a.e.w, on ? I : 0, on ? I - c0 : 0);
    };
    auto start_n = [&](auto& op, const LoopTile& t) {
        op.start(a.e.x + t.first * in, t.expert >= 0 ? t.rows : 0);
    };
    auto begin = [&](auto nt, const LoopTile& t, auto& acc) {
        using S = Shape<decltype(nt)::value>;
        if constexpr (LORA) adapters_of<S::kF, S::kN>(a, t, t.ft * (kTileF / 2) + S::wf() / 2, S::wn(), acc);
    };
    run_tiles(a.e, ftiles, in, lds, fo, start_f, start_n, begin, [&](auto nt, const LoopTile& t, auto& acc) {
        using S = Shape<decltype(nt)::value>;
        constexpr int KF = S::kF, KN = S::kN;
        const int wn = S::wn();
        const int32_t c0 = t.ft * (kTileF / 2) + S::wf() / 2;  // the wave's first column of act
        // acc[2 p][n][j], acc[2 p + 1][n][j]: g and u of column c0 + 16 p + 4 q + j, row wn + 16 n + i
        uint16_t* const act = static_cast<uint16_t*>(a.e.out);
        float w[KN];
        int32_t slot[KN];
        auto row_of = [&](int n) { return t.first + min(wn + n * 16 + i, t.rows - 1); };
        row_weights<KN>(a, row_of, w, slot);
        v2u ga[BACKWARD ? KN : 1][KF / 2];
        if constexpr (BACKWARD) {
#pragma unroll
            for (int n = 0; n < KN; ++n)
#pragma unroll
                for (int p = 0; p < KF / 2; ++p)
                    ga[n][p] = *reinterpret_cast<const v2u*>(a.grad_act + row_of(n) * I + min(c0 + p * 16 + q * 4, I - 4));
        }
#pragma unroll
        for (int n = 0; n < KN; ++n) {
            const int64_t r = row_of(n);
            const bool on = wn + n * 16 + i < t.rows;
            float sum = 0.0f;
#pragma unroll
            for (int p = 0; p < KF / 2; ++p) {
                const int32_t c = c0 + p * 16 + q * 4;
                const bool in = on && c < I;
                const f32x4 g = acc[2 * p][n], u = acc[2 * p + 1][n];
                float y[4], gg[4], gu[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float s = fast_sigmoid(g[j]), silu = g[j] * s;
                    y[j] = w[n] * (silu * u[j]);
                    if constexpr (BACKWARD) {
                        const float d = j % 2 ? bf16_hi(ga[n][p][j / 2]) : bf16_lo(ga[n][p][j / 2]), wd = w[n] * d;
                        sum += in ? d * (silu * u[j]) : 0.0f;
                        gg[j] = wd * u[j] * (s * (1.0f + g[j] * (1.0f - s)));
                        gu[j] = wd * silu;
                    }
                }
                if (!in) continue;
                if (act != nullptr)
                    *reinterpret_cast<v2u*>(act + r * I + c) = v2u{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
                if constexpr (BACKWARD) {
                    uint16_t* const gh = a.grad_h + r * 2 * I + c;
                    *reinterpret_cast<v2u*>(gh) = v2u{pack_bf16x2(gg[0], gg[1]), pack_bf16x2(gg[2], gg[3])};
                    *reinterpret_cast<v2u*>(gh + I) = v2u{pack_bf16x2(gu[0], gu[1]), pack_bf16x2(gu[2], gu[3])};
                }
            }
            if constexpr (BACKWARD) {
                if (a.parts == nullptr) continue;
                sum += __shfl_xor(sum, 16, kWave);
                sum += __shfl_xor(sum, 32, kWave);
                // the wave's columns are KF / 4 parts: the sum in the first, zeros in the others
                const int32_t parts = (I + kGatedPart - 1) / kGatedPart, part = c0 / kGatedPart + q;
                if (q < KF / 4 && on && slot[n] >= 0 && part < parts) a.parts[(int64_t)slot[n] * parts + part] = q == 0 ? sum : 0.0f;
            }
        }
    });
}

// grad_probs[t, k]: the parts of the slot's row in order; 0 where the slot has none.
__global__ __launch_bounds__(256) void k_gated_probs(BlockArgs a) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= (int64_t)a.T * a.K) return;
    const int32_t row = a.token_row[at / a.K * a.Kp + at % a.K], parts = (a.I + kGatedPart - 1) / kGatedPart;
    float sum = 0.0f;
    if (row >= 0 && row < a.e.R)
        for (int32_t p = 0; p < parts; ++p) sum += a.parts[at * parts + p];
    a.grad_probs[at] = sum;
}

template <bool BACKWARD>
hipError_t gated(const BlockArgs& a, hipStream_t stream) {
    const int32_t ftiles = (a.I + kTileF / 2 - 1) / (kTileF / 2);
    unsigned blocks;
    if (const hipError_t e = loop_blocks(a.e, ftiles, blocks)) return e;
    if (blocks == 0) return hipSuccess;
    if (a.l.rank > 0)
        hipLaunchKernelGGL((k_gated<BACKWARD, true>), dim3(blocks), dim3(kLoopThreads), 0, stream, a, ftiles);
    else
        hipLaunchKernelGGL((k_gated<BACKWARD, false>), dim3(blocks), dim3(kLoopThreads), 0, stream, a, ftiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gated(const BlockArgs& a, hipStream_t stream) { return gated<false>(a, stream); }

hipError_t launch_gated_bwd(const BlockArgs& a, hipStream_t stream) {
    if (const hipError_t e = gated<true>(a, stream)) return e;
    const int64_t slots = (int64_t)a.T * a.K;
    if (a.grad_probs == nullptr || slots == 0) return hipSuccess;
    hipLaunchKernelGGL(k_gated_probs, dim3((unsigned)((slots + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace epx
