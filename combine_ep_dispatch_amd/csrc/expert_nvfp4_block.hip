// The gated block over 4-bit weights, and the 4-bit product with adapters: the
// tiles of the 4-bit product with other ends, and bound by what bounds that: 8 rows of 8
// experts of 4096 x 7168 31 us, 576 rows of 65 250 us (4.3 TB/s), 3890 rows of 32 328 to
// 339 us (670 to 700 TFLOP/s; conversions, LDS reads and matrix instructions overlap little).  With
// 8 adapters of rank 16 576 rows take 266 to 282: each (adapter, 32 values of rank) is a round
// trip to memory behind the tile's last step.
//   act[r, i] = w_r silu(g) u,  g = rowscale[e, i] sum_h x[r, h] e2m1 e4m3 (+ adapters),  u: row I + i
#include "gated_device.h"
#include "lora_device.h"
#include "nvfp4_tile.h"

namespace epx {
namespace {

// A wave of 16 features has 8 of the gate and 8 of the up projection, in the lower
// and upper half of its lanes; one of 32 has 16 of each, in its two fragments.
template <int NT, int FW, int WAVES, int L, int BUFS, bool WORDS, bool GATED, bool LORA>
__global__ __launch_bounds__(WAVES * kWave) void k_nvfp4_block(BlockArgs a, int32_t ftiles) {
    using Tile = Nvfp4Tile<NT, FW, WAVES, L, BUFS, WORDS, GATED>;
    constexpr int KF = FW / 16, KN = NT / 16;
    __shared__ __align__(1024) uint8_t lds[BUFS * Tile::kBuffer];
    __shared__ int32_t scan[16];
    Tile::run(a.e, ftiles, lds, scan, [&](const RowTile& t, int32_t f0, int64_t row0, f32x4 (&acc)[KF][KN]) {
        const int lane = threadIdx.x & (kWave - 1), i = lane % 16, q = lane / 16;
        const int32_t features = GATED ? a.I : a.e.on;
        // feature `at` (0..15) of fragment g: its place among the projection's, and whether it is the up projection's
        auto feature = [&](int g, int at) { return f0 + (!GATED ? g * 16 + at : KF == 1 ? at % 8 : at); };
        auto up = [&](int g, int at) { return !GATED ? 0 : KF == 1 ? at / 8 : g; };
#pragma unroll
        for (int g = 0; g < KF; ++g) {
            const int32_t fe = feature(g, q * 4);
            const v2u rs = fe < features ? *reinterpret_cast<const v2u*>(a.e.rowscale + row0 + up(g, q * 4) * features + (fe - f0)) : v2u{};
            const f32x4 s = {bf16_lo(rs.x), bf16_hi(rs.x), bf16_lo(rs.y), bf16_hi(rs.y)};
#pragma unroll
            for (int n = 0; n < KN; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[g][n][j] *= s[j];
        }
        if constexpr (LORA)
            add_adapters<KF, KN>(a, t.first, t.rows, 0, [&](int g, int32_t ad, int32_t c) {
                const int32_t fe = feature(g, i);
                const int64_t pair = (int64_t)ad * (a.e.E + a.e.shared) + t.expert;
                if (fe >= features) return bf16x8{};
                return *reinterpret_cast<const bf16x8*>(a.l.b + (pair * a.e.on + up(g, i) * features + fe) * a.l.rank + c * 8);
            }, acc);
        uint16_t* const out = static_cast<uint16_t*>(a.e.out);
        float w[KN];
        int32_t slot[KN];
        if constexpr (GATED) row_weights<KN>(a, [&](int n) { return t.first + min(n * 16 + i, t.rows - 1); }, w, slot);
#pragma unroll
        for (int n = 0; n < KN; ++n) {
            const int32_t r = n * 16 + i;
            f32x4 upper;
            if constexpr (GATED && KF == 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j) upper[j] = __shfl_xor(acc[0][n][j], 32, kWave);
                if (lane >= 32) continue;
            }
            if (r >= t.rows) continue;
            if constexpr (GATED) {
                const int32_t fe = feature(0, q * 4);
                if (fe >= features) continue;
                if constexpr (KF == 2) upper = acc[KF - 1][n];
                float y[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = w[n] * (acc[0][n][j] * fast_sigmoid(acc[0][n][j]) * upper[j]);
                *reinterpret_cast<v2u*>(out + (t.first + r) * features + fe) = v2u{pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
            } else {
#pragma unroll
                for (int g = 0; g < KF; ++g) {
                    const int32_t fe = feature(g, q * 4);
                    if (fe < features)
                        *reinterpret_cast<v2u*>(out + (t.first + r) * features + fe) =
                            v2u{pack_bf16x2(acc[g][n][0], acc[g][n][1]), pack_bf16x2(acc[g][n][2], acc[g][n][3])};
                }
            }
        }
    });
}

// BYTES: steps that LDS holds where the scales travel as bytes.
template <int NT, int FW, int WAVES, int L, int BUFS, int BYTES, bool GATED, bool LORA>
hipError_t block(const BlockArgs& a, hipStream_t stream) {
    constexpr int kF = FW * WAVES;
    const int32_t ftiles = (a.e.on + kF - 1) / kF;
    const int64_t tiles = max_row_tiles(a.e, NT) * ftiles, blocks = (tiles + 7) / 8 * 8;
    if (tiles == 0) return hipSuccess;
    if (const hipError_t e = check_grid(blocks, WAVES * kWave)) return e;
    if (a.e.in % 64 == 0)
        hipLaunchKernelGGL((k_nvfp4_block<NT, FW, WAVES, L, BUFS, true, GATED, LORA>), dim3((unsigned)blocks),
                           dim3(WAVES * kWave), 0, stream, a, ftiles);
    else
        hipLaunchKernelGGL((k_nvfp4_block<NT, FW, WAVES, L, BYTES, false, GATED, LORA>), dim3((unsigned)blocks),
                           dim3(WAVES * kWave), 0, stream, a, ftiles);
    return hipGetLastError();
}

// By the rows a group has on average, as the product without an end of its own.
template <bool GATED, bool LORA>
hipError_t by_size(const BlockArgs& a, hipStream_t stream) {
    const int64_t groups = a.e.slots < a.e.E + a.e.shared ? a.e.slots : a.e.E + a.e.shared;
    if (groups == 0) return hipSuccess;
    const int64_t mean = a.e.slots / groups;
    if (mean <= 13) return block<16, 16, 4, 256, 3, 3, GATED, LORA>(a, stream);
    if (mean <= 26) return block<32, 16, 4, 256, 2, 2, GATED, LORA>(a, stream);
    if (mean <= 56) return block<64, 32, 8, 128, 2, 2, GATED, LORA>(a, stream);
    return block<128, 32, 8, 128, 3, 2, GATED, LORA>(a, stream);
}

}  // namespace

hipError_t launch_gated_nvfp4(const BlockArgs& a, hipStream_t stream) {
    return a.l.rank > 0 ? by_size<true, true>(a, stream) : by_size<true, false>(a, stream);
}

hipError_t launch_gemm_nvfp4_lora(const BlockArgs& a, hipStream_t stream) { return by_size<false, true>(a, stream); }

}  // namespace epx
