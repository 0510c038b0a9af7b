// Tiles of 256 features by up to 256 rows whose product ends in an epilogue of
// its own: the gated block and the products with adapters.
#pragma once

#include <type_traits>

#include "expert_tile.h"
#include "lora_device.h"

namespace epx {

constexpr int kLoopWaves = 4;
constexpr int kLoopThreads = kLoopWaves * kWave;
constexpr int kTileF = 256, kTileN = 256;  // features (of both projections, where gated) and rows of a tile
constexpr int kLoopLds = 160 * 1024;       // all of it: one workgroup a CU

// The gated block's feature operand: 16 rows of the gate and 16 of the up
// projection in turn, so that a lane of a wave has both of a column of act.
struct GatedOperand : RowsOperand<kTileF, kLoopWaves> {
    const uint16_t* up;

    // p: the expert's weights; a0: first column of act; inter: their number
    __device__ __forceinline__ void init(const uint16_t* p, int32_t a0, int32_t inter, int32_t l) {
        const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
        base = p + (int64_t)a0 * l;
        up = base + (int64_t)inter * l;
        ld = len = l;
        records = uniform(min(kTileF / 2, inter - a0) * l * 2);
        chunk[0] = (lane % 8) ^ (lane / 16);
        chunk[1] = chunk[0] ^ 4;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int at = w * kLoads + j;  // 8 rows of LDS: half of a gate's or an up's 16
            voff[j] = (at / 4 * 16 + at % 2 * 8 + lane / 8) * l * 2 + chunk[j % 2] * 16;
        }
    }
    __device__ __forceinline__ void load(uint16_t* lds, int32_t l0, int j) const {
        const int w = uniform((int32_t)(threadIdx.x / kWave));
        load_to_lds<16>(j / 2 % 2 ? up : base, records, lds + (w * kLoads + j) * 512,
                        l0 + chunk[j % 2] * 8 < len ? voff[j] + l0 * 2 : kOutside);
    }
};

// A wave's KF x KN fragments of 16 features by 16 rows, from feature wf and row
// wn of the tile on, summed over L and added to acc.  LDS holds NT rows a step.
// meanwhile() runs behind the first loads, which are under way meanwhile.
template <typename FOp, typename NOp, int NT, int KF, int KN, typename Meanwhile>
__device__ __forceinline__ void tile_loop(const FOp& fo, const NOp& no, uint16_t* lds, int wf, int wn, int32_t len,
                                          f32x4 (&acc)[KF][KN], Meanwhile meanwhile) {
    // LDS is a ring of whole steps of both operands; with 256 rows, of which two
    // steps and a half fit, of units of one operand's step, F's and N's in turn.
    constexpr bool kUnits = NT == kTileF;
    constexpr int kUnit = kTileF * kStepL, kBuffer = kUnits ? kUnit : (kTileF + NT) * kStepL;
    constexpr int kRing = kLoopLds / 2 / kBuffer;
    constexpr int kAheadF = kUnits ? 2 : kRing - 1, kAheadN = kUnits ? 1 : kRing - 1;
    constexpr int kFL = FOp::kLoads, kNL = NOp::kLoads;
    static_assert(kUnits ? kRing == 5 : kRing >= 3, "");
    auto ring = [](int32_t v) { return v >= kRing ? v - kRing : v; };
    auto f_at = [&](int32_t slot) { return lds + slot * kBuffer; };
    auto n_at = [&](int32_t slot) { return kUnits ? lds + ring(slot + 1) * kBuffer : lds + slot * kBuffer + kUnit; };
    auto load_f = [&](int32_t s, int32_t slot, int j0, int j1) {
#pragma unroll
        for (int j = j0; j < j1; ++j) fo.load(f_at(slot), s * kStepL, j);
    };
    auto load_n = [&](int32_t s, int32_t slot, int j0, int j1) {
#pragma unroll
        for (int j = j0; j < j1; ++j) no.load(n_at(slot), s * kStepL, j);
    };
    constexpr int kStride = kUnits ? 2 : 1;  // slots of a step
#pragma unroll
    for (int s = 0; s < kAheadF; ++s) {
        if (s < kAheadN) load_n(s, s * kStride, 0, kNL);
        load_f(s, s * kStride, 0, kFL);
    }
    load_n(kAheadN, kAheadN * kStride, 0, kNL);
    meanwhile();
    // 256 results in accumulation registers, the operands in the other 256: left
    // to itself the compiler moves results between the two in every step
#pragma unroll
    for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int n = 0; n < KN; ++n) in_agprs(acc[f][n]);
    // Step 0 has landed when only what was issued behind it is outstanding
    // (loads return in order, and past the end they still count and write zeros).
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAheadF - 1) * kFL + kAheadN * kNL) : "memory");
    lds_barrier();
    constexpr int kReads = KF + KN;  // of half a step
    bf16x8 fa[2][KF], fb[2][KN];
    auto read = [&](int half, int32_t slot, int r) {
        if (r < KN)
            fb[half][r] = NOp::fragment(n_at(slot), wn + r * 16, half);
        else
            fa[half][r - KN] = FOp::fragment(f_at(slot), wf + (r - KN) * 16, half);
    };
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(0, 0, r);
    // Each half of a step multiplies the fragments that the half before read, and
    // reads the next one's: first the second half's, then, behind the barrier, the
    // next step's first.  By that barrier every wave has read all of this step,
    // whose buffers are filled from then on.
    constexpr int kSpread = KF - 1;  // the reads end before the last products: they have returned by the barrier
    const int32_t steps = (len + kStepL - 1) / kStepL;
    int32_t slot = 0;
    for (int32_t s = 0; s < steps; ++s) {
        const int32_t ahead = ring(slot + (kUnits ? 4 : kRing - 1)), after = ring(slot + kStride);
#pragma unroll
        for (int f = 0; f < KF; ++f) {
            __builtin_amdgcn_sched_barrier(0);
            load_f(s + kAheadF, ahead, f * kFL / KF, (f + 1) * kFL / KF);
#pragma unroll
            for (int r = min(f, kSpread) * kReads / kSpread; r < min(f + 1, kSpread) * kReads / kSpread; ++r) read(1, slot, r);
#pragma unroll
            for (int n = 0; n < KN; ++n)
                acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[0][f], fb[0][n], acc[f][n], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        // the next step has landed, in every wave
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kUnits ? kFL : (kRing - 2) * (kFL + kNL)) : "memory");
        lds_barrier();
        const int32_t freed = kUnits ? ring(slot + 4) : slot;  // its N unit is this step's F unit
#pragma unroll
        for (int f = 0; f < KF; ++f) {
            __builtin_amdgcn_sched_barrier(0);
            load_n(s + 1 + kAheadN, freed, f * kNL / KF, (f + 1) * kNL / KF);
#pragma unroll
            for (int r = min(f, kSpread) * kReads / kSpread; r < min(f + 1, kSpread) * kReads / kSpread; ++r) read(0, after, r);
#pragma unroll
            for (int n = 0; n < KN; ++n)
                acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[1][f], fb[1][n], acc[f][n], 0, 0, 0);
        }
        slot = after;
    }
    // No load may land in LDS that belongs to another workgroup by then.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Results of one row tile, with the shape that its rows ask for: the 4 waves
// take 128 features by 128 rows each, or, of at most 128 rows, 64 by all.
template <typename Go>
__device__ __forceinline__ void by_rows(int32_t rows, Go go) {
    if (rows > 128)
        go(std::integral_constant<int, 256>{});
    else if (rows > 64)
        go(std::integral_constant<int, 128>{});
    else if (rows > 32)
        go(std::integral_constant<int, 64>{});
    else
        go(std::integral_constant<int, 32>{});
}

template <int NT>
struct Shape {
    static constexpr int kWavesN = NT == kTileN ? 2 : 1;
    static constexpr int kF = kTileF / (kLoopWaves / kWavesN) / 16, kN = NT / kWavesN / 16;
    // first feature and row of this wave
    static __device__ __forceinline__ int wf() { return uniform((int32_t)(threadIdx.x / kWave)) / kWavesN * kF * 16; }
    static __device__ __forceinline__ int wn() { return uniform((int32_t)(threadIdx.x / kWave)) % kWavesN * kN * 16; }
};

}  // namespace epx
