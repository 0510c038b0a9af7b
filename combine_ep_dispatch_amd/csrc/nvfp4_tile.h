// The tiles of the experts' product over 4-bit weights, whatever ends them.
#pragma once

#include "expert_device.h"

namespace epx {

// E4M3 byte `at` (0..3) of a word.
__device__ __forceinline__ float e4m3_of(uint32_t word, int at) {
    switch (at) {
        case 0: return __builtin_amdgcn_cvt_f32_fp8((int)word, 0);
        case 1: return __builtin_amdgcn_cvt_f32_fp8((int)word, 1);
        case 2: return __builtin_amdgcn_cvt_f32_fp8((int)word, 2);
        default: return __builtin_amdgcn_cvt_f32_fp8((int)word, 3);
    }
}

// e2m1(code) * scale of 8 codes.
__device__ __forceinline__ bf16x8 weights8(uint32_t codes, float scale) {
    v4u o;
    f32x2_t p;
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
    o.x = pack_bf16x2(p.x * scale, p.y * scale);
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
    o.y = pack_bf16x2(p.x * scale, p.y * scale);
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
    o.z = pack_bf16x2(p.x * scale, p.y * scale);
    p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
    o.w = pack_bf16x2(p.x * scale, p.y * scale);
    return __builtin_bit_cast(bf16x8, o);
}

// LDS rows are swizzled, chunk c of 16 bytes of row r at c ^ swizzle(r).  A
// 16-byte LDS read serves 16 lanes at a time, and those are rows 0-3 and 12-15
// of one quarter q with rows 4-11 of the next: the swizzles keep these apart
// for q even and odd (rows with bits 2 and 3 alike go to other chunks than the
// rest, whatever q adds).
__device__ __forceinline__ int swizzle_row(int r) { return (r % 16) ^ (r & 4) << 1; }            // 16 chunks or more
__device__ __forceinline__ int swizzle_codes8(int r) { return r / 2 % 8; }                       // 8 chunks
__device__ __forceinline__ int swizzle_codes4(int r) { return (r / 4 % 2) | ((r / 4 ^ r / 8) & 1) << 1; }  // 4 chunks

// NT rows and WAVES * FW features a tile, L values a step, BUFS steps in LDS.
// WORDS: every feature's scales start at a word (in_dim is a multiple of 64)
// and travel as words; otherwise each scale is loaded as a byte, into a word.
// GATED: the features of a wave are FW / 2 rows of the gate projection, then as
// many of the up projection (a.on counts both).
template <int NT, int FW, int WAVES, int L, int BUFS, bool WORDS, bool GATED>
struct Nvfp4Tile {
    static_assert(FW * L == 4096, "a wave's scales are 64 words, its codes two loads");
    static constexpr int kThreads = WAVES * kWave;
    static constexpr int kFeatures = WAVES * FW;
    static constexpr int kLane = L / 4;                        // values of a lane and step
    static constexpr int kCodeRow = L / 2, kCodeChunks = kCodeRow / 16;
    static constexpr int kScaleBytes = WORDS ? 256 : 1024;     // of a wave
    static constexpr int kScaleLoads = kScaleBytes / 256;
    static constexpr int kRowBytes = L * 2, kRowChunks = kRowBytes / 16;
    static constexpr int kRowLoads = NT * kRowBytes / 1024 / WAVES;
    static constexpr int kLoads = 2 + kScaleLoads + kRowLoads;  // of a wave and step
    static constexpr int kCodes = kFeatures * kCodeRow, kScales = WAVES * kScaleBytes;
    static constexpr int kBuffer = kCodes + kScales + NT * kRowBytes;
    // Many rows: the next step's loads go between this step's products, and the
    // next group's operands are made while the matrix pipe works on this one's
    // (213 -> 197 us at 122 rows a group; few rows gain nothing).
    static constexpr bool kSpread = NT >= 64;
    static_assert(kRowLoads >= 1 && (BUFS - 2) * kLoads < 64, "");

    // Computes the workgroup's tile and hands its results to epilogue(t, f0, row0, acc):
    // row tile, first feature of the wave (gated: column of act) and its row of the
    // weights, acc[g][n][j]: feature 16 g + 4 q + j of the wave, row 16 n + i.
    template <typename Epilogue>
    static __device__ __forceinline__ void run(const ExpertArgs& a, int32_t ftiles, uint8_t* lds, int32_t* scan,
                                               Epilogue epilogue) {
        const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
        const int i = lane % 16, q = lane / 16;
        int32_t f;
        const RowTile t = find_row_tile<kThreads, NT>(
            a, scan, [&](int32_t rt, int32_t& ft) { return xcd_tile(rt, ftiles, ft); }, f);
        if (t.expert < 0) return;
        constexpr int kPart = GATED ? FW / 2 : FW;  // features of a wave that follow each other
        const int32_t in = a.in, features = GATED ? a.on / 2 : a.on, f0 = uniform(f * (kFeatures / FW * kPart) + w * kPart);
        const int64_t row0 = (int64_t)t.expert * a.on + f0;
        const int32_t frows = uniform(max(min(kPart, features - f0), 0));  // 0: this wave only helps with the rows
        const int32_t cpitch = in / 2, spitch = in / 16;
        // gated: the scales of the wave's rows of both projections lie apart; of no rows, nothing may be read
        const int32_t srows = uniform(GATED && frows > 0 ? features + frows : frows);
        const uint8_t* const codes = a.codes + row0 * cpitch;
        const uint8_t* const scales = a.scales + row0 * spitch;
        const uint16_t* const x = a.x + t.first * in;

        // A wave's loads of a step: where the lane's bytes are in the operands'
        // step 0, and the first value they hold.
        int32_t off[kLoads], first[kLoads];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = j * (64 / kCodeChunks) + lane / kCodeChunks;
            const int c = (lane % kCodeChunks) ^ (L == 256 ? swizzle_codes8(r) : swizzle_codes4(r));
            off[j] = r % kPart * cpitch + c * 16;  // gated: load 0 is the gate's, load 1 the up projection's
            first[j] = c * 32;
        }
#pragma unroll
        for (int j = 0; j < kScaleLoads; ++j) {
            constexpr int kPer = WORDS ? L / 64 : L / 16;  // words or scales of a feature
            const int at = j * kWave + lane, r = at / kPer, c = at % kPer;
            off[2 + j] = (r / kPart * features + r % kPart) * spitch + c * (WORDS ? 4 : 1);
            first[2 + j] = c * (L / kPer);
        }
#pragma unroll
        for (int j = 0; j < kRowLoads; ++j) {
            const int r = (w * kRowLoads + j) * (64 / kRowChunks) + lane / kRowChunks;
            const int c = (lane % kRowChunks) ^ swizzle_row(r);
            off[2 + kScaleLoads + j] = r * in * 2 + c * 16;
            first[2 + kScaleLoads + j] = c * 8;
        }
        // Step s of this wave's features and of its share of the rows; lanes past
        // the end of the summed dimension read nothing.  (The last 16 codes of a
        // feature may end in the middle of a lane's 16 bytes: what follows them
        // meets zeros of the rows, or the end of the buffer.)
        auto load = [&](int32_t s, int j) {
            uint8_t* const to = lds + s % BUFS * kBuffer;
            const int32_t l0 = s * L;
            const bool on = l0 + L <= in || l0 + first[j] < in;
            if (j < 2)
                load_to_lds<16>(GATED && j == 1 ? codes + (int64_t)features * cpitch : codes, frows * cpitch,
                                to + w * (FW * kCodeRow) + j * 1024, on ? off[j] + l0 / 2 : kOutside);
            else if (j < 2 + kScaleLoads)
                load_to_lds<WORDS ? 4 : 1>(scales, srows * spitch,
                                           to + kCodes + w * kScaleBytes + (j - 2) * 256,
                                           on ? off[j] + l0 / 16 : kOutside);
            else
                load_to_lds<16>(x, t.rows * in * 2, to + kCodes + kScales + (w * kRowLoads + j - 2 - kScaleLoads) * 1024,
                                on ? off[j] + l0 * 2 : kOutside);
        };
        f32x4 acc[FW / 16][NT / 16] = {};
        const int32_t steps = (in + L - 1) / L;
        for (int s = 0; s < BUFS - 1; ++s)
#pragma unroll
            for (int j = 0; j < kLoads; ++j) load(s, j);
        for (int32_t s = 0; s < steps; ++s) {
            // This step's loads have landed when only the later steps' are
            // outstanding: loads return in order, and past the end they still
            // count, and write zeros.  Behind the barrier every wave's have, and
            // every wave is done with the last step's buffer, which is filled next.
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((BUFS - 2) * kLoads) : "memory");
            lds_barrier();
            if (!kSpread) {
#pragma unroll
                for (int j = 0; j < kLoads; ++j) load(s + BUFS - 1, j);
            }
            const uint8_t* const from = lds + s % BUFS * kBuffer;
            v4u cw[FW / 16][kLane / 32];
            float sc[FW / 16][kLane / 16];
#pragma unroll
            for (int g = 0; g < FW / 16; ++g) {
                const int r = g * 16 + i;
                const uint8_t* const p = from + (w * FW + r) * kCodeRow;
                const uint8_t* const ps = from + kCodes + w * kScaleBytes;
#pragma unroll
                for (int h = 0; h < kLane / 32; ++h) {
                    const int c = h * 4 + q;  // the chunk of 32 codes; its blocks are 2 c and 2 c + 1
                    cw[g][h] = *reinterpret_cast<const v4u*>(p + (c ^ (L == 256 ? swizzle_codes8(r) : swizzle_codes4(r))) * 16);
                    const int b = r * (L / 16) + c * 2;
                    if constexpr (WORDS) {
                        const uint32_t two = *reinterpret_cast<const uint16_t*>(ps + b);
                        sc[g][2 * h] = e4m3_of(two, 0);
                        sc[g][2 * h + 1] = e4m3_of(two, 1);
                    } else {
                        const v2u two = *reinterpret_cast<const v2u*>(ps + b * 4);
                        sc[g][2 * h] = e4m3_of(two.x, 0);
                        sc[g][2 * h + 1] = e4m3_of(two.y, 0);
                    }
                }
            }
            const uint8_t* const rows = from + kCodes + kScales + i * kRowBytes;
            constexpr int kGroups = kLane / 8;  // of 8 values a lane: one matrix instruction each way
            bf16x8 wv[2][FW / 16], xv[2][NT / 16];
            auto operands = [&](int j) {
#pragma unroll
                for (int g = 0; g < FW / 16; ++g) wv[j % 2][g] = weights8(cw[g][j / 4][j % 4], sc[g][j / 2]);
#pragma unroll
                for (int n = 0; n < NT / 16; ++n)
                    xv[j % 2][n] = *reinterpret_cast<const bf16x8*>(rows + n * 16 * kRowBytes +
                                                                    (((j / 4 * 4 + q) * 4 + j % 4) ^ swizzle_row(i)) * 16);
            };
            operands(0);
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                if constexpr (kSpread) {
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int k = j * kLoads / kGroups; k < (j + 1) * kLoads / kGroups; ++k) load(s + BUFS - 1, k);
                }
                if (j + 1 < kGroups) operands(j + 1);
#pragma unroll
                for (int n = 0; n < NT / 16; ++n)
#pragma unroll
                    for (int g = 0; g < FW / 16; ++g)
                        acc[g][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j % 2][g], xv[j % 2][n], acc[g][n], 0, 0, 0);
                if constexpr (kSpread) {
                    __builtin_amdgcn_sched_group_barrier(0x100, NT / 16, 0);  // LDS reads, then
#pragma unroll
                    for (int n = 0; n < NT / 16 * (FW / 16); ++n) {
                        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);  // a matrix instruction and
                        __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);  // its share of the conversions, in turn
                    }
                }
            }
        }
        // No load may land in LDS that belongs to another workgroup by then.
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        epilogue(t, f0, row0, acc);
    }
};

}  // namespace epx
