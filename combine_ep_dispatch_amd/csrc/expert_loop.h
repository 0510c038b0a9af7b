// Tiles of 256 features by up to 256 rows whose product ends in an epilogue of
// its own: the gated block and the products with adapters.
#pragma once

#include <type_traits>
#include <utility>

#include "expert_tile.h"
#include "lora_device.h"

namespace epx {

constexpr int kLoopWaves = 4;
constexpr int kLoopThreads = kLoopWaves * kWave;
constexpr int kTileF = 256, kTileN = 256;  // features (of both projections, where gated) and rows of a tile
constexpr int kLoopLds = 160 * 1024;       // all of it: one workgroup a CU

// A load of 16 bytes a lane to LDS (16 l for lane l), as load_to_lds, in two parts
// that other instructions go between: where to, in m0, and the load, at least one
// wait state later.  Its descriptor is one that no vector instruction writes from
// settled() on: it needs no wait states of its own.  Nothing the compiler puts
// between the two uses m0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int OFF>
__device__ __forceinline__ void aim16(uint32_t to) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_add_u32 m0, %0, %1" ::"s"(to), "n"(OFF) : "memory", "m0", "scc");
#endif
}
__device__ __forceinline__ void load16(i32x4 rs, int32_t voff) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("buffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(voff), "s"(rs) : "memory");
#endif
}
// Both at once.
template <int OFF>
__device__ __forceinline__ void aim_and_load16(uint32_t to, i32x4 rs, int32_t voff) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds" ::"s"(to), "n"(OFF), "v"(voff),
                 "s"(rs)
                 : "memory", "m0", "scc");
#endif
}
#pragma clang diagnostic pop

__device__ __forceinline__ i32x4 descriptor(const void* base, int32_t bytes) {
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    return {(int32_t)uniform((uint32_t)p), (int32_t)uniform((uint32_t)(p >> 32) & 0xFFFFu), uniform(bytes), kBufferWord3};
}

// rs, whose words were written 5 wait states ago at least.
__device__ __forceinline__ i32x4 settled(i32x4 rs) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("s_nop 4" : "+s"(rs));
#endif
    return rs;
}

// bytes further: the base by scalar additions.
__device__ __forceinline__ void move_on(i32x4& rs, int64_t bytes) {
    const uint64_t p = ((uint64_t)(uint32_t)rs[1] << 32 | (uint32_t)rs[0]) + bytes;
    rs[0] = (int32_t)(uint32_t)p;
    rs[1] = (int32_t)(uint32_t)(p >> 32);
}

// The operands as expert_tile.h lays them out, loaded step after step: a lane's
// offsets stay, the descriptors move on.  (A vector instruction between two matrix
// instructions costs about 9 cycles: with an addition for each load the loop took
// 272 000 instead of 256 000.)
template <int BM>
struct LoopRows : RowsOperand<BM, kLoopWaves> {
    using Base = RowsOperand<BM, kLoopWaves>;
    i32x4 rs;
    int32_t left;  // values of L from the next step on

    __device__ __forceinline__ void init(const uint16_t* p, int32_t rows, int32_t pitch, int32_t l) {
        Base::init(p, rows, pitch, l);
        rs = settled(descriptor(p, this->records));
        left = l;
        if (left < kStepL) trim();
    }
    // The last step, in part: chunks past its end are outside.  Behind it everything is.
    __device__ __forceinline__ void trim() {
        if (left <= 0) rs[2] = 0;
#pragma unroll
        for (int j = 0; j < Base::kLoads; ++j)
            if (this->chunk[j % 2] * 8 >= left) this->voff[j] = kOutside;
    }
    __device__ __forceinline__ void advance() {
        move_on(rs, kStepL * 2);
        rs[2] -= kStepL * 2;
        left -= kStepL;
        if (left < kStepL) trim();
    }
    __device__ __forceinline__ i32x4 source(int) const { return rs; }
    // Where a lane's values of half a step are in the operand's LDS tile, from row m0
    // on, and the fragment 16 f rows further.
    static __device__ __forceinline__ int32_t lane_at(int m0, int half) {
        const int lane = threadIdx.x & (kWave - 1), i = lane % 16, q = lane / 16;
        return (m0 + i) * kStepL + ((half * 4 + q) ^ (i / 2)) * 8;
    }
    static __device__ __forceinline__ bf16x8 fragment_at(const uint16_t* p, int f, int, int) {
        return *reinterpret_cast<const bf16x8*>(p + f * 16 * kStepL);
    }
};

// The gated block's feature operand: 16 rows of the gate and 16 of the up
// projection in turn, so that a lane of a wave has both of a column of act.
struct GatedOperand : LoopRows<kTileF> {
    i32x4 up;

    // p: the expert's weights; a0: first column of act; inter: their number
    __device__ __forceinline__ void init(const uint16_t* p, int32_t a0, int32_t inter, int32_t l) {
        const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
        const uint16_t* const gate = p + (int64_t)a0 * l;
        Base::init(gate, min(kTileF / 2, inter - a0), l, l);
        rs = settled(descriptor(gate, records));
        up = settled(descriptor(gate + (int64_t)inter * l, records));
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int at = w * kLoads + j;  // 8 rows of LDS: half of a gate's or an up's 16
            voff[j] = (at / 4 * 16 + at % 2 * 8 + lane / 8) * l * 2 + chunk[j % 2] * 16;
        }
        left = l;
        if (left < kStepL) trim();
    }
    __device__ __forceinline__ void advance() {
        LoopRows<kTileF>::advance();
        move_on(up, kStepL * 2);
        up[2] = rs[2];
    }
    __device__ __forceinline__ i32x4 source(int j) const { return j / 2 % 2 ? up : rs; }
};

struct LoopCols : ColsOperand<kTileF, kLoopWaves> {
    using Base = ColsOperand<kTileF, kLoopWaves>;
    i32x4 rs;
    int32_t l0;  // the next step's first row

    __device__ __forceinline__ void init(const uint16_t* p, int32_t cols, int32_t pitch, int32_t l, int32_t m0) {
        Base::init(p, cols, pitch, l, m0);
        rs = settled(descriptor(p, records(0)));
        l0 = 0;
    }
    __device__ __forceinline__ void advance() {
        move_on(rs, (int64_t)kStepL * ld * 2);
        l0 += kStepL;
        const int32_t rows = min(len - l0, kStepL);
        rs[2] = rows > 0 ? rows * ld * 2 - cut : 0;
    }
    __device__ __forceinline__ i32x4 source(int) const { return rs; }
    static __device__ __forceinline__ int32_t lane_at(int, int) { return 0; }
    static __device__ __forceinline__ bf16x8 fragment_at(const uint16_t* p, int f, int m0, int half) {
        return fragment(p, m0 + f * 16, half);
    }
};

// A wave's loads of an operand's next step, to its part of LDS.
template <typename Op, int... J>
__device__ __forceinline__ void load_step(Op& op, uint32_t to, std::integer_sequence<int, J...>) {
    (aim_and_load16<J * 1024>(to, op.source(J), op.voff[J]), ...);
    op.advance();
}

// f(integral_constant<int, 0>), f(integral_constant<int, 1>), ...
template <typename F, int... K>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, K...>) {
    (f(std::integral_constant<int, K>{}), ...);
}

// A wave's KF x KN fragments of 16 features by 16 rows, from feature wf and row
// wn of the tile on, summed over L and added to acc.  LDS holds NT rows a step.
// meanwhile() runs behind the first loads, which are under way meanwhile.
template <typename FOp, typename NOp, int NT, int KF, int KN, typename Meanwhile>
__device__ __forceinline__ void tile_loop(FOp fo, NOp no, uint16_t* lds, int wf, int wn, int32_t len,
                                          f32x4 (&acc)[KF][KN], Meanwhile meanwhile) {
    // LDS is a ring of whole steps of both operands; with 256 rows, of which two
    // steps and a half fit, of units of one operand's step, F's and N's in turn.
    constexpr bool kUnits = NT == kTileF;
    constexpr int kUnit = kTileF * kStepL, kBuffer = kUnits ? kUnit : (kTileF + NT) * kStepL;
    constexpr int kRing = kLoopLds / 2 / kBuffer;
    constexpr int kAheadF = kUnits ? 2 : kRing - 1, kAheadN = kUnits ? 1 : kRing - 1;
    constexpr int kFL = FOp::kLoads, kNL = NOp::kLoads;
    static_assert(kUnits ? kRing == 5 : kRing >= 3, "");
    const int w = uniform((int32_t)(threadIdx.x / kWave));
    const uint32_t base = uniform((uint32_t)(uintptr_t)(EPX_LDS const void*)lds);
    auto ring = [](int32_t v) { return v >= kRing ? v - kRing : v; };
    // element of LDS where a step's operands begin, by the step's slot
    auto f_at = [&](int32_t slot) { return slot * kBuffer; };
    auto n_at = [&](int32_t slot) { return kUnits ? ring(slot + 1) * kBuffer : slot * kBuffer + kUnit; };
    auto f_to = [&](int32_t slot) { return base + f_at(slot) * 2 + w * kFL * 1024; };
    auto n_to = [&](int32_t slot) { return base + n_at(slot) * 2 + w * kNL * 1024; };
    auto load_f = [&](int32_t slot) { load_step(fo, f_to(slot), std::make_integer_sequence<int, kFL>{}); };
    auto load_n = [&](int32_t slot) { load_step(no, n_to(slot), std::make_integer_sequence<int, kNL>{}); };
    constexpr int kStride = kUnits ? 2 : 1;  // slots of a step
#pragma unroll
    for (int s = 0; s < kAheadF; ++s) {
        if (s < kAheadN) load_n(s * kStride);
        load_f(s * kStride);
    }
    load_n(kAheadN * kStride);
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
    const uint16_t* const lane_f[2] = {lds + FOp::lane_at(wf, 0), lds + FOp::lane_at(wf, 1)};
    const uint16_t* const lane_n[2] = {lds + NOp::lane_at(wn, 0), lds + NOp::lane_at(wn, 1)};
    auto read = [&](int half, const uint16_t* f, const uint16_t* n, int r) {
        if (r < KN)
            fb[half][r] = NOp::fragment_at(n, r, wn, half);
        else
            fa[half][r - KN] = FOp::fragment_at(f, r - KN, wf, half);
    };
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(0, lane_f[0] + f_at(0), lane_n[0] + n_at(0), r);
    // Each half of a step multiplies the fragments that the half before read, and
    // reads the next one's: first the second half's, then, behind the barrier, the
    // next step's first.  By that barrier every wave has read all of this step,
    // whose buffers are filled from then on.  Loads and reads go one by one between
    // the matrix instructions, each of which leaves time to issue three others.
    constexpr int kProducts = KF * KN;
    constexpr int kReadGap = (kProducts - 1) / kReads < 3 ? (kProducts - 1) / kReads : 3;
    static_assert(kReadGap >= 1, "");
    const int32_t steps = (len + kStepL - 1) / kStepL;
    int32_t slot = 0;
    auto half_step = [&](auto half_, int32_t from, auto& op, uint32_t to, auto loads) {
        constexpr int half = decltype(half_)::value, kLoads = decltype(loads)::value, kGap = kProducts / kLoads;
        static_assert(kGap >= 1, "");
        const uint16_t *const f_from = lane_f[half ^ 1] + f_at(from), *const n_from = lane_n[half ^ 1] + n_at(from);
        each([&](auto k_) {
            constexpr int k = decltype(k_)::value, f = k / KN, n = k % KN, j = k / kGap;
            __builtin_amdgcn_sched_barrier(0);
            acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[half][f], fb[half][n], acc[f][n], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (k % kReadGap == 0 && k / kReadGap < kReads) read(half ^ 1, f_from, n_from, k / kReadGap);
            if constexpr (j < kLoads && kGap == 1) {
                aim_and_load16<j * 1024>(to, op.source(j), op.voff[j]);
            } else if constexpr (j < kLoads && k % kGap == 0) {
                aim16<j * 1024>(to);
            } else if constexpr (j < kLoads && k % kGap == 1) {
                load16(op.source(j), op.voff[j]);
            }
        }, std::make_integer_sequence<int, kProducts>{});
        __builtin_amdgcn_sched_barrier(0);
        op.advance();
    };
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, 1>;
    for (int32_t s = 0; s < steps; ++s) {
        const int32_t after = ring(slot + kStride);
        half_step(First{}, slot, fo, f_to(ring(slot + (kUnits ? 4 : kRing - 1))),
                  std::integral_constant<int, kFL>{});
        // the next step has landed, in every wave
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kUnits ? kFL : (kRing - 2) * (kFL + kNL)) : "memory");
        lds_barrier();
        // of the freed units, N's of the step after the next takes this step's F's
        half_step(Second{}, after, no, n_to(kUnits ? ring(slot + 4) : slot),
                  std::integral_constant<int, kNL>{});
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
