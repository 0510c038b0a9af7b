// Tiles of 256 features by up to 256 rows whose product ends in an epilogue of
// its own: the gated block and the products with adapters.  A workgroup of 4 waves
// a CU takes tile after tile; the loads run on from one to the next.
//
// Full tiles are as large as registers and LDS hold: 64 KiB come through L2 for
// 2 x 256 x 256 x 64 operations a step and CU.  A wave's 128 x 128 results fill its 256
// accumulation registers.  LDS reads, loads and what advances them go one by one
// between the matrix instructions.  32 experts of 4096 x 7168, 32 768 rows, us: loads
// and reads ahead of each step's products 1745, between them 1650, a workgroup a CU
// whose loads run on into the next tile 1496.  A step then takes 2290 cycles, 2048 of
// them matrix instructions.
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
constexpr int kCus = 256;

struct LoopTile {
    int32_t expert;  // -1: no such tile
    int32_t rows;    // of the tile, 1..kTileN
    int32_t ft;      // its feature tile
    int64_t first;   // its first receive row
};

// Tiles come in three kinds, by their rows; each kind fills LDS in its own way.
constexpr int kKinds = 3;
constexpr int kKindRows[kKinds] = {kTileN, 128, 32};  // at most

// The tiles that a workgroup takes in turn, kind after kind.  A group is cut into
// as few tiles as can be, of one height: 896 rows are 4 of 224.  From five tiles on
// they are full ones and what is left over, if that is at most half of one, which
// then reads the weights once more.  32 experts of 4096 x 7168, us for one height and
// for full tiles and the rest: 300 rows 605 and 750, 384 632 and 772, 520 918 and 1018,
// 600 1053 and 1060, 776 1335 and 1381, 896 1328 and 1446, 1040 1645 and 1645, 996
// to 1060 rows (a training step's) 1605 and 1510, where one height is 9 tiles a CU and
// the other 8 and a rest.  Every wave keeps, for the run of groups that each lane looks
// after, how many row tiles of each kind come before and up to it; no memory but the
// layout's is used.  Of each kind each XCD takes an eighth, in blocks of 4 row tiles by
// all feature tiles, whose operands the workgroups that run together share in its L2,
// and hands them out in turn.
struct LoopTiles {
    int32_t before[kKinds], upto[kKinds];  // of this lane's groups
    int32_t total[kKinds], ftiles, per;
    int32_t rows_, first_;  // of this lane's only group, where it has one

    // Rows of a group that become a tile of their own, behind its full ones.
    static __device__ __forceinline__ int32_t left_over(int32_t rows) {
        const int32_t rest = rows % kTileN;
        return rows <= kKindRows[1] ? rows : rows > 4 * kTileN && rest <= kKindRows[1] ? rest : 0;
    }
    static __device__ __forceinline__ int32_t tiles_of(int32_t rows, int kind) {
        const int32_t rest = left_over(rows);
        if (kind == 0) return (rows - rest + kTileN - 1) / kTileN;
        return kind == 1 ? rest > kKindRows[2] : rest > 0 && rest <= kKindRows[2];
    }
    __device__ __forceinline__ void init(const ExpertArgs& a, int32_t f) {
        const int lane = threadIdx.x & (kWave - 1);
        ftiles = f;
        per = (a.NG + kWave - 1) / kWave;
        int32_t mine[kKinds] = {};
        rows_ = first_ = 0;
        for (int g = lane * per; g < min((lane + 1) * per, a.NG); ++g) {
            const GroupRows r = group_rows(a, g);
            rows_ = r.rows;
            first_ = (int32_t)r.first;
#pragma unroll
            for (int k = 0; k < kKinds; ++k) mine[k] += tiles_of(r.rows, k);
        }
#pragma unroll
        for (int k = 0; k < kKinds; ++k) {
            upto[k] = wave_inclusive_sum(mine[k]);
            before[k] = upto[k] - mine[k];
            total[k] = __builtin_amdgcn_readlane(upto[k], kWave - 1);
        }
    }
    // How many tiles of a kind this workgroup's XCD takes, and the first of them.
    __device__ __forceinline__ int32_t share(int kind, int32_t& from) const {
        const int32_t tiles = total[kind] * ftiles, each = (tiles + 7) / 8;
        from = (int32_t)(blockIdx.x % 8) * each;
        return max(min(each, tiles - from), 0);
    }
    // The n-th tile of the kind of this workgroup: its turns go on from one kind to
    // the next, so that all workgroups get as many tiles, give or take one.
    template <int KIND>
    __device__ __forceinline__ LoopTile get(const ExpertArgs& a, int32_t n) const {
        const int32_t turns = uniform((int32_t)(gridDim.x / 8));
        int32_t from = 0, before_us = 0;
#pragma unroll
        for (int k = 0; k < KIND; ++k) before_us += share(k, from);
        const int32_t mine = share(KIND, from);
        int32_t at = uniform((int32_t)(blockIdx.x / 8)) - before_us % turns;
        at = uniform((at < 0 ? at + turns : at) + n * turns);
        if (at >= mine) return {-1, 1, 0, 0};
        const int32_t all = from + at, block = all / (4 * ftiles), r0 = block * 4, height = min(4, total[KIND] - r0);
        const int32_t in = all - block * 4 * ftiles, want = r0 + in % height, ft = in / height;
        const bool owner = want >= before[KIND] && want < upto[KIND];
        int32_t expert = 0, rows = 0, first = 0;
        if (owner) {
            const int lane = threadIdx.x & (kWave - 1);
            int32_t b = before[KIND];
            for (int g = lane * per; g < min((lane + 1) * per, a.NG); ++g) {
                const GroupRows r = per == 1 ? GroupRows{first_, rows_} : group_rows(a, g);
                const int32_t c = tiles_of(r.rows, KIND);
                if (want < b + c) {
                    const int32_t rest = left_over(r.rows), cut = r.rows - rest;  // cut: in tiles of one height
                    const int32_t height = KIND == 0 ? ((cut + c - 1) / c + 15) / 16 * 16 : rest;
                    const int32_t skip = KIND == 0 ? (want - b) * height : cut;
                    expert = group_expert(a, g);
                    rows = KIND == 0 ? min(height, cut - skip) : rest;
                    first = (int32_t)(r.first + skip);
                    break;
                }
                b += c;
            }
        }
        const int l = __builtin_ctzll(__builtin_amdgcn_ballot_w64(owner) | 1ull << 63);
        return {__builtin_amdgcn_readlane(expert, l), __builtin_amdgcn_readlane(rows, l), uniform(ft),
                __builtin_amdgcn_readlane(first, l)};
    }
};

// Workgroups of a launch, and whether the tiles can be counted in 32 bits.
inline hipError_t loop_blocks(const ExpertArgs& a, int32_t ftiles, unsigned& blocks) {
    const int64_t tiles = max_row_tiles(a, kTileN) * ftiles;
    blocks = (unsigned)((tiles < kCus ? tiles : kCus) + 7) / 8 * 8;
    return tiles >= int64_t(1) << 31 ? hipErrorInvalidConfiguration : hipSuccess;
}

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

// rs in scalar registers, written 5 wait states ago at least.
__device__ __forceinline__ i32x4 settled(i32x4 rs) {
#pragma unroll
    for (int k = 0; k < 4; ++k) rs[k] = uniform(rs[k]);
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
// offsets stay, the descriptors move on (advance()).  start() sets an operand to a
// tile's first step; ready(s) comes before the loads of step s wherever that may be
// one that L ends in, or one behind it, which loads zeros.
template <int BM>
struct LoopRows : RowsOperand<BM, kLoopWaves> {
    using Base = RowsOperand<BM, kLoopWaves>;
    i32x4 rs;

    __device__ __forceinline__ void offsets() { Base::init(nullptr, 0, this->ld, this->len); }
    __device__ __forceinline__ void init(int32_t l) { Base::init(nullptr, 0, l, l); }
    __device__ __forceinline__ void start(const uint16_t* p, int32_t rows) {
        rs = settled(descriptor(p, rows * this->ld * 2));
    }
    __device__ __forceinline__ void trim(int32_t s) {
#pragma unroll
        for (int j = 0; j < Base::kLoads; ++j)
            this->voff[j] = s * kStepL + this->chunk[j % 2] * 8 >= this->len ? kOutside : this->voff[j];
    }
    __device__ __forceinline__ void ready(int32_t s, bool ragged) {
        if (!ragged) return;
        offsets();
        trim(s);
    }
    __device__ __forceinline__ void advance() {
        move_on(rs, kStepL * 2);
        rs[2] -= min(rs[2], kStepL * 2);
    }
    __device__ __forceinline__ void settle() { rs = settled(rs); }
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

    __device__ __forceinline__ void offsets() {
        const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int at = w * kLoads + j;  // 8 rows of LDS: half of a gate's or an up's 16
            voff[j] = (at / 4 * 16 + at % 2 * 8 + lane / 8) * ld * 2 + chunk[j % 2] * 16;
        }
    }
    __device__ __forceinline__ void init(int32_t l) {
        Base::init(nullptr, 0, l, l);
        offsets();
    }
    // gate: the tile's first row of the gate projection; inter rows behind it the up's; cols: rows left of each
    __device__ __forceinline__ void start(const uint16_t* gate, int32_t inter, int32_t cols) {
        const int32_t bytes = min(kTileF / 2, cols) * ld * 2;
        rs = settled(descriptor(gate, bytes));
        up = settled(descriptor(gate + (int64_t)inter * ld, bytes));
    }
    __device__ __forceinline__ void ready(int32_t s, bool ragged) {
        if (!ragged) return;
        offsets();
        trim(s);
    }
    __device__ __forceinline__ void advance() {
        LoopRows<kTileF>::advance();
        move_on(up, kStepL * 2);
        up[2] = rs[2];
    }
    __device__ __forceinline__ void settle() {
        rs = settled(rs);
        up = settled(up);
    }
    __device__ __forceinline__ i32x4 source(int j) const { return j / 2 % 2 ? up : rs; }
};

struct LoopCols : ColsOperand<kTileF, kLoopWaves> {
    using Base = ColsOperand<kTileF, kLoopWaves>;
    i32x4 rs;

    // p: the weights' column f0; cols: columns from it on; pitch, rows: the weights'
    __device__ __forceinline__ void start(const uint16_t* p, int32_t f0, int32_t cols, int32_t pitch, int32_t rows) {
        Base::init(p, cols, pitch, rows, f0);
        rs = settled(descriptor(p, records(0)));
    }
    __device__ __forceinline__ void ready(int32_t s, bool) { rs[2] = records(s * kStepL); }
    __device__ __forceinline__ void advance() { move_on(rs, (int64_t)kStepL * ld * 2); }
    __device__ __forceinline__ void settle() {
        rs = settled(rs);
        len = uniform(len);
        cut = uniform(cut);
    }
    __device__ __forceinline__ i32x4 source(int) const { return rs; }
    static __device__ __forceinline__ int32_t lane_at(int, int) { return 0; }
    static __device__ __forceinline__ bf16x8 fragment_at(const uint16_t* p, int f, int m0, int half) {
        return fragment(p, m0 + f * 16, half);
    }
};

// f(integral_constant<int, 0>), f(integral_constant<int, 1>), ...
template <typename F, int... K>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, K...>) {
    (f(std::integral_constant<int, K>{}), ...);
}

// What a tile's rows ask for: the 4 waves take 128 features by half of the rows
// each, or, of at most 128 rows, 64 by all.
template <int NT>
struct Shape {
    static constexpr int kWavesN = NT > 128 ? 2 : 1;
    static constexpr int kF = kTileF / (kLoopWaves / kWavesN) / 16, kN = NT / kWavesN / 16;
    // first feature and row of this wave
    static __device__ __forceinline__ int wf() { return uniform((int32_t)(threadIdx.x / kWave)) / kWavesN * kF * 16; }
    static __device__ __forceinline__ int wn() { return uniform((int32_t)(threadIdx.x / kWave)) % kWavesN * kN * 16; }
};

// (A shape's code is up to 20 KB, and a kernel's has to stay within the reach of its
// branches, 128 KB: 224 and 160 rows gained 3 % where groups had as many.)
template <int KIND, typename Go>
__device__ __forceinline__ void by_rows(int32_t rows, Go go) {
    if constexpr (KIND == 0) {
        if (rows > 192)
            go(std::integral_constant<int, 256>{});
        else
            go(std::integral_constant<int, 192>{});
    } else {
        go(std::integral_constant<int, kKindRows[KIND]>{});
    }
}

// This workgroup's tiles of a kind.  start_f(fo, tile) and start_n(no, tile) set the operands to a tile; begin(shape, tile, acc) may add to the
// results beforehand; end(shape, tile, acc) takes them: acc[f][n], 16 features by 16
// rows each, from feature Shape::wf() and row Shape::wn() of the tile on.
//
// LDS is a ring: of whole steps, three for tiles of up to 128 rows and four for up
// to 32; of full tiles, whose steps are 64 KiB, of five units of 32 KiB, a step of
// one operand each, F's and N's in turn (step s's are units 2 s and 2 s + 1).  A step
// loads the one kAhead behind it into what the step before it has left.
template <int KIND, typename FOp, typename StartF, typename StartN, typename Begin, typename End>
__device__ __forceinline__ void run_kind(const ExpertArgs& a, const LoopTiles& tiles, int32_t len, uint16_t* lds,
                                         FOp& fo, StartF start_f, StartN start_n, Begin begin, End end) {
    constexpr bool kUnits = KIND == 0;
    constexpr int kRows = kKindRows[KIND];
    using NOp = LoopRows<kRows>;
    constexpr int kUnit = kTileF * kStepL, kSlot = kUnits ? kUnit : (kTileF + kRows) * kStepL;
    constexpr int kRing = kLoopLds / 2 / kSlot, kStride = kUnits ? 2 : 1, kAhead = kUnits ? 2 : kRing - 1;
    constexpr int kFL = FOp::kLoads, kNL = NOp::kLoads;
    static_assert(kUnits ? kRing == 5 : kRing >= 3, "");
    LoopTile t = tiles.get<KIND>(a, 0), next;
    if (t.expert < 0) return;
    const int w = uniform((int32_t)(threadIdx.x / kWave));
    const uint32_t base = uniform((uint32_t)(uintptr_t)(EPX_LDS const void*)lds);
    auto ring = [](int32_t v) { return v >= kRing ? v - kRing : v; };
    // element of LDS where a step's operands begin, by its slot
    auto f_at = [](int32_t slot) { return slot * kSlot; };
    auto n_at = [&](int32_t slot) { return kUnits ? ring(slot + 1) * kSlot : slot * kSlot + kUnit; };
    auto f_to = [&](int32_t slot) { return base + f_at(slot) * 2 + w * kFL * 1024; };
    auto n_to = [&](int32_t slot) { return base + n_at(slot) * 2 + w * kNL * 1024; };
    // With more steps a tile than kAhead the loads reach into the next one, no further.
    const int32_t steps = max((len + kStepL - 1) / kStepL, kAhead + 1);
    const bool ragged = len != steps * kStepL;
    NOp no;
    no.init(len);
    start_f(fo, t);
    start_n(no, t);
    auto load = [&](auto& op, uint32_t to, auto loads) {
        each([&](auto j_) {
            constexpr int j = decltype(j_)::value;
            aim_and_load16<j * 1024>(to, op.source(j), op.voff[j]);
        }, std::make_integer_sequence<int, decltype(loads)::value>{});
        op.advance();
    };
#pragma unroll
    for (int s = 0; s < kAhead; ++s) {
        fo.ready(s, ragged);
        no.ready(s, ragged);
        load(fo, f_to(s * kStride), std::integral_constant<int, kFL>{});
        load(no, n_to(s * kStride), std::integral_constant<int, kNL>{});
    }
    // Step 0 has landed when only what was issued behind it is outstanding: loads
    // return in order, and out of range they still count and write zeros.
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 1) * (kFL + kNL)) : "memory");
    lds_barrier();
    int32_t slot = 0;
    for (int32_t n = 1;; ++n) {
        next = tiles.get<KIND>(a, n);
        by_rows<KIND>(t.rows, [&](auto nt) {
            constexpr int NT = decltype(nt)::value, KF = Shape<NT>::kF, KN = Shape<NT>::kN;
            const int wf = Shape<NT>::wf(), wn = Shape<NT>::wn();
            // The compiler takes what comes out of the previous tile's branches for
            // different from lane to lane.
            slot = uniform(slot);
            fo.settle();
            no.settle();
            f32x4 acc[KF][KN] = {};
            begin(nt, t, acc);
            // 256 results in accumulation registers, the operands in the other 256: left
            // to itself the compiler moves results between the two in every step
#pragma unroll
            for (int f = 0; f < KF; ++f)
#pragma unroll
                for (int n = 0; n < KN; ++n) in_agprs(acc[f][n]);
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
            // The first step's first half; behind the previous tile's last barrier it has landed.
#pragma unroll
            for (int r = 0; r < kReads; ++r) read(0, lane_f[0] + f_at(slot), lane_n[0] + n_at(slot), r);
            // Each half of a step multiplies the fragments that the half before read, and
            // reads the next one's: first the second half's, then, behind the barrier, the
            // next step's first.  By that barrier every wave has read all of this step.
            // Loads and reads go one by one between the matrix instructions, each of which
            // leaves time to issue three others.
            constexpr int kProducts = KF * KN;
            constexpr int kReadGap = (kProducts - 1) / kReads < 3 ? (kProducts - 1) / kReads : 3;
            static_assert(kReadGap >= 1, "");
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
            // The steps whose loads L neither begins nor ends with; the one that loads the
            // last; those that load the next tile's first.
#pragma nounroll
            for (int part = 0; part < 2 + kAhead; ++part) {
                if (part == 2) {
                    start_f(fo, next);
                    start_n(no, next);
                }
                const int32_t ahead = part == 0 ? kAhead : part == 1 ? steps - 1 : part - 2;
                fo.ready(ahead, ragged);
                no.ready(ahead, ragged);
                for (int32_t s = part == 0 ? steps - kAhead - 1 : 1; s > 0; --s) {
                    const int32_t after = ring(slot + kStride), free = ring(slot + (kUnits ? 4 : kAhead));
                    half_step(std::integral_constant<int, 0>{}, slot, fo, f_to(free), std::integral_constant<int, kFL>{});
                    // the next step has landed, in every wave, when only later ones are outstanding
                    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kAhead - 2) * (kFL + kNL) + kFL) : "memory");
                    lds_barrier();
                    half_step(std::integral_constant<int, 1>{}, after, no, n_to(free), std::integral_constant<int, kNL>{});
                    slot = after;
                }
            }
            end(nt, t, acc);
        });
        t = next;
        if (t.expert < 0) break;
    }
    // No load of any wave may land in LDS that belongs to the next kind, or another workgroup,
    // by then: those of the tile that is not there write zeros behind the last step's barrier.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    lds_barrier();
}

// All tiles of this workgroup.
template <typename FOp, typename StartF, typename StartN, typename Begin, typename End>
__device__ __forceinline__ void run_tiles(const ExpertArgs& a, int32_t ftiles, int32_t len, uint16_t* lds, FOp& fo,
                                          StartF start_f, StartN start_n, Begin begin, End end) {
    LoopTiles tiles;
    tiles.init(a, ftiles);
    run_kind<0>(a, tiles, len, lds, fo, start_f, start_n, begin, end);
    run_kind<1>(a, tiles, len, lds, fo, start_f, start_n, begin, end);
    run_kind<2>(a, tiles, len, lds, fo, start_f, start_n, begin, end);
}

}  // namespace epx
