// The experts' products with bf16 weights: every receive row times its
// expert's weights, and both gradients.
//   forward   y[r, n]     = sum_h x[r, h] w[e, n, h]
//   input's   gx[r, h]    = sum_n gy[r, n] w[e, n, h]
//   weights'  gw[e, n, h] = sum_r gy[r, n] x[r, h]
// Each is a product of a feature operand F (the output's contiguous dimension,
// and the rows of the matrix instruction's result, so that a lane stores
// consecutive values) and a row operand N, summed over a dimension L that is
// contiguous in an operand (rows) or its rows (columns).
//
// Tiles of 256 features by 256 or 128 rows, 8 waves of 128 x 64 or 64 x 64
// results in registers; steps of 64 values of L, two and a half or three of
// them in LDS, copied there by the loads themselves, one barrier a step.  Where
// those would be few, the forward product and the input's gradient take tiles of
// 64 by 64 (k_expert_small); the weights' gradient has the 256 by 256 ones alone,
// each of which sums all rows of its expert: 4 experts of 128 x 128 with 4096 rows
// each are 4 workgroups and take 86 us, of 1536 x 2048 (192 workgroups) 114.
//
// What bounds them: with few rows an expert HBM, which reads each weight once
// (16 tokens of 8 of 32 experts, 4096 x 7168: 1.88 GB in 321 us, 5.9 TB/s of
// the 6.0 that reading alone reaches); with many the way from L2 to LDS, 64 KiB
// a step and CU beside 128 matrix instructions a SIMD.  32768 rows, same experts:
// 1827 us, 1053 TFLOP/s (a library product of that size: 1298 us in the same run);
// the matrix pipes are busy for 52 % of the cycles, LDS reads have no bank
// conflicts, 4.9 GB come from beyond L2; 11 % of the tiles' rows are past their
// group's end.  Gradients of 49152 rows, 64 experts of 2048 x 1416: input's 344 us
// (829 TFLOP/s), weights' 359 (794; fp32 447, added to fp32 641, which write 743
// MB and read as much); 1416 fills 92 % of 6 tiles.  Measured instead, for the
// 32768 rows when they took 1784 us: the loads alone 1530, the products alone
// 1230; steps of 32 values, four in LDS, 2190 (64-byte requests); dword touches
// into L2 ahead of the loads 2000; the barrier in the middle of a step 1850; tiles
// in another order of L 1850.
#include <type_traits>

#include "expert_device.h"

namespace epx {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kWideThreads = 512;
constexpr int kStepL = 64;                 // values of L a step: whole 128-byte lines of rows
constexpr int kFeatures = 256;             // features of a wide tile
constexpr int kSmall = 64;                 // features and rows of a small one

// One operand's step of BM x kStepL values, copied to LDS by the loads
// themselves (16 bytes a lane, 1 KiB a wave and load, to consecutive LDS
// addresses; the lanes pick their global addresses so that the LDS tile comes
// out swizzled).  Loads past the operand's end write zeros.
//
// Rows: L contiguous.  LDS row m (128 bytes) holds its 8 chunks of 16 bytes at
// c ^ (m / 2 % 8): the 16 rows of a fragment's quarter fall on all banks.
template <int BM>
struct RowsOperand {
    static constexpr int kLoads = BM / 64;  // of each wave and step
    const uint16_t* base;
    int32_t ld, len, records;
    int32_t voff[kLoads], chunk[2];

    // rows: valid rows from base on; pitch: theirs; l: values of L
    __device__ __forceinline__ void init(const uint16_t* p, int32_t rows, int32_t pitch, int32_t l) {
        const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
        base = p;
        ld = pitch;
        len = l;
        records = uniform(rows * ld * 2);
        chunk[0] = (lane % 8) ^ (lane / 16) ^ (w * kLoads % 2 * 4);
        chunk[1] = chunk[0] ^ 4;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            voff[j] = ((w * kLoads + j) * 8 + lane / 8) * ld * 2 + chunk[j % 2] * 16;
    }
    __device__ __forceinline__ void load(uint16_t* lds, int32_t l0, int j) const {
        const int w = uniform((int32_t)(threadIdx.x / kWave));
        load_to_lds<16>(base, records, lds + (w * kLoads + j) * 512,
                        l0 + chunk[j % 2] * 8 < len ? voff[j] + l0 * 2 : kOutside);
    }
    // Fragment of 16 rows from m0 on, values [32 kk, 32 kk + 32) of the step.
    static __device__ __forceinline__ bf16x8 fragment(const uint16_t* lds, int m0, int kk) {
        const int lane = threadIdx.x & (kWave - 1), i = lane % 16, q = lane / 16;
        return *reinterpret_cast<const bf16x8*>(lds + (m0 + i) * kStepL + ((kk * 4 + q) ^ (i / 2)) * 8);
    }
};

// Columns: L strided.  LDS row l holds its BM values in 32-byte pairs of
// chunks at p ^ swizzle(l), so that the transposing reads of 4 rows by 16
// lanes, and of two such groups, fall on different banks.
template <int BM>
struct ColsOperand {
    static constexpr int kLoads = BM / 64;
    static constexpr int kPerRow = BM / 8;         // lanes of one LDS row
    static constexpr int kRows = kWave / kPerRow;  // LDS rows of one load
    const uint16_t* base;
    int32_t ld, len, cut;
    int32_t voff[kLoads];

    // p: column m0 of the operand; cols: valid columns from p on; pitch: of rows; l: rows
    __device__ __forceinline__ void init(const uint16_t* p, int32_t cols, int32_t pitch, int32_t l, int32_t m0) {
        const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
        base = p;
        ld = pitch;
        len = l;
        cut = m0 * 2;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int r = (w * kLoads + j) * kRows + lane / kPerRow, c = lane % kPerRow;
            const int col = (((c / 2) ^ swizzle(r)) * 2 + c % 2) * 8;
            voff[j] = col < cols ? r * ld * 2 + col * 2 : kOutside;
        }
    }
    static __device__ __forceinline__ int swizzle(int l) { return ((l & 3) | ((l >> 1) & 4)) & (BM / 16 - 1); }
    // Bytes of the rows of a step, from base's column on.
    __device__ __forceinline__ int32_t records(int32_t l0) const {
        const int32_t rows = min(len - l0, kStepL);
        return uniform(rows > 0 ? rows * ld * 2 - cut : 0);
    }
    __device__ __forceinline__ void load(uint16_t* lds, int32_t l0, int j) const {
        const int w = uniform((int32_t)(threadIdx.x / kWave));
        load_to_lds<16>(base + (int64_t)l0 * ld, records(l0), lds + (w * kLoads + j) * 512, voff[j]);
    }
    static __device__ __forceinline__ bf16x8 fragment(const uint16_t* lds, int m0, int kk) {
        const int lane = threadIdx.x & (kWave - 1), i = lane % 16, q = lane / 16;
        const int l = kk * 32 + q * 8 + i / 4;
        [[maybe_unused]] const uint16_t* p = lds + l * BM + ((m0 / 16) ^ swizzle(l)) * 16 + i % 4 * 4;
        s16x4 lo = {}, hi = {};
#ifdef __HIP_DEVICE_COMPILE__
        lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((EPX_LDS s16x4*)p);
        hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((EPX_LDS s16x4*)(p + 4 * BM));
#endif
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
};

enum Product { kForward, kInputGrad, kWeightGrad };

// A workgroup's tile of BF features by NT rows, and its operands.
template <Product P, int BF, int NT>
struct Tile {
    using FOp = typename std::conditional<P == kForward, RowsOperand<BF>, ColsOperand<BF>>::type;
    using NOp = typename std::conditional<P == kWeightGrad, ColsOperand<NT>, RowsOperand<NT>>::type;
    FOp fo;
    NOp no;
    int32_t expert, f0, rows, len;  // len: of L
    int64_t first;                  // row of the result

    // false: no such tile.  scan: LDS, free again on return.
    __device__ __forceinline__ bool init(const ExpertArgs& a, int32_t ftiles, int32_t ntiles, int32_t* scan) {
        int32_t f;
        if constexpr (P == kWeightGrad) {
            const int32_t n = xcd_tile_in_turn((a.E + a.shared) * ntiles, ftiles, f);
            if (n == kNoTile) return false;
            expert = n / ntiles;
            const int32_t n0 = (n - expert * ntiles) * NT;
            f0 = f * BF;
            const int32_t g = expert < a.E ? expert / a.E_loc * a.G + a.shared + expert % a.E_loc : a.src_seg * a.G;
            const GroupRows r = group_rows(a, g);
            len = r.rows;
            rows = min(NT, a.on - n0);
            first = (int64_t)expert * a.on + n0;
            fo.init(a.x + r.first * a.in + f0, a.in - f0, a.in, len, f0);
            no.init(a.gy + r.first * a.on + n0, rows, a.on, len, n0);
        } else {
            const RowTile t = find_row_tile<kWideThreads, NT>(
                a, scan, [&](int32_t rt, int32_t& ft) { return xcd_tile(rt, ftiles, ft); }, f);
            if (t.expert < 0) return false;
            __syncthreads();  // the words that named the tile become step 0
            expert = t.expert;
            rows = t.rows;
            first = t.first;
            f0 = f * BF;
            const uint16_t* we = a.w + (int64_t)expert * a.on * a.in;
            if constexpr (P == kForward) {
                len = a.in;
                fo.init(we + (int64_t)f0 * a.in, min(BF, a.on - f0), a.in, len);
                no.init(a.x + first * a.in, rows, a.in, len);
            } else {
                len = a.on;
                fo.init(we + f0, a.in - f0, a.in, len, f0);
                no.init(a.gy + first * a.on, rows, a.on, len);
            }
        }
        return true;
    }
};

// Four results, at and on, in the output's type.
template <Product P>
__device__ __forceinline__ void store4(const ExpertArgs& a, int64_t at, f32x4 v) {
    if (P == kWeightGrad && a.grad_type != EP_GRAD_BF16) {
        f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at);
        *o = a.grad_type == EP_GRAD_F32_ADD ? *o + v : v;
    } else {
        const v2u o = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        *reinterpret_cast<v2u*>(static_cast<uint16_t*>(a.out) + at) = o;
    }
}

template <Product P, int NT>
__global__ __launch_bounds__(kWideThreads) void k_expert_wide(ExpertArgs a, int32_t ftiles, int32_t ntiles) {
    using T = Tile<P, kFeatures, NT>;
    using FOp = typename T::FOp;
    using NOp = typename T::NOp;
    constexpr int kWavesN = NT / 64, kWavesF = 8 / kWavesN;  // a wave's tile: 64 rows
    constexpr int kF = kFeatures / kWavesF / 16, kN = 4;     // its fragments
    constexpr bool kUnits = NT == 256;
    constexpr int kUnit = kFeatures * kStepL, kBuffer = (kFeatures + NT) * kStepL;
    static_assert(kF >= kN, "the second half's N fragments are read beside F's");
    __shared__ __align__(1024) uint16_t lds[kUnits ? 5 * kUnit : 3 * kBuffer];
    const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
    const int wf = w / kWavesN * (kFeatures / kWavesF), wn = w % kWavesN * 64;
    const int32_t F = P == kForward ? a.on : a.in;
    T tile;
    if (!tile.init(a, ftiles, ntiles, reinterpret_cast<int32_t*>(lds))) return;
    const FOp& fo = tile.fo;
    const NOp& no = tile.no;
    const int32_t f0 = tile.f0, rows = tile.rows, len = tile.len;
    const int64_t first = tile.first;

    f32x4 acc[kF][kN] = {};
    // What LDS holds: for tiles of 128 rows three steps, of both operands; for
    // tiles of 256 five units of one operand's step, F's and N's in turn, which
    // is half a step more in flight than two whole steps.
    constexpr int kLoads = FOp::kLoads + NOp::kLoads;  // of a wave and step
    constexpr int kSlots = kUnits ? 5 : 3;
    auto next = [](int32_t v) { return v == kSlots - 1 ? 0 : v + 1; };
    const int32_t steps = (len + kStepL - 1) / kStepL;
    const bool busy = wn < rows;  // a wave past the tile's last row only loads
    int32_t in_slot = 0, out_slot = kUnits ? 3 : 2;  // to use, and to fill, next
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        uint16_t* const to = lds + s * (kUnits ? 2 * kUnit : kBuffer);
#pragma unroll
        for (int j = 0; j < FOp::kLoads; ++j) fo.load(to, s * kStepL, j);
        if (kUnits && s == 1) break;
#pragma unroll
        for (int j = 0; j < NOp::kLoads; ++j) no.load(to + kUnit, s * kStepL, j);
    }
    for (int32_t s = 0; s < steps; ++s) {
        // This step's loads have landed when only the later ones are
        // outstanding: loads return in order, and past the end they still
        // count, and write zeros.  Behind the barrier every wave's have, and
        // every wave is done with the last step's LDS, which is filled next.
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kUnits ? FOp::kLoads : kLoads) : "memory");
        lds_barrier();
        uint16_t *to_f, *to_n;
        const uint16_t *lf, *ln;
        if constexpr (kUnits) {  // N of the next step, then F of the one after it
            to_n = lds + out_slot * kUnit;
            out_slot = next(out_slot);
            to_f = lds + out_slot * kUnit;
            lf = lds + in_slot * kUnit;
            in_slot = next(in_slot);
            ln = lds + in_slot * kUnit;
        } else {
            to_f = lds + out_slot * kBuffer;
            to_n = to_f + kUnit;
            lf = lds + in_slot * kBuffer;
            ln = lf + kUnit;
        }
        out_slot = next(out_slot);
        in_slot = next(in_slot);
        auto load = [&](int j) {
            if (j < NOp::kLoads)
                no.load(to_n, (s + (kUnits ? 1 : 2)) * kStepL, j);
            else
                fo.load(to_f, (s + 2) * kStepL, j - NOp::kLoads);
        };
        if (!busy) {
#pragma unroll
            for (int j = 0; j < kLoads; ++j) load(j);
            continue;
        }
        bf16x8 fa[2][kF], fb[2][kN];
#pragma unroll
        for (int n = 0; n < kN; ++n) fb[0][n] = NOp::fragment(ln, wn + n * 16, 0);
#pragma unroll
        for (int f = 0; f < kF; ++f) fa[0][f] = FOp::fragment(lf, wf + f * 16, 0);
        // The loads and the second half's LDS reads go between the matrix
        // instructions of the first half.  All loads first keep every wave from
        // its products until the 64 of the workgroup are issued (1930 instead of
        // 1830 us); without the scheduling barriers the compiler collects them
        // at the end (2210 us).
#pragma unroll
        for (int f = 0; f < kF; ++f) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = f * kLoads / kF; j < (f + 1) * kLoads / kF; ++j) load(j);
            fa[1][f] = FOp::fragment(lf, wf + f * 16, 1);
            if (f < kN) fb[1][f] = NOp::fragment(ln, wn + f * 16, 1);
#pragma unroll
            for (int n = 0; n < kN; ++n)
                acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[0][f], fb[0][n], acc[f][n], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < kF; ++f)
#pragma unroll
            for (int n = 0; n < kN; ++n)
                acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[1][f], fb[1][n], acc[f][n], 0, 0, 0);
    }
    // No load may land in LDS that belongs to another workgroup by then.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // acc[f][n][j]: feature f0 + wf + 16 f + 4 (lane / 16) + j, row wn + 16 n + lane % 16
#pragma unroll
    for (int n = 0; n < kN; ++n) {
        const int32_t row = wn + n * 16 + lane % 16;
        if (row >= rows) continue;
#pragma unroll
        for (int f = 0; f < kF; ++f) {
            const int32_t fe = f0 + wf + f * 16 + lane / 16 * 4;
            if (fe >= F) continue;
            store4<P>(a, (first + row) * F + fe, acc[f][n]);
        }
    }
}

// Tiles of 64 features by 64 rows, for launches whose wide tiles would leave
// CUs without work: the same sums in the same order, ten steps in LDS, used in
// pairs (one at a time: 21 instead of 17 us for a row of 4096 values by 128
// features).  Bound by the latency of a pair, 0.5 us, where the wide tiles take
// 0.8 us a step.  A wave has 16 features by 32 rows.
template <Product P>
__global__ __launch_bounds__(kWideThreads) void k_expert_small(ExpertArgs a, int32_t ftiles, int32_t ntiles) {
    using T = Tile<P, kSmall, kSmall>;
    constexpr int kSlots = 5, kUnit = kSmall * kStepL, kBuffer = 4 * kUnit, kLoads = 4;  // loads of a wave and pair of steps
    static_assert(2 * (T::FOp::kLoads + T::NOp::kLoads) == kLoads, "");
    __shared__ __align__(1024) uint16_t lds[kSlots * kBuffer];
    const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
    const int wf = w % 4 * 16, wn = w / 4 * 32;
    const int32_t F = P == kForward ? a.on : a.in;
    T tile;
    if (!tile.init(a, ftiles, ntiles, reinterpret_cast<int32_t*>(lds))) return;
    const int32_t rows = tile.rows, steps = (tile.len + 2 * kStepL - 1) / (2 * kStepL);
    const bool busy = wn < rows;
    auto load = [&](int32_t s, int32_t slot) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            tile.fo.load(lds + slot * kBuffer + h * 2 * kUnit, (s * 2 + h) * kStepL, 0);
            tile.no.load(lds + slot * kBuffer + (h * 2 + 1) * kUnit, (s * 2 + h) * kStepL, 0);
        }
    };
    f32x4 acc[2] = {};
#pragma unroll
    for (int s = 0; s < kSlots - 1; ++s) load(s, s);
    int32_t slot = 0, to = kSlots - 1;
    for (int32_t s = 0; s < steps; ++s) {
        // As in the wide tiles: this step's loads have landed, in every wave,
        // and the last step's buffer is free.
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kSlots - 2) * kLoads) : "memory");
        lds_barrier();
        load(s + kSlots - 1, to);
        if (busy) {
            bf16x8 fa[4], fb[4][2];
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
                const uint16_t *lf = lds + slot * kBuffer + kk / 2 * 2 * kUnit, *ln = lf + kUnit;
                fa[kk] = T::FOp::fragment(lf, wf, kk % 2);
#pragma unroll
                for (int n = 0; n < 2; ++n) fb[kk][n] = T::NOp::fragment(ln, wn + n * 16, kk % 2);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                    acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[kk], fb[kk][n], acc[n], 0, 0, 0);
        }
        to = slot;
        slot = slot == kSlots - 1 ? 0 : slot + 1;
    }
    // No load may land in LDS that belongs to another workgroup by then.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int32_t fe = tile.f0 + wf + lane / 16 * 4;
    if (fe >= F) return;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int32_t row = wn + n * 16 + lane % 16;
        if (row < rows) store4<P>(a, (tile.first + row) * F + fe, acc[n]);
    }
}

// Tiles of a launch with tiles of BF features by NT rows.
template <Product P>
int64_t tiles_of(const ExpertArgs& a, int bf, int nt, int32_t& ftiles, int32_t& ntiles) {
    const int32_t F = P == kForward ? a.on : a.in;
    ftiles = (F + bf - 1) / bf;
    ntiles = (a.on + nt - 1) / nt;
    int64_t rtiles = P == kWeightGrad ? (int64_t)ntiles * (a.E + a.shared) : max_row_tiles(a, nt);
    if (P == kWeightGrad) rtiles = (rtiles + 15) / 16 * 16;  // whole turns of the XCDs
    return rtiles * ftiles;
}

template <Product P, int BF, int NT>
hipError_t launch(const ExpertArgs& a, hipStream_t stream) {
    int32_t ftiles, ntiles;
    const int64_t blocks = (tiles_of<P>(a, BF, NT, ftiles, ntiles) + 7) / 8 * 8;
    if (blocks == 0) return hipSuccess;
    if (const hipError_t e = check_grid(blocks, kWideThreads)) return e;
    if constexpr (BF == kSmall)
        hipLaunchKernelGGL((k_expert_small<P>), dim3((unsigned)blocks), dim3(kWideThreads), 0, stream, a, ftiles, ntiles);
    else
        hipLaunchKernelGGL((k_expert_wide<P, NT>), dim3((unsigned)blocks), dim3(kWideThreads), 0, stream, a, ftiles,
                           ntiles);
    return hipGetLastError();
}

// Small tiles where they are few.  Forward, us with small and with wide tiles:
// 8 experts with a row, 7168 values, 512 features (64 small tiles) 27 and 87,
// 2048 features (256) 38 and 91, 4096 (512) 86 and 112; 32 experts with 4 rows,
// 4096 values, 512 features (272) 24 and 52, 1024 (544) 44 and 54, 2048 (1088)
// 151 and 122; 128 rows, 2048 values, 512 features (768) 36 and 50, 1024 (1536)
// 72 and 52.  Input's gradient, timed with the weights' behind it, which has no
// small form and takes the same time on both sides: 32 experts with 4 rows of 4096
// values, 512 features (272) 73 and 102, 1024 (544) 174 and 160.
// Wide row tiles by the rows a group has on average.  Forward over 32 experts of
// 4096 x 7168, us at 16, 64, 128, 256 and 512 rows a group: 128-row tiles 317
// 335 454 716 1128, 256-row tiles 330 363 405 689 1008 (128 rows on average fill
// a second tile of 128 in half of the groups).
template <Product P>
hipError_t by_size(const ExpertArgs& a, hipStream_t stream) {
    int32_t ftiles, ntiles;
    if (tiles_of<P>(a, kSmall, kSmall, ftiles, ntiles) <= (P == kForward ? 768 : 512)) return launch<P, kSmall, kSmall>(a, stream);
    const int64_t groups = a.slots < a.E + a.shared ? a.slots : a.E + a.shared;
    return a.slots >= 96 * groups ? launch<P, kFeatures, 256>(a, stream) : launch<P, kFeatures, 128>(a, stream);
}

}  // namespace

hipError_t launch_expert_gemm(const ExpertArgs& a, hipStream_t stream) { return by_size<kForward>(a, stream); }
hipError_t launch_expert_gemm_bwd_x(const ExpertArgs& a, hipStream_t stream) { return by_size<kInputGrad>(a, stream); }
hipError_t launch_expert_gemm_bwd_w(const ExpertArgs& a, hipStream_t stream) {
    return launch<kWeightGrad, kFeatures, 256>(a, stream);
}

}  // namespace epx
