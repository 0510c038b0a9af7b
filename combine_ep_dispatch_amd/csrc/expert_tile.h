// The operands of a tile of the experts' products on their way through LDS:
// steps of kStepL values of the summed dimension L, copied there by the loads
// themselves.
#pragma once

#include "expert_device.h"

namespace epx {

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kStepL = 64;  // values of L a step: whole 128-byte lines of rows

// The wave among the WAVES that share an operand; alone, each has its own.
template <int WAVES>
__device__ __forceinline__ int32_t wave_of() {
    return WAVES == 1 ? 0 : uniform((int32_t)(threadIdx.x / kWave));
}

// One operand's step of BM x kStepL values, copied to LDS by the loads
// themselves (16 bytes a lane, 1 KiB a wave and load, to consecutive LDS
// addresses; the lanes pick their global addresses so that the LDS tile comes
// out swizzled).  Loads past the operand's end write zeros.
//
// Rows: L contiguous.  LDS row m (128 bytes) holds its 8 chunks of 16 bytes at
// c ^ (m / 2 % 8): the 16 rows of a fragment's quarter fall on all banks.
template <int BM, int WAVES>
struct RowsOperand {
    static constexpr int kLoads = BM / 8 / WAVES;  // of each wave and step
    const uint16_t* base;
    int32_t ld, len, records;
    int32_t voff[kLoads], chunk[2];

    // rows: valid rows from base on; pitch: theirs; l: values of L
    __device__ __forceinline__ void init(const uint16_t* p, int32_t rows, int32_t pitch, int32_t l) {
        const int lane = threadIdx.x & (kWave - 1), w = wave_of<WAVES>();
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
        const int w = wave_of<WAVES>();
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
template <int BM, int WAVES>
struct ColsOperand {
    static constexpr int kLoads = BM / 8 / WAVES;
    static constexpr int kPerRow = BM / 8;         // lanes of one LDS row
    static constexpr int kRows = kWave / kPerRow;  // LDS rows of one load
    const uint16_t* base;
    int32_t ld, len, cut;
    int32_t voff[kLoads];

    // p: column m0 of the operand; cols: valid columns from p on; pitch: of rows; l: rows
    __device__ __forceinline__ void init(const uint16_t* p, int32_t cols, int32_t pitch, int32_t l, int32_t m0) {
        const int lane = threadIdx.x & (kWave - 1), w = wave_of<WAVES>();
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
        const int w = wave_of<WAVES>();
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

}  // namespace epx
