// The experts' product over 4-bit weights: y[r, n] = rowscale[e, n] *
// sum_h x[r, h] e2m1(code) e4m3(scale).  Tiles of 64 features by 64 rows are
// built from 32 values of the summed dimension at a time, staged in LDS with
// it contiguous.
#include "expert_device.h"

namespace epx {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kGemmThreads = 256;
constexpr int kTile = 64;   // results of a tile, each way
constexpr int kStep = 32;   // values of L a step
constexpr int kPitch = 40;  // LDS row pitch in bf16

// Operand rows m0.. (of `rows`), L contiguous: element (m, l) at p[m * ld + l].
__device__ __forceinline__ void stage_rows(uint16_t* lds, const uint16_t* p, int64_t ld, int32_t m0, int32_t rows,
                                           int32_t l0, int32_t len) {
    const int m = threadIdx.x / 4, c = threadIdx.x % 4 * 8;
    v4u v = {0, 0, 0, 0};
    if (m0 + m < rows && l0 + c < len) v = *reinterpret_cast<const v4u*>(p + (int64_t)(m0 + m) * ld + l0 + c);
    *reinterpret_cast<v4u*>(lds + m * kPitch + c) = v;
}

// 4-bit rows: half a block (8 codes) a thread, times the block's scale.
__device__ __forceinline__ void stage_nvfp4(uint16_t* lds, const uint8_t* codes, const uint8_t* scales, int64_t in,
                                            int32_t m0, int32_t rows, int32_t l0, int32_t len) {
    const int m = threadIdx.x / 4, c = threadIdx.x % 4 * 8;
    v4u o = {0, 0, 0, 0};
    if (m0 + m < rows && l0 + c < len) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(codes + (int64_t)(m0 + m) * (in / 2) + (l0 + c) / 2);
        const float s = e4m3_decode_signed(scales[(int64_t)(m0 + m) * (in / 16) + (l0 + c) / 16]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = pack_bf16x2(e2m1_decode((q >> (8 * j)) & 15) * s, e2m1_decode((q >> (8 * j + 4)) & 15) * s);
    }
    *reinterpret_cast<v4u*>(lds + m * kPitch + c) = o;
}

__global__ __launch_bounds__(kGemmThreads) void k_expert_nvfp4(ExpertArgs a, int32_t ftiles) {
    __shared__ uint16_t lf[kTile * kPitch], ln[kTile * kPitch];
    __shared__ int32_t ls[16];
    const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
    int32_t f;
    const RowTile t = find_row_tile<kGemmThreads, kTile>(
        a, ls,
        [&](int32_t, int32_t& ft) {
            ft = blockIdx.x % ftiles;
            return (int32_t)(blockIdx.x / ftiles);
        },
        f);
    if (t.expert < 0) return;
    const int32_t f0 = f * kTile;
    const uint8_t* codes = a.codes + (int64_t)t.expert * a.on * (a.in / 2);
    const uint8_t* scales = a.scales + (int64_t)t.expert * a.on * (a.in / 16);
    f32x4 acc[4] = {};
    for (int32_t l0 = 0; l0 < a.in; l0 += kStep) {
        __syncthreads();
        stage_nvfp4(lf, codes, scales, a.in, f0, a.on, l0, a.in);
        stage_rows(ln, a.x + t.first * a.in, a.in, 0, t.rows, l0, a.in);
        __syncthreads();
        const bf16x8 fa = *reinterpret_cast<const bf16x8*>(lf + (w * 16 + lane % 16) * kPitch + lane / 16 * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x8 fb = *reinterpret_cast<const bf16x8*>(ln + (i * 16 + lane % 16) * kPitch + lane / 16 * 8);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, fb, acc[i], 0, 0, 0);
        }
    }
    // acc[i][j]: feature f0 + 16 w + 4 (lane / 16) + j, row 16 i + lane % 16
    const int32_t fe = f0 + w * 16 + lane / 16 * 4;
    if (fe >= a.on) return;
    float rs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) rs[j] = bf16_lo(a.rowscale[(int64_t)t.expert * a.on + fe + j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t n = i * 16 + lane % 16;
        if (n >= t.rows) continue;
        uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + (t.first + n) * a.on + fe);
        o[0] = pack_bf16x2(acc[i][0] * rs[0], acc[i][1] * rs[1]);
        o[1] = pack_bf16x2(acc[i][2] * rs[2], acc[i][3] * rs[3]);
    }
}

}  // namespace

hipError_t launch_expert_gemm_nvfp4(const ExpertArgs& a, hipStream_t stream) {
    const int32_t ftiles = (a.on + kTile - 1) / kTile;
    const int64_t blocks = max_row_tiles(a, kTile) * ftiles;
    if (blocks == 0) return hipSuccess;
    if (blocks * kGemmThreads > 0xFFFFFFFFll) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_expert_nvfp4, dim3((unsigned)blocks), dim3(kGemmThreads), 0, stream, a, ftiles);
    return hipGetLastError();
}

}  // namespace epx
