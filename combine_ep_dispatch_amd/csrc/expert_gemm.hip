// The experts' products: every receive row times its expert's weights, and
// both gradients.
//   forward      y[r, n]  = sum_h x[r, h] w[e, n, h]
//   4-bit        the same, w[e, n, h] = e2m1 * e4m3 * rowscale[e, n]
//   input's      gx[r, h] = sum_n gy[r, n] w[e, n, h]
//   weights'     gw[e, n, h] = sum_r gy[r, n] x[r, h]
// Each is a product of an F operand (features: the output's contiguous
// dimension, the rows of the matrix instruction's result) and an N operand
// over a summed dimension L.  Tiles of 64 x 64 results are built from 32
// values of L at a time, staged in LDS with L contiguous.
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

// Operand columns m0.. (of `cols`), L the rows: element (m, l) at p[l * ld + m].
__device__ __forceinline__ void stage_cols(uint16_t* lds, const uint16_t* p, int64_t ld, int32_t m0, int32_t cols,
                                           int32_t l0, int32_t len) {
    const int l = threadIdx.x / 8, c = threadIdx.x % 8 * 8;
    v4u v = {0, 0, 0, 0};
    if (l0 + l < len && m0 + c < cols) v = *reinterpret_cast<const v4u*>(p + (int64_t)(l0 + l) * ld + m0 + c);
#pragma unroll
    for (int j = 0; j < 8; ++j) lds[(c + j) * kPitch + l] = (uint16_t)(v[j / 2] >> (j % 2 * 16));
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

enum Product { kForward, kNvfp4, kInputGrad, kWeightGrad };

template <Product P>
__global__ __launch_bounds__(kGemmThreads) void k_expert_simple(ExpertArgs a, int32_t ftiles, int32_t ntiles) {
    __shared__ uint16_t lf[kTile * kPitch], ln[kTile * kPitch];
    __shared__ int32_t ls[16];
    const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
    const int32_t F = P == kForward || P == kNvfp4 ? a.on : a.in;
    int32_t expert, f0, n0 = 0, nrows, len;
    int64_t first = 0;
    if (P == kWeightGrad) {
        // one tile of one expert's gradient; a group that has no part in it
        // (a segment's shared group) is left out
        const int32_t f = blockIdx.x % ftiles, n = blockIdx.x / ftiles % ntiles;
        expert = blockIdx.x / ftiles / ntiles;
        f0 = f * kTile;
        n0 = n * kTile;
        const int32_t g = expert < a.E ? expert / a.E_loc * a.G + a.shared + expert % a.E_loc : a.src_seg * a.G;
        const GroupRows r = group_rows(a, g);
        first = r.first;
        len = r.rows;
        nrows = a.on;
    } else {
        int32_t f;
        const RowTile t = find_row_tile<kGemmThreads, kTile>(
            a, ls,
            [&](int32_t, int32_t& ft) {
                ft = blockIdx.x % ftiles;
                return (int32_t)(blockIdx.x / ftiles);
            },
            f);
        if (t.expert < 0) return;
        expert = t.expert;
        first = t.first;
        nrows = t.rows;
        f0 = f * kTile;
        len = P == kInputGrad ? a.on : a.in;
    }
    f32x4 acc[4] = {};
    for (int32_t l0 = 0; l0 < len; l0 += kStep) {
        __syncthreads();
        if (P == kForward) stage_rows(lf, a.w + (int64_t)expert * a.on * a.in, a.in, f0, a.on, l0, len);
        if (P == kNvfp4)
            stage_nvfp4(lf, a.codes + (int64_t)expert * a.on * (a.in / 2), a.scales + (int64_t)expert * a.on * (a.in / 16),
                        a.in, f0, a.on, l0, len);
        if (P == kInputGrad) stage_cols(lf, a.w + (int64_t)expert * a.on * a.in, a.in, f0, a.in, l0, len);
        if (P == kWeightGrad) stage_cols(lf, a.x + first * a.in, a.in, f0, a.in, l0, len);
        if (P == kForward || P == kNvfp4) stage_rows(ln, a.x + first * a.in, a.in, 0, nrows, l0, len);
        if (P == kInputGrad) stage_rows(ln, a.gy + first * a.on, a.on, 0, nrows, l0, len);
        if (P == kWeightGrad) stage_cols(ln, a.gy + first * a.on, a.on, n0, a.on, l0, len);
        __syncthreads();
        const bf16x8 fa = *reinterpret_cast<const bf16x8*>(lf + (w * 16 + lane % 16) * kPitch + lane / 16 * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x8 fb = *reinterpret_cast<const bf16x8*>(ln + (i * 16 + lane % 16) * kPitch + lane / 16 * 8);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, fb, acc[i], 0, 0, 0);
        }
    }
    // acc[i][j]: feature f0 + 16 w + 4 (lane / 16) + j, row 16 i + lane % 16
    const int32_t f = f0 + w * 16 + lane / 16 * 4;
    if (f >= F) return;
    float rs[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    if (P == kNvfp4)
#pragma unroll
        for (int j = 0; j < 4; ++j) rs[j] = bf16_lo(a.rowscale[(int64_t)expert * a.on + f + j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int32_t n = n0 + i * 16 + lane % 16;
        if (n >= nrows) continue;
        const int64_t at = (P == kWeightGrad ? (int64_t)expert * a.on + n : first + n) * F + f;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = P == kNvfp4 ? acc[i][j] * rs[j] : acc[i][j];
        if (P == kWeightGrad && a.grad_type != EP_GRAD_BF16) {
            f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + at);
            f32x4 s = {v[0], v[1], v[2], v[3]};
            if (a.grad_type == EP_GRAD_F32_ADD) s += *o;
            *o = s;
        } else {
            uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at);
            o[0] = pack_bf16x2(v[0], v[1]);
            o[1] = pack_bf16x2(v[2], v[3]);
        }
    }
}

template <Product P>
hipError_t product(const ExpertArgs& a, hipStream_t stream) {
    const int32_t F = P == kForward || P == kNvfp4 ? a.on : a.in;
    const int32_t ftiles = (F + kTile - 1) / kTile, ntiles = (a.on + kTile - 1) / kTile;
    const int64_t blocks =
        P == kWeightGrad ? (int64_t)ftiles * ntiles * (a.E + a.shared) : max_row_tiles(a, kTile) * ftiles;
    if (blocks == 0) return hipSuccess;
    if (blocks * kGemmThreads > 0xFFFFFFFFll) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_expert_simple<P>, dim3((unsigned)blocks), dim3(kGemmThreads), 0, stream, a, ftiles, ntiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm(const ExpertArgs& a, hipStream_t stream) { return product<kForward>(a, stream); }
hipError_t launch_expert_gemm_nvfp4(const ExpertArgs& a, hipStream_t stream) { return product<kNvfp4>(a, stream); }
hipError_t launch_expert_gemm_bwd_x(const ExpertArgs& a, hipStream_t stream) { return product<kInputGrad>(a, stream); }
hipError_t launch_expert_gemm_bwd_w(const ExpertArgs& a, hipStream_t stream) { return product<kWeightGrad>(a, stream); }

}  // namespace epx
