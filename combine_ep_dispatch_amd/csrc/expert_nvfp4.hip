// The experts' product over 4-bit weights: y[r, n] = rowscale[e, n] *
// sum_h x[r, h] e2m1(code) e4m3(scale).
#include "expert_device.h"

namespace epx {
namespace {

constexpr int kFewThreads = 256;

// E4M3 byte `at` (0..3) of a word.
__device__ __forceinline__ float e4m3_of(uint32_t word, int at) {
    switch (at) {
        case 0: return __builtin_amdgcn_cvt_f32_fp8((int)word, 0);
        case 1: return __builtin_amdgcn_cvt_f32_fp8((int)word, 1);
        case 2: return __builtin_amdgcn_cvt_f32_fp8((int)word, 2);
        default: return __builtin_amdgcn_cvt_f32_fp8((int)word, 3);
    }
}

// e2m1(code) * e4m3(scale) of 8 codes: at most 2 by 4 significant bits, exact in bf16.
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

// Few rows: the weights stream from memory into registers, 16 features a
// wave; lane (i, q) holds feature i and, of every chunk of KC values of the
// summed dimension, the KC / 4 from q * KC / 4 on, so that its loads are 16
// consecutive bytes and its block scales are whole.  The matrix instruction
// does not care which value is which as long as both operands agree: the
// rows, staged in LDS, are read in the same order.
// WK waves share the summed dimension, 4 / WK the features.  WORDS: every
// feature's scales start at a word (in_dim is a multiple of 64).
//
// Two chunks of weights are in flight in registers and the rows' chunks go
// round three LDS buffers, so that one barrier a chunk is enough: a wave
// stages chunk c + 2, into the buffer of chunk c - 1, only after the barrier
// of chunk c, which every wave reaches after computing chunk c - 1.
template <int NR, int KC, int WK, bool WORDS>
__global__ __launch_bounds__(kFewThreads) void k_nvfp4_few(ExpertArgs a, int32_t ftiles) {
    static_assert(KC == 512 || KC == 256, "a row's chunk is one load of a wave or half of one");
    constexpr int kWN = 4 / WK;
    constexpr int kLane = KC / 4;        // values of a lane and chunk
    constexpr int kCodes = kLane / 32;   // its 16-byte code loads
    constexpr int kScales = kLane / 64;  // its 4-byte scale words
    constexpr int kPitch = KC * 2 + 16;  // LDS bytes of a row's chunk: 16 rows fall on different banks
    constexpr int kBuffer = WK * NR * kPitch;
    __shared__ __align__(16) uint8_t lds[3 * kBuffer];
    __shared__ __align__(16) int32_t scan[16];
    const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave));
    const int i = lane % 16, q = lane / 16, wn = w % kWN, wk = w / kWN;
    int32_t f;
    const RowTile t = find_row_tile<kFewThreads, NR>(
        a, scan, [&](int32_t rt, int32_t& ft) { return xcd_tile(rt, ftiles, ft); }, f);
    if (t.expert < 0) return;
    const int32_t in = a.in, f0 = uniform((f * kWN + wn) * 16);
    const int64_t row0 = (int64_t)t.expert * a.on + f0;
    const int32_t frows = max(min(16, a.on - f0), 0);  // 0: this wave only helps with the staging
    const int32_t cpitch = in / 2, spitch = in / 16;
    const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(a.codes + row0 * cpitch), (short)0, uniform(frows * cpitch), kBufferWord3);
    const __amdgpu_buffer_rsrc_t rsc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(a.scales + row0 * spitch), (short)0, uniform(frows * spitch), kBufferWord3);
    const int32_t voff_c = i * cpitch + q * (kLane / 2), voff_s = i * spitch + q * (kLane / 16);

    struct Chunk {
        v4u codes[kCodes];
        uint32_t scales[kScales];
    };
    const int32_t chunks = (in + WK * KC - 1) / (WK * KC);
    // Weights of chunk c of this wave: values [l, l + KC), l = (c WK + wk) KC.
    // Past a feature's end the next one's codes arrive (zeros past the last).
    auto load = [&](Chunk& ch, int32_t c) {
        const int32_t l = (c * WK + wk) * KC;
#pragma unroll
        for (int j = 0; j < kCodes; ++j) ch.codes[j] = __builtin_amdgcn_raw_buffer_load_b128(rc, voff_c + l / 2 + j * 16, 0, 2);
#pragma unroll
        for (int j = 0; j < kScales; ++j) {
            const int32_t at = voff_s + l / 16 + j * 4;
            if constexpr (WORDS) {
                ch.scales[j] = __builtin_amdgcn_raw_buffer_load_b32(rsc, at, 0, 0);
            } else {  // features whose scales start between words
                uint32_t v = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    v |= (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rsc, at + b, 0, 0) << (8 * b);
                ch.scales[j] = v;
            }
        }
    };
    // The rows' part of chunk c: row r at r * kPitch of the wave group's buffer.
    auto stage = [&](int32_t c) {
        const int32_t l = (c * WK + wk) * KC;
        uint8_t* to = lds + (c % 3) * kBuffer + wk * NR * kPitch;
        const int32_t voff = l + lane * 8 < in ? (l + lane * 8) * 2 : kOutside;
        for (int r = wn; r < t.rows; r += kWN)
            if (KC == 512 || lane < 32)
                load_to_lds(a.x + (t.first + r) * in, in * 2, reinterpret_cast<uint16_t*>(to + r * kPitch), voff);
    };
    f32x4 acc[NR / 16] = {};
    auto compute = [&](const Chunk& ch, int32_t c) {
        const uint8_t* from = lds + (c % 3) * kBuffer + wk * NR * kPitch + i * kPitch + q * (kLane * 2);
        const int32_t left = (in - (c * WK + wk) * KC - q * kLane) / 16;  // of this lane's blocks: those before the end
        uint32_t sc[kScales];
#pragma unroll
        for (int j = 0; j < kScales; ++j) {
            const int n = min(max(left - 4 * j, 0), 4);
            sc[j] = n == 4 ? ch.scales[j] : ch.scales[j] & ((1u << (8 * n)) - 1);
        }
#pragma unroll
        for (int j = 0; j < kLane / 8; ++j) {
            const bf16x8 wv = weights8(ch.codes[j / 4][j % 4], e4m3_of(sc[j / 8], j / 2 % 4));
#pragma unroll
            for (int n = 0; n < NR / 16; ++n) {
                const bf16x8 xv = *reinterpret_cast<const bf16x8*>(from + n * 16 * kPitch + j * 16);
                acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xv, acc[n], 0, 0, 0);
            }
        }
    };
    Chunk ch[2];
    stage(0);
    load(ch[0], 0);
    asm volatile("" ::: "memory");  // chunk 0's loads are the older ones
    if (chunks > 1) {
        stage(1);
        load(ch[1], 1);
    }
    for (int32_t c = 0; c < chunks; c += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (c + h >= chunks) break;
            // This chunk's rows are in LDS once all loads but the next chunk's
            // weights have returned (loads return in order).
            if (c + h + 1 < chunks)
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kCodes + kScales) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            lds_barrier();
            compute(ch[h], c + h);
            asm volatile("" ::: "memory");
            if (c + h + 2 < chunks) {
                stage(c + h + 2);
                load(ch[h], c + h + 2);
            }
        }
    }
    if constexpr (WK > 1) {  // the waves' shares, added in their order
        f32x4* part = reinterpret_cast<f32x4*>(lds);
        __syncthreads();
        if (wk > 0)
#pragma unroll
            for (int n = 0; n < NR / 16; ++n) part[(((wk - 1) * kWN + wn) * (NR / 16) + n) * kWave + lane] = acc[n];
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int s = 0; s < WK - 1; ++s)
#pragma unroll
            for (int n = 0; n < NR / 16; ++n) acc[n] += part[((s * kWN + wn) * (NR / 16) + n) * kWave + lane];
    }
    // acc[n][j]: feature f0 + 4 q + j, row 16 n + i
    const int32_t fe = f0 + q * 4;
    if (fe >= a.on) return;
    const v2u rs = *reinterpret_cast<const v2u*>(a.rowscale + row0 + q * 4);
#pragma unroll
    for (int n = 0; n < NR / 16; ++n) {
        const int32_t r = n * 16 + i;
        if (r >= t.rows) continue;
        const v2u o = {pack_bf16x2(acc[n][0] * bf16_lo(rs.x), acc[n][1] * bf16_hi(rs.x)),
                       pack_bf16x2(acc[n][2] * bf16_lo(rs.y), acc[n][3] * bf16_hi(rs.y))};
        *reinterpret_cast<v2u*>(static_cast<uint16_t*>(a.out) + (t.first + r) * a.on + fe) = o;
    }
}

template <int NR, int KC, int WK>
hipError_t few(const ExpertArgs& a, hipStream_t stream) {
    constexpr int kF = 64 / WK;
    const int32_t ftiles = (a.on + kF - 1) / kF;
    const int64_t tiles = max_row_tiles(a, NR) * ftiles, blocks = (tiles + 7) / 8 * 8;
    if (tiles == 0) return hipSuccess;
    if (blocks * kFewThreads > 0xFFFFFFFFll) return hipErrorInvalidValue;
    if (a.in % 64 == 0)
        hipLaunchKernelGGL((k_nvfp4_few<NR, KC, WK, true>), dim3((unsigned)blocks), dim3(kFewThreads), 0, stream, a,
                           ftiles);
    else
        hipLaunchKernelGGL((k_nvfp4_few<NR, KC, WK, false>), dim3((unsigned)blocks), dim3(kFewThreads), 0, stream, a,
                           ftiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm_nvfp4(const ExpertArgs& a, hipStream_t stream) {
    const int64_t groups = a.slots < a.E + a.shared ? a.slots : a.E + a.shared;
    if (groups == 0) return hipSuccess;
    const int64_t mean = a.slots / groups;
    if (mean > 24) return few<64, 256, 1>(a, stream);
    if (mean > 10) return few<32, 256, 1>(a, stream);
    if (groups * ((a.on + 63) / 64) < 256) return few<16, 256, 4>(a, stream);
    return few<16, 512, 1>(a, stream);
}

}  // namespace epx
