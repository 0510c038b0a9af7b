// Low-rank adapters of many requests beside the experts' products.  Row r, of
// expert e and of a token with adapter d:
//   u[r] = s_d A[d, e] x[r]                     (k_lora_down)
//   y[r] = w[e] x[r] + B[d, e] u[r]             (k_product, forward)
// and the gradients, w fixed:
//   gu[r] = s_d B[d, e]^T gy[r]                 (k_lora_down over B)
//   gx[r] = w[e]^T gy[r] + A[d, e]^T gu[r]      (k_product, input's gradient)
//   gA[d, e] = sum_r gu[r]^T x[r],  gB[d, e] = sum_r gy[r]^T u[r]   (k_lora_bwd_w)
// The second product of an adapter is added to the experts' own in the registers that
// hold it, before anything is rounded; the adapters' rows need not be sorted.
//
// 32 experts of 4096 x 7168: 128 rows of 16 adapters of rank 16 328 to 345 us for u and the
// product, bound by reading 1.92 GB of weights; 16 experts of 2048 x 1416, 4092 rows,
// every token another of 5 adapters, rank 64: 145 to 170 us, of 16 290, of 256 850.  A
// training step of 4 adapters of rank 16 over 32 experts of 2048 x 2048, 32 768 rows: 734
// to 775 us, of which the two products take 278 and 310 (990 and 890 TFLOP/s); of 256 2660.
#include "expert_loop.h"

namespace epx {
namespace {

enum Product { kForward, kInputGrad };

template <Product P>
__global__ __launch_bounds__(kLoopThreads) __attribute__((amdgpu_waves_per_eu(1, 1))) void k_product(BlockArgs a, int32_t ftiles) {
    using FOp = typename std::conditional<P == kForward, LoopRows<kTileF>, LoopCols>::type;
    __shared__ __align__(1024) uint16_t lds[kLoopLds / 2];
    const int lane = threadIdx.x & (kWave - 1), i = lane % 16, q = lane / 16;
    const int32_t F = P == kForward ? a.e.on : a.e.in, L = P == kForward ? a.e.in : a.e.on;
    FOp fo;
    if constexpr (P == kForward) fo.init(L);
    auto start_f = [&](FOp& op, const LoopTile& t) {
        const int32_t f0 = t.ft * kTileF;
        const bool on = t.expert >= 0;
        const uint16_t* const we = a.e.w + (on ? (int64_t)t.expert * a.e.on * a.e.in : 0);
        if constexpr (P == kForward)
            op.start(we + (int64_t)f0 * L, on ? min(kTileF, F - f0) : 0);
        else
            op.start(we + f0, f0, F - f0, F, on ? L : 0);
    };
    auto start_n = [&](auto& op, const LoopTile& t) {
        op.start((P == kForward ? a.e.x : a.e.gy) + t.first * L, t.expert >= 0 ? t.rows : 0);
    };
    auto begin = [&](auto nt, const LoopTile& t, auto& acc) {
        using S = Shape<decltype(nt)::value>;
        const int32_t f0 = t.ft * kTileF + S::wf();
        add_adapters<S::kF, S::kN>(a, t.first, t.rows, S::wn(), [&](int f, int32_t ad, int32_t c) {
            const int32_t fe = f0 + f * 16 + i, rank = a.l.rank;
            const int64_t pair = (int64_t)ad * (a.e.E + a.e.shared) + t.expert;
            bf16x8 v = {};
            if (fe >= F) return v;
            if constexpr (P == kForward) {
                v = *reinterpret_cast<const bf16x8*>(a.l.b + (pair * F + fe) * rank + c * 8);
            } else {
                const __bf16* const p = reinterpret_cast<const __bf16*>(a.l.a) + (pair * rank + c * 8) * F + fe;
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = p[(int64_t)k * F];
            }
            return v;
        }, acc);
    };
    run_tiles(a.e, ftiles, L, lds, fo, start_f, start_n, begin, [&](auto nt, const LoopTile& t, auto& acc) {
        using S = Shape<decltype(nt)::value>;
        constexpr int KF = S::kF, KN = S::kN;
        const int wn = S::wn(), wf = S::wf();
        const int32_t f0 = t.ft * kTileF;
        // acc[f][n][j]: feature f0 + wf + 16 f + 4 q + j, row wn + 16 n + i
#pragma unroll
        for (int n = 0; n < KN; ++n) {
            const int32_t row = wn + n * 16 + i;
            if (row >= t.rows) continue;
            uint16_t* const out = static_cast<uint16_t*>(a.e.out) + (t.first + row) * F;
#pragma unroll
            for (int f = 0; f < KF; ++f) {
                const int32_t fe = f0 + wf + f * 16 + q * 4;
                if (fe < F)
                    *reinterpret_cast<v2u*>(out + fe) =
                        v2u{pack_bf16x2(acc[f][n][0], acc[f][n][1]), pack_bf16x2(acc[f][n][2], acc[f][n][3])};
            }
        }
    });
}

template <Product P>
hipError_t product(const BlockArgs& a, hipStream_t stream) {
    const int32_t F = P == kForward ? a.e.on : a.e.in, ftiles = (F + kTileF - 1) / kTileF;
    unsigned blocks;
    if (const hipError_t e = loop_blocks(a.e, ftiles, blocks)) return e;
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((k_product<P>), dim3(blocks), dim3(kLoopThreads), 0, stream, a, ftiles);
    return hipGetLastError();
}

constexpr int kDownWaves = 4;
constexpr int kDownThreads = kDownWaves * kWave;

// The adapter's weights as a wave's operand: A, rank rows along L, or for gu B,
// whose rows of rank values are L.  Past the rank: zeros.
template <bool BWD, int P>
struct AdapterOperand : std::conditional<BWD, ColsOperand<P, 1>, RowsOperand<P, 1>>::type {
    using Base = typename std::conditional<BWD, ColsOperand<P, 1>, RowsOperand<P, 1>>::type;
    __device__ __forceinline__ void start(const uint16_t* p, int32_t rank, int32_t l) {
        if constexpr (BWD)
            Base::init(p, rank, rank, l, 0);
        else
            Base::init(p, rank, l, l);
    }
};

// u of NT rows, P >= rank.  Each of 4 waves by itself sums every fourth step of 64
// values, kept under way kRing - 1 steps ahead in its own part of LDS; the workgroup
// adds the four up in order.  The workgroups of a tile (blockIdx.y) share its
// adapters: with few tiles, as in a decode step, each adapter's weights are read by
// a workgroup of their own.  BWD: gu, from gy and B.
// Bound by the rows' bytes for many rows: 32 768 of 7168, rank 32, 124 to 148 us (470 MB,
// 3.2 to 3.8 TB/s), of 2048, rank 16, 40 us (3.4 TB/s); by latency for few: 128 rows of 7168 with
// 16 adapters 13 us (fragments from memory to registers, without LDS: 264 and 20 us).
template <bool BWD, int P, int NT>
__global__ __launch_bounds__(kDownThreads) void k_lora_down(BlockArgs a, float* u) {
    using Op = AdapterOperand<BWD, P>;
    constexpr int kStep = (NT + P) * kStepL;  // elements of a wave's step
    constexpr int kRing = NT + P <= 32 ? 4 : NT + P <= 96 ? 3 : 2;
    constexpr int kFL = P / 8, kNL = NT / 8, KP = P / 16, KN = NT / 16;
    constexpr int kPart = kDownWaves * NT * (P + 1) * 4, kLds = kDownWaves * kRing * kStep * 2;
    static_assert(kPart <= kLds && kLds <= 160 * 1024 && (kRing - 1) * (kFL + kNL) < 64, "");
    __shared__ __align__(1024) uint8_t lds[kLds];
    __shared__ int32_t scan[kDownWaves + 3], ads[NT];
    int32_t none;
    const RowTile t = find_row_tile<kDownThreads, NT>(
        a.e, scan, [&](int32_t rt, int32_t& f) { return xcd_tile(rt, 1, f); }, none);
    if (t.expert < 0) return;
    const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave)), i = lane % 16, q = lane / 16;
    const int32_t L = BWD ? a.e.on : a.e.in, rank = a.l.rank, steps = (L + kStepL - 1) / kStepL;
    const uint16_t* const x = (BWD ? a.e.gy : a.e.x) + t.first * L;
    if ((int32_t)threadIdx.x < NT) ads[threadIdx.x] = (int32_t)threadIdx.x < t.rows ? row_adapter(a, t.first + threadIdx.x) : -1;
    __syncthreads();
    int32_t ad[KN];
#pragma unroll
    for (int n = 0; n < KN; ++n) ad[n] = ads[n * 16 + i];
    uint16_t* const mine = reinterpret_cast<uint16_t*>(lds) + w * kRing * kStep;
    float* const part = reinterpret_cast<float*>(lds);
    RowsOperand<NT, 1> no;
    int32_t at = 0;
    for (int32_t cur = next_adapter(ad, -1); cur != kNoAdapter; cur = next_adapter(ad, cur), ++at) {
        if (at % (int32_t)gridDim.y != (int32_t)blockIdx.y) continue;
        const int64_t pair = (int64_t)cur * (a.e.E + a.e.shared) + t.expert;
        Op fo;
        fo.start((BWD ? a.l.b : a.l.a) + pair * rank * L, rank, L);
        no.init(x, t.rows, L, L);
#pragma unroll
        for (int j = 0; j < kNL; ++j)  // rows of other adapters: zeros, and not read
            no.voff[j] = ads[j * 8 + lane / 8] == cur ? no.voff[j] : kOutside;
        auto load = [&](int32_t s, int slot) {
            const int32_t l0 = uniform((s * kDownWaves + w) * kStepL);
#pragma unroll
            for (int j = 0; j < kFL; ++j) fo.load(mine + slot * kStep, l0, j);
#pragma unroll
            for (int j = 0; j < kNL; ++j) no.load(mine + slot * kStep + P * kStepL, l0, j);
        };
        f32x4 acc[KP][KN] = {};
#pragma unroll
        for (int s = 0; s < kRing - 1; ++s) load(s, s);
        const int32_t turns = (steps - w + kDownWaves - 1) / kDownWaves;
        int32_t slot = 0;
        for (int32_t s = 0; s < turns; ++s) {
            load(s + kRing - 1, slot == 0 ? kRing - 1 : slot - 1);
            // this step has landed when only the later ones are outstanding
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kRing - 1) * (kFL + kNL)) : "memory");
            const uint16_t *const lf = mine + slot * kStep, *const ln = lf + P * kStepL;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                bf16x8 fv[KP], nv[KN];
#pragma unroll
                for (int k = 0; k < KP; ++k) fv[k] = Op::fragment(lf, k * 16, kk);
#pragma unroll
                for (int n = 0; n < KN; ++n) nv[n] = RowsOperand<NT, 1>::fragment(ln, n * 16, kk);
#pragma unroll
                for (int k = 0; k < KP; ++k)
#pragma unroll
                    for (int n = 0; n < KN; ++n) acc[k][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv[k], nv[n], acc[k][n], 0, 0, 0);
            }
            // what was read is in registers before the next step's loads overwrite it
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            slot = slot == kRing - 1 ? 0 : slot + 1;
        }
        // no load of any wave may land among the parts
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int k = 0; k < KP; ++k)
#pragma unroll
            for (int n = 0; n < KN; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[(w * NT + n * 16 + i) * (P + 1) + k * 16 + q * 4 + j] = acc[k][n][j];
        __syncthreads();
        const float s = a.l.scale != nullptr ? a.l.scale[cur] : 1.0f;
        for (int at = threadIdx.x; at < NT * P; at += kDownThreads) {
            const int r = at / P, p = at % P;
            if (p >= rank || ads[r] != cur) continue;
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kDownWaves; ++k) v += part[(k * NT + r) * (P + 1) + p];
            u[(t.first + r) * rank + p] = s * v;
        }
        __syncthreads();
    }
    if (blockIdx.y != 0) return;
    // rows without an adapter: zeros
    for (int at = threadIdx.x; at < NT * P; at += kDownThreads) {
        const int r = at / P, p = at % P;
        if (p < rank && r < t.rows && ads[r] < 0) u[(t.first + r) * rank + p] = 0.0f;
    }
}

// Tiles of 64 rows, which read an adapter's weights a quarter as often, where they
// are enough to fill the CUs; of 16, shared by their adapters' workgroups, for less.
template <bool BWD, int P, int NT>
hipError_t down(const BlockArgs& a, float* u, hipStream_t stream) {
    const int64_t tiles = max_row_tiles(a.e, NT), blocks = (tiles + 7) / 8 * 8;
    if (blocks == 0) return hipSuccess;
    const int share = tiles <= 2 * kCus ? (a.l.n < NT ? a.l.n : NT) : 1;
    if (const hipError_t e = check_grid(blocks, kDownThreads)) return e;
    hipLaunchKernelGGL((k_lora_down<BWD, P, NT>), dim3((unsigned)blocks, (unsigned)share), dim3(kDownThreads), 0, stream, a, u);
    return hipGetLastError();
}

template <bool BWD>
hipError_t down_by_size(const BlockArgs& a, float* u, hipStream_t stream) {
    const bool many = a.e.slots >= 64 * kCus;
    if (a.l.rank <= 16) return many ? down<BWD, 16, 64>(a, u, stream) : down<BWD, 16, 16>(a, u, stream);
    if (a.l.rank <= 32) return many ? down<BWD, 32, 64>(a, u, stream) : down<BWD, 32, 16>(a, u, stream);
    if (a.l.rank <= 64) return many ? down<BWD, 64, 64>(a, u, stream) : down<BWD, 64, 16>(a, u, stream);
    return down<BWD, 128, 16>(a, u, stream);
}

constexpr int kGradThreads = 256, kGradRows = 64, kGradCols = 256;  // rows a step, columns of a tile
constexpr int kLook = 4, kList = kLook * kGradThreads;               // rows that a thread, and all, look through at a time

// Gradients of one adapter's weights of one expert, columns c0 on: sum over the
// rows r of the expert whose tokens have the adapter of v[r]^T d[r], d = x (of
// width in; result [rank, in]) or gy (out; result [out, rank]), v = gu or u.  The
// rows are picked out in order, 64 a step; d's go through registers to LDS.  No
// workgroup shares a result with another: the order of the sums is the rows'.
// 32 experts, 4 adapters of rank 16, 32 768 rows of 2048: 41 to 46 us, bound by the
// rows' reads (134 MB, 3.0 TB/s; 88 us with a step's loads behind the one before).
// Every adapter's workgroups look through all rows of their expert.
template <int KP, bool OUT>
__global__ __launch_bounds__(kGradThreads, KP <= 2 ? 3 : KP == 4 ? 2 : 1)  // as many workgroups as LDS holds
void k_lora_bwd_w(BlockArgs a, const float* v, void* out, int32_t ctiles) {
    using XOp = ColsOperand<kGradCols, 4>;
    // v as three bf16 whose sum it is (24 significant bits): the sums over the rows are
    // as good as 32-bit products' would be
    constexpr int P = KP * 16, kParts = 3;
    using VOp = ColsOperand<P, 4>;
    __shared__ __align__(1024) uint16_t xs[kGradRows * kGradCols], vs[kParts][kGradRows * P];
    __shared__ int32_t list[kList + kGradRows], counts[5];
    const int lane = threadIdx.x & (kWave - 1), w = uniform((int32_t)(threadIdx.x / kWave)), i = lane % 16, q = lane / 16;
    const int32_t EX = a.e.E + a.e.shared, rank = a.l.rank, C = OUT ? a.e.on : a.e.in;
    const int32_t ct = blockIdx.x % ctiles, pair = blockIdx.x / ctiles, ad = pair / EX, expert = pair % EX, c0 = ct * kGradCols;
    const int32_t g = expert < a.e.E ? expert / a.e.E_loc * a.e.G + a.e.shared + expert % a.e.E_loc : a.e.src_seg * a.e.G;
    const GroupRows rows = group_rows(a.e, g);
    const uint16_t* const d = (OUT ? a.e.gy : a.e.x) + rows.first * C + c0;
    const float* const vv = v + rows.first * rank;
    f32x4 acc[4][KP];
    constexpr int kX = kGradRows * kGradCols / 8 / kGradThreads;  // 16-byte pieces of d that a thread copies a step
    auto sums = [&](auto again) {
        constexpr bool kAgain = decltype(again)::value;
#pragma unroll
        for (int f = 0; f < 4; ++f)
#pragma unroll
            for (int k = 0; k < KP; ++k) acc[f][k] = f32x4{};
        int32_t have = 0;  // rows in the list
        for (int32_t r0 = 0; r0 < rows.rows || have > 0; r0 += kList) {
            // append the next rows' matches
            int32_t of[kLook];
            row_adapters<kLook>(
                a, [&](int k) { return rows.first + min(r0 + k * kGradThreads + (int32_t)threadIdx.x, rows.rows - 1); },
                [&](int k) { return r0 + k * kGradThreads + (int32_t)threadIdx.x < rows.rows; }, of);
#pragma unroll
            for (int k = 0; k < kLook; ++k) {
                const bool mine = of[k] == ad;
                const uint64_t m = __builtin_amdgcn_ballot_w64(mine);
                if (lane == 0) counts[w] = __popcll(m);
                __syncthreads();
                int32_t at = have;
                for (int o = 0; o < 4; ++o) {
                    if (o == w && mine) list[at + lanes_below(m)] = r0 + k * kGradThreads + (int32_t)threadIdx.x;
                    at += counts[o];
                }
                have = at;
                __syncthreads();
            }
            const bool last = r0 + kList >= rows.rows;
            const int32_t turns = last ? (have + kGradRows - 1) / kGradRows : have / kGradRows, done = turns * kGradRows;
            // a step's rows on their way to LDS, while the step before is multiplied
            v4u xr[kX];
            f32x4 vr[KP];
            auto fetch = [&](int32_t turn) {
                const int32_t from = turn * kGradRows, n = min(kGradRows, have - from);
                // d: 64 rows of 32 chunks of 8 values
#pragma unroll
                for (int k = 0; k < kX; ++k) {
                    const int at = k * kGradThreads + threadIdx.x, r = at / 32, c = at % 32;
                    xr[k] = v4u{};
                    if (r < n && c0 + c * 8 < C) xr[k] = *reinterpret_cast<const v4u*>(d + (int64_t)list[from + r] * C + c * 8);
                }
                // v: 64 rows of KP * 4 chunks of 4 values
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    const int at = k * kGradThreads + threadIdx.x, r = at / (KP * 4), p = at % (KP * 4) * 4;
                    vr[k] = f32x4{};
                    if (r < n && p < rank) vr[k] = *reinterpret_cast<const f32x4*>(vv + (int64_t)list[from + r] * rank + p);
                }
            };
            if (turns > 0) fetch(0);
            for (int32_t turn = 0; turn < turns; ++turn) {
#pragma unroll
                for (int k = 0; k < kX; ++k) {
                    const int at = k * kGradThreads + threadIdx.x, r = at / 32, c = at % 32;
                    *reinterpret_cast<v4u*>(xs + r * kGradCols + (((c / 2) ^ XOp::swizzle(r)) * 2 + c % 2) * 8) = xr[k];
                }
#pragma unroll
                for (int k = 0; k < KP; ++k) {
                    const int at = k * kGradThreads + threadIdx.x, r = at / (KP * 4), c = at % (KP * 4);
                    f32x4 left = vr[k];
#pragma unroll
                    for (int o = 0; o < kParts; ++o) {
                        const v2u w = {pack_bf16x2(left[0], left[1]), pack_bf16x2(left[2], left[3])};
                        *reinterpret_cast<v2u*>(vs[o] + r * P + ((c / 4) ^ VOp::swizzle(r)) * 16 + c % 4 * 4) = w;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float h = j % 2 ? bf16_hi(w[j / 2]) : bf16_lo(w[j / 2]);
                            left[j] = __builtin_isinf(h) ? 0.0f : left[j] - h;  // an infinity leaves nothing
                        }
                    }
                }
                lds_barrier();
                if (turn + 1 < turns) fetch(turn + 1);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    bf16x8 xf[4];
#pragma unroll
                    for (int f = 0; f < 4; ++f) xf[f] = XOp::fragment(xs, w * 64 + f * 16, kk);
#pragma unroll
                    for (int k = 0; k < kParts * KP; ++k) {
                        const bf16x8 vf = VOp::fragment(vs[k / KP], k % KP * 16, kk);
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            if (kAgain && k == KP) xf[f] = only_finite(xf[f]);
                            f32x4& s = acc[f][k % KP];
                            s = OUT ? __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, xf[f], s, 0, 0, 0)
                                    : __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[f], vf, s, 0, 0, 0);
                        }
                    }
                }
                lds_barrier();
            }
            // what is left of the list moves to its front
            const int32_t left = max(have - done, 0);
            int32_t keep = 0;
            if ((int32_t)threadIdx.x < left) keep = list[done + threadIdx.x];
            __syncthreads();
            if ((int32_t)threadIdx.x < left) list[threadIdx.x] = keep;
            have = left;
            __syncthreads();
        }
    };
    sums(std::false_type{});
    // Where a sum is NaN all are made once more, with the infinities of d times the first part
    // of v alone: times the other two they may be NaN where the sum is infinite.
    bool nan = false;
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int k = 0; k < KP; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) nan |= acc[f][k][j] != acc[f][k][j];
    const uint64_t any = __builtin_amdgcn_ballot_w64(nan);
    if (lane == 0) counts[w] = any != 0;
    __syncthreads();
    const bool again = uniform(counts[0] | counts[1] | counts[2] | counts[3]) != 0;
    __syncthreads();
    if (again) sums(std::true_type{});
    // acc[f][k][j]: column c = c0 + 64 w + 16 f + .., value p = 16 k + .. of the rank;
    // the four of a lane lie along the result's rows
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
        for (int k = 0; k < KP; ++k) {
            const int32_t c = c0 + w * 64 + f * 16 + (OUT ? i : q * 4), p = k * 16 + (OUT ? q * 4 : i);
            if (c >= C || p >= rank) continue;
            const int64_t at = (int64_t)pair * rank * C + (OUT ? (int64_t)c * rank + p : (int64_t)p * C + c);
            const f32x4 s = acc[f][k];
            if (a.e.grad_type == EP_GRAD_BF16) {
                *reinterpret_cast<v2u*>(static_cast<uint16_t*>(out) + at) = v2u{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
            } else {
                f32x4* const o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + at);
                *o = a.e.grad_type == EP_GRAD_F32_ADD ? *o + s : s;
            }
        }
}

int32_t grad_tiles(int32_t columns) { return (columns + kGradCols - 1) / kGradCols; }
int64_t grad_blocks(const BlockArgs& a, int32_t columns) {
    return (int64_t)a.l.n * (a.e.E + a.e.shared) * grad_tiles(columns);
}

template <int KP, bool OUT>
hipError_t bwd_w(const BlockArgs& a, const float* v, void* out, hipStream_t stream) {
    const int32_t ctiles = grad_tiles(OUT ? a.e.on : a.e.in);
    const int64_t blocks = grad_blocks(a, OUT ? a.e.on : a.e.in);
    hipLaunchKernelGGL((k_lora_bwd_w<KP, OUT>), dim3((unsigned)blocks), dim3(kGradThreads), 0, stream, a, v, out,
                       ctiles);
    return hipGetLastError();
}

template <bool OUT>
hipError_t bwd_w_by_rank(const BlockArgs& a, const float* v, void* out, hipStream_t stream) {
    if (a.l.rank <= 16) return bwd_w<1, OUT>(a, v, out, stream);
    if (a.l.rank <= 32) return bwd_w<2, OUT>(a, v, out, stream);
    if (a.l.rank <= 64) return bwd_w<4, OUT>(a, v, out, stream);
    return bwd_w<8, OUT>(a, v, out, stream);
}

}  // namespace

hipError_t launch_gemm_lora(const BlockArgs& a, hipStream_t stream) { return product<kForward>(a, stream); }
hipError_t launch_gemm_bwd_x_lora(const BlockArgs& a, hipStream_t stream) { return product<kInputGrad>(a, stream); }
hipError_t launch_lora_down(const BlockArgs& a, float* u, hipStream_t stream) { return down_by_size<false>(a, u, stream); }
hipError_t launch_lora_bwd_u(const BlockArgs& a, float* u, hipStream_t stream) { return down_by_size<true>(a, u, stream); }
hipError_t check_lora_bwd_w(const BlockArgs& a) {
    const hipError_t e = check_grid(grad_blocks(a, a.e.in), kGradThreads);
    return e != hipSuccess ? e : check_grid(grad_blocks(a, a.e.on), kGradThreads);
}
hipError_t launch_lora_bwd_w(const BlockArgs& a, const float* grad_u, void* grad_a, void* grad_b, hipStream_t stream) {
    if (const hipError_t e = bwd_w_by_rank<false>(a, grad_u, grad_a, stream)) return e;
    return bwd_w_by_rank<true>(a, a.u, grad_b, stream);
}

}  // namespace epx
