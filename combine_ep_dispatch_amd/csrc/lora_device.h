// What the kernels with low-rank adapters share: which adapter a row has, and
// adding B u (or A^T u) to a wave's results in registers.
#pragma once

#include "expert_device.h"

namespace epx {

// The adapter of receive row r, -1 for none, whatever the layout and the ids hold.
__device__ __forceinline__ int32_t row_adapter(const BlockArgs& a, int64_t r) {
    const int32_t t = a.src_info[2 * r];
    if (t < 0 || t >= a.T) return -1;
    const int32_t ad = a.l.token_adapter[t];
    return ad < 0 || ad >= a.l.n ? -1 : ad;
}

// As row_adapter for COUNT rows of this lane, row(n) each (any row of the buffer), -1
// where on(n) is false.  All loads go out together, twice.
template <int COUNT, typename Row, typename On>
__device__ __forceinline__ void row_adapters(const BlockArgs& a, Row row, On on, int32_t (&ad)[COUNT]) {
    int32_t t[COUNT];
#pragma unroll
    for (int n = 0; n < COUNT; ++n) t[n] = a.src_info[2 * row(n)];
#pragma unroll
    for (int n = 0; n < COUNT; ++n) ad[n] = a.l.token_adapter[t[n] < 0 || t[n] >= a.T ? 0 : t[n]];
#pragma unroll
    for (int n = 0; n < COUNT; ++n) ad[n] = !on(n) || t[n] < 0 || t[n] >= a.T || ad[n] < 0 || ad[n] >= a.l.n ? -1 : ad[n];
}

// The smallest of the adapters `ad` (COUNT of each of the 16 lanes i; the
// quarters of the wave hold the same) past `last`, kNoAdapter if there is none.
constexpr int32_t kNoAdapter = INT32_MAX;
template <int COUNT>
__device__ __forceinline__ int32_t next_adapter(const int32_t (&ad)[COUNT], int32_t last) {
    int32_t v = kNoAdapter;
#pragma unroll
    for (int n = 0; n < COUNT; ++n) v = ad[n] > last ? min(v, ad[n]) : v;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) v = min(v, __shfl_xor(v, o, kWave));
    return uniform(v);
}

// Eight values as bf16: rounded, or, with `rest`, what the rounding left.  Both
// together have 16 significant bits, so that products with u are off by 2^-16 of
// their terms, next to the result's 2^-8; one bf16 alone would add a rounding of its
// own where the adapters make most of the result.  An infinity leaves nothing (not NaN).
__device__ __forceinline__ bf16x8 split8(const f32x4 a, const f32x4 b, bool rest) {
    v4u o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float x = j < 2 ? a[2 * j] : b[2 * j - 4], y = j < 2 ? a[2 * j + 1] : b[2 * j - 3];
        const uint32_t w = pack_bf16x2(x, y);
        const float rx = __builtin_isinf(bf16_lo(w)) ? 0.0f : x - bf16_lo(w);
        const float ry = __builtin_isinf(bf16_hi(w)) ? 0.0f : y - bf16_hi(w);
        o[j] = rest ? pack_bf16x2(rx, ry) : w;
    }
    return __builtin_bit_cast(bf16x8, o);
}

// Whether one of the values is an infinity or NaN: all exponent bits set.
__device__ __forceinline__ bool not_finite(const bf16x8 v) {
    const v4u w = __builtin_bit_cast(v4u, v);
    uint32_t carry = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) carry |= (w[j] & 0x7F807F80u) + 0x00800080u;
    return (carry & 0x80008000u) != 0;
}

// v with zeros in place of infinities and NaN.  Where a value goes into products in parts,
// the others than the first meet only finite factors: an infinity times the first part
// is infinite already, and times a rest of 0, or of the other sign, it would make that NaN.
__device__ __forceinline__ bf16x8 only_finite(const bf16x8 v) {
    v4u w = __builtin_bit_cast(v4u, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t carry = (w[j] & 0x7F807F80u) + 0x00800080u;
        w[j] &= ~((carry >> 15 & 0x00010001u) * 0xFFFFu);
    }
    return __builtin_bit_cast(bf16x8, w);
}

// acc[f][n] += the adapters' part of a wave's results: 16 features a fragment f
// by 16 rows a fragment n, summed over u rounded to bf16 and then over what the
// rounding left (2 rank values), 32 of them a step.  weights(f, ad, c): this lane's 8
// values [8 c, 8 c + 8) of the rank of its feature of fragment f.  Every adapter that
// one of the rows has is multiplied with all of them, with u zero in the rows of
// others.  Steps whose weights hold an infinity or NaN come afterwards, and are added
// to the adapter's own rows alone: nothing that an adapter or another row holds
// reaches a row that does not use it.  There what the rounding left meets no infinity.  Bound by the loads' latency, some 0.8 us for each
// adapter and step of a tile; loads a step ahead gained nothing.  (Selecting in every step moves all results
// from accumulation to vector registers and back: 32 experts of 4096 x 7168, 4096
// tokens of 8, rank 32, 2010 us.)
template <int KF, int KN, typename Weights>
__device__ __forceinline__ void add_adapters(const BlockArgs& a, int64_t first, int32_t rows, int32_t wn, Weights weights,
                                             f32x4 (&acc)[KF][KN]) {
    const int lane = threadIdx.x & (kWave - 1), i = lane % 16, q = lane / 16;
    int32_t ad[KN];
    row_adapters<KN>(
        a, [&](int n) { return first + min(wn + n * 16 + i, rows - 1); }, [&](int n) { return wn + n * 16 + i < rows; }, ad);
    const int32_t chunks = uniform(a.l.rank / 4);  // of 8 values: the rounded ones, then the rests
    const float* const u = a.u + (first + wn + i) * a.l.rank;
    auto load_u = [&](f32x4 (&v)[KN][2], int32_t cur, int32_t c) {
        const int32_t at = (c >= chunks / 2 ? c - chunks / 2 : c) * 8;
#pragma unroll
        for (int n = 0; n < KN; ++n) {
            v[n][0] = v[n][1] = f32x4{};
            if (c < chunks && ad[n] == cur) {
                const f32x4* const p = reinterpret_cast<const f32x4*>(u + n * 16 * a.l.rank + at);
                v[n][0] = p[0];
                v[n][1] = p[1];
            }
        }
    };
    auto load_w = [&](int f, int32_t cur, int32_t c) {
        bf16x8 w = {};
        if (c < chunks) w = weights(f, cur, c < chunks / 2 ? c : c - chunks / 2);
        return w;
    };
    int32_t any_bad = 0;
#pragma unroll
    for (int f = 0; f < KF; ++f)
#pragma unroll
        for (int n = 0; n < KN; ++n) in_agprs(acc[f][n]);
    for (int32_t cur = next_adapter(ad, -1); cur != kNoAdapter; cur = next_adapter(ad, cur)) {
        for (int32_t c0 = 0; c0 < chunks; c0 += 4) {
            bf16x8 wv[KF];
            f32x4 uv[KN][2];
#pragma unroll
            for (int f = 0; f < KF; ++f) wv[f] = load_w(f, cur, c0 + q);
            load_u(uv, cur, c0 + q);
            bool bad = false;
#pragma unroll
            for (int f = 0; f < KF; ++f) bad |= not_finite(wv[f]);
            if (__builtin_amdgcn_ballot_w64(bad) != 0) {
                any_bad = 1;
                continue;
            }
#pragma unroll
            for (int n = 0; n < KN; ++n) {
                if (__builtin_amdgcn_ballot_w64(ad[n] == cur) == 0) continue;
                const bf16x8 v = split8(uv[n][0], uv[n][1], c0 + q >= chunks / 2);
#pragma unroll
                for (int f = 0; f < KF; ++f) {
                    acc[f][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[f], v, acc[f][n], 0, 0, 0);
                    in_agprs(acc[f][n]);
                }
            }
        }
    }
    if (uniform(any_bad) == 0) return;
    // Few fragments of features at a time: the selections need their results in
    // vector registers, and all 256 at once would not fit beside the operands.
    constexpr int kBlock = KF < 2 ? KF : 2;
#pragma unroll
    for (int f0 = 0; f0 < KF; f0 += kBlock) {
        for (int32_t cur = next_adapter(ad, -1); cur != kNoAdapter; cur = next_adapter(ad, cur)) {
            for (int32_t c0 = 0; c0 < chunks; c0 += 4) {
                bool bad = false;
#pragma unroll
                for (int f = 0; f < KF; ++f) bad |= not_finite(load_w(f, cur, c0 + q));
                if (__builtin_amdgcn_ballot_w64(bad) == 0) continue;
                bf16x8 wv[kBlock];
                f32x4 uv[KN][2];
                load_u(uv, cur, c0 + q);
#pragma unroll
                for (int f = 0; f < kBlock; ++f) {
                    wv[f] = load_w(f0 + f, cur, c0 + q);
                    if (c0 + q >= chunks / 2) wv[f] = only_finite(wv[f]);
                }
#pragma unroll
                for (int n = 0; n < KN; ++n) {
                    const bf16x8 v = split8(uv[n][0], uv[n][1], c0 + q >= chunks / 2);
#pragma unroll
                    for (int f = 0; f < kBlock; ++f) {
                        const f32x4 s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[f], v, acc[f0 + f][n], 0, 0, 0);
                        acc[f0 + f][n] = ad[n] == cur ? s : acc[f0 + f][n];
                    }
                }
            }
        }
        // done with: into accumulation registers, out of the next block's way
#pragma unroll
        for (int f = 0; f < kBlock; ++f)
#pragma unroll
            for (int n = 0; n < KN; ++n) in_agprs(acc[f0 + f][n]);
    }
}

}  // namespace epx
