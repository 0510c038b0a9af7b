// What the experts' product kernels share: which rows belong to which
// expert, and the tiles of a launch.
#pragma once

#include "epx_device.h"

namespace epx {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

#define EPX_LDS __attribute__((address_space(3)))

[[maybe_unused]] constexpr int kBufferWord3 = 0x00020000;  // buffer descriptor word 3: 32-bit data, raw addressing
constexpr int kOutside = 0x7FFFFFF0;                       // an offset past every descriptor's end: loads zeros

// BYTES (16, 4 or 1) a lane from offset voff of a buffer of `bytes` bytes to
// LDS: lane l's 16 at lds + 16 l, its 4 at lds + 4 l, its 1 as a word at
// lds + 4 l; zeros for words past the buffer's end.  base, bytes and lds are the
// same in all lanes.  The instruction's scalar offset stays 0: the range check
// does not count it.  Written out, because the compiler waits for every load in
// flight (vmcnt 0) before any LDS read that follows its builtin.
// Nothing waits for this load by itself: whoever reads the LDS bytes waits for
// vmcnt first.  The compiler puts no wait states before an instruction in here:
// an SGPR that a vector instruction wrote (uniform() is one) may be read by a
// memory instruction 5 wait states later at the earliest, m0, which holds the
// LDS address, 1 later.  The write of m0 is one, s_nop 3 four.  m0 is declared as
// written: the compiler warns that it is reserved, but otherwise takes a value of
// its own there for unchanged.
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const void* base, int32_t bytes, const void* lds, int32_t voff) {
#ifdef __HIP_DEVICE_COMPILE__
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const i32x4 rs = {(int32_t)uniform((uint32_t)p), (int32_t)uniform((uint32_t)(p >> 32) & 0xFFFFu), uniform(bytes),
                      kBufferWord3};
    const uint32_t to = uniform((uint32_t)(uintptr_t)(EPX_LDS const void*)lds);
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(voff),
                     "s"(rs)
                     : "memory", "m0");
    else if constexpr (BYTES == 4)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to), "v"(voff),
                     "s"(rs)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_ubyte %1, %2, 0 offen lds" ::"s"(to), "v"(voff),
                     "s"(rs)
                     : "memory", "m0");
#endif
}
#pragma clang diagnostic pop

// Results of matrix instructions kept in accumulation registers from here on.
__device__ __forceinline__ void in_agprs(f32x4& v) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("" : "+a"(v));
#endif
}

// A group's rows in the receive buffers, whatever the layout holds: [first,
// first + rows) lies inside [0, R).
struct GroupRows {
    int64_t first;
    int32_t rows;
};

__device__ __forceinline__ GroupRows group_rows(const ExpertArgs& a, int32_t g) {
    const int32_t s = g / a.G, gl = g - s * a.G;
    const int64_t off = a.row_offsets[s * (a.G + 1) + gl];
    int64_t n = a.counts[g];
    if (a.C > 0) n = min(n, (int64_t)a.C - off);  // rows past the capacity were dropped
    const int64_t first = (int64_t)a.seg_base[s] + off;
    n = first < 0 || first > a.R ? 0 : min(n, a.R - first);
    return {first, n > 0 ? (int32_t)n : 0};
}

// The expert whose weights group g uses; the shared expert is the last.
__device__ __forceinline__ int32_t group_expert(const ExpertArgs& a, int32_t g) {
    const int32_t s = g / a.G, gl = g - s * a.G;
    return gl < a.shared ? a.E : s * a.E_loc + gl - a.shared;
}

// A launch of `blocks` workgroups fits one grid (a count of work-items in 32
// bits); the entry points answer EP_EINVAL to the error.
inline hipError_t check_grid(int64_t blocks, int threads) {
    return blocks * threads > 0xFFFFFFFFll ? hipErrorInvalidConfiguration : hipSuccess;
}

// Most row tiles of BM rows that the groups can need: every group with rows
// has at most one part tile.
inline int64_t max_row_tiles(const ExpertArgs& a, int bm) {
    const int64_t groups = a.slots < a.E + a.shared ? a.slots : a.E + a.shared;
    return a.slots / bm + groups;
}

struct RowTile {
    int32_t expert;  // -1: no such tile
    int32_t rows;    // rows of the tile, 1..BM
    int64_t first;   // its first receive row
};

// The row tile that pick(number of row tiles, other) asks for, groups in
// order.  Every thread of the workgroup (THREADS of them) takes part; lds
// holds THREADS / 64 + 3 words.  Each thread counts the tiles of a run of
// groups; an exclusive sum over the threads gives the run that holds the tile.
template <int THREADS, int BM, typename Pick>
__device__ __forceinline__ RowTile find_row_tile(const ExpertArgs& a, int32_t* lds, Pick pick, int32_t& other) {
    constexpr int kWaves = THREADS / kWave;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), w = tid / kWave;
    const int per = (a.NG + THREADS - 1) / THREADS;
    const int g0 = tid * per, g1 = min(g0 + per, a.NG);
    int32_t mine = 0;
    for (int g = g0; g < g1; ++g) mine += (group_rows(a, g).rows + BM - 1) / BM;
    const int32_t upto = wave_inclusive_sum(mine);
    if (lane == kWave - 1) lds[w] = upto;
    if (tid == 0) lds[kWaves] = -1;
    __syncthreads();
    int32_t base = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        if (i < w) base += lds[i];
        total += lds[i];
    }
    const int32_t want = pick(uniform(total), other);
    int32_t before = base + upto - mine;
    if (want >= before && want < before + mine) {
        for (int g = g0; g < g1; ++g) {
            const GroupRows r = group_rows(a, g);
            const int32_t n = (r.rows + BM - 1) / BM;
            if (want < before + n) {
                const int32_t skip = (want - before) * BM;
                lds[kWaves] = group_expert(a, g);
                lds[kWaves + 1] = min(BM, r.rows - skip);
                lds[kWaves + 2] = (int32_t)(r.first + skip);
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    RowTile t;
    t.expert = uniform(lds[kWaves]);
    t.rows = uniform(lds[kWaves + 1]);
    t.first = uniform(lds[kWaves + 2]);
    return t;
}

constexpr int32_t kNoTile = INT32_MAX;

// The tile of this workgroup among row_tiles x ftiles: its row tile (kNoTile:
// none) and, in f, its feature tile.  Workgroups are handed to the 8 XCDs in
// turn: XCD x takes the x-th eighth of the tiles, in blocks of 4 row tiles by
// all feature tiles, so that the workgroups that run together on it share
// operands in its L2.
__device__ __forceinline__ int32_t xcd_tile(int32_t row_tiles, int32_t ftiles, int32_t& f) {
    const int32_t total = row_tiles * ftiles, per = (total + 7) / 8;
    const int32_t b = (int32_t)(blockIdx.x / 8), at = (int32_t)(blockIdx.x % 8) * per + b;
    f = 0;
    if (b >= per || at >= total) return kNoTile;
    const int32_t block = at / (4 * ftiles), r0 = block * 4, height = min(4, row_tiles - r0);
    const int32_t in = at - block * 4 * ftiles;
    f = uniform(in / height);
    return uniform(r0 + in % height);
}

// As xcd_tile for the weights' gradients, whose tiles cost as much as their
// experts have rows: the XCDs take blocks of 2 row tiles by all feature tiles
// in turn, so that no XCD gets all the busy experts (with an eighth each,
// experts of 400 to 2200 rows left seven XCDs waiting for the first).
__device__ __forceinline__ int32_t xcd_tile_in_turn(int32_t row_tiles, int32_t ftiles, int32_t& f) {
    const int32_t b = (int32_t)(blockIdx.x / 8), unit = 2 * ftiles;
    const int32_t r0 = (b / unit * 8 + (int32_t)(blockIdx.x % 8)) * 2, height = min(2, row_tiles - r0);
    f = 0;
    if (height <= 0) return kNoTile;
    const int32_t in = b % unit;
    if (in >= height * ftiles) return kNoTile;
    f = uniform(in / height);
    return uniform(r0 + in % height);
}

}  // namespace epx
