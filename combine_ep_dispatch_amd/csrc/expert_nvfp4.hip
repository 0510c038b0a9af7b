// The experts' product over 4-bit weights: y[r, n] = rowscale[e, n] *
// sum_h x[r, h] e2m1(code) e4m3(scale).
//
// Tiles of features by rows; the codes, their block scales and the rows of L
// values at a time go to LDS by the loads themselves, several steps ahead;
// each wave turns the codes of its own features into bf16 operands of the
// matrix instruction (a code times its block scale has at most 2 + 4
// significant bits: exact in bf16) and multiplies them with all rows of the
// tile.  Lane (i, q) of a wave takes feature i and 32 values, two whole blocks,
// of every 128 of the step; which value of a step is which does not matter to
// the sum as long as the rows are read in the same order.
//
// What bounds it: with one row an expert the latency of the first loads and
// HBM (8 experts of 4096 x 7168, 132 MB: 30 us, 4.4 TB/s; loads alone 26, all
// but the loads 25); at 8 rows HBM and the conversions (65 experts, 1.09 GB:
// 256 us, 4.3 TB/s; loads alone 242, of which the 4-byte loads of the scales
// are 55, all but the loads 143; vector instructions for 68 % of the cycles); at
// 122 rows the conversions, two instructions a weight and row tile, and the matrix
// instructions of tiles that 122 rows fill three quarters of (32 experts of 7168 x
// 2048: 197 us, 581 TFLOP/s; loads alone 137, all but the loads 159; the matrix
// pipes are busy for 33 % of the cycles).  32 experts of 4096 x 7168 with 1024
// rows each: 1981 us, 971 TFLOP/s.  Few tiles are slow: 4 experts of 512 x 2048
// with 64 rows are 8 workgroups with work, 32 us.  Measured instead: scales as 64-byte windows
// load in 187 us instead of 242, but two of them in LDS cost a workgroup a CU
// (254-274 us in all), and one, taken to registers for four steps, gains nothing
// (262, and 36 us instead of 32 for one row); 4 waves of 64 features by 128 rows
// for prompts, 233 us instead of 194; half the products of tiles that are at most
// half full, 193.
#include "nvfp4_tile.h"

namespace epx {
namespace {

// WORDS: the block scales travel as words.
template <int NT, int FW, int WAVES, int L, int BUFS, bool WORDS>
__global__ __launch_bounds__(WAVES * kWave) void k_nvfp4(ExpertArgs a, int32_t ftiles) {
    using Tile = Nvfp4Tile<NT, FW, WAVES, L, BUFS, WORDS, false>;
    __shared__ __align__(1024) uint8_t lds[BUFS * Tile::kBuffer];
    __shared__ int32_t scan[16];
    Tile::run(a, ftiles, lds, scan, [&](const RowTile& t, int32_t f0, int64_t row0, const f32x4 (&acc)[FW / 16][NT / 16]) {
        const int lane = threadIdx.x & (kWave - 1), i = lane % 16, q = lane / 16;
        // acc[g][n][j]: feature f0 + 16 g + 4 q + j, row 16 n + i
#pragma unroll
        for (int g = 0; g < FW / 16; ++g) {
            const int32_t fe = g * 16 + q * 4;
            if (f0 + fe >= a.on) continue;
            const v2u rs = *reinterpret_cast<const v2u*>(a.rowscale + row0 + fe);
#pragma unroll
            for (int n = 0; n < NT / 16; ++n) {
                const int32_t r = n * 16 + i;
                if (r >= t.rows) continue;
                const v2u o = {pack_bf16x2(acc[g][n][0] * bf16_lo(rs.x), acc[g][n][1] * bf16_hi(rs.x)),
                               pack_bf16x2(acc[g][n][2] * bf16_lo(rs.y), acc[g][n][3] * bf16_hi(rs.y))};
                *reinterpret_cast<v2u*>(static_cast<uint16_t*>(a.out) + (t.first + r) * a.on + f0 + fe) = o;
            }
        }
    });
}

// BYTES: steps that LDS holds where the scales travel as bytes.
template <int NT, int FW, int WAVES, int L, int BUFS, int BYTES>
hipError_t nvfp4(const ExpertArgs& a, hipStream_t stream) {
    constexpr int kF = FW * WAVES;
    const int32_t ftiles = (a.on + kF - 1) / kF;
    const int64_t tiles = max_row_tiles(a, NT) * ftiles, blocks = (tiles + 7) / 8 * 8;
    if (tiles == 0) return hipSuccess;
    if (const hipError_t e = check_grid(blocks, WAVES * kWave)) return e;
    if (a.in % 64 == 0)
        hipLaunchKernelGGL((k_nvfp4<NT, FW, WAVES, L, BUFS, true>), dim3((unsigned)blocks), dim3(WAVES * kWave), 0,
                           stream, a, ftiles);
    else
        hipLaunchKernelGGL((k_nvfp4<NT, FW, WAVES, L, BYTES, false>), dim3((unsigned)blocks), dim3(WAVES * kWave), 0,
                           stream, a, ftiles);
    return hipGetLastError();
}

}  // namespace

// By the rows a group has on average.  Measured over 64 experts of 4096 x 7168,
// us at 8, 12, 16, 24, 32 and 64 rows a group:
//   16-row tiles    257  286  343  444  516  854
//   32              289  301  307  333  424  659
//   64              334  339  347  351  365  505
//   128             424  436  440  446  450  482
hipError_t launch_expert_gemm_nvfp4(const ExpertArgs& a, hipStream_t stream) {
    const int64_t groups = a.slots < a.E + a.shared ? a.slots : a.E + a.shared;
    if (groups == 0) return hipSuccess;
    const int64_t mean = a.slots / groups;
    if (mean <= 13) return nvfp4<16, 16, 4, 256, 3, 3>(a, stream);
    if (mean <= 26) return nvfp4<32, 16, 4, 256, 2, 2>(a, stream);
    if (mean <= 56) return nvfp4<64, 32, 8, 128, 2, 2>(a, stream);
    return nvfp4<128, 32, 8, 128, 3, 2>(a, stream);
}

}  // namespace epx
