// fp8_quantize.hip -- matrices to 8-bit floats with a scale for each block.
//
//   s = max(amax |x| / top, 2^-126) over the block (`pow2`: the next power of
//   two), q = fp8(x * (1 / s)); blocks of 1 x 128 ("row") or 128 x 128
//   ("tile"), and the same of the transposed matrix.
//
// All of it is bound by memory: each x is read once and gives one byte, or
// two with the transposed copy.
#include "fp8_common.h"

namespace pg {

namespace {

// Rows only: 16 lanes hold one block of a row, 8 values each, so its amax
// takes four lane rotations and nothing is shared between rows.  A thread
// takes R rows of a block; R = 1 spreads few rows over more workgroups.
template <int XT, int R>
__global__ void __launch_bounds__(256) quantize_rows(QuantizeArgs a) {
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
    const unsigned kblocks = (unsigned)((a.K + kBlock - 1) / kBlock);
    const int64_t kb = blockIdx.x % kblocks, k0 = kb * kBlock + c * 8;
    const int64_t m0 = (int64_t)(blockIdx.x / kblocks) * (16 * R) + g;
    const int n = (int)min((int64_t)8, max((int64_t)0, a.K - k0));
    float f[R][8];
    Raw8<XT> raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t m = m0 + 16 * i;
        raw[i] = fetch8<XT>(a.X, m * a.ldx + k0, k0, m < a.M ? n : 0);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        settle8<XT>(raw[i], k0, n);
        to_f32<XT>(raw[i], f[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t m = m0 + 16 * i;
        const float s = block_scale(max16(amax8(f[i])), a.e5m2, a.pow2);
        const i32x2q v = to_fp8x8(f[i], 1.0f / s, a.e5m2);
        if (m < a.M) {
            store_fp8x8(a.Q + m * a.ldq + k0, n, v);
            if (c == 0) a.S[m * a.s_row + kb * a.s_blk] = s;
        }
    }
}

// A 128 x 128 tile per workgroup: thread (c, g) holds the R x 8 values of
// rows R g .. and columns 8 c ...  The 16 threads of a row block are lanes of
// one 16-lane row, those of a column are spread over the waves, so column
// (and tile) maxima pass through LDS.  The transposed bytes pass through LDS
// too: written R at a time, they leave in rows of 128.
// Measured with both directions, bf16, rows: 8192^2 48.3 us at R = 4 (5.6
// TB/s), 50.8 at 8, 64.6 at 2; but with one tile per CU or fewer a thread's own
// arithmetic counts (66 x 320: 9.8 us at R = 8, 6.2 at 2).
template <int XT, bool TILE, int R>
__global__ void __launch_bounds__(2048 / R) quantize_tile(QuantizeArgs a) {
    constexpr int LD = kBlock + 16;              // a transposed row in LDS
    constexpr int T = 2048 / R, WAVES = T / 64;
    __shared__ __attribute__((aligned(16))) uint8_t tr[kBlock * LD];
    __shared__ float part[WAVES][kBlock];
    const int tid = threadIdx.x, c = tid & 15, g = tid >> 4, wave = tid >> 6, lane = tid & 63;
    const unsigned kblocks = (unsigned)((a.K + kBlock - 1) / kBlock);
    const int64_t kb = blockIdx.x % kblocks, mb = blockIdx.x / kblocks;
    const int64_t k0 = kb * kBlock + c * 8, m0 = mb * kBlock + g * R;
    const int n = (int)min((int64_t)8, max((int64_t)0, a.K - k0));
    float f[R][8];
    Raw8<XT> raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t m = m0 + i;
        raw[i] = fetch8<XT>(a.X, m * a.ldx + k0, k0, m < a.M ? n : 0);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        settle8<XT>(raw[i], k0, n);
        to_f32<XT>(raw[i], f[i]);
    }
    float r_tile = 0.0f, col[8];                 // reciprocal scales
    if constexpr (TILE) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) m = fmaxf(m, amax8(f[i]));
        m = max16(m);
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        if (lane == 0) part[0][wave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) m = fmaxf(m, part[0][w]);
        const float s = block_scale(m, a.e5m2, a.pow2);
        r_tile = 1.0f / s;
        if (tid == 0) {
            if (a.Q != nullptr) a.S[mb * a.s_row + kb * a.s_blk] = s;
            if (a.QT != nullptr) a.ST[kb * a.st_row + mb * a.st_blk] = s;
        }
    } else {
        // a column's maximum over the wave's rows, then over the waves: one
        // thread per column finishes it, and leaves the reciprocal for all
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < R; ++i) m = fmaxf(m, fabsf(f[i][j]));
            m = fmaxf(m, __shfl_xor(m, 16));
            m = fmaxf(m, __shfl_xor(m, 32));
            if (lane < 16) part[wave][c * 8 + j] = m;
        }
        __syncthreads();
        if (tid < kBlock) {
            float m = part[0][tid];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) m = fmaxf(m, part[w][tid]);
            const float s = block_scale(m, a.e5m2, a.pow2);
            const int64_t k = kb * kBlock + tid;
            if (k < a.K) a.ST[k * a.st_row + mb * a.st_blk] = s;
            part[0][tid] = 1.0f / s;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) col[j] = part[0][c * 8 + j];
    }
    if (a.Q != nullptr) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int64_t m = m0 + i;
            float r = r_tile;
            if constexpr (!TILE) {
                const float s = block_scale(max16(amax8(f[i])), a.e5m2, a.pow2);
                r = 1.0f / s;
                if (c == 0 && m < a.M) a.S[m * a.s_row + kb * a.s_blk] = s;
            }
            const i32x2q v = to_fp8x8(f[i], r, a.e5m2);
            if (m < a.M) store_fp8x8(a.Q + m * a.ldq + k0, n, v);
        }
    }
    if (a.QT == nullptr) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float r = TILE ? r_tile : col[j];
        uint8_t* to = tr + (c * 8 + j) * LD + g * R;
        if constexpr (R == 2) {
            *(uint16_t*)to = (uint16_t)to_fp8x4(f[0][j] * r, f[1][j] * r, 0.0f, 0.0f, a.e5m2);
        } else {
#pragma unroll
            for (int q = 0; q < R / 4; ++q)
                *(int*)(to + 4 * q) = to_fp8x4(f[4 * q][j] * r, f[4 * q + 1][j] * r, f[4 * q + 2][j] * r,
                                               f[4 * q + 3][j] * r, a.e5m2);
        }
    }
    __syncthreads();
    const int64_t mt = mb * kBlock + (tid & 7) * 16;
    const int nt = (int)min((int64_t)16, a.M - mt);
#pragma unroll
    for (int i = 0; i < kBlock * 8 / T; ++i) {
        const int row = i * (T / 8) + (tid >> 3);
        const int64_t k = kb * kBlock + row;
        if (k >= a.K || nt <= 0) continue;
        const i32x4q v = *(const i32x4q*)(tr + row * LD + (tid & 7) * 16);
        uint8_t* dst = a.QT + k * a.ldqt + mt;
        if (nt == 16) {
            *(i32x4u*)dst = v;
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e < nt) dst[e] = (uint8_t)((uint32_t)v[e >> 2] >> (8 * (e & 3)));
        }
    }
}

constexpr unsigned kFewTiles = 256;      // one per CU (4096 x 2048, 512 tiles: 10.3 us at R = 4, 12.2 at 2)

template <int XT>
hipError_t launch(const QuantizeArgs& a, bool tile, hipStream_t stream) {
    const int rows = quantize_rows_per_group(a.M, a.K, tile || a.QT != nullptr);
    const dim3 grid((unsigned)(((int64_t)a.K + kBlock - 1) / kBlock * (((int64_t)a.M + rows - 1) / rows)));
    if (tile || a.QT != nullptr) {
        const bool few = grid.x <= kFewTiles;
        if (tile && few)
            hipLaunchKernelGGL((quantize_tile<XT, true, 2>), grid, dim3(1024), 0, stream, a);
        else if (tile)
            hipLaunchKernelGGL((quantize_tile<XT, true, 4>), grid, dim3(quantize_threads(true)), 0, stream, a);
        else if (few)
            hipLaunchKernelGGL((quantize_tile<XT, false, 2>), grid, dim3(1024), 0, stream, a);
        else
            hipLaunchKernelGGL((quantize_tile<XT, false, 4>), grid, dim3(quantize_threads(true)), 0, stream, a);
    } else if (rows == 16)
        hipLaunchKernelGGL((quantize_rows<XT, 1>), grid, dim3(quantize_threads(false)), 0, stream, a);
    else
        hipLaunchKernelGGL((quantize_rows<XT, 4>), grid, dim3(quantize_threads(false)), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

int quantize_rows_per_group(int64_t M, int64_t K, bool tile) {
    if (tile) return kBlock;
    return (K + kBlock - 1) / kBlock * ((M + 15) / 16) <= 2048 ? 16 : 64;
}

hipError_t launch_quantize(const QuantizeArgs& a, int xtype, bool tile, hipStream_t stream) {
    switch (xtype) {
    case XT_F16: return launch<XT_F16>(a, tile, stream);
    case XT_BF16: return launch<XT_BF16>(a, tile, stream);
    default: return launch<XT_F32>(a, tile, stream);
    }
}

}  // namespace pg
