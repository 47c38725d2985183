// fp8_gemm.h -- products of 8-bit float matrices with a scale for each block
// of 128: what the kernels share.
//
//   C[i][j] = sum over blocks kb of SA[i][kb] * SB[jb][kb] * t,
//   t = sum over k in block kb of A[i][k] * B[j][k],
//
// A is M x K and B (the second factor's transpose) N x K, both with K
// contiguous; jb is j / 128 for "tile" scales of B and j for "row" scales.
// One block of 128 is exactly one 16x16x128 matrix instruction, so a block
// costs a wave one instruction and four multiply-adds per 16x16 piece of C:
// t comes out of the matrix core and goes, times the blocks' scales, into
// fp32 accumulators.
//
// Precision.  The 8-bit matrix instructions form a block's sum with fewer
// bits than fp32: on normal data their sums are 1.3e-5 to 2e-5 off (2-norm,
// measured; all of the 8-bit shapes alike), far below the half step of a
// 16-bit output (2^-8 and 2^-11 of the value).  For fp32 outputs (gradients
// that are accumulated) that would be the largest error by far, so those widen
// both operands to bf16 -- every 8-bit value is one exactly -- and take four
// 16x16x32 bf16 instructions a block, which are 1e-8 off, at half the rate.
//
// The second factor's fragment is the instruction's first operand, so a lane
// (r = lane % 16, g = lane / 16) ends up with row r and columns 4 g .. +3 of a
// 16x16 piece.  Operand order inside a block: lane group g holds bytes
// 16 g .. +15 and 64 + 16 g .. +15 of the block, the same for both operands.
#ifndef PIPEGEMM_FP8_GEMM_H
#define PIPEGEMM_FP8_GEMM_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_common.h"
#include "tile_layout.h"

namespace pg {

struct Fp8Args {
    const uint8_t* A;
    const uint8_t* B;
    const float* SA;         // scale (i, kb) at i * sa_row + kb * sa_blk
    const float* SB;
    void* C;
    int64_t lda, ldb, ldc, sa_row, sa_blk, sb_row, sb_blk;
    int32_t M, N, K;
    int32_t tiles_m, tiles_n;
    int32_t c_type;          // XT_*
    int32_t accumulate;      // C += (fp32)
    int32_t vec_c;           // four neighbouring outputs are one aligned store
};

// Tile classes: the workgroup's part of C, and the waves that share its K.
enum Fp8Tile : int { FP8_TILE_256 = 0, FP8_TILE_128 = 1, FP8_TILE_64 = 2, FP8_TILE_64x32 = 3, FP8_TILE_32 = 4,
                     FP8_TILE_16 = 5, FP8_TILE_COUNT = 6 };
struct Fp8Shape { int bm, bn, waves, wk; };
constexpr Fp8Shape fp8_shape(int t) {
    return t == FP8_TILE_256 ? Fp8Shape{256, 256, 8, 1}
         : t == FP8_TILE_128 ? Fp8Shape{128, 128, 4, 1}
         : t == FP8_TILE_64 ? Fp8Shape{64, 64, 8, 8}
         : t == FP8_TILE_64x32 ? Fp8Shape{64, 32, 8, 8}
         : t == FP8_TILE_32 ? Fp8Shape{32, 32, 8, 8}
                            : Fp8Shape{16, 16, 16, 16};
}
// Tiles staged through LDS (whole 16-byte chunks); the others read operands
// straight into registers.
constexpr bool fp8_staged(int t) { return t == FP8_TILE_256 || t == FP8_TILE_128; }

// The kernel for a call: a_type, b_type, row scales of B, fp32 output, and
// (register-fed tiles) rows that do not start or end on 16 bytes.
const void* fp8_stream_kernel(int tile, int a_type, int b_type, bool sb_rows, bool exact, bool bytes);
const void* fp8_staged_kernel(int tile, int a_type, int b_type, bool sb_rows, bool exact);

#if defined(__HIPCC__)

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

#define PG_LDS __attribute__((address_space(3)))

// Raw buffer resource, word 3 of the gfx9 family; an offset past its range,
// from which loads give zero.
constexpr int kBufferWord3 = 0x00020000;
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc((void*)p, 0, 0x7fffffff, kBufferWord3);
}

// Eight 8-bit floats (two words) as bf16, exactly.
template <int T>
__device__ __forceinline__ bf16x8 widen(int lo, int hi) {
    bf16x2 a, b, c, d;
    if constexpr (T == FP8_E5M2) {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.0f, true);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.0f, true);
    } else {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    }
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A fragment as the matrix instruction takes it: 32 bytes per lane, or
// (EXACT) the same widened to bf16.
template <int T, bool EXACT> struct Frag { i32x8 v; };
template <int T> struct Frag<T, true> { bf16x8 v[4]; };

template <int T, bool EXACT>
__device__ __forceinline__ Frag<T, EXACT> fragment(i32x4 lo, i32x4 hi) {
    Frag<T, EXACT> f;
    if constexpr (EXACT) {
        f.v[0] = widen<T>(lo[0], lo[1]);
        f.v[1] = widen<T>(lo[2], lo[3]);
        f.v[2] = widen<T>(hi[0], hi[1]);
        f.v[3] = widen<T>(hi[2], hi[3]);
    } else {
        f.v = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
    return f;
}

// One block's sum for a 16x16 piece.
template <int AT, int BT, bool EXACT>
__device__ __forceinline__ f32x4 block_sum(const Frag<BT, EXACT>& x, const Frag<AT, EXACT>& y) {
    f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (EXACT) {
#pragma unroll
        for (int h = 0; h < 4; ++h) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x.v[h], y.v[h], t, 0, 0, 0);
    } else {
        t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x.v, y.v, t, BT, AT, 0, 0, 0, 0);
    }
    return t;
}

// C[m][n .. n+3], rounded once to C's type; columns at or past N are left.
template <bool EXACT>
__device__ __forceinline__ void store_c(const Fp8Args& a, int64_t m, int64_t n, f32x4 v) {
    if constexpr (EXACT) {
        float* p = (float*)a.C + m * a.ldc + n;
        if (a.vec_c && n + 4 <= a.N) {
            if (a.accumulate) v += *(const f32x4*)p;
            *(f32x4*)p = v;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.N) p[e] = a.accumulate ? p[e] + v[e] : v[e];
        }
    } else {
        uint16_t* p = (uint16_t*)a.C + m * a.ldc + n;
        i32x2 w;
        if (a.c_type == XT_BF16) {
            w = i32x2{__builtin_bit_cast(int, bf16x2{(__bf16)v[0], (__bf16)v[1]}),
                      __builtin_bit_cast(int, bf16x2{(__bf16)v[2], (__bf16)v[3]})};
        } else {
            typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
            w = i32x2{__builtin_bit_cast(int, f16x2{(_Float16)v[0], (_Float16)v[1]}),
                      __builtin_bit_cast(int, f16x2{(_Float16)v[2], (_Float16)v[3]})};
        }
        if (a.vec_c && n + 4 <= a.N) {
            *(i32x2*)p = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.N) p[e] = (uint16_t)((uint32_t)w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

#endif

}  // namespace pg

#endif
