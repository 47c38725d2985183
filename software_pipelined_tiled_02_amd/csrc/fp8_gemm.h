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
    int32_t c_lines;         // C's rows start on 128 bytes, and nothing is read from them
};

// Tile classes: the workgroup's part of C, its waves, and how many of them
// share each piece of C, every one with blocks of K of its own (64K4: 64 x 64
// like 64, but its four waves do).
enum Fp8Tile : int { FP8_TILE_256 = 0, FP8_TILE_256x128 = 1, FP8_TILE_128 = 2, FP8_TILE_64 = 3, FP8_TILE_64K4 = 4,
                     FP8_TILE_64x32 = 5, FP8_TILE_32 = 6, FP8_TILE_16x32 = 7, FP8_TILE_16 = 8, FP8_TILE_COUNT = 9 };
struct Fp8Shape { int bm, bn, waves, wk; };
constexpr Fp8Shape fp8_shape(int t) {
    return t == FP8_TILE_256 ? Fp8Shape{256, 256, 8, 1}
         : t == FP8_TILE_256x128 ? Fp8Shape{256, 128, 8, 1}
         : t == FP8_TILE_128 ? Fp8Shape{128, 128, 8, 1}
         : t == FP8_TILE_64 ? Fp8Shape{64, 64, 4, 1}
         : t == FP8_TILE_64K4 ? Fp8Shape{64, 64, 4, 4}
         : t == FP8_TILE_64x32 ? Fp8Shape{64, 32, 4, 4}
         : t == FP8_TILE_32 ? Fp8Shape{32, 32, 8, 8}
         : t == FP8_TILE_16x32 ? Fp8Shape{16, 32, 8, 8}
                               : Fp8Shape{16, 16, 16, 16};
}
// Tiles staged through LDS (whole 16-byte chunks); the others read operands
// straight into registers.
constexpr bool fp8_staged(int t) { return t <= FP8_TILE_64x32; }

// What a tile class costs, for the choice between them: workgroups a CU holds
// at a time, and microseconds per block of 128 of a round of workgroups that
// gives no CU more than one (`some`) or fills every CU (`all`), and per round
// besides.  Measured on an MI355X with operands in the caches, at N = 4096
// and M = 32 to 4096, K = 512 to 8192 (fp32 outputs, whose blocks cost more,
// there too and at 1024^2 x 4096 and 4096^2 x 8200); microseconds at K = 4096 by
// the class chosen and the next best:
//   M = 32: 64x32 7.4, 16x32 8.4           M = 64: 64x32 8.1, 64x64k4 9.4
//   M = 128: 64x32 8.2, 64x64k4 9.4        M = 256: 64x64k4 10.3, 64x64 11.1
//   M = 512: 64x64 17.1, 64x64k4 18.4      M = 640: 128x128 18.9, 64x64 24.9
//   M = 1024: 128x128 22.3, 256x128 28.8   M = 2048: 256x128 34.6, 128x128 42.1
//   M = 4096: 256x256 57.8, 256x128 68.4
// and in fp32 M = 32: 16x32 8.9, 64x32 10.5; M = 128: 64x32 11.2, 64x64k4
// 14.4; M = 256: 64x64k4 14.9, 64x64 18.8; M = 512: 64x64 26.8, 64x64k4 27.9.
struct Fp8Cost { int per_cu; double some, all, round; };
constexpr Fp8Cost fp8_cost(int t, bool exact) {
    return t == FP8_TILE_256 ? Fp8Cost{1, 1.30, 1.65, 6.0}
         : t == FP8_TILE_256x128 ? (exact ? Fp8Cost{1, 1.75, 1.95, 5.0} : Fp8Cost{1, 0.78, 0.93, 5.0})
         : t == FP8_TILE_128 ? (exact ? Fp8Cost{1, 1.00, 1.16, 4.0} : Fp8Cost{1, 0.50, 0.60, 4.0})
         : t == FP8_TILE_64 ? (exact ? Fp8Cost{2, 0.47, 0.71, 2.8} : Fp8Cost{2, 0.24, 0.42, 2.5})
         : t == FP8_TILE_64K4 ? (exact ? Fp8Cost{1, 0.31, 0.31, 3.8} : Fp8Cost{1, 0.18, 0.18, 3.4})
         : t == FP8_TILE_64x32 ? (exact ? Fp8Cost{1, 0.21, 0.21, 3.2} : Fp8Cost{1, 0.13, 0.13, 2.9})
         : t == FP8_TILE_32 ? (exact ? Fp8Cost{2, 0.22, 0.47, 3.5} : Fp8Cost{2, 0.20, 0.44, 2.6})
         : t == FP8_TILE_16x32 ? Fp8Cost{2, 0.16, 0.34, 2.2}
                               : Fp8Cost{2, 0.12, 0.21, 2.5};
}
constexpr double fp8_time(int t, bool exact, int64_t workgroups, int64_t blocks, int64_t cus) {
    const Fp8Cost c = fp8_cost(t, exact);
    const int64_t slots = cus * c.per_cu, full = workgroups / slots, rest = workgroups % slots;
    const double last = rest == 0 ? 0.0 : rest <= cus ? c.some : c.all;
    return blocks * (full * c.all + last) + (full + (rest > 0 ? 1 : 0)) * c.round;
}

// The kernel for a call: a_type, b_type, row scales of B, fp32 output, and
// (register-fed tiles) rows that do not start or end on 16 bytes.
const void* fp8_stream_kernel(int tile, int a_type, int b_type, bool sb_rows, bool exact, bool bytes);
const void* fp8_staged_kernel(int tile, int a_type, int b_type, bool sb_rows, bool exact);
const void* fp8_waves_kernel(int tile, int a_type, int b_type, bool sb_rows, bool exact);

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

// Workgroup b of n runs on XCD b mod 8, each of which has an L2 of its own.
// The tile it takes: every XCD gets a run of neighbouring tiles.
__device__ __forceinline__ int by_xcd(unsigned b, unsigned n) {
    const unsigned x = b & 7, each = n >> 3, more = n & 7;
    return (int)(x * each + (x < more ? x : more) + (b >> 3));
}

// Tile number `tile`: each XCD gets a run of tiles, in bands of 4 tile rows,
// so that what it holds at a time shares rows of A and of B in its L2.
template <int BM, int BN>
__device__ __forceinline__ void place_tile(const Fp8Args& a, int tile, int& m0, int& n0) {
    constexpr int kBand = 4;
    const int w = by_xcd(tile, a.tiles_m * a.tiles_n);
    const int band = kBand * a.tiles_n, gi = w / band, first = gi * kBand;
    const int rows = min(a.tiles_m - first, kBand), in = w - gi * band;
    m0 = (first + in % rows) * BM;
    n0 = in / rows * BN;
}

// At most N of this wave's loads are still in flight (vmcnt; loads retire in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("" ::: "memory");
}
// Barrier behind this wave's LDS accesses.
__device__ __forceinline__ void barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// This wave's LDS accesses are done.
__device__ __forceinline__ void wait_lds() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (0 << 8));
    asm volatile("" ::: "memory");
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

// Four values rounded to bf16 or fp16 (nearest even).
__device__ __forceinline__ i32x2 to_16(f32x4 v, int type) {
    if (type == XT_BF16)
        return i32x2{__builtin_bit_cast(int, bf16x2{(__bf16)v[0], (__bf16)v[1]}),
                     __builtin_bit_cast(int, bf16x2{(__bf16)v[2], (__bf16)v[3]})};
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return i32x2{__builtin_bit_cast(int, f16x2{(_Float16)v[0], (_Float16)v[1]}),
                 __builtin_bit_cast(int, f16x2{(_Float16)v[2], (_Float16)v[3]})};
}

// C[m][n .. n+3], rounded once to C's type; columns at or past N are left.
template <bool EXACT>
__device__ __forceinline__ void store_c(const Fp8Args& a, int64_t m, int64_t n, f32x4 v) {
    if constexpr (EXACT) {
        float* p = (float*)a.C + m * a.ldc + n;
        if (n + 4 <= a.N) {
            if (a.accumulate) v += __builtin_bit_cast(f32x4, (i32x4q)*(const i32x4u*)p);
            *(i32x4u*)p = __builtin_bit_cast(i32x4q, v);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.N) p[e] = a.accumulate ? p[e] + v[e] : v[e];
        }
    } else {
        uint16_t* p = (uint16_t*)a.C + m * a.ldc + n;
        const i32x2 w = to_16(v, a.c_type);
        if (n + 4 <= a.N) {
            *(i32x2u*)p = w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.N) p[e] = (uint16_t)((uint32_t)w[e >> 1] >> (16 * (e & 1)));
        }
    }
}

// The epilogue's LDS: per wave, a strip of 16 rows of its block of C, each row
// padded by 16 bytes (so that the rows of a column fall in different banks).
constexpr int strip_row(int fn, int size) { return 16 * fn * size + 16; }
constexpr int epilogue_lds(int waves, int fn, int size) { return waves * 16 * strip_row(fn, size); }

// A wave's block of FM x FN pieces at (m0, n0).  A lane holds 4 neighbouring
// columns, 8 or 16 bytes, of a row; stored like that, an instruction would
// write 32-byte runs of 16 rows.  A strip of 16 rows goes through the wave's
// own part of LDS instead and leaves 16 bytes per lane, whole rows of the block
// at a time (256x256 tiles, 4096^3: 4 us less, at 8192^3 30 us less of 490).
// STREAM: past the caches where C's rows start on whole lines (8192 x 4096 x
// 256 fp32: 43.6 us, 49.0 through them; 2048 x 4096^2 bf16 35.7 and 37.3);
// pieces of lines are joined there (8192 x 8190 x 512 bf16: 60.5 us, past them 76.6;
// 6384 x 2731 x 128 fp32 23.7 and 30.4).
template <bool EXACT, int FM, int FN, bool STREAM>
__device__ __forceinline__ void store_block(const Fp8Args& a, uint8_t PG_LDS* smem, int wave, int m0, int n0,
                                            const f32x4 (&acc)[FM][FN]) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    constexpr int SIZE = EXACT ? 4 : 2, ROW = strip_row(FN, SIZE), CHUNKS = FN * SIZE;   // 16-byte chunks of a row
    if (m0 + 16 * FM <= a.M && n0 + 16 * FN <= a.N) {
        uint8_t PG_LDS* strip = smem + wave * 16 * ROW;     // (a wave's LDS accesses keep their order)
        constexpr int Q = (16 * CHUNKS + 63) / 64;
        const auto target = [&](int i, int q) {
            const int row = (q * 64 + lane) / CHUNKS, c = (q * 64 + lane) % CHUNKS;
            return (i32x4u*)((uint8_t*)a.C + ((int64_t)(m0 + 16 * i + row) * a.ldc + n0) * SIZE + c * 16);
        };
        // What C holds (accumulate), a strip ahead: behind the stores each
        // load would be waited for in turn (8192 x 4096 x 512: 101 us, 89 so).
        f32x4 old[2][Q];
        const auto fetch = [&](int i) {
            if constexpr (EXACT)
                if (a.accumulate)
#pragma unroll
                    for (int q = 0; q < Q; ++q)
                        if ((q * 64 + lane) / CHUNKS < 16) old[i & 1][q] = __builtin_bit_cast(f32x4, (i32x4)*target(i, q));
        };
        fetch(0);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            if (i + 1 < FM) fetch(i + 1);
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                uint8_t PG_LDS* p = strip + r * ROW + (16 * j + 4 * g) * SIZE;
                if constexpr (EXACT) *(f32x4 PG_LDS*)p = acc[i][j];
                else *(i32x2 PG_LDS*)p = to_16(acc[i][j], a.c_type);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int row = (q * 64 + lane) / CHUNKS, c = (q * 64 + lane) % CHUNKS;
                if (row >= 16) break;
                i32x4 v = *(const i32x4 PG_LDS*)(strip + row * ROW + c * 16);
                i32x4u* dst = target(i, q);
                if constexpr (EXACT)
                    if (a.accumulate) v = __builtin_bit_cast(i32x4, __builtin_bit_cast(f32x4, v) + old[i & 1][q]);
                if (STREAM && a.c_lines) {
                    asm volatile("" ::: "memory");       // (or the two stores become a plain one)
                    __builtin_nontemporal_store(v, dst);
                    asm volatile("" ::: "memory");
                } else {
                    *dst = v;
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t m = m0 + 16 * i + r;
        if (m >= a.M) continue;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int64_t n = n0 + 16 * j + 4 * g;
            if (n < a.N) store_c<EXACT>(a, m, n, acc[i][j]);
        }
    }
}

#endif

}  // namespace pg

#endif
