// fp8_common.h -- what the 8-bit kernels share: types, argument blocks,
// conversions, and the scale of a block.  Device helpers are inline; the
// argument blocks are plain structs the host fills.
//
// 8-bit floats are the OCP types gfx950 converts and multiplies: e4m3 (top
// 448, one NaN, no infinity) and e5m2 (top 57344).  A block is kBlock = 128
// values (or 128 x 128) with one fp32 scale s; a stored value q stands for
// q * s.
#ifndef PIPEGEMM_FP8_COMMON_H
#define PIPEGEMM_FP8_COMMON_H

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pg {

enum Fp8Type : int { FP8_E4M3 = 0, FP8_E5M2 = 1 };
enum XType : int { XT_F16 = 1, XT_BF16 = 2, XT_F32 = 3 };   // the GEMM_* values of the float types

constexpr int kBlock = 128;

struct QuantizeArgs {
    const void* X;
    uint8_t* Q;              // M x K, or NULL
    float* S;                // scale (row m or row block, k block) at m * s_row + kb * s_blk
    uint8_t* QT;             // K x M, or NULL
    float* ST;               // scale (row k or row block, m block) at k * st_row + mb * st_blk
    int64_t ldx, ldq, ldqt, s_row, s_blk, st_row, st_blk;
    int32_t M, K;
    int32_t e5m2, pow2;
};

struct RmsArgs {
    const void* X;
    const void* R;           // residual, or NULL
    const void* W;
    void* H;                 // x + residual, or NULL
    void* Y;                 // the normalised row in X's type, or NULL
    uint8_t* Q;              // or NULL
    float* S;
    float* rstd;             // or NULL
    int64_t ldx, ldr, ldh, ldy, ldq, s_row, s_blk;
    int32_t M, D;
    float eps;
    int32_t e5m2, pow2, w_f32;
};

struct RmsBackwardArgs {
    const void* DY;
    const void* H;
    const void* W;
    const float* rstd;
    const void* DH;          // gradient that reaches h from elsewhere, or NULL
    void* DX;
    float* parts;            // [groups][D rounded up to 4] partial sums of dw
    float* DW;
    int64_t lddy, ldh, lddh, lddx;
    int32_t M, D, groups;    // groups: parts of dw
    int32_t w_f32;
    int32_t in_place;        // DX's bytes meet DY's or H's
};

#if defined(__HIPCC__)

typedef int i32x4q __attribute__((ext_vector_type(4)));
typedef int i32x2q __attribute__((ext_vector_type(2)));

template <int XT> struct XTypeOf { typedef float type; };
template <> struct XTypeOf<XT_F16> { typedef _Float16 type; };
template <> struct XTypeOf<XT_BF16> { typedef __bf16 type; };

// Accesses of 8 and 16 bytes at any address: gfx950 reads and writes them
// whole, so rows need no alignment beyond their elements' (8192 x 9300 bf16
// rows, 4 bytes off 16, element by element: three times the time).
typedef i32x4q i32x4u __attribute__((aligned(1)));
typedef i32x2q i32x2u __attribute__((aligned(1)));

// Eight consecutive elements as they lie in memory.
template <int XT> struct Raw8 { typename XTypeOf<XT>::type v __attribute__((ext_vector_type(8))); };

// Elements k .. k + 7 of a row, of which the row has the first `n`; element k
// lies at base + at.  Where the row ends among them the access moves back to
// end with it, and settle8, called when the values are needed, moves them to
// their places: element by element, each load is waited for on the spot
// (norm's backward pass in bf16, 7763 x 276: 21.6 us against 16.0).  The
// elements in front are dropped, so they may be changing.
template <int XT>
__device__ __forceinline__ Raw8<XT> fetch8(const void* base, int64_t at, int64_t k, int n) {
    typedef typename XTypeOf<XT>::type T;
    const T* p = (const T*)base + at;
    Raw8<XT> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = (T)0.0f;
    if (n >= 8 || (n > 0 && k >= 8)) {
        p -= 8 - min(n, 8);
        if constexpr (XT == XT_F32) {
            struct Two { i32x4q a, b; } two = {*(const i32x4u*)p, *(const i32x4u*)(p + 4)};
            r = __builtin_bit_cast(Raw8<XT>, two);
        } else {
            r = __builtin_bit_cast(Raw8<XT>, (i32x4q)*(const i32x4u*)p);
        }
    } else if (n > 0) {                      // a row of less than 8
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) r.v[e] = p[e];
    }
    return r;
}

// The n elements at their places, zeros behind them.
template <int XT>
__device__ __forceinline__ void settle8(Raw8<XT>& r, int64_t k, int n) {
    typedef typename XTypeOf<XT>::type T;
    if (n <= 0 || n >= 8 || k < 8) return;
#pragma unroll
    for (int by = 4; by > 0; by >>= 1)
        if ((8 - n) & by) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r.v[e] = e + by < 8 ? r.v[e + by < 8 ? e + by : 0] : (T)0.0f;
        }
}

template <int XT>
__device__ __forceinline__ void to_f32(const Raw8<XT>& r, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)r.v[e];
}

// Both, and the values as fp32.
template <int XT>
__device__ __forceinline__ void load8(const void* base, int64_t at, int64_t k, int n, float (&f)[8]) {
    Raw8<XT> r = fetch8<XT>(base, at, k, n);
    settle8<XT>(r, k, n);
    to_f32<XT>(r, f);
}

// Eight consecutive elements rounded to the type (nearest even), those
// before `n`.
template <int XT>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, const float (&f)[8]) {
    typedef typename XTypeOf<XT>::type T;
    T* p = (T*)base + at;
    if (n >= 8) {
        Raw8<XT> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = (T)f[e];
        if constexpr (XT == XT_F32) {
            struct Two { i32x4q a, b; };
            const Two two = __builtin_bit_cast(Two, r);
            *(i32x4u*)p = two.a;
            *(i32x4u*)(p + 4) = two.b;
        } else {
            *(i32x4u*)p = __builtin_bit_cast(i32x4q, r);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = (T)f[e];
    }
}

// A value rounded to the type (nearest even), as fp32.
template <int XT>
__device__ __forceinline__ float rounded(float x) {
    return (float)(typename XTypeOf<XT>::type)x;
}

// Four values to 8 bits each, rounded to nearest even.
__device__ __forceinline__ int to_fp8x4(float a, float b, float c, float d, bool e5m2) {
    int v = 0;
    if (e5m2) {
        v = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, v, false);
        v = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, v, true);
    } else {
        v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, v, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    }
    return v;
}

__device__ __forceinline__ i32x2q to_fp8x8(const float (&f)[8], float r, bool e5m2) {
    return i32x2q{to_fp8x4(f[0] * r, f[1] * r, f[2] * r, f[3] * r, e5m2),
                  to_fp8x4(f[4] * r, f[5] * r, f[6] * r, f[7] * r, e5m2)};
}

// The scale of a block whose largest |x| is amax: amax / top, or the next
// power of two, at least the smallest normal number (so that 1 / s is
// finite, and a block of zeros gives zeros).  |x| * (1 / s) exceeds `top` by
// three roundings of 2^-24 at most, far below the half step at which the
// conversion would leave the type's range.
__device__ __forceinline__ float block_scale(float amax, bool e5m2, bool pow2) {
    float s = amax / (e5m2 ? 57344.0f : 448.0f);
    s = s < 0x1p-126f ? 0x1p-126f : s;
    if (pow2) s = __uint_as_float((__float_as_uint(s) + 0x007fffffu) & 0x7f800000u);
    return s;
}

// Largest value of the 16 lanes of a row (DPP rotations inside the row).
__device__ __forceinline__ float max16(float x) {
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xf, 0xf, true)));   // row_ror:8
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x124, 0xf, 0xf, true)));   // row_ror:4
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x122, 0xf, 0xf, true)));   // row_ror:2
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x121, 0xf, 0xf, true)));   // row_ror:1
    return x;
}

// Sum over the wave, the same in every lane.
__device__ __forceinline__ float sum64(float x) {
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xf, 0xf, true));
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x124, 0xf, 0xf, true));
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x122, 0xf, 0xf, true));
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x121, 0xf, 0xf, true));
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

__device__ __forceinline__ float amax8(const float (&f)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
    return m;
}

// Eight 8-bit values to a row, those before `n`.
__device__ __forceinline__ void store_fp8x8(uint8_t* p, int n, i32x2q v) {
    if (n >= 8) {
        *(i32x2u*)p = v;
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = (uint8_t)((uint32_t)v[e >> 2] >> (8 * (e & 3)));
    }
}

#endif

// Launchers (fp8_quantize.hip, fp8_rms.hip); each enqueues on the current device.
hipError_t launch_quantize(const QuantizeArgs& a, int xtype, bool tile, hipStream_t stream);
// Rows of one workgroup (blocks of 128 columns each), and its threads where
// there are many; a launch takes less than 2^32 threads.
int quantize_rows_per_group(int64_t M, int64_t K, bool tile);
constexpr int quantize_threads(bool tile) { return tile ? 512 : 256; }
hipError_t launch_rms(const RmsArgs& a, int xtype, hipStream_t stream);
struct RmsBackwardForm;      // fp8_rms_plan.h
hipError_t launch_rms_backward(const RmsBackwardArgs& a, const RmsBackwardForm& form, int xtype, hipStream_t stream);

}  // namespace pg

#endif
