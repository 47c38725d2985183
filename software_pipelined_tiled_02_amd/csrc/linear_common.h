// linear_common.h -- what the feed-forward kernels share: the argument block,
// the activations, and what is done with the fp32 sums of a product before
// they are stored.
//
//   linear           C = act(A B + A2 B2 + bias) + residual, and Z, act's argument
//   gated            H = act(X Wg^T + bg) * (X Wu^T + bu), and G and U
//   gated_backward   dH = dY W: dG = dH U act'(G), dU = dH act(G), and H
//   weight_gradient  dW = dC^T A in fp32, and the sums of dC's columns
//
// Operands are bf16 or fp16 and products are summed in fp32 by the matrix
// cores; everything up to a result's one rounding to the operands' type is
// fp32 too.  In a kernel's terms each is a product of M x N sums (gated: two)
// over K, with an ending of its own.
#ifndef PIPEGEMM_LINEAR_COMMON_H
#define PIPEGEMM_LINEAR_COMMON_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_common.h"

namespace pg {

enum Ending : int { END_LINEAR = 0, END_GATED = 1, END_GATED_BACKWARD = 2, END_WEIGHT = 3 };
enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

struct LinearArgs {
    const void* A[2];        // linear: the two products' first factors
    const void* B[2];        // ... and second ones; gated: Wg and Wu
    const void* in[2];       // linear: residual; gated_backward: G, U (each may be NULL but G)
    void* out[3];            // linear: C, Z; gated: H, G, U; gated_backward: dG, dU, H; weight_gradient: dW
    const void* bias[2];     // linear: bias; gated: bg, bu
    float* sums;             // weight_gradient: sums of dC's columns, or NULL
    int64_t lda[2], ldb[2], ldi[2], ldo[3];
    int32_t M, N, K;         // sums are M x N
    int32_t tiles_m, tiles_n;
    int32_t act, bias_f32, accumulate;
    int32_t apart;           // some of the factors' rows do not start on 16 bytes
};

// Tile classes: the workgroup's part of the sums (gated: half of the columns are
// the second product's), and its waves.  From 64K4 on each wave takes K-tiles of
// its own.
enum LinearTile : int { LINEAR_TILE_256 = 0, LINEAR_TILE_128x256 = 1, LINEAR_TILE_128 = 2, LINEAR_TILE_64 = 3,
                        LINEAR_TILE_64K4 = 4, LINEAR_TILE_64x32 = 5, LINEAR_TILE_32 = 6, LINEAR_TILE_16x32 = 7,
                        LINEAR_TILE_16 = 8, LINEAR_TILE_COUNT = 9 };
struct LinearShape { int bm, bn, waves; };
constexpr LinearShape linear_shape(int t) {
    return t == LINEAR_TILE_256 ? LinearShape{256, 256, 4}
         : t == LINEAR_TILE_128x256 ? LinearShape{128, 256, 4}
         : t == LINEAR_TILE_128 ? LinearShape{128, 128, 4}
         : t == LINEAR_TILE_64 ? LinearShape{64, 64, 4}
         : t == LINEAR_TILE_64K4 ? LinearShape{64, 64, 4}
         : t == LINEAR_TILE_64x32 ? LinearShape{64, 32, 4}
         : t == LINEAR_TILE_32 ? LinearShape{32, 32, 8}
         : t == LINEAR_TILE_16x32 ? LinearShape{16, 32, 8}
                                  : LinearShape{16, 16, 8};
}
constexpr bool linear_few_tile(int t) { return t >= LINEAR_TILE_64K4; }

// The kernel for a call: XT_F16 or XT_BF16, a tile class (NULL: the operator does not
// have it), and whether there is a second product (linear) or sums of A's rows
// (weight gradients).
const void* linear_rc_kernel(int xt, int tile, bool pair);
const void* linear_rr_kernel(int xt, int tile, bool pair);
const void* gated_kernel(int xt, int tile);
const void* gated_backward_kernel(int xt, int tile);
const void* weight_gradient_kernel(int xt, int tile, bool sums);

#if defined(__HIPCC__)

// Both tails are formed 2^8 times as large, and z's part of a result 2^-8 times: the
// factor's value may lie below 2^-126, where exp2 and rcp give 0, and the
// result's not (silu(-88) = -5.3e-37; factors themselves: -0).

// The distribution function of the normal distribution at -|z|, from
// e = 2^8 exp(-z^2 / 2): e times half of exp(x^2) erfc(x), x = |z| / sqrt 2,
// which is a polynomial in t = 1 / (1 + 0.54 x) to 4e-6 (fitted here, by least
// squares with weights moved to the largest relative errors).  5e-6 off for |z| <
// 6 in fp32, a hundredth of fp16's half step; the far tail keeps its relative error.
__device__ __forceinline__ float normal_exp(float z) { return __builtin_amdgcn_exp2f(fmaf(-0.721347520f * z, z, 8.0f)); }
__device__ __forceinline__ float normal_tail(float z, float e) {
    constexpr float s = 0x1p-8f;
    const float t = __builtin_amdgcn_rcpf(fmaf(0.381837662f, fabsf(z), 1.0f));
    float p = fmaf(0.0480623953f * s, t, -0.155210704f * s);
    p = fmaf(p, t, 0.105571732f * s);
    p = fmaf(p, t, 0.063943103f * s);
    p = fmaf(p, t, 0.133146182f * s);
    p = fmaf(p, t, 0.152152315f * s);
    p = fmaf(p, t, 0.152334273f * s);
    return e * p * t;
}

// silu(z) = z s(z) and gelu_tanh(z) = z s(2 sqrt(2 / pi) (z + 0.044715 z^3)), s the
// logistic function: both are z s(z (c1 + c3 z^2)).  s through exp2, so the
// constants hold -log2 e.  Past |z| = 128 s is 0 or 1 in fp32, and is taken there:
// its argument's terms overflow.
struct Logistic { float c1, c3; };
__device__ __forceinline__ Logistic logistic_of(int act) {
    return act == ACT_SILU ? Logistic{-1.44269504f, 0.0f} : Logistic{-2.30220818f, -0.102943240f};
}
__device__ __forceinline__ float within128(float z) { return __builtin_amdgcn_fmed3f(z, -128.0f, 128.0f); }   // (a NaN too)
__device__ __forceinline__ float logistic_256(float z, Logistic l) {  // 2^8 s, |z| <= 128
    return __builtin_amdgcn_rcpf(0x1p-8f + __builtin_amdgcn_exp2f(fmaf(z, fmaf(l.c3 * z, z, l.c1), -8.0f)));
}

// Values through the activation.  The branches are the same for a whole
// launch.  A NaN stays one.
template <int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
    if (act == ACT_NONE) return;
    if (act == ACT_RELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = v[e] < 0.0f ? 0.0f : v[e];
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float q = normal_tail(v[e], normal_exp(v[e]));
            v[e] *= v[e] > 0.0f ? 1.0f - q : q;
        }
    } else {
        const Logistic l = logistic_of(act);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = 0x1p-8f * v[e] * logistic_256(within128(v[e]), l);
    }
}

// The activation a and its derivative d at N values.  The derivative past |z|
// = 128 is taken there: 0 or 1 in fp32.  A NaN stays one in both.
template <int N>
__device__ __forceinline__ void activate_slope(int act, const float (&z)[N], float (&a)[N], float (&d)[N]) {
    if (act == ACT_NONE) {
#pragma unroll
        for (int e = 0; e < N; ++e) { a[e] = z[e]; d[e] = 1.0f; }
    } else if (act == ACT_RELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            a[e] = z[e] < 0.0f ? 0.0f : z[e];
            d[e] = z[e] > 0.0f ? 1.0f : z[e] <= 0.0f ? 0.0f : z[e];
        }
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float c = within128(z[e]);
            const float x = normal_exp(c);
            const float q = normal_tail(c, x), p = c > 0.0f ? 1.0f - q : q;
            a[e] = z[e] * p;
            d[e] = z[e] == z[e] ? fmaf(0.398942280f * 0x1p-8f * c, x, p) : z[e];
        }
    } else {
        const Logistic l = logistic_of(act);
        const float k1 = -0.693147181f * l.c1, k3 = -2.07944154f * l.c3;        // q' = k1 + k3 z^2, back from base 2
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const float c = within128(z[e]);
            const float s256 = logistic_256(c, l), s = 0x1p-8f * s256;
            a[e] = 0x1p-8f * z[e] * s256;
            d[e] = z[e] == z[e] ? fmaf(0x1p-8f * c * s256 * (1.0f - s), fmaf(k3 * c, c, k1), s) : z[e];
        }
    }
}

// Eight neighbouring values of a row, `left` of them before its end (WHOLE: eight
// or more; else the access is one that fetch8 and store8 describe).
template <int XT, bool WHOLE>
__device__ __forceinline__ Raw8<XT> get8(const void* base, int64_t at, int64_t n, int left) {
    if constexpr (!WHOLE) {
        return fetch8<XT>(base, at, n, left);
    } else if constexpr (XT == XT_F32) {
        const float* p = (const float*)base + at;
        struct Two { i32x4q a, b; } two = {*(const i32x4u*)p, *(const i32x4u*)(p + 4)};
        return __builtin_bit_cast(Raw8<XT>, two);
    } else {
        return __builtin_bit_cast(Raw8<XT>, (i32x4q)*(const i32x4u*)((const uint16_t*)base + at));
    }
}
template <int XT, bool WHOLE>
__device__ __forceinline__ void read8(Raw8<XT> r, int64_t n, int left, float* f) {
    if constexpr (!WHOLE) settle8<XT>(r, n, left);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)r.v[e];
}
template <int XT, bool WHOLE>
__device__ __forceinline__ void put8(void* base, int64_t at, int left, const float* f) {
    typedef typename XTypeOf<XT>::type T;
    if constexpr (!WHOLE) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f[e];
        store8<XT>(base, at, left, v);
    } else {
        Raw8<XT> r;
#pragma unroll
        for (int e = 0; e < 8; ++e) r.v[e] = (T)f[e];
        T* p = (T*)base + at;
        if constexpr (XT == XT_F32) {
            struct Two { i32x4q a, b; };
            const Two two = __builtin_bit_cast(Two, r);
            *(i32x4u*)p = two.a;
            *(i32x4u*)(p + 4) = two.b;
        } else {
            *(i32x4u*)p = __builtin_bit_cast(i32x4q, r);
        }
    }
}

// What an ending reads beside the sums, for eight neighbouring outputs.
template <int XT, int END>
struct Beside { Raw8<XT> a, b; Raw8<XT_F32> c; };

template <int XT, int END, bool WHOLE>
__device__ __forceinline__ Beside<XT, END> fetch_beside(const LinearArgs& p, int64_t m, int64_t n) {
    Beside<XT, END> r;
    const int left = p.N - (int)n;
    if constexpr (END == END_LINEAR || END == END_GATED_BACKWARD)
        if (p.in[0] != nullptr) r.a = get8<XT, WHOLE>(p.in[0], m * p.ldi[0] + n, n, left);
    if constexpr (END == END_GATED_BACKWARD)
        if (p.in[1] != nullptr) r.b = get8<XT, WHOLE>(p.in[1], m * p.ldi[1] + n, n, left);
    if constexpr (END == END_WEIGHT)
        if (p.accumulate) r.c = get8<XT_F32, WHOLE>(p.out[0], m * p.ldo[0] + n, n, left);
    return r;
}

// The biases of eight neighbouring columns.
template <int END>
struct Biases { float v[8], u[8]; };

template <int XT, int END>
__device__ __forceinline__ Biases<END> fetch_biases(const LinearArgs& p, int64_t n) {
    Biases<END> b;
    const auto fetch = [&](const void* from, float (&f)[8]) {
        const int left = p.N - (int)n;
        if (from == nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = 0.0f;
        } else if (p.bias_f32) {
            load8<XT_F32>(from, n, n, left, f);
        } else {
            load8<XT>(from, n, n, left, f);
        }
    };
    if constexpr (END == END_LINEAR || END == END_GATED) fetch(p.bias[0], b.v);
    if constexpr (END == END_GATED) fetch(p.bias[1], b.u);
    return b;
}

// The ending for outputs (m + q step, n .. n + 7), q < Q, rows m .. < M and n < N:
// v holds their sums, u (gated) the second product's.
template <int XT, int END, bool WHOLE, int Q>
__device__ __forceinline__ void finish(const LinearArgs& p, int64_t m, int64_t step, int64_t n, Beside<XT, END> (&beside)[Q],
                                       const Biases<END>& bias, float (&v)[8 * Q], float (&u)[8 * Q]) {
    const int left = p.N - (int)n;
    const auto put = [&](int which, const float (&f)[8 * Q]) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            put8<XT, WHOLE>(p.out[which], (m + q * step) * p.ldo[which] + n, left, f + 8 * q);
    };
    if constexpr (END == END_LINEAR) {
#pragma unroll
        for (int e = 0; e < 8 * Q; ++e) v[e] += bias.v[e % 8];
        if (p.out[1] != nullptr) put(1, v);
        activate(p.act, v);
        if (p.in[0] != nullptr) {
            float r[8 * Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) read8<XT, WHOLE>(beside[q].a, n, left, r + 8 * q);
#pragma unroll
            for (int e = 0; e < 8 * Q; ++e) v[e] += r[e];
        }
        put(0, v);
    } else if constexpr (END == END_GATED) {
#pragma unroll
        for (int e = 0; e < 8 * Q; ++e) {
            v[e] += bias.v[e % 8];
            u[e] += bias.u[e % 8];
        }
        if (p.out[1] != nullptr) {
            put(1, v);
            put(2, u);
        }
        activate(p.act, v);
#pragma unroll
        for (int e = 0; e < 8 * Q; ++e) v[e] *= u[e];
        put(0, v);
    } else if constexpr (END == END_GATED_BACKWARD) {
        float a[8 * Q], d[8 * Q];
        {
            float g[8 * Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) read8<XT, WHOLE>(beside[q].a, n, left, g + 8 * q);
            activate_slope(p.act, g, a, d);
        }
        if (p.in[1] != nullptr) {
            float w[8 * Q], x[8 * Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) read8<XT, WHOLE>(beside[q].b, n, left, w + 8 * q);
#pragma unroll
            for (int e = 0; e < 8 * Q; ++e) {
                x[e] = v[e] * a[e];
                d[e] *= w[e];
                a[e] *= w[e];
            }
            put(1, x);
        }
        if (p.out[2] != nullptr) put(2, a);
#pragma unroll
        for (int e = 0; e < 8 * Q; ++e) v[e] *= d[e];
        put(0, v);
    } else {
        if (p.accumulate) {
            float c[8 * Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) read8<XT_F32, WHOLE>(beside[q].c, n, left, c + 8 * q);
#pragma unroll
            for (int e = 0; e < 8 * Q; ++e) v[e] += c[e];
        }
#pragma unroll
        for (int q = 0; q < Q; ++q)
            put8<XT_F32, WHOLE>(p.out[0], (m + q * step) * p.ldo[0] + n, left, v + 8 * q);
    }
}

#endif

}  // namespace pg

#endif
