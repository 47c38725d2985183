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
    int32_t products;        // added into one sum: 1 or 2
    int32_t tiles_m, tiles_n;
    int32_t act, bias_f32, accumulate;
};

// Tile classes: the workgroup's part of the sums (gated: half of the columns are
// the second product's), and its waves.
enum LinearTile : int { LINEAR_TILE_256 = 0, LINEAR_TILE_128 = 1, LINEAR_TILE_64 = 2, LINEAR_TILE_COUNT = 3 };
struct LinearShape { int bm, bn, waves; };
constexpr LinearShape linear_shape(int t) {
    return t == LINEAR_TILE_256 ? LinearShape{256, 256, 8} : t == LINEAR_TILE_128 ? LinearShape{128, 128, 8} : LinearShape{64, 64, 4};
}

// The kernel for a call: XT_F16 or XT_BF16, a tile class, and whether all
// rows of the factors start on 16 bytes (NULL: the class needs that).
const void* linear_rc_kernel(int xt, int tile, bool rows16);
const void* linear_rr_kernel(int xt, int tile, bool rows16);
const void* gated_kernel(int xt, int tile, bool rows16);
const void* gated_backward_kernel(int xt, int tile, bool rows16);
const void* weight_gradient_kernel(int xt, int tile, bool rows16, bool sums);

#if defined(__HIPCC__)

// The distribution function of the normal distribution at -|z|, from
// e = exp(-z^2 / 2): e times half of exp(x^2) erfc(x), x = |z| / sqrt 2, which is
// a polynomial in t = 1 / (1 + 0.54 x) to 4e-6 (fitted here, by least
// squares with weights moved to the largest relative errors).  5e-6 off for |z| <
// 6 in fp32, a hundredth of fp16's half step; the far tail keeps its relative error.
__device__ __forceinline__ float normal_tail(float z, float e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.381837662f, fabsf(z), 1.0f));
    float p = fmaf(0.0480623953f, t, -0.155210704f);
    p = fmaf(p, t, 0.105571732f);
    p = fmaf(p, t, 0.063943103f);
    p = fmaf(p, t, 0.133146182f);
    p = fmaf(p, t, 0.152152315f);
    p = fmaf(p, t, 0.152334273f);
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
__device__ __forceinline__ float logistic(float z, Logistic l) {      // |z| <= 128
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * fmaf(l.c3 * z, z, l.c1)));
}

// Eight values through the activation.  The branches are the same for a whole
// launch.  A NaN stays one.
__device__ __forceinline__ void activate(int act, float (&v)[8]) {
    if (act == ACT_NONE) return;
    if (act == ACT_RELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] < 0.0f ? 0.0f : v[e];
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float q = normal_tail(v[e], __builtin_amdgcn_exp2f(-0.721347520f * v[e] * v[e]));
            v[e] *= v[e] > 0.0f ? 1.0f - q : q;
        }
    } else {
        const Logistic l = logistic_of(act);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= logistic(within128(v[e]), l);
    }
}

// The activation a and its derivative d at eight values.  The derivative past |z|
// = 128 is taken there: 0 or 1 in fp32.  A NaN stays one in both.
__device__ __forceinline__ void activate_slope(int act, const float (&z)[8], float (&a)[8], float (&d)[8]) {
    if (act == ACT_NONE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) { a[e] = z[e]; d[e] = 1.0f; }
    } else if (act == ACT_RELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            a[e] = z[e] < 0.0f ? 0.0f : z[e];
            d[e] = z[e] > 0.0f ? 1.0f : z[e] <= 0.0f ? 0.0f : z[e];
        }
    } else if (act == ACT_GELU) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = within128(z[e]);
            const float x = __builtin_amdgcn_exp2f(-0.721347520f * c * c);
            const float q = normal_tail(c, x), p = c > 0.0f ? 1.0f - q : q;
            a[e] = z[e] * p;
            d[e] = z[e] == z[e] ? fmaf(0.398942280f * c, x, p) : z[e];
        }
    } else {
        const Logistic l = logistic_of(act);
        const float k1 = -0.693147181f * l.c1, k3 = -2.07944154f * l.c3;        // q' = k1 + k3 z^2, back from base 2
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = within128(z[e]);
            const float s = logistic(c, l);
            a[e] = z[e] * s;
            d[e] = z[e] == z[e] ? fmaf(c * s * (1.0f - s), fmaf(k3 * c, c, k1), s) : z[e];
        }
    }
}

// What an ending reads beside the sums, for eight neighbouring outputs.
template <int XT, int END>
struct Beside { Raw8<XT> a, b; };

template <int XT, int END>
__device__ __forceinline__ Beside<XT, END> fetch_beside(const LinearArgs& p, int64_t m, int64_t n) {
    Beside<XT, END> r;
    const int left = p.N - (int)n;
    if constexpr (END == END_LINEAR || END == END_GATED_BACKWARD)
        if (p.in[0] != nullptr) r.a = fetch8<XT>(p.in[0], m * p.ldi[0] + n, n, left);
    if constexpr (END == END_GATED_BACKWARD)
        if (p.in[1] != nullptr) r.b = fetch8<XT>(p.in[1], m * p.ldi[1] + n, n, left);
    return r;
}

// v += bias.
template <int XT>
__device__ __forceinline__ void add_bias(const LinearArgs& p, int which, int64_t n, float (&v)[8]) {
    if (p.bias[which] == nullptr) return;
    float b[8];
    const int left = p.N - (int)n;
    if (p.bias_f32) load8<XT_F32>(p.bias[which], n, n, left, b);
    else load8<XT>(p.bias[which], n, n, left, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += b[e];
}

// The ending for outputs (m, n .. n + 7), m < M, n < N: v holds their sums,
// u (gated) the second product's.
template <int XT, int END>
__device__ __forceinline__ void finish8(const LinearArgs& p, int64_t m, int64_t n, Beside<XT, END>& beside, float (&v)[8],
                                        float (&u)[8]) {
    const int left = p.N - (int)n;
    if constexpr (END == END_LINEAR) {
        add_bias<XT>(p, 0, n, v);
        if (p.out[1] != nullptr) store8<XT>(p.out[1], m * p.ldo[1] + n, left, v);
        activate(p.act, v);
        if (p.in[0] != nullptr) {
            float r[8];
            settle8<XT>(beside.a, n, left);
            to_f32<XT>(beside.a, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += r[e];
        }
        store8<XT>(p.out[0], m * p.ldo[0] + n, left, v);
    } else if constexpr (END == END_GATED) {
        add_bias<XT>(p, 0, n, v);
        add_bias<XT>(p, 1, n, u);
        if (p.out[1] != nullptr) {
            store8<XT>(p.out[1], m * p.ldo[1] + n, left, v);
            store8<XT>(p.out[2], m * p.ldo[2] + n, left, u);
        }
        activate(p.act, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= u[e];
        store8<XT>(p.out[0], m * p.ldo[0] + n, left, v);
    } else if constexpr (END == END_GATED_BACKWARD) {
        float g[8], a[8], d[8];
        settle8<XT>(beside.a, n, left);
        to_f32<XT>(beside.a, g);
        activate_slope(p.act, g, a, d);
        if (p.in[1] != nullptr) {
            float w[8], x[8];
            settle8<XT>(beside.b, n, left);
            to_f32<XT>(beside.b, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) { x[e] = v[e] * a[e]; d[e] *= w[e]; a[e] *= w[e]; }
            store8<XT>(p.out[1], m * p.ldo[1] + n, left, x);
        }
        if (p.out[2] != nullptr) store8<XT>(p.out[2], m * p.ldo[2] + n, left, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= d[e];
        store8<XT>(p.out[0], m * p.ldo[0] + n, left, v);
    } else {
        if (p.accumulate) {
            float c[8];
            load8<XT_F32>(p.out[0], m * p.ldo[0] + n, n, left, c);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += c[e];
        }
        store8<XT_F32>(p.out[0], m * p.ldo[0] + n, left, v);
    }
}

#endif

}  // namespace pg

#endif
