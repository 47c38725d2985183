// fp8_rms.hip -- root-mean-square norm with the residual's addition and an
// 8-bit output, and its backward pass.
//
//   forward:  h = x + residual, rounded to x's type (what the residual
//             stream keeps is what is normalised); rstd = 1 / sqrt(mean h^2 +
//             eps); y = h rstd w; y in blocks of 128 to 8 bits.
//   backward: dx = dh + rstd (w dy - h rstd^2 mean(w dy h)),
//             dw = sum over rows of dy h rstd.
//
// Both are bound by memory, so a row is read once and stays in registers
// (fp32) between its statistics and its output: TPR threads hold it, 8
// consecutive values per thread and step, NC steps.  A block of 128 is 16
// neighbouring lanes.
#include "fp8_common.h"

namespace pg {

namespace {

// Sum over the TPR threads of a row, the same in each (red: one slot per
// wave; a caller in a loop alternates between two).
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
    x = sum64(x);
    if constexpr (TPR > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) red[wave] = x;
        __syncthreads();
        x = 0.0f;
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) x += red[w];
    }
    return x;
}

template <int XT>
__device__ __forceinline__ void load_w(const void* W, int64_t at, int n, bool vec, bool w_f32, float (&w)[8]) {
    if (w_f32)
        load8<XT_F32>(W, at, n, vec, w);
    else
        load8<XT>(W, at, n, vec, w);
}

template <int XT, int TPR, int NC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rms_kernel(RmsArgs a) {
    __shared__ float red[TPR > 64 ? TPR / 64 : 1];
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;          // rows per workgroup
    const int t = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
    if (m >= a.M) return;                                    // RPW > 1 only: whole waves, no barrier follows
    float f[NC][8];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t k = ((int64_t)i * TPR + t) * 8;
        const int n = (int)min((int64_t)8, max((int64_t)0, a.D - k));
        load8<XT>(a.X, n > 0 ? m * a.ldx + k : 0, n, a.vec, f[i]);
        if (a.R != nullptr) {
            float r[8];
            load8<XT>(a.R, n > 0 ? m * a.ldr + k : 0, n, a.vec, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[i][e] = rounded<XT>(f[i][e] + r[e]);
        }
        if (a.H != nullptr && n > 0) store8<XT>(a.H, m * a.ldh + k, n, a.vec, f[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sq += f[i][e] * f[i][e];
    }
    sq = row_sum<TPR>(sq, red);
    const float rstd = 1.0f / sqrtf(sq / (float)a.D + a.eps);
    if (a.rstd != nullptr && t == 0) a.rstd[m] = rstd;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int64_t k = ((int64_t)i * TPR + t) * 8;
        const int n = (int)min((int64_t)8, max((int64_t)0, a.D - k));
        float w[8];
        load_w<XT>(a.W, n > 0 ? k : 0, n, a.vec, a.w_f32, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * rstd * w[e];
        if (a.Y != nullptr && n > 0) store8<XT>(a.Y, m * a.ldy + k, n, a.vec, f[i]);
        if (a.Q != nullptr) {
            const float s = block_scale(max16(amax8(f[i])), a.e5m2, a.pow2);
            const i32x2q v = to_fp8x8(f[i], 1.0f / s, a.e5m2);
            if (n > 0) {
                store_fp8x8(a.Q + m * a.ldq + k, n, a.vec, v);
                if ((t & 15) == 0) a.S[m * a.s_row + (k / kBlock) * a.s_blk] = s;
            }
        }
    }
}

// Row group g of `groups` takes rows g, g + groups, ...: it keeps its part
// of dw in registers over them and writes it once, to parts[g].  AHEAD: the
// next row is loaded before the current one's sum, so that two rows per
// group are on their way (8192 x 4096: 86 us without it, 53 with it).  Rows of more
// than 8192 values leave a thread no registers for that, and have loads enough in flight.
template <int XT, int TPR, int NC, bool AHEAD>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rms_backward_kernel(RmsBackwardArgs a) {
    __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    const int t = threadIdx.x % TPR;
    const int group = blockIdx.x * RPW + threadIdx.x / TPR;
    if (group >= a.groups) return;                           // whole waves, RPW > 1 only
    struct Row {
        Raw8<XT> dy[NC], h[NC], dh[NC];
        float rstd;
    };
    auto load_row = [&](Row& x, int64_t m) {
        x.rstd = a.rstd[m];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
            x.dy[i] = load_raw8<XT>(a.DY, n > 0 ? m * a.lddy + k : 0, n, a.vec);
            x.h[i] = load_raw8<XT>(a.H, n > 0 ? m * a.ldh + k : 0, n, a.vec);
            if (a.DH != nullptr) x.dh[i] = load_raw8<XT>(a.DH, n > 0 ? m * a.lddh + k : 0, n, a.vec);
        }
    };
    float w[NC][8], dw[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
        load_w<XT>(a.W, n > 0 ? k : 0, n, a.vec, a.w_f32, w[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
    }
    Row x;
    load_row(x, group);
    int turn = 0;
    for (int64_t m = group; m < a.M; m += a.groups) {
        Row next;
        const bool more = m + a.groups < a.M;
        if (AHEAD && more) load_row(next, m + a.groups);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dy = (float)x.dy[i].v[e], h = (float)x.h[i].v[e];
                dw[i][e] += dy * (h * x.rstd);
                dot += dy * w[i][e] * h;
            }
        dot = row_sum<TPR>(dot, red[turn]);
        turn ^= 1;
        const float c = x.rstd * x.rstd * (dot / (float)a.D);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
            float dx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dx[e] = x.rstd * ((float)x.dy[i].v[e] * w[i][e] - (float)x.h[i].v[e] * c);
                if (a.DH != nullptr) dx[e] += (float)x.dh[i].v[e];
            }
            if (n > 0) store8<XT>(a.DX, m * a.lddx + k, n, a.vec, dx);
        }
        if (more) {
            if constexpr (AHEAD) x = next;
            else load_row(x, m + a.groups);
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
        // parts' rows are D values: on 16 bytes where D is a multiple of 4
        if (n > 0) store8<XT_F32>(a.parts, (int64_t)group * a.D + k, n, (a.D & 3) == 0, dw[i]);
    }
}

// dw = the sum of the groups' parts, in a fixed order: 16 columns per
// workgroup, 64 threads per 4 columns over the groups (64 g-th, each taking
// every 64th part), then their sums in turn.
__global__ void __launch_bounds__(256) rms_backward_sum(RmsBackwardArgs a) {
    typedef float f32x4v __attribute__((ext_vector_type(4)));
    __shared__ f32x4v red[64][4];
    const int c = threadIdx.x & 3, g = threadIdx.x >> 2;
    const int k = blockIdx.x * 16 + c * 4;
    f32x4v s = {0.0f, 0.0f, 0.0f, 0.0f};
    if ((a.D & 3) == 0) {
        if (k < a.D) {
#pragma unroll 8
            for (int p = g; p < a.groups; p += 64) s += *(const f32x4v*)(a.parts + (int64_t)p * a.D + k);
        }
    } else {
        for (int p = g; p < a.groups; p += 64)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k + e < a.D) s[e] += a.parts[(int64_t)p * a.D + k + e];
    }
    red[g][c] = s;
    __syncthreads();
    if (threadIdx.x < 16 && blockIdx.x * 16 + threadIdx.x < a.D) {
        const float* col = (const float*)red + threadIdx.x;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) sum += col[i * 16];
        a.DW[blockIdx.x * 16 + threadIdx.x] = sum;
    }
}

template <int XT, int TPR, int NC>
hipError_t forward(const RmsArgs& a, hipStream_t stream) {
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    hipLaunchKernelGGL((rms_kernel<XT, TPR, NC>), dim3((unsigned)((a.M + RPW - 1) / RPW)), dim3(TPR < 256 ? 256 : TPR),
                       0, stream, a);
    return hipGetLastError();
}

template <int XT>
hipError_t forward_for(const RmsArgs& a, hipStream_t stream) {
    if (a.D <= 512) return forward<XT, 64, 1>(a, stream);
    if (a.D <= 1024) return forward<XT, 64, 2>(a, stream);
    if (a.D <= 2048) return forward<XT, 256, 1>(a, stream);
    if (a.D <= 4096) return forward<XT, 256, 2>(a, stream);
    if (a.D <= 8192) return forward<XT, 256, 4>(a, stream);
    if (a.D <= 16384) return forward<XT, 1024, 2>(a, stream);
    return forward<XT, 1024, 4>(a, stream);
}

template <int XT, int TPR, int NC, bool AHEAD>
hipError_t backward(const RmsBackwardArgs& a, hipStream_t stream) {
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    if (a.groups > 0) {                  // no rows: dw is zero
        hipLaunchKernelGGL((rms_backward_kernel<XT, TPR, NC, AHEAD>), dim3((unsigned)((a.groups + RPW - 1) / RPW)),
                           dim3(TPR < 256 ? 256 : TPR), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(rms_backward_sum, dim3((unsigned)((a.D + 15) / 16)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int XT>
hipError_t backward_for(const RmsBackwardArgs& a, hipStream_t stream) {
    if (a.D <= 512) return backward<XT, 64, 1, true>(a, stream);
    if (a.D <= 1024) return backward<XT, 64, 2, true>(a, stream);
    if (a.D <= 2048) return backward<XT, 256, 1, true>(a, stream);
    if (a.D <= 4096) return backward<XT, 256, 2, true>(a, stream);
    if (a.D <= 8192) return backward<XT, 512, 2, true>(a, stream);
    if (a.D <= 16384) return backward<XT, 1024, 2, false>(a, stream);
    return backward<XT, 1024, 4, false>(a, stream);
}

}  // namespace

int rms_backward_groups(int64_t M, int64_t D, int num_cus) {
    // two workgroups of 256 threads per CU (one of 1024), each with as many
    // groups as it holds rows at a time
    const int64_t most = (int64_t)num_cus * (D <= 1024 ? 8 : D <= 8192 ? 2 : 1);
    return (int)(M < most ? M : most);
}

hipError_t launch_rms(const RmsArgs& a, int xtype, hipStream_t stream) {
    switch (xtype) {
    case XT_F16: return forward_for<XT_F16>(a, stream);
    case XT_BF16: return forward_for<XT_BF16>(a, stream);
    default: return forward_for<XT_F32>(a, stream);
    }
}

hipError_t launch_rms_backward(const RmsBackwardArgs& a, int xtype, hipStream_t stream) {
    switch (xtype) {
    case XT_F16: return backward_for<XT_F16>(a, stream);
    case XT_BF16: return backward_for<XT_BF16>(a, stream);
    default: return backward_for<XT_F32>(a, stream);
    }
}

}  // namespace pg
