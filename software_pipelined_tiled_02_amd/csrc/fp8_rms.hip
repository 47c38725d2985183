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
__device__ __forceinline__ void load_w(const void* W, int64_t at, int n, bool w_f32, float (&w)[8]) {
    if (w_f32)
        load8<XT_F32>(W, at, n, w);
    else
        load8<XT>(W, at, n, w);
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
        load8<XT>(a.X, n > 0 ? m * a.ldx + k : 0, n, f[i]);
        if (a.R != nullptr) {
            float r[8];
            load8<XT>(a.R, n > 0 ? m * a.ldr + k : 0, n, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[i][e] = rounded<XT>(f[i][e] + r[e]);
        }
        if (a.H != nullptr && n > 0) store8<XT>(a.H, m * a.ldh + k, n, f[i]);
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
        load_w<XT>(a.W, n > 0 ? k : 0, n, a.w_f32, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * rstd * w[e];
        if (a.Y != nullptr && n > 0) store8<XT>(a.Y, m * a.ldy + k, n, f[i]);
        if (a.Q != nullptr) {
            const float s = block_scale(max16(amax8(f[i])), a.e5m2, a.pow2);
            const i32x2q v = to_fp8x8(f[i], 1.0f / s, a.e5m2);
            if (n > 0) {
                store_fp8x8(a.Q + m * a.ldq + k, n, v);
                if ((t & 15) == 0) a.S[m * a.s_row + (k / kBlock) * a.s_blk] = s;
            }
        }
    }
}

// How a backward pass holds its rows.  kAhead: in registers, the next row
// loaded before the current one's sum, so that two rows per group are on
// their way (8192 x 4096 bf16: 86 us without, 53 with).  kHold: in registers,
// one at a time.  kTwice: read for the sum and again (from the caches) for dx.
// The longer the row, the fewer registers a thread has for each value of it:
// 8192 values and fewer go ahead (16-bit ones up to 12288); a form that spills
// costs more than it gives (4096 x 16384 bf16: 242 us ahead, 116 held).
enum Holding { kAhead, kHold, kTwice };

// Row group g of `groups` takes rows g, g + groups, ...: it keeps its part
// of dw in registers over them and writes it once, to parts[g].
template <int XT, int TPR, int NC, int HOLDING>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rms_backward_kernel(RmsBackwardArgs a) {
    __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    constexpr bool KEEP = HOLDING == kAhead;                 // the weight stays in registers too
    constexpr int NH = HOLDING == kTwice ? 1 : NC;
    const int t = threadIdx.x % TPR;
    const int group = blockIdx.x * RPW + threadIdx.x / TPR;
    if (group >= a.groups) return;                           // whole waves, RPW > 1 only
    struct Row {
        Raw8<XT> dy[NH], h[NH], dh[NH];
        float rstd;
    };
    auto load_part = [&](Row& x, int64_t m, int i, bool with_dh) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k)), q = HOLDING == kTwice ? 0 : i;
        x.dy[q] = load_raw8<XT>(a.DY, n > 0 ? m * a.lddy + k : 0, n);
        x.h[q] = load_raw8<XT>(a.H, n > 0 ? m * a.ldh + k : 0, n);
        if (with_dh && a.DH != nullptr) x.dh[q] = load_raw8<XT>(a.DH, n > 0 ? m * a.lddh + k : 0, n);
    };
    auto load_row = [&](Row& x, int64_t m) {
        x.rstd = a.rstd[m];
        if constexpr (HOLDING != kTwice) {
#pragma unroll
            for (int i = 0; i < NC; ++i) load_part(x, m, i, true);
        }
    };
    auto weight = [&](int i, float (&w)[8]) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
        load_w<XT>(a.W, n > 0 ? k : 0, n, a.w_f32, w);
    };
    float kept[KEEP ? NC : 1][8], dw[NC][8];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        if constexpr (KEEP) weight(i, kept[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
    }
    Row x;
    load_row(x, group);
    int turn = 0;
    for (int64_t m = group; m < a.M; m += a.groups) {
        Row next;
        const bool more = m + a.groups < a.M;
        if (HOLDING == kAhead && more) load_row(next, m + a.groups);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int q = HOLDING == kTwice ? 0 : i;
            if constexpr (HOLDING == kTwice) load_part(x, m, i, false);
            if constexpr (!KEEP) weight(i, kept[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dy = (float)x.dy[q].v[e], h = (float)x.h[q].v[e];
                dw[i][e] += dy * (h * x.rstd);
                dot += dy * kept[KEEP ? i : 0][e] * h;
            }
            if constexpr (HOLDING == kTwice) __builtin_amdgcn_sched_barrier(0);
        }
        dot = row_sum<TPR>(dot, red[turn]);
        turn ^= 1;
        const float c = x.rstd * x.rstd * (dot / (float)a.D);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k)), q = HOLDING == kTwice ? 0 : i;
            float dx[8];
            if constexpr (HOLDING == kTwice) load_part(x, m, i, true);
            if constexpr (!KEEP) weight(i, kept[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dx[e] = x.rstd * ((float)x.dy[q].v[e] * kept[KEEP ? i : 0][e] - (float)x.h[q].v[e] * c);
                if (a.DH != nullptr) dx[e] += (float)x.dh[q].v[e];
            }
            if (n > 0) store8<XT>(a.DX, m * a.lddx + k, n, dx);
            if constexpr (HOLDING == kTwice) __builtin_amdgcn_sched_barrier(0);
        }
        if (more) {
            if constexpr (HOLDING == kAhead) x = next;
            else load_row(x, m + a.groups);
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
        if (n > 0) store8<XT_F32>(a.parts, group * rms_parts_row(a.D) + k, n, dw[i]);
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
    if (k < a.D) {       // (past D, to the row's end, whatever lies there goes into sums that nobody stores)
        const int64_t row = rms_parts_row(a.D);
#pragma unroll 8
        for (int p = g; p < a.groups; p += 64) s += *(const f32x4v*)(a.parts + p * row + k);
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

template <int XT, int TPR, int NC, int HOLDING>
hipError_t backward(const RmsBackwardArgs& a, hipStream_t stream) {
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    if (a.groups > 0) {                  // no rows: dw is zero
        hipLaunchKernelGGL((rms_backward_kernel<XT, TPR, NC, HOLDING>), dim3((unsigned)((a.groups + RPW - 1) / RPW)),
                           dim3(TPR < 256 ? 256 : TPR), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(rms_backward_sum, dim3((unsigned)((a.D + 15) / 16)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int XT>
hipError_t backward_for(const RmsBackwardArgs& a, hipStream_t stream) {
    if (a.D <= 512) return backward<XT, 64, 1, kAhead>(a, stream);
    if (a.D <= 1024) return backward<XT, 64, 2, kAhead>(a, stream);
    if (a.D <= 2048) return backward<XT, 256, 1, kAhead>(a, stream);
    if (a.D <= 4096) return backward<XT, 256, 2, kAhead>(a, stream);
    if (a.D <= 8192) return backward<XT, 512, 2, kAhead>(a, stream);
    if (a.D <= 12288 && XT != XT_F32) return backward<XT, 512, 3, XT == XT_F32 ? kHold : kAhead>(a, stream);
    if (a.D <= 16384) return backward<XT, 1024, 2, kHold>(a, stream);
    return backward<XT, 1024, 4, kTwice>(a, stream);
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
