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
#include "fp8_rms_plan.h"

namespace pg {

namespace {

// Sum over the TPR threads of a row, the same in each (red: one slot per
// wave; a caller in a loop alternates between two).
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {     // TPR > 64: the workgroup's only row
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
__device__ __forceinline__ void load_w(const void* W, int64_t k, int n, bool w_f32, float (&w)[8]) {
    if (w_f32)
        load8<XT_F32>(W, k, k, n, w);
    else
        load8<XT>(W, k, k, n, w);
}

template <int XT, int TPR, int NC>
__global__ void __launch_bounds__(rms_group_threads(TPR)) rms_kernel(RmsArgs a) {
    __shared__ float red[TPR > 64 ? TPR / 64 : 1];
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;          // rows per workgroup
    const int t = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
    if (m >= a.M) return;                                    // RPW > 1 only: whole waves, no barrier follows
    // All loads go out before the first store: h may be x or r, so the compiler
    // keeps the order it finds (8192 x 8192 bf16: 94.1 us chunk by chunk, 91.3
    // so; without a residual 54.3 and 48.4).
    Raw8<XT> x[NC], r[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
        x[i] = fetch8<XT>(a.X, m * a.ldx + k, k, n);
        if (a.R != nullptr) r[i] = fetch8<XT>(a.R, m * a.ldr + k, k, n);
    }
    float f[NC][8];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
        settle8<XT>(x[i], k, n);
        to_f32<XT>(x[i], f[i]);
        if (a.R != nullptr) {
            settle8<XT>(r[i], k, n);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[i][e] = rounded<XT>(f[i][e] + (float)r[i].v[e]);
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
        load_w<XT>(a.W, k, n, a.w_f32, w);
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

// How a backward pass of many rows holds them.  Ahead: in registers, the next
// row loaded before the current one's sum, so that two rows per group are on
// their way (8192 x 4096 bf16: 86 us without, 52 with).  Otherwise one at a
// time: the longer the row, the fewer registers a thread has for each value
// of it, and two rows of 16384 go to scratch (4096 x 16384 bf16: 242 us ahead,
// 112 held).  fp8_rms_plan.h chooses; the launches refuse a row that a form
// does not take.

// Row group g of `groups` takes rows g, g + groups, ...: it keeps its part
// of dw in registers over them and writes it once, to parts[g].
template <int XT, int TPR, int NC, bool AHEAD, bool WHOLE>       // WHOLE: D is a multiple of 8
__global__ void __launch_bounds__(TPR == 64 ? 256 : TPR) rms_backward_kernel(RmsBackwardArgs a) {
    __shared__ float red[2][TPR > 64 ? TPR / 64 : 1];
    constexpr int RPW = TPR == 64 ? 4 : 1;                   // rows of several waves meet at barriers: one each
    constexpr bool KEEP = AHEAD;                             // the weight stays in registers too
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
            const int k = (i * TPR + t) * 8, n = WHOLE ? (k < a.D ? 8 : 0) : min(8, max(0, a.D - k));
            x.dy[i] = fetch8<XT>(a.DY, m * a.lddy + k, k, n);
            x.h[i] = fetch8<XT>(a.H, m * a.ldh + k, k, n);
            if (a.DH != nullptr) x.dh[i] = fetch8<XT>(a.DH, m * a.lddh + k, k, n);
        }
    };
    auto weight = [&](int i, float (&w)[8]) {
        const int k = (i * TPR + t) * 8, n = WHOLE ? (k < a.D ? 8 : 0) : min(8, max(0, a.D - k));
        load_w<XT>(a.W, k, n, a.w_f32, w);
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
        if (AHEAD && more) load_row(next, m + a.groups);
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
            if constexpr (!WHOLE) {
                settle8<XT>(x.dy[i], k, n);
                settle8<XT>(x.h[i], k, n);
            }
            if constexpr (!KEEP) weight(i, kept[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dy = (float)x.dy[i].v[e], h = (float)x.h[i].v[e];
                dw[i][e] += dy * (h * x.rstd);
                dot += dy * kept[KEEP ? i : 0][e] * h;
            }
        }
        dot = row_sum<TPR>(dot, red[turn]);
        turn ^= 1;
        const float c = x.rstd * x.rstd * (dot / (float)a.D);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int k = (i * TPR + t) * 8, n = WHOLE ? (k < a.D ? 8 : 0) : min(8, max(0, a.D - k));
            float dx[8];
            if (!WHOLE && a.DH != nullptr) settle8<XT>(x.dh[i], k, n);
            if constexpr (!KEEP) weight(i, kept[0]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dx[e] = x.rstd * ((float)x.dy[i].v[e] * kept[KEEP ? i : 0][e] - (float)x.h[i].v[e] * c);
                if (a.DH != nullptr) dx[e] += (float)x.dh[i].v[e];
            }
            if (n > 0) store8<XT>(a.DX, m * a.lddx + k, n, dx);
        }
        if (more) {
            if constexpr (AHEAD) x = next;
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

// The other form of the backward pass, for fewer rows and for the longest:
// dw takes only the rows' rstd, which is given, not their sums, so it needs
// nothing from dx.  The first workgroups take a row each (TPR threads per
// row), the others 64 or 128 columns of dw over a part of the rows each: 8 or
// 16 lanes across, the other threads down, their sums added in turn.  dy and h
// are read twice, mostly from the caches, but dw's parts are few, none for
// 512 rows and fewer, which take one launch (bf16 with dh, 16 x 4096: 5.1 us,
// 8.3 in groups and two launches; 512 x 4096: 6.9 and 14.8).
// 64 columns give short rows more workgroups (512 x 1024: 5.6 us against 8.2), 128
// read longer pieces (1024 x 8192: 25 us against 21).
// Where dx takes the place of dy or h the dw workgroups go first, in a launch
// of their own: side by side they would read what a row has overwritten.
template <int XT, int TPR, int NC, int AT_ONCE>      // rows on their way per thread
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) rms_backward_columns(RmsBackwardArgs a, int first) {
    constexpr int T = TPR < 256 ? 256 : TPR, RPW = T / TPR, LANES = columns_lanes(TPR), COLUMNS = LANES * 8, DOWN = T / LANES;
    __shared__ float sums[DOWN][COLUMNS + 4];
    const int row_groups = (a.M + RPW - 1) / RPW, block = (int)blockIdx.x + first;
    if (block >= row_groups) {
        const int c = threadIdx.x % LANES, g = threadIdx.x / LANES;
        const int blocks = (a.D + COLUMNS - 1) / COLUMNS, part = (block - row_groups) / blocks;
        const int k0 = (block - row_groups) % blocks * COLUMNS, k = k0 + c * 8, n = min(8, max(0, a.D - k));
        const int parts = max(1, a.groups), rows = (a.M + parts - 1) / parts;
        const int64_t to = min((int64_t)a.M, (int64_t)(part + 1) * rows);
        float dw[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = 0.0f;
        for (int64_t m0 = (int64_t)part * rows + g; m0 < to; m0 += AT_ONCE * DOWN) {
            Raw8<XT> dy[AT_ONCE], h[AT_ONCE];
            float rstd[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                const int64_t m = m0 + i * DOWN;
                dy[i] = fetch8<XT>(a.DY, m * a.lddy + k, k, m < to ? n : 0);
                h[i] = fetch8<XT>(a.H, m * a.ldh + k, k, m < to ? n : 0);
                rstd[i] = m < to ? a.rstd[m] : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                settle8<XT>(dy[i], k, n);
                settle8<XT>(h[i], k, n);
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[e] += (float)dy[i].v[e] * ((float)h[i].v[e] * rstd[i]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[g][c * 8 + e] = dw[e];
        __syncthreads();
        const int col = k0 + (int)threadIdx.x;
        if (threadIdx.x < COLUMNS && col < a.D) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < DOWN; ++i) s += sums[i][threadIdx.x];
            (a.groups > 0 ? a.parts + part * rms_parts_row(a.D) : a.DW)[col] = s;
        }
        return;
    }
    const int t = threadIdx.x % TPR;
    const int64_t m = (int64_t)block * RPW + threadIdx.x / TPR;
    if (m >= a.M) return;                                    // whole waves, RPW > 1 only
    const float rstd = a.rstd[m];
    float dy[NC][8], h[NC][8];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
        float w[8];
        load8<XT>(a.DY, m * a.lddy + k, k, n, dy[i]);
        load8<XT>(a.H, m * a.ldh + k, k, n, h[i]);
        load_w<XT>(a.W, k, n, a.w_f32, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dy[i][e] *= w[e];
            dot += dy[i][e] * h[i][e];
        }
    }
    dot = row_sum<TPR>(dot, sums[0]);
    const float c = rstd * rstd * (dot / (float)a.D);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int k = (i * TPR + t) * 8, n = min(8, max(0, a.D - k));
        float dx[8], dh[8];
        if (a.DH != nullptr) load8<XT>(a.DH, m * a.lddh + k, k, n, dh);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dx[e] = rstd * (dy[i][e] - h[i][e] * c);
            if (a.DH != nullptr) dx[e] += dh[e];
        }
        if (n > 0) store8<XT>(a.DX, m * a.lddx + k, n, dx);
    }
}

constexpr int form_key(int tpr, int nc) { return 8 * tpr + nc; }

template <int XT, int TPR, int NC>
hipError_t forward(const RmsArgs& a, hipStream_t stream) {
    if (a.D > TPR * NC * 8) return hipErrorInvalidValue;
    hipLaunchKernelGGL((rms_kernel<XT, TPR, NC>), dim3((unsigned)rms_row_groups(a.M, TPR)), dim3(rms_group_threads(TPR)), 0,
                       stream, a);
    return hipGetLastError();
}

template <int XT>
hipError_t forward_for(const RmsArgs& a, hipStream_t stream) {
    const RmsForm f = rms_form(a.M, a.D);
    switch (form_key(f.tpr, f.nc)) {
    case form_key(64, 1): return forward<XT, 64, 1>(a, stream);
    case form_key(64, 2): return forward<XT, 64, 2>(a, stream);
    case form_key(256, 1): return forward<XT, 256, 1>(a, stream);
    case form_key(256, 2): return forward<XT, 256, 2>(a, stream);
    case form_key(256, 4): return forward<XT, 256, 4>(a, stream);
    case form_key(512, 1): return forward<XT, 512, 1>(a, stream);
    case form_key(1024, 1): return forward<XT, 1024, 1>(a, stream);
    case form_key(1024, 2): return forward<XT, 1024, 2>(a, stream);
    case form_key(1024, 4): return forward<XT, 1024, 4>(a, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t sum_parts(const RmsBackwardArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(rms_backward_sum, dim3((unsigned)((a.D + 15) / 16)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int XT, int TPR, int NC, bool AHEAD, bool WHOLE>
hipError_t backward(const RmsBackwardArgs& a, hipStream_t stream) {
    constexpr int RPW = TPR == 64 ? 4 : 1;
    if ((WHOLE && a.D % 8 != 0) || a.D > TPR * NC * 8) return hipErrorInvalidValue;
    hipLaunchKernelGGL((rms_backward_kernel<XT, TPR, NC, AHEAD, WHOLE>), dim3((unsigned)((a.groups + RPW - 1) / RPW)),
                       dim3(TPR * RPW), 0, stream, a);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess ? e : sum_parts(a, stream);
}

template <int XT, int TPR, int NC, int AT_ONCE>
hipError_t launch_columns(const RmsBackwardArgs& a, hipStream_t stream) {
    constexpr int T = rms_group_threads(TPR), COLUMNS = columns_lanes(TPR) * 8;
    if (a.D > TPR * NC * 8) return hipErrorInvalidValue;
    const int rows = (int)rms_row_groups(a.M, TPR);
    const int columns = (a.D + COLUMNS - 1) / COLUMNS * (a.groups > 0 ? a.groups : 1);
    const bool apart = a.in_place && rows > 0;
    const auto launch = [&](int workgroups, int first) {
        hipLaunchKernelGGL((rms_backward_columns<XT, TPR, NC, AT_ONCE>), dim3((unsigned)workgroups), dim3(T), 0, stream,
                           a, first);
        return hipGetLastError();
    };
    hipError_t e = hipSuccess;
    if (apart) e = launch(columns, rows);
    if (e == hipSuccess) e = launch(apart ? rows : rows + columns, 0);
    return e != hipSuccess || a.groups == 0 ? e : sum_parts(a, stream);
}

// Eight 16-bit rows at once where there are as many (512 x 4096: 6.3 us, 7.7
// with four); up to 128 rows, four take them all (1 x 4096 in a graph: 4.5 us with
// eight, 3.2 with four).
template <int XT, int TPR, int NC>
hipError_t backward_columns(const RmsBackwardArgs& a, hipStream_t stream) {
    if constexpr (XT != XT_F32 && columns_lanes(TPR) == 8)
        if (a.M > 128) return launch_columns<XT, TPR, NC, 8>(a, stream);
    return launch_columns<XT, TPR, NC, 4>(a, stream);
}

template <int XT>
hipError_t backward_for(const RmsBackwardArgs& a, const RmsBackwardForm& f, hipStream_t stream) {
    const int key = form_key(f.tpr, f.nc);
    if (f.by_columns) {
        switch (key) {
        case form_key(64, 1): return backward_columns<XT, 64, 1>(a, stream);
        case form_key(64, 2): return backward_columns<XT, 64, 2>(a, stream);
        case form_key(256, 1): return backward_columns<XT, 256, 1>(a, stream);
        case form_key(256, 2): return backward_columns<XT, 256, 2>(a, stream);
        case form_key(512, 2): return backward_columns<XT, 512, 2>(a, stream);
        case form_key(1024, 2): return backward_columns<XT, 1024, 2>(a, stream);
        case form_key(1024, 4): return backward_columns<XT, 1024, 4>(a, stream);
        default: return hipErrorInvalidValue;
        }
    }
    switch (key) {
    case form_key(64, 1): return backward<XT, 64, 1, true, false>(a, stream);
    case form_key(128, 1): return backward<XT, 128, 1, true, false>(a, stream);
    case form_key(256, 1): return backward<XT, 256, 1, true, false>(a, stream);
    case form_key(512, 1): return backward<XT, 512, 1, true, false>(a, stream);
    case form_key(1024, 1): return backward<XT, 1024, 1, true, false>(a, stream);
    case form_key(512, 3):
        if constexpr (XT != XT_F32) return backward<XT, 512, 3, true, false>(a, stream);
        else return hipErrorInvalidValue;
    case form_key(1024, 2):
        if (f.whole) return backward<XT, 1024, 2, false, true>(a, stream);
        if constexpr (XT == XT_F32) return backward<XT, 1024, 2, false, false>(a, stream);
        else return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_rms(const RmsArgs& a, int xtype, hipStream_t stream) {
    switch (xtype) {
    case XT_F16: return forward_for<XT_F16>(a, stream);
    case XT_BF16: return forward_for<XT_BF16>(a, stream);
    default: return forward_for<XT_F32>(a, stream);
    }
}

hipError_t launch_rms_backward(const RmsBackwardArgs& a, const RmsBackwardForm& form, int xtype, hipStream_t stream) {
    switch (xtype) {
    case XT_F16: return backward_for<XT_F16>(a, form, stream);
    case XT_BF16: return backward_for<XT_BF16>(a, form, stream);
    default: return backward_for<XT_F32>(a, form, stream);
    }
}

}  // namespace pg
