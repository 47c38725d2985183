// linear_abi.hip -- the C ABI of the feed-forward operators
// (include/pipegemm.h): argument checks, choice of kernel, launch.  Host code
// only.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "pipegemm.h"
#include "handle.h"
#include "linear_common.h"

namespace {

constexpr int kDefaultCus = 256;  // MI355X; used when no device is at hand

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0; }
bool is_half(int t) { return t == GEMM_F16 || t == GEMM_BF16; }
bool is_act(int a) { return a >= GEMM_ACT_NONE && a <= GEMM_ACT_SILU; }
bool is_form(int f) { return f >= GEMM_FORM_LINEAR_RC && f <= GEMM_FORM_WEIGHT_GRADIENT; }
bool is_pair(int f) { return f == GEMM_FORM_LINEAR_RC_PAIR || f == GEMM_FORM_LINEAR_RR_PAIR; }

// A factor of a product: `rows` rows of `cols` values, K along them (`inside`)
// or across.
struct Operand {
    const void* p;
    int64_t ld, rows, cols;
    bool inside;
    // Of a single row no distance counts, and the kernels' offsets are formed with the row's own length.
    int64_t step() const { return rows > 1 ? ld : (cols + 7) / 8 * 8; }
};

// Whether all of a factor's rows start on 16 bytes: the others' last K-tiles go through registers.
bool rows16(const Operand& o) { return aligned(o.p, 16) && o.step() % 8 == 0; }

// extra: a second product (linear), sums of DC's columns (weight gradients).
const void* kernel(int form, int dtype, int tile, bool extra) {
    const int xt = dtype == GEMM_BF16 ? pg::XT_BF16 : pg::XT_F16;
    switch (form) {
    case GEMM_FORM_LINEAR_RC: return pg::linear_rc_kernel(xt, tile, extra);
    case GEMM_FORM_LINEAR_RR: return pg::linear_rr_kernel(xt, tile, extra);
    case GEMM_FORM_GATED: return pg::gated_kernel(xt, tile);
    case GEMM_FORM_GATED_BACKWARD: return pg::gated_backward_kernel(xt, tile);
    default: return pg::weight_gradient_kernel(xt, tile, extra);
    }
}

// Microseconds that the classes take: for a K-tile when few workgroups are there,
// and when every CU has all that fit (`resident`); for the start and the ending of
// a workgroup.  Fitted to 5000 times of 630 calls of all forms (1 to 8192 rows, 64 to
// 8192 columns and depth, factors from HBM).  Rows on 2 bytes were not fitted by
// themselves since they go straight into LDS: they take the factor of rows on 4.  Over
// 300 other calls of the kernels as they are the class of the least time takes 0.7%
// (rows on 16 bytes), 3.1% (on 4) and 1.7% (on 2) longer than the best one on average,
// 1.6 times at worst; with the largest class that gives every CU a workgroup it was
// 17% (factors in the caches), and three times as long at worst.  64 x 8192 x 8192:
// 64x32 31.8 us, 32x32 41.4; 1024 x 4096 x 4096: 128x128 38, 256x256 78; 1 x 4096 x
// 4096: 16x16 8.6, 64x64 25.8.
struct Cost { double few, all, ends; int resident; };
constexpr Cost kCost[pg::LINEAR_TILE_COUNT] = {{0.95, 1.80, 9.8, 1}, {0.60, 0.99, 5.8, 1}, {0.35, 0.63, 3.9, 1},
                                               {0.20, 0.67, 2.1, 3}, {0.79, 1.16, 2.9, 1}, {0.60, 0.91, 2.3, 1},
                                               {0.85, 1.20, 1.7, 1}, {0.63, 0.82, 1.9, 1}, {0.52, 0.63, 1.7, 1}};

double linear_time(int tile, int form, bool r16, int64_t tiles, int64_t k_tiles, int num_cus) {
    const Cost& c = kCost[tile];
    const bool waves = pg::linear_few_tile(tile);            // (each has K-tiles of its own)
    // factors with K outside are read by the transposing reads; rows that start inside lines touch more of these
    double k = form == GEMM_FORM_LINEAR_RC || form == GEMM_FORM_GATED ? 1.0 : 1.08;
    k *= r16 ? 1.0 : 1.55;
    const double ends = c.ends * (form == GEMM_FORM_GATED_BACKWARD ? 1.6 : 1.0);
    const int64_t own = waves ? ceil_div(k_tiles, pg::linear_shape(tile).waves) : k_tiles;
    const int64_t slots = (int64_t)c.resident * num_cus, rounds = tiles / slots, rest = tiles % slots;
    double time = (double)rounds * (ends + (double)own * k * c.all);
    if (rest > 0) time += ends + (double)own * k * (c.few + (c.all - c.few) * (double)rest / (double)slots);
    return time;
}

struct Plan {
    gemm_linear_info_t info;
    const void* fn;
    int64_t tiles_m, tiles_n;
};

// The kernel for M x N sums over K (weight gradients: M and N are the weight's
// rows and columns, K the tokens).  No HIP call.
int plan_sums(int form, int64_t M, int64_t N, int64_t K, int dtype, bool r16, bool extra, int tile, int num_cus, Plan* plan) {
    const bool gated = form == GEMM_FORM_GATED;
    auto tiles = [&](int t) {
        const pg::LinearShape sh = pg::linear_shape(t);
        return ceil_div(M, sh.bm) * ceil_div(N, gated ? sh.bn / 2 : sh.bn);
    };
    // a launch has fewer than 2^32 threads
    auto fits = [&](int t) { return tiles(t) < ((int64_t)1 << 32) / (64 * pg::linear_shape(t).waves); };
    int tc = tile;
    if (tc == GEMM_LINEAR_TILE_AUTO) {
        double best = 0.0;
        for (int t = 0; t < pg::LINEAR_TILE_COUNT; ++t) {
            if (kernel(form, dtype, t, extra) == nullptr || !fits(t)) continue;
            const int64_t products = extra && form <= GEMM_FORM_LINEAR_RR ? 2 : 1;
            const double time = linear_time(t, form, r16, tiles(t), products * ceil_div(K, 64), num_cus);
            if (tc == GEMM_LINEAR_TILE_AUTO || time < best) {
                tc = t;
                best = time;
            }
        }
    }
    if (tc == GEMM_LINEAR_TILE_AUTO || !fits(tc)) return GEMM_ERR_UNSUPPORTED;
    plan->fn = kernel(form, dtype, tc, extra);
    if (plan->fn == nullptr) return GEMM_ERR_UNSUPPORTED;
    const pg::LinearShape sh = pg::linear_shape(tc);
    const bool any = M > 0 && N > 0;
    plan->tiles_m = any ? ceil_div(M, sh.bm) : 0;
    plan->tiles_n = any ? ceil_div(N, gated ? sh.bn / 2 : sh.bn) : 0;
    const int64_t grid = plan->tiles_m * plan->tiles_n;
    gemm_linear_info_t& in = plan->info;
    memset(&in, 0, sizeof in);
    in.tile = tc;
    in.block_m = sh.bm;
    in.block_n = gated ? sh.bn / 2 : sh.bn;
    in.threads = 64 * sh.waves;
    in.rows16 = r16 ? 1 : 0;
    in.grid = grid;
    in.k_tiles = ceil_div(K, 64);
    return GEMM_OK;
}

// Checks of sizes that all forms share.
int check_sizes(int64_t M, int64_t N, int64_t K, int dtype, int tile) {
    if (!is_half(dtype) || tile < GEMM_LINEAR_TILE_AUTO || tile >= pg::LINEAR_TILE_COUNT) return GEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
    if (M > INT_MAX - 512 || N > INT_MAX - 512 || K > INT_MAX - 512) return GEMM_ERR_UNSUPPORTED;
    return GEMM_OK;
}
int check_factor(const Operand& o) {
    if (o.p == nullptr || o.ld < o.cols) return GEMM_ERR_INVALID_ARG;
    if (!aligned(o.p, 2)) return GEMM_ERR_ALIGNMENT;
    return GEMM_OK;
}
// A tile's 32-bit offsets: K along the rows, of up to 256 rows that are there;
// across them, of 64 rows of K whether they are there or not (those that are
// not have to lie past the last one's end).
bool factor_fits(const Operand& o) {
    const int64_t rows = o.inside ? std::min<int64_t>(o.rows, 256) : 64;
    return (__int128)rows * o.step() * 2 + 1024 <= (int64_t)1 << 31;
}
// Rows of results, or of what is read beside the sums.
int check_rows(const void* p, int64_t ld, int64_t N, int size, bool needed) {
    if (p == nullptr) return needed ? GEMM_ERR_INVALID_ARG : GEMM_OK;
    if (ld < N) return GEMM_ERR_INVALID_ARG;
    return aligned(p, size) ? GEMM_OK : GEMM_ERR_ALIGNMENT;
}
int first_of(std::initializer_list<int> codes) {
    for (int c : codes)
        if (c != GEMM_OK) return c;
    return GEMM_OK;
}

int launch(gemm_handle_t h, const Plan& plan, pg::LinearArgs& a, void* stream) {
    a.tiles_m = (int32_t)plan.tiles_m;
    a.tiles_n = (int32_t)plan.tiles_n;
    a.apart = plan.info.rows16 ? 0 : 1;
    void* kargs[] = {&a};
    return pg::on_device(h, [&] {
        const hipError_t e = hipLaunchKernel(plan.fn, dim3((unsigned)plan.info.grid), dim3((unsigned)plan.info.threads), kargs, 0,
                                             (hipStream_t)stream);
        return e == hipSuccess ? hipGetLastError() : e;
    });
}

}  // namespace

extern "C" {

int gemm_query_linear(int form, int64_t M, int64_t N, int64_t K, int dtype, int rows_on_16, int tile, gemm_linear_info_t* info) {
    const bool pair = is_pair(form);
    if (pair) form -= GEMM_FORM_LINEAR_RC_PAIR - GEMM_FORM_LINEAR_RC;
    if (info == nullptr || !is_form(form) || (rows_on_16 != 0 && rows_on_16 != 1)) return GEMM_ERR_INVALID_ARG;
    const int rc = check_sizes(M, N, K, dtype, tile);
    if (rc != GEMM_OK) return rc;
    Plan plan;
    const bool weight = form == GEMM_FORM_WEIGHT_GRADIENT;
    const int got = plan_sums(form, weight ? N : M, weight ? K : N, weight ? M : K, dtype, rows_on_16 == 1, pair, tile, kDefaultCus,
                              &plan);
    if (got == GEMM_OK) *info = plan.info;
    return got;
}

int gemm_linear(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int layout, int activation, int bias_dtype,
                int tile, const void* A, int64_t lda, const void* B, int64_t ldb, const void* A2, int64_t lda2,
                const void* B2, int64_t ldb2, const void* bias, const void* R, int64_t ldr, void* Z, int64_t ldz, void* C,
                int64_t ldc, void* stream) {
    if (h == nullptr || !is_act(activation)) return GEMM_ERR_INVALID_ARG;
    if (layout != GEMM_LAYOUT_RC && layout != GEMM_LAYOUT_RR) return GEMM_ERR_INVALID_ARG;
    int rc = check_sizes(M, N, K, dtype, tile);
    if (rc != GEMM_OK) return rc;
    if (bias != nullptr && bias_dtype != GEMM_F32 && bias_dtype != dtype) return GEMM_ERR_INVALID_ARG;
    if ((A2 == nullptr) != (B2 == nullptr)) return GEMM_ERR_INVALID_ARG;
    const bool any = M > 0 && N > 0, reads = any && K > 0, rr = layout == GEMM_LAYOUT_RR;
    const int products = A2 != nullptr ? 2 : 1;
    const Operand o[4] = {{A, lda, M, K, true}, {B, ldb, rr ? K : N, rr ? N : K, !rr},
                          {A2, lda2, M, K, true}, {B2, ldb2, rr ? K : N, rr ? N : K, !rr}};
    bool r16 = true;
    if (reads)
        for (int i = 0; i < 2 * products; ++i) {
            if ((rc = check_factor(o[i])) != GEMM_OK) return rc;
            if (!factor_fits(o[i])) return GEMM_ERR_UNSUPPORTED;
            r16 = r16 && rows16(o[i]);
        }
    if (!any) return GEMM_OK;
    rc = first_of({check_rows(R, ldr, N, 2, false), check_rows(Z, ldz, N, 2, false), check_rows(C, ldc, N, 2, true)});
    if (rc != GEMM_OK) return rc;
    if (bias != nullptr && !aligned(bias, bias_dtype == GEMM_F32 ? 4 : 2)) return GEMM_ERR_ALIGNMENT;
    Plan plan;
    rc = plan_sums(rr ? GEMM_FORM_LINEAR_RR : GEMM_FORM_LINEAR_RC, M, N, K, dtype, r16, products == 2, tile, h->num_cus, &plan);
    if (rc != GEMM_OK) return rc;
    pg::LinearArgs a;
    memset(&a, 0, sizeof a);
    for (int q = 0; q < 2; ++q) {
        a.A[q] = o[2 * q].p;
        a.lda[q] = reads ? o[2 * q].step() : 0;
        a.B[q] = o[2 * q + 1].p;
        a.ldb[q] = reads ? o[2 * q + 1].step() : 0;
    }
    a.in[0] = R;
    a.ldi[0] = ldr;
    a.out[0] = C;
    a.ldo[0] = ldc;
    a.out[1] = Z;
    a.ldo[1] = ldz;
    a.bias[0] = bias;
    a.bias_f32 = bias_dtype == GEMM_F32;
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.act = activation;
    return launch(h, plan, a, stream);
}

int gemm_gated(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int activation, int bias_dtype, int tile,
               const void* X, int64_t ldx, const void* WG, int64_t ldwg, const void* WU, int64_t ldwu, const void* BG,
               const void* BU, void* G, int64_t ldg, void* U, int64_t ldu, void* H, int64_t ldh, void* stream) {
    if (h == nullptr || !is_act(activation)) return GEMM_ERR_INVALID_ARG;
    int rc = check_sizes(M, N, K, dtype, tile);
    if (rc != GEMM_OK) return rc;
    if ((BG != nullptr || BU != nullptr) && bias_dtype != GEMM_F32 && bias_dtype != dtype) return GEMM_ERR_INVALID_ARG;
    if ((G == nullptr) != (U == nullptr)) return GEMM_ERR_INVALID_ARG;
    const bool any = M > 0 && N > 0, reads = any && K > 0;
    const Operand o[3] = {{X, ldx, M, K, true}, {WG, ldwg, N, K, true}, {WU, ldwu, N, K, true}};
    bool r16 = true;
    if (reads)
        for (int i = 0; i < 3; ++i) {
            if ((rc = check_factor(o[i])) != GEMM_OK) return rc;
            if (!factor_fits(o[i])) return GEMM_ERR_UNSUPPORTED;
            r16 = r16 && rows16(o[i]);
        }
    if (!any) return GEMM_OK;
    rc = first_of({check_rows(G, ldg, N, 2, false), check_rows(U, ldu, N, 2, false), check_rows(H, ldh, N, 2, true)});
    if (rc != GEMM_OK) return rc;
    const int bias_size = bias_dtype == GEMM_F32 ? 4 : 2;
    if (!aligned(BG, bias_size) || !aligned(BU, bias_size)) return GEMM_ERR_ALIGNMENT;
    Plan plan;
    rc = plan_sums(GEMM_FORM_GATED, M, N, K, dtype, r16, false, tile, h->num_cus, &plan);
    if (rc != GEMM_OK) return rc;
    pg::LinearArgs a;
    memset(&a, 0, sizeof a);
    a.A[0] = X;
    a.lda[0] = reads ? o[0].step() : 0;
    a.B[0] = WG;
    a.ldb[0] = reads ? o[1].step() : 0;
    a.B[1] = WU;
    a.ldb[1] = reads ? o[2].step() : 0;
    a.out[0] = H;
    a.ldo[0] = ldh;
    a.out[1] = G;
    a.ldo[1] = ldg;
    a.out[2] = U;
    a.ldo[2] = ldu;
    a.bias[0] = BG;
    a.bias[1] = BU;
    a.bias_f32 = bias_dtype == GEMM_F32;
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.act = activation;
    return launch(h, plan, a, stream);
}

int gemm_gated_backward(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int activation, int tile,
                        const void* DY, int64_t lddy, const void* W, int64_t ldw, const void* G, int64_t ldg,
                        const void* U, int64_t ldu, void* DG, int64_t lddg, void* DU, int64_t lddu, void* H, int64_t ldh,
                        void* stream) {
    if (h == nullptr || !is_act(activation)) return GEMM_ERR_INVALID_ARG;
    int rc = check_sizes(M, N, K, dtype, tile);
    if (rc != GEMM_OK) return rc;
    const bool any = M > 0 && N > 0, reads = any && K > 0;
    const Operand o[2] = {{DY, lddy, M, K, true}, {W, ldw, K, N, false}};
    bool r16 = true;
    if (reads)
        for (int i = 0; i < 2; ++i) {
            if ((rc = check_factor(o[i])) != GEMM_OK) return rc;
            if (!factor_fits(o[i])) return GEMM_ERR_UNSUPPORTED;
            r16 = r16 && rows16(o[i]);
        }
    if (!any) return GEMM_OK;
    if ((U == nullptr) != (DU == nullptr)) return GEMM_ERR_INVALID_ARG;
    rc = first_of({check_rows(G, ldg, N, 2, true), check_rows(U, ldu, N, 2, false), check_rows(DG, lddg, N, 2, true),
                   check_rows(DU, lddu, N, 2, false), check_rows(H, ldh, N, 2, false)});
    if (rc != GEMM_OK) return rc;
    Plan plan;
    rc = plan_sums(GEMM_FORM_GATED_BACKWARD, M, N, K, dtype, r16, false, tile, h->num_cus, &plan);
    if (rc != GEMM_OK) return rc;
    pg::LinearArgs a;
    memset(&a, 0, sizeof a);
    a.A[0] = DY;
    a.lda[0] = reads ? o[0].step() : 0;
    a.B[0] = W;
    a.ldb[0] = reads ? o[1].step() : 0;
    a.in[0] = G;
    a.ldi[0] = ldg;
    a.in[1] = U;
    a.ldi[1] = ldu;
    a.out[0] = DG;
    a.ldo[0] = lddg;
    a.out[1] = DU;
    a.ldo[1] = lddu;
    a.out[2] = H;
    a.ldo[2] = ldh;
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.act = activation;
    return launch(h, plan, a, stream);
}

int gemm_weight_gradient(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int accumulate, int tile,
                         const void* DC, int64_t lddc, const void* A, int64_t lda, float* DW, int64_t lddw, float* DB,
                         void* stream) {
    if (h == nullptr || (accumulate != 0 && accumulate != 1)) return GEMM_ERR_INVALID_ARG;
    int rc = check_sizes(M, N, K, dtype, tile);
    if (rc != GEMM_OK) return rc;
    const bool any = N > 0 && K > 0, reads = any && M > 0;
    if (N > 0 && K == 0 && DB != nullptr) return GEMM_ERR_UNSUPPORTED;      // no tile would add them
    const Operand o[2] = {{DC, lddc, M, N, false}, {A, lda, M, K, false}};
    bool r16 = true;
    if (reads)
        for (int i = 0; i < 2; ++i) {
            if ((rc = check_factor(o[i])) != GEMM_OK) return rc;
            if (!factor_fits(o[i])) return GEMM_ERR_UNSUPPORTED;
            r16 = r16 && rows16(o[i]);
        }
    if (!any) return GEMM_OK;
    rc = first_of({check_rows(DW, lddw, K, 4, true), aligned(DB, 4) ? GEMM_OK : GEMM_ERR_ALIGNMENT});
    if (rc != GEMM_OK) return rc;
    Plan plan;
    rc = plan_sums(GEMM_FORM_WEIGHT_GRADIENT, N, K, M, dtype, r16, DB != nullptr, tile, h->num_cus, &plan);
    if (rc != GEMM_OK) return rc;
    pg::LinearArgs a;
    memset(&a, 0, sizeof a);
    a.A[0] = DC;
    a.lda[0] = reads ? o[0].step() : 0;
    a.B[0] = A;
    a.ldb[0] = reads ? o[1].step() : 0;
    a.out[0] = DW;
    a.ldo[0] = lddw;
    a.sums = DB;
    a.M = (int32_t)N;
    a.N = (int32_t)K;
    a.K = (int32_t)M;
    a.accumulate = accumulate;
    return launch(h, plan, a, stream);
}

}  // extern "C"
