// fp8_abi.hip -- the C ABI of the 8-bit operators (include/pipegemm.h):
// argument checks, choice of kernel, launch.  Host code only.
#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "pipegemm.h"
#include "handle.h"
#include "fp8_common.h"
#include "fp8_gemm.h"
#include "fp8_rms_plan.h"

namespace {

constexpr int kDefaultCus = 256;  // MI355X; used when no device is at hand
constexpr int64_t kBlock = pg::kBlock;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0; }
bool is_fp8(int t) { return t == GEMM_E4M3 || t == GEMM_E5M2; }
bool is_float(int t) { return t == GEMM_F16 || t == GEMM_BF16 || t == GEMM_F32; }
int size_of(int t) { return t == GEMM_F32 ? 4 : 2; }
int fp8_of(int t) { return t == GEMM_E5M2 ? pg::FP8_E5M2 : pg::FP8_E4M3; }

// rows x blocks scales span less than the buffer range, past which loads give
// zero: a scale's address is the sum of its row's and its block's parts.
bool scales_fit(int64_t rows, int64_t row, int64_t blocks, int64_t blk) {
    return 4 * ((rows > 1 ? (__int128)rows * row : 0) + (blocks > 1 ? (__int128)blocks * blk : 0)) <= INT_MAX;
}

// A tile's rows span less than 2^31 bytes, with 4096 to spare: the loops address
// up to 16 blocks past K, with the bit that puts them out of range (2^31), and
// so large an offset would carry out of 32 bits and come back in range.
bool rows_fit(int64_t rows, int64_t ld, int64_t K) {
    return (rows > 1 ? (__int128)rows * ld : K) + 4096 <= (int64_t)1 << 31;
}

struct Plan {
    gemm_fp8_info_t info;
    const void* fn;
    int64_t tiles_m, tiles_n;
};

// Every check of the product, then its kernel.  No HIP call.
int plan_product(int64_t M, int64_t N, int64_t K, int a_type, int b_type, int c_dtype, int b_scale_rows, int accumulate,
                 int tile, const void* A, int64_t lda, const void* SA, int64_t sa_row, int64_t sa_blk, const void* B,
                 int64_t ldb, const void* SB, int64_t sb_row, int64_t sb_blk, const void* C, int64_t ldc, int num_cus,
                 bool query, Plan* plan) {
    if (!is_fp8(a_type) || !is_fp8(b_type) || !is_float(c_dtype)) return GEMM_ERR_INVALID_ARG;
    if (b_scale_rows != 1 && b_scale_rows != kBlock) return GEMM_ERR_INVALID_ARG;
    if (tile < GEMM_FP8_TILE_AUTO || tile >= pg::FP8_TILE_COUNT) return GEMM_ERR_INVALID_ARG;
    if (accumulate != 0 && accumulate != 1) return GEMM_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 0 || lda < 0 || ldb < 0 || ldc < 0) return GEMM_ERR_INVALID_ARG;
    if (sa_row < 0 || sa_blk < 0 || sb_row < 0 || sb_blk < 0) return GEMM_ERR_INVALID_ARG;
    const bool has_c = M > 0 && N > 0, reads = has_c && K > 0;
    if (reads && !query && (A == nullptr || B == nullptr || SA == nullptr || SB == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (reads && (lda < K || ldb < K)) return GEMM_ERR_INVALID_ARG;
    if (has_c && ((C == nullptr && !query) || ldc < N)) return GEMM_ERR_INVALID_ARG;
    if (accumulate && c_dtype != GEMM_F32) return GEMM_ERR_UNSUPPORTED;
    if (!aligned(C, size_of(c_dtype)) || !aligned(SA, 4) || !aligned(SB, 4)) return GEMM_ERR_ALIGNMENT;
    if (M > INT_MAX || N > INT_MAX || K > INT_MAX - kBlock) return GEMM_ERR_UNSUPPORTED;

    // Rows that start on 16 bytes can be staged through LDS whatever K is (a
    // chunk that holds one byte of a row lies in one page with it); rows at
    // any address, and pieces of chunks, are read into registers.
    const bool rows16 = !reads || (aligned(A, 16) && aligned(B, 16) && lda % 16 == 0 && ldb % 16 == 0);
    const bool exact = c_dtype == GEMM_F32;
    const bool bytes = reads && (!rows16 || K % 16 != 0);
    const int at = fp8_of(a_type), bt = fp8_of(b_type);
    auto kernel = [&](int t) -> const void* {
        if (!pg::fp8_staged(t)) return pg::fp8_stream_kernel(t, at, bt, b_scale_rows == 1, exact, bytes);
        if (!rows16) return nullptr;
        const void* fn = pg::fp8_staged_kernel(t, at, bt, b_scale_rows == 1, exact);
        return fn != nullptr ? fn : pg::fp8_waves_kernel(t, at, bt, b_scale_rows == 1, exact);
    };
    // A class's launch, and its 32-bit offsets inside a tile (of `rows` rows of
    // A) and to the scales that a tile takes.
    const int64_t kb = ceil_div(K, kBlock);
    auto fits = [&](int t, int64_t rows) {
        const pg::Fp8Shape sh = pg::fp8_shape(t);
        if (has_c && ceil_div(M, sh.bm) * ceil_div(N, sh.bn) >= ((int64_t)1 << 32) / (64 * sh.waves)) return false;
        const int64_t a_rows = std::min(rows, M), b_rows = std::min<int64_t>(sh.bn, N);
        return !reads || (rows_fit(a_rows, lda, K) && rows_fit(b_rows, ldb, K) && scales_fit(a_rows, sa_row, kb, sa_blk) &&
                          scales_fit(b_scale_rows == 1 ? b_rows : ceil_div(b_rows, kBlock), sb_row, kb, sb_blk));
    };
    // The class that takes the least time by the measured costs, of those that
    // fit.  (Where only tiles of 16 rows do, which read B for each 16 rows of A,
    // the caller has to ask for one.)
    int tc = tile;
    if (tc == GEMM_FP8_TILE_AUTO) {
        double best = 0.0;
        for (int t = 0; t < pg::FP8_TILE_COUNT; ++t) {
            const pg::Fp8Shape sh = pg::fp8_shape(t);
            if (kernel(t) == nullptr) continue;
            // A handful of rows leave a staged tile of 64 mostly loading copies
            // of A (1 x 8192 x 8192, B not in the caches: 64x32 15.9 us, 16x32
            // 13.9; 16 rows, in the caches: 13.0 and 14.2).
            if (M <= 8 && pg::fp8_staged(t)) continue;
            const double time = pg::fp8_time(t, exact, ceil_div(M, sh.bm) * ceil_div(N, sh.bn), kb, num_cus);
            if ((tc == GEMM_FP8_TILE_AUTO || time < best) && fits(t, std::max(sh.bm, 32))) {
                tc = t;
                best = time;
            }
        }
        if (tc == GEMM_FP8_TILE_AUTO) return GEMM_ERR_UNSUPPORTED;
    }
    plan->fn = kernel(tc);
    if (plan->fn == nullptr) return rows16 ? GEMM_ERR_UNSUPPORTED : GEMM_ERR_ALIGNMENT;
    const pg::Fp8Shape sh = pg::fp8_shape(tc);
    if (!fits(tc, sh.bm)) return GEMM_ERR_UNSUPPORTED;
    plan->tiles_m = has_c ? ceil_div(M, sh.bm) : 0;
    plan->tiles_n = has_c ? ceil_div(N, sh.bn) : 0;
    const int64_t grid = plan->tiles_m * plan->tiles_n;
    gemm_fp8_info_t& in = plan->info;
    memset(&in, 0, sizeof in);
    in.tile = tc;
    in.block_m = sh.bm;
    in.block_n = sh.bn;
    in.waves_k = sh.wk;
    in.threads = 64 * sh.waves;
    in.staged = pg::fp8_staged(tc) ? 1 : 0;
    in.widened = exact ? 1 : 0;
    // 256x256: one workgroup per CU stays and takes tile after tile
    in.grid = tc == pg::FP8_TILE_256 && grid > num_cus ? num_cus : grid;
    in.c_tiles = grid;
    in.k_blocks = kb;
    return GEMM_OK;
}

}  // namespace

extern "C" {

int gemm_query_fp8(int64_t M, int64_t N, int64_t K, int a_type, int b_type, int c_dtype, int b_scale_rows,
                   int accumulate, int tile, const void* A, int64_t lda, const float* SA, int64_t sa_row,
                   int64_t sa_blk, const void* B, int64_t ldb, const float* SB, int64_t sb_row, int64_t sb_blk,
                   const void* C, int64_t ldc, gemm_fp8_info_t* info) {
    if (info == nullptr) return GEMM_ERR_INVALID_ARG;
    Plan plan;
    const int rc = plan_product(M, N, K, a_type, b_type, c_dtype, b_scale_rows, accumulate, tile, A, lda, SA, sa_row,
                                sa_blk, B, ldb, SB, sb_row, sb_blk, C, ldc, kDefaultCus, true, &plan);
    if (rc == GEMM_OK) *info = plan.info;
    return rc;
}

int gemm_run_fp8(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int a_type, int b_type, int c_dtype,
                 int b_scale_rows, int accumulate, int tile, const void* A, int64_t lda, const float* SA,
                 int64_t sa_row, int64_t sa_blk, const void* B, int64_t ldb, const float* SB, int64_t sb_row,
                 int64_t sb_blk, void* C, int64_t ldc, void* stream) {
    if (h == nullptr) return GEMM_ERR_INVALID_ARG;
    Plan plan;
    const int rc = plan_product(M, N, K, a_type, b_type, c_dtype, b_scale_rows, accumulate, tile, A, lda, SA, sa_row,
                                sa_blk, B, ldb, SB, sb_row, sb_blk, C, ldc, h->num_cus, false, &plan);
    if (rc != GEMM_OK) return rc;
    if (plan.info.grid == 0) return GEMM_OK;
    pg::Fp8Args a;
    a.A = (const uint8_t*)A;
    a.B = (const uint8_t*)B;
    a.SA = SA;
    a.SB = SB;
    a.C = C;
    const bool reads = K > 0;            // else strides are unchecked, and every load is out of range by its bit alone
    a.lda = reads ? lda : 0;
    a.ldb = reads ? ldb : 0;
    a.ldc = ldc;
    a.sa_row = reads ? sa_row : 0;
    a.sa_blk = reads ? sa_blk : 0;
    a.sb_row = reads ? sb_row : 0;
    a.sb_blk = reads ? sb_blk : 0;
    a.M = (int32_t)M;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.tiles_m = (int32_t)plan.tiles_m;
    a.tiles_n = (int32_t)plan.tiles_n;
    a.c_type = c_dtype;
    a.accumulate = accumulate;
    a.c_lines = !accumulate && aligned(C, 128) && ldc * size_of(c_dtype) % 128 == 0;
    void* kargs[] = {&a};
    return pg::on_device(h, [&] {
        const hipError_t e = hipLaunchKernel(plan.fn, dim3((unsigned)plan.info.grid), dim3((unsigned)plan.info.threads),
                                             kargs, 0, (hipStream_t)stream);
        return e == hipSuccess ? hipGetLastError() : e;
    });
}

int gemm_quantize_fp8(gemm_handle_t h, int64_t M, int64_t K, int x_dtype, int fp8_type, int block_rows, int pow2,
                      const void* X, int64_t ldx, void* Q, int64_t ldq, float* S, int64_t s_row, int64_t s_blk,
                      void* QT, int64_t ldqt, float* ST, int64_t st_row, int64_t st_blk, void* stream) {
    if (h == nullptr || !is_float(x_dtype) || !is_fp8(fp8_type)) return GEMM_ERR_INVALID_ARG;
    if (block_rows != 1 && block_rows != kBlock) return GEMM_ERR_INVALID_ARG;
    if (pow2 != 0 && pow2 != 1) return GEMM_ERR_INVALID_ARG;
    if (M < 0 || K < 0 || ldx < 0 || ldq < 0 || ldqt < 0) return GEMM_ERR_INVALID_ARG;
    if (s_row < 0 || s_blk < 0 || st_row < 0 || st_blk < 0) return GEMM_ERR_INVALID_ARG;
    const bool any = M > 0 && K > 0;
    if (any && Q == nullptr && QT == nullptr) return GEMM_ERR_INVALID_ARG;
    if (any && (X == nullptr || ldx < K)) return GEMM_ERR_INVALID_ARG;
    if (any && Q != nullptr && (S == nullptr || ldq < K)) return GEMM_ERR_INVALID_ARG;
    if (any && QT != nullptr && (ST == nullptr || ldqt < M)) return GEMM_ERR_INVALID_ARG;
    const int sz = size_of(x_dtype);
    if (!aligned(X, sz) || !aligned(S, 4) || !aligned(ST, 4)) return GEMM_ERR_ALIGNMENT;
    if (M > INT_MAX || K > INT_MAX) return GEMM_ERR_UNSUPPORTED;
    const bool tile = block_rows == kBlock;
    const bool both = tile || QT != nullptr;
    const int64_t groups = ceil_div(M, pg::quantize_rows_per_group(M, K, both)) * ceil_div(K, kBlock);
    if (groups >= ((int64_t)1 << 32) / pg::quantize_threads(both)) return GEMM_ERR_UNSUPPORTED;
    if (!any) return GEMM_OK;
    pg::QuantizeArgs a;
    a.X = X;
    a.Q = (uint8_t*)Q;
    a.S = S;
    a.QT = (uint8_t*)QT;
    a.ST = ST;
    a.ldx = ldx;
    a.ldq = ldq;
    a.ldqt = ldqt;
    a.s_row = s_row;
    a.s_blk = s_blk;
    a.st_row = st_row;
    a.st_blk = st_blk;
    a.M = (int32_t)M;
    a.K = (int32_t)K;
    a.e5m2 = fp8_type == GEMM_E5M2;
    a.pow2 = pow2;
    return pg::on_device(h, [&] { return pg::launch_quantize(a, x_dtype, tile, (hipStream_t)stream); });
}

int gemm_rms_fp8(gemm_handle_t h, int64_t M, int64_t D, int x_dtype, int w_dtype, int fp8_type, int pow2, float eps,
                 const void* X, int64_t ldx, const void* R, int64_t ldr, const void* W, void* H, int64_t ldh, void* Y,
                 int64_t ldy, void* Q, int64_t ldq, float* S, int64_t s_row, int64_t s_blk, float* rstd, void* stream) {
    if (h == nullptr || !is_float(x_dtype) || !is_fp8(fp8_type)) return GEMM_ERR_INVALID_ARG;
    if (w_dtype != x_dtype && w_dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
    if (pow2 != 0 && pow2 != 1) return GEMM_ERR_INVALID_ARG;
    if (!(eps >= 0.0f)) return GEMM_ERR_INVALID_ARG;
    if (M < 0 || D < 0 || ldx < 0 || ldr < 0 || ldh < 0 || ldy < 0 || ldq < 0 || s_row < 0 || s_blk < 0)
        return GEMM_ERR_INVALID_ARG;
    const bool any = M > 0 && D > 0;
    if (any && Q == nullptr && Y == nullptr) return GEMM_ERR_INVALID_ARG;
    if (any && (X == nullptr || ldx < D || W == nullptr)) return GEMM_ERR_INVALID_ARG;
    if (any && ((R != nullptr && ldr < D) || (H != nullptr && ldh < D) || (Y != nullptr && ldy < D)))
        return GEMM_ERR_INVALID_ARG;
    if (any && Q != nullptr && (S == nullptr || ldq < D)) return GEMM_ERR_INVALID_ARG;
    const int sz = size_of(x_dtype);
    if (!aligned(X, sz) || !aligned(R, sz) || !aligned(H, sz) || !aligned(Y, sz) || !aligned(W, size_of(w_dtype)) ||
        !aligned(S, 4) || !aligned(rstd, 4))
        return GEMM_ERR_ALIGNMENT;
    if (M > GEMM_RMS_MAX_ROWS || D > GEMM_RMS_MAX_D || !pg::rms_launches(M, D)) return GEMM_ERR_UNSUPPORTED;
    if (!any) return GEMM_OK;
    pg::RmsArgs a;
    a.X = X;
    a.R = R;
    a.W = W;
    a.H = H;
    a.Y = Y;
    a.Q = (uint8_t*)Q;
    a.S = S;
    a.rstd = rstd;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.ldq = ldq;
    a.s_row = s_row;
    a.s_blk = s_blk;
    a.M = (int32_t)M;
    a.D = (int32_t)D;
    a.eps = eps;
    a.e5m2 = fp8_type == GEMM_E5M2;
    a.pow2 = pow2;
    a.w_f32 = w_dtype == GEMM_F32;
    return pg::on_device(h, [&] { return pg::launch_rms(a, x_dtype, (hipStream_t)stream); });
}

int64_t gemm_rms_backward_workspace(int64_t M, int64_t D) {
    if (M < 0 || D < 0 || M > GEMM_RMS_MAX_ROWS || D > GEMM_RMS_MAX_D) return 0;
    return pg::rms_backward_form(M, D, false, kDefaultCus).parts * pg::rms_parts_row(D) * 4;
}

int gemm_rms_backward(gemm_handle_t h, int64_t M, int64_t D, int x_dtype, int w_dtype, const void* DY, int64_t lddy,
                      const void* H, int64_t ldh, const void* W, const float* rstd, const void* DH, int64_t lddh,
                      void* DX, int64_t lddx, float* DW, void* workspace, int64_t workspace_bytes, void* stream) {
    if (h == nullptr || !is_float(x_dtype)) return GEMM_ERR_INVALID_ARG;
    if (w_dtype != x_dtype && w_dtype != GEMM_F32) return GEMM_ERR_INVALID_ARG;
    if (M < 0 || D < 0 || lddy < 0 || ldh < 0 || lddh < 0 || lddx < 0 || workspace_bytes < 0) return GEMM_ERR_INVALID_ARG;
    const bool any = M > 0 && D > 0;
    if (D > 0 && DW == nullptr) return GEMM_ERR_INVALID_ARG;
    if (any && (DY == nullptr || H == nullptr || W == nullptr || rstd == nullptr || DX == nullptr))
        return GEMM_ERR_INVALID_ARG;
    if (any && (lddy < D || ldh < D || lddx < D || (DH != nullptr && lddh < D))) return GEMM_ERR_INVALID_ARG;
    const int sz = size_of(x_dtype);
    if (!aligned(DY, sz) || !aligned(H, sz) || !aligned(DH, sz) || !aligned(DX, sz) || !aligned(W, size_of(w_dtype)) ||
        !aligned(rstd, 4) || !aligned(DW, 4) || !aligned(workspace, 16))
        return GEMM_ERR_ALIGNMENT;
    if (M > GEMM_RMS_MAX_ROWS || D > GEMM_RMS_MAX_D) return GEMM_ERR_UNSUPPORTED;
    const pg::RmsBackwardForm form = pg::rms_backward_form(M, D, x_dtype == GEMM_F32, kDefaultCus);
    if (!pg::rms_backward_launches(form, M, D)) return GEMM_ERR_UNSUPPORTED;
    const int64_t needed = gemm_rms_backward_workspace(M, D);
    if (needed > 0 && (workspace == nullptr || workspace_bytes < needed)) return GEMM_ERR_INVALID_ARG;
    if (D == 0) return GEMM_OK;
    pg::RmsBackwardArgs a;
    a.DY = DY;
    a.H = H;
    a.W = W;
    a.rstd = rstd;
    a.DH = DH;
    a.DX = DX;
    a.parts = (float*)workspace;
    a.DW = DW;
    a.lddy = lddy;
    a.ldh = ldh;
    a.lddh = lddh;
    a.lddx = lddx;
    a.M = (int32_t)M;
    a.D = (int32_t)D;
    a.groups = form.parts;
    a.w_f32 = w_dtype == GEMM_F32;
    const auto meets = [&](const void* p, int64_t ld) {      // the byte ranges of DX and p
        const uintptr_t x = (uintptr_t)DX, y = (uintptr_t)p;
        return any && x < y + ((uintptr_t)(M - 1) * ld + D) * sz && y < x + ((uintptr_t)(M - 1) * lddx + D) * sz;
    };
    a.in_place = meets(DY, lddy) || meets(H, ldh);
    return pg::on_device(h, [&] { return pg::launch_rms_backward(a, form, x_dtype, (hipStream_t)stream); });
}

}  // extern "C"
