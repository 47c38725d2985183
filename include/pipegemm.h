/*
 * pipegemm.h -- C ABI of the software-pipelined tiled GEMM for AMD Instinct
 * MI355X (gfx950).
 *
 * Operation.  gemm_run computes C = A * B,
 *     C[i][j] = sum_{k=0}^{K-1} A[i][k] * B[k][j],   0 <= i < M, 0 <= j < N,
 * the product the "CUDA Kernel Study: Pipelining" README benchmarks (Example
 * Code: "C = A x B") and that "Part 4 -- Pipelining and Occupancy"
 * (gpucourse.com) writes out as the triple loop of section 4.3.  The K loop
 * runs over BK-wide tiles restructured into prologue / main loop / epilogue
 * so that the global->LDS copy of the next tile overlaps the matrix-core
 * work on the current one ("pipeline-gpu-kernel", step 3; the README's
 * ping-pong and multi-stage cases).  Pipelining reorders loads only; the
 * arithmetic is that of the unpipelined loop ("pipeline-gpu-kernel", step 5).
 *
 * Element types (input -> accumulator -> output):
 *   GEMM_I8   int8  -> int32 (exact; wraps modulo 2^32 like the uint32_t
 *                     reference at the end of the gpucourse section 4.3)
 *   GEMM_F16  fp16  -> fp32  -> fp16 (round to nearest even)
 *   GEMM_BF16 bf16  -> fp32  -> bf16 (round to nearest even)
 *   GEMM_F32  fp32  -> fp32  -> fp32
 *
 * Layouts (leading dimensions are in elements):
 *   A is always row-major M x K:  A(i,k) = A[i*lda + k], lda >= K.
 *   GEMM_LAYOUT_RR: B row-major K x N:     B(k,j) = B[k*ldb + j], ldb >= N.
 *   GEMM_LAYOUT_RC: B column-major K x N:  B(k,j) = B[j*ldb + k], ldb >= K.
 *   C is always row-major M x N:  C(i,j) = C[i*ldc + j], ldc >= N.
 *
 * Alignment:
 *   C: 16-byte aligned, ldc a multiple of 4 elements.  Layout RR: N a
 *     multiple of 16 bytes worth of elements.
 *   A and B, GEMM_VARIANT_DIRECT: 16-byte aligned, lda and ldb times the
 *     element size multiples of 16 bytes, K a multiple of 16 bytes worth of
 *     elements (its copies move whole aligned 16-byte chunks).
 *   A and B, GEMM_VARIANT_REG: aligned to their element size; any K, lda and
 *     ldb.  When K is not a multiple of 16 bytes worth of elements the chunk
 *     holding column K-1 of each row is read in exact 8/4/2/1-byte pieces
 *     (the bounds-checked fallback for the last tile that "pipeline-gpu-kernel"
 *     names under its pitfalls, cp.async boundary handling): no byte past
 *     column K-1 of a row is read.  Rows and pointers that are not 16-byte
 *     aligned are read with unaligned 16-byte loads.
 *
 * Pipeline depth and load path:
 *   stages in [1, 4].
 *   GEMM_VARIANT_DIRECT: global -> LDS copies that bypass registers (the
 *     README's cp.async case; here the LDS-DMA form of buffer loads).  An
 *     LDS ring of `stages` slots with stages-1 tiles in flight; stages = 1 is
 *     the serial load-sync-compute-sync loop of the README's Background.
 *     The 256x256 tiles keep their full K-tile at stages = 3 by splitting
 *     the ring by operand: three slots for A (two tiles in flight), two for
 *     B (one in flight), 160 KiB in all; at stages = 4 they halve the
 *     K-tile (four whole slots).
 *   GEMM_VARIANT_REG: global -> VGPR -> LDS (the README's ping-pong case).
 *     min(stages, 2) LDS slots and max(1, stages-1) register staging sets,
 *     each a tile in flight; stages = 1 is the skill's register-only prefetch
 *     into a single buffer (step 1, "if it fails"), stages = 2 the classic
 *     double buffer.
 *   For a fixed dtype, layout and tile every (stages, variant) pair adds
 *   the same products in the same k order (the instances built from 16x16
 *   matrix-core blocks as well as those built from 32x32 ones), so all of
 *   them return bit-identical C.
 *
 * Memory ownership.  The caller allocates, owns and frees A, B, C and the
 * stream; they are device pointers (hipMalloc or torch CUDA tensors) on the
 * handle's device.  The library allocates no device memory; its code object
 * holds one static array of GEMM_NOALLOC_SCRATCH_BYTES per device, the
 * workspace of gemm_run_splitk_noalloc.  A and B are only read.  C must not
 * overlap A or B.
 *
 * Errors.  Every entry point returns GEMM_OK (0) or one of the codes below;
 * nothing is thrown across the ABI.  Argument checks run before any HIP call,
 * so a rejected call has no side effect.  gemm_run, gemm_run_splitk,
 * gemm_run_streamk and gemm_run_splitk_noalloc are asynchronous: each
 * enqueues one kernel launch on `stream` (and nothing else, so a graph can
 * capture it) and returns; faults during execution surface at the caller's
 * next synchronisation of that stream.
 */
#ifndef PIPEGEMM_H
#define PIPEGEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMM_I8 = 0, GEMM_F16 = 1, GEMM_BF16 = 2, GEMM_F32 = 3 } gemm_dtype_t;
typedef enum { GEMM_LAYOUT_RR = 0, GEMM_LAYOUT_RC = 1 } gemm_layout_t;
typedef enum { GEMM_VARIANT_REG = 0, GEMM_VARIANT_DIRECT = 1 } gemm_variant_t;

enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = 1,  /* NULL handle/pointer, negative size, bad enum,
                                  leading dimension too small, stages not in [1,4] */
    GEMM_ERR_ALIGNMENT = 2,    /* an alignment rule above is broken: C's, RR's N,
                                  A/B not element-aligned, or (direct variant
                                  only) A/B rows or K not whole 16-byte chunks */
    GEMM_ERR_UNSUPPORTED = 3,  /* no kernel instance fits the LDS budget, an
                                  operand tile row span exceeds 2^31 bytes, or
                                  (gemm_run_splitk) more than one split with
                                  more than 16384 C tiles */
    GEMM_ERR_HIP = 4,          /* a HIP runtime call failed (no device, launch
                                  failure); see gemm_last_hip_error */
    GEMM_ERR_SCRATCH = 5       /* gemm_run_splitk_noalloc: the split-K workspace
                                  the call needs exceeds
                                  GEMM_NOALLOC_SCRATCH_BYTES */
};

/* Size of the library's static scratch buffer (one per device), the
 * workspace of gemm_run_splitk_noalloc: 32 MiB. */
#define GEMM_NOALLOC_SCRATCH_BYTES (32 * 1024 * 1024)

/* Tile classes selectable with gemm_set_tile.  GEMM_TILE_256x256_W8 is the
 * 256x256 tile run by 8 waves (2 per SIMD) instead of 4; it is never chosen
 * automatically (its register-staged instances spill a few registers).
 * GEMM_TILE_AUTO lets the library choose the largest of the 4-wave tiles
 * that still gives at least one workgroup per compute unit. */
enum { GEMM_TILE_AUTO = -1, GEMM_TILE_256x256 = 0, GEMM_TILE_128x128 = 1, GEMM_TILE_32x64 = 2,
       GEMM_TILE_256x256_W8 = 3 };

typedef struct gemm_handle_s *gemm_handle_t;

/* What gemm_run would launch for a given call (see gemm_query). */
typedef struct {
    int32_t tile;            /* GEMM_TILE_* actually chosen */
    int32_t block_m, block_n, block_k;
    int32_t waves_m, waves_n;
    int32_t threads;         /* per workgroup */
    int32_t lds_slots;       /* slots of the LDS ring (the split ring of
                                the 256x256 tiles at 3 direct stages: 3 for
                                A, 2 for B) */
    int32_t reg_sets;        /* VGPR staging sets (0 for the direct variant) */
    int32_t tiles_in_flight; /* K-tiles loading while one is multiplied
                                (split ring: 2 for A, 1 for B) */
    int32_t lds_bytes;       /* LDS per workgroup */
    int32_t loads_per_tile;  /* 16-byte loads per lane per K-tile */
    int64_t grid;            /* workgroups launched */
    int64_t k_tiles;         /* ceil(K / block_k) */
    int32_t k_tail;          /* K mod block_k; 0 means no ragged last tile */
    int32_t c_tiles;         /* C tiles; above grid when each workgroup of a
                                256x256 tile computes several in turn (then
                                grid = one workgroup per CU) */
    int32_t splits;          /* K splits per C tile (1: none); see gemm_run_splitk */
    int32_t mfma_block;      /* edge of the MFMA blocks the kernel uses: 16
                                (4-wave 256x256 tile, 2-3 direct stages, either
                                layout, int8/fp16/bf16) or 32; both give the
                                same bits */
    int64_t workspace_bytes; /* workspace gemm_run_splitk needs (0 when splits = 1),
                                or gemm_run_streamk (see there) */
    int32_t waves_k;         /* waves sharing each C block, each taking its own
                                run of every K-tile's k-steps; their partial
                                sums are added in LDS after the K loop (1: none) */
    int32_t sk_tiles;        /* gemm_run_streamk: C tiles shared out stream-K
                                (the last sk_tiles of the c_tiles); the others
                                run data-parallel.  0 otherwise */
} gemm_config_info_t;

/* Bind a handle to HIP device `device`.  Allocates host memory for the
 * handle only.  The first call for a device also sets up that device's copy
 * of the static scratch buffer of gemm_run_splitk_noalloc: it looks up its
 * address and clears its arrival counters with one small kernel on the null
 * stream, waiting for it (so call it outside any graph capture).  Returns
 * GEMM_ERR_INVALID_ARG for a NULL `out` or a negative device, GEMM_ERR_HIP
 * when the device does not exist or that set-up fails. */
int gemm_create(gemm_handle_t *out, int device);

/* C = A * B on `stream` (a hipStream_t; NULL is the null stream).  Argument
 * checks as described above; M, N or K may be 0 (M or N = 0 does nothing,
 * K = 0 writes C = 0).  Launches on the handle's device. */
int gemm_run(gemm_handle_t h, int64_t M, int64_t N, int64_t K,
             int dtype, int layout, int stages, int variant,
             const void *A, int64_t lda, const void *B, int64_t ldb,
             void *C, int64_t ldc, void *stream);

/* C = A * B with K split over `splits` workgroups per C tile, for shapes with
 * fewer C tiles than compute units (a partial wave: skinny or small M x N
 * with a long K).  The split count is the analogue, across workgroups, of
 * what the pages do within one: more independent loads in flight per unit of
 * C; "CUDA Kernel Study: Pipelining" (Detailed Analysis) and "Part 4 --
 * Pipelining and Occupancy" (gpucourse.com) tie the gain of pipelining to
 * the occupancy it leaves.
 *   splits >= 1 asks for that many (1 = gemm_run); 0 lets the library take
 *   the smallest that gives every CU a workgroup, but at most 8 and with at
 *   least two K units per split (the last split reads every partial tile,
 *   so the final sum grows with the count).  The count used is clamped
 *   to [1, min(64, K / largest K-tile of the tile class)] and reported by
 *   gemm_query_splitk.  Each split takes whole units of the class's largest
 *   K-tile (the ragged rest goes to the last split), so for a given split
 *   count every (stages, variant) pair still returns bit-identical C.
 *   Each split writes its fp32 (int32 for GEMM_I8) accumulators to the
 *   workspace and counts itself in an arrival counter; the split that
 *   arrives last adds the partial tiles in split order 0, 1, ..., rounds
 *   once and stores C.  No workgroup waits for another, and the result does
 *   not depend on which one arrives last.  int8 stays exact.
 * Workspace: caller-owned device memory of at least
 *   info.workspace_bytes = 65536 + c_tiles * splits * block_m * block_n * 4
 *   bytes, 256-byte aligned, overlapping none of A, B, C.  Its first 65536
 *   bytes hold the arrival counters and must be zero before its first use;
 *   every call that completes leaves them zero again, so one workspace
 *   serves any later call, of any shape, on the same stream.  Calls that
 *   share a workspace must not run concurrently (two streams race).
 *   NULL / 0 is accepted when the split count used is 1.
 * Errors: as gemm_run; also GEMM_ERR_INVALID_ARG for splits < 0, a NULL or
 * too small workspace when splits > 1 are used, GEMM_ERR_ALIGNMENT for a
 * workspace not 256-byte aligned, GEMM_ERR_UNSUPPORTED for splits > 1 with
 * more than 16384 C tiles. */
int gemm_run_splitk(gemm_handle_t h, int64_t M, int64_t N, int64_t K,
                    int dtype, int layout, int stages, int variant, int splits,
                    const void *A, int64_t lda, const void *B, int64_t ldb,
                    void *C, int64_t ldc, void *workspace, int64_t workspace_bytes,
                    void *stream);

/* C = A * B with the tiles shared out stream-K over `grid` workgroups
 * (0: one per compute unit), for shapes whose C tiles do not fill a whole
 * number of rounds of the grid (a partial last wave: e.g. 400 tiles of
 * 256 x 256 on 256 CUs take two rounds of gemm_run, the second 56% full).
 * This is the other half of the split-K / stream-K pair "CUDA Kernel Study:
 * Pipelining" (Detailed Analysis) and "Part 4 -- Pipelining and Occupancy"
 * (gpucourse.com, section 4.2: occupancy and waves of blocks) point to.
 *   Every full round of `grid` tiles but the last runs as in gemm_run (one
 *   tile per workgroup at a time).  The remaining sk_tiles tiles (between
 *   one and two rounds' worth, or all of them when there are fewer than two
 *   rounds) are cut into units of the tile class's largest K-tile, numbered
 *   tile by tile, and workgroup g takes the g-th of `grid` equal runs of
 *   units (sizes differ by at most one).  A tile covered by one workgroup is
 *   stored as in gemm_run; a tile split between several is summed from
 *   their fp32 (int32 for GEMM_I8) partial tiles by whichever arrives last,
 *   in K order, so the result does not depend on arrival order, every
 *   (stages, variant) pair returns bit-identical C for a given grid, and
 *   int8 stays exact.  Float results may differ from gemm_run's in the last
 *   bits (the partial sums are grouped differently).
 *   The grid used is min(grid, sk_tiles x units); gemm_query_streamk
 *   reports it, sk_tiles and the workspace size.
 * Workspace: caller-owned device memory of at least info.workspace_bytes =
 *   65536 + 2 x grid x block_m x block_n x 4 bytes, 256-byte aligned,
 *   overlapping none of A, B, C; its first 65536 bytes are arrival counters
 *   that must be zero before the first use and are zero again after every
 *   completed call (as for gemm_run_splitk, whose workspace it may share).
 *   Calls that share a workspace must not run concurrently.  NULL / 0 is
 *   accepted when sk_tiles is 0 (M or N = 0).
 * Errors: as gemm_run; also GEMM_ERR_INVALID_ARG for grid < 0 or a NULL or
 * too small workspace, GEMM_ERR_ALIGNMENT for a workspace not 256-byte
 * aligned, GEMM_ERR_UNSUPPORTED for more than 16384 C tiles or a grid whose
 * partial tiles would pass 2 GiB. */
int gemm_run_streamk(gemm_handle_t h, int64_t M, int64_t N, int64_t K,
                     int dtype, int layout, int stages, int variant, int grid,
                     const void *A, int64_t lda, const void *B, int64_t ldb,
                     void *C, int64_t ldc, void *workspace, int64_t workspace_bytes,
                     void *stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc):
 * gemm_run_splitk with the library's own static scratch buffer as its
 * workspace, so the caller passes no workspace and nothing is allocated.
 *   Same arguments, checks and results as gemm_run_splitk (bit for bit:
 * same kernels, same split count), without `workspace` / `workspace_bytes`.
 * The buffer is a file-scope device array of GEMM_NOALLOC_SCRATCH_BYTES per
 * device, held until the process ends; gemm_create sets it up for its
 * device.  A call whose split-K workspace (info.workspace_bytes of
 * gemm_query_splitk) exceeds that size returns GEMM_ERR_SCRATCH before any
 * HIP call; with one split (splits = 1, or the automatic choice taking one)
 * no scratch is used.  The call calls no hipMalloc, hipFree or allocating
 * routine and enqueues one kernel launch on `stream`.
 *   Every call on a device shares that device's buffer, which keeps the
 * last call's contents; its arrival counters are zero after every completed
 * call.  Calls that overlap on one device (e.g. on two streams) race on the
 * buffer and must not be issued. */
int gemm_run_splitk_noalloc(gemm_handle_t h, int64_t M, int64_t N, int64_t K,
                            int dtype, int layout, int stages, int variant, int splits,
                            const void *A, int64_t lda, const void *B, int64_t ldb,
                            void *C, int64_t ldc, void *stream);

/* Release a handle.  NULL is a no-op.  Does not synchronise any stream. */
int gemm_destroy(gemm_handle_t h);

/* Force a tile class for later gemm_run calls on this handle
 * (GEMM_TILE_AUTO restores the automatic choice). */
int gemm_set_tile(gemm_handle_t h, int tile);

/* The configuration gemm_run would use, after the same argument checks, with
 * no HIP call and no device access.  Pointers are never dereferenced: a
 * non-NULL pointer is checked for alignment, a NULL one is taken as "not
 * given" and skipped.  The tile is chosen for a 256-CU device (MI355X).
 * `tile` is a GEMM_TILE_* value. */
int gemm_query(int64_t M, int64_t N, int64_t K, int dtype, int layout, int stages,
               int variant, int tile, const void *A, int64_t lda, const void *B,
               int64_t ldb, const void *C, int64_t ldc, gemm_config_info_t *info);

/* gemm_query for gemm_run_splitk: the same, with the split count (and the
 * workspace size) that call would use. */
int gemm_query_splitk(int64_t M, int64_t N, int64_t K, int dtype, int layout, int stages,
                      int variant, int tile, int splits, const void *A, int64_t lda,
                      const void *B, int64_t ldb, const void *C, int64_t ldc,
                      gemm_config_info_t *info);

/* gemm_query for gemm_run_streamk: the tile, grid, sk_tiles and workspace
 * size that call would use (for a 256-CU device when grid = 0). */
int gemm_query_streamk(int64_t M, int64_t N, int64_t K, int dtype, int layout, int stages,
                       int variant, int tile, int grid, const void *A, int64_t lda,
                       const void *B, int64_t ldb, const void *C, int64_t ldc,
                       gemm_config_info_t *info);

/* Resources and occupancy of the kernel instance gemm_run would launch for a
 * call (see gemm_occupancy), the figures the "Part 4 -- Pipelining and
 * Occupancy" page (section 4.2) reads from the occupancy calculator. */
typedef struct {
    int32_t blocks_per_cu;   /* hipOccupancyMaxActiveBlocksPerMultiprocessor at
                                the instance's block size (no dynamic LDS) */
    int32_t waves_per_cu;    /* blocks_per_cu x waves per block (4 SIMDs per CU) */
    int32_t num_regs;        /* hipFuncGetAttributes numRegs: vector registers
                                per lane as the runtime reports them */
    int32_t lds_bytes;       /* static LDS per workgroup (sharedSizeBytes) */
    int32_t scratch_bytes;   /* private scratch per lane (localSizeBytes; 0 =
                                no register spill) */
    int32_t threads;         /* per workgroup */
} gemm_occupancy_t;

/* The occupancy of the instance gemm_run would launch on this handle (its
 * tile override, its device) for a call of this shape, dtype, layout,
 * stages and variant; pointers are not needed (the checks of gemm_query).
 * Makes HIP calls (function attributes, occupancy) on the handle's device;
 * launches nothing.  Errors: those of gemm_query, GEMM_ERR_INVALID_ARG for a
 * NULL handle or `out`, GEMM_ERR_HIP when a HIP call fails. */
int gemm_occupancy(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int layout,
                   int stages, int variant, gemm_occupancy_t *out);

/* ---- 8-bit floating point, with a scale for each block of 128 -------------
 *
 * One linear layer through 8 bits: gemm_rms_fp8 or gemm_quantize_fp8 make an
 * 8-bit matrix and its scales, gemm_run_fp8 multiplies two of them, and
 * gemm_rms_backward is the norm's backward pass.  (The product's own
 * backward pass is two more products: dX = dY * W with W quantised by tiles
 * and transposed, dW = dY^T * X with both quantised along the rows of X.)
 *
 * Types.  GEMM_E4M3 (largest value 448, no infinity) and GEMM_E5M2 (57344)
 * are the OCP 8-bit floats, torch's float8_e4m3fn and float8_e5m2.  A stored
 * value q of a block with scale s stands for q * s; s is fp32.
 *
 * Blocks are 128 consecutive values of a row (block_rows 1, "row") or 128
 * rows by 128 columns (block_rows 128, "tile"); the last ones may be shorter.
 * The scale of row (or row block) i and block b is at
 * S[i * s_row + b * s_blk], both strides in elements, zero allowed; s_row = 1
 * is the fastest for the product.
 *
 * Quantisation of a block (rounding to nearest even, everything in fp32):
 *   s = max(amax |x| / largest, 2^-126); with pow2 = 1 rounded up to a power of two;
 *   q = fp8(x * (1 / s)).
 * A NaN stays a NaN in its place and does not enter amax; an infinity gives
 * its block an infinite scale (every value of it then stands for NaN).
 *
 * All of these are asynchronous, allocate nothing, and enqueue one kernel
 * (gemm_rms_backward: up to two, up to three where DX takes the place of DY or
 * H) on `stream`, on the handle's device; any number of calls may overlap, on
 * any streams (gemm_rms_backward: each with its own workspace).  A captured
 * graph can hold them.  Outputs must not overlap inputs or one another, but
 * where stated.  Sizes of zero are accepted. */
enum { GEMM_E4M3 = 16, GEMM_E5M2 = 17 };

/* Part of C that one workgroup of gemm_run_fp8 computes.  Those down to
 * 64x32 stage operands through LDS and need rows that start on 16 bytes; the
 * others take any address.  From 64x64_K4 on each wave takes blocks of K of
 * its own (gemm_fp8_info_t's waves_k).  GEMM_FP8_TILE_AUTO: the one that takes the least time
 * by what each cost in measurements, of those (of 32 rows and more) that can
 * address the call's operands and scales. */
enum { GEMM_FP8_TILE_AUTO = -1, GEMM_FP8_TILE_256x256 = 0, GEMM_FP8_TILE_256x128 = 1, GEMM_FP8_TILE_128x128 = 2,
       GEMM_FP8_TILE_64x64 = 3, GEMM_FP8_TILE_64x64_K4 = 4, GEMM_FP8_TILE_64x32 = 5, GEMM_FP8_TILE_32x32 = 6,
       GEMM_FP8_TILE_16x32 = 7, GEMM_FP8_TILE_16x16 = 8 };

typedef struct {
    int32_t tile;        /* GEMM_FP8_TILE_* chosen */
    int32_t block_m, block_n;
    int32_t waves_k;     /* waves that share a piece's K */
    int32_t threads;     /* per workgroup */
    int32_t staged;      /* 1: operands pass through LDS */
    int32_t widened;     /* 1: multiplied as bf16 (fp32 outputs) */
    int32_t reserved;
    int64_t grid;        /* workgroups */
    int64_t k_blocks;    /* ceil(K / 128) */
    int64_t c_tiles;     /* tiles of C; above grid where workgroups take several in turn */
} gemm_fp8_info_t;

/* C = A * B of 8-bit matrices, each block of products times its scales:
 *   C[i][j] = sum over blocks b of SA[i][b] * SB[jb][b] *
 *             sum over k in block b of A[i][k] * B[j][k],
 * A row-major M x K with "row" scales; B column-major K x N (its N x K
 * transpose, K contiguous: layout RC) with "tile" scales (b_scale_rows 128,
 * jb = j / 128) or "row" scales (b_scale_rows 1, jb = j).
 * a_type, b_type: GEMM_E4M3 or GEMM_E5M2, in any combination.  c_dtype:
 * GEMM_F16, GEMM_BF16 or GEMM_F32; sums over blocks are fp32, rounded once.
 * The sum inside a block is the matrix core's: for 16-bit outputs that of
 * the 8-bit instructions (about 2e-5 off on normal data: each product to about
 * 2^-13 of the largest of 8 neighbours, whatever the sum cancels to); for
 * fp32 outputs both operands are widened to bf16, exactly, and it is fp32's
 * (half the rate).  The order of the sums is fixed for a
 * call's sizes and tile class.
 * accumulate = 1 (fp32 only): C += instead.
 * Leading dimensions are in elements, C may have any; an operand whose base
 * and leading dimension are not multiples of 16 bytes is read into
 * registers by smaller tiles, slower (64 x 4096 x 4100: twice the time of
 * aligned rows, 4096 x 4096 x 4100: 20 times).  No byte at or past column K of
 * a row counts, whatever it holds.
 * Errors: GEMM_ERR_INVALID_ARG (NULL, a negative size or stride, an unknown
 * type, a leading dimension below K or N), GEMM_ERR_ALIGNMENT (C, SA or SB
 * not element-aligned, or a staged tile asked for with other rows than it
 * takes), GEMM_ERR_UNSUPPORTED (accumulate without GEMM_F32, the 256x256
 * tile with it, a tile's rows, or the scales of all its blocks, spanning 2^31
 * bytes),
 * GEMM_ERR_HIP. */
int gemm_run_fp8(gemm_handle_t h, int64_t M, int64_t N, int64_t K,
                 int a_type, int b_type, int c_dtype, int b_scale_rows, int accumulate, int tile,
                 const void *A, int64_t lda, const float *SA, int64_t sa_row, int64_t sa_blk,
                 const void *B, int64_t ldb, const float *SB, int64_t sb_row, int64_t sb_blk,
                 void *C, int64_t ldc, void *stream);

/* What gemm_run_fp8 would launch on a 256-CU device, after the same checks;
 * no HIP call.  NULL pointers are "not given" and skipped. */
int gemm_query_fp8(int64_t M, int64_t N, int64_t K,
                   int a_type, int b_type, int c_dtype, int b_scale_rows, int accumulate, int tile,
                   const void *A, int64_t lda, const float *SA, int64_t sa_row, int64_t sa_blk,
                   const void *B, int64_t ldb, const float *SB, int64_t sb_row, int64_t sb_blk,
                   const void *C, int64_t ldc, gemm_fp8_info_t *info);

/* X (M x K; GEMM_F16, GEMM_BF16 or GEMM_F32) to 8 bits.  Q, S: X by blocks
 * of block_rows x 128.  QT, ST: its transpose (K x M), by blocks of 1 x 128
 * along M, or 128 x 128 (the same values and scales as Q's, transposed).
 * Either pair may be NULL, not both.  Only columns before K (M) of Q (QT) are
 * written.  Errors as above; GEMM_ERR_UNSUPPORTED for 2^24 and more workgroups
 * of 64 x 128 values, 2^23 of 128 x 128 by tiles or with a transpose (about
 * 2^37 values). */
int gemm_quantize_fp8(gemm_handle_t h, int64_t M, int64_t K, int x_dtype, int fp8_type, int block_rows, int pow2,
                      const void *X, int64_t ldx, void *Q, int64_t ldq, float *S, int64_t s_row, int64_t s_blk,
                      void *QT, int64_t ldqt, float *ST, int64_t st_row, int64_t st_blk, void *stream);

#define GEMM_RMS_MAX_D 32768
#define GEMM_RMS_MAX_ROWS (1 << 22)

/* Root-mean-square norm of each row of x + residual, to 8 bits:
 *   h = x + residual, rounded to x's type; rstd = 1 / sqrt(mean(h^2) + eps);
 *   y = h * rstd * w in fp32; Q, S: y by blocks of 1 x 128.
 * X, R, H, Y: M x D of x_dtype (GEMM_F16, GEMM_BF16, GEMM_F32).  W: D
 * values of w_dtype (x_dtype or GEMM_F32).  R may be NULL (h = x); H (h), Y
 * (y, rounded), Q with S, and rstd (M fp32 values) are written where they are
 * not NULL, and one of Q and Y must be given.  H may be X or R (in
 * place).  With D = 0 nothing is written.  GEMM_ERR_UNSUPPORTED above
 * GEMM_RMS_MAX_D or GEMM_RMS_MAX_ROWS, and where the launch would have 2^32
 * threads: GEMM_RMS_MAX_ROWS rows of more than 8192; for the backward pass
 * within 16384 rows of GEMM_RMS_MAX_ROWS, of more than 16384, or more than 12288
 * and no multiple of 8. */
int gemm_rms_fp8(gemm_handle_t h, int64_t M, int64_t D, int x_dtype, int w_dtype, int fp8_type, int pow2, float eps,
                 const void *X, int64_t ldx, const void *R, int64_t ldr, const void *W, void *H, int64_t ldh,
                 void *Y, int64_t ldy, void *Q, int64_t ldq, float *S, int64_t s_row, int64_t s_blk, float *rstd,
                 void *stream);

/* The norm's backward pass, from dy = dL/dy and h, rstd of the forward pass:
 *   dx = dh + rstd (w dy - h rstd^2 mean(w dy h)), dw = sum over rows of dy h rstd.
 * DH (may be NULL): the gradient that reaches h from elsewhere.  dx is the
 * gradient of x and of the residual alike; DX may be DY, DH or H (in place).  DW: D
 * fp32 values, overwritten; rows are added in a fixed order.  workspace:
 * gemm_rms_backward_workspace bytes of device memory, 16-byte aligned, any
 * contents (few rows take none: 0, NULL). */
int gemm_rms_backward(gemm_handle_t h, int64_t M, int64_t D, int x_dtype, int w_dtype,
                      const void *DY, int64_t lddy, const void *H, int64_t ldh, const void *W, const float *rstd,
                      const void *DH, int64_t lddh, void *DX, int64_t lddx, float *DW,
                      void *workspace, int64_t workspace_bytes, void *stream);
int64_t gemm_rms_backward_workspace(int64_t M, int64_t D);

/* ---- a feed-forward block in 16 bits, forward and backward ------------------
 *
 * Products of bf16 or fp16 matrices (dtype GEMM_BF16 or GEMM_F16) with what
 * stands next to them in a feed-forward block done in the same kernel:
 *   H = gemm_gated(X, Wg, Wu), Y = gemm_linear(H, Wd, residual X) forward;
 *   dG, dU, H = gemm_gated_backward(dY, Wd, G, U),
 *   dX = gemm_linear(dG, Wg, dU, Wu, residual dY; layout RR),
 *   dW = gemm_weight_gradient(dG, X), ... backward.
 * Products are summed in fp32 and everything up to an output's rounding is
 * fp32; each output is rounded once, to nearest even, to dtype (weight
 * gradients stay fp32).  The order of the sums is fixed for a call's sizes,
 * alignment and tile class.
 *
 * Activations: relu(z) = max(z, 0), its derivative 0 at 0; gelu(z) = z F(z),
 * F the normal distribution's function; gelu_tanh(z) = z (1 + tanh(sqrt(2 /
 * pi) (z + 0.044715 z^3))) / 2; silu(z) = z / (1 + exp(-z)).  Each is within
 * 2^-16 of its value of z as summed, a derivative within 2^-16 of its two terms (act(z) = z s(z):
 * s and z s'); what is under 2^-126 in size may be 0.  A NaN stays one.
 *
 * Leading dimensions are in elements; all rows may lie at any address that is
 * aligned to their elements; rows on 16 bytes, and with whole lines of 128, are
 * fastest.  No value of
 * a factor outside its matrix counts, whatever it holds.
 *
 * Asynchronous: each enqueues one kernel on `stream`, on the handle's device,
 * and nothing else; nothing is allocated; any number may overlap, and a graph
 * can capture them.  Outputs must not overlap inputs or one another, but where
 * stated.  Sizes of zero are accepted.  Errors: GEMM_ERR_INVALID_ARG (NULL, a
 * negative size, an unknown type, a leading dimension below the row's length),
 * GEMM_ERR_ALIGNMENT (a pointer not aligned to its elements), GEMM_ERR_UNSUPPORTED (a tile class that the
 * operator does not have; 256 rows of a factor with K along its rows, or 64 of
 * one with K across them, that span 2^31 bytes; 2^32 threads), GEMM_ERR_HIP. */
enum { GEMM_ACT_NONE = 0, GEMM_ACT_RELU = 1, GEMM_ACT_GELU = 2, GEMM_ACT_GELU_TANH = 3, GEMM_ACT_SILU = 4 };

/* Part of the sums that one workgroup computes (gated: half of its columns are
 * the second product's).  From 64x64_K4 on each wave takes parts of K of its
 * own.  Weight gradients have
 * those down to 32x32, gated layers those down to 16x32.  GEMM_LINEAR_TILE_AUTO: chosen by
 * the call's sizes. */
enum { GEMM_LINEAR_TILE_AUTO = -1, GEMM_LINEAR_TILE_256x256 = 0, GEMM_LINEAR_TILE_128x256 = 1, GEMM_LINEAR_TILE_128x128 = 2,
       GEMM_LINEAR_TILE_64x64 = 3, GEMM_LINEAR_TILE_64x64_K4 = 4, GEMM_LINEAR_TILE_64x32 = 5, GEMM_LINEAR_TILE_32x32 = 6,
       GEMM_LINEAR_TILE_16x32 = 7, GEMM_LINEAR_TILE_16x16 = 8 };

enum { GEMM_FORM_LINEAR_RC = 0, GEMM_FORM_LINEAR_RR = 1, GEMM_FORM_GATED = 2, GEMM_FORM_GATED_BACKWARD = 3,
       GEMM_FORM_WEIGHT_GRADIENT = 4,
       GEMM_FORM_LINEAR_RC_PAIR = 16, GEMM_FORM_LINEAR_RR_PAIR = 17 };    /* with A2 and B2: for the query */

typedef struct {
    int32_t tile;              /* GEMM_LINEAR_TILE_* chosen */
    int32_t block_m, block_n;  /* outputs of one workgroup */
    int32_t threads;           /* per workgroup */
    int32_t rows16;            /* 1: all the factors' rows start on 16 bytes */
    int32_t reserved;
    int64_t grid;              /* workgroups */
    int64_t k_tiles;           /* ceil(K / 64), K the length of a product's sums */
} gemm_linear_info_t;

/* C = act(A B + A2 B2 + bias) + R, and Z = the activation's argument.
 * A: M x K.  Layout RC: B is column-major (its N x K transpose, as a layer's
 * weight lies); RR: row-major K x N.  A2 and B2: as A and B, both NULL or none.
 * bias: N values of bias_dtype (dtype or GEMM_F32), R: M x N, Z: M x N, each may
 * be NULL.  C, and only C, may take R's place (the same address and leading
 * dimension). */
int gemm_linear(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int layout, int activation, int bias_dtype,
                int tile, const void *A, int64_t lda, const void *B, int64_t ldb, const void *A2, int64_t lda2,
                const void *B2, int64_t ldb2, const void *bias, const void *R, int64_t ldr, void *Z, int64_t ldz,
                void *C, int64_t ldc, void *stream);

/* H = act(G) * U with G = X Wg + bg and U = X Wu + bu.  X: M x K; WG, WU: the
 * N x K transposes of Wg and Wu; BG, BU: N values of bias_dtype, each may be
 * NULL; G, U: M x N, both NULL or none; H: M x N.  H is formed of G and U
 * before their rounding. */
int gemm_gated(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int activation, int bias_dtype, int tile,
               const void *X, int64_t ldx, const void *WG, int64_t ldwg, const void *WU, int64_t ldwu, const void *BG,
               const void *BU, void *G, int64_t ldg, void *U, int64_t ldu, void *H, int64_t ldh, void *stream);

/* With dH = DY W: DG = dH U act'(G), DU = dH act(G), and H = act(G) U again;
 * U and DU NULL: DG = dH act'(G), H = act(G).  DY: M x K, W: row-major K x N (the
 * weight of the layer that takes H, as it lies), the others M x N; H may be
 * NULL.  dH is not rounded. */
int gemm_gated_backward(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int activation, int tile,
                        const void *DY, int64_t lddy, const void *W, int64_t ldw, const void *G, int64_t ldg,
                        const void *U, int64_t ldu, void *DG, int64_t lddg, void *DU, int64_t lddu, void *H, int64_t ldh,
                        void *stream);

/* DW (N x K, fp32) = DC^T A, DC: M x N, A: M x K; DB: N fp32 values, the sums of
 * DC's columns, or NULL.  accumulate = 1: DW += and DB +=.  DB needs K > 0. */
int gemm_weight_gradient(gemm_handle_t h, int64_t M, int64_t N, int64_t K, int dtype, int accumulate, int tile,
                         const void *DC, int64_t lddc, const void *A, int64_t lda, float *DW, int64_t lddw, float *DB,
                         void *stream);

/* What a call of these sizes would launch on a 256-CU device (rows_on_16:
 * whether all its factors' rows start on 16 bytes); M, N and K as the call
 * takes them.  A second product counts in the choice of the class, so such a
 * call has a form of its own here; a bias, a bias's gradient and what else an
 * operator reads or keeps do not.  No HIP call. */
int gemm_query_linear(int form, int64_t M, int64_t N, int64_t K, int dtype, int rows_on_16, int tile,
                      gemm_linear_info_t *info);

/* Static text for a status code (never NULL). */
const char *gemm_status_string(int status);

/* The last hipError_t seen by this thread's failing call (0 if none). */
int gemm_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* PIPEGEMM_H */
