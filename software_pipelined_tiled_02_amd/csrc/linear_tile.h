// linear_tile.h -- the feed-forward kernels' tiles: a workgroup's BM x BN sums
// over K, staged through LDS.
//
// A factor lies in memory with K along its rows ("K inside": a layer's input,
// and its weight in the forward pass) or with K across them ("K outside": the
// weight in the backward pass, both factors of a weight's gradient).  A K-tile
// is 64 deep.  K inside, it is staged as rows of 128 bytes, 16-byte chunks
// swizzled as tile_layout.h describes, and a fragment (16 rows x 32 deep) is
// one 16-byte read per lane; K outside, as 64 rows of the tile's width, and
// the same fragment is two of gfx950's transposing reads.
//
// The K loop is a ring of SLOTS K-tiles.  A K-tile is multiplied row of pieces
// by row of pieces (16 x 16 each).  Once the last row's fragments are in
// registers the wave waits for the next K-tile and crosses the one barrier;
// under the last row's matrix instructions it reads the next K-tile's first
// fragments, and starts the loads that take the place of the one it has read.
#ifndef PIPEGEMM_LINEAR_TILE_H
#define PIPEGEMM_LINEAR_TILE_H

#include "fp8_gemm.h"
#include "linear_common.h"

namespace pg {

typedef _Float16 f16x8l __attribute__((ext_vector_type(8)));

constexpr int kDeep = 64;                    // values of K in a K-tile

template <int XT>
__device__ __forceinline__ f32x4 multiply16(i32x4 x, i32x4 y, f32x4 c) {
    if constexpr (XT == XT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8l, x), __builtin_bit_cast(f16x8l, y), c, 0, 0, 0);
}

// At most N of this wave's LDS accesses are still in flight.
template <int N>
__device__ __forceinline__ void wait_reads() {
    static_assert(N >= 0 && N < 16, "lgkmcnt range");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4) | (N << 8));
    asm volatile("" ::: "memory");
}

// Tile number `tile`: each XCD gets a run of tiles, in bands of 4 tile rows.
__device__ __forceinline__ void place_linear(const LinearArgs& a, int tile, int& tm, int& tn) {
    constexpr int kBand = 4;
    const int w = by_xcd(tile, a.tiles_m * a.tiles_n);
    const int band = kBand * a.tiles_n, gi = w / band, first = gi * kBand;
    const int rows = min(a.tiles_m - first, kBand), in = w - gi * band;
    tm = first + in % rows;
    tn = in / rows;
}

// One factor's part of a tile: ROWS rows (of A, or of B's transpose), staged by
// T threads.  INSIDE: K along the rows.  SPLIT: rows 0-15 of each 32 belong to
// the first of two matrices, rows 16-31 to the second (gated).
template <bool INSIDE, int ROWS, int T, bool SPLIT>
struct Factor {
    static constexpr int L = ROWS * 8 / T;               // chunks of 16 bytes per lane and K-tile
    static constexpr int BYTES = ROWS * 128;
    static constexpr int CR = ROWS / 8;                  // K outside: chunks of a row
    static_assert(ROWS * 8 % T == 0 && L >= 1, "whole chunks per lane");
    static_assert(INSIDE ? T % 128 == 0 : T % (16 * CR) == 0, "a lane's chunks have one place in the swizzle's period");

    const uint8_t* base;             // this wave's matrix, at the tile's first row (column), k = 0
    int64_t ld;                      // bytes from row to row
    uint32_t off[L];                 // a lane's chunks
    int at;                          // K inside: the chunks' first k in a K-tile; K outside: their first column in the tile
    int left;                        // K outside: columns of the matrix from the tile's first on

    // rows: of the matrix from the tile's first on; elements and ld in elements of 2 bytes.
    __device__ __forceinline__ void locate(const void* p, int64_t first, int64_t ld_, int rows, int wave) {
        const int tid = threadIdx.x;
        ld = ld_ * 2;
        left = rows;
        if constexpr (INSIDE) {
            base = (const uint8_t*)p + first * ld;
            const int c = (tid % 8) ^ swz(8, tid / 8);
            at = c * 8;
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int row = (j * T + tid) / 8, r = SPLIT ? (row / 32) * 16 + row % 16 : row;
                // rows past the matrix read one of it: they only feed sums that are not stored
                off[j] = (uint32_t)(r < rows ? r : 0) * (uint32_t)ld + c * 16;
            }
        } else {
            static_assert(INSIDE || !SPLIT, "");
            base = (const uint8_t*)p + first * 2;
            const int k = tid / CR, c = (tid % CR) ^ swz_rr(DT_F16, ROWS * 2, k);
            at = c * 8;
#pragma unroll
            for (int j = 0; j < L; ++j) off[j] = (uint32_t)(j * T / CR + k) * (uint32_t)ld + (c * 8 < rows ? c * 16 : 0);
        }
    }
};

template <int XT, int END, bool AIN, bool BIN, bool DIRECT, int BM, int BN, int WM, int WN, int SLOTS, bool SUMS>
struct Tile {
    static constexpr bool SPLIT = END == END_GATED;
    static constexpr int T = WM * WN * 64;
    static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    typedef Factor<AIN, BM, T, false> FA;
    typedef Factor<BIN, BN, T, SPLIT> FB;
    static constexpr int LA = FA::L, LB = FB::L, LPT = LA + LB;
    static constexpr int SLOT = FA::BYTES + FB::BYTES;
    static constexpr int STRIP_ROW = WTN * 4 + 16, STRIP = 16 * STRIP_ROW;     // fp32, rows padded to other banks
    static constexpr int LDS = max3(SLOTS * SLOT, WM * WN * STRIP, 0);
    static constexpr int OUTS = SPLIT ? WTN / 2 : WTN;   // a wave's outputs per row
    static_assert(LDS <= kLdsBudget && FM % 2 == 0 && (!SPLIT || FN % 2 == 0), "tile");
    static_assert(DIRECT || SLOTS == 2, "register-staged K-tiles: two slots");

    struct State {
        FA a;
        FB b;
        int m0, n0, wave, K, KB, nt;         // nt: K-tiles of all products
        int product;                         // the one that the factors' places are of
    };

    __device__ static __forceinline__ void locate(const LinearArgs& p, State& s, int q) {
        s.product = q;
        s.a.locate(p.A[q], s.m0, p.lda[q], p.M - s.m0, s.wave);
        // gated: a load's 8 rows, and all of a wave's loads, belong to one matrix
        const int w = SPLIT ? (s.wave >> 1) & 1 : q;
        s.b.locate(p.B[w], s.n0, p.ldb[w], p.N - s.n0, s.wave);
    }

    // Where K-tile t's loads come from: one past the last moves nothing (all its
    // offsets are out of range), so that the number in flight is always the same.
    struct Issue {
        __amdgpu_buffer_rsrc_t ra, rb;
        uint32_t outa, outb;                 // K inside: the out-of-range bit for chunks past K
        int rem;                             // values of K from the K-tile's first on
        uint8_t PG_LDS* to;
    };
    template <class F, bool INSIDE>
    __device__ static __forceinline__ __amdgpu_buffer_rsrc_t resource(const F& f, int kb, int rem) {
        int64_t size = rem > 0 ? 0x7fffffff : 0;
        if constexpr (!INSIDE) size = rem > 0 ? min((int64_t)rem * f.ld, (int64_t)0x7fffffff) : 0;
        return __builtin_amdgcn_make_buffer_rsrc((void*)(f.base + (int64_t)kb * (INSIDE ? 128 : kDeep * f.ld)), 0, (int)size,
                                                 kBufferWord3);
    }
    __device__ static __forceinline__ Issue start(const LinearArgs& p, State& s, uint8_t PG_LDS* smem, int t, int slot) {
        if (END == END_LINEAR && t == s.KB && s.product == 0 && p.products == 2) locate(p, s, 1);
        const int kb = END == END_LINEAR && t >= s.KB && p.products == 2 ? t - s.KB : t;
        Issue x;
        x.rem = t < s.nt ? s.K - kb * kDeep : 0;
        x.ra = resource<FA, AIN>(s.a, kb, x.rem);
        x.rb = resource<FB, BIN>(s.b, kb, x.rem);
        x.outa = AIN && s.a.at >= x.rem ? kOutside : 0u;
        x.outb = BIN && s.b.at >= x.rem ? kOutside : 0u;
        x.to = smem + slot * SLOT;
        return x;
    }
    // Load q of a K-tile's LPT, straight into LDS.
    __device__ static __forceinline__ void load(const State& s, const Issue& x, int q) {
        if (q < LA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(x.ra, (void PG_LDS*)(x.to + (q * T + 64 * s.wave) * kChunk), 16,
                                                     s.a.off[q] | x.outa, 0, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                x.rb, (void PG_LDS*)(x.to + FA::BYTES + ((q - LA) * T + 64 * s.wave) * kChunk), 16,
                s.b.off[q - LA] | x.outb, 0, 0, 0);
    }

    // K inside and not a multiple of 8: the values at and past K of the chunk
    // that holds K - 1 become zero (what lies there may be a NaN).
    template <int ROWS>
    __device__ static __forceinline__ void clear_rows(uint8_t PG_LDS* rows, int k) {
        const int c = k / 8, keep = k % 8;
        for (int row = threadIdx.x; row < ROWS; row += T) {
            i32x4 PG_LDS* p = (i32x4 PG_LDS*)(rows + (row * 8 + (c ^ swz(8, row))) * kChunk);
            i32x4 v = *p;
#pragma unroll
            for (int w = 0; w < 4; ++w) v[w] = keep >= 2 * w + 2 ? v[w] : keep == 2 * w + 1 ? v[w] & 0xffff : 0;
            *p = v;
        }
    }
    __device__ static __forceinline__ bool cut(const State& s, int t) {      // K-tile t has such a chunk
        return (AIN || BIN) && s.K % 8 != 0 && (t == s.KB - 1 || t == s.nt - 1);
    }
    __device__ static __forceinline__ void clear_tail(const State& s, uint8_t PG_LDS* slot) {
        if constexpr (AIN) clear_rows<BM>(slot, s.K % kDeep);
        if constexpr (BIN) clear_rows<BN>(slot + FA::BYTES, s.K % kDeep);
        barrier();
    }

    // ---- rows at any address: through registers ---------------------------------

    // Eight values of which `n` are there; the others become zero and are not read.
    __device__ static __forceinline__ i32x4 load_some(__amdgpu_buffer_rsrc_t r, uint32_t off, int n) {
        const uint32_t vb = n > 0 && n < 8 ? 2u * n : 0u;
        i32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, n >= 8 ? off : kOutside, 0, 0);
        const i32x2 p8 = __builtin_amdgcn_raw_buffer_load_b64(r, (vb & 8) ? off : kOutside, 0, 0);
        const int p4 = (int)__builtin_amdgcn_raw_buffer_load_b32(r, (vb & 4) ? off + (vb & 8) : kOutside, 0, 0);
        const int p2 = (int)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (vb & 2) ? off + (vb & 12) : kOutside, 0, 0);
        const uint32_t d4 = (vb & 8) >> 2, d2 = (vb & 12) >> 2;
        v[0] |= p8[0] | (d4 == 0 ? p4 : 0) | (d2 == 0 ? p2 : 0);
        v[1] |= p8[1] | (d2 == 1 ? p2 : 0);
        v[2] |= (d4 == 2 ? p4 : 0) | (d2 == 2 ? p2 : 0);
        v[3] |= d2 == 3 ? p2 : 0;
        return v;
    }
    template <class F, bool INSIDE>
    __device__ static __forceinline__ void gather(const F& f, __amdgpu_buffer_rsrc_t r, uint32_t out, int rem, i32x4* v) {
        const bool ragged = INSIDE ? rem > 0 && rem < kDeep : f.left < F::CR * 8;
#pragma unroll
        for (int j = 0; j < F::L; ++j) {
            // (K outside: a chunk's place past the matrix was moved to its first one, whole or not)
            if (ragged) v[j] = load_some(r, f.off[j], INSIDE ? rem - f.at : min(f.at < f.left ? f.left - f.at : f.left, 8));
            else v[j] = __builtin_amdgcn_raw_buffer_load_b128(r, f.off[j] | out, 0, 0);
        }
    }
    __device__ static __forceinline__ void gather(const State& s, const Issue& x, i32x4 (&v)[LPT]) {
        gather<FA, AIN>(s.a, x.ra, x.outa, x.rem, v);
        gather<FB, BIN>(s.b, x.rb, x.outb, x.rem, v + LA);
    }
    __device__ static __forceinline__ void put(const Issue& x, const i32x4 (&v)[LPT]) {
#pragma unroll
        for (int j = 0; j < LA; ++j) *(i32x4 PG_LDS*)(x.to + (j * T + threadIdx.x) * kChunk) = v[j];
#pragma unroll
        for (int j = 0; j < LB; ++j) *(i32x4 PG_LDS*)(x.to + FA::BYTES + (j * T + threadIdx.x) * kChunk) = v[LA + j];
    }

    // ---- fragments -------------------------------------------------------------------

    // Lane (r = lane % 16, g = lane / 16) of a fragment holds row r and values
    // 8 g .. + 7 of its 32 deep.  K inside: `lane[h]` is that chunk's offset in
    // 16 rows, at depth 32 h.  K outside: `lane[i]` is the offset of what the
    // lane hands to the first transposing read of fragment i: 4 columns of row
    // 8 g + (lane % 16) / 4; the second read is 4 rows on.
    template <bool INSIDE, int ROWS, int F>
    struct Reader {
        static constexpr int N = INSIDE ? 2 : F;
        uint32_t lane[N];
        __device__ __forceinline__ void locate(int first) {      // the wave's first row of the tile
            const int l = threadIdx.x & 63, r = l & 15, g = l >> 4;
            if constexpr (INSIDE) {
#pragma unroll
                for (int h = 0; h < 2; ++h) lane[h] = (uint32_t)((first + r) * 8 + ((4 * h + g) ^ swz(8, r))) * kChunk;
            } else {
                const int k = rr_lane_k(DT_F16, true, l);
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    const int n = first + 16 * i + rr_lane_n(DT_F16, true, l);
                    lane[i] = (uint32_t)(k * ROWS * 2 + ((n / 8) ^ swz_rr(DT_F16, ROWS * 2, k)) * kChunk + n % 8 * 2);
                }
            }
        }
        __device__ __forceinline__ i32x4 read(const uint8_t PG_LDS* rows, int i, int h) const {
            if constexpr (INSIDE) {
                return *(const i32x4 PG_LDS*)(rows + lane[h] + i * 16 * 128);
            } else {
                // Inline assembly: behind loads into LDS the compiler drains every
                // load before a transposing read, which it cannot tell apart from
                // them.  It does not see these reads' latency either, so the loop
                // waits for them itself.
                const uint32_t p = (uint32_t)(uintptr_t)(rows + lane[i]);
                i32x2 lo, hi;
                if (h == 0)
                    asm volatile("ds_read_b64_tr_b16 %0, %2\n\tds_read_b64_tr_b16 %1, %2 offset:%3"
                                 : "=&v"(lo), "=&v"(hi) : "v"(p), "i"(4 * ROWS * 2) : "memory");
                else
                    asm volatile("ds_read_b64_tr_b16 %0, %2 offset:%3\n\tds_read_b64_tr_b16 %1, %2 offset:%4"
                                 : "=&v"(lo), "=&v"(hi) : "v"(p), "i"(32 * ROWS * 2), "i"(36 * ROWS * 2) : "memory");
                return i32x4{lo[0], lo[1], hi[0], hi[1]};
            }
        }
    };
    typedef Reader<AIN, BM, FM> RA;
    typedef Reader<BIN, BN, FN> RB;

    __device__ static __forceinline__ void run(const LinearArgs& p, uint8_t PG_LDS* smem) {
        State s;
        s.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        s.K = p.K;
        s.KB = (p.K + kDeep - 1) / kDeep;
        s.nt = END == END_LINEAR ? s.KB * p.products : s.KB;
        int tm, tn;
        place_linear(p, blockIdx.x, tm, tn);
        s.m0 = tm * BM;
        s.n0 = tn * (SPLIT ? BN / 2 : BN);
        locate(p, s, 0);
        const int wm = s.wave / WN, wn = s.wave % WN;
        RA ra;
        RB rb;
        ra.locate(wm * WTM);
        rb.locate(wn * WTN);

        f32x4 acc[FM][FN], sums[SUMS ? FM : 1];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < (SUMS ? FM : 1); ++i) sums[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const bool adds = SUMS && tn == 0;
        const int one = XT == XT_BF16 ? 0x3f803f80 : 0x3c003c00;
        const i32x4 ones = {one, one, one, one};

        i32x4 staged[DIRECT ? 1 : LPT];
        Issue x;
        if constexpr (DIRECT) {
#pragma unroll
            for (int t = 0; t < SLOTS; ++t) {
                x = start(p, s, smem, t, t);
#pragma unroll
                for (int q = 0; q < LPT; ++q) load(s, x, q);
            }
            wait_loads<(SLOTS - 1) * LPT>();
        } else {
            x = start(p, s, smem, 0, 0);
            gather(s, x, staged);
            put(x, staged);
            x = start(p, s, smem, 1, 1);
            gather(s, x, staged);
        }
        barrier();
        if (DIRECT && cut(s, 0)) clear_tail(s, smem);

        i32x4 fa[2][2], fb[FN][2];
        auto tile_a = [&](int slot) { return smem + slot * SLOT; };
        auto tile_b = [&](int slot) { return smem + slot * SLOT + FA::BYTES; };
#pragma unroll
        for (int h = 0; h < 2; ++h) fa[0][h] = ra.read(tile_a(0), 0, h);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < FN; ++j) fb[j][h] = rb.read(tile_b(0), j, h);

        constexpr bool WAITS = !AIN || !BIN;     // the transposing reads' own waits
        int slot = 0;
        for (int t = 0; t < s.nt; ++t) {
            const int next = slot + 1 == SLOTS ? 0 : slot + 1;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                if (i + 1 == FM) {
                    // every fragment of K-tile t is read: on to the next one
                    if constexpr (DIRECT) {
                        wait_loads<(SLOTS - 2) * LPT>();     // K-tile t + 1 has landed (this wave's part)
                        barrier();                           // ... everyone's, and slot t is free
                        if (cut(s, t + 1)) clear_tail(s, smem + next * SLOT);
                        x = start(p, s, smem, t + SLOTS, slot);
                    } else {
                        // (slot `next` was read before the last barrier)
                        x.to = smem + next * SLOT;
                        put(x, staged);
                        barrier();
                        x = start(p, s, smem, t + 2, slot);
                        gather(s, x, staged);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (WAITS) {
                        // the row's fragments have landed; a K-tile's first row: all but B's second halves, then those
                        if (i == 0 && h == 0) wait_reads<FN * (BIN ? 1 : 2)>();
                        else if (h == 0 || i == 0) wait_reads<0>();
                        __builtin_amdgcn_sched_barrier(0);
                    }
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        const int u = h * FN + j;
                        acc[i][j] = multiply16<XT>(fb[j][h], fa[i & 1][h], acc[i][j]);
                        if constexpr (SUMS) {
                            if (adds && j == 0 && i % WN == wn) sums[i] = multiply16<XT>(ones, fa[i & 1][h], sums[i]);
                        }
                        if (i + 1 < FM) {
                            // the next row's fragments (a K-tile's second row: behind the wait for B's second halves)
                            if (u == (i == 0 ? FN : 0)) {
                                fa[(i + 1) & 1][0] = ra.read(tile_a(slot), i + 1, 0);
                                fa[(i + 1) & 1][1] = ra.read(tile_a(slot), i + 1, 1);
                            }
                        } else {
                            if (u == 0) {
                                fa[0][0] = ra.read(tile_a(next), 0, 0);
                                fa[0][1] = ra.read(tile_a(next), 0, 1);
                            }
                            fb[j][h] = rb.read(tile_b(next), j, h);
                            if constexpr (DIRECT) {
#pragma unroll
                                for (int q = u * LPT / (2 * FN); q < (u + 1) * LPT / (2 * FN); ++q) load(s, x, q);
                            }
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            slot = next;
        }
        wait_loads<0>();                     // no write into LDS outlives the K loop, and no read is in flight
        barrier();
        if constexpr (WAITS) {
            // the last reads' registers are not free before that
            asm volatile("" ::"v"(fa[0][0]), "v"(fa[0][1]));
#pragma unroll
            for (int j = 0; j < FN; ++j) asm volatile("" ::"v"(fb[j][0]), "v"(fb[j][1]));
        }

        if constexpr (SUMS) {
            if (adds)
#pragma unroll
                for (int i = 0; i < FM; ++i) {
                    // every column of the piece is the row's sum
                    const int m = s.m0 + wm * WTM + 16 * i + (threadIdx.x & 15);
                    if (i % WN == wn && (threadIdx.x & 63) < 16 && m < p.M)
                        p.sums[m] = p.accumulate ? p.sums[m] + sums[i][0] : sums[i][0];
                }
        }
        store(p, s, smem, wm, wn, acc);
    }

    // A wave's sums: 16 rows at a time go through its own strip of LDS and
    // come back as eight neighbouring columns per lane, whole rows of the
    // wave's block at a time, for the ending.
    __device__ static __forceinline__ void store(const LinearArgs& p, const State& s, uint8_t PG_LDS* smem, int wm, int wn,
                                                 const f32x4 (&acc)[FM][FN]) {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
        constexpr int LANES = OUTS / 8, PASS = 64 / LANES, Q = 16 / PASS > 0 ? 16 / PASS : 1;
        uint8_t PG_LDS* strip = smem + s.wave * STRIP;
        const int row = lane / LANES, c = lane % LANES * 8;
        const int64_t n = s.n0 + wn * OUTS + c;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int64_t m = s.m0 + wm * WTM + 16 * i + row;
            Beside<XT, END> beside[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (row < 16 && m + q * PASS < p.M && n < p.N) beside[q] = fetch_beside<XT, END>(p, m + q * PASS, n);
#pragma unroll
            for (int j = 0; j < FN; ++j) *(f32x4 PG_LDS*)(strip + r * STRIP_ROW + (16 * j + 4 * g) * 4) = acc[i][j];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (row >= 16) break;
                const uint8_t PG_LDS* at = strip + (row + q * PASS) * STRIP_ROW + (SPLIT ? c / 16 * 32 + c % 16 : c) * 4;
                float v[8], u[8];
                const f32x4 v0 = *(const f32x4 PG_LDS*)at, v1 = *(const f32x4 PG_LDS*)(at + 16);
                f32x4 u0 = v0, u1 = v1;
                if constexpr (SPLIT) {
                    u0 = *(const f32x4 PG_LDS*)(at + 64);
                    u1 = *(const f32x4 PG_LDS*)(at + 80);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) { v[e] = v0[e]; v[4 + e] = v1[e]; u[e] = u0[e]; u[4 + e] = u1[e]; }
                if (m + q * PASS < p.M && n < p.N) finish8<XT, END>(p, m + q * PASS, n, beside[q], v, u);
            }
        }
    }
};

template <int XT, int END, bool AIN, bool BIN, bool DIRECT, int BM, int BN, int WM, int WN, int SLOTS, bool SUMS>
__global__ void __launch_bounds__(512) linear_tile(LinearArgs p) {
    typedef Tile<XT, END, AIN, BIN, DIRECT, BM, BN, WM, WN, SLOTS, SUMS> S;
    __shared__ __attribute__((aligned(16))) uint8_t smem[S::LDS];
    S::run(p, (uint8_t PG_LDS*)smem);
}

// The classes of one ending: waves in rows x columns, so that a wave's rows of
// outputs are as long as they can be.
template <int XT, int END, bool AIN, bool BIN, bool SUMS>
const void* linear_by_tile(int tile, bool rows16) {
    constexpr bool G = END == END_GATED;
    switch (tile) {
    case LINEAR_TILE_256:
        return rows16 ? (const void*)&linear_tile<XT, END, AIN, BIN, true, 256, 256, G ? 4 : 2, G ? 2 : 4, 2, SUMS> : nullptr;
    case LINEAR_TILE_128:
        return rows16 ? (const void*)&linear_tile<XT, END, AIN, BIN, true, 128, 128, G ? 4 : 2, G ? 2 : 4, 4, SUMS>
                      : (const void*)&linear_tile<XT, END, AIN, BIN, false, 128, 128, G ? 4 : 2, G ? 2 : 4, 2, SUMS>;
    case LINEAR_TILE_64:
        return rows16 ? (const void*)&linear_tile<XT, END, AIN, BIN, true, 64, 64, 2, 2, 4, SUMS>
                      : (const void*)&linear_tile<XT, END, AIN, BIN, false, 64, 64, 2, 2, 2, SUMS>;
    default: return nullptr;
    }
}
template <int END, bool AIN, bool BIN, bool SUMS>
const void* linear_by_type(int xt, int tile, bool rows16) {
    return xt == XT_BF16 ? linear_by_tile<XT_BF16, END, AIN, BIN, SUMS>(tile, rows16)
                         : linear_by_tile<XT_F16, END, AIN, BIN, SUMS>(tile, rows16);
}

}  // namespace pg

#endif
