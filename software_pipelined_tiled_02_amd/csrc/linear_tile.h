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
// The K loop goes through rings of SA K-tiles of A and SB of B, with one barrier a
// K-tile, in which each wave reads its fragments behind matrix instructions of the
// fragments before.
//
// Large products are bound by the matrix cores at the clock that power leaves
// them: 256 x 256 tiles take 2352 cycles a K-tile, of which 2048 are matrix
// instructions (bf16 8192^3 742 us, 1480 TFLOP/s; K outside in both factors,
// 8192 x 4096 x 8192, 409 us, 1340).  Smaller tiles are bound by LDS and the CU's
// loads: per K-tile 128 x 256 moves 96 KB of fragments and 48 KB of loads beside
// 1024 cycles of products, 128 x 128 64 and 32 KB beside 512 (1024 x 4096 x 4096,
// one tile per CU: 32 us, 1060 TFLOP/s; 38 us with factors from HBM).
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

// The same written in place: the sum's registers are the destination's, and lie
// in the second half of the register file.  (Left to itself the compiler moves
// a wave's 64 sums of four between registers at every K-tile.)  It does not see
// these as matrix instructions, so the loop pads their hazards itself.
template <int XT>
__device__ __forceinline__ void multiply16_in_place(i32x4 x, i32x4 y, i32x4& c) {
    if constexpr (XT == XT_BF16) asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(x), "v"(y));
    else asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(x), "v"(y));
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

// Swizzle of a K-tile whose factor has K outside: row k (of `row_bytes`) has its
// 16-byte chunk c in place c ^ out_swz.  A clock of the transposing read takes 32
// bytes of rows 0-3 and of rows 8-11 (of each 16); rows of 256 bytes or more all
// start in one bank, of which these 8 pieces have to fill all 64 (tile_layout.h has
// the probe's figures): bits 0, 1 and 3 of k move a piece.  Shorter rows start
// 128 or 64 bytes apart, and need fewer of them.
constexpr int out_swz(int row_bytes, int k) {
    return row_bytes >= 256 ? swz_rr(DT_F16, row_bytes, k)
         : row_bytes == 128 ? ((k >> 1) & 1) * 4 ^ ((k >> 3) & 1) * 2
         : row_bytes == 64  ? ((k >> 3) & 1) * 2
                            : 0;
}

// K as whole K-tiles and the values of one more, which is multiplied first.  Rows
// that do not start on 16 bytes (`apart`) have their last K-tile there, whole or
// not: all the others are read without a look at where rows and the matrix end.
// With K outside, their last row's last value may share a dword with the next row's
// first one, so that many bytes more (`over`) are in range.
struct Depth { int whole, part, over; };
__device__ __forceinline__ Depth depth_of(int K, bool apart) {
    const int whole = (apart && K > 0 ? K - 1 : K) / kDeep;
    return Depth{whole, K - whole * kDeep, apart ? 2 : 0};
}

// Eight values of which `n` are there; the others become zero and are not read.
__device__ __forceinline__ i32x4 load_some(__amdgpu_buffer_rsrc_t r, uint32_t off, int n) {
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

// One factor's part of a tile: ROWS rows (of A, or of B's transpose), staged by
// T threads (64: a wave by itself).  INSIDE: K along the rows.  SPLIT: rows 0-15
// of each 32 belong to the first of two matrices, rows 16-31 to the second
// (gated): a load's 8 rows belong to one, and so do all of a wave's where several
// waves share the loads.
template <bool INSIDE, int ROWS, int T, bool SPLIT, int P>
struct Factor {
    static constexpr int L = ROWS * 8 / T;               // chunks of 16 bytes per lane and K-tile
    static constexpr int BYTES = ROWS * 128;
    static constexpr int CR = ROWS / 8;                  // K outside: chunks of a row
    static_assert(ROWS * 8 % T == 0 && L >= 1, "whole chunks per lane");
    // A lane's chunks have one place in the swizzle's period of 16 rows, or (loads 8
    // rows apart) two in turn, 2 chunks apart.
    static constexpr bool TURNS = INSIDE ? T % 128 != 0 : T % (16 * CR) != 0;
    static_assert(INSIDE ? T % 64 == 0 : T % (8 * CR) == 0, "places in the swizzle's period");
    static_assert((swz(8, 0) ^ swz(8, 8)) == 2 && (swz(8, 7) ^ swz(8, 15)) == 2, "the swizzle's row bit 3");
    static constexpr bool BOTH = SPLIT && T == 64;       // loads of the two matrices in turn

    const uint8_t* base[P];          // this wave's matrix of each product, at the tile's first row (column), k = 0
    int64_t ld[P];                   // bytes from row to row
    uint32_t off[P][L];              // a lane's chunks
    int at;                          // K inside: the chunks' first k in a K-tile; K outside: their first column in the tile
    int left;                        // rows (K outside: columns) of the matrix from the tile's first on
    const uint8_t* base_u;           // BOTH: of the second matrix
    const uint8_t* from_u;

    // The K-tile whose loads are next.  The order in which they are multiplied:
    // each product's last one, where it goes apart, then all others, from
    // number `first` on and round to it again.  Behind the last, a K-tile moves
    // nothing (all is out of range), so that the number of loads in flight is
    // always the same.
    const uint8_t* from;             // its first row or column
    int size;                        // bytes from there on that may be read
    int rem;                         // values of K from there on
    int kb;                          // its number among those behind the ones apart, of all products
    int more;                        // K-tiles from this one on
    bool second;                     // of the second product

    __device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(int j) const {
        return __builtin_amdgcn_make_buffer_rsrc((void*)(BOTH && ((j >> 1) & 1) ? from_u : from), 0, size, kBufferWord3);
    }
    __device__ __forceinline__ uint32_t offset(int j) const { return P == 2 && second ? off[P - 1][j] : off[0][j]; }
    // The same, out of range where the chunk lies past K (K outside: the size sees to that).
    __device__ __forceinline__ uint32_t offset_in(int j) const {
        return offset(j) | (INSIDE && (TURNS && (j & 1) ? at ^ 16 : at) >= rem ? kOutside : 0u);
    }

    // Load j of the K-tile, straight into LDS (16 bytes from any address: all K-tiles
    // through registers took 50 us at 500 x 4104 x 4100, this 42).  `part`: it may not be
    // a whole one.
    __device__ __forceinline__ void load(int j, uint8_t PG_LDS* to, int wave, bool part = false) const {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(resource(j), (void PG_LDS*)(to + (j * T + 64 * wave) * kChunk), 16,
                                                 part ? offset_in(j) : offset(j), 0, 0, 0);
    }
    __device__ __forceinline__ void load_all(uint8_t PG_LDS* to, int wave) const {
#pragma unroll
        for (int j = 0; j < L; ++j) load(j, to, wave, true);
    }

    // The K-tile through registers: the chunks at the ends of rows are read only as far
    // as these go.
    __device__ __forceinline__ void carry(uint8_t PG_LDS* to, int tid) const {
        const bool ragged = INSIDE ? rem < kDeep : left < CR * 8;
        i32x4 v[L];
#pragma unroll
        for (int j = 0; j < L; ++j) {
            const int c = TURNS && (j & 1) ? at ^ 16 : at;
            // (K outside: a chunk's place past the matrix was moved to its first one, whole or not)
            if (ragged) v[j] = load_some(resource(j), offset(j), INSIDE ? rem - c : min(c < left ? left - c : left, 8));
            else v[j] = __builtin_amdgcn_raw_buffer_load_b128(resource(j), offset(j), 0, 0);
        }
#pragma unroll
        for (int j = 0; j < L; ++j) *(i32x4 PG_LDS*)(to + (j * T + tid) * kChunk) = v[j];
    }

    // K-tile number i of the order.
    __device__ __forceinline__ void start(int i, Depth d, int first) {
        const int parts = d.part != 0 ? P : 0;
        more = parts + P * d.whole - i;
        int q = 0, k = d.whole;
        rem = d.part;
        kb = first;
        if (i >= parts) {
            kb = i - parts + first;
            kb = kb >= P * d.whole ? kb - P * d.whole : kb;
            q = P == 2 && kb >= d.whole ? 1 : 0;
            k = q ? kb - d.whole : kb;
            rem = kDeep;
        } else {
            q = i;
        }
        second = q == 1;
        const int64_t row = second ? ld[P - 1] : ld[0];
        from = (second ? base[P - 1] : base[0]) + (int64_t)k * (INSIDE ? 128 : kDeep * row);
        rem = more > 0 ? rem : 0;
        size = more <= 0 ? 0 : INSIDE ? 0x7fffffff : (int)(rem * row) + (i >= parts ? d.over : 0);
        if constexpr (BOTH) from_u = base_u + (int64_t)k * 128;
    }
    // On to the next one, both whole (or behind the last).  Without a branch: one
    // in the K loop costs some 50 cycles where it is taken (256 x 256 tiles: 2706
    // cycles a K-tile with three of them, 2460 without).
    __device__ __forceinline__ void next(Depth d) {
        const int64_t row = P == 2 && second ? ld[P - 1] : ld[0];
        const uint8_t* to = from + (INSIDE ? 128 : kDeep * row);
        ++kb;
        --more;
        if constexpr (P == 2) {
            second = kb == d.whole ? true : second;
            to = kb == d.whole ? base[P - 1] : to;
        }
        const bool round = kb == P * d.whole;
        to = round ? base[0] : to;
        second = round ? false : second;
        kb = round ? 0 : kb;
        from = to;
        size = more > 0 ? (INSIDE ? 0x7fffffff : (int)(kDeep * (P == 2 && second ? ld[P - 1] : ld[0])) + d.over) : 0;
    }

    // Product q's matrix p; elements of 2 bytes, ld_ in elements.  tid: of T.
    // BOTH: p_u, ld_u are the second matrix's.
    __device__ __forceinline__ void locate(int tid, int q, const void* p, int64_t first, int64_t ld_, int rows,
                                           const void* p_u = nullptr, int64_t ld_u = 0) {
        ld[q] = ld_ * 2;
        left = rows;
        if constexpr (INSIDE) {
            base[q] = (const uint8_t*)p + first * ld[q];
            if constexpr (BOTH) base_u = (const uint8_t*)p_u + first * ld_u * 2;
            const int c = (tid % 8) ^ swz(8, tid / 8);
            at = c * 8;
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int row = (j * T + tid) / 8, r = SPLIT ? (row / 32) * 16 + row % 16 : row;
                const int64_t step = BOTH && ((j >> 1) & 1) ? ld_u * 2 : ld[q];
                // rows past the matrix read one of it: they only feed sums that are not stored
                off[q][j] = (uint32_t)(r < rows ? r : 0) * (uint32_t)step + (TURNS && (j & 1) ? c ^ 2 : c) * 16;
            }
        } else {
            base[q] = (const uint8_t*)p + first * 2;
            const int k = tid / CR, c = (tid % CR) ^ out_swz(ROWS * 2, k);
            at = c * 8;
#pragma unroll
            for (int j = 0; j < L; ++j) {
                const int cj = TURNS && (j & 1) ? c ^ 2 : c;
                off[q][j] = (uint32_t)(j * T / CR + k) * (uint32_t)ld[q] + (cj * 8 < rows ? cj * 16 : 0);
            }
        }
    }
};

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
                lane[i] = (uint32_t)(k * ROWS * 2 + ((n / 8) ^ out_swz(ROWS * 2, k)) * kChunk + n % 8 * 2);
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

// K inside and not a multiple of 8: the values at and past K of the chunk
// that holds K - 1 become zero (what lies there may be a NaN).
template <int ROWS, int T>
__device__ __forceinline__ void clear_rows(int tid, uint8_t PG_LDS* rows, int k) {
    const int c = k / 8, keep = k % 8;
    for (int row = tid; row < ROWS; row += T) {
        i32x4 PG_LDS* p = (i32x4 PG_LDS*)(rows + (row * 8 + (c ^ swz(8, row))) * kChunk);
        i32x4 v = *p;
#pragma unroll
        for (int w = 0; w < 4; ++w) v[w] = keep >= 2 * w + 2 ? v[w] : keep == 2 * w + 1 ? v[w] & 0xffff : 0;
        *p = v;
    }
}

// Sums of A's rows in vector instructions: pair e of a chunk's eight values, added.
// (Beside matrix instructions in inline assembly others, in branches, made the
// compiler move their sums.)
template <int XT>
__device__ __forceinline__ float add_pair(i32x4 chunk, int e, float sum) {
    const uint32_t w = (uint32_t)(e == 0 ? chunk[0] : e == 1 ? chunk[1] : e == 2 ? chunk[2] : chunk[3]);
    if constexpr (XT == XT_BF16) {
        return sum + __uint_as_float(w << 16) + __uint_as_float(w & 0xffff0000u);
    } else {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 h = __builtin_bit_cast(f16x2, w);
        return sum + (float)h[0] + (float)h[1];
    }
}

template <int XT, int END, bool AIN, bool BIN, int BM, int BN, int WM, int WN, int SA, int SB, int EXTRA>
struct Tile {
    static constexpr bool SPLIT = END == END_GATED;
    static constexpr bool SUMS = END == END_WEIGHT && EXTRA != 0;        // of A's rows too
    static constexpr int P = END == END_LINEAR && EXTRA != 0 ? 2 : 1;    // products
    static constexpr int T = WM * WN * 64;
    static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    typedef Factor<AIN, BM, T, false, P> FA;
    typedef Factor<BIN, BN, T, SPLIT, P> FB;
    static constexpr int LA = FA::L, LB = FB::L, LPT = LA + LB;
    static constexpr int RING_A = SA * FA::BYTES, RING = RING_A + SB * FB::BYTES;
    // Loads that may be in flight when K-tile t + 1 has to be there: those of B's
    // K-tiles t + 2 .. t + SB - 1 and of A's t + 2 .. t + SA - 1.
    static constexpr int FLYING = (SB - 2) * LB + (SA - 2) * LA;
    // The ending's parts of LDS: PIECES rows of pieces of each wave at a time, in
    // fp32, rows padded to other banks.
    static constexpr int STRIP_ROW = WTN * 4 + 16, PIECES = FM == 8 ? 4 : FM;
    static constexpr int LDS = max3(RING, WM * WN * PIECES * 16 * STRIP_ROW, 0);
    static constexpr bool QUADS = FM == 8 && FN == 8;    // one wave per SIMD
    static constexpr int OUTS = SPLIT ? WTN / 2 : WTN;   // a wave's outputs per row
    static_assert(LDS <= kLdsBudget && FM % 2 == 0 && (!SPLIT || FN % 2 == 0), "tile");
    static_assert(QUADS ? SA == 3 && SB == 2 : SA == SB, "slots");

    struct State {
        FA a;
        FB b;
        int m0, n0, wave, nt;                // nt: K-tiles of all products
        Depth deep;
        bool apart;                          // rows that do not start on 16 bytes
        int rot;                             // the K-tile that is multiplied first
    };

    // What clear_rows clears, in the K-tiles in places 0 .. P - 1, once they have landed.
    template <class PA, class PB>
    __device__ static __forceinline__ void clear_tails(const State& s, PA tile_a, PB tile_b) {
        if (!(AIN || BIN) || s.apart || s.deep.part % 8 == 0) return;
        wait_loads<0>();
        barrier();
#pragma unroll
        for (int t = 0; t < P; ++t) {
            if constexpr (AIN) clear_rows<BM, T>(threadIdx.x, tile_a(t), s.deep.part);
            if constexpr (BIN) clear_rows<BN, T>(threadIdx.x, tile_b(t), s.deep.part);
        }
        barrier();
    }

    // K-tile number t of the order, one of the first, into its places.
    __device__ static __forceinline__ void begin(const State& s, int t, uint8_t PG_LDS* a, uint8_t PG_LDS* b) {
        if (t < P && s.apart) {
            s.a.carry(a, threadIdx.x);
            s.b.carry(b, threadIdx.x);
        } else {
            s.b.load_all(b, s.wave);
            s.a.load_all(a, s.wave);
        }
    }

    // ---- fragments -------------------------------------------------------------------

    typedef Reader<AIN, BM, FM> RA;
    typedef Reader<BIN, BN, FN> RB;

    __device__ static __forceinline__ void run(const LinearArgs& p, uint8_t PG_LDS* smem) {
        State s;
        s.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        s.apart = p.apart != 0;
        s.deep = depth_of(p.K, s.apart);
        s.nt = P * ((p.K + kDeep - 1) / kDeep);
        int tm, tn;
        place_linear(p, blockIdx.x, tm, tn);
        s.m0 = tm * BM;
        s.n0 = tn * (SPLIT ? BN / 2 : BN);
        // With more tiles than one round, XCD x starts at K-tile 9 x.
        s.rot = gridDim.x > 256 && s.deep.whole > 0 ? (int)((blockIdx.x & 7) * 9u % (unsigned)(P * s.deep.whole)) : 0;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            s.a.locate(threadIdx.x, q, p.A[q], s.m0, p.lda[q], p.M - s.m0);
            // gated: a load's 8 rows, and all of a wave's loads, belong to one matrix
            const int w = SPLIT ? (s.wave >> 1) & 1 : q;
            s.b.locate(threadIdx.x, q, p.B[w], s.n0, p.ldb[w], p.N - s.n0);
        }
        const int wm = s.wave / WN, wn = s.wave % WN;
        RA ra;
        RB rb;
        ra.locate(wm * WTM);
        rb.locate(wn * WTN);

        if constexpr (QUADS) {
            // (apart to the end: where the two ways met, the sums would be moved before they are there)
            if (SUMS && tn == 0) run_quads<SUMS>(p, s, smem, ra, rb, wm, wn);
            else run_quads<false>(p, s, smem, ra, rb, wm, wn);
        } else {
            run_steps(p, s, smem, ra, rb, wm, wn, tn == 0);
        }
    }

    // Sums of A's rows: products with a fragment of ones, whose every column is
    // the row's sum.
    __device__ static __forceinline__ i32x4 ones() {
        constexpr int two = XT == XT_BF16 ? 0x3f803f80 : 0x3c003c00;
        return i32x4{two, two, two, two};
    }
    __device__ static __forceinline__ void store_sums(const LinearArgs& p, int first, float v) {
        const int m = first + (threadIdx.x & 15);
        if ((threadIdx.x & 63) < 16 && m < p.M) p.sums[m] = p.accumulate ? p.sums[m] + v : v;
    }

    // ---- both steps' fragments in registers ----------------------------------------------
    //
    // A K-tile is two steps, 32 deep each.  While a step's pieces are multiplied, the
    // other set of registers takes the next step's fragments, evenly, since LDS
    // is nearly as busy as the matrix cores (a 128 x 256 tile by four waves: 96 KB of
    // fragments and 48 KB of loads in 1024 cycles of products).  When the first
    // step is done all of a K-tile's fragments are in registers: there the wave
    // waits for the next K-tile and crosses the barrier.  The loads that take the
    // place of the K-tile it has read are spread from there on too, over a K-tile's
    // time.  The loop begins behind the barrier, where no LDS read is in flight:
    // across its end the compiler would wait for all of them.  (Row by row of
    // pieces, loads in a burst behind the barrier: 500 x 8192 x 4096 gated 62.8 us
    // by 128 x 256 tiles, this 54.1; 1024 x 4096 x 4096 36.8 and 32 by 128 x 128.)
    struct Steps {
        f32x4 acc[FM][FN], sums[SUMS ? FM : 1];
        i32x4 fa[2][FM], fb[2][FN];
        bool adds;                           // this wave adds up rows of A (every WN-th row of pieces)
    };
    static constexpr bool WAITS = !AIN || !BIN;              // the transposing reads' own waits
    static constexpr int UNITS = FM * FN, READS = FM + FN;   // matrix instructions and fragments of a step

    // Unit `u` of the two steps behind the hand-over: its load, if it has one.
    __device__ static __forceinline__ void spread(const State& s, int u, uint8_t PG_LDS* a_to, uint8_t PG_LDS* b_to) {
        const int q = u * LPT / (2 * UNITS);
        if ((u + 1) * LPT / (2 * UNITS) > q) {
            if (q < LB) s.b.load(q, b_to, s.wave);
            else s.a.load(q - LB, a_to, s.wave);
        }
    }
    // Fragment r of step H of the K-tile at `a`, `b`, in the order of their use.
    template <int H>
    __device__ static __forceinline__ void read_one(const RA& ra, const RB& rb, Steps& f, const uint8_t PG_LDS* a,
                                                    const uint8_t PG_LDS* b, int r) {
        if (r == 0) f.fa[H][0] = ra.read(a, 0, H);
        else if (r <= FN) f.fb[H][r - 1] = rb.read(b, r - 1, H);
        else f.fa[H][r - FN] = ra.read(a, r - FN, H);
    }
    // Step H, under which the next step's fragments are read from the K-tile at
    // `a`, `b` (MORE).
    template <int H, bool MORE>
    __device__ static __forceinline__ void step_of_two(const State& s, const RA& ra, const RB& rb, Steps& f, const uint8_t PG_LDS* a,
                                                       const uint8_t PG_LDS* b, uint8_t PG_LDS* a_to, uint8_t PG_LDS* b_to, int wn) {
        if constexpr (WAITS) {
            wait_reads<0>();
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            const int i = u / FN, j = u % FN;
            f.acc[i][j] = multiply16<XT>(f.fb[H][j], f.fa[H][i], f.acc[i][j]);
            if constexpr (SUMS) {
                if (f.adds && j == 0 && i % WN == wn) f.sums[i] = multiply16<XT>(ones(), f.fa[H][i], f.sums[i]);
            }
            if constexpr (MORE) {
                // all of them in the first three quarters of the step
                constexpr int SPAN = UNITS * 3 / 4 > 0 ? UNITS * 3 / 4 : 1;
#pragma unroll
                for (int r = 0; r < READS; ++r)
                    if (r * SPAN / READS == u) read_one<1 - H>(ra, rb, f, a, b, r);
                spread(s, (H == 1 ? 0 : UNITS) + u, a_to, b_to);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    __device__ static __forceinline__ void run_steps(const LinearArgs& p, State& s, uint8_t PG_LDS* smem, const RA& ra, const RB& rb,
                                                    int wm, int wn, bool first_columns) {
        Steps f;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) f.acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < (SUMS ? FM : 1); ++i) f.sums[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        f.adds = SUMS && first_columns;
        auto tile_a = [&](int slot) { return smem + slot * FA::BYTES; };
        auto tile_b = [&](int slot) { return smem + RING_A + slot * FB::BYTES; };
        auto first_fragments = [&] {
#pragma unroll
            for (int r = 0; r < READS; ++r) read_one<0>(ra, rb, f, tile_a(0), tile_b(0), r);
        };
        // The first SB - 1 K-tiles, and of the next one what a second step takes.
        static_assert(SA == SB && SB > P && LPT % 2 == 0, "");
#pragma unroll
        for (int t = 0; t < SB; ++t) {
            s.a.start(t, s.deep, s.rot);
            s.b.start(t, s.deep, s.rot);
            if (t + 1 < SB) {
                begin(s, t, tile_a(t), tile_b(t));
            } else {
#pragma unroll
                for (int u = 0; u < UNITS; ++u) spread(s, u, tile_a(t), tile_b(t));
            }
        }
        wait_loads<(SB - 2) * LPT + LPT / 2>();
        barrier();
        clear_tails(s, tile_a, tile_b);
        if (s.nt > 0) {
            first_fragments();
            step_of_two<0, true>(s, ra, rb, f, tile_a(0), tile_b(0), tile_a(SB - 1), tile_b(SB - 1), wn);
            int slot = 0;
            for (int t = 0; t + 1 < s.nt; ++t) {
                const int next = slot + 1 == SB ? 0 : slot + 1;
                s.a.next(s.deep);
                s.b.next(s.deep);
                wait_loads<(SB - 2) * LPT>();            // K-tile t + 1 has landed (this wave's part)
                barrier();                               // ... everyone's, and K-tile t's place is free
                step_of_two<1, true>(s, ra, rb, f, tile_a(next), tile_b(next), tile_a(slot), tile_b(slot), wn);
                step_of_two<0, true>(s, ra, rb, f, tile_a(next), tile_b(next), tile_a(slot), tile_b(slot), wn);
                slot = next;
            }
            step_of_two<1, false>(s, ra, rb, f, nullptr, nullptr, nullptr, nullptr, wn);
        }
        wait_loads<0>();                     // no write into LDS outlives the K loop
        barrier();
        if constexpr (SUMS) {
            if (f.adds)
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    if (i % WN == wn) store_sums(p, s.m0 + wm * WTM + 16 * i, f.sums[i][0]);
        }
        store(p, s, smem, wm, wn, f.acc);
    }

    // ---- 128 x 128 sums per wave, one wave per SIMD -----------------------------------
    //
    // The sums fill half of the register file, and both factors' fragments of a
    // step (32 deep) leave no room for a second set.  So there is one, refilled in
    // the order in which it is used: a step runs four quadrants of 16 pieces, (A
    // 0-3, B 0-3), (A 0-3, B 4-7), (A 4-7, B 0-3), (A 4-7, B 4-7).  It reads its
    // own B 4-7 and A 4-7 under the first, the next step's A 0-3 under the third
    // and its B 0-3 under the fourth.  The second step of a K-tile waits for the
    // next K-tile and crosses the barrier behind the first quadrant, when all of
    // its own reads are done.  (Eight waves of 128 x 64 read 192 KB of fragments a
    // K-tile, these four 128: 8192 x 8192 x 8200 920 and 832 us.)
    struct Frags { i32x4 a[8], b[8]; };

    // The fragments that a K-tile starts with have landed, and their registers
    // are not free before that.
    __device__ static __forceinline__ void settle(const Frags& f) {
        if constexpr (!AIN || !BIN) {
            wait_reads<0>();
#pragma unroll
            for (int j = 0; j < 4; ++j) asm volatile("" ::"v"(f.a[j]), "v"(f.b[j]) : "memory");
        }
    }

    // The loads of `factor`'s next K-tile go out in units [U0, 64) of the step.
    template <int H, bool BAR, bool ADDS, class F>
    __device__ static __forceinline__ void step(State& s, uint8_t PG_LDS* smem, const RA& ra, const RB& rb,
                                                Frags& f, i32x4 (&acc)[8][8], const uint8_t PG_LDS* a, const uint8_t PG_LDS* b,
                                                const uint8_t PG_LDS* na, const uint8_t PG_LDS* nb, F& factor,
                                                uint8_t PG_LDS* to, float (&sums)[ADDS ? 8 : 1]) {
        constexpr int U0 = BAR ? 16 : 0, NL = F::L;
        constexpr int PA = AIN ? 1 : 2, PB = BIN ? 1 : 2;    // LDS reads of a fragment
#pragma unroll
        for (int u = 0; u < 64; ++u) {
            const int q = u / 16, i = u % 16;
            if constexpr (!AIN || !BIN) {
                if (u == 0) wait_reads<0>();
                if (!BAR && u == 16) wait_reads<4 * PA < 15 ? 4 * PA : 15>();
                if (!BAR && u == 32) wait_reads<0>();
            }
            const int m = (q >> 1) * 4 + i / 4, n = (q & 1) * 4 + i % 4;
            multiply16_in_place<XT>(f.b[n], f.a[m], acc[m][n]);
            if constexpr (ADDS)
                if (q & 1) sums[m] = add_pair<XT>(f.a[m], i % 4, sums[m]);
            if (q == 0 && (i & 1) == 0) {
                const int r = i / 2;
                if (r < 4) f.b[4 + r] = rb.read(b, 4 + r, H);
                else f.a[r] = ra.read(a, r, H);
            }
            if (q == 2 && (i & 3) == 0) f.a[i / 4] = ra.read(na, i / 4, 1 - H);
            if (q == 3 && i < 4) f.b[i] = rb.read(nb, i, 1 - H);
            if (u >= U0) {
                const int j = (u - U0) * NL / (64 - U0);     // at most one load a unit
                if ((u - U0 + 1) * NL / (64 - U0) > j) factor.load(j, to, s.wave);
                if (u == 63) factor.next(s.deep);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (BAR && u == 15) {
                wait_loads<FLYING>();
                barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    template <bool ADDS>
    __device__ static __forceinline__ void multiply_quads(State& s, uint8_t PG_LDS* smem, const RA& ra, const RB& rb, Frags& f,
                                                          i32x4 (&acc)[8][8], float (&sums)[ADDS ? 8 : 1]) {
        auto tile_a = [&](int slot) { return smem + slot * FA::BYTES; };
        auto tile_b = [&](int slot) { return smem + RING_A + slot * FB::BYTES; };
        int slot_a = 0, slot_b = 0;
        for (int t = 0; t < s.nt; ++t) {
            const int next_a = slot_a == 2 ? 0 : slot_a + 1, next_b = slot_b ^ 1, prev_a = slot_a == 0 ? 2 : slot_a - 1;
            asm volatile("s_nop 4" ::: "memory");
            step<0, false, ADDS>(s, smem, ra, rb, f, acc, tile_a(slot_a), tile_b(slot_b), tile_a(slot_a), tile_b(slot_b), s.a,
                           tile_a(prev_a), sums);
            step<1, true, ADDS>(s, smem, ra, rb, f, acc, tile_a(slot_a), tile_b(slot_b), tile_a(next_a), tile_b(next_b), s.b,
                          tile_b(slot_b), sums);
            slot_a = next_a;
            slot_b = next_b;
        }
        settle(f);
    }

    template <bool ADDS>
    __device__ static __forceinline__ void run_quads(const LinearArgs& p, State& s, uint8_t PG_LDS* smem, const RA& ra, const RB& rb,
                                                     int wm, int wn) {
        i32x4 acc[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
        auto tile_a = [&](int slot) { return smem + slot * FA::BYTES; };
        auto tile_b = [&](int slot) { return smem + RING_A + slot * FB::BYTES; };
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            s.a.start(t, s.deep, s.rot);
            s.b.start(t, s.deep, s.rot);
            begin(s, t, tile_a(t), tile_b(t));
        }
        wait_loads<LA + LB>();
        barrier();
        clear_tails(s, tile_a, tile_b);
        s.a.start(2, s.deep, s.rot);
        s.b.start(2, s.deep, s.rot);
        Frags f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f.a[i] = ra.read(tile_a(0), i, 0);
            f.b[i] = rb.read(tile_b(0), i, 0);
        }
        settle(f);
        float sums[ADDS ? 8 : 1];
#pragma unroll
        for (int i = 0; i < (ADDS ? 8 : 1); ++i) sums[i] = 0.0f;
        multiply_quads<ADDS>(s, smem, ra, rb, f, acc, sums);
        asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
        wait_loads<0>();
        barrier();
        if constexpr (ADDS) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // lane (r, g) has added chunk g of each step's row r
                float v = sums[i] + __shfl_xor(sums[i], 16);
                v += __shfl_xor(v, 32);
                if (wn == 0) store_sums(p, s.m0 + wm * WTM + 16 * i, v);
            }
        }
        f32x4 c[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) c[i][j] = __builtin_bit_cast(f32x4, acc[i][j]);
        store(p, s, smem, wm, wn, c);
    }

    // A wave's sums go through its own part of LDS, as many rows at a time as fit,
    // and come back as eight neighbouring columns per lane, whole rows of
    // the wave's block at a time, for the ending.  A block that lies inside the
    // matrix takes several passes at a time, without tests, their loads and the next
    // ones' in flight together; any other goes row by row.  Neither loop is
    // unrolled further: code that is run once is waited for (256 x 256 tiles at 4096^3,
    // all of it unrolled: 61000 cycles of a tile's 240000).
    __device__ static __forceinline__ void store(const LinearArgs& p, const State& s, uint8_t PG_LDS* smem, int wm, int wn,
                                                 const f32x4 (&acc)[FM][FN]) {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
        constexpr int LANES = OUTS / 8, ROWS = 64 / LANES;           // lanes of a row, rows of a pass
        constexpr int PASSES = PIECES * 16 / ROWS > 0 ? PIECES * 16 / ROWS : 1;
        // (gated_backward's values of four passes would not fit the registers)
        constexpr int MOST = END == END_GATED_BACKWARD ? 2 : 4, Q = PASSES < MOST ? PASSES : MOST, GROUPS = PASSES / Q;
        static_assert(FM % PIECES == 0 && PASSES % Q == 0, "whole parts");
        uint8_t PG_LDS* part = smem + s.wave * (PIECES * 16 * STRIP_ROW);
        const int row = lane / LANES, c = lane % LANES * 8;
        const int mw = s.m0 + wm * WTM, nw = s.n0 + wn * OUTS;
        const int64_t n = nw + c;
        const bool whole = mw + WTM <= p.M && nw + OUTS <= p.N && ROWS <= PIECES * 16;
        const bool in = n < p.N && row < PIECES * 16;
        Biases<END> bias;
        if (in) bias = fetch_biases<XT, END>(p, n);
        const auto values = [&](int at, float* v, float* u) {
            const uint8_t PG_LDS* from = part + at * STRIP_ROW + (SPLIT ? c / 16 * 32 + c % 16 : c) * 4;
            const f32x4 v0 = *(const f32x4 PG_LDS*)from, v1 = *(const f32x4 PG_LDS*)(from + 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[e] = v0[e]; v[4 + e] = v1[e]; }
            if constexpr (SPLIT) {
                const f32x4 u0 = *(const f32x4 PG_LDS*)(from + 64), u1 = *(const f32x4 PG_LDS*)(from + 80);
#pragma unroll
                for (int e = 0; e < 4; ++e) { u[e] = u0[e]; u[4 + e] = u1[e]; }
            }
        };
#pragma unroll 1
        for (int i0 = 0; i0 < FM; i0 += PIECES) {
            const int64_t m0 = mw + 16 * i0 + row;
            Beside<XT, END> beside[Q], next[Q];
            if (whole) {
#pragma unroll
                for (int q = 0; q < Q; ++q) next[q] = fetch_beside<XT, END, true>(p, m0 + q * ROWS, n);
            }
#pragma unroll
            for (int k = 0; k < FM; k += PIECES)
                if (k == i0)
#pragma unroll
                    for (int i = 0; i < PIECES; ++i)
#pragma unroll
                        for (int j = 0; j < FN; ++j)
                            *(f32x4 PG_LDS*)(part + (16 * i + r) * STRIP_ROW + (16 * j + 4 * g) * 4) = acc[k + i][j];
            if (whole) {
#pragma unroll 1
                for (int k = 0; k < GROUPS; ++k) {
#pragma unroll
                    for (int q = 0; q < Q; ++q) beside[q] = next[q];
                    float v[8 * Q], u[8 * Q];
#pragma unroll
                    for (int q = 0; q < Q; ++q) values(row + (k * Q + q) * ROWS, v + 8 * q, u + 8 * q);
                    if (k + 1 < GROUPS) {
#pragma unroll
                        for (int q = 0; q < Q; ++q) next[q] = fetch_beside<XT, END, true>(p, m0 + ((k + 1) * Q + q) * ROWS, n);
                    }
                    finish<XT, END, true, Q>(p, m0 + k * Q * ROWS, ROWS, n, beside, bias, v, u);
                }
            } else {
#pragma unroll 1
                for (int q = 0; q < PASSES; ++q) {
                    const int64_t m = m0 + q * ROWS;
                    if (!in || m >= p.M) continue;
                    Beside<XT, END> one[1] = {fetch_beside<XT, END, false>(p, m, n)};
                    float v[8], u[8];
                    values(row + q * ROWS, v, u);
                    finish<XT, END, false, 1>(p, m, 0, n, one, bias, v, u);
                }
            }
        }
    }
};

template <int XT, int END, bool AIN, bool BIN, int BM, int BN, int WM, int WN, int SA, int SB, int EXTRA>
__global__ void __launch_bounds__(WM * WN * 64) linear_tile(LinearArgs p) {
    typedef Tile<XT, END, AIN, BIN, BM, BN, WM, WN, SA, SB, EXTRA> S;
    __shared__ __attribute__((aligned(16))) uint8_t smem[S::LDS];
    S::run(p, (uint8_t PG_LDS*)smem);
}

// The classes of one ending.  EXTRA: a second product (linear), sums of A's rows
// (weight gradients).
template <int XT, int END, bool AIN, bool BIN, int EXTRA>
const void* linear_by_tile(int tile) {
    switch (tile) {
    case LINEAR_TILE_256: return (const void*)&linear_tile<XT, END, AIN, BIN, 256, 256, 2, 2, 3, 2, EXTRA>;
    case LINEAR_TILE_128x256: return (const void*)&linear_tile<XT, END, AIN, BIN, 128, 256, 2, 2, 3, 3, EXTRA>;
    case LINEAR_TILE_128: return (const void*)&linear_tile<XT, END, AIN, BIN, 128, 128, 2, 2, 4, 4, EXTRA>;
    case LINEAR_TILE_64: return (const void*)&linear_tile<XT, END, AIN, BIN, 64, 64, 2, 2, 3, 3, EXTRA>;
    default: return nullptr;
    }
}
template <int END, bool AIN, bool BIN, int EXTRA>
const void* linear_by_type(int xt, int tile) {
    return xt == XT_BF16 ? linear_by_tile<XT_BF16, END, AIN, BIN, EXTRA>(tile) : linear_by_tile<XT_F16, END, AIN, BIN, EXTRA>(tile);
}

}  // namespace pg

#endif
