// fp8_staged.hip -- 8-bit products of many rows: tiles staged through LDS.
//
// A workgroup computes a BM x BN tile of C; a K-tile is one block of 128, so
// each block's scales are applied exactly once per piece of C.  Operands and
// scales go from memory straight into LDS (16 and 4 bytes per lane) into a
// ring of SLOTS, swizzled as tile_layout.h describes; one barrier per K-tile.
#include "fp8_gemm.h"

namespace pg {

namespace {

template <int AT, int BT, bool SBROW, bool EXACT, int BM, int BN, int WM, int WN, int SLOTS, bool LOOP>
struct Staged {
    static constexpr int T = WM * WN * 64;
    static constexpr int WTM = BM / WM, WTN = BN / WN, FM = WTM / 16, FN = WTN / 16;
    static constexpr int CPR = kBlock / kChunk;                  // 8 chunks of 16 bytes per row
    static constexpr int LA = BM * CPR / T, LB = BN * CPR / T;   // chunks per lane and K-tile
    static constexpr int LPT = LA + LB + 1;                      // loads per lane and K-tile, one of them scales
    static constexpr int A_BYTES = BM * kBlock, B_BYTES = BN * kBlock, S_OFF = A_BYTES + B_BYTES;
    static constexpr int SLOT = S_OFF + T * 4;
    // The epilogue's strips take the ring's place, or (LOOP) lie behind it, so
    // that the next tile's first loads can go out before the stores.
    static constexpr int STRIPS = LOOP ? SLOTS * SLOT : 0;
    static constexpr int LDS = max3(SLOTS * SLOT, STRIPS + epilogue_lds(WM * WN, FN, EXACT ? 4 : 2), 0);
    static_assert(T <= 512 && BM + BN <= T && BM % 64 == 0, "a scale per lane, whole waves of A's");
    static_assert(LDS <= kLdsBudget, "LDS");
    static_assert(WTN <= kBlock && kBlock % WTN == 0 && (BN % kBlock == 0 || kBlock % BN == 0),
                  "a wave's columns share a tile scale");

    struct State {
        __amdgpu_buffer_rsrc_t ra, rb, rs;
        uint32_t offa[LA], offb[LB], offs;
        uint32_t s_blk;                      // bytes from one block's scale to the next, of this wave's operand
        int kc;                              // first k of the lane's chunks
        int wave, K, KB, ragged, rot;
        int m0, n0;                          // the tile
    };

    // K-tiles in the order they are multiplied: a ragged last one first, the
    // others from `rot` on.
    __device__ static __forceinline__ int block_of(const State& s, int t) {
        const int nb = s.KB - s.ragged, q = t - s.ragged + s.rot;
        return t < s.ragged ? s.KB - 1 : q >= nb ? q - nb : q;
    }

    // Where the loads of K-tile t go and start.  One at or past KB moves
    // nothing (every offset is out of range: zeros into a slot no later tile
    // reads), so the number of loads in flight is the same at each boundary.
    struct Issue {
        uint8_t PG_LDS* base;
        uint32_t so, ss;                     // byte offsets of the K-tile, and of its scales
        uint32_t out;                        // the out-of-range bit for chunks past K
    };
    template <bool FIRST>
    __device__ static __forceinline__ Issue start(const State& s, uint8_t PG_LDS* smem, int t, int slot) {
        const int kb = block_of(s, t);
        Issue x;
        x.base = smem + slot * SLOT;
        x.so = __builtin_amdgcn_readfirstlane(t < s.KB ? (uint32_t)kb * kBlock : kOutside);
        x.ss = __builtin_amdgcn_readfirstlane(t < s.KB ? (uint32_t)kb * s.s_blk : kOutside);
        x.out = FIRST && t < s.KB && kb * kBlock + s.kc >= s.K ? kOutside : 0u;     // (never on top of x.so's)
        return x;
    }
    // Load q of a K-tile's LPT: chunks of A, chunks of B, then the scales.
    __device__ static __forceinline__ void load(const State& s, const Issue& x, int q) {
        if (q < LA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s.ra, (void PG_LDS*)(x.base + (q * T + 64 * s.wave) * kChunk), 16,
                                                     s.offa[q] | x.out, x.so, 0, 0);
        else if (q < LA + LB)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                s.rb, (void PG_LDS*)(x.base + A_BYTES + ((q - LA) * T + 64 * s.wave) * kChunk), 16,
                s.offb[q - LA] | x.out, x.so, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rs, (void PG_LDS*)(x.base + S_OFF + 256 * s.wave), 4, s.offs,
                                                     x.ss, 0, 0);
    }
    template <bool FIRST>
    __device__ static __forceinline__ void issue(const State& s, uint8_t PG_LDS* smem, int t, int slot) {
        const Issue x = start<FIRST>(s, smem, t, slot);
#pragma unroll
        for (int q = 0; q < LPT; ++q) load(s, x, q);
    }

    // K not a multiple of 16: the bytes at and past K of the chunk that holds
    // K - 1 become zero, in both operands (what lies there may be a NaN).
    __device__ static __forceinline__ void clear_tail(const State& s, uint8_t PG_LDS* smem) {
        const int k = s.K % kBlock, c = k / 16, keep = k % 16;
        const int row = threadIdx.x;         // one row per lane: A's, then B's
        if (row >= BM + BN) return;
        i32x4 PG_LDS* p = (i32x4 PG_LDS*)(smem + (row * CPR + (c ^ swz(CPR, row))) * kChunk);
        i32x4 v = *p;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int left = keep - 4 * w;
            v[w] = left >= 4 ? v[w] : left <= 0 ? 0 : v[w] & (int)((1u << (8 * left)) - 1u);
        }
        *p = v;
    }

    __device__ static __forceinline__ i32x4 chunk(const uint8_t PG_LDS* rows, uint32_t off) {
        return *(const i32x4 PG_LDS*)(rows + off);
    }

    // Tile number `tile`: where it is, and where a lane's loads start.
    __device__ static __forceinline__ void locate(const Fp8Args& a, State& s, int tile) {
        const int tid = threadIdx.x, ntiles = a.tiles_m * a.tiles_n;
        int m0, n0;
        place_tile<BM, BN>(a, tile, m0, n0);
        s.m0 = m0;
        s.n0 = n0;
        // With more tiles than one round, XCD x starts at K-tile 9 x: read at
        // one k by every XCD, rows at equal distances gather on a few memory
        // channels (8192 x 8192 x 8200: 545 us without, 517 with; one round,
        // whose operands the caches hold, gains nothing).
        const int nb = s.KB - s.ragged;
        s.rot = ntiles > 256 && nb > 0 ? (int)((tile & 7) * 9u % (unsigned)nb) : 0;
        s.ra = buffer_at(a.A + (int64_t)m0 * a.lda);
        s.rb = buffer_at(a.B + (int64_t)n0 * a.ldb);
        // Chunk p = j T + tid of a tile lies in row p / 8; the swizzle has
        // period 16 in the row, so a lane's k is the same for each j.
        const int c = (tid % CPR) ^ swz(CPR, tid / CPR);
        s.kc = c * kChunk;
#pragma unroll
        for (int j = 0; j < LA; ++j) {
            const int row = (j * T + tid) / CPR;
            s.offa[j] = (uint32_t)(m0 + row < a.M ? row : 0) * (uint32_t)a.lda + c * kChunk;
        }
#pragma unroll
        for (int j = 0; j < LB; ++j) {
            const int row = (j * T + tid) / CPR;
            s.offb[j] = (uint32_t)(n0 + row < a.N ? row : 0) * (uint32_t)a.ldb + c * kChunk;
        }
        // Scales: lane i < BM takes row i of A, lane BM + j column j (lanes
        // past them column 0's again, so that every wave issues one load).
        if (s.wave < BM / 64) {
            s.rs = buffer_at(a.SA + (int64_t)m0 * a.sa_row);
            s.offs = (uint32_t)(m0 + tid < a.M ? tid : 0) * (uint32_t)(a.sa_row * 4);
            s.s_blk = (uint32_t)(a.sa_blk * 4);
        } else {
            const int col = tid - BM, n = col < BN && n0 + col < a.N ? col : 0;
            s.rs = buffer_at(a.SB + (int64_t)(SBROW ? n0 : n0 / kBlock) * a.sb_row);
            s.offs = (uint32_t)(SBROW ? n : n / kBlock) * (uint32_t)(a.sb_row * 4);
            s.s_blk = (uint32_t)(a.sb_blk * 4);
        }
    }

    // The first SLOTS - 1 K-tiles' loads.
    __device__ static __forceinline__ void fill(const State& s, uint8_t PG_LDS* smem) {
        issue<true>(s, smem, 0, 0);
#pragma unroll
        for (int t = 1; t < SLOTS - 1; ++t) issue<false>(s, smem, t, t);
    }

    __device__ static __forceinline__ void run(const Fp8Args& a, uint8_t PG_LDS* smem) {
        State s;
        s.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        s.K = a.K;
        s.KB = (a.K + kBlock - 1) / kBlock;
        s.ragged = a.K % kBlock != 0 ? 1 : 0;
        const int wm = s.wave / WN, wn = s.wave % WN;
        f32x4 acc[FM][FN];
        int tile = blockIdx.x;
        locate(a, s, tile);
        fill(s, smem);
        while (true) {
            multiply(a, s, smem, acc);
            // (no write into LDS is left in flight, and every wave is here)
            const int m0 = s.m0 + wm * WTM, n0 = s.n0 + wn * WTN;
            tile += gridDim.x;
            const bool more = LOOP && tile < a.tiles_m * a.tiles_n;
            if (more) {
                locate(a, s, tile);
                fill(s, smem);
            }
            store_block<EXACT, FM, FN, (BM * BN >= 128 * 128)>(a, smem + STRIPS, s.wave, m0, n0, acc);
            if (!more) return;
        }
    }

    // One tile's K loop, its first loads under way.
    __device__ static __forceinline__ void multiply(const Fp8Args& a, const State& s, uint8_t PG_LDS* smem,
                                                    f32x4 (&acc)[FM][FN]) {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
        const int wm = s.wave / WN, wn = s.wave % WN;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        // LDS offsets of the lane's two chunks of a 16-row fragment at row 0
        // of a tile (fragments start at multiples of 16, the swizzle's period)
        const uint32_t rd0 = (uint32_t)(r * CPR + (g ^ swz(CPR, r))) * kChunk;
        const uint32_t rd1 = (uint32_t)(r * CPR + ((4 + g) ^ swz(CPR, r))) * kChunk;

        wait_loads<(SLOTS - 2) * LPT>();
        barrier();
        if (a.K % 16 != 0) {
            clear_tail(s, smem);
            barrier();
        }
        // The K loop, one unit per 16x16 piece of the wave's block.  A unit
        // issues its matrix instruction, then adds the sum that the unit LAG
        // before it left (so the instruction's latency passes under the
        // others'), then its share of the next fragment's LDS reads and of
        // the next K-tile's loads; a fence keeps that order.  The last LAG
        // sums of a K-tile are added under the next one's first reads.
        constexpr int NU = FM * FN, LAG = NU > 3 ? 3 : 1, RING = LAG + 1;
        constexpr int PER = (LPT + NU - 1) / NU;         // loads per unit, from the first on
        f32x4 sum[RING];                     // sums not added yet: unit u's in u % RING
        f32x4 sbv[SBROW ? FN : 1];
        float sa[FM];
#pragma unroll
        for (int q = 0; q < RING; ++q) sum[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < (SBROW ? FN : 1); ++j) sbv[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] = 0.0f;
        auto add = [&](int u) {
            const int i = u / FN, j = u % FN;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][j][e] = fmaf(sum[u % RING][e], SBROW ? sa[i] * sbv[SBROW ? j : 0][e] : sa[i], acc[i][j][e]);
        };
        static_assert(NU % RING == 0, "units of the next K-tile start at ring slot 0");
        int slot = 0;
        for (int t = 0; t < s.KB; ++t) {
            const int free_slot = slot == 0 ? SLOTS - 1 : slot - 1;
            const Issue next = start<false>(s, smem, t + SLOTS - 1, free_slot);
            const uint8_t PG_LDS* ta = smem + slot * SLOT + wm * WTM * kBlock;
            const uint8_t PG_LDS* tb = smem + slot * SLOT + A_BYTES + wn * WTN * kBlock;
            const float PG_LDS* psa = (const float PG_LDS*)(smem + slot * SLOT + S_OFF) + wm * WTM;
            const float PG_LDS* psb = (const float PG_LDS*)(smem + slot * SLOT + S_OFF) + BM + wn * WTN;
            Frag<BT, EXACT> fb[FN];
            Frag<AT, EXACT> fa[2];
            auto read_a = [&](int i) {
                return fragment<AT, EXACT>(chunk(ta, i * 16 * kBlock + rd0), chunk(ta, i * 16 * kBlock + rd1));
            };
            fa[0] = read_a(0);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[j] = fragment<BT, EXACT>(chunk(tb, j * 16 * kBlock + rd0), chunk(tb, j * 16 * kBlock + rd1));
            float sa_next[FM], sb_next = 0.0f;
            f32x4 sbv_next[SBROW ? FN : 1];
#pragma unroll
            for (int i = 0; i < FM; ++i) sa_next[i] = psa[16 * i + r];
            if constexpr (SBROW) {
#pragma unroll
                for (int j = 0; j < FN; ++j) sbv_next[j] = *(const f32x4 PG_LDS*)(psb + 16 * j + 4 * g);
            } else {
                sb_next = psb[0];
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = NU - LAG; u < NU; ++u) add(u);      // the K-tile before's last
#pragma unroll
            for (int i = 0; i < FM; ++i) sa[i] = SBROW ? sa_next[i] : sa_next[i] * sb_next;
            if constexpr (SBROW) {
#pragma unroll
                for (int j = 0; j < FN; ++j) sbv[j] = sbv_next[j];
            }
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int i = u / FN, j = u % FN;
                sum[u % RING] = block_sum<AT, BT, EXACT>(fb[j], fa[i & 1]);
                if (u >= LAG) add(u - LAG);
                if (j == 0 && i + 1 < FM) fa[(i + 1) & 1] = read_a(i + 1);
#pragma unroll
                for (int q = u * PER; q < (u + 1) * PER && q < LPT; ++q) load(s, next, q);
                __builtin_amdgcn_sched_barrier(0);
            }
            wait_loads<(SLOTS - 2) * LPT>();   // K-tile t + 1 has landed (this wave's part)
            barrier();                         // ... everyone's, and slot t is free
            slot = slot + 1 == SLOTS ? 0 : slot + 1;
        }
#pragma unroll
        for (int u = NU - LAG; u < NU; ++u) add(u);
        wait_loads<0>();                       // no write into LDS outlives the K loop
        barrier();
    }
};

// A bound of 512 threads, for tiles of fewer too, keeps a kernel to 256
// registers per thread: given more, the compiler leaves the matrix
// instructions' sums in those that vector instructions cannot read, a copy
// for each multiply-add (64 x 64 tiles, 256 x 4096 x 4096: 11.6 us, 11.1 so).
template <int AT, int BT, bool SBROW, bool EXACT, int BM, int BN, int WM, int WN, int SLOTS, bool LOOP>
__global__ void __launch_bounds__(512) fp8_staged_tile(Fp8Args a) {
    typedef Staged<AT, BT, SBROW, EXACT, BM, BN, WM, WN, SLOTS, LOOP> S;
    __shared__ __attribute__((aligned(16))) uint8_t smem[S::LDS];
    S::run(a, (uint8_t PG_LDS*)smem);
}

// Waves and slots of each tile class.  More slots than two hide the memory's
// latency where a K-tile is multiplied in less time than it takes to arrive.
// The 256x256 tile's workgroups stay and take tile after tile.
template <int AT, int BT, bool SBROW, bool EXACT>
const void* by_tile(int tile) {
    switch (tile) {
    case FP8_TILE_256:
        if constexpr (EXACT) return nullptr;     // the widened fragments leave no registers for 128 accumulators
        else return (const void*)&fp8_staged_tile<AT, BT, SBROW, EXACT, 256, 256, 2, 4, 2, true>;
    case FP8_TILE_256x128: return (const void*)&fp8_staged_tile<AT, BT, SBROW, EXACT, 256, 128, 4, 2, 3, false>;
    case FP8_TILE_128: return (const void*)&fp8_staged_tile<AT, BT, SBROW, EXACT, 128, 128, 2, 4, 4, false>;
    case FP8_TILE_64: return (const void*)&fp8_staged_tile<AT, BT, SBROW, EXACT, 64, 64, 2, 2, 4, false>;
    default: return nullptr;
    }
}
template <int AT, int BT>
const void* by_mode(int tile, bool sb_rows, bool exact) {
    if (sb_rows) return exact ? by_tile<AT, BT, true, true>(tile) : by_tile<AT, BT, true, false>(tile);
    return exact ? by_tile<AT, BT, false, true>(tile) : by_tile<AT, BT, false, false>(tile);
}

}  // namespace

const void* fp8_staged_kernel(int tile, int a_type, int b_type, bool sb_rows, bool exact) {
    if (a_type == FP8_E4M3)
        return b_type == FP8_E4M3 ? by_mode<FP8_E4M3, FP8_E4M3>(tile, sb_rows, exact)
                                  : by_mode<FP8_E4M3, FP8_E5M2>(tile, sb_rows, exact);
    return b_type == FP8_E4M3 ? by_mode<FP8_E5M2, FP8_E4M3>(tile, sb_rows, exact)
                              : by_mode<FP8_E5M2, FP8_E5M2>(tile, sb_rows, exact);
}

}  // namespace pg
