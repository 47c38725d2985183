// fp8_waves.hip -- 8-bit products of few tiles: waves that take whole blocks.
//
// With one small tile per CU a staged tile whose waves share each K-tile waits
// at a barrier per K-tile, each wave reads a part of the tile that another
// reads too, and (fp32 outputs) widens it again.  Here a wave takes a block of K
// by itself: it waits only for its own loads, and reads and widens each byte
// once.  Measured at 256 x 4096 x 4096, 64 x 64 tiles, against waves in 2 x 2
// with a barrier per K-tile: 10.2 us against 11.1, fp32 14.9 against 18.8; 64 x
// 8192 x 8192, 64 x 32 tiles: 14.1 against 16.7 (4.9 TB/s: bound by memory).
// What is left in fp32 is the widening: 276 vector instructions to a K-tile's
// 64 matrix instructions.
#include "fp8_gemm.h"

namespace pg {

namespace {

// A workgroup computes a BM x BN tile of C.  Each of its W waves takes every
// W-th block of K of it, each the whole tile, through a ring of SLOTS K-tiles of
// its own; at the end their sums are added in turn.
template <int AT, int BT, bool SBROW, bool EXACT, int BM, int BN, int W, int SLOTS>
struct Waves {
    static constexpr int FM = BM / 16, FN = BN / 16;
    static constexpr int CPR = kBlock / kChunk;                  // 8 chunks of 16 bytes per row
    static constexpr int LA = BM / 8, LB = BN / 8;               // loads of 8 rows each
    static constexpr int LPT = LA + LB + 2;                      // and of the scales
    static constexpr int A_BYTES = BM * kBlock, S_OFF = A_BYTES + BN * kBlock;
    static constexpr int SLOT = S_OFF + 2 * 256, RING = SLOTS * SLOT;
    static constexpr int PARTS = W * FM * FN * 1024;             // every wave's sums
    static constexpr int LDS = max3(W * RING, PARTS + epilogue_lds(W, FN, EXACT ? 4 : 2), 0);
    static_assert(BM == 64 && BN <= 64 && FM == W, "a scale per lane; a wave stores 16 rows");
    static_assert(LDS <= kLdsBudget, "LDS");

    struct State {
        __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
        uint32_t offa[LA], offb[LB], offsa, offsb, sa_blk, sb_blk;
        int kc;                              // first k of the lane's chunks in rows 0-7 of 16; rows 8-15: kc ^ 32
        int K, KB, ragged;
    };

    // K-tiles in the order they are multiplied: a ragged last one first.
    __device__ static __forceinline__ int block_of(const State& s, int t) { return t < s.ragged ? s.KB - 1 : t - s.ragged; }

    struct Issue {
        uint8_t PG_LDS* base;
        uint32_t so, ssa, ssb;               // byte offsets of the K-tile, and of its scales
        uint32_t out[2];                     // the out-of-range bit for chunks past K
    };
    // K-tiles at or past KB move nothing, so that the number of loads in
    // flight is the same at each step.
    template <bool FIRST>
    __device__ static __forceinline__ Issue start(const State& s, uint8_t PG_LDS* slot, int t) {
        const int kb = block_of(s, t);
        Issue x;
        x.base = slot;
        x.so = __builtin_amdgcn_readfirstlane(t < s.KB ? (uint32_t)kb * kBlock : kOutside);
        x.ssa = __builtin_amdgcn_readfirstlane(t < s.KB ? (uint32_t)kb * s.sa_blk : kOutside);
        x.ssb = __builtin_amdgcn_readfirstlane(t < s.KB ? (uint32_t)kb * s.sb_blk : kOutside);
#pragma unroll
        for (int h = 0; h < 2; ++h)                          // (never on top of x.so's)
            x.out[h] = FIRST && t < s.KB && kb * kBlock + (s.kc ^ (32 * h)) >= s.K ? kOutside : 0u;
        return x;
    }
    __device__ static __forceinline__ void load(const State& s, const Issue& x, int q) {
        if (q < LA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s.ra, (void PG_LDS*)(x.base + q * 1024), 16,
                                                     s.offa[q] | x.out[q & 1], x.so, 0, 0);
        else if (q < LA + LB)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rb, (void PG_LDS*)(x.base + A_BYTES + (q - LA) * 1024), 16,
                                                     s.offb[q - LA] | x.out[(q - LA) & 1], x.so, 0, 0);
        else if (q == LA + LB)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rsa, (void PG_LDS*)(x.base + S_OFF), 4, s.offsa, x.ssa, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(s.rsb, (void PG_LDS*)(x.base + S_OFF + 256), 4, s.offsb, x.ssb, 0, 0);
    }

    // K not a multiple of 16: the bytes at and past K of the chunk that holds
    // K - 1 become zero, in both operands (what lies there may be a NaN).
    __device__ static __forceinline__ void clear_tail(const State& s, uint8_t PG_LDS* slot) {
        const int k = s.K % kBlock, c = k / 16, keep = k % 16;
        for (int row = threadIdx.x & 63; row < BM + BN; row += 64) {
            i32x4 PG_LDS* p = (i32x4 PG_LDS*)(slot + (row * CPR + (c ^ swz(CPR, row))) * kChunk);
            i32x4 v = *p;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int left = keep - 4 * w;
                v[w] = left >= 4 ? v[w] : left <= 0 ? 0 : v[w] & (int)((1u << (8 * left)) - 1u);
            }
            *p = v;
        }
    }

    __device__ static __forceinline__ void run(const Fp8Args& a, uint8_t PG_LDS* smem) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
        uint8_t PG_LDS* ring = smem + wave * RING;
        State s;
        s.K = a.K;
        s.KB = (a.K + kBlock - 1) / kBlock;
        s.ragged = a.K % kBlock != 0 ? 1 : 0;
        int m0, n0;
        place_tile<BM, BN>(a, blockIdx.x, m0, n0);
        s.ra = buffer_at(a.A + (int64_t)m0 * a.lda);
        s.rb = buffer_at(a.B + (int64_t)n0 * a.ldb);
        s.rsa = buffer_at(a.SA + (int64_t)m0 * a.sa_row);
        s.rsb = buffer_at(a.SB + (int64_t)(SBROW ? n0 : n0 / kBlock) * a.sb_row);
        s.sa_blk = (uint32_t)(a.sa_blk * 4);
        s.sb_blk = (uint32_t)(a.sb_blk * 4);
        // Load j takes rows 8 j + lane / 8; the swizzle has period 16 in the
        // row, and rows 8-15 have chunk ^ 2 where rows 0-7 have chunk.
        const int c0 = (lane % CPR) ^ swz(CPR, lane / CPR);
        static_assert((swz(CPR, 0) ^ swz(CPR, 8)) == 2 && (swz(CPR, 7) ^ swz(CPR, 15)) == 2, "the swizzle's row bit 3");
        s.kc = c0 * kChunk;
#pragma unroll
        for (int j = 0; j < LA; ++j) {
            const int row = j * 8 + lane / CPR;
            s.offa[j] = (uint32_t)(m0 + row < a.M ? row : 0) * (uint32_t)a.lda + (s.kc ^ (32 * (j & 1)));
        }
#pragma unroll
        for (int j = 0; j < LB; ++j) {
            const int row = j * 8 + lane / CPR;
            s.offb[j] = (uint32_t)(n0 + row < a.N ? row : 0) * (uint32_t)a.ldb + (s.kc ^ (32 * (j & 1)));
        }
        s.offsa = (uint32_t)(m0 + lane < a.M ? lane : 0) * (uint32_t)(a.sa_row * 4);
        s.offsb = SBROW && lane < BN && n0 + lane < a.N ? (uint32_t)lane * (uint32_t)(a.sb_row * 4) : 0u;

        {
            const Issue x = start<true>(s, ring, wave);
#pragma unroll
            for (int q = 0; q < LPT; ++q) load(s, x, q);
        }
#pragma unroll
        for (int i = 1; i < SLOTS; ++i) {
            const Issue x = start<false>(s, ring + i * SLOT, wave + i * W);
#pragma unroll
            for (int q = 0; q < LPT; ++q) load(s, x, q);
        }

        f32x4 acc[FM][FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // (fp8_staged.hip describes the units.)  The K-tile's fragments are
        // all read before its first unit, so that its slot can take the
        // loads of K-tile t + SLOTS W at once; widened ones leave no
        // registers for that, and A's are read as they are needed.
        constexpr int NU = FM * FN, LAG = 3, SUMS = LAG + 1, NA = EXACT ? 2 : FM;
        constexpr int U0 = EXACT ? (FM - 1) * FN : 0;            // the slot's last read lies before this unit
        constexpr int PER = (LPT + NU - U0 - 1) / (NU - U0);
        f32x4 sum[SUMS];
        f32x4 sbv[SBROW ? FN : 1];
        float sa[FM];
#pragma unroll
        for (int q = 0; q < SUMS; ++q) sum[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < (SBROW ? FN : 1); ++j) sbv[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < FM; ++i) sa[i] = 0.0f;
        auto add = [&](int u) {
            const int i = u / FN, j = u % FN;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[i][j][e] = fmaf(sum[u % SUMS][e], SBROW ? sa[i] * sbv[SBROW ? j : 0][e] : sa[i], acc[i][j][e]);
        };
        static_assert(NU % SUMS == 0, "units of the next K-tile start at slot 0");
        const uint32_t rd0 = (uint32_t)(r * CPR + (g ^ swz(CPR, r))) * kChunk;
        const uint32_t rd1 = (uint32_t)(r * CPR + ((4 + g) ^ swz(CPR, r))) * kChunk;
        auto chunk = [&](const uint8_t PG_LDS* rows, uint32_t off) { return *(const i32x4 PG_LDS*)(rows + off); };
        int at = 0;
        for (int t = wave; t < s.KB; t += W) {
            uint8_t PG_LDS* slot = ring + at * SLOT;
            wait_loads<(SLOTS - 1) * LPT>();                     // K-tile t has landed
            if (t == 0 && s.K % 16 != 0) clear_tail(s, slot);
            const float PG_LDS* ps = (const float PG_LDS*)(slot + S_OFF);
            Frag<BT, EXACT> fb[FN];
            Frag<AT, EXACT> fa[NA];
            auto read_a = [&](int i) {
                return fragment<AT, EXACT>(chunk(slot, i * 16 * kBlock + rd0), chunk(slot, i * 16 * kBlock + rd1));
            };
            fa[0] = read_a(0);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                fb[j] = fragment<BT, EXACT>(chunk(slot + A_BYTES, j * 16 * kBlock + rd0),
                                            chunk(slot + A_BYTES, j * 16 * kBlock + rd1));
            float sa_next[FM], sb_next = 0.0f;
            f32x4 sbv_next[SBROW ? FN : 1];
#pragma unroll
            for (int i = 0; i < FM; ++i) sa_next[i] = ps[16 * i + r];
            if constexpr (SBROW) {
#pragma unroll
                for (int j = 0; j < FN; ++j) sbv_next[j] = *(const f32x4 PG_LDS*)(ps + 64 + 16 * j + 4 * g);
            } else {
                sb_next = ps[64];
            }
            if constexpr (!EXACT) {
#pragma unroll
                for (int i = 1; i < FM; ++i) fa[i] = read_a(i);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int u = NU - LAG; u < NU; ++u) add(u);          // the K-tile before's last
#pragma unroll
            for (int i = 0; i < FM; ++i) sa[i] = SBROW ? sa_next[i] : sa_next[i] * sb_next;
            if constexpr (SBROW) {
#pragma unroll
                for (int j = 0; j < FN; ++j) sbv[j] = sbv_next[j];
            }
            const Issue next = start<false>(s, slot, t + SLOTS * W);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const int i = u / FN, j = u % FN;
                if (u == U0) wait_lds();                         // the slot is free
                sum[u % SUMS] = block_sum<AT, BT, EXACT>(fb[j], fa[i % NA]);
                if (u >= LAG) add(u - LAG);
                if (EXACT && j == 0 && i + 1 < FM) fa[(i + 1) % NA] = read_a(i + 1);
                if (u >= U0) {
#pragma unroll
                    for (int q = (u - U0) * PER; q < (u - U0 + 1) * PER && q < LPT; ++q) load(s, next, q);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            at = at + 1 == SLOTS ? 0 : at + 1;
        }
#pragma unroll
        for (int u = NU - LAG; u < NU; ++u) add(u);
        wait_loads<0>();                     // no write into LDS outlives the K loop
        barrier();
        // The waves' sums, in their order; wave w stores rows 16 w .. 16 w + 15.
        f32x4 PG_LDS* parts = (f32x4 PG_LDS*)smem;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) parts[((wave * FM + i) * FN + j) * 64 + lane] = acc[i][j];
        barrier();
        f32x4 c[1][FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            c[0][j] = parts[(wave * FN + j) * 64 + lane];
#pragma unroll
            for (int w = 1; w < W; ++w) c[0][j] += parts[((w * FM + wave) * FN + j) * 64 + lane];
        }
        store_block<EXACT, 1, FN, false>(a, smem + PARTS, wave, m0 + 16 * wave, n0, c);
    }
};

// Twice the threads: 256 registers each, as fp8_staged.hip explains
// (256 x 4096 x 4096: 10.4 us without, 10.0 with).
template <int AT, int BT, bool SBROW, bool EXACT, int BM, int BN, int W, int SLOTS>
__global__ void __launch_bounds__(2 * W * 64) fp8_waves_tile(Fp8Args a) {
    typedef Waves<AT, BT, SBROW, EXACT, BM, BN, W, SLOTS> S;
    __shared__ __attribute__((aligned(16))) uint8_t smem[S::LDS];
    S::run(a, (uint8_t PG_LDS*)smem);
}

template <int AT, int BT, bool SBROW, bool EXACT>
const void* by_tile(int tile) {
    switch (tile) {
    case FP8_TILE_64K4: return (const void*)&fp8_waves_tile<AT, BT, SBROW, EXACT, 64, 64, 4, 2>;
    case FP8_TILE_64x32: return (const void*)&fp8_waves_tile<AT, BT, SBROW, EXACT, 64, 32, 4, 3>;
    default: return nullptr;
    }
}
template <int AT, int BT>
const void* by_mode(int tile, bool sb_rows, bool exact) {
    if (sb_rows) return exact ? by_tile<AT, BT, true, true>(tile) : by_tile<AT, BT, true, false>(tile);
    return exact ? by_tile<AT, BT, false, true>(tile) : by_tile<AT, BT, false, false>(tile);
}

}  // namespace

const void* fp8_waves_kernel(int tile, int a_type, int b_type, bool sb_rows, bool exact) {
    if (a_type == FP8_E4M3)
        return b_type == FP8_E4M3 ? by_mode<FP8_E4M3, FP8_E4M3>(tile, sb_rows, exact)
                                  : by_mode<FP8_E4M3, FP8_E5M2>(tile, sb_rows, exact);
    return b_type == FP8_E4M3 ? by_mode<FP8_E5M2, FP8_E4M3>(tile, sb_rows, exact)
                              : by_mode<FP8_E5M2, FP8_E5M2>(tile, sb_rows, exact);
}

}  // namespace pg
