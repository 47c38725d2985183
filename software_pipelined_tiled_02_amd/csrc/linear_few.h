// linear_few.h -- feed-forward products of few tiles: waves that take whole
// K-tiles by themselves.
//
// With one small tile per CU, or less, what counts is how many loads are in
// flight.  Here a wave takes K-tiles of its own, every W-th of them, through a
// ring of its own in LDS: it waits only for its own loads, and there is no barrier
// in the loop.  At the end the waves' sums are added in turn, each thread taking
// eight neighbouring outputs to their ending.
//
// Bound by memory: 1 x 4096 x 4096 from HBM takes 8.3 us by 16 x 16 tiles (4.1
// TB/s; 25.8 by the 64 x 64 tiles of linear_tile.h), a gated layer of one token with
// 4096 inputs and 8192 outputs 26.8 us by 16 x 32 (5.0 TB/s), 64 x 8192 x 8192 32.5 us
// by 64 x 32 (4.2 TB/s; 52 by 64 x 64).
#ifndef PIPEGEMM_LINEAR_FEW_H
#define PIPEGEMM_LINEAR_FEW_H

#include "linear_tile.h"

namespace pg {

template <int XT, int END, bool AIN, bool BIN, int BM, int BN, int W, int SLOTS, int EXTRA>
struct Few {
    static constexpr bool SPLIT = END == END_GATED;
    static constexpr bool SUMS = END == END_WEIGHT && EXTRA != 0;
    static constexpr int P = END == END_LINEAR && EXTRA != 0 ? 2 : 1;
    static constexpr int FM = BM / 16, FN = BN / 16, OUTS = SPLIT ? BN / 2 : BN;
    typedef Factor<AIN, BM, 64, false, P> FA;
    typedef Factor<BIN, BN, 64, SPLIT, P> FB;
    static constexpr int LPT = FA::L + FB::L;
    static constexpr int SLOT = FA::BYTES + FB::BYTES, RING = SLOTS * SLOT;
    static constexpr int PARTS = W * FM * FN * 1024;             // every wave's sums
    static constexpr int LDS = max3(W * RING, PARTS + (SUMS ? W * BM * 4 : 0), 0);
    static_assert(LDS <= kLdsBudget && (!SPLIT || FN % 2 == 0) && SLOTS * LPT < 64, "");
    typedef Reader<AIN, BM, FM> RA;
    typedef Reader<BIN, BN, FN> RB;

    __device__ static __forceinline__ void run(const LinearArgs& p, uint8_t PG_LDS* smem) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        uint8_t PG_LDS* ring = smem + wave * RING;
        // tiles of one column strip are neighbours: they share B
        const unsigned w = by_xcd(blockIdx.x, gridDim.x);
        const int m0 = (int)(w % (unsigned)p.tiles_m) * BM, tn = (int)(w / (unsigned)p.tiles_m), n0 = tn * OUTS;
        const bool apart = p.apart != 0;
        const Depth deep = depth_of(p.K, apart);
        const int nt = P * ((p.K + kDeep - 1) / kDeep), parts = deep.part != 0 ? P : 0;
        // XCD x starts at K-tile 9 x: with every row read at the same k, rows at equal
        // distances would gather the reads on a few channels.
        const int first = deep.whole > 0 ? (int)((blockIdx.x & 7) * 9u % (unsigned)(P * deep.whole)) : 0;
        FA a;
        FB b;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            a.locate(lane, q, p.A[q], m0, p.lda[q], p.M - m0);
            b.locate(lane, q, p.B[q], n0, p.ldb[q], p.N - n0, p.B[1], p.ldb[1]);
        }
        RA ra;
        RB rb;
        ra.locate(0);
        rb.locate(0);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            a.start(wave + i * W, deep, first);
            b.start(wave + i * W, deep, first);
            if (i == 0 && wave < parts && apart) {
                a.carry(ring, lane);
                b.carry(ring + FA::BYTES, lane);
            } else {
                a.load_all(ring + i * SLOT, 0);
                b.load_all(ring + i * SLOT + FA::BYTES, 0);
            }
        }
        f32x4 acc[FM][FN];
        float sums[SUMS ? FM : 1];
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < (SUMS ? FM : 1); ++i) sums[i] = 0.0f;

        int at = 0;
        for (int t = wave; t < nt; t += W) {
            uint8_t PG_LDS* slot = ring + at * SLOT;
            wait_loads<(SLOTS - 1) * LPT>();                     // K-tile t has landed
            if ((AIN || BIN) && t < parts && !apart && deep.part % 8 != 0) {
                if constexpr (AIN) clear_rows<BM, 64>(lane, slot, deep.part);
                if constexpr (BIN) clear_rows<BN, 64>(lane, slot + FA::BYTES, deep.part);
            }
            i32x4 fa[FM][2], fb[FN][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int i = 0; i < FM; ++i) fa[i][h] = ra.read(slot, i, h);
#pragma unroll
                for (int j = 0; j < FN; ++j) fb[j][h] = rb.read(slot + FA::BYTES, j, h);
            }
            wait_reads<0>();                                     // the slot is free
            if constexpr (!AIN || !BIN) {
                // (the transposing reads' registers are not what the compiler may move or use before that)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(fa[i][h])::"memory");
#pragma unroll
                    for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(fb[j][h])::"memory");
                }
            }
            a.start(t + SLOTS * W, deep, first);
            b.start(t + SLOTS * W, deep, first);
            a.load_all(slot, 0);
            b.load_all(slot + FA::BYTES, 0);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < FM; ++i) {
#pragma unroll
                    for (int j = 0; j < FN; ++j) acc[i][j] = multiply16<XT>(fb[j][h], fa[i][h], acc[i][j]);
                    if constexpr (SUMS) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) sums[i] = add_pair<XT>(fa[i][h], e, sums[i]);
                    }
                }
            at = at + 1 == SLOTS ? 0 : at + 1;
        }
        wait_loads<0>();                     // no write into LDS outlives the K loop
        barrier();

        f32x4 PG_LDS* all = (f32x4 PG_LDS*)smem;
        float PG_LDS* all_sums = (float PG_LDS*)(smem + PARTS);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j) all[((wave * FM + i) * FN + j) * 64 + lane] = acc[i][j];
        if constexpr (SUMS) {
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                float v = sums[i] + __shfl_xor(sums[i], 16);
                v += __shfl_xor(v, 32);
                if (lane < 16) all_sums[wave * BM + 16 * i + lane] = v;
            }
        }
        barrier();
        if (SUMS && tn == 0)
            for (int i = threadIdx.x; i < BM; i += 64 * W) {
                float v = all_sums[i];
#pragma unroll
                for (int q = 1; q < W; ++q) v += all_sums[q * BM + i];
                if (m0 + i < p.M) p.sums[m0 + i] = p.accumulate ? p.sums[m0 + i] + v : v;
            }
        // Eight neighbouring outputs at a time: columns 8 h .. + 7 of row r of a piece
        // are lanes (r, 2 h) and (r, 2 h + 1) of it.
        for (int o = threadIdx.x; o < BM * OUTS / 8; o += 64 * W) {
            const int row = o % BM, c = o / BM, r = row % 16, h = c % 2;
            const int64_t m = m0 + row, n = n0 + 8 * c;
            if (m >= p.M || n >= p.N) continue;
            Beside<XT, END> beside[1] = {fetch_beside<XT, END, false>(p, m, n)};
            const Biases<END> bias = fetch_biases<XT, END>(p, n);
            float v[8], u[8];
            const auto sum = [&](int j, float (&f)[8]) {
                f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll
                for (int q = 0; q < W; ++q) {
                    const f32x4 PG_LDS* from = all + ((q * FM + row / 16) * FN + j) * 64 + r + 32 * h;
                    x += from[0];
                    y += from[16];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) { f[e] = x[e]; f[4 + e] = y[e]; }
            };
            sum(SPLIT ? c / 2 * 2 : c / 2, v);
            if constexpr (SPLIT) sum(c / 2 * 2 + 1, u);
            finish<XT, END, false, 1>(p, m, 0, n, beside, bias, v, u);
        }
    }
};

// A bound of 512 threads, for fewer too, keeps a kernel to 256 registers per
// thread: given more, the compiler holds the sums where vector instructions cannot
// read them.
template <int XT, int END, bool AIN, bool BIN, int BM, int BN, int W, int SLOTS, int EXTRA>
__global__ void __launch_bounds__(512) linear_few(LinearArgs p) {
    typedef Few<XT, END, AIN, BIN, BM, BN, W, SLOTS, EXTRA> S;
    __shared__ __attribute__((aligned(16))) uint8_t smem[S::LDS];
    S::run(p, (uint8_t PG_LDS*)smem);
}

// The classes of one ending.
template <int XT, int END, bool AIN, bool BIN, int EXTRA>
const void* few_by_tile(int tile) {
    switch (tile) {
    case LINEAR_TILE_64K4: return (const void*)&linear_few<XT, END, AIN, BIN, 64, 64, 4, 2, EXTRA>;
    case LINEAR_TILE_64x32: return (const void*)&linear_few<XT, END, AIN, BIN, 64, 32, 4, 3, EXTRA>;
    case LINEAR_TILE_32: return (const void*)&linear_few<XT, END, AIN, BIN, 32, 32, 8, 2, EXTRA>;
    case LINEAR_TILE_16x32:
        if constexpr (AIN) return (const void*)&linear_few<XT, END, AIN, BIN, 16, 32, 8, 3, EXTRA>;
        else return nullptr;
    case LINEAR_TILE_16:
        if constexpr (AIN && END != END_GATED) return (const void*)&linear_few<XT, END, AIN, BIN, 16, 16, 8, 4, EXTRA>;
        else return nullptr;
    default: return nullptr;
    }
}
template <int END, bool AIN, bool BIN, int EXTRA>
const void* few_by_type(int xt, int tile) {
    return xt == XT_BF16 ? few_by_tile<XT_BF16, END, AIN, BIN, EXTRA>(tile) : few_by_tile<XT_F16, END, AIN, BIN, EXTRA>(tile);
}

}  // namespace pg

#endif
