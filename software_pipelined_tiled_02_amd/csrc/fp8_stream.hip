// fp8_stream.hip -- 8-bit products of few rows, and of rows at any address:
// operands go from memory straight into registers.
//
// With few rows of A the product is bound by reading B once, so what counts
// is how many loads are in flight and that no CU idles: a workgroup takes a
// small piece of C, its waves share K (wave w takes blocks w, w + WK, ...,
// so together they read WK x 128 consecutive bytes of each row), and their
// partial sums are added through LDS in wave order, by all waves at once.
// Nothing needs a workspace, and the sum's order is fixed.
#include "fp8_gemm.h"

namespace pg {

namespace {

template <int AT, int BT, bool SBROW, bool EXACT, bool BYTES, int MB, int NB, int WK>
struct Stream {
    static constexpr int BM = 16 * MB, BN = 16 * NB, T = 64 * WK;

    // What a wave holds of one block: operands, and their scales.
    struct Block {
        i32x4 a[MB][2], b[NB][2];
        float sa[MB], sb[SBROW ? NB : 1][SBROW ? 4 : 1];
    };

    struct State {
        __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
        uint32_t offa[MB], offb[NB];       // byte offset of the lane's first chunk at block 0
        uint32_t offsa[MB], offsb[SBROW ? NB : 1][SBROW ? 4 : 1];
        uint32_t sa_blk, sb_blk;           // bytes from one block's scale to the next
        int K, KB, kc;                     // kc: first k of the lane's first chunk
        int rot;                           // the block that is multiplied first
    };

    // 16 bytes of a row from k on, of which only those before K are read:
    // a partial chunk in pieces of 8, 4, 2 and 1 bytes by the binary digits of
    // its length, each at its own place; the rest is zero.
    __device__ static __forceinline__ i32x4 chunk_before(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff, int rem) {
        const uint32_t vb = rem > 0 && rem < 16 ? (uint32_t)rem : 0u;
        i32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, rem >= 16 ? off : kOutside, soff, 0);
        const i32x2 p8 = __builtin_amdgcn_raw_buffer_load_b64(r, (vb & 8) ? off : kOutside, soff, 0);
        const int p4 = (int)__builtin_amdgcn_raw_buffer_load_b32(r, (vb & 4) ? off + (vb & 8) : kOutside, soff, 0);
        uint32_t t = __builtin_amdgcn_raw_buffer_load_b16(r, (vb & 2) ? off + (vb & 12) : kOutside, soff, 0);
        t |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r, (vb & 1) ? off + (vb & 14) : kOutside, soff, 0) << (8 * (vb & 2));
        const uint32_t d4 = (vb & 8) >> 2, dt = (vb & 12) >> 2;
        v[0] |= p8[0] | (d4 == 0 ? p4 : 0) | (dt == 0 ? (int)t : 0);
        v[1] |= p8[1] | (dt == 1 ? (int)t : 0);
        v[2] |= (d4 == 2 ? p4 : 0) | (dt == 2 ? (int)t : 0);
        v[3] |= (dt == 3 ? (int)t : 0);
        return v;
    }

    // The k-th block in the order they are multiplied; one at or past KB gives
    // zeros, scales too.
    __device__ static __forceinline__ void load(const State& s, Block& x, int k) {
        const int kb = k >= s.KB ? k : k + s.rot >= s.KB ? k + s.rot - s.KB : k + s.rot;
        const uint32_t soff = __builtin_amdgcn_readfirstlane((uint32_t)kb * kBlock);
        const int rem = s.K - (kb * kBlock + s.kc);        // bytes of the row from the lane's first chunk on
        if (BYTES && kb == s.KB - 1) {
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) x.a[i][h] = chunk_before(s.ra, s.offa[i] + 64 * h, soff, rem - 64 * h);
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) x.b[j][h] = chunk_before(s.rb, s.offb[j] + 64 * h, soff, rem - 64 * h);
        } else {
            // offsets are below 2^31, so the bit puts them out of range
            const uint32_t out0 = rem > 0 ? 0u : kOutside, out1 = rem > 64 ? 0u : kOutside;
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                x.b[j][0] = __builtin_amdgcn_raw_buffer_load_b128(s.rb, s.offb[j] | out0, soff, 0);
                x.b[j][1] = __builtin_amdgcn_raw_buffer_load_b128(s.rb, (s.offb[j] + 64) | out1, soff, 0);
            }
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                x.a[i][0] = __builtin_amdgcn_raw_buffer_load_b128(s.ra, s.offa[i] | out0, soff, 0);
                x.a[i][1] = __builtin_amdgcn_raw_buffer_load_b128(s.ra, (s.offa[i] + 64) | out1, soff, 0);
            }
        }
        const uint32_t past = kb < s.KB ? 0u : kOutside;
        const uint32_t ka = __builtin_amdgcn_readfirstlane(kb < s.KB ? (uint32_t)kb * s.sa_blk : 0u);
        const uint32_t kbb = __builtin_amdgcn_readfirstlane(kb < s.KB ? (uint32_t)kb * s.sb_blk : 0u);
#pragma unroll
        for (int i = 0; i < MB; ++i)
            x.sa[i] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(s.rsa, s.offsa[i] | past, ka, 0));
        constexpr int NS = SBROW ? NB : 1, NE = SBROW ? 4 : 1;
#pragma unroll
        for (int j = 0; j < NS; ++j)
#pragma unroll
            for (int e = 0; e < NE; ++e)
                x.sb[j][e] = __int_as_float(__builtin_amdgcn_raw_buffer_load_b32(s.rsb, s.offsb[j][e] | past, kbb, 0));
    }

    __device__ static __forceinline__ void add(const Block& x, f32x4 (&acc)[MB][NB]) {
        Frag<BT, EXACT> fb[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) fb[j] = fragment<BT, EXACT>(x.b[j][0], x.b[j][1]);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const Frag<AT, EXACT> fa = fragment<AT, EXACT>(x.a[i][0], x.a[i][1]);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                const f32x4 t = block_sum<AT, BT, EXACT>(fb[j], fa);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][j][e] = fmaf(t[e], x.sa[i] * x.sb[SBROW ? j : 0][SBROW ? e : 0], acc[i][j][e]);
            }
        }
    }

    __device__ static __forceinline__ void run(const Fp8Args& a, f32x4 PG_LDS* sums) {
        const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int r = lane & 15, g = lane >> 4;
        // tiles of one column strip are neighbours: they share B
        const unsigned w = by_xcd(blockIdx.x, gridDim.x);
        const int m0 = (int)(w % (unsigned)a.tiles_m) * BM, n0 = (int)(w / (unsigned)a.tiles_m) * BN;

        State s;
        s.K = a.K;
        s.KB = (a.K + kBlock - 1) / kBlock;
        s.kc = 16 * g;
        // XCD x starts at block 9 x: with every row read at the same k, the
        // rows' equal distances would gather the reads on a few channels.
        s.rot = s.KB > 0 ? (int)((blockIdx.x & 7) * 9u % (unsigned)s.KB) : 0;
        s.ra = buffer_at(a.A + (int64_t)m0 * a.lda);
        s.rb = buffer_at(a.B + (int64_t)n0 * a.ldb);
        s.rsa = buffer_at(a.SA + (int64_t)m0 * a.sa_row);
        s.rsb = buffer_at(a.SB + (int64_t)(SBROW ? n0 : n0 / kBlock) * a.sb_row);
        s.sa_blk = (uint32_t)(a.sa_blk * 4);
        s.sb_blk = (uint32_t)(a.sb_blk * 4);
        // Rows past M (columns past N) read row 0 of the tile: they only feed
        // outputs that are not stored.
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            const int row = m0 + 16 * i + r < a.M ? 16 * i + r : 0;
            s.offa[i] = (uint32_t)row * (uint32_t)a.lda + 16 * g;
            s.offsa[i] = (uint32_t)row * (uint32_t)(a.sa_row * 4);
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int row = n0 + 16 * j + r < a.N ? 16 * j + r : 0;
            s.offb[j] = (uint32_t)row * (uint32_t)a.ldb + 16 * g;
            if constexpr (SBROW) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int col = 16 * j + 4 * g + e;
                    s.offsb[j][e] = (uint32_t)(n0 + col < a.N ? col : 0) * (uint32_t)(a.sb_row * 4);
                }
            }
        }
        if constexpr (!SBROW) s.offsb[0][0] = 0;    // BN divides 128: one scale for the whole strip

        f32x4 acc[MB][NB];
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        if constexpr (BYTES) {
            Block x;
            for (int k = wave; k < s.KB; k += WK) {
                load(s, x, k);
                add(x, acc);
            }
        } else {
            // Two blocks in flight: the next one's loads are issued before the
            // current one is multiplied (the fences keep the compiler from
            // moving them next to their use).  Three and four were slower: the
            // registers they take cost waves (1x1024x8192: 7.5, 8.2, 8.6 us).
            Block x[2];
            load(s, x[0], wave);
            for (int k = wave; k < s.KB;) {
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                    if (d > 0 && k >= s.KB) break;
                    load(s, x[d ^ 1], k + WK);
                    __builtin_amdgcn_sched_barrier(0);
                    add(x[d], acc);
                    __builtin_amdgcn_sched_barrier(0);
                    k += WK;
                }
            }
        }

        // Partial sums to LDS, [wave][piece][lane]; then each thread adds
        // four neighbouring outputs over the waves, in wave order.
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int j = 0; j < NB; ++j) sums[(wave * MB * NB + i * NB + j) * 64 + lane] = acc[i][j];
        __syncthreads();
        for (int q = threadIdx.x; q < MB * NB * 64; q += T) {
            f32x4 v = sums[q];
#pragma unroll
            for (int p = 1; p < WK; ++p) v += sums[p * MB * NB * 64 + q];
            const int piece = q >> 6, ql = q & 63;
            const int64_t m = m0 + 16 * (piece / NB) + (ql & 15), c = n0 + 16 * (piece % NB) + 4 * (ql >> 4);
            if (m < a.M && c < a.N) store_c<EXACT>(a, m, c, v);
        }
    }
};

template <int AT, int BT, bool SBROW, bool EXACT, bool BYTES, int MB, int NB, int WK>
__global__ void __launch_bounds__(64 * WK) fp8_stream(Fp8Args a) {
    __shared__ __attribute__((aligned(16))) f32x4 sums[WK * MB * NB * 64];
    Stream<AT, BT, SBROW, EXACT, BYTES, MB, NB, WK>::run(a, (f32x4 PG_LDS*)sums);
}

template <int AT, int BT, bool SBROW, bool EXACT, bool BYTES>
const void* by_tile(int tile) {
    switch (tile) {
    case FP8_TILE_32: return (const void*)&fp8_stream<AT, BT, SBROW, EXACT, BYTES, 2, 2, 8>;
    case FP8_TILE_16x32: return (const void*)&fp8_stream<AT, BT, SBROW, EXACT, BYTES, 1, 2, 8>;
    case FP8_TILE_16: return (const void*)&fp8_stream<AT, BT, SBROW, EXACT, BYTES, 1, 1, 16>;
    default: return nullptr;
    }
}
template <int AT, int BT, bool SBROW, bool EXACT>
const void* by_bytes(int tile, bool bytes) {
    return bytes ? by_tile<AT, BT, SBROW, EXACT, true>(tile) : by_tile<AT, BT, SBROW, EXACT, false>(tile);
}
template <int AT, int BT>
const void* by_mode(int tile, bool sb_rows, bool exact, bool bytes) {
    if (sb_rows) return exact ? by_bytes<AT, BT, true, true>(tile, bytes) : by_bytes<AT, BT, true, false>(tile, bytes);
    return exact ? by_bytes<AT, BT, false, true>(tile, bytes) : by_bytes<AT, BT, false, false>(tile, bytes);
}

}  // namespace

const void* fp8_stream_kernel(int tile, int a_type, int b_type, bool sb_rows, bool exact, bool bytes) {
    if (a_type == FP8_E4M3)
        return b_type == FP8_E4M3 ? by_mode<FP8_E4M3, FP8_E4M3>(tile, sb_rows, exact, bytes)
                                  : by_mode<FP8_E4M3, FP8_E5M2>(tile, sb_rows, exact, bytes);
    return b_type == FP8_E4M3 ? by_mode<FP8_E5M2, FP8_E4M3>(tile, sb_rows, exact, bytes)
                              : by_mode<FP8_E5M2, FP8_E5M2>(tile, sb_rows, exact, bytes);
}

}  // namespace pg
