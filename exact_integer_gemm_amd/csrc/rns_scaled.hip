// The block-scaled 8-bit product on gfx950: Y = sum over 128-wide blocks of
// the contraction of sa sb (va . vb).
//
// Which matrix instructions carry the inner products goes by the output's
// type.  The 8-bit instructions align the products they add (64 or 128 of
// them) to the largest and keep about 14 bits below it; their running sum is
// binary32.  Measured on normal deviates that fill e4m3's range, the result is
// off by 1.5e-5 of its norm (values spread over 2^14: 5.8e-5) at any length of
// the contraction: nothing beside a bfloat16's 1.7e-3 or a binary16's 2.1e-4,
// so outputs of 16 bits take them.  A binary32 output takes the bfloat16
// instructions instead, at half the rate: every 8-bit value is a bfloat16, and
// their sums are off by 4e-8 on the same operands.
#include <type_traits>

#include "rns_scaled_device.h"

namespace rns {

struct MmArgs {
    const uint8_t *a, *b;
    const void *as, *bs;
    int64_t lda, ldb;
    int64_t as_row, as_blk, bs_row, bs_blk;
    int32_t a_shift, b_shift;       // log2 of the rows that share a scale: 0 or 7
    void *y;
    int64_t ldy;
    int32_t M, N, K;
    int32_t tiles_m, tiles_n;
    int32_t y_type;
    int32_t e8m0;                   // both scale arrays: 8-bit exponents, or binary32
    int32_t split;                  // parts along K
    float *partial;                 // [split][M][partial_ld]
    int64_t partial_ld;
};

// Four consecutive columns n .. n + 3 of row m.
__device__ __forceinline__ void store4(const MmArgs &g, int m, int n, const float (&v)[4]) {
    const int64_t at = (int64_t)m * g.ldy + n;
    if (g.y_type == RNS_T_F32) {
        float *y = (float *)g.y + at;
        if (n + 4 <= g.N && ((uintptr_t)y & 15) == 0) *(v4f *)y = v4f{v[0], v[1], v[2], v[3]};
        else
            for (int e = 0; e < 4; e++)
                if (n + e < g.N) y[e] = v[e];
        return;
    }
    uint32_t h[4];
#pragma unroll
    for (int e = 0; e < 4; e++) h[e] = g.y_type == RNS_T_BF16 ? bf16_bits(v[e]) : f16_bits(v[e]);
    uint16_t *y = (uint16_t *)g.y + at;
    if (n + 4 <= g.N && ((uintptr_t)y & 7) == 0) *(v2u *)y = v2u{h[0] | h[1] << 16, h[2] | h[3] << 16};
    else
        for (int e = 0; e < 4; e++)
            if (n + e < g.N) y[e] = (uint16_t)h[e];
}

// ---- any alignment ----------------------------------------------------------------
// 64 x 64 tiles, four waves of 32 x 32, one 128-wide block of the contraction
// per step through LDS.  The matrix instruction takes b as its first operand,
// so a lane's sixteen sums belong to one row m of Y (lane % 32) and to columns
// 8 q + 4 (lane / 32) + e: four at a time are neighbours in memory.
constexpr int kPitch = 128 + 16;    // LDS bytes between rows: a fragment read's 32 rows start in different banks

template <int ST, int AT, bool WIDE>
__global__ __launch_bounds__(256) void mm_general_kernel(MmArgs g) {
    __shared__ alignas(16) uint8_t lds[2][64 * kPitch];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int half = lane >> 5, l32 = lane & 31, wm = wave & 1, wn = wave >> 1;
    const int tm = blockIdx.x / g.tiles_n, tn = blockIdx.x - tm * g.tiles_n;
    const int m0 = tm * 64, n0 = tn * 64;
    const bool vec = (((uintptr_t)g.a | (uintptr_t)g.b | (uintptr_t)g.lda | (uintptr_t)g.ldb) & 15) == 0;

    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; i++) acc[i] = 0.f;
    const int lr = tid >> 2, lc = (tid & 3) * 32;           // this thread's row and bytes of a step
    const int m = m0 + wm * 32 + l32;
    for (int k0 = 0, kb = 0; k0 < g.K; k0 += 128, kb++) {
#pragma unroll
        for (int op = 0; op < 2; op++) {
            const int row = (op ? n0 : m0) + lr;
            const bool in = row < (op ? g.N : g.M);
            const uint8_t *src = (op ? g.b + row * g.ldb : g.a + row * g.lda) + k0 + lc;
            uint32_t w[8];
            if (in && vec && k0 + lc + 32 <= g.K) {
                const v4u x = *(const v4u *)src, y = *(const v4u *)(src + 16);
#pragma unroll
                for (int i = 0; i < 4; i++) w[i] = x[i], w[4 + i] = y[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    w[i] = 0;
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (in && k0 + lc + 4 * i + e < g.K) w[i] |= (uint32_t)src[4 * i + e] << (8 * e);
                }
            }
            uint8_t *dst = lds[op] + lr * kPitch + lc;
            *(v4u *)dst = v4u{w[0], w[1], w[2], w[3]};
            *(v4u *)(dst + 16) = v4u{w[4], w[5], w[6], w[7]};
        }
        __syncthreads();
        v16f p{};
#pragma unroll
        for (int kk = 0; kk < 2; kk++) {
            // which entries meet in an instruction is a permutation of the step that both operands share
            const uint8_t *ra = lds[0] + (wm * 32 + l32) * kPitch + kk * 64 + half * 32;
            const uint8_t *rb = lds[1] + (wn * 32 + l32) * kPitch + kk * 64 + half * 32;
            v8i af, bf;
            *(v4i *)&af = *(const v4i *)ra;
            *((v4i *)&af + 1) = *(const v4i *)(ra + 16);
            *(v4i *)&bf = *(const v4i *)rb;
            *((v4i *)&bf + 1) = *(const v4i *)(rb + 16);
            if constexpr (WIDE) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen8<RNS_T_E4M3>(bf[2 * i], bf[2 * i + 1]),
                                                                widen8<AT>(af[2 * i], af[2 * i + 1]), p, 0, 0, 0);
            } else {
                p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bf, af, p, 0, AT == RNS_T_E5M2, 0, 0, 0, 0);
            }
        }
        const float sa = scale_factor<ST>(
            load_scale<ST>(g.as, (int64_t)(min(m, g.M - 1) >> g.a_shift) * g.as_row + kb * g.as_blk));
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int n = min(n0 + wn * 32 + 8 * (i >> 2) + 4 * half + (i & 3), g.N - 1);
            const float sb =
                scale_factor<ST>(load_scale<ST>(g.bs, (int64_t)(n >> g.b_shift) * g.bs_row + kb * g.bs_blk));
            acc[i] += scaled(p[i], sa, sb);
        }
        __syncthreads();
    }
    if (m < g.M)
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const int n = n0 + wn * 32 + 8 * q + 4 * half;
            const float v[4] = {acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
            if (n < g.N) store4(g, m, n, v);
        }
}

// ---- the contraction's end ----------------------------------------------------------
// Sixteen bytes of a row from byte k on; those at or past K are cleared.
__device__ __forceinline__ v4u clear_tail(v4u w, int k, int K) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int left = K - (k + 4 * i);
        if (left < 4) w[i] = left <= 0 ? 0u : w[i] & ((1u << (8 * left)) - 1);
    }
    return w;
}

// ---- up to 16 rows of a ------------------------------------------------------------------
// A few tokens against a weight: the weight's bytes, read once, are what it
// costs.  A workgroup takes 16 rows of b and all of a; its waves share the
// 128-wide blocks of the contraction and read both operands straight into the
// registers of v_mfma_f32_16x16x128_f8f6f4 (lane l: row l % 16, bytes
// 32 (l / 16) .. + 31 of the block, so four lanes read one row's 128-byte
// line), two blocks at a time and two such batches ahead.  b is the first
// operand: a lane's four sums belong to one token and four neighbouring columns
// of Y.  The waves' sums meet in LDS and are added in wave order.
//
// Exponent scales are the instruction's own, one load for a's and one for b's;
// binary32 scales are applied by significands and exponents, beside the memory.
// 1 x 4096 x 4096, bfloat16 outputs, on a weight that has left the caches: 6.8
// us of GPU time (e8m0 5.9), of which a launch is 2.3 and the weight at a
// copy's rate 3.6; 1 x 16384 x 8192: 27 us, 5.0 TB/s.  32 rows of b to a
// workgroup halve what is read of a, which comes from L2, and were slower (7.3
// us where 16 took 5.4).
constexpr int kSkinnyBlocks = 2, kSkinnyAhead = 2;
struct Frag {
    v4u lo, hi;
};
__device__ __forceinline__ v8i frag_words(const Frag &f) {
    return v8i{(int)f.lo[0], (int)f.lo[1], (int)f.lo[2], (int)f.lo[3],
               (int)f.hi[0], (int)f.hi[1], (int)f.hi[2], (int)f.hi[3]};
}

template <int ST, int AT, bool WIDE>
__global__ __launch_bounds__(1024) void mm_skinny_kernel(MmArgs g) {
    constexpr int U = kSkinnyBlocks, D = kSkinnyAhead;
    extern __shared__ float part[];                         // [waves][64][4]
    const int tid = threadIdx.x, lane = tid & 63, waves = blockDim.x >> 6;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int n0 = blockIdx.x * 16, kb_all = (g.K + 127) >> 7;

    // rows past the last are the last, and their sums are not stored
    const uint8_t *brow = g.b + (int64_t)min(n0 + l16, g.N - 1) * g.ldb;
    const int m = min(l16, g.M - 1);
    const uint8_t *arow = g.a + (int64_t)m * g.lda;
    const int64_t as_row = (int64_t)(m >> g.a_shift) * g.as_row;
    v4f acc{0, 0, 0, 0};

    constexpr bool HWS = ST == RNS_T_E8M0 && !WIDE;          // the instruction applies the scales: those of its lane's rows
    struct Batch {
        Frag b[U], a[U];
        uint32_t sa[U], sb[U][4];
    };
    const int last_chunk = (g.K - 1) & ~15;
    // Blocks kb0 .. kb0 + U - 1; what lies past K is read from K's last chunk, and cleared or left out by `work`.
    auto fetch = [&](int kb0, Batch &x) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int at = (kb0 + u) * 128 + quad * 32, lo = min(at, last_chunk), hi = min(at + 16, last_chunk);
            x.b[u] = Frag{*(const v4u *)(brow + lo), *(const v4u *)(brow + hi)};
            x.a[u] = Frag{*(const v4u *)(arow + lo), *(const v4u *)(arow + hi)};
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int kb = min(kb0 + u, kb_all - 1);
            x.sa[u] = load_scale<ST>(g.as, as_row + kb * g.as_blk);
            if (HWS) {
                x.sb[u][0] = load_scale<ST>(g.bs, (min(n0 + l16, g.N - 1) >> g.b_shift) * g.bs_row + kb * g.bs_blk);
            } else if (g.b_shift) {
                // 16 rows that start at a multiple of 16 share a block
                x.sb[u][0] = load_scale<ST>(g.bs, (n0 >> 7) * g.bs_row + kb * g.bs_blk);
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    x.sb[u][e] = load_scale<ST>(g.bs, min(n0 + quad * 4 + e, g.N - 1) * g.bs_row + kb * g.bs_blk);
            }
        }
    };
    auto work = [&](int kb0, Batch &x) {
        if ((g.K & 127) != 0 && kb0 + U >= kb_all) {
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int at = (kb0 + u) * 128 + quad * 32;
                x.b[u] = Frag{clear_tail(x.b[u].lo, at, g.K), clear_tail(x.b[u].hi, at + 16, g.K)};
                x.a[u] = Frag{clear_tail(x.a[u].lo, at, g.K), clear_tail(x.a[u].hi, at + 16, g.K)};
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (kb0 + u >= kb_all) break;                    // a block past the end adds nothing, whatever its scale
            const v8i wb = frag_words(x.b[u]), wa = frag_words(x.a[u]);
            if constexpr (HWS) {
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wb, wa, acc, 0, AT == RNS_T_E5M2, 0, (int)x.sb[u][0], 0,
                                                                       (int)x.sa[u]);
                continue;
            }
            v4f p{0, 0, 0, 0};
            if constexpr (WIDE) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<RNS_T_E4M3>(wb[2 * i], wb[2 * i + 1]),
                                                                widen8<AT>(wa[2 * i], wa[2 * i + 1]), p, 0, 0, 0);
            } else {
                p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wb, wa, p, 0, AT == RNS_T_E5M2, 0, 0, 0, 0);
            }
            const float sa = scale_factor<ST>(x.sa[u]);
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[e] += scaled(p[e], sa, scale_factor<ST>(x.sb[u][g.b_shift ? 0 : e]));
        }
    };
    // While there are as many batches again, no load stands behind a branch: one that may not have been issued would
    // have to be waited for as if it had not.
    const int stride = waves * U, n = (kb_all - wave * U + stride - 1) / stride;   // this wave's batches
    Batch ring[D];
    auto start = [&](int i) { return (wave + i * waves) * U; };
#pragma unroll
    for (int i = 0; i < D; i++)
        if (i < n) fetch(start(i), ring[i]);
    int i = 0;
    for (; i + 2 * D <= n; i += D)
#pragma unroll
        for (int d = 0; d < D; d++) {
            work(start(i + d), ring[d]);
            fetch(start(i + d + D), ring[d]);
        }
    for (; i < n; i += D)
#pragma unroll
        for (int d = 0; d < D; d++) {
            if (i + d >= n) break;
            work(start(i + d), ring[d]);
            if (i + d + D < n) fetch(start(i + d + D), ring[d]);
        }
    *(v4f *)&part[(wave * 64 + lane) * 4] = acc;
    __syncthreads();
    if (tid < 64) {
        v4f s{0, 0, 0, 0};
        for (int w = 0; w < waves; w++) s += *(const v4f *)&part[(w * 64 + lane) * 4];
        const int n = n0 + quad * 4;
        const float v[4] = {s[0], s[1], s[2], s[3]};
        if (l16 < g.M && n < g.N) store4(g, l16, n, v);
    }
}

// ---- T x T tiles, T = 64 or 128 -----------------------------------------------------------
// T = 128: eight waves, each with a 64 x 32 part of the tile, one workgroup
// on a compute unit; T = 64: four waves of 32 x 32, two workgroups, or (KG =
// 2) one of two such groups, each with its own ring and half of the blocks,
// whose sums meet in LDS.  A ring of four 128-wide blocks of the contraction
// in LDS: while the fragments of one are in the matrix cores, those of the
// next are read from LDS into registers and the three after that are on their
// way, straight from memory (global_load_lds, 16 bytes a lane).  One barrier
// a block keeps the waves together: a wave first waits for its own loads of
// the next block and for its fragments of this one, and behind the barrier
// requests the block four further into this one's place, which every wave has
// read.
//
// LDS rows are 128 bytes; 16-byte chunk c of row r lies at chunk c ^ swz8(r),
// so that the 16 rows of a fragment read spread over the banks; the loads
// fetch chunk (lane % 8) ^ swz8(row) into place lane % 8.  Chunks past K are
// fetched from a block of zeros, and of the chunk that K ends inside the lane
// that fetched it clears the rest.  Scales travel beside, one word for each row
// of a and of b (a byte arrives with zeros above it).
//
// HWS: both scale arrays are powers of two, which v_mfma_scale applies to the
// operands itself.  Otherwise a block's product starts from zero and is scaled
// into the sum by fused multiply-adds (BROW: b's scales differ by row); a block
// with scales far from one first, by significands and exponents.
//
// A block's fragments cost more to read from LDS (T = 128: 96 KiB at 128 bytes
// a clock, 0.32 us) than to multiply (0.21 us at the instructions' rate);
// measured, a block takes 0.65 us (both arrays powers of two) to 0.85, and 1.5
// to 1.8 with a binary32 result.  2048 x 2048 x 4096, one tile to a compute unit:
// 24 us; binary32 scales 27, those of single rows of b 30; binary32 results 51
// and 58.
__device__ __attribute__((aligned(16))) const uint32_t kZeros[4] = {0, 0, 0, 0};

__device__ __forceinline__ int swz8(int row) { return (row ^ (row >> 3)) & 7; }

__device__ __forceinline__ void direct_load(const void *src, v4u *dst) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

// A scale straight into LDS, one word a lane: a byte arrives with zeros above it.
__device__ __forceinline__ void direct_scale(const void *s, bool e8m0, int64_t i, uint32_t *dst) {
    if (e8m0)
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)((const uint8_t *)s + i),
                                         (__attribute__((address_space(3))) void *)dst, 1, 0, 0);
    else
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)((const float *)s + i),
                                         (__attribute__((address_space(3))) void *)dst, 4, 0, 0);
}

// Work item -> tile: consecutive workgroups go to the 8 XCDs in turn, so
// workgroup i takes tile (i % 8) G / 8 + i / 8 and an XCD works through one run
// of tiles; a run walks down four tile rows before it moves to the next column.
__device__ __forceinline__ void locate_tile(int i, int G, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int xcd = i & 7;
    const int t = xcd * (G >> 3) + min(xcd, G & 7) + (i >> 3);
    const int per = 4 * tiles_n, band = t / per, first = band * 4;
    const int rows = min(4, tiles_m - first), in = t - band * per;
    tn = in / rows;
    tm = first + in - tn * rows;
}

template <int N>
__device__ __forceinline__ void wait_loads() {               // at most N of this wave's loads outstanding
    __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0f70);
}
typedef __attribute__((address_space(3))) const uint8_t *lds_bytes;
typedef __attribute__((address_space(3))) const v4u *lds_chunk;

template <int T, int KG, int AT, bool WIDE, bool HWS, bool BROW>
__global__ __launch_bounds__(T * 4 * KG) void mm_tile_kernel(MmArgs g) {
    constexpr int RING = 4, LOADS = 5;                       // blocks in LDS; a wave's loads of a block
    constexpr int THREADS = T * 4, STEP = T / 2;             // threads of a group
    constexpr int FI = T / 32;                               // 16-row fragments of a that a wave has; of b it has two
    // [place]: T rows of a, T rows of b, 8 chunks each; then the scales, twice.  One array: beside a second shared
    // variable the compiler waits for all direct loads before every fragment read.
    constexpr int SIZE = RING * T * 16 + RING * T;
    __shared__ v4u shared[SIZE * KG];
    const int tid = threadIdx.x % THREADS, lane = tid & 63;
    const int group = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / THREADS);
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    v4u(*lds)[T * 16] = (v4u(*)[T * 16])(shared + group * SIZE);
    uint32_t(*scales)[T * 4] = (uint32_t(*)[T * 4])(shared + group * SIZE + RING * T * 16);
    const int quad = lane >> 4, l16 = lane & 15, wm = wave & 1, wn = wave >> 1;

    int tm, tn;
    const int tiles = g.tiles_m * g.tiles_n;
    const int part = blockIdx.x / tiles;
    locate_tile(blockIdx.x - part * tiles, tiles, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * T, n0 = tn * T;
    const int kb_all = (g.K + 127) >> 7;
    // this part's blocks; of two groups the first takes half, and one more of an odd number
    int first = (int)((int64_t)kb_all * part / g.split), last = (int)((int64_t)kb_all * (part + 1) / g.split);
    const int count = (last - first + KG - 1) / KG;
    const int steady = min(last, g.K >> 7) - (first + count * (KG - 1)) - RING - 1;   // steps that all groups have
    if (group) first += count;
    last = min(last, first + count);

    // requests: rows STEP q + 8 wave + lane / 8 of a and of b, q = 0, 1, past the last row the last row, at 32-bit
    // offsets from the tile's first (pitches are below 2^22)
    const int row0 = wave * 8 + (lane >> 3);
    auto column = [&](int q) { return ((lane & 7) ^ swz8(row0 + STEP * q)) * 16; };   // T = 128: the same for both
    const uint8_t *abase = g.a + (int64_t)m0 * g.lda, *bbase = g.b + (int64_t)n0 * g.ldb;
    uint32_t off[4];
#pragma unroll
    for (int q = 0; q < 2; q++) {
        off[q] = (uint32_t)min(row0 + STEP * q, g.M - 1 - m0) * (uint32_t)g.lda + column(q);
        off[2 + q] = (uint32_t)min(row0 + STEP * q, g.N - 1 - n0) * (uint32_t)g.ldb + column(q);
    }
    // scales: the waves in turn fetch 64 rows of a, then of b, each; the second half of the waves the same once more
    // (every wave has as many loads)
    const bool of_a = (wave & (T / 64)) == 0, e8m0 = HWS || (WIDE && g.e8m0);   // (8-bit instructions: HWS)
    const int srow = (T == 128 ? (wave & 1) * 64 : 0) + lane, es = e8m0 ? 1 : 4;
    const uint8_t *sbase = (const uint8_t *)(of_a ? g.as : g.bs);
    const int64_t sblk = (of_a ? g.as_blk : g.bs_blk) * es;
    const uint8_t *sat = sbase + es * (of_a ? (int64_t)(min(m0 + srow, g.M - 1) >> g.a_shift) * g.as_row
                                            : (int64_t)(min(n0 + srow, g.N - 1) >> g.b_shift) * g.bs_row);
    // request i = 0 .. 4 of a block; `whole`: the block ends before K
    auto request = [&](auto whole, int kb, int i) {
        if (i == 4) {
            direct_scale(sat + kb * sblk, e8m0, 0, scales[kb & (RING - 1)] + wave * 64);
            return;
        }
        uint32_t o = off[i];
        asm volatile("" : "+v"(o));                          // a 32-bit offset from a uniform address, not a kept pointer
        const uint8_t *p = (i < 2 ? abase : bbase) + (int64_t)kb * 128 + o;
        if constexpr (!decltype(whole)::value)
            if (kb * 128 + column(i & 1) >= g.K) p = (const uint8_t *)kZeros;
        direct_load(p, lds[kb & (RING - 1)] + i * THREADS + wave * 64);
    };
    auto trim = [&](int kb) {
#pragma unroll 1
        for (int q = 0; q < 4; q++) {
            const int k = kb * 128 + column(q & 1);
            if (k >= g.K || k + 16 <= g.K) continue;
            v4u *at = lds[kb & (RING - 1)] + q * THREADS + wave * 64 + lane;
            *at = clear_tail(*at, k, g.K);
        }
    };

    v4f acc[FI][2];                                          // [16 rows of a][16 rows of b]
#pragma unroll
    for (int i = 0; i < FI; i++)
#pragma unroll
        for (int j = 0; j < 2; j++) acc[i][j] = v4f{0, 0, 0, 0};
    // Fragment row 16 f + l16 of a region: chunk 2 quad + t of it lies at chunk (2 quad + t) ^ swz8(l16) ^ 2 (f % 4).
    const uint32_t at0 = l16 * 128 + (((quad * 2) ^ swz8(l16)) * 16);
    const lds_bytes lds0 = (lds_bytes)&shared[group * SIZE];
    auto fragment = [&](uint32_t region, int f) -> v8i {     // region: a multiple of 64 rows and f below 4, or of 32
        const uint32_t a = (at0 ^ (32 * (f & 3))) + region + f * 2048;
        return frag_words(Frag{*(lds_chunk)(lds0 + a), *(lds_chunk)(lds0 + (a ^ 16))});
    };
    auto factor = [&](uint32_t w) { return e8m0 ? e8m0_factor(w) : __uint_as_float(w); };

    const std::true_type yes;
    const std::false_type no;
    struct Block {
        v8i fa[FI], fb[2];
        uint32_t sa[FI], sb[2];
    };
    auto read = [&](int kb, Block &r) {
        // fragment rows: of a from wm T / 2 on, of b from 32 wn on
        const uint32_t place = (kb & (RING - 1)) * (T * 256);
        const uint32_t A = place + (T == 128 ? wm * 8192 : 0), B = place + T * 128 + (wn >> 1) * 8192;
        const uint32_t *sc = scales[kb & (RING - 1)];
#pragma unroll
        for (int j = 0; j < 2; j++) r.fb[j] = fragment(B, (wn & 1) * 2 + j);
#pragma unroll
        for (int i = 0; i < FI; i++) r.fa[i] = fragment(A, (T == 128 ? 0 : wm * 2) + i);
#pragma unroll
        for (int i = 0; i < FI; i++) r.sa[i] = sc[wm * STEP + i * 16 + l16];
        if (HWS)
#pragma unroll
            for (int j = 0; j < 2; j++) r.sb[j] = sc[T + wn * 32 + j * 16 + l16];
        if (!HWS && !BROW) r.sb[0] = sc[T];                  // T rows from a multiple of T share theirs
    };
    // own loads of block kb are here, as far as there is one; its last chunk is clean
    auto arrived = [&](int kb) {
        if (kb + 2 < last) wait_loads<2 * LOADS>();
        else if (kb + 1 < last) wait_loads<LOADS>();
        else wait_loads<0>();
        if (kb == kb_all - 1 && (g.K & 15) != 0) trim(kb);
    };
    auto fence = [&]() {
        __builtin_amdgcn_s_waitcnt(0xc07f);                  // lgkmcnt(0)
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    // STEADY: the block that this step requests is there and whole, so that the loop over such steps has no branches
    auto step = [&](auto steady, int kb, const Block &r, Block &next) {
        constexpr bool S = decltype(steady)::value;
        if (KG > 1 && !S && kb >= last) {                    // the other group has one more
            fence();
            return;
        }
        v4u sb[2];
        if (BROW && !HWS)
#pragma unroll
            for (int j = 0; j < 2; j++) sb[j] = *(const v4u *)&scales[kb & (RING - 1)][T + wn * 32 + j * 16 + 4 * quad];
        if (S) wait_loads<2 * LOADS>();
        else if (kb + 1 < last) arrived(kb + 1);
        fence();
        if (S || kb + 1 < last) read(kb + 1, next);
        __builtin_amdgcn_sched_barrier(0);
        // row fragment by row fragment, the requests between
        auto requests = [&](int i) {
            if (S || kb + RING < last) {
                constexpr int EACH = 4 / FI;
#pragma unroll
                for (int l = 0; l < EACH; l++) request(steady, kb + RING, i * EACH + l);
                if (i == FI - 1) request(steady, kb + RING, 4);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        if constexpr (HWS) {
#pragma unroll
            for (int i = 0; i < FI; i++) {
#pragma unroll
                for (int j = 0; j < 2; j++)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        r.fb[j], r.fa[i], acc[i][j], 0, AT == RNS_T_E5M2, 0, (int)r.sb[j], 0, (int)r.sa[i]);
                requests(i);
            }
        } else {
            v4f p[FI][2];
            float s[FI], fb[2][4];                           // BROW: a's scales and b's; otherwise the products of both
            Extent x;
            auto look = [&](int i) {
                s[i] = BROW ? factor(r.sa[i]) : factor(r.sa[i]) * factor(r.sb[0]);
                x.add(s[i]);
                if constexpr (BROW)
#pragma unroll
                    for (int k = i * 8 / FI; k < (i + 1) * 8 / FI; k++) {
                        fb[k >> 2][k & 3] = factor(sb[k >> 2][k & 3]);
                        x.add(fb[k >> 2][k & 3]);
                    }
            };
            if constexpr (WIDE) {
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    v8bf wa[FI], wb[2];
#pragma unroll
                    for (int j = 0; j < 2; j++) wb[j] = widen8<RNS_T_E4M3>(r.fb[j][2 * q], r.fb[j][2 * q + 1]);
#pragma unroll
                    for (int i = 0; i < FI; i++) wa[i] = widen8<AT>(r.fa[i][2 * q], r.fa[i][2 * q + 1]);
#pragma unroll
                    for (int i = 0; i < FI; i++)
#pragma unroll
                        for (int j = 0; j < 2; j++)
                            p[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                wb[j], wa[i], q == 0 ? v4f{0, 0, 0, 0} : p[i][j], 0, 0, 0);
                    if (q < FI) {
                        look(q);
                        requests(q);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < FI; i++) {
#pragma unroll
                    for (int j = 0; j < 2; j++)
                        p[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            r.fb[j], r.fa[i], v4f{0, 0, 0, 0}, 0, AT == RNS_T_E5M2, 0, 0, 0, 0);
                    look(i);                                 // while the matrix cores are at work
                    requests(i);
                }
            }
            if (__any(BROW ? x.beyond(kScaleLow, kScaleHigh) : x.beyond(kSmallestNormal, kLargestFinite))) {
                // the products scaled, and factors of one
#pragma unroll
                for (int i = 0; i < FI; i++)
#pragma unroll
                    for (int j = 0; j < 2; j++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            p[i][j][e] = scaled(p[i][j][e], factor(r.sa[i]), BROW ? fb[j][e] : factor(r.sb[0]));
#pragma unroll
                for (int i = 0; i < FI; i++) s[i] = 1.f;
#pragma unroll
                for (int k = 0; k < 8; k++) fb[k >> 2][k & 3] = 1.f;
            }
#pragma unroll
            for (int i = 0; i < FI; i++)
#pragma unroll
                for (int j = 0; j < 2; j++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        acc[i][j][e] = BROW ? __builtin_fmaf(p[i][j][e] * s[i], fb[j][e], acc[i][j][e])
                                            : __builtin_fmaf(p[i][j][e], s[i], acc[i][j][e]);
        }
    };

#pragma unroll 1
    for (int i = first; i < min(first + RING, last); i++)
#pragma unroll
        for (int l = 0; l < LOADS; l++) request(no, i, l);
    if (first + 3 < last) wait_loads<3 * LOADS>();           // block `first` is here
    else wait_loads<0>();
    if (first == kb_all - 1 && (g.K & 15) != 0) trim(first);
    fence();
    Block even, odd;
    read(first, even);
    int done = 0;
    for (; done < steady; done += 2) {
        step(yes, first + done, even, odd);
        step(yes, first + done + 1, odd, even);
    }
    for (; done < count; done++) {
        step(no, first + done, even, odd);
        even = odd;
    }

    constexpr int PITCH = T + 4;                             // floats
    float *stage = (float *)shared;
    if constexpr (KG > 1) {
        // the second group's sums onto the first's
        fence();
        if (group)
#pragma unroll
            for (int i = 0; i < FI; i++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    *(v4f *)(stage + (wm * STEP + 16 * i + l16) * PITCH + wn * 32 + j * 16 + 4 * quad) = acc[i][j];
        fence();
        if (group) return;
#pragma unroll
        for (int i = 0; i < FI; i++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                acc[i][j] += *(const v4f *)(stage + (wm * STEP + 16 * i + l16) * PITCH + wn * 32 + j * 16 + 4 * quad);
    }

    const bool half = g.split == 1 && g.y_type != RNS_T_F32, bf16 = g.y_type == RNS_T_BF16;
    if (half && m0 + T <= g.M && n0 + T <= g.N && g.ldy % 8 == 0 && ((uintptr_t)g.y & 15) == 0) {
#pragma unroll
        for (int i = 0; i < FI; i++) {
            // neighbouring quads trade, so that each has eight neighbouring columns: quads 0 and 2 of the first
            // sixteen, quads 1 and 3 of the second
            uint32_t w[2][2];
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float x = acc[i][j][2 * e], y = acc[i][j][2 * e + 1];
                    w[j][e] = bf16 ? bf16_bits(x) | bf16_bits(y) << 16 : f16_bits(x) | f16_bits(y) << 16;
                }
            const auto r0 = __builtin_amdgcn_permlane16_swap(w[0][0], w[1][0], false, false);
            const auto r1 = __builtin_amdgcn_permlane16_swap(w[0][1], w[1][1], false, false);
            *(v4u *)((uint16_t *)g.y + (int64_t)(m0 + wm * STEP + 16 * i + l16) * g.ldy + n0 + wn * 32 +
                     (quad & 1) * 16 + (quad >> 1) * 8) = v4u{r0[0], r1[0], r0[1], r1[1]};
        }
        return;
    }
    // Anything else goes through LDS, so that the code that stores it is there once: a launch that is over soon
    // waits for its instructions too.
    fence();
#pragma unroll
    for (int i = 0; i < FI; i++)
#pragma unroll
        for (int j = 0; j < 2; j++)
            *(v4f *)(stage + (wm * STEP + 16 * i + l16) * PITCH + wn * 32 + j * 16 + 4 * quad) = acc[i][j];
    fence();
#pragma unroll 1
    for (int i = tid; i < T * T / 4; i += THREADS) {
        const int r = i / (T / 4), c = (i % (T / 4)) * 4, m = m0 + r, n = n0 + c;
        if (m >= g.M || n >= g.N) continue;
        const v4f x = *(const v4f *)(stage + r * PITCH + c);
        const float v[4] = {x[0], x[1], x[2], x[3]};
        if (g.split > 1) *(v4f *)(g.partial + ((int64_t)part * g.M + m) * g.partial_ld + n) = x;   // the pitch covers n + 3
        else store4(g, m, n, v);
    }
}

// ---- 256 x 256 tiles ----------------------------------------------------------------------
// Many tiles, 16-bit outputs.  Eight waves, two on a SIMD, each with a 128 x 64
// part of the tile; two groups of four alternate between reading fragments and
// computing, one group in each at any time, so that a SIMD's matrix core always
// has one wave's instructions to run while its other wave waits on LDS.
//
// A 128-wide block of the contraction takes two turns: the first reads all of
// the wave's fragments of b and the upper 64 of its rows of a, the second the
// lower 64 rows.  LDS holds two blocks (128 KiB).  What a block's first turn
// has read (b, and rows 0..63 and 128..191 of a: "first part") is free once
// both groups are past it, half a block before the rest, and is requested anew
// for the block after next at once: in the compute phase of the second turn;
// the rest ("second part") in the compute phase of the next first turn.  So
// loads have about a whole block's time to arrive.  The phases' order:
//
//   read 1 (block j)    fragments and scales; wait: the second part of j is here
//   compute 1           request the second part of j + 1
//   read 2              fragments and scales; wait: first part and scales of j + 1 are here
//   compute 2           request the scales and the first part of j + 2 (the scales into one of four places:
//                       group 1 may still be reading those of j)
//
// each followed by a barrier, group 1 one phase behind group 0.  A wave waits
// for its own loads before the barrier behind which another wave may read what
// they brought; a part is requested only after the barrier behind which every
// wave has read its last contents.
//
// v_mfma_f32_16x16x128_f8f6f4 takes a whole block in one instruction.  With
// binary32 scales its four sums a lane are scaled into the total by vector
// instructions that run while the next products are in the matrix core; a
// phase's last three are left to the following read phase, which has time to
// spare.
//
// The matrix cores bound it: 8192 x 8192 x 8192 in 400 to 500 us (both arrays
// powers of two, 2.2 to 2.7 PFLOP/s), 540 to 620 with binary32 scales, whose
// vector instructions share the issue slots (taking each scale apart is 3% of
// it); the library's product with one scale for each whole operand takes 390 to
// 430.  4096 x 4096 x 4096: 57 to 61 us, 83 with binary32 scales, 51 there.
// b times a, times 2^(eb - 127) and 2^(byte i of ea - 127).
template <int AT>
__device__ __forceinline__ v4f scaled_product(const v8i &b, const v8i &a, int i, uint32_t eb, uint32_t ea) {
    constexpr v4f zero{0, 0, 0, 0};
    constexpr int type = AT == RNS_T_E5M2;
    if (i == 0) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, zero, 0, type, 0, (int)eb, 0, (int)ea);
    if (i == 1) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, zero, 0, type, 0, (int)eb, 1, (int)ea);
    if (i == 2) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, zero, 0, type, 0, (int)eb, 2, (int)ea);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, zero, 0, type, 0, (int)eb, 3, (int)ea);
}

template <int AT, bool HWS>
__global__ __launch_bounds__(512) void mm_big_kernel(MmArgs g) {
    // 256 rows of a, 256 rows of b, 8 chunks each, twice; then four places for scales.  One array: beside a second
    // shared variable the compiler waits for all direct loads before every fragment read.
    __shared__ v4u shared[2 * 4096 + 4 * 512 / 4];
    v4u(*lds)[4096] = (v4u(*)[4096])shared;
    uint32_t(*scales)[512] = (uint32_t(*)[512])(shared + 2 * 4096);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), group = wave >> 2;
    const int quad = lane >> 4, l16 = lane & 15, wm = wave & 1, wn = wave >> 1;
    int tm, tn;
    locate_tile(blockIdx.x, g.tiles_m * g.tiles_n, g.tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * 256, n0 = tn * 256;
    const int kbs = (g.K + 127) >> 7;

    // Scales travel through LDS: thread t fetches that of row t of a (t < 256: waves 0 to 3) or of row t - 256 of b,
    // at a 32-bit offset from the tile's first (the host has checked that they fit).
    constexpr int es = HWS ? 1 : 4;
    const int srow = (wave < 4 ? m0 : n0) + (tid & 255), s0 = wave < 4 ? m0 : n0, shift = wave < 4 ? g.a_shift : g.b_shift;
    const int64_t sstride = (wave < 4 ? g.as_row : g.bs_row) * es, sblk = (wave < 4 ? g.as_blk : g.bs_blk) * es;
    const uint8_t *sbase = (const uint8_t *)(wave < 4 ? g.as : g.bs) + (int64_t)(s0 >> shift) * sstride;
    const uint32_t soff = (uint32_t)((min(srow, (wave < 4 ? g.M : g.N) - 1) >> shift) - (s0 >> shift)) * (uint32_t)sstride;
    auto request_scales = [&](int kb) {
        uint32_t off = soff;
        asm volatile("" : "+v"(off));
        direct_scale(sbase + (int64_t)kb * sblk + off, HWS, 0, scales[kb & 3] + wave * 64);
    };

    // The lane index, read afresh where it is wanted: nothing derived from it is kept across the loop, whose registers
    // are all taken.
    auto lane_now = []() {
        int l;
        asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
        return l;
    };
    // byte of this lane's chunk in its row of 128
    auto chunk_at = [&](int ln) { return ((ln & 7) ^ (ln >> 3) ^ wave) * 16; };
    // requests: rows 64 q + 8 wave + lane / 8 of a and of b, q = 0 .. 3.  A lane whose row is past the operand's last
    // reads that one's last chunk of the block instead (what it brings is not stored): offsets are cut off there,
    // which leaves those of the last row itself alone.
    const uint32_t last_a = (uint32_t)min(255, g.M - 1 - m0) * (uint32_t)g.lda;
    const uint32_t last_b = (uint32_t)min(255, g.N - 1 - n0) * (uint32_t)g.ldb;
    const uint8_t *abase = g.a + (int64_t)m0 * g.lda, *bbase = g.b + (int64_t)n0 * g.ldb;
    const uint32_t off_a = (uint32_t)(wave * 8 + (lane >> 3)) * (uint32_t)g.lda + chunk_at(lane);
    const uint32_t off_b = (uint32_t)(wave * 8 + (lane >> 3)) * (uint32_t)g.ldb + chunk_at(lane);
    auto request = [&](auto whole, int kb, int q) {
        uint32_t off = q < 4 ? off_a : off_b;
        asm volatile("" : "+v"(off));                        // not to be kept eight times over
        const int chunks = decltype(whole)::value ? 112 : min(112, ((g.K + 15) & ~15) - 16 - kb * 128);
        off = min(off + (uint32_t)(64 * (q & 3)) * (uint32_t)(q < 4 ? g.lda : g.ldb), (q < 4 ? last_a : last_b) + chunks);
        const uint8_t *p = (q < 4 ? abase : bbase) + (int64_t)kb * 128 + off;
        if constexpr (!decltype(whole)::value)
            if (kb * 128 + chunk_at(lane_now()) >= g.K) p = (const uint8_t *)kZeros;
        direct_load(p, lds[kb & 1] + q * 512 + wave * 64);
    };
    // A chunk that K ends inside: the lane that fetched it clears its bytes from K on, once it is here and before the
    // barrier that shows it to the other waves.
    const bool straddle = (g.K & 15) != 0;
    auto trim = [&](int kb, bool first) {
        const int ln = lane_now(), c16 = chunk_at(ln);
        if (kb * 128 + c16 >= g.K || kb * 128 + c16 + 16 <= g.K) return;
#pragma unroll 1
        for (int q = 0; q < 8; q++) {
            if (((q & 1) == 0 || q >= 4) != first) continue;
            v4u *at = lds[kb & 1] + q * 512 + wave * 64 + ln;
            *at = clear_tail(*at, kb * 128 + c16, g.K);
        }
    };

    // request i = 0 .. 6 of a block's first part; of its second part there are two, for q = 1 and 3
    auto request_first = [&](auto whole, int kb, int i) {
        if (i == 0) request_scales(kb);
        else request(whole, kb, i < 3 ? (i - 1) * 2 : i + 1);
    };
    v4f acc[8][4];                                           // [16 rows of a][16 rows of b]
#pragma unroll
    for (int i = 0; i < 8; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = v4f{0, 0, 0, 0};
    v8i fa[4], fb[4];
    // Binary32 scales: the products of the last LAG instructions, not yet scaled into their sums.  The first ones are
    // zeros, scaled by zero.
    constexpr int LAG = 3;
    v4f p[LAG + 1];
#pragma unroll
    for (int i = 0; i <= LAG; i++) p[i] = v4f{0, 0, 0, 0};
    // Fragment row 16 f + l16 of a region: chunk 2 quad + t of it lies at chunk (2 quad + t) ^ swz8(l16) ^ 2 (f % 4),
    // so one byte offset serves every fragment, with bits 5 and 6 turned by f and bit 4 by t.
    const uint32_t at0 = l16 * 128 + (((quad * 2) ^ swz8(l16)) * 16);
    const lds_bytes lds0 = (lds_bytes)&shared[0];
    auto fragment = [&](uint32_t region, int f) -> v8i {
        const uint32_t a = (at0 ^ (32 * (f & 3))) + region + f * 2048;
        return frag_words(Frag{*(lds_chunk)(lds0 + a), *(lds_chunk)(lds0 + (a ^ 16))});
    };
    // Binary32 scales: the instruction takes their powers of two (a's four in the bytes of ea, b's in eb), which it applies
    // before anything is rounded, so that nothing leaves binary32's range before the result does; what is left of b's
    // scale is rb, and of both s.
    uint32_t sa[4], sb[4], ea = 0x7f7f7f7f, eb = 127;
    float s[4] = {0, 0, 0, 0}, rb = 1;
    auto scale_in = [&](v4f &to, const v4f &from, float f) {
#pragma unroll
        for (int e = 0; e < 4; e++) to[e] = __builtin_fmaf(from[e], f, to[e]);
    };
    // the scales of block kb for rows 64 h .. of this wave, as they are; asked for before the fragments, they are worked on
    // while those are on their way
    auto read_scales = [&](int kb, int h) {
        const uint32_t *sc = scales[kb & 3];
#pragma unroll
        for (int i = 0; i < 4; i++) sa[i] = sc[wm * 128 + h * 64 + i * 16 + l16];
        if (HWS && h == 0)
#pragma unroll
            for (int j = 0; j < 4; j++) sb[j] = sc[256 + wn * 64 + 16 * j + l16];
        if (!HWS && h == 0) sb[0] = sc[256 + wn * 64];
        __builtin_amdgcn_sched_barrier(0);
    };
    auto split_scales = [&](int h) {
        if constexpr (!HWS) {
            if (h == 0) {
                const Split b = split_scale<1, 253>(__uint_as_float(sb[0]));
                eb = b.e;
                rb = b.r;
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const Split a = split_scale<1, 253>(__uint_as_float(sa[i]));
                ea = i == 0 ? a.e : ea | a.e << 8 * i;
                s[i] = a.r * rb;
            }
        }
    };
    // the products that a compute phase left unscaled: the last ones of row fragment 3
    auto finish = [&](int h) {
        if constexpr (!HWS)
#pragma unroll
            for (int t = 16 - LAG; t < 16; t++) scale_in(acc[4 * h + 3][t & 3], p[t & LAG], s[3]);
    };
    auto fence = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    // Rows 64 h .. of this wave: sixteen instructions, each followed by the scaling of the product LAG before it, which
    // is done by then, and by one of the phase's requests where it has one left.
    auto compute = [&](int h, auto requests) {
#pragma unroll
        for (int t = 0; t < 16; t++) {
            const int i = t >> 2, j = t & 3;
            if constexpr (HWS) {
                acc[4 * h + i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    fb[j], fa[i], acc[4 * h + i][j], 0, AT == RNS_T_E5M2, 0, (int)sb[j], 0, (int)sa[i]);
            } else {
                p[t & LAG] = scaled_product<AT>(fb[j], fa[i], i, eb, ea);
                if (t >= LAG) {
                    const int u = t - LAG;
                    scale_in(acc[4 * h + (u >> 2)][u & 3], p[u & LAG], s[u >> 2]);
                }
            }
            requests(t);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // One block.  STEADY: blocks j + 1 and j + 2 are there and whole, so that the loop over such blocks has no
    // branches and every wait's count is known.
    auto block = [&](auto steady, int j) {
        constexpr bool S = decltype(steady)::value;
        const uint32_t A = (j & 1) * 65536 + wm * 16384, B = (j & 1) * 65536 + 32768 + wn * 8192;
        // read 1
        read_scales(j, 0);
#pragma unroll
        for (int f = 0; f < 4; f++) fb[f] = fragment(B, f), fa[f] = fragment(A, f);
        finish(1);
        split_scales(0);
        if (S || j + 1 < kbs) wait_loads<7>();
        else wait_loads<0>();
        if (!S && straddle && j == kbs - 1) trim(j, false);
        __builtin_amdgcn_s_waitcnt(0xc07f);                  // the fragments
        fence();
        // compute 1
        compute(0, [&](int t) {
            if ((S || j + 1 < kbs) && t % 6 == 1 && t < 8) request(steady, j + 1, t / 6 * 2 + 1);
        });
        fence();
        // read 2
        read_scales(j, 1);
#pragma unroll
        for (int f = 0; f < 4; f++) fa[f] = fragment(A, 4 + f);
        finish(0);
        split_scales(1);
        if (S || j + 1 < kbs) wait_loads<2>();
        else wait_loads<0>();
        if (!S && straddle && j + 2 == kbs) trim(j + 1, true);
        __builtin_amdgcn_s_waitcnt(0xc07f);
        fence();
        // compute 2
        compute(1, [&](int t) {
            if ((S || j + 2 < kbs) && t % 2 == 1 && t < 14) request_first(steady, j + 2, t / 2);
        });
        fence();
    };
    const std::true_type yes;
    const std::false_type no;

    // the blocks before the loop; the first part of block 0 is here when they are done
    auto begin = [&](auto whole) {
#pragma unroll
        for (int i = 0; i < 7; i++) request_first(whole, 0, i);
        request(whole, 0, 1);
        request(whole, 0, 3);
        if (decltype(whole)::value || kbs > 1) {
#pragma unroll
            for (int i = 0; i < 7; i++) request_first(whole, 1, i);
            wait_loads<2 + 7>();
        } else {
            wait_loads<0>();
            if (straddle) trim(0, true);
            __builtin_amdgcn_s_waitcnt(0xc07f);              // lgkmcnt(0)
        }
        __builtin_amdgcn_s_barrier();
        if (group == 1) fence();
    };
    const int steady = (g.K >> 7) - 2;                       // blocks with two whole ones behind them
    int j = 0;
    if (steady > 0) {
        begin(yes);
        for (; j < steady; j++) block(yes, j);
    } else {
        begin(no);
    }
    for (; j < kbs; j++) block(no, j);
    if (group == 0) fence();
    finish(1);

    // A lane holds, of its row, columns 4 quad .. + 3 of each of four groups of 16.  The quads trade (a 4 x 4
    // transposition of the wave's 16-lane rows) so that each has one whole group: 32 neighbouring bytes.
    const int ln = lane_now(), end_quad = ln >> 4;
    const int ma = m0 + wm * 128 + (ln & 15), nb = n0 + wn * 64;
    const bool whole = m0 + 256 <= g.M && n0 + 256 <= g.N && g.ldy % 8 == 0 && ((uintptr_t)g.y & 15) == 0;
    const bool bf16 = g.y_type == RNS_T_BF16;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int m = ma + 16 * i;
        if (whole) {
            uint32_t w[4][2];
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float x = acc[i][j][2 * e], y = acc[i][j][2 * e + 1];
                    w[j][e] = bf16 ? bf16_bits(x) | bf16_bits(y) << 16 : f16_bits(x) | f16_bits(y) << 16;
                }
#pragma unroll
            for (int e = 0; e < 2; e++) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const auto r = __builtin_amdgcn_permlane32_swap(w[j][e], w[j + 2][e], false, false);
                    w[j][e] = r[0];
                    w[j + 2][e] = r[1];
                }
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const auto r = __builtin_amdgcn_permlane16_swap(w[j][e], w[j + 1][e], false, false);
                    w[j][e] = r[0];
                    w[j + 1][e] = r[1];
                }
            }
            uint16_t *y = (uint16_t *)g.y + (int64_t)m * g.ldy + nb + end_quad * 16;
            *(v4u *)y = v4u{w[0][0], w[0][1], w[1][0], w[1][1]};
            *(v4u *)(y + 8) = v4u{w[2][0], w[2][1], w[3][0], w[3][1]};
        } else {
            // an edge: through this wave's own corner of LDS, so that the code that stores it is short
            float *stage = (float *)shared + wave * 16 * 68;
#pragma unroll
            for (int j = 0; j < 4; j++) *(v4f *)(stage + (ln & 15) * 68 + j * 16 + 4 * end_quad) = acc[i][j];
            __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll 1
            for (int k = ln; k < 256; k += 64) {
                const int r = k >> 4, c = (k & 15) * 4, row = m0 + wm * 128 + 16 * i + r, n = nb + c;
                const v4f x = *(const v4f *)(stage + r * 68 + c);
                const float v[4] = {x[0], x[1], x[2], x[3]};
                if (row < g.M && n < g.N) store4(g, row, n, v);
            }
        }
    }
}

// Y from the parts of a product that was split along K, added in order.
__global__ __launch_bounds__(256) void mm_join_kernel(MmArgs g) {
    const int64_t per_row = g.partial_ld / 4, count = per_row * g.M;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
        const int m = (int)(i / per_row), n = (int)(i - m * per_row) * 4;
        if (n >= g.N) continue;
        v4f s{0, 0, 0, 0};
        for (int p = 0; p < g.split; p++) s += *(const v4f *)(g.partial + ((int64_t)p * g.M + m) * g.partial_ld + n);
        const float v[4] = {s[0], s[1], s[2], s[3]};
        store4(g, m, n, v);
    }
}

}  // namespace rns

using namespace rns;

namespace {

bool operand_ok(const rns_scaled_t *o, int64_t rows, int64_t K) {
    if (!o || (o->type != RNS_T_E4M3 && o->type != RNS_T_E5M2)) return false;
    if (o->scale_type != RNS_T_F32 && o->scale_type != RNS_T_E8M0) return false;
    if (o->block_rows != 1 && o->block_rows != 128) return false;
    if (o->scale_type == RNS_T_F32 && (uintptr_t)o->scales % 4) return false;
    return o->ld >= K && o->ld <= RNS_SCALED_LD_MAX && o->s_row >= 0 && o->s_blk >= 0 && rows >= 0;
}

int device_cus() {
    static int cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
    if (dev < 64 && cached[dev] > 0) return cached[dev];
    int cus = 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1) return 256;
    if (dev < 64) cached[dev] = cus;
    return cus;
}

enum Path { kGeneral, kSkinny, kSmall, kPair, kTile, kBig };

struct MmPlan {
    Path path;
    int split;
    int64_t partial_ld;
    size_t bytes;
};

// Rows on 16-byte boundaries that can be read to the next one.
bool aligned(const rns_scaled_t *o) {
    return (uintptr_t)o->values % 16 == 0 && o->ld % 16 == 0 && o->readable;
}

MmPlan plan_mm(int64_t M, int64_t N, int64_t K, const rns_scaled_t *a, const rns_scaled_t *b, bool wide) {
    MmPlan p{kGeneral, 1, 0, 0};
    if (M == 0 || N == 0 || K == 0 || !aligned(a) || !aligned(b)) return p;
    // Figures here: GPU time of one product among others, on operands that have left the caches where those are small.
    // Up to 16 rows read the weight straight into registers: 16 x 4096 x 4096 in 7.5 us, against 10.4 in tiles of 64
    // that split the contraction.  With over 8 rows and much of a weight to read the tiles win, whose rows of a are not
    // fetched again for every 16 of b: 16 x 16384 x 8192 in 34 us against 36, 16 x 1024 x 16384 in 12.8 against 18.
    // At twice the instructions, for 32-bit outputs, they do not (16 x 4096 x 4096 in 14 against 7.7).
    if (M <= 16 && (wide || M <= 8 || (N * K < (int64_t)1 << 26 && K <= 8192))) {
        p.path = kSkinny;
        return p;
    }
    // Tiles of 256 where those of 128 take more than twice as many rounds of the chip: 3328 x 3328 x 4096 (one round
    // against three) in 52 us against 66, with binary32 scales 74 against 75; 2816 x 2816 x 4096 (one against two) in 50
    // against 45, and 72 against 52.  Of two blocks only, 8192 x 8192 x 256 takes 48 against 72, but with binary32 scales
    // 87 against 75.  They have no form for 32-bit outputs, nor for binary32 scales of single rows of b,
    // and scale offsets inside a tile are 32-bit there.
    const int cus = device_cus();
    const int64_t far = (int64_t)1 << 20;
    if (!wide && (a->scale_type == RNS_T_E8M0 || b->block_rows == 128) && a->s_row < far && b->s_row < far &&
        div_up(div_up(M, 128) * div_up(N, 128), cus) > 2 * div_up(div_up(M, 256) * div_up(N, 256), cus)) {
        p.path = kBig;
        return p;
    }
    // Tiles of 64 where those of 128 would fill at most half of the chip: 777 x 1100 x 650 in 7.1 us against 11.2, 512 x
    // 4096 x 4096 in 18 against 21 (binary32 scales 20 against 25); but 1000 x 3001 x 1537, three quarters of the chip,
    // in 19.6 against 16.7.  And where the rows do not fill half of one: 48 x 32768 x 4096 in 34 us against 39.
    const int64_t blocks = div_up(K, 128);
    p.path = M <= 64 || div_up(M, 128) * div_up(N, 128) * 2 <= cus ? kSmall : kTile;
    // Where those are at most one to a compute unit, a tile's workgroup is two groups of waves that share its blocks (1024
    // x 1024 x 8192 in 19 us against 24 by one group; 777 x 1100 x 650 in 7.1 against 7.5, binary32 scales), and
    // where they are at most one to two units the contraction is split besides, while each part keeps at least 16
    // blocks: 48 x 8192 x 4096 in 14.0 us against 14.6, 64 x 4096 x 8192 in 14.8 against 23.6; parts of eight: 48 x 2048
    // x 2048 in 9.0 us against 8.3.
    const int64_t tiles = div_up(M, 64) * div_up(N, 64);
    if (p.path == kSmall && tiles <= cus && blocks >= 2) {
        p.path = kPair;
        while (tiles * p.split * 2 <= cus && blocks / (p.split * 2) >= 16) p.split *= 2;
    }
    if (p.split > 1) {
        p.partial_ld = div_up(N, 4) * 4;
        p.bytes = (size_t)(p.split * M * p.partial_ld * 4);
    }
    return p;
}

template <int AT, bool WIDE>
void launch_skinny(const MmArgs &g, hipStream_t s) {
    // as many waves as there are batches of blocks to share, up to 16 where few workgroups leave the chip idle
    const int64_t kb = div_up(g.K, 128), grid = div_up(g.N, 16);
    const int most = grid * 2 <= device_cus() ? 16 : 8;
    int waves = 1;
    while (waves < most && waves * kSkinnyBlocks < kb) waves *= 2;
    const dim3 blocks((unsigned)grid), threads(64 * waves);
    const size_t lds = (size_t)waves * 64 * 16;
    if (g.e8m0) hipLaunchKernelGGL((mm_skinny_kernel<RNS_T_E8M0, AT, WIDE>), blocks, threads, lds, s, g);
    else hipLaunchKernelGGL((mm_skinny_kernel<RNS_T_F32, AT, WIDE>), blocks, threads, lds, s, g);
}

template <int T, int KG, int AT, bool WIDE>
void launch_tile(dim3 grid, const MmArgs &g, hipStream_t s) {
    const dim3 threads(4 * T * KG);
    if (!WIDE && g.e8m0) hipLaunchKernelGGL((mm_tile_kernel<T, KG, AT, WIDE, !WIDE, false>), grid, threads, 0, s, g);
    else if (g.b_shift) hipLaunchKernelGGL((mm_tile_kernel<T, KG, AT, WIDE, false, false>), grid, threads, 0, s, g);
    else hipLaunchKernelGGL((mm_tile_kernel<T, KG, AT, WIDE, false, true>), grid, threads, 0, s, g);
}

template <int AT, bool WIDE>
void launch_mm(const MmPlan &p, const MmArgs &g, hipStream_t s) {
    if (p.path == kSkinny) {
        launch_skinny<AT, WIDE>(g, s);
        return;
    }
    if (p.path == kGeneral) {
        const dim3 grid((unsigned)(g.tiles_m * g.tiles_n));
        if (g.e8m0) hipLaunchKernelGGL((mm_general_kernel<RNS_T_E8M0, AT, WIDE>), grid, dim3(256), 0, s, g);
        else hipLaunchKernelGGL((mm_general_kernel<RNS_T_F32, AT, WIDE>), grid, dim3(256), 0, s, g);
        return;
    }
    const dim3 grid((unsigned)(g.tiles_m * g.tiles_n * g.split));
    if constexpr (!WIDE)
        if (p.path == kBig) {
            if (g.e8m0) hipLaunchKernelGGL((mm_big_kernel<AT, true>), grid, dim3(512), 0, s, g);
            else hipLaunchKernelGGL((mm_big_kernel<AT, false>), grid, dim3(512), 0, s, g);
            return;
        }
    if (p.path == kTile) launch_tile<128, 1, AT, WIDE>(grid, g, s);
    else if (p.path == kPair) launch_tile<64, 2, AT, WIDE>(grid, g, s);
    else launch_tile<64, 1, AT, WIDE>(grid, g, s);
    if (g.split > 1) {
        const int64_t blocks = div_up(g.partial_ld / 4 * g.M, 256);
        hipLaunchKernelGGL(mm_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, g);
    }
}

bool sizes_ok(int64_t M, int64_t N, int64_t K) {
    const int64_t top = RNS_SCALED_DIM_MAX - 1024;         // padded tiles stay inside int32
    return M >= 0 && N >= 0 && K >= 0 && M <= top && N <= top && K <= RNS_SCALED_LD_MAX;
}

}  // namespace

extern "C" {

int rns_scaled_workspace_size(int64_t M, int64_t N, int64_t K, const rns_scaled_t *a, const rns_scaled_t *b,
                              size_t *bytes) {
    if (!bytes || !sizes_ok(M, N, K) || !operand_ok(a, M, K) || !operand_ok(b, N, K)) return RNS_E_ARG;
    const size_t wide = plan_mm(M, N, K, a, b, true).bytes, half = plan_mm(M, N, K, a, b, false).bytes;
    *bytes = wide > half ? wide : half;                      // whatever the output's type
    return RNS_OK;
}

int rns_scaled_mm_nt(int64_t M, int64_t N, int64_t K, const rns_scaled_t *a, const rns_scaled_t *b, void *y,
                     int32_t y_type, int64_t ldy, void *ws, size_t ws_bytes, hipStream_t stream) {
    if (!sizes_ok(M, N, K) || !operand_ok(a, M, K) || !operand_ok(b, N, K)) return RNS_E_ARG;
    if (b->type != RNS_T_E4M3 || a->scale_type != b->scale_type) return RNS_E_ARG;
    if (y_type != RNS_T_F32 && y_type != RNS_T_BF16 && y_type != RNS_T_F16) return RNS_E_ARG;
    if (M == 0 || N == 0) return RNS_OK;
    if (!y || ldy < N || (uintptr_t)y % (y_type == RNS_T_F32 ? 4 : 2)) return RNS_E_ARG;
    if (K > 0 && (!a->values || !b->values || !a->scales || !b->scales)) return RNS_E_ARG;
    const bool wide = y_type == RNS_T_F32;
    const MmPlan p = plan_mm(M, N, K, a, b, wide);
    if (p.bytes > 0 && (!ws || (uintptr_t)ws % 16)) return RNS_E_ARG;
    if (ws_bytes < p.bytes) return RNS_E_WORKSPACE;
    const int tile = p.path == kBig ? 256 : p.path == kTile ? 128 : 64;
    MmArgs g{(const uint8_t *)a->values, (const uint8_t *)b->values, a->scales, b->scales, a->ld, b->ld,
             a->s_row, a->s_blk, b->s_row, b->s_blk, a->block_rows == 128 ? 7 : 0, b->block_rows == 128 ? 7 : 0,
             y, ldy, (int32_t)M, (int32_t)N, (int32_t)K, 0, 0, y_type, a->scale_type == RNS_T_E8M0,
             p.split, (float *)ws, p.partial_ld};
    if (div_up(M, tile) * div_up(N, tile) * p.split > 0x7fffffff) return RNS_E_ARG;
    g.tiles_m = (int32_t)div_up(M, tile);
    g.tiles_n = (int32_t)div_up(N, tile);
    if (a->type == RNS_T_E4M3) wide ? launch_mm<RNS_T_E4M3, true>(p, g, stream) : launch_mm<RNS_T_E4M3, false>(p, g, stream);
    else wide ? launch_mm<RNS_T_E5M2, true>(p, g, stream) : launch_mm<RNS_T_E5M2, false>(p, g, stream);
    return hipGetLastError() == hipSuccess ? RNS_OK : RNS_E_HIP;
}

}  // extern "C"
