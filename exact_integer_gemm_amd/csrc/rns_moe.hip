// A mixture-of-experts layer for a few tokens on block-scaled 8-bit weights.
// What it costs is the chosen experts' weights, read once: the kernels stream
// them and keep everything else (tokens, routing, activations) in cache.
#include "rns_scaled_device.h"

namespace rns {

constexpr int kMaxT = RNS_MOE_MAX_TOKENS, kMaxE = RNS_MOE_MAX_EXPERTS, kMaxTop = RNS_MOE_MAX_TOP_K;
constexpr int kMaxPairs = kMaxT * kMaxTop;
constexpr int kMaxParts = 4;

// What the first workgroup of the first product kernel leaves for the second:
// the experts that some token chose ("slots", ascending), where each one's
// tokens start in the list of all pairs, and the list.
struct MoeTable {
    int32_t active;
    int16_t expert[kMaxE];
    int16_t base[kMaxE + 1];
    uint8_t token[kMaxPairs];
};

struct MoeArgs {
    rns_moe_t a;
    float *logits;          // [parts][T][E]: sums over `parts` pieces of H
    MoeTable *table;
    uint16_t *act;          // [2][T * top_k][I] bfloat16, by pair: the activation's high and low parts
    int32_t parts;
    int32_t kbh, kbi;       // 128-wide blocks of H and of I
};

// Sixteen rows of an 8-bit weight times bfloat16 columns, over one 128-wide
// block: lane l holds row l % 16, bytes 32 (l / 16) .. + 31 of the block, and
// four matrix instructions take eight of them each, against the same eight
// entries of column l % 16.  Which entries meet in an instruction is a
// permutation of the block that both operands share.
struct WeightFrag {
    v4u lo, hi;             // 32 bytes
};
// The power of two in a block's scale goes into the weights: their products are as large as the results are, however
// large the tokens' entries.
__device__ __forceinline__ void widen(const WeightFrag &w, float power, v8bf (&o)[4]) {
    o[0] = widen8<RNS_T_E4M3>(w.lo[0], w.lo[1], power);
    o[1] = widen8<RNS_T_E4M3>(w.lo[2], w.lo[3], power);
    o[2] = widen8<RNS_T_E4M3>(w.hi[0], w.hi[1], power);
    o[3] = widen8<RNS_T_E4M3>(w.hi[2], w.hi[3], power);
}
template <int ST>
__device__ __forceinline__ Split split_weight(uint32_t s) {
    return split_scale<127 - 100, 127 + 100>(scale_factor<ST>(s));
}
// Bytes `at` .. at + 31 of a row of `len` bytes (a multiple of 16), and entries
// at .. at + 31 of a bfloat16 row of `len`.  What lies past the row's end is
// some other part of it, for the trim below to clear when the piece is used:
// a load into registers that were cleared first would wait for every load
// before it.
__device__ __forceinline__ WeightFrag load_weight(const uint8_t *row, int at, int len) {
    return WeightFrag{*(const v4u *)(row + min(at, len - 16)), *(const v4u *)(row + min(at + 16, len - 16))};
}
__device__ __forceinline__ void load_column(const uint16_t *row, int at, int len, v8bf (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i++) o[i] = *(const v8bf *)(row + min(at + 8 * i, len - 8));
}
__device__ __forceinline__ void trim(WeightFrag &w, int at, int len) {
    if (at >= len) w.lo = v4u{0, 0, 0, 0};
    if (at + 16 >= len) w.hi = v4u{0, 0, 0, 0};
}
__device__ __forceinline__ void trim(v8bf (&o)[4], int at, int len) {
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (at + 8 * i >= len) o[i] = v8bf{0, 0, 0, 0, 0, 0, 0, 0};
}
// Zero, by a way that the compiler cannot see through: an address with it in is a vector's, whose load is counted
// with the others instead of waited for on its own.
__device__ __forceinline__ int vector_zero() {
    int z = 0;
    asm volatile("" : "+v"(z));
    return z;
}

// ---- router ---------------------------------------------------------------------
// Partial logits: one workgroup for 16 experts, every token and one piece of
// H, its waves sharing the piece.  Products of bfloat16 numbers are exact in
// binary32; a binary32 router's are taken by fused multiply-adds.  A launch and
// one trip to memory bound it: 3 us for a token, 64 experts, H 2048 (256 KiB of
// router), 7 for 32 tokens, H 4096.
constexpr int kRouterWaves = 4;

template <int RT>
__global__ __launch_bounds__(kRouterWaves * 64) void moe_router_kernel(MoeArgs g) {
    __shared__ float part[kRouterWaves][kMaxT][17];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int l16 = lane & 15, quad = lane >> 4;
    const int T = g.a.T, E = g.a.E, H = g.a.H;
    const int tile = blockIdx.x / g.parts, piece = blockIdx.x - tile * g.parts;
    const int e0 = tile * 16;
    // pieces of whole runs of 32
    const int runs = (H + 31) >> 5, end = min(H, (runs * (piece + 1) / g.parts) * 32);
    const int begin = (runs * piece / g.parts) * 32;
    const uint16_t *x = (const uint16_t *)g.a.x;
    const int groups = (T + 15) >> 4;
    if constexpr (RT == RNS_T_BF16) {
        v4f acc[4];
#pragma unroll
        for (int t = 0; t < 4; t++) acc[t] = v4f{0, 0, 0, 0};
        const uint16_t *row = (const uint16_t *)g.a.router + (int64_t)min(e0 + l16, E - 1) * H;
        constexpr int U = 4;                               // steps whose loads are requested together
        for (int h0 = begin + wave * 32; h0 < end; h0 += U * kRouterWaves * 32) {
            v4u w[U], v[U][4];
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int h = h0 + u * kRouterWaves * 32 + quad * 8;
                w[u] = v4u{0, 0, 0, 0};
                if (h < end) w[u] = *(const v4u *)(row + h);
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    v[u][t] = v4u{0, 0, 0, 0};
                    if (t < groups && h < end && t * 16 + l16 < T)
                        v[u][t] = *(const v4u *)(x + (int64_t)(t * 16 + l16) * H + h);
                }
            }
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int t = 0; t < 4; t++)
                    if (t < groups)
                        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(v8bf, w[u]), __builtin_bit_cast(v8bf, v[u][t]), acc[t], 0, 0, 0);
        }
#pragma unroll
        for (int t = 0; t < 4; t++)
            if (t < groups)
#pragma unroll
                for (int i = 0; i < 4; i++) part[wave][t * 16 + l16][quad * 4 + i] = acc[t][i];
    } else {
        // lane (l16, quad) sums its share of expert e0 + l16
        const float *row = (const float *)g.a.router + (int64_t)min(e0 + l16, E - 1) * H;
        for (int t = 0; t < T; t++) {
            float s = 0.f;
            for (int h = begin + (wave * 4 + quad) * 4; h < end; h += kRouterWaves * 16) {
                const v4f w = *(const v4f *)(row + h);
                const v2u v = *(const v2u *)(x + (int64_t)t * H + h);
                s = __builtin_fmaf(w[0], bf16_float(v[0] & 0xffff), s);
                s = __builtin_fmaf(w[1], bf16_float(v[0] >> 16), s);
                s = __builtin_fmaf(w[2], bf16_float(v[1] & 0xffff), s);
                s = __builtin_fmaf(w[3], bf16_float(v[1] >> 16), s);
            }
            s += __shfl_xor(s, 16);
            s += __shfl_xor(s, 32);
            if (quad == 0) part[wave][t][l16] = s;
        }
    }
    __syncthreads();
    for (int i = tid; i < T * 16; i += kRouterWaves * 64) {
        const int t = i >> 4, e = e0 + (i & 15);
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kRouterWaves; w++) s += part[w][t][i & 15];
        if (e < E) g.logits[((int64_t)piece * T + t) * E + e] = s;
    }
}

// ---- routing ----------------------------------------------------------------------
// Every workgroup of the first product kernel works the routing out for itself
// from the logits, which costs it about two microseconds beside the weights'
// first bytes: a wave takes a token and finds its largest logits one after the
// other.
struct Routing {
    MoeTable t;
    uint64_t mask[kMaxE];           // tokens that chose the expert
    int16_t slot[kMaxE];
    uint8_t id[kMaxT][kMaxTop];
    float p[kMaxT][kMaxTop];
    float weight[kMaxPairs];        // by pair, as t.token
};

// A 32-bit key in the order of the floats, NaN below all, never 0.
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(f);
    if ((b & 0x7fffffffu) > 0x7f800000u) return 1;
    if ((b & 0x7fffffffu) == 0) return 0x80000000u;        // -0 and +0 are equal
    return b >> 31 ? ~b : b | 0x80000000u;
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {  // a lane without a source takes 0
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = dpp_max<0x111>(v);                                  // row_shr 1, 2, 4, 8: a row of 16's maximum in its last lane
    v = dpp_max<0x112>(v);
    v = dpp_max<0x114>(v);
    v = dpp_max<0x118>(v);
    v = dpp_max<0x142>(v);                                  // row_bcast 15, 31: the wave's in lane 63
    v = dpp_max<0x143>(v);
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The next token's logits are on their way while this one's are searched, and
// the pieces of a logit are requested together.
template <int NT>
__device__ __forceinline__ void build_routing(const MoeArgs &g, Routing &r) {
    constexpr int PER = kMaxE / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int T = g.a.T, E = g.a.E, top = g.a.top_k;
    for (int i = tid; i < kMaxE; i += NT) r.mask[i] = 0;
    __syncthreads();
    float next[PER];
    auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < PER; i++) {
            next[i] = 0.f;
            if (64 * i >= E || t >= T) continue;
            const float *at = g.logits + (int64_t)t * E + min(lane + 64 * i, E - 1);
            float piece[kMaxParts];
#pragma unroll
            for (int s = 0; s < kMaxParts; s++) piece[s] = at[(int64_t)min(s, g.parts - 1) * T * E];
#pragma unroll
            for (int s = 0; s < kMaxParts; s++) next[i] += s < g.parts ? piece[s] : 0.f;
        }
    };
    fetch(wave);
    for (int t = wave; t < T; t += NT / 64) {
        float l[PER];
        uint32_t key[PER];
#pragma unroll
        for (int i = 0; i < PER; i++) {
            l[i] = next[i];
            key[i] = lane + 64 * i < E ? order_key(l[i]) : 0;      // 0: no expert, or taken
        }
        fetch(t + NT / 64);
        float first = 0.f, mine = 0.f, total = 0.f;
        for (int j = 0; j < top; j++) {
            uint32_t m = key[0];
#pragma unroll
            for (int i = 1; i < PER; i++) m = max(m, key[i]);
            m = wave_max(m);
            int best = -1;
            float value = 0.f;
#pragma unroll
            for (int i = 0; i < PER; i++) {
                if (64 * i >= E) continue;
                const uint64_t at = __ballot(key[i] == m);
                if (best < 0 && at) {                      // uniform: the lowest index with the largest key
                    const int src = __ffsll((long long)at) - 1;
                    best = src + 64 * i;
                    value = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(l[i]), src));
                    if (lane == src) key[i] = 0;
                }
            }
            if (j == 0) first = value;
            const float p = expf(value - first);
            total += p;
            if (lane == j) mine = p;
            if (lane == 0) {
                r.id[t][j] = (uint8_t)best;
                atomicOr((unsigned long long *)&r.mask[best], 1ull << t);
            }
        }
        if (!g.a.renormalize) {
            total = 0.f;
#pragma unroll
            for (int i = 0; i < PER; i++)
                if (lane + 64 * i < E) total += expf(l[i] - first);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
        }
        if (lane < top) r.p[t][lane] = mine / total;
    }
    __syncthreads();
    if (wave == 0) {
        int n = 0, pairs = 0;
        for (int i = 0; i < PER && 64 * i < E; i++) {
            const int e = lane + 64 * i;
            const uint64_t mask = r.mask[e];
            const int count = __popcll(mask);
            int before = count;                            // pairs of the experts up to this one
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(before, d);
                if (lane >= d) before += o;
            }
            const uint64_t any = __ballot(mask != 0);
            if (mask) {
                const int slot = n + __popcll(any & ((1ull << lane) - 1));
                r.slot[e] = (int16_t)slot;
                r.t.expert[slot] = (int16_t)e;
                r.t.base[slot] = (int16_t)(pairs + before - count);
            }
            n += __popcll(any);
            pairs += __builtin_amdgcn_readlane(before, 63);
        }
        if (lane == 0) {
            r.t.active = n;
            r.t.base[n] = (int16_t)pairs;
        }
    }
    __syncthreads();
    for (int i = tid; i < T * top; i += NT) {
        const int t = i / top, j = i - t * top, e = r.id[t][j];
        const int at = r.t.base[r.slot[e]] + __popcll(r.mask[e] & ((1ull << t) - 1));
        r.t.token[at] = (uint8_t)t;
        r.weight[at] = r.p[t][j];
    }
    __syncthreads();
}

// ---- gate and up products, activation ------------------------------------------------
// An item is one active expert and 16 entries of I: 16 gate rows and the 16 up
// rows that go with them, times that expert's tokens in groups of 16.  The
// four waves share H, each fetching its next block while it works on this one;
// their partial sums meet in LDS.  The weights' bytes bound it: 1 token, 8 of 64
// experts, H 2048, I 1024: 12.6 us for 34 MB, of which a launch and the routing
// are 5; 32 tokens, 4 each, H 4096, I 1040: 105 us for 477 MB, 4.5 TB/s.
constexpr int kInWaves = 4, kInThreads = kInWaves * 64;

template <int ST>
__global__ __launch_bounds__(kInThreads) void moe_in_kernel(MoeArgs g) {
    __shared__ Routing r;
    __shared__ float part[kInWaves][2][4][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int H = g.a.H, I = g.a.I, T = g.a.T, top = g.a.top_k;
    const uint16_t *x = (const uint16_t *)g.a.x;
    build_routing<kInThreads>(g, r);
    if (blockIdx.x == 0) {
        for (int i = tid; i < T * top; i += kInThreads) {
            const int t = i / top, j = i - t * top;
            if (g.a.ids) g.a.ids[i] = r.id[t][j];
            if (g.a.probs) g.a.probs[i] = r.p[t][j];
        }
        for (int i = tid; i < (int)(sizeof(MoeTable) / 4); i += kInThreads)
            ((uint32_t *)g.table)[i] = ((const uint32_t *)&r.t)[i];
    }
    struct Fetched {
        WeightFrag gate, up;
        v8bf col[4];
        uint32_t sg, su;
    };
    const int tiles = (I + 15) >> 4, zero = vector_zero();
    for (int item = blockIdx.x; item < r.t.active * tiles; item += gridDim.x) {
        const int slot = item / tiles, i0 = (item - slot * tiles) * 16;
        const int64_t e = r.t.expert[slot];
        const int base = r.t.base[slot], count = r.t.base[slot + 1] - base;
        const uint8_t *gate = (const uint8_t *)g.a.w_in + (e * 2 * I + i0 + l16) * H;
        const uint8_t *up = gate + (int64_t)I * H;
        const int64_t sg = e * g.a.si[0] + (i0 >> 7) * g.a.si[2], su = sg + g.a.si[1];
        for (int t0 = 0; t0 < count; t0 += 16) {
            // a column without a token takes the group's first: its products go nowhere
            const bool on = t0 + l16 < count;
            const uint16_t *col = x + (int64_t)r.t.token[base + (on ? t0 + l16 : t0)] * H;
            auto fetch = [&](int kb, Fetched &f) {
                const int at = kb * 128 + quad * 32;
                f.gate = load_weight(gate, at, H);
                f.up = load_weight(up, at, H);
                load_column(col, at, H, f.col);
                f.sg = load_scale<ST>(g.a.w_in_scales, sg + kb * g.a.si[3] + zero);
                f.su = load_scale<ST>(g.a.w_in_scales, su + kb * g.a.si[3] + zero);
            };
            v4f ag{0, 0, 0, 0}, au{0, 0, 0, 0};
            auto work = [&](int kb, Fetched &f) {
                v8bf w[4];
                v4f pg{0, 0, 0, 0}, pu{0, 0, 0, 0};
                if ((kb + 1) * 128 > H) {
                    const int at = kb * 128 + quad * 32;
                    trim(f.gate, at, H);
                    trim(f.up, at, H);
                    trim(f.col, at, H);
                }
                const Split sg = split_weight<ST>(f.sg), su = split_weight<ST>(f.su);
                widen(f.gate, sg.power(), w);
#pragma unroll
                for (int i = 0; i < 4; i++) pg = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], f.col[i], pg, 0, 0, 0);
                widen(f.up, su.power(), w);
#pragma unroll
                for (int i = 0; i < 4; i++) pu = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], f.col[i], pu, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    ag[i] = __builtin_fmaf(pg[i], sg.r, ag[i]);
                    au[i] = __builtin_fmaf(pu[i], su.r, au[i]);
                }
            };
            Fetched f[2];
            int kb = wave;
            if (kb < g.kbh) fetch(kb, f[0]);
            if (kb + kInWaves < g.kbh) fetch(kb + kInWaves, f[1]);
            for (; kb < g.kbh; kb += 2 * kInWaves) {
                work(kb, f[0]);
                if (kb + 2 * kInWaves < g.kbh) fetch(kb + 2 * kInWaves, f[0]);
                if (kb + kInWaves < g.kbh) work(kb + kInWaves, f[1]);
                if (kb + 3 * kInWaves < g.kbh) fetch(kb + 3 * kInWaves, f[1]);
            }
#pragma unroll
            for (int i = 0; i < 4; i++) {
                part[wave][0][i][lane] = ag[i];
                part[wave][1][i][lane] = au[i];
            }
            __syncthreads();
            {
                // thread (i, lane): row 4 (lane / 16) + i of the tile, token lane % 16 of the group
                const int i = wave;
                float sgate = 0.f, sup = 0.f;
#pragma unroll
                for (int w = 0; w < kInWaves; w++) sgate += part[w][0][i][lane], sup += part[w][1][i][lane];
                if (on) {
                    const int pair = base + t0 + l16;
                    const float h = sgate / (1.f + expf(-sgate)) * sup * r.weight[pair];
                    const int64_t at = (int64_t)pair * I + i0 + quad * 4 + i;
                    const uint32_t hi = bf16_bits(h);
                    g.act[at] = (uint16_t)hi;
                    // an infinite high part is all of it
                    const float rest = fabsf(bf16_float(hi)) <= 3.4028235e38f ? h - bf16_float(hi) : 0.f;
                    g.act[(int64_t)T * top * I + at] = (uint16_t)bf16_bits(rest);
                }
            }
            __syncthreads();
        }
    }
}

// ---- down product and the sum over experts ---------------------------------------------
// A workgroup makes 16 entries of H for every token.  Block kb of I of expert
// e is wave (e + kb) % 8's, whatever else there is to do: the waves' shares
// are even, and the order of a token's sum depends on nothing but its own
// experts.  A wave fetches a few blocks ahead and adds each one's products to
// its own copy of the 16 entries in LDS; the copies are added in wave order.
// A token outside an expert has no part in its products.  1 token (as above):
// 11.7 us for 17 MB, a launch, the table and the first bytes' way 7 of them; 32
// tokens: 75 us for 238 MB, 3.2 TB/s.
constexpr int kOutWaves = 8, kOutThreads = kOutWaves * 64;
constexpr int kWeights = 4, kColumns = 2;                   // blocks fetched ahead: weights from memory, activations from L2

template <int ST>
__global__ __launch_bounds__(kOutThreads) void moe_out_kernel(MoeArgs g) {
    __shared__ MoeTable tab;
    __shared__ v4f sum[kOutWaves][kMaxT][4];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, quad = lane >> 4;
    const int H = g.a.H, I = g.a.I, T = g.a.T;
    for (int i = tid; i < (int)(sizeof(MoeTable) / 4); i += kOutThreads)
        ((uint32_t *)&tab)[i] = ((const uint32_t *)g.table)[i];
    for (int i = tid; i < kOutWaves * kMaxT * 4; i += kOutThreads) (&sum[0][0][0])[i] = v4f{0, 0, 0, 0};
    __syncthreads();
    const int h0 = blockIdx.x * 16;
    const int64_t low = (int64_t)T * g.a.top_k * I;
    const int zero = vector_zero();
    const int active = __builtin_amdgcn_readfirstlane(tab.active);
    // Lane i holds slot chunk + i's expert and where its pairs begin and end: a lane is read in a few cycles, LDS in a
    // hundred.
    int chunk = 0, in_chunk = 0, of_expert = 0, of_base = 0, of_end = 0;
    struct Place {
        int slot, kb, e;                                     // slot within the chunk
    };
    auto advance = [&](Place &p) {                           // to this wave's next block; there has to be one
        p.kb += kOutWaves;
        while (p.kb >= g.kbi && p.slot + 1 < in_chunk) {
            p.e = __builtin_amdgcn_readlane(of_expert, ++p.slot);
            p.kb = (wave - p.e) & (kOutWaves - 1);
        }
    };
    struct Weights {
        WeightFrag w;
        uint32_t s;
    };
    struct Columns {
        v8bf hi[4], lo[4];
        int token;                                           // of this lane's column, or -1
    };
    const uint8_t *rows = (const uint8_t *)g.a.w_out + (int64_t)h0 * I;
    const int64_t scales0 = (h0 >> 7) * g.a.so[1];
    auto fetch_weights = [&](const Place &p, Weights &f) {
        f.w = load_weight(rows + (int64_t)p.e * H * I + l16 * I, p.kb * 128 + quad * 32, I);
        f.s = load_scale<ST>(g.a.w_out_scales, p.e * g.a.so[0] + scales0 + p.kb * g.a.so[2] + zero);
    };
    auto fetch_columns = [&](const Place &p, int t0, Columns &f) {
        // a column without a token takes the group's first: its products go nowhere
        const int first = __builtin_amdgcn_readlane(of_base, p.slot) + t0, at = p.kb * 128 + quad * 32;
        const bool on = first + l16 < __builtin_amdgcn_readlane(of_end, p.slot);
        const int pair = on ? first + l16 : first;
        f.token = on ? tab.token[pair] : -1;
        const uint16_t *col = g.act + (int64_t)pair * I;
        load_column(col, at, I, f.hi);
        load_column(col + low, at, I, f.lo);
    };
    auto work = [&](const Place &p, Weights &f, Columns &c) {
        const int at = p.kb * 128 + quad * 32;
        const bool tail = (p.kb + 1) * 128 > I;
        v8bf w[4];
        if (tail) trim(f.w, at, I);
        const Split scale = split_weight<ST>(f.s);
        widen(f.w, scale.power(), w);
        const int base = __builtin_amdgcn_readlane(of_base, p.slot), end = __builtin_amdgcn_readlane(of_end, p.slot);
        for (int t0 = 0; base + t0 < end; t0 += 16) {        // more than 16 tokens: the others with the weights at hand
            if (t0 > 0) fetch_columns(p, t0, c);
            if (tail) {
                trim(c.hi, at, I);
                trim(c.lo, at, I);
            }
            v4f o{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], c.lo[i], o, 0, 0, 0);
                o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], c.hi[i], o, 0, 0, 0);
            }
            if (c.token >= 0) {
                v4f &to = sum[wave][c.token][quad];
                v4f s = to;
#pragma unroll
                for (int i = 0; i < 4; i++) s[i] = __builtin_fmaf(o[i], scale.r, s[i]);
                to = s;
            }
        }
    };
    for (; chunk < active; chunk += 64) {
        in_chunk = min(64, active - chunk);
        const int mine = min(chunk + lane, active - 1);
        of_expert = tab.expert[mine];
        of_base = tab.base[mine];
        of_end = tab.base[mine + 1];
        Weights w[kWeights];
        Columns c[kColumns];
        // this wave's blocks in the chunk
        int n = 0;
        if (chunk + lane < active) {
            const int kb = (wave - of_expert) & (kOutWaves - 1);
            n = kb < g.kbi ? (g.kbi - 1 - kb) / kOutWaves + 1 : 0;
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
        n = __builtin_amdgcn_readfirstlane(n);
        const int e = __builtin_amdgcn_readlane(of_expert, 0);
        Place at{0, ((wave - e) & (kOutWaves - 1)) - kOutWaves, e};
        advance(at);
        Place next_w = at, next_c = at;
#pragma unroll
        for (int i = 0; i < kWeights; i++)
            if (i < n) {
                if (i) advance(next_w);
                fetch_weights(next_w, w[i]);
            }
#pragma unroll
        for (int i = 0; i < kColumns; i++)
            if (i < n) {
                if (i) advance(next_c);
                fetch_columns(next_c, 0, c[i]);
            }
        // While everything that is fetched ahead is there, without a branch: a load that may not have been issued would
        // have to be waited for as if it had not.
        int k = 0;
        for (; k + 2 * kWeights <= n; k += kWeights)
#pragma unroll
            for (int i = 0; i < kWeights; i++) {
                work(at, w[i], c[i % kColumns]);
                advance(at);
                advance(next_w);
                fetch_weights(next_w, w[i]);
                advance(next_c);
                fetch_columns(next_c, 0, c[i % kColumns]);
            }
        for (; k < n; k += kWeights)
#pragma unroll
            for (int i = 0; i < kWeights; i++) {
                if (k + i >= n) break;
                work(at, w[i], c[i % kColumns]);
                advance(at);
                if (k + i + kWeights < n) {
                    advance(next_w);
                    fetch_weights(next_w, w[i]);
                }
                if (k + i + kColumns < n) {
                    advance(next_c);
                    fetch_columns(next_c, 0, c[i % kColumns]);
                }
            }
    }
    __syncthreads();
    for (int i = tid; i < T * 4; i += kOutThreads) {
        const int t = i >> 2, q = i & 3;
        v4f s = sum[0][t][q];
#pragma unroll
        for (int w = 1; w < kOutWaves; w++) s += sum[w][t][q];
        *(v2u *)((uint16_t *)g.a.y + (int64_t)t * H + h0 + q * 4) =
            v2u{bf16_bits(s[0]) | bf16_bits(s[1]) << 16, bf16_bits(s[2]) | bf16_bits(s[3]) << 16};
    }
}

}  // namespace rns

using namespace rns;

namespace {

bool moe_shape_ok(int64_t T, int64_t E, int64_t H, int64_t I, int64_t top_k) {
    return T >= 0 && T <= RNS_MOE_MAX_TOKENS && E >= 1 && E <= RNS_MOE_MAX_EXPERTS && top_k >= 1 &&
           top_k <= RNS_MOE_MAX_TOP_K && top_k <= E && H >= 16 && H % 16 == 0 && I >= 16 && I % 16 == 0 &&
           H <= (1 << 20) && I <= (1 << 20);
}

// Pieces of H for the router, each of at least 256, at most four: each piece's logits are read back by every workgroup of
// the next kernel.
int router_parts(int64_t H) {
    const int64_t most = H / 256 < 1 ? 1 : H / 256;
    return (int)(most < kMaxParts ? most : kMaxParts);
}

int64_t logits_bytes(int64_t T, int64_t E, int64_t H) { return div_up(router_parts(H) * T * E * 4, 256) * 256; }
constexpr int64_t kTableBytes = (sizeof(MoeTable) + 255) / 256 * 256;

}  // namespace

extern "C" {

int rns_moe_workspace_size(int32_t T, int32_t E, int32_t H, int32_t I, int32_t top_k, size_t *bytes) {
    if (!bytes || !moe_shape_ok(T, E, H, I, top_k)) return RNS_E_ARG;
    *bytes = (size_t)(logits_bytes(T, E, H) + kTableBytes + (int64_t)2 * T * top_k * I * 2);
    return RNS_OK;
}

int rns_moe_layer(const rns_moe_t *args, void *ws, size_t ws_bytes, hipStream_t stream) {
    if (!args) return RNS_E_ARG;
    const rns_moe_t &a = *args;
    size_t need = 0;
    if (rns_moe_workspace_size(a.T, a.E, a.H, a.I, a.top_k, &need) != RNS_OK) return RNS_E_ARG;
    if (a.router_type != RNS_T_BF16 && a.router_type != RNS_T_F32) return RNS_E_ARG;
    if (a.scale_type != RNS_T_F32 && a.scale_type != RNS_T_E8M0) return RNS_E_ARG;
    for (int i = 0; i < 4; i++)
        if (a.si[i] < 0 || (i < 3 && a.so[i] < 0)) return RNS_E_ARG;
    if (a.T == 0) return RNS_OK;
    if (!a.x || !a.router || !a.w_in || !a.w_in_scales || !a.w_out || !a.w_out_scales || !a.y || !ws) return RNS_E_ARG;
    if (a.scale_type == RNS_T_F32 && ((uintptr_t)a.w_in_scales | (uintptr_t)a.w_out_scales) % 4) return RNS_E_ARG;
    if (((uintptr_t)a.ids | (uintptr_t)a.probs) % 4) return RNS_E_ARG;
    if (((uintptr_t)a.x | (uintptr_t)a.router | (uintptr_t)a.w_in | (uintptr_t)a.w_out | (uintptr_t)a.y) % 16 ||
        (uintptr_t)ws % 256)
        return RNS_E_ARG;
    if (ws_bytes < need) return RNS_E_WORKSPACE;
    uint8_t *w = (uint8_t *)ws;
    const int64_t lb = logits_bytes(a.T, a.E, a.H);
    MoeArgs g{a, (float *)w, (MoeTable *)(w + lb), (uint16_t *)(w + lb + kTableBytes), router_parts(a.H),
              (int32_t)div_up(a.H, 128), (int32_t)div_up(a.I, 128)};
    const unsigned router_grid = (unsigned)(div_up(a.E, 16) * g.parts);
    if (a.router_type == RNS_T_BF16)
        hipLaunchKernelGGL((moe_router_kernel<RNS_T_BF16>), dim3(router_grid), dim3(kRouterWaves * 64), 0, stream, g);
    else
        hipLaunchKernelGGL((moe_router_kernel<RNS_T_F32>), dim3(router_grid), dim3(kRouterWaves * 64), 0, stream, g);
    // as many workgroups as stay resident, each with several items where there are more
    const int64_t items = (int64_t)(a.T * a.top_k < a.E ? a.T * a.top_k : a.E) * div_up(a.I, 16);
    // At most two workgroups to a compute unit, which go on to further items: each works out the routing for itself.  32
    // tokens of 64 experts, H 4096, I 1040, the layer's GPU time: 182 us; at most 256 workgroups 206, 1024 191, 4096 266.
    const dim3 in_grid((unsigned)(items < 512 ? items : 512)), out_grid((unsigned)(a.H / 16));
    if (a.scale_type == RNS_T_F32) {
        hipLaunchKernelGGL((moe_in_kernel<RNS_T_F32>), in_grid, dim3(kInThreads), 0, stream, g);
        hipLaunchKernelGGL((moe_out_kernel<RNS_T_F32>), out_grid, dim3(kOutThreads), 0, stream, g);
    } else {
        hipLaunchKernelGGL((moe_in_kernel<RNS_T_E8M0>), in_grid, dim3(kInThreads), 0, stream, g);
        hipLaunchKernelGGL((moe_out_kernel<RNS_T_E8M0>), out_grid, dim3(kOutThreads), 0, stream, g);
    }
    return hipGetLastError() == hipSuccess ? RNS_OK : RNS_E_HIP;
}

}  // extern "C"
