// The block quantiser: 8-bit floating-point values with one scale for each
// block of 128 columns (of one row, or of 128 rows), of a matrix and, from the
// same read, of its transpose.  Both kernels are bound by the bytes they move:
// each entry is read once and kept in registers between the search for its
// block's largest magnitude and its rounding.
#include "rns_scaled_device.h"

namespace rns {

struct QuantArgs {
    const void *x;
    int64_t ldx, R, C;
    uint8_t *q, *qt;
    int64_t ldq, ldqt;
    void *s, *st;
    int64_t s_ld, st_ld;
    int32_t nblk;          // column blocks
    int32_t log_cols;      // row kernel: log2 of the column blocks a workgroup covers
    int32_t col_groups;    // row kernel: groups of that many column blocks
};

constexpr float kLargestFloat = 3.4028235e38f;

// ---- the rule -----------------------------------------------------------------
// Both types' largest values are 1.75 * 2^top (top 8 or 15).
template <bool E5M2>
struct Format {
    static constexpr float largest = E5M2 ? 57344.f : 448.f;
    static constexpr int top = E5M2 ? 15 : 8;
    static constexpr float small_scale = E5M2 ? 0x1p-86f : 0x1p-93f;    // see `quotient`
};

// A block's scale: the binary32 number, or the biased exponent; and what its
// entries are multiplied by (the exponent's power of two is exact, so that is
// the quotient; otherwise fl(1 / s)).
struct Scale {
    float s, r;
    uint32_t e;
};

// x over s, correctly rounded, without the divider's full sequence: with r =
// fl(1 / s), one correction by the exact remainder brings x r to within one
// unit in the last place, and from such a value the next gives the rounded
// quotient, as long as the remainders are exact: their last bit is that of q
// times that of s, which has to be 2^-149 or more.  The smallest q whose
// rounding matters is half the type's smallest step, 2^-10 for E4M3 and 2^-17
// for E5M2, with last bits 2^-33 and 2^-40; so s has to be at least 2^-93 or
// 2^-86, whose last bits are 2^-116 and 2^-109.  (Smaller q all become zero.)
__device__ __forceinline__ float quotient(float x, float s, float r) {
    float q = x * r;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
    return __builtin_fmaf(__builtin_fmaf(-q, s, x), r, q);
}

// The smallest 2^e with amax <= 1.75 * 2^(top + e): e = exponent(amax) - top,
// one more where amax's mantissa exceeds 1.75 (then adding 2^21 - 1 to its
// bits carries into the exponent), at least -127.
template <bool E8M0, bool E5M2>
__device__ __forceinline__ Scale block_scale(float amax) {
    Scale b{1.f, 1.f, 127};
    if (amax > 0.f) {
        if constexpr (E8M0) {
            const int e = (int)((__float_as_uint(amax) + 0x1fffffu) >> 23) - Format<E5M2>::top;
            b.e = (uint32_t)max(e, 0);
            b.r = __uint_as_float((254 - b.e) << 23);
        } else {
            b.s = fmaxf(amax / Format<E5M2>::largest, 1.17549435e-38f);
            b.r = 1.f / b.s;
        }
    }
    return b;
}

// Four quotients to four bytes.  The largest rounds to at most the type's
// largest value, so nothing finite overflows; the conversion gives an infinity
// as NaN in E4M3.
template <bool E5M2>
__device__ __forceinline__ uint32_t pack4_8(float a, float b, float c, float d) {
    if constexpr (E5M2)
        return (uint32_t)__builtin_amdgcn_cvt_pk_bf8_f32(c, d, __builtin_amdgcn_cvt_pk_bf8_f32(a, b, 0, false), true);
    else
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}
template <bool E8M0, bool E5M2>
__device__ __forceinline__ v2u pack8(const float (&v)[8], float s, float r) {
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; i++) y[i] = E8M0 ? v[i] * r : quotient(v[i], s, r);
    return v2u{pack4_8<E5M2>(y[0], y[1], y[2], y[3]), pack4_8<E5M2>(y[4], y[5], y[6], y[7])};
}

template <bool E8M0>
__device__ __forceinline__ void store_scale(void *s, int64_t i, const Scale &b) {
    if constexpr (E8M0) ((uint8_t *)s)[i] = (uint8_t)b.e;
    else ((float *)s)[i] = b.s;
}

// ---- entries ----------------------------------------------------------------------
// Sixteen bytes at any entry: a global load takes every alignment, a misaligned one a little slower.
typedef v4u v4u_any __attribute__((aligned(2)));
typedef v4f v4f_any __attribute__((aligned(4)));

template <int XT>
__device__ __forceinline__ float entry(const void *x, int64_t i) {
    if constexpr (XT == RNS_T_F32) return ((const float *)x)[i];
    else if constexpr (XT == RNS_T_BF16) return bf16_float(((const uint16_t *)x)[i]);
    else return f16_float(((const uint16_t *)x)[i]);
}

// Entries c .. c + 7 of a row of C >= 8 entries, zero past its end: where the
// row ends inside them, its last eight moved down.
template <int XT>
__device__ __forceinline__ void load8(const void *row, int64_t c, int64_t C, float (&v)[8]) {
    const int64_t at = min(c, C - 8);
    const int gone = (int)min(c - at, (int64_t)8);
    if constexpr (XT == RNS_T_F32) {
        const v4f a = *(const v4f_any *)((const float *)row + at), b = *(const v4f_any *)((const float *)row + at + 4);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = a[i], v[4 + i] = b[i];
        if (gone) {
#pragma unroll
            for (int step = 8; step; step >>= 1)
                if (gone & step)
#pragma unroll
                    for (int i = 0; i < 8; i++) v[i] = i + step < 8 ? v[i + step < 8 ? i + step : 0] : 0.f;
        }
    } else {
        v4u w = *(const v4u_any *)((const uint16_t *)row + at);
        if (gone) {
            uint64_t lo = w[0] | (uint64_t)w[1] << 32, hi = w[2] | (uint64_t)w[3] << 32;
            const int sh = 16 * (gone & 3);
            if (gone & 8) lo = hi = 0;
            if (gone & 4) lo = hi, hi = 0;
            if (sh) lo = lo >> sh | hi << (64 - sh), hi >>= sh;
            w = v4u{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
        }
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = XT == RNS_T_BF16 ? bf16_float(w[i] & 0xffff) : f16_float(w[i] & 0xffff);
            v[2 * i + 1] = XT == RNS_T_BF16 ? bf16_float(w[i] >> 16) : f16_float(w[i] >> 16);
        }
    }
}

// The larger of m and |x|: a NaN x leaves m, an infinite one makes it infinite, which the callers look for.
__device__ __forceinline__ float grow(float m, float x) { return fmaxf(m, fabsf(x)); }

// ---- any entries at all -------------------------------------------------------------
// One block (rows x 128 columns of x, or of its transpose) by one workgroup,
// entry by entry from memory and with the divider: blocks with infinities,
// with very small scales, and matrices of fewer than eight columns.  Short
// code, seldom run.
template <int XT, bool E8M0, bool E5M2>
__device__ __forceinline__ void quantize_slowly(const QuantArgs &g, int64_t r0, int64_t c0, bool square, bool transposed) {
    __shared__ float all;
    const int64_t R = transposed ? g.C : g.R, C = transposed ? g.R : g.C;
    uint8_t *q = transposed ? g.qt : g.q;
    const int64_t ldq = transposed ? g.ldqt : g.ldq, s_ld = transposed ? g.st_ld : g.s_ld;
    const auto at = [&](int64_t r, int64_t c) { return transposed ? c * g.ldx + r : r * g.ldx + c; };
    const int t = threadIdx.x;                               // 256 threads; row r0 + t for t < 128
    const int64_t r = r0 + t;
    const int n = (int)min((int64_t)128, C - c0);
    if (t == 0) all = 0.f;
    __syncthreads();
    float m = 0.f;
    if (t < 128 && r < R)
#pragma unroll 1
        for (int c = 0; c < n; c++) {
            const float a = fabsf(entry<XT>(g.x, at(r, c0 + c)));
            if (a <= kLargestFloat) m = fmaxf(m, a);
        }
    if (square) {
        // maxima of non-negative floats: their bits are in the same order
        if (m > 0.f) atomicMax((unsigned *)&all, __float_as_uint(m));
        __syncthreads();
        m = all;
    }
    if (t < 128 && r < R) {
        const Scale b = block_scale<E8M0, E5M2>(m);
#pragma unroll 1
        for (int c = 0; c < 128; c++) {
            const float x = c < n ? entry<XT>(g.x, at(r, c0 + c)) : 0.f;
            q[r * ldq + c0 + c] = (uint8_t)pack4_8<E5M2>(E8M0 ? x * b.r : x / b.s, 0.f, 0.f, 0.f);
        }
        const int64_t row = square ? r0 / 128 : r;
        if (!square || t == 0) store_scale<E8M0>(transposed ? g.st : g.s, c0 / 128 * s_ld + row, b);
    }
    __syncthreads();
}

template <int XT, bool E8M0, bool E5M2>
__global__ __launch_bounds__(256) void quantize_any_kernel(QuantArgs g, int square, int both) {
    const int64_t rb = blockIdx.x / (uint32_t)g.nblk;
    const int blk = (int)(blockIdx.x - rb * g.nblk);
    quantize_slowly<XT, E8M0, E5M2>(g, rb * 128, (int64_t)blk * 128, square, false);
    if (both) quantize_slowly<XT, E8M0, E5M2>(g, (int64_t)blk * 128, rb * 128, square, true);
}

// ---- row blocks of one orientation --------------------------------------------
// Sixteen lanes take one block, eight entries each; a workgroup takes 2^log_cols
// neighbouring column blocks of 16 >> log_cols rows.  16 x 2048 bfloat16: 2.6 us,
// a launch and one trip to memory.
template <int XT, bool E8M0, bool E5M2>
__global__ __launch_bounds__(256) void quantize_rows_kernel(QuantArgs g) {
    const int group = threadIdx.x >> 4, l16 = threadIdx.x & 15;
    const int64_t rg = blockIdx.x / (uint32_t)g.col_groups;
    const int cg = (int)(blockIdx.x - rg * g.col_groups);
    const int blk = (cg << g.log_cols) + (group & ((1 << g.log_cols) - 1));
    const int64_t row = rg * (16 >> g.log_cols) + (group >> g.log_cols);
    if (blk >= g.nblk || row >= g.R) return;
    const int64_t c = (int64_t)blk * RNS_SCALE_BLOCK + l16 * 8;
    const void *x = (const uint8_t *)g.x + row * g.ldx * (XT == RNS_T_F32 ? 4 : 2);
    float v[8];
    load8<XT>(x, c, g.C, v);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = grow(m, v[i]);
    m = row_max(m);
    const bool infinite = !(m <= kLargestFloat);
    if (infinite) {                                          // all sixteen lanes of the block
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (fabsf(v[i]) <= kLargestFloat) m = grow(m, v[i]);
        m = row_max(m);
    }
    const Scale b = block_scale<E8M0, E5M2>(m);
    v2u w;
    if (!E8M0 && (infinite || b.s < Format<E5M2>::small_scale)) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = v[i] / b.s;
        w = v2u{pack4_8<E5M2>(y[0], y[1], y[2], y[3]), pack4_8<E5M2>(y[4], y[5], y[6], y[7])};
    } else {
        w = pack8<E8M0, E5M2>(v, b.s, b.r);
    }
    *(v2u *)(g.q + row * g.ldq + c) = w;
    if (l16 == 0) store_scale<E8M0>(g.s, (int64_t)blk * g.s_ld + row, b);
}

// ---- 128 x 128 tiles: square blocks, and both orientations ----------------------
// A thread holds an 8 x 8 patch: rows 8 (tid / 16) .., columns 8 (tid % 16) ...
// Row maxima are taken over 16 lanes, column maxima through LDS over the 16
// patches below one another; then each of the 256 threads works out one row's
// or one column's scale, which the others read back.  8192 x 4096 bfloat16 both
// ways: 27 us, 134 MB at 4.9 TB/s, a copy's rate; 3001 x 4097 binary32, square
// blocks, both ways: 18 us, 4.2 TB/s with rows off every boundary.  A patch of
// eight rows makes every store of the transpose eight neighbouring bytes.
template <int XT, bool SQUARE, bool BOTH, bool E8M0, bool E5M2>
__global__ __launch_bounds__(256) void quantize_tile_kernel(QuantArgs g) {
    __shared__ float part[16][128];                          // column maxima of each row of patches; or of the waves
    __shared__ float rmax[128];
    __shared__ float div[256], mul[256];                     // scales and multipliers: rows, then columns
    const int tid = threadIdx.x, l16 = tid & 15, rg = tid >> 4;
    const int64_t rb = blockIdx.x / (uint32_t)g.nblk;
    const int blk = (int)(blockIdx.x - rb * g.nblk);
    const int64_t r0 = rb * 128 + rg * 8, c0 = (int64_t)blk * 128 + l16 * 8;
    const int rows = (int)min((int64_t)8, g.R - r0);         // of this patch; none or fewer in the last tile
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; i++)
        load8<XT>((const uint8_t *)g.x + min(r0 + i, g.R - 1) * g.ldx * (XT == RNS_T_F32 ? 4 : 2), c0, g.C, v[i]);
    if (rows < 8)
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (i >= rows)
#pragma unroll
                for (int j = 0; j < 8; j++) v[i][j] = 0.f;

    Scale mine;
    if constexpr (SQUARE) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 8; j++) m = grow(m, v[i][j]);
        m = row_max(m);
        if (l16 == 0) rmax[rg] = m;
        __syncthreads();
        m = row_max(rmax[l16]);
        mine = block_scale<E8M0, E5M2>(m);
        if (!(m <= kLargestFloat) || (!E8M0 && mine.s < Format<E5M2>::small_scale)) {     // the same in every thread
            quantize_slowly<XT, E8M0, E5M2>(g, rb * 128, (int64_t)blk * 128, true, false);
            if (BOTH) quantize_slowly<XT, E8M0, E5M2>(g, (int64_t)blk * 128, rb * 128, true, true);
            return;
        }
        if (tid == 0) {
            store_scale<E8M0>(g.s, (int64_t)blk * g.s_ld + rb, mine);
            if (BOTH) store_scale<E8M0>(g.st, rb * g.st_ld + blk, mine);
        }
    } else {
        float cm[8];
#pragma unroll
        for (int j = 0; j < 8; j++) cm[j] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                m = grow(m, v[i][j]);
                cm[j] = grow(cm[j], v[i][j]);
            }
            m = row_max(m);
            if (l16 == 0) rmax[rg * 8 + i] = m;
        }
#pragma unroll
        for (int j = 0; j < 8; j += 4) *(v4f *)&part[rg][l16 * 8 + j] = v4f{cm[j], cm[j + 1], cm[j + 2], cm[j + 3]};
        __syncthreads();
        float m;
        const int k = tid & 127;
        if (tid < 128) {
            m = rmax[k];
        } else {
            m = part[0][k];
#pragma unroll
            for (int i = 1; i < 16; i++) m = fmaxf(m, part[i][k]);
        }
        mine = block_scale<E8M0, E5M2>(m);
        div[tid] = mine.s;
        mul[tid] = mine.r;
        const bool bad = !(m <= kLargestFloat) || (!E8M0 && mine.s < Format<E5M2>::small_scale);
        if (__syncthreads_or(bad)) {
            quantize_slowly<XT, E8M0, E5M2>(g, rb * 128, (int64_t)blk * 128, false, false);
            quantize_slowly<XT, E8M0, E5M2>(g, (int64_t)blk * 128, rb * 128, false, true);
            return;
        }
        if (tid < 128) {
            if (rb * 128 + k < g.R) store_scale<E8M0>(g.s, (int64_t)blk * g.s_ld + rb * 128 + k, mine);
        } else {
            if ((int64_t)blk * 128 + k < g.C) store_scale<E8M0>(g.st, rb * g.st_ld + (int64_t)blk * 128 + k, mine);
        }
    }
    uint8_t *to = g.q + r0 * g.ldq + c0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int k = rg * 8 + i;
        if (i < rows)
            *(v2u *)(to + i * g.ldq) = SQUARE ? pack8<E8M0, E5M2>(v[i], mine.s, mine.r)
                                              : pack8<E8M0, E5M2>(v[i], E8M0 ? 1.f : div[k], mul[k]);
    }
    if constexpr (BOTH) {
        uint8_t *tt = g.qt + c0 * g.ldqt + r0;
        const int cols = (int)min((int64_t)8, g.C - c0);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int k = 128 + l16 * 8 + j;
            float col[8];
#pragma unroll
            for (int i = 0; i < 8; i++) col[i] = v[i][j];
            if (j < cols)
                *(v2u *)(tt + j * g.ldqt) = SQUARE ? pack8<E8M0, E5M2>(col, mine.s, mine.r)
                                                   : pack8<E8M0, E5M2>(col, E8M0 ? 1.f : div[k], mul[k]);
        }
    }
}

}  // namespace rns

using namespace rns;

namespace {

template <int XT, bool E8M0, bool E5M2>
void launch_quantize(const QuantArgs &g, bool square, bool both, unsigned grid, hipStream_t s) {
    if (g.C < 8)
        hipLaunchKernelGGL((quantize_any_kernel<XT, E8M0, E5M2>), dim3(grid), dim3(256), 0, s, g, (int)square, (int)both);
    else if (!square && !both)
        hipLaunchKernelGGL((quantize_rows_kernel<XT, E8M0, E5M2>), dim3(grid), dim3(256), 0, s, g);
    else if (!square)
        hipLaunchKernelGGL((quantize_tile_kernel<XT, false, true, E8M0, E5M2>), dim3(grid), dim3(256), 0, s, g);
    else if (both)
        hipLaunchKernelGGL((quantize_tile_kernel<XT, true, true, E8M0, E5M2>), dim3(grid), dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL((quantize_tile_kernel<XT, true, false, E8M0, E5M2>), dim3(grid), dim3(256), 0, s, g);
}

template <int XT>
void launch_quantize(const QuantArgs &g, bool square, bool both, bool e8m0, bool e5m2, unsigned grid, hipStream_t s) {
    if (e8m0) e5m2 ? launch_quantize<XT, true, true>(g, square, both, grid, s)
                   : launch_quantize<XT, true, false>(g, square, both, grid, s);
    else e5m2 ? launch_quantize<XT, false, true>(g, square, both, grid, s)
              : launch_quantize<XT, false, false>(g, square, both, grid, s);
}

}  // namespace

extern "C" int rns_block_quantize(int64_t R, int64_t C, const void *x, int32_t x_type, int64_t ldx, int32_t type,
                                  int32_t block_rows, int32_t scale_type, void *q, int64_t ldq, void *s, int64_t s_ld,
                                  void *qt, int64_t ldqt, void *st, int64_t st_ld, hipStream_t stream) {
    if (R < 0 || C < 0 || R > RNS_SCALED_DIM_MAX || C > RNS_SCALED_DIM_MAX) return RNS_E_ARG;
    if (x_type != RNS_T_F32 && x_type != RNS_T_BF16 && x_type != RNS_T_F16) return RNS_E_ARG;
    if (type != RNS_T_E4M3 && type != RNS_T_E5M2) return RNS_E_ARG;
    if (scale_type != RNS_T_F32 && scale_type != RNS_T_E8M0) return RNS_E_ARG;
    if (block_rows != 1 && block_rows != 128) return RNS_E_ARG;
    if (R == 0 || C == 0) return RNS_OK;
    if (!x || !q || !s || (qt == nullptr) != (st == nullptr)) return RNS_E_ARG;
    const bool square = block_rows == 128, both = qt != nullptr;
    const int64_t nblk = div_up(C, 128), rblk = div_up(R, 128);
    if (ldx < C || ldq < C || ldq % 128 || s_ld < (square ? rblk : R)) return RNS_E_ARG;
    if (both && (ldqt < R || ldqt % 128 || st_ld < (square ? nblk : C))) return RNS_E_ARG;
    if ((uintptr_t)q % 8 || (uintptr_t)qt % 8) return RNS_E_ARG;
    const int es = x_type == RNS_T_F32 ? 4 : 2;
    if ((uintptr_t)x % es || (scale_type == RNS_T_F32 && ((uintptr_t)s % 4 || (uintptr_t)st % 4))) return RNS_E_ARG;
    QuantArgs g{x, ldx, R, C, (uint8_t *)q, (uint8_t *)qt, ldq, ldqt, s, st, s_ld, st_ld, (int32_t)nblk,
                0, 1};
    int64_t grid = rblk * nblk;
    if (!square && !both && C >= 8) {
        while (g.log_cols < 4 && (1 << g.log_cols) < nblk) g.log_cols++;
        g.col_groups = (int32_t)div_up(nblk, 1 << g.log_cols);
        grid = div_up(R, 16 >> g.log_cols) * g.col_groups;
    }
    if (grid > 0x7fffffff) return RNS_E_ARG;
    const bool e8m0 = scale_type == RNS_T_E8M0, e5m2 = type == RNS_T_E5M2;
    if (x_type == RNS_T_F32) launch_quantize<RNS_T_F32>(g, square, both, e8m0, e5m2, (unsigned)grid, stream);
    else if (x_type == RNS_T_BF16) launch_quantize<RNS_T_BF16>(g, square, both, e8m0, e5m2, (unsigned)grid, stream);
    else launch_quantize<RNS_T_F16>(g, square, both, e8m0, e5m2, (unsigned)grid, stream);
    return hipGetLastError() == hipSuccess ? RNS_OK : RNS_E_HIP;
}
