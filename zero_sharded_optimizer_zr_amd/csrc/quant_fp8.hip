// Block quantization of a 16-bit matrix to e4m3 or e5m2 codes with E8M0 scales,
// along rows, along columns (the transposed copy) or in 128 x 128 blocks (gfx950).
//
// For a group with largest magnitude amax the scale is the smallest power of
// two 2^e with amax <= MAX * 2^e and the code is RNE(x * 2^-e).  The product is
// exact, so a code is rounded once, and the exponent comes from amax's bits
// (scale_byte), so codes and scales are exact functions of the input.
//
// Bound by HBM: 2 bytes read and 1 or 2 written per element.  Sources are read once,
// so their loads pass the caches by.
#include "fp8.hpp"

namespace zr {

struct QuantArgs {
    const uint16_t *src;
    int64_t rows, cols, ld;
    uint8_t *q;
    int64_t ldq;
    uint8_t *scales;
    uint8_t *qt;
    int64_t ldqt;
    uint8_t *scales_t;
    int64_t gc, gr;  // groups along a row and along a column
};

// fp32 pattern of a magnitude's 16 bits.
template <typename T>
__device__ __forceinline__ uint32_t wide_bits(uint32_t h)
{
    return __float_as_uint(widen<T>((uint16_t)h));
}

// Largest magnitude (16 bits) of eight elements.
__device__ __forceinline__ uint32_t amax8(u32x4 w)
{
    const uint32_t m = max2(max2(abs2(w[0]), abs2(w[1])), max2(abs2(w[2]), abs2(w[3])));
    return max_u32(m & 0xffffu, m >> 16);
}

template <typename T, int kFormat>
__device__ __forceinline__ u32x2 codes8(u32x4 w, uint32_t s)
{
    const float inv = inverse_scale(s);
    return u32x2{codes4<kFormat>(T::lo(w[0]), T::hi(w[0]), T::lo(w[1]), T::hi(w[1]), inv, s),
                 codes4<kFormat>(T::lo(w[2]), T::hi(w[2]), T::lo(w[3]), T::hi(w[3]), inv, s)};
}

// ---------------------------------------------------------- groups along rows --

// A row of 16 lanes holds a group, 8 elements per lane, so a wave holds 4
// consecutive groups (of one row or of consecutive rows) and its accesses cover
// whole lines; the maximum is four DPP steps.  Each XCD takes 64 consecutive tiles of
// 16 groups at a time: 8192 x 11008 bf16 in 47 us, 5.7 TB/s (in launch order 56 at a state
// of 50).  1 x 4096 takes 2 us, a launch.  With rows off 16 bytes the same bytes come from
// memory, but the vector cache is accessed 2.2 times as often and bounds: 8192 x 4095 in 30
// us, 8192 x 4096 in 20.
template <typename T, int kFormat>
__global__ __launch_bounds__(kBlock) void quantize_rows_kernel(QuantArgs a, int64_t groups)
{
    const int lane = threadIdx.x & 63;
    const int64_t stride = (int64_t)gridDim.x * (kBlock / 16);
    int64_t base = first_tile<64>() * (kBlock / 16) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 4;
    for (; base < groups; base += stride) {
        // row and group of the wave's first group, then of this lane's
        int64_t row = 0, g = base;
        if (a.rows > 1) {
            row = groups <= 0xffffffffll ? (int64_t)((uint32_t)base / (uint32_t)a.gc) : base / a.gc;
            g = base - row * a.gc;
        }
        g += lane >> 4;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const bool over = g >= a.gc;
            row += over;
            g -= over ? a.gc : 0;
        }
        const bool live = row < a.rows;
        const int64_t col = g * kGroup + (lane & 15) * kVec;
        const int64_t n = live ? a.cols - col : 0;
        const u32x4 w = load8<true>(a.src + row * a.ld + col, n);
        const uint32_t s = scale_byte<kFormat>(wide_bits<T>(group_max(amax8(w))));
        store_codes8<false>(a.q + row * a.ldq + col, codes8<T, kFormat>(w, s), n);
        if (live && (lane & 15) == 0)
            a.scales[row * a.gc + g] = (uint8_t)s;
    }
}

// ------------------------------------------------- tiles with a transposed copy --

// One workgroup quantizes a tile of 128 x 128 elements.  Thread t holds the 8 x 8
// elements of rows 8 (t / 16) ... and columns 8 (t % 16) ..., so a row of 16 lanes
// holds 128 columns of 8 rows, and the tile is read from memory once for both
// copies.  Row maxima are DPP steps; column maxima go through LDS across the 4
// waves.  The transposed codes are made 8 rows to an 8-byte word and turned in
// LDS, whose 8-byte slots are permuted by the column's lane (slot ^ column / 8) so
// that the 16 lanes of a write fall into different banks.  Tiles go down the columns
// (consecutive ones write neighbouring pieces of a transposed row), in runs of 16 to an
// XCD.  11008 x 4096 in blocks, both copies: 39 us, 4.6 TB/s (codes alone 30, transpose
// alone 27); 5003 x 12288 by rows and columns: 57 us, 4.3 TB/s (columns alone 38): a row of
// a tile is 256 bytes of a source row and 128 of a copy's, shorter runs than a copy's.  The 8 x 8 elements of a thread need the registers
// of two workgroups to a compute unit: bounded to 4 or 5 they spill (92 and 120 us).
template <typename T, int kFormat, bool kBlocks>
__global__ __launch_bounds__(kBlock) void quantize_tile_kernel(QuantArgs a, int64_t tiles)
{
    __shared__ u32x2 turn[kGroup * 16];
    __shared__ u32x4 colmax[4][16];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, tr = t >> 4, tc = t & 15;
    for (int64_t tile = first_tile<16>(); tile < tiles; tile += gridDim.x) {
        const int64_t gcol = tile / a.gr, grow = tile - gcol * a.gr;
        const int64_t r0 = grow * kGroup + tr * kVec, c0 = gcol * kGroup + tc * kVec;
        u32x4 w[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            w[i] = load8<true>(a.src + (r0 + i) * a.ld + c0, r0 + i < a.rows ? a.cols - c0 : 0);
        // column maxima over this thread's rows, over the wave's, over the tile's
        u32x4 cm;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t m = abs2(w[0][h]);
#pragma unroll
            for (int i = 1; i < kVec; ++i)
                m = max2(m, abs2(w[i][h]));
            m = max2(m, (uint32_t)__shfl_xor((int)m, 16, 64));
            m = max2(m, (uint32_t)__shfl_xor((int)m, 32, 64));
            cm[h] = m;
        }
        __syncthreads();  // the last tile's LDS reads are done
        if (lane < 16)
            colmax[wave][lane] = cm;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const u32x4 o = colmax[j][tc];
#pragma unroll
            for (int h = 0; h < 4; ++h)
                cm[h] = max2(cm[h], o[h]);
        }
        uint32_t block = 0;  // the block's scale
        if (kBlocks)
            block = scale_byte<kFormat>(wide_bits<T>(group_max(amax8(cm))));
        // codes in row order
        if (a.q) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const uint32_t s = kBlocks ? block : scale_byte<kFormat>(wide_bits<T>(group_max(amax8(w[i]))));
                if (r0 + i < a.rows) {
                    store_codes8(a.q + (r0 + i) * a.ldq + c0, codes8<T, kFormat>(w[i], s), a.cols - c0);
                    if (!kBlocks && tc == 0)
                        a.scales[(r0 + i) * a.gc + gcol] = (uint8_t)s;
                }
            }
            if (kBlocks && t == 0)
                a.scales[grow * a.gc + gcol] = (uint8_t)block;
        }
        if (!a.qt)
            continue;
        // codes in column order: 8 rows of one column to a word
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const uint32_t m = j % 2 ? cm[j / 2] >> 16 : cm[j / 2] & 0xffffu;
            const uint32_t s = kBlocks ? block : scale_byte<kFormat>(wide_bits<T>(m));
            const float inv = inverse_scale(s);
            float f[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                f[i] = j % 2 ? T::hi(w[i][j / 2]) : T::lo(w[i][j / 2]);
            turn[(tc * kVec + j) * 16 + (tr ^ tc)] = u32x2{codes4<kFormat>(f[0], f[1], f[2], f[3], inv, s),
                                                          codes4<kFormat>(f[4], f[5], f[6], f[7], inv, s)};
            if (!kBlocks && tr == 0 && c0 + j < a.cols)
                a.scales_t[(c0 + j) * a.gr + grow] = (uint8_t)s;
        }
        if (kBlocks && t == 0)
            a.scales_t[gcol * a.gr + grow] = (uint8_t)block;
        __syncthreads();
        // thread t writes 8 rows' codes (slot t % 16) of columns t / 16 + 16 p
#pragma unroll
        for (int p = 0; p < kVec; ++p) {
            const int col = tr + 16 * p;
            const int64_t c = gcol * kGroup + col, r = grow * kGroup + tc * kVec;
            if (c < a.cols)
                store_codes8(a.qt + c * a.ldqt + r, turn[col * 16 + (tc ^ (col >> 3))], a.rows - r);
        }
    }
}

namespace {

template <typename T, int kFormat>
zr_status quantize_run(const QuantArgs &a, int32_t block_rows, hipStream_t st)
{
    if (block_rows == 1 && !a.qt) {
        QuantArgs f = a;
        // rows without gaps whose groups are whole are one long row
        if (f.cols % kGroup == 0 && f.ld == f.cols && f.ldq == f.cols) {
            f.cols *= f.rows;
            f.gc *= f.rows;
            f.rows = 1;
        }
        const int64_t groups = f.rows * f.gc;
        const dim3 grid = grid_of((groups + kBlock / 16 - 1) / (kBlock / 16));
        return launch(quantize_rows_kernel<T, kFormat>, grid, dim3(kBlock), 0, st, f, groups);
    }
    const int64_t tiles = a.gr * a.gc;
    const dim3 grid = grid_of(tiles);
    return block_rows == 1 ? launch(quantize_tile_kernel<T, kFormat, false>, grid, dim3(kBlock), 0, st, a, tiles)
                           : launch(quantize_tile_kernel<T, kFormat, true>, grid, dim3(kBlock), 0, st, a, tiles);
}

}  // namespace
}  // namespace zr

using namespace zr;

extern "C" zr_status zr_quantize_fp8(const void *src, zr_dtype dtype, int64_t rows, int64_t cols, int64_t ld,
                                     int32_t block_rows, zr_fp8_format format, uint8_t *q, int64_t ldq,
                                     uint8_t *scales, uint8_t *qt, int64_t ldqt, uint8_t *scales_t, void *stream)
{
    clear_error();
    const char *who = "zr_quantize_fp8";
    if (dtype != ZR_BF16 && dtype != ZR_F16)
        return fail(ZR_EINVAL, "%s: dtype = %d, must be ZR_BF16 or ZR_F16", who, dtype);
    if (format != ZR_E4M3 && format != ZR_E5M2)
        return fail(ZR_EINVAL, "%s: format = %d, must be ZR_E4M3 or ZR_E5M2", who, format);
    if (block_rows != 1 && block_rows != kGroup)
        return fail(ZR_EINVAL, "%s: block_rows = %d, must be 1 or 128", who, block_rows);
    if ((!q) != (!scales) || (!qt) != (!scales_t))
        return fail(ZR_EINVAL, "%s: codes without scales or scales without codes", who);
    const bool both_absent = !q && !qt;
    if (rows < 0 || cols < 0)
        return fail(ZR_EINVAL, "%s: negative rows or cols", who);
    if (rows == 0 || cols == 0)
        return ZR_OK;
    if (!src || both_absent)
        return fail(ZR_EINVAL, "%s: NULL src or no output", who);
    int64_t src_n, q_n = 0, qt_n = 0;
    if (!matrix_extent(rows, cols, ld, 2, &src_n) || (q && !matrix_extent(rows, cols, ldq, 1, &q_n)) ||
        (qt && !matrix_extent(cols, rows, ldqt, 1, &qt_n)))
        return fail(ZR_EINVAL, "%s: row distance below the row length, or a matrix past int64", who);
    if (!aligned_to(src, 2))
        return fail(ZR_EALIGN, "%s: src must be 2-byte aligned", who);
    const int64_t gc = (cols + kGroup - 1) / kGroup, gr = (rows + kGroup - 1) / kGroup;
    {
        const void *p[5] = {src, q, scales, qt, scales_t};
        int64_t b[5] = {src_n, q_n, (block_rows == 1 ? rows : gr) * gc, qt_n, (block_rows == 1 ? cols : gc) * gr};
        int x, y;
        if (any_overlap(p, b, 5, &x, &y))
            return fail(ZR_EINVAL, "%s: buffers %d and %d overlap", who, x, y);
    }
    const QuantArgs a{static_cast<const uint16_t *>(src), rows, cols, ld, q, ldq, scales, qt, ldqt, scales_t, gc, gr};
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == ZR_BF16)
        return format == ZR_E4M3 ? quantize_run<BF16, ZR_E4M3>(a, block_rows, st)
                                 : quantize_run<BF16, ZR_E5M2>(a, block_rows, st);
    return format == ZR_E4M3 ? quantize_run<F16, ZR_E4M3>(a, block_rows, st)
                             : quantize_run<F16, ZR_E5M2>(a, block_rows, st);
}
