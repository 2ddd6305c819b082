// Product of two matrices of 8-bit codes with E8M0 scales per 128 of the summed
// axis: out[i][j] = sum_k A[i][k] B[j][k] (gfx950).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 codes by 128 x 16 and adds
// the 16 x 16 products, each scaled by an E8M0 byte per row and 32 of the summed
// axis, to fp32 accumulators.  A scale per 128 is one byte for the instruction's
// whole depth, so the scales cost no arithmetic, and the order in which a lane
// group takes the 128 codes does not matter as long as both operands agree.
// The first operand is B (output columns) and the second A (output rows): a
// lane's four accumulators are then four neighbours of one output row.
//
// Precision.  On its 8-bit path the matrix unit adds each run of 8 consecutive
// products of a lane before it adds to the accumulators: the 8 are aligned to the
// largest and cut below 2^-13 of it (measured: with products 1 and 2^-j in one run
// 2^-13 is kept and 2^-14 lost; across runs, and against the accumulator, sums are
// fp32).  On normal data that leaves the sum 1.4e-5 off, a hundredth of a rounding
// to bf16 and a tenth of one to fp16, so 16-bit outputs take that path.  An fp32
// output would keep that error, so its codes are widened to bf16 (exact: at most 3
// mantissa bits; the scale is applied by the conversion), whose products the matrix
// unit adds in fp32 (7e-8 off), at half the rate.
#include "fp8.hpp"

namespace zr {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

struct MatmulArgs {
    const uint8_t *a, *b, *sa, *sb;
    int64_t lda, ldb, m, n, k, kb;  // kb: groups of the summed axis
    int32_t b_shift;                // rows of B that share a scale: 2^b_shift
    void *out;
    int64_t ldo;
    int32_t dtype, accumulate;
};

constexpr int kAccum = 4;  // accumulators of a lane in a 16 x 16 tile

// acc (column j .. j + 3 of row i) to out, the first `n` of them.
__device__ __forceinline__ void store_out(const MatmulArgs &p, int64_t i, int64_t j, f32x4 acc, int64_t n)
{
    const int64_t at = i * p.ldo + j;
#pragma unroll
    for (int e = 0; e < kAccum; ++e) {
        if (e >= n)
            break;
        if (p.dtype == ZR_F32) {
            float *o = static_cast<float *>(p.out) + at + e;
            *o = p.accumulate ? *o + acc[e] : acc[e];
        } else {
            uint16_t *o = static_cast<uint16_t *>(p.out) + at + e;
            if (p.dtype == ZR_BF16)
                *o = narrow<BF16>(p.accumulate ? widen<BF16>(*o) + acc[e] : acc[e]);
            else
                *o = narrow<F16>(p.accumulate ? widen<F16>(*o) + acc[e] : acc[e]);
        }
    }
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes times a power of two, as bf16.
template <int kFormat>
__device__ __forceinline__ bf16x8 widen8(int lo, int hi, float scale)
{
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int w = i < 2 ? lo : hi;
        bf16x2 p;
        if constexpr (kFormat == ZR_E4M3)
            p = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true)
                      : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
        else
            p = i % 2 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, true)
                      : __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, false);
        o[2 * i] = p[0];
        o[2 * i + 1] = p[1];
    }
    return o;
}

// A lane's 32 codes of a 16 x 128 operand from two 16-byte pieces.
__device__ __forceinline__ i32x8 operand(u32x4 lo, u32x4 hi)
{
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

__device__ __forceinline__ i32x8 operand_at(const uint8_t *p)
{
    return operand(*reinterpret_cast<const u32x4 *>(p), *reinterpret_cast<const u32x4 *>(p + 16));
}

// acc += B's 16 rows times A's 16 rows over one group of 128: codes fb and fa (any
// order of the 128 in which both agree), scale bytes sb and sa in the low byte.
template <int kFormatA, bool kWide>
__device__ __forceinline__ f32x4 multiply(i32x8 fb, int sb, i32x8 fa, int sa, f32x4 acc)
{
    if constexpr (!kWide) {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb, fa, acc, ZR_E4M3, kFormatA, 0, sb, 0, sa);
    } else {
        const float xb = __uint_as_float((uint32_t)sb << 23), xa = __uint_as_float((uint32_t)sa << 23);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<ZR_E4M3>(fb[2 * i], fb[2 * i + 1], xb),
                                                          widen8<kFormatA>(fa[2 * i], fa[2 * i + 1], xa), acc, 0, 0, 0);
        return acc;
    }
}

// Any alignment and any sizes: a workgroup computes 64 x 64 outputs, its codes
// staged through LDS byte by byte with zeros outside the matrices.
constexpr int kAnyTile = 64;
constexpr int kAnyRow = kGroup + 16;  // LDS bytes of a staged row

template <int kFormatA, bool kWide>
__global__ __launch_bounds__(kBlock) void matmul_any_kernel(MatmulArgs p, int64_t tiles_n, int64_t tiles)
{
    __shared__ __attribute__((aligned(16))) uint8_t la[kAnyTile * kAnyRow], lb[kAnyTile * kAnyRow];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, row = lane & 15, quad = lane >> 4;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t i0 = tile / tiles_n * kAnyTile, j0 = tile % tiles_n * kAnyTile;
        f32x4 acc[4] = {};
        for (int64_t g = 0; g < p.kb; ++g) {
            __syncthreads();
            for (int e = t; e < kAnyTile * kGroup; e += kBlock) {
                const int r = e / kGroup, c = e % kGroup;
                const int64_t kk = g * kGroup + c;
                la[r * kAnyRow + c] = i0 + r < p.m && kk < p.k ? p.a[(i0 + r) * p.lda + kk] : 0;
                lb[r * kAnyRow + c] = j0 + r < p.n && kk < p.k ? p.b[(j0 + r) * p.ldb + kk] : 0;
            }
            __syncthreads();
            const int64_t j = j0 + wave * 16 + row;
            const int sb = j < p.n ? p.sb[(j >> p.b_shift) * p.kb + g] : 0;
            const i32x8 fb = operand_at(lb + (wave * 16 + row) * kAnyRow + quad * 32);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int64_t i = i0 + x * 16 + row;
                const int sa = i < p.m ? p.sa[i * p.kb + g] : 0;
                const i32x8 fa = operand_at(la + (x * 16 + row) * kAnyRow + quad * 32);
                acc[x] = multiply<kFormatA, kWide>(fb, sb, fa, sa, acc[x]);
            }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int64_t i = i0 + x * 16 + row, j = j0 + wave * 16 + quad * 4;
            if (i < p.m)
                store_out(p, i, j, acc[x], p.n - j);
        }
    }
}

// ------------------------------------------------------------- large products --

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kBig = 256;                  // output rows and columns of a workgroup
constexpr int kBigThreads = 512;           // 8 waves: 2 down the rows x 4 across the columns
constexpr int kBigStage = 2 * kBig * kGroup;  // LDS bytes of one group of both operands

__device__ __forceinline__ f32x16 multiply32(i32x8 b, int sb, i32x8 a, int sa, f32x16 acc)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, ZR_E4M3, ZR_E4M3, 0, sb, 0, sa);
}

// Byte offset of 16-byte piece `piece` (of 8) of row `row` in a staged tile.
__device__ __forceinline__ int staged(int row, int piece) { return row * kGroup + ((piece ^ (row & 7)) << 4); }

struct ScaleWords {
    const uint8_t *base;  // of the tile's first row
    int32_t limit;        // last offset a word may be read at
};

// Four scale bytes from byte `at` on.
__device__ __forceinline__ uint32_t scale_word(const ScaleWords &s, int32_t at)
{
    const int32_t from = at < s.limit ? at : s.limit;
    uint32_t w;
    __builtin_memcpy(&w, s.base + from, 4);
    return w >> (8 * (at - from));
}

template <int kFormatA>
__global__ __launch_bounds__(kBigThreads, 2) void matmul_big_kernel(MatmulArgs p, int64_t tiles_m, int64_t tiles_n)
{
    __shared__ __attribute__((aligned(1024))) uint8_t stage0[kBigStage], stage1[kBigStage];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = (wave >> 2) * 128, wn = (wave & 3) * 64, row = lane & 31, half = lane >> 5;
    const int64_t tiles = tiles_m * tiles_n;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t tm = tile / tiles_n, tn = tile % tiles_n;
        const int64_t i0 = tm * kBig, j0 = tn * kBig;
        const int rows_a = (int)(p.m - i0 < kBig ? p.m - i0 : kBig), rows_b = (int)(p.n - j0 < kBig ? p.n - j0 : kBig);
        const int64_t left_a = (p.m - 1 - i0) * p.lda + p.k, left_b = (p.n - 1 - j0) * p.ldb + p.k;
        const int64_t most = 0xfffffff0ll;
        const auto ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p.a + i0 * p.lda), 0,
                                                          (int)(uint32_t)(((left_a < most ? left_a : most) + 15) & ~15ll), 0x00027000);
        const auto rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p.b + j0 * p.ldb), 0,
                                                          (int)(uint32_t)(((left_b < most ? left_b : most) + 15) & ~15ll), 0x00027000);
        // staging: a wave's instruction fills 8 rows; row r of 8, piece lane % 8
        uint32_t at_a[4], at_b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = (j * 8 + wave) * 8 + (lane >> 3);
            const int piece = (lane & 7) ^ (r & 7);
            const int xa = r < rows_a ? r : rows_a - 1, xb = r < rows_b ? r : rows_b - 1;
            at_a[j] = (uint32_t)xa * (uint32_t)p.lda + piece * 16;
            at_b[j] = (uint32_t)xb * (uint32_t)p.ldb + piece * 16;
        }
        const auto load = [&](uint8_t *stage, int64_t g) {
            typedef __attribute__((address_space(3))) void *lds_ptr;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr)(stage + (j * 8 + wave) * 1024), 16, at_a[j], (int)(g * kGroup), 0, 0);
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)(stage + kBig * kGroup + (j * 8 + wave) * 1024), 16, at_b[j], (int)(g * kGroup), 0, 0);
            }
        };
        const int32_t kb = (int32_t)p.kb;
        ScaleWords sa{p.sa + i0 * kb, (int32_t)((p.m - i0) * kb - 4 < (1 << 30) ? (p.m - i0) * kb - 4 : (1 << 30))};
        const int64_t sb_rows = ((p.n - 1) >> p.b_shift) + 1, sb0 = j0 >> p.b_shift;
        ScaleWords sb{p.sb + sb0 * kb, (int32_t)((sb_rows - sb0) * kb - 4 < (1 << 30) ? (sb_rows - sb0) * kb - 4 : (1 << 30))};
        int32_t sat[4], sbt[2];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = wm + x * 32 + row;
            sat[x] = (r < rows_a ? r : rows_a - 1) * kb;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int r = wn + x * 32 + row;
            sbt[x] = ((r < rows_b ? r : rows_b - 1) >> p.b_shift) * kb;
        }
        uint32_t ca[4], cb[2], na[4], nb[2];
        const auto load_scales = [&](int32_t g) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
                na[x] = scale_word(sa, sat[x] + g);
#pragma unroll
            for (int x = 0; x < 2; ++x)
                nb[x] = scale_word(sb, sbt[x] + g);
        };
        f32x16 acc[2][4] = {};
        const auto compute = [&](const uint8_t *stage) {
            i32x8 fb[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = kBig + wn + x * 32 + row;
                    fb[x][h] = operand(*reinterpret_cast<const u32x4 *>(stage + staged(r, h * 4 + half * 2)),
                                       *reinterpret_cast<const u32x4 *>(stage + staged(r, h * 4 + half * 2 + 1)));
                }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                i32x8 fa[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = wm + y * 32 + row;
                    fa[h] = operand(*reinterpret_cast<const u32x4 *>(stage + staged(r, h * 4 + half * 2)),
                                    *reinterpret_cast<const u32x4 *>(stage + staged(r, h * 4 + half * 2 + 1)));
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[x][h], fa[h], acc[x][y], ZR_E4M3, kFormatA, 0, (int)cb[x], 0, (int)ca[y]);
            }
        };
        const auto step = [&](uint8_t *stage, uint8_t *next, int32_t g) {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __builtin_amdgcn_s_barrier();
            if (g + 1 < kb)
                load(next, g + 1);
            if ((g & 3) == 0) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    ca[x] = na[x];
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    cb[x] = nb[x];
                if (g + 4 < kb)
                    load_scales(g + 4);
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    ca[x] >>= 8;
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    cb[x] >>= 8;
            }
            if (g + 1 == kb && p.k % kGroup) {  // zeros behind the last code of every row
                const int tail = (int)(p.k % kGroup);
                uint8_t *line = stage + t * kGroup;
                for (int piece = tail / 16; piece < 8; ++piece) {
                    u32x4 *w = reinterpret_cast<u32x4 *>(line + ((piece ^ (t & 7)) << 4));
                    u32x4 v = *w;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int keep = tail - piece * 16 - e * 4;  // bytes of the word that stay
                        v[e] = keep >= 4 ? v[e] : keep <= 0 ? 0u : v[e] & ((1u << (8 * keep)) - 1u);
                    }
                    *w = v;
                }
                __syncthreads();
            }
            compute(stage);
        };
        __syncthreads();
        load(stage0, 0);
        load_scales(0);
        for (int32_t g = 0; g < kb; g += 2) {
            step(stage0, stage1, g);
            if (g + 1 < kb)
                step(stage1, stage0, g + 1);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            const int64_t i = i0 + wm + y * 32 + row;
            if (i >= p.m)
                continue;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int64_t j = j0 + wn + x * 32 + e * 8 + half * 4;
                    store_out(p, i, j, f32x4{acc[x][y][4 * e], acc[x][y][4 * e + 1], acc[x][y][4 * e + 2], acc[x][y][4 * e + 3]}, p.n - j);
                }
        }
    }
}

namespace {

template <int kFormatA, bool kWide>
zr_status matmul_run(const MatmulArgs &p, hipStream_t st)
{
    if constexpr (!kWide) {
        const bool aligned = aligned_to(p.a, 16) && aligned_to(p.b, 16) && p.lda % 16 == 0 && p.ldb % 16 == 0 &&
                             p.lda < (1 << 23) && p.ldb < (1 << 23) && p.m * p.kb >= 4 && (((p.n - 1) >> p.b_shift) + 1) * p.kb >= 4;
        if (aligned && p.k > 0 && p.m > 256 && p.n >= 256) {
            const int64_t bm = (p.m + kBig - 1) / kBig, bn = (p.n + kBig - 1) / kBig;
            return launch(matmul_big_kernel<kFormatA>, grid_of(bm * bn), dim3(kBigThreads), 0, st, p, bm, bn);
        }
    }
    const int64_t tn = (p.n + kAnyTile - 1) / kAnyTile, tiles = tn * ((p.m + kAnyTile - 1) / kAnyTile);
    return launch(matmul_any_kernel<kFormatA, kWide>, grid_of(tiles), dim3(kBlock), 0, st, p, tn, tiles);
}

}  // namespace
}  // namespace zr

using namespace zr;

extern "C" zr_status zr_matmul_fp8(const uint8_t *a, int64_t lda, const uint8_t *a_scales, zr_fp8_format a_format,
                                   const uint8_t *b, int64_t ldb, const uint8_t *b_scales, int32_t b_block_rows,
                                   int64_t m, int64_t n, int64_t k, void *out, zr_dtype out_dtype, int64_t ldo,
                                   int32_t accumulate, void *stream)
{
    clear_error();
    const char *who = "zr_matmul_fp8";
    if (a_format != ZR_E4M3 && a_format != ZR_E5M2)
        return fail(ZR_EINVAL, "%s: a_format = %d, must be ZR_E4M3 or ZR_E5M2", who, a_format);
    if (out_dtype != ZR_BF16 && out_dtype != ZR_F16 && out_dtype != ZR_F32)
        return fail(ZR_EINVAL, "%s: out_dtype = %d, must be ZR_BF16, ZR_F16 or ZR_F32", who, out_dtype);
    if (b_block_rows != 1 && b_block_rows != kGroup)
        return fail(ZR_EINVAL, "%s: b_block_rows = %d, must be 1 or 128", who, b_block_rows);
    if (accumulate != 0 && accumulate != 1)
        return fail(ZR_EINVAL, "%s: accumulate = %d, must be 0 or 1", who, accumulate);
    if (m < 0 || n < 0 || k < 0)
        return fail(ZR_EINVAL, "%s: negative size", who);
    if (m == 0 || n == 0 || (k == 0 && accumulate))
        return ZR_OK;
    const int64_t size = out_dtype == ZR_F32 ? 4 : 2;
    if (!out || (k > 0 && (!a || !b || !a_scales || !b_scales)))
        return fail(ZR_EINVAL, "%s: NULL buffer", who);
    int64_t na = 0, nb = 0, no;
    if (!matrix_extent(m, n, ldo, size, &no) ||
        (k > 0 && (!matrix_extent(m, k, lda, 1, &na) || !matrix_extent(n, k, ldb, 1, &nb))))
        return fail(ZR_EINVAL, "%s: row distance below the row length, or a matrix past int64", who);
    if (!aligned_to(out, size))
        return fail(ZR_EALIGN, "%s: out must be %d-byte aligned", who, (int)size);
    const int64_t kb = (k + kGroup - 1) / kGroup;
    const int64_t sb_rows = b_block_rows == 1 ? n : (n + kGroup - 1) / kGroup;
    {
        const void *p[4] = {a, b, a_scales, b_scales};
        const int64_t bytes[4] = {na, nb, m * kb, sb_rows * kb};
        for (int i = 0; i < 4; ++i)
            if (p[i] && overlaps(out, no, p[i], bytes[i]))
                return fail(ZR_EINVAL, "%s: out overlaps another buffer", who);
    }
    const MatmulArgs p{a, b, a_scales, b_scales, lda, ldb, m, n, k, kb, b_block_rows == 1 ? 0 : 7, out, ldo,
                       out_dtype, accumulate};
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (out_dtype == ZR_F32)
        return a_format == ZR_E4M3 ? matmul_run<ZR_E4M3, true>(p, st) : matmul_run<ZR_E5M2, true>(p, st);
    return a_format == ZR_E4M3 ? matmul_run<ZR_E4M3, false>(p, st) : matmul_run<ZR_E5M2, false>(p, st);
}
