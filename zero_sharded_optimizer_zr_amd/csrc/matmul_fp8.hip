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
// mantissa bits; the scale is applied by the conversion, and elements past bf16's
// range are taken smaller, see lower_scales), whose products the matrix unit adds in
// fp32 (7e-8 off), at half the rate.
//
// Four kernels: waves that split the summed axis (few rows, any alignment), 128 x 64
// outputs by two teams, 128 x 128 through a ring in LDS, and 256 x 256 for the large
// products; matmul_run says which is taken when.
#include "fp8.hpp"

namespace zr {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float any_f32x4 __attribute__((ext_vector_type(4), aligned(4)));

struct MatmulArgs {
    const uint8_t *a, *b, *sa, *sb;
    int64_t lda, ldb, m, n, k, kb;  // kb: groups of the summed axis
    int32_t b_shift;                // rows of B that share a scale: 2^b_shift
    void *out;
    int64_t ldo;
    int32_t dtype, accumulate;
};

constexpr int kCus = 256;             // compute units
// Groups are counted in 32 bits, by a few at a time past the last one.
constexpr int32_t kMostGroups = INT32_MAX - 64;
constexpr int kWaitLoads = 0x0f70;   // s_waitcnt vmcnt(0)
constexpr int kWaitAll = 0x0070;     // s_waitcnt vmcnt(0) lgkmcnt(0)
constexpr int kWaitStage = 0x0071;   // s_waitcnt vmcnt(1) lgkmcnt(0)

constexpr int kAccum = 4;  // accumulators of a lane in a 16 x 16 tile

// Four (or eight) sums, columns j ... of row i, to out: the first `n` of them.
template <typename T>
__device__ __forceinline__ u32x2 add4(u32x2 old, f32x4 v, bool accumulate)
{
    if (accumulate)
        v += f32x4{T::lo(old[0]), T::hi(old[0]), T::lo(old[1]), T::hi(old[1])};
    return u32x2{T::pack(v[0], v[1]), T::pack(v[2], v[3])};
}

// The old values of an accumulating product are waited for where they are loaded:
// the compiler, which does not know there whether anything was, would wait again in
// the loop that follows, for every load in flight.
__device__ __forceinline__ void store_out(const MatmulArgs &p, int64_t i, int64_t j, f32x4 v, int64_t n)
{
    const int64_t at = i * p.ldo + j;
    const bool vec = n >= kAccum;  // at any address
    if (p.dtype == ZR_F32) {
        float *o = static_cast<float *>(p.out) + at;
        if (p.accumulate) {
            f32x4 old = {0.0f, 0.0f, 0.0f, 0.0f};
            if (vec) {
                old = *(global_ptr<const any_f32x4>)o;
            } else {
#pragma unroll
                for (int e = 0; e < kAccum; ++e)
                    if (e < n)
                        old[e] = o[e];
            }
            __builtin_amdgcn_s_waitcnt(kWaitLoads);
            v += old;
        }
        if (vec) {
            *(global_ptr<any_f32x4>)o = v;
            return;
        }
#pragma unroll
        for (int e = 0; e < kAccum; ++e)
            if (e < n)
                o[e] = v[e];
        return;
    }
    uint16_t *o = static_cast<uint16_t *>(p.out) + at;
    u32x2 w = {0, 0};
    if (p.accumulate) {
        if (vec) {
            w = *(global_ptr<const any_u32x2>)o;
        } else {
#pragma unroll
            for (int e = 0; e < kAccum; ++e)
                if (e < n)
                    w[e / 2] |= (uint32_t)o[e] << (16 * (e % 2));
        }
        __builtin_amdgcn_s_waitcnt(kWaitLoads);
    }
    w = p.dtype == ZR_BF16 ? add4<BF16>(w, v, p.accumulate) : add4<F16>(w, v, p.accumulate);
    if (vec) {
        *(global_ptr<any_u32x2>)o = w;
        return;
    }
#pragma unroll
    for (int e = 0; e < kAccum; ++e)
        if (e < n)
            o[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
}

// The same for eight sums and a 16-bit out.  Stored through the caches.  Past them it is 2 to
// 8 % faster after short sums (16384 x 16384 by k = 512 253 us against 266, by 2048 556
// against 563) but slower where rows are not whole lines (2900 x 2950 x 400 24.8 against 22.5),
// with accumulation (16384 x 16384 x 1024 573 against 559) and after long sums (16384 x 11008 x
// 4096 641 against 638).
__device__ __forceinline__ void store_out(const MatmulArgs &p, int64_t i, int64_t j, f32x4 lo, f32x4 hi, int64_t n)
{
    uint16_t *o = static_cast<uint16_t *>(p.out) + i * p.ldo + j;
    u32x4 w = {0, 0, 0, 0};
    if (p.accumulate) {
        w = load8(o, n);
        __builtin_amdgcn_s_waitcnt(kWaitLoads);
    }
    const u32x2 a = {w[0], w[1]}, b = {w[2], w[3]};
    u32x2 c, d;
    if (p.dtype == ZR_BF16) {
        c = add4<BF16>(a, lo, p.accumulate);
        d = add4<BF16>(b, hi, p.accumulate);
    } else {
        c = add4<F16>(a, lo, p.accumulate);
        d = add4<F16>(b, hi, p.accumulate);
    }
    w = u32x4{c[0], c[1], d[0], d[1]};
    store8(o, w, n);
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes times a power of two, as bf16.
template <int kFormat>
__device__ __forceinline__ bf16x8 widen8(uint32_t lo, uint32_t hi, float scale)
{
    bf16x8 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int w = (int)(i < 2 ? lo : hi);
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

// Elements past bf16's range.  A scale byte from kFar on (247 for e4m3, 240 for e5m2; 255
// is NaN) makes elements of 2^128 and more, which the widening would turn into infinities
// although their products may be small: the largest bf16 value's own code is 2^128.
// Where a group has such a scale, its row or column is widened 2^16 times smaller, and
// the sums of that row or column are taken 2^16 times smaller over this group; all others
// keep their bits.  Sums below 2^-90, which could lose bits, stay as they are: the products
// they meet are zeros, and the sum is right without the factor, or multiples of 2^-52 (a
// code of at least 2^-16 or 2^-9 times 2^(kFar - 16 - 127) times at least 2^-133), beside
// which they are nothing (2^-38 of the result).  Looking for such scales, which are rare,
// takes 1 to 3 % (11008 x 4096 x 8192 752 us at 739 without, 333 x 4096 x 4096 21.0 at 20.4).
template <int kFormat>
constexpr uint32_t kFar = kFormat == ZR_E4M3 ? 247 : 240;

// The lowered scales of a lane's accumulators and the sums held as they are.
struct Lowered {
    uint32_t marks;  // a bit for accumulator e of column tile z at z * kAccum + e, for row tile y at 16 + y
    uint64_t held;   // a bit for each accumulator
};

template <int kFormat>
__device__ __forceinline__ bool is_far(uint32_t s)
{
    return s >= kFar<kFormat> && s < 255u;
}

// How often an accumulator is taken 2^16 times smaller: 0, 1 or 2.
__device__ __forceinline__ int times(uint32_t marks, int y, int at)
{
    return (int)(marks >> at & 1) + (int)(marks >> (16 + y) & 1);
}

// One tile's sums after another, and back where the products take them (kPinned: in the
// matrix unit's registers): few registers are free.
template <bool kPinned>
__device__ __forceinline__ void one_tile(f32x4 &v, Lowered &low)
{
    if constexpr (kPinned)
        asm volatile("" : "+a"(v), "+v"(low.marks), "+v"(low.held));
    else
        asm volatile("" : "+v"(v), "+v"(low.marks), "+v"(low.held));
}

// Lowers the scales of a group, and the sums, where needed; false if nowhere.
template <bool kPinned, int kFormatA, int MT, int NT>
__device__ __forceinline__ bool lower_scales(uint32_t *ca, uint32_t *cb, f32x4 (&acc)[MT][NT], Lowered &low)
{
    // one maximum over both operands: the lower limit of the two, here, for either
    uint32_t most = ca[0];
#pragma unroll
    for (int y = 1; y < MT; ++y)
        most = max_u32(most, ca[y]);
#pragma unroll
    for (int z = 0; z < NT; ++z)
        most = max_u32(most, cb[z]);
    if (!__any(most >= kFar<kFormatA>))
        return false;
    low = {0, 0};
#pragma unroll
    for (int y = 0; y < MT; ++y) {
        const bool far = is_far<kFormatA>(ca[y]);
        low.marks |= (uint32_t)far << (16 + y);
        ca[y] -= far ? 16 : 0;
    }
    // this lane has the scale of one row of B in each tile, and accumulators of four
#pragma unroll
    for (int z = 0; z < NT; ++z) {
        const bool far = is_far<ZR_E4M3>(cb[z]);
        const uint64_t lanes = __ballot(far);
        low.marks |= (uint32_t)(lanes >> ((threadIdx.x & 63) / 16 * kAccum) & 15) << (z * kAccum);
        cb[z] -= far ? 16 : 0;
    }
#pragma unroll
    for (int y = 0; y < MT; ++y)
#pragma unroll
        for (int z = 0; z < NT; ++z) {
            f32x4 v = acc[y][z];
            one_tile<kPinned>(v, low);
#pragma unroll
            for (int e = 0; e < kAccum; ++e) {
                const bool hold = !(__builtin_fabsf(v[e]) >= 0x1p-90f);
                v[e] = __builtin_ldexpf(v[e], hold ? 0 : -16 * times(low.marks, y, z * kAccum + e));
                low.held |= (uint64_t)hold << ((y * NT + z) * kAccum + e);
            }
            one_tile<kPinned>(v, low);
            acc[y][z] = v;
        }
    return true;
}

// Sums stay in the matrix unit's registers where paths meet.
template <int MT, int NT>
__device__ __forceinline__ void pin(f32x4 (&acc)[MT][NT])
{
#pragma unroll
    for (int y = 0; y < MT; ++y)
#pragma unroll
        for (int z = 0; z < NT; ++z)
            asm volatile("" : "+a"(acc[y][z]));
}

// After the group's products.
template <bool kPinned, int MT, int NT>
__device__ __forceinline__ void raise_sums(f32x4 (&acc)[MT][NT], Lowered &low)
{
#pragma unroll
    for (int y = 0; y < MT; ++y)
#pragma unroll
        for (int z = 0; z < NT; ++z) {
            f32x4 v = acc[y][z];
            one_tile<kPinned>(v, low);
#pragma unroll
            for (int e = 0; e < kAccum; ++e) {
                // no product came to a held sum that is still small
                const bool alone = (low.held >> ((y * NT + z) * kAccum + e) & 1) && __builtin_fabsf(v[e]) < 0x1p-60f;
                v[e] = __builtin_ldexpf(v[e], alone ? 0 : 16 * times(low.marks, y, z * kAccum + e));
            }
            one_tile<kPinned>(v, low);
            acc[y][z] = v;
        }
}

// A lane's 32 codes of an operand from two 16-byte pieces.
__device__ __forceinline__ i32x8 operand(u32x4 lo, u32x4 hi)
{
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// ------------------------------------------------------- few rows, any alignment --

// A wave computes 16 MT x 16 NT outputs over a range of groups, its operands loaded
// straight into registers (a lane's 32 codes of a group are pieces `quad` and `quad`
// + 4 of its row: 16 rows x 64 bytes an instruction), `kAhead` groups ahead of their
// use.  `split` waves of a workgroup share a tile and take a part of the groups each;
// their sums meet in LDS and are added in wave order.  So a product with few
// tiles still occupies the chip, without a workspace.  Bound by the bytes of B and by
// the latency of the few loads a wave makes: 1 x 11008 x 4096 (m x n x k) 13.7 us, 3.3
// TB/s; 1 x 32000 x 4096 26 us, 5.0 TB/s; 32 x 11008 x 4096 18 us; 1 x 512 x 512 4 us, a
// launch.  Rows off 16 bytes have no other kernel: 1000 x 4096 x 4096 50 us (24 on them),
// 4096 x 4096 x 4096 201 (66).
constexpr int kSplitThreads = 512;
constexpr int kSplitWaves = kSplitThreads / 64;

// 16 codes at `p`, of which `n` belong to the row; the others count as zeros.
// Nothing behind the row is read.
__device__ __forceinline__ u32x4 codes16(const uint8_t *p, int n)
{
    u32x4 w = {0, 0, 0, 0};
    if (n >= 16) {
        __builtin_memcpy(&w, (global_ptr<const uint8_t>)p, 16);
    } else {
#pragma unroll 1
        for (int e = 0; e < n; ++e) {
            const uint32_t byte = (uint32_t)load_global(p + e) << (8 * (e % 4));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] |= e / 4 == i ? byte : 0u;
        }
    }
    return w;
}

// Each of the four rows of 16 lanes, spread over all four.
__device__ __forceinline__ void spread_quads(uint32_t v, uint32_t *out)
{
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    out[0] = lo[0];
    out[1] = lo[1];
    out[2] = hi[0];
    out[3] = hi[1];
}

// One group's operands and scales of a wave's tile.
template <int MT, int NT>
struct SplitGroup {
    u32x4 a[MT][2], b[NT][2];
    uint32_t sa, sb;  // of row 16 quad + lane % 16
};

// acc += the products of one group.
template <int kFormatA, bool kWide, int MT, int NT>
__device__ __forceinline__ void multiply_group(const SplitGroup<MT, NT> &s, f32x4 (&acc)[MT][NT])
{
    uint32_t ca[4], cb[4];
    spread_quads(s.sa, ca);
    spread_quads(s.sb, cb);
    if constexpr (!kWide) {
#pragma unroll
        for (int y = 0; y < MT; ++y)
#pragma unroll
            for (int z = 0; z < NT; ++z)
                acc[y][z] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    operand(s.b[z][0], s.b[z][1]), operand(s.a[y][0], s.a[y][1]), acc[y][z], ZR_E4M3, kFormatA, 0,
                    (int)cb[z], 0, (int)ca[y]);
    } else {
        Lowered low;
        const bool far = lower_scales<false, kFormatA>(ca, cb, acc, low);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 8 codes of each lane at a time
            const int h = i / 2, e = i % 2 * 2;
            bf16x8 b[NT];
#pragma unroll
            for (int z = 0; z < NT; ++z)
                b[z] = widen8<ZR_E4M3>(s.b[z][h][e], s.b[z][h][e + 1], __uint_as_float(cb[z] << 23));
#pragma unroll
            for (int y = 0; y < MT; ++y) {
                const bf16x8 a = widen8<kFormatA>(s.a[y][h][e], s.a[y][h][e + 1], __uint_as_float(ca[y] << 23));
#pragma unroll
                for (int z = 0; z < NT; ++z)
                    acc[y][z] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[z], a, acc[y][z], 0, 0, 0);
            }
        }
        if (far)
            raise_sums<false>(acc, low);
    }
}

template <int kFormatA, bool kWide, int MT, int NT, int kAhead>
__global__ __launch_bounds__(kSplitThreads, 2) void matmul_split_kernel(MatmulArgs p, int32_t split, int64_t tiles_m,
                                                                        int64_t rounds)
{
    __shared__ f32x4 part[kSplitWaves][MT * NT][64];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int row = lane & 15, quad = lane >> 4;
    const int share = wave % split, slot = wave / split, slots = kSplitWaves / split;
    const int32_t kb = (int32_t)p.kb, whole = (int32_t)(p.k / kGroup);
    const int64_t tiles_n = (p.n + 16 * NT - 1) / (16 * NT), tiles = tiles_m * tiles_n;
    for (int64_t round = blockIdx.x; round < rounds; round += gridDim.x) {
        // one run of rounds per XCD; neighbouring tiles share their rows of B
        const int64_t x = round % kXcds, each = rounds / kXcds, more = rounds % kXcds;
        const int64_t tile = (x * each + (x < more ? x : more) + round / kXcds) * slots + slot;
        const bool live = tile < tiles;
        const int64_t i0 = live ? tile % tiles_m * (16 * MT) : 0, j0 = live ? tile / tiles_m * (16 * NT) : 0;
        const uint8_t *pa[MT], *pb[NT];
#pragma unroll
        for (int y = 0; y < MT; ++y) {
            const int64_t i = i0 + y * 16 + row;
            pa[y] = p.a + (i < p.m ? i : p.m - 1) * p.lda + quad * 16;
        }
#pragma unroll
        for (int z = 0; z < NT; ++z) {
            const int64_t j = j0 + z * 16 + row;
            pb[z] = p.b + (j < p.n ? j : p.n - 1) * p.ldb + quad * 16;
        }
        const int64_t ia = i0 + lane, jb = j0 + lane;
        const uint8_t *psa = p.sa + (ia < p.m ? ia : p.m - 1) * kb;
        const uint8_t *psb = p.sb + ((jb < p.n ? jb : p.n - 1) >> p.b_shift) * kb;
        f32x4 acc[MT][NT] = {};
        // loads the group at the pointers and moves them on
        const auto load = [&](SplitGroup<MT, NT> &s) {
#pragma unroll
            for (int z = 0; z < NT; ++z) {
                __builtin_memcpy(&s.b[z][0], (global_ptr<const uint8_t>)pb[z], 16);
                __builtin_memcpy(&s.b[z][1], (global_ptr<const uint8_t>)pb[z] + 64, 16);
                pb[z] += kGroup;
            }
#pragma unroll
            for (int y = 0; y < MT; ++y) {
                __builtin_memcpy(&s.a[y][0], (global_ptr<const uint8_t>)pa[y], 16);
                __builtin_memcpy(&s.a[y][1], (global_ptr<const uint8_t>)pa[y] + 64, 16);
                pa[y] += kGroup;
            }
            s.sa = load_global(psa++);
            s.sb = load_global(psb++);
        };
        // this wave's share of the whole groups
        const int32_t first = (int32_t)((int64_t)whole * share / split), end = (int32_t)((int64_t)whole * (share + 1) / split);
#pragma unroll
        for (int y = 0; y < MT; ++y)
            pa[y] += (int64_t)first * kGroup;
#pragma unroll
        for (int z = 0; z < NT; ++z)
            pb[z] += (int64_t)first * kGroup;
        psa += first;
        psb += first;
        if (live) {
            SplitGroup<MT, NT> s[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (first + u < end)
                    load(s[u]);
            for (int32_t g = first; g < end; g += kAhead)
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (g + u < end)
                        multiply_group<kFormatA, kWide>(s[u], acc);
                    if (g + u + kAhead < end)
                        load(s[u]);
                }
            if (whole < kb && share == split - 1) {  // the short last group
                const int left = (int)(p.k - (int64_t)whole * kGroup) - quad * 16;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int z = 0; z < NT; ++z)
                        s[0].b[z][h] = codes16(pb[z] + h * 64, left - h * 64);
#pragma unroll
                    for (int y = 0; y < MT; ++y)
                        s[0].a[y][h] = codes16(pa[y] + h * 64, left - h * 64);
                }
                s[0].sa = load_global(psa);
                s[0].sb = load_global(psb);
                multiply_group<kFormatA, kWide>(s[0], acc);
            }
        }
        if (split == 1) {
            if (live) {
#pragma unroll
                for (int y = 0; y < MT; ++y)
#pragma unroll
                    for (int z = 0; z < NT; ++z) {
                        const int64_t i = i0 + y * 16 + row, j = j0 + z * 16 + quad * 4;
                        if (i < p.m)
                            store_out(p, i, j, acc[y][z], p.n - j);
                    }
            }
            continue;
        }
        __syncthreads();  // the last round's sums have been read
#pragma unroll
        for (int y = 0; y < MT; ++y)
#pragma unroll
            for (int z = 0; z < NT; ++z)
                part[wave][y * NT + z][lane] = acc[y][z];
        __syncthreads();
        for (int c = wave; c < slots * MT * NT; c += kSplitWaves) {
            const int sl = c / (MT * NT), yz = c % (MT * NT);
            const int64_t other = tile - slot + sl;
            if (other >= tiles)
                break;
            f32x4 sum = part[sl * split][yz][lane];
            for (int w = 1; w < split; ++w)
                sum += part[sl * split + w][yz][lane];
            const int64_t i = other % tiles_m * (16 * MT) + yz / NT * 16 + row;
            const int64_t j = other / tiles_m * (16 * NT) + yz % NT * 16 + quad * 4;
            if (i < p.m)
                store_out(p, i, j, sum, p.n - j);
        }
    }
}

// ------------------------------------------------------------- large products --

typedef float f32x16 __attribute__((ext_vector_type(16)));

// A workgroup of four waves computes 256 x 256 outputs, a wave 128 x 128 (the accumulators
// take half of a SIMD's registers; fewer outputs to a wave would read LDS more often than
// it can answer).  A group of both operands is 64 KB of LDS; one is multiplied while the
// next is loaded, and workgroups stay for several tiles, so that a tile's first loads fall
// under the last products of the one before.
//
// 16384 x 11008 x 4096: 617 to 654 us (by the card), 2.26 to 2.4 PFLOP/s, accumulating 757
// where 642 without; 16384 cubed 2.6 PFLOP/s; 11008 x 4096 x 8111 (e5m2) 306 to 325 us.  A
// group takes 1.55 us, 0.85 of them products at full clock.  Power is one bound: with zeros for codes a group takes 1.2 us, with random ones the clock falls to 1.9
// GHz (the matrix unit alone, fed from registers, reaches 4.95 and 4.0 PFLOP/s).  Issue is the
// other: without loads, reads of LDS and scales the same loop reaches 3.8.  A tile's end
// takes 9.5 us, in which all workgroups store 33 MB at once.  Measured and not kept: 16 x 16 x
// 128 instructions (682 us at a state of 655), scales read as bytes so that nothing waits at
// mid-group (1.5 to 3 % slower), results packed before they are turned (spills), loads by half
// groups, which gives them twice the time but makes twice the requests (700 us), and no wait
// for a tile's stores in the next one's first group (1 % slower).
constexpr int kBig = 256;                    // output rows and columns of a workgroup
constexpr int kOperandStage = kBig * kGroup;  // LDS bytes of one group of one operand
constexpr int kStage = 2 * kOperandStage;
constexpr int kScaleBlock = 4 * kBig * 4;     // LDS bytes of four groups' scales of both operands

// Byte offset of 16-byte piece `piece` (of 8) of row `row` in a staged operand: 16
// rows' pieces of one column of pieces fall into all 64 banks.
__device__ __forceinline__ int staged(int row, int piece) { return row * kGroup + ((piece ^ (row >> 1 & 7)) << 4); }

// 16 (or 4) bytes of each lane from `rsrc` at byte `at` + `k` into LDS from byte `to`
// + `plus` (a constant) on, lane after lane.  No vector register is written; the caller waits
// on vmcnt.  In assembly because the compiler would wait for every such load before any
// read of the same LDS array, also of another stage.  m0 holds the LDS address; the
// compiler keeps it for itself (hence its warning), and sets it anew wherever it needs it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t at, int k, uint32_t to, int plus)
{
    asm volatile("s_add_u32 m0, %3, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 :: "v"(at), "s"(rsrc), "s"(k), "s"(to), "i"(plus) : "m0", "scc");
}

__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t at, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :: "v"(at), "s"(rsrc), "s"(to) : "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t *p, int64_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0,
                                             (int)(uint32_t)(bytes < 0xfffffff0ll ? bytes : 0xfffffff0ll), 0x00027000);
}

// One operand of the tile that is being loaded: `here` of its kBig rows exist, the
// others are replaced by the last one (their results are dropped).
struct BigOperand {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t at[8];  // this lane's byte offsets in the eight blocks of 32 rows
    int32_t here;
    uint32_t row0;   // row of the scales that the tile's first row has
};

// Byte offset of row r (or of the last one).
__device__ __forceinline__ uint32_t row_at(int r, int here, int64_t ld)
{
    uint32_t x = (uint32_t)(r < here ? r : here - 1) * (uint32_t)ld;
    asm("" : "+v"(x));  // a 32-bit product
    return x;
}

__device__ __forceinline__ BigOperand big_operand(const uint8_t *q, int64_t ld, int64_t rows, int64_t k, int64_t r0,
                                                  int shift)
{
    const int t = threadIdx.x;
    BigOperand o;
    // up to the end of the 16-byte piece that holds the last code
    o.rsrc = buffer(q + r0 * ld, ((rows - 1 - r0) * ld + k + 15) & ~15ll);
    o.here = (int)(rows - r0 < kBig ? rows - r0 : kBig);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = j * 32 + (t >> 3);
        o.at[j] = row_at(r, o.here, ld) + (((t & 7) ^ (r >> 1 & 7)) << 4);
    }
    o.row0 = (uint32_t)(r0 >> shift);
    return o;
}

template <int kFormatA>
__global__ __launch_bounds__(kBlock, 1) void matmul_big_kernel(MatmulArgs p, int32_t tiles_m, int32_t tiles_n)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage];
    __shared__ __attribute__((aligned(1024))) uint32_t words[2 * kScaleBlock / 4];
    __shared__ uint32_t dump[64];  // what a prefetch brings; never read
    __shared__ f32x4 turn[4][32 * 8];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = (wave >> 1) * 128, wn = (wave & 1) * 128, row = lane & 31, half = lane >> 5;
    const int32_t tiles = tiles_m * tiles_n;
    const int32_t kb = (int32_t)p.kb;
    const int tail = (int)(p.k % kGroup);  // codes of a last, short group
    typedef __attribute__((address_space(3))) uint8_t *lds_address;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_address)lds;
    const uint32_t dump0 = (uint32_t)(uintptr_t)(lds_address)reinterpret_cast<uint8_t *>(dump);
    const uint32_t words0 = (uint32_t)(uintptr_t)(lds_address)reinterpret_cast<uint8_t *>(words);

    const auto tile_at = [&](int32_t v, int64_t *i0, int64_t *j0) {
        // one run of tiles per XCD; within it, strips of kStrip tile rows (8 and 16: slower)
        constexpr int32_t kStrip = 4;
        const int32_t x = v % kXcds, each = tiles / kXcds, more = tiles % kXcds;
        const int32_t i = x * each + (x < more ? x : more) + v / kXcds;
        const int32_t strip = i / (kStrip * tiles_n), r0 = strip * kStrip;
        const int32_t high = tiles_m - r0 < kStrip ? tiles_m - r0 : kStrip;
        const int32_t in = i - strip * kStrip * tiles_n;
        *i0 = (int64_t)(r0 + in % high) * kBig;
        *j0 = (int64_t)(in / high) * kBig;
    };

    // Scales: aligned words that hold the bytes of four groups (of two words, where
    // the bytes of a row start inside one), read no further than the word of the
    // array's last byte.
    const uint32_t low_a = (uint32_t)(uintptr_t)p.sa & 3, low_b = (uint32_t)(uintptr_t)p.sb & 3;
    const uint32_t bytes_a = (uint32_t)(p.m * p.kb) + low_a;
    const uint32_t bytes_b = (uint32_t)((((p.n - 1) >> p.b_shift) + 1) * p.kb) + low_b;
    const auto rsa = buffer(p.sa - low_a, (bytes_a + 3) & ~3u), rsb = buffer(p.sb - low_b, (bytes_b + 3) & ~3u);
    const bool split = (low_a | low_b | (p.kb & 3)) != 0;

    // The loader: the tile and group that are loaded next, two groups ahead.  After the
    // last tile it goes on with that tile's operands; nothing uses them.
    int32_t load_tile = blockIdx.x, load_g = 0;
    uint32_t load_words = 0;  // half of `words` that is filled next
    BigOperand oa, ob;
    uint32_t ahead;           // this lane's row for prefetches
    const auto open_tile = [&]() {
        int64_t i0, j0;
        tile_at(load_tile, &i0, &j0);
        oa = big_operand(p.a, p.lda, p.m, p.k, i0, 0);
        ob = big_operand(p.b, p.ldb, p.n, p.k, j0, p.b_shift);
        // a quarter of the rows of each operand: neighbouring tiles share the rest
        const int quarter = (int)((wave < 2 ? j0 : i0) / kBig & 3) * 64 + (wave & 1) * 32 + lane;
        ahead = lane < 32 ? row_at(quarter, wave < 2 ? oa.here : ob.here, wave < 2 ? p.lda : p.ldb) : kNowhere;
    };
    const auto load_piece = [&](uint32_t stage, int j) {  // j-th of 16 pieces of this wave
        const BigOperand &o = j & 1 ? oa : ob;
        load16_to_lds(o.rsrc, o.at[j / 2], load_g * kGroup, lds0 + stage + wave * 1024,
                      (j & 1 ? 0 : kOperandStage) + j / 2 * 4096);
    };
    const auto load_done = [&]() {
        if (load_g % 4 == 0) {
            const uint32_t to = words0 + load_words + wave * 256, g = (uint32_t)load_g;
            const uint32_t ra = oa.row0 + (uint32_t)(t < oa.here ? t : oa.here - 1);
            const uint32_t rb = ob.row0 + ((uint32_t)(t < ob.here ? t : ob.here - 1) >> p.b_shift);
            const uint32_t xa = (ra * (uint32_t)kb + g + low_a) & ~3u, xb = (rb * (uint32_t)kb + g + low_b) & ~3u;
            load4_to_lds(rsa, xa, to);
            load4_to_lds(rsb, xb, to + 2048);
            if (split) {
                const uint32_t last_a = (bytes_a - 1) & ~3u, last_b = (bytes_b - 1) & ~3u;
                load4_to_lds(rsa, xa < last_a ? xa + 4 : last_a, to + 1024);
                load4_to_lds(rsb, xb < last_b ? xb + 4 : last_b, to + 3 * 1024);
            }
            load_words ^= kScaleBlock;
        }
        if (++load_g == kb) {
            load_g = 0;
            load_tile += gridDim.x;
            if (load_tile < tiles)
                open_tile();
        }
    };
    // Brings the lines of the group kAhead further on into the L2, where the loads of
    // the XCD's workgroups, which run side by side, would all wait for them (12 % of the
    // time).
    const auto prefetch = [&]() {
        constexpr int32_t kAhead = 1;
        const int32_t g = load_g + kAhead;
        load4_to_lds(wave < 2 ? oa.rsrc : ob.rsrc, group_of_row(ahead, g, kb), dump0);
    };
    // zeros from code `tail` on in every row of a stage
    const auto clear_tail = [&](uint32_t at) {
        for (int r = t; r < 2 * kBig; r += kBlock)
            for (int q = tail / 4; q < kGroup / 4; ++q) {
                uint32_t *w = reinterpret_cast<uint32_t *>(lds + at + staged(r, q / 4) + q % 4 * 4);
                *w = q == tail / 4 ? *w & ((1u << (8 * (tail % 4))) - 1u) : 0u;
            }
        __syncthreads();
    };

    i32x8 fa[2][4], fb[2][4];
    uint32_t ca[4], cb[4];  // scales of the current group, in the low byte
    f32x16 acc[4][4];
    const auto read_one = [&](uint32_t stage, int f, int i) {  // i-th of 8 operands
        const int x = i / 2, r = (i & 1 ? wm : kBig + wn) + x * 32 + row;
        const i32x8 v = operand(*reinterpret_cast<const u32x4 *>(lds + stage + staged(r, f * 4 + half * 2)),
                                *reinterpret_cast<const u32x4 *>(lds + stage + staged(r, f * 4 + half * 2 + 1)));
        (i & 1 ? fa[f][x] : fb[f][x]) = v;
    };
    const auto multiply_one = [&](int f, int i) {
        const int x = i & 3, y = i >> 2;
        acc[x][y] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[f][x], fa[f][y], acc[x][y], ZR_E4M3, kFormatA,
                                                                    0, (int)cb[x], 0, (int)ca[y]);
        asm volatile("" : "+a"(acc[x][y]));  // here, not where the sum is next used
    };
    // The scales of four groups from `words`, for a tile whose first rows' scales are
    // row_a and row_b.
    const auto read_scales = [&](uint32_t from, uint32_t row_a, uint32_t row_b, uint32_t *wa, uint32_t *wb) {
        const uint32_t *w = words + from / 4;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            wa[x] = w[wm + x * 32 + row];
            wb[x] = w[512 + wn + x * 32 + row];
        }
        if (split) {  // rows 32 apart start at the same byte of a word
            const uint32_t sa = (row_a + wm + row) * (uint32_t)kb + low_a;
            const uint32_t sb = (row_b + ((wn + row) >> p.b_shift)) * (uint32_t)kb + low_b;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                wa[x] = __builtin_amdgcn_alignbyte(w[256 + wm + x * 32 + row], wa[x], sa);
                wb[x] = __builtin_amdgcn_alignbyte(w[768 + wn + x * 32 + row], wb[x], sb);
            }
        }
    };
    const auto clear_acc = [&]() {
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                acc[x][y] = f32x16{};
    };

    f32x4 *const mine = turn[wave];
    int32_t tile = blockIdx.x;
    if (tile >= tiles)
        return;
    open_tile();
#pragma unroll
    for (int j = 0; j < 16; ++j)
        load_piece(0, j);
    load_done();
    clear_acc();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kWaitAll);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    uint32_t stage = 0, from = 0, row_a = oa.row0, row_b = ob.row0;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        load_piece(kStage, j);
    load_done();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        read_one(0, 0, i);
    read_scales(from, row_a, row_b, ca, cb);
    from ^= kScaleBlock;
    for (;;) {
        for (int32_t g = 0; g < kb; ++g) {
            const bool last = g + 1 == kb;
            // first half of the group, from registers; the second half's operands are read
            prefetch();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                multiply_one(0, i);
                if (i < 8)
                    read_one(stage, 1, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            // the next group has landed (all but the prefetch), in every wave, and this
            // group's stage has been read by all
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(kWaitStage);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            if (tail && g + 2 == kb)
                clear_tail(stage ^ kStage);
            const bool fresh = last || (g & 3) == 3;
            uint32_t wa[4], wb[4];
            if (fresh) {  // of the next four groups, or of the next tile, which is already being loaded
                row_a = last ? oa.row0 : row_a;
                row_b = last ? ob.row0 : row_b;
                read_scales(from, row_a, row_b, wa, wb);
                from ^= kScaleBlock;
            } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    wa[x] = ca[x] >> 8;
                    wb[x] = cb[x] >> 8;
                }
            }
            // second half; the next group's first operands are read, and the group after
            // it is loaded into this one's place
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                multiply_one(1, i);
                load_piece(stage, i);
                if (i < 8)
                    read_one(stage ^ kStage, 0, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            load_done();
            stage ^= kStage;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                ca[x] = wa[x];
                cb[x] = wb[x];
            }
        }
        // Results: 32 x 32 at a time through the wave's own LDS (16-byte pieces,
        // permuted by the row), so that four lanes store 64 bytes of a row.
        int64_t i0, j0;
        tile_at(tile, &i0, &j0);
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16 &v = acc[x][y];  // columns 8 q + 4 half ... of the 32
                    mine[row * 8 + ((q * 2 + half) ^ (row & 7))] = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll 1
                for (int r = lane >> 2; r < 32; r += 16) {
                    const int piece = (lane & 3) * 2;
                    const f32x4 lo = mine[r * 8 + (piece ^ (r & 7))], hi = mine[r * 8 + ((piece + 1) ^ (r & 7))];
                    const int64_t i = i0 + wm + y * 32 + r, j = j0 + wn + x * 32 + piece * 4;
                    if (i < p.m)
                        store_out(p, i, j, lo, hi, p.n - j);
                }
                __builtin_amdgcn_wave_barrier();
            }
        tile += gridDim.x;
        if (tile >= tiles)
            break;
        clear_acc();
    }
    __builtin_amdgcn_s_waitcnt(kWaitAll);  // no load into LDS outlives the workgroup
}

// ------------------------------------------------------------ middling products --

// A workgroup computes 128 x 128 outputs, a wave 64 x 64, through a ring of kRing
// groups of both operands in LDS, with the operands of the next group read into
// registers while one is multiplied.  For products with too few 256 x 256 tiles to
// occupy the chip, and for fp32 outputs.  A group takes 0.5 us for 0.21 us of products:
// the one wave of a SIMD issues reads, loads and control one after another (the order in
// which they are spread between the products makes no difference).
// 1000 x 4096 x 4096 24 us; fp32 outputs, bound by the matrix unit's bf16 rate and by the
// widening: 11008 x 4096 x 8192 739 to 757 us (by the card), 1.0 PFLOP/s; accumulating 825.
constexpr int kMid = 128;
constexpr int kRing = 4;
constexpr int kMidOperand = kMid * kGroup;
constexpr int kMidStage = 2 * kMidOperand;
constexpr int kMidWords = 2 * kMid * 16;      // LDS bytes of eight groups' scales of both operands
constexpr int kMidWordRing = 8;               // more than the blocks of eight (or fewer) groups in use at once
constexpr int kWaitRing = 0x4070;             // s_waitcnt vmcnt(16) lgkmcnt(0): all but two stages

template <int kFormatA, bool kWide>
__global__ __launch_bounds__(kBlock, 1) void matmul_mid_kernel(MatmulArgs p, int32_t tiles_m, int32_t tiles_n)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[kRing * kMidStage];
    __shared__ __attribute__((aligned(1024))) uint8_t words[kMidWordRing * kMidWords];
    const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64, row = lane & 15, quad = lane >> 4;
    const int32_t tiles = tiles_m * tiles_n, kb = (int32_t)p.kb;
    const int tail = (int)(p.k % kGroup);
    typedef __attribute__((address_space(3))) uint8_t *lds_address;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_address)lds, words0 = (uint32_t)(uintptr_t)(lds_address)words;

    // one run of tiles per XCD, down the columns of tiles: they share their rows of B
    const auto tile_at = [&](int32_t v, int64_t *i0, int64_t *j0) {
        const int32_t x = v % kXcds, each = tiles / kXcds, more = tiles % kXcds;
        const int32_t i = x * each + (x < more ? x : more) + v / kXcds;
        *i0 = (int64_t)(i % tiles_m) * kMid;
        *j0 = (int64_t)(i / tiles_m) * kMid;
    };

    // Scales: the 16 bytes from the word on that holds a row's first byte of eight
    // groups; words behind the array's last one read as zeros.
    const uint32_t low_a = (uint32_t)(uintptr_t)p.sa & 3, low_b = (uint32_t)(uintptr_t)p.sb & 3;
    const auto rsa = buffer(p.sa - low_a, (p.m * kb + low_a + 3) & ~3ll);
    const auto rsb = buffer(p.sb - low_b, ((((p.n - 1) >> p.b_shift) + 1) * kb + low_b + 3) & ~3ll);

    // The loader, kRing groups ahead; after the last tile it goes on with that tile's
    // operands, which nothing uses.
    int32_t load_tile = blockIdx.x, load_g = 0;
    uint32_t load_words = 0;
    __amdgpu_buffer_rsrc_t ra, rb;
    uint32_t at_a[4], at_b[4], at_s;
    const auto open_tile = [&]() {
        int64_t i0, j0;
        tile_at(load_tile, &i0, &j0);
        ra = buffer(p.a + i0 * p.lda, ((p.m - 1 - i0) * p.lda + p.k + 15) & ~15ll);
        rb = buffer(p.b + j0 * p.ldb, ((p.n - 1 - j0) * p.ldb + p.k + 15) & ~15ll);
        const int here_a = (int)(p.m - i0 < kMid ? p.m - i0 : kMid), here_b = (int)(p.n - j0 < kMid ? p.n - j0 : kMid);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = j * 32 + (t >> 3);
            const uint32_t piece = (uint32_t)((t & 7) ^ (r >> 1 & 7)) << 4;
            at_a[j] = row_at(r, here_a, p.lda) + piece;
            at_b[j] = row_at(r, here_b, p.ldb) + piece;
        }
        // waves 0 and 1 bring A's scales, waves 2 and 3 B's
        const int r = t & 127;
        const uint32_t sr = wave < 2 ? (uint32_t)i0 + (uint32_t)(r < here_a ? r : here_a - 1)
                                     : (uint32_t)(j0 + (r < here_b ? r : here_b - 1)) >> p.b_shift;
        at_s = sr * (uint32_t)kb + (wave < 2 ? low_a : low_b);
    };
    const auto load_piece = [&](uint32_t stage, int j) {  // j-th of 8 pieces of this wave
        load16_to_lds(j & 1 ? ra : rb, j & 1 ? at_a[j / 2] : at_b[j / 2], load_g * kGroup,
                      lds0 + stage + wave * 1024, (j & 1 ? 0 : kMidOperand) + j / 2 * 4096);
    };
    const auto load_done = [&]() {
        if (load_g % 8 == 0) {
            load16_to_lds(wave < 2 ? rsa : rsb, (at_s + (uint32_t)load_g) & ~3u, 0, words0 + load_words + wave * 1024,
                          0);
            load_words = load_words == (kMidWordRing - 1) * kMidWords ? 0 : load_words + kMidWords;
        }
        if (++load_g == kb) {
            load_g = 0;
            load_tile += gridDim.x;
            if (load_tile < tiles)
                open_tile();
        }
    };
    const auto clear_tail = [&](uint32_t at) {
        for (int q = tail / 4; q < kGroup / 4; ++q) {
            uint32_t *w = reinterpret_cast<uint32_t *>(lds + at + staged(t, q / 4) + q % 4 * 4);
            *w = q == tail / 4 ? *w & ((1u << (8 * (tail % 4))) - 1u) : 0u;
        }
        __syncthreads();
    };

    SplitGroup<4, 4> f[2];
    uint32_t ca[2][4], cb[2][4];
    f32x4 acc[4][4];
    // i-th of 16 reads of the operands of the group at `stage`
    const auto read_one = [&](uint32_t stage, int e, int i) {
        const int x = i >> 2, piece = quad + (i >> 1 & 1) * 4;
        if (i & 1)
            f[e].a[x][i >> 1 & 1] = *reinterpret_cast<const u32x4 *>(lds + stage + staged(wm + x * 16 + row, piece));
        else
            f[e].b[x][i >> 1 & 1] = *reinterpret_cast<const u32x4 *>(lds + stage + staged(kMid + wn + x * 16 + row, piece));
    };
    // the scales of the next group: its place in `words` and this lane's bytes in it
    uint32_t word = 0, first_a = 0, first_b = 0;
    const auto first_bytes = [&](int64_t i0, int64_t j0) {  // rows 16 apart start at the same byte of a word
        const int64_t ia = i0 + wm + row, jb = j0 + wn + row;
        first_a = (uint32_t)(wm + row) * 16 + (((uint32_t)ia * (uint32_t)kb + low_a) & 3);
        first_b = (uint32_t)(kMid + wn + row) * 16 + (((uint32_t)(jb >> p.b_shift) * (uint32_t)kb + low_b) & 3);
    };
    const auto read_scale = [&](int e, int i, int32_t g) {  // i-th of 8
        const uint8_t *w = words + word + (g & 7) + i / 2 * 256;
        (i & 1 ? ca : cb)[e][i / 2] = w[i & 1 ? first_a : first_b];
    };
    const auto clear_acc = [&]() {
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                acc[y][z] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                asm volatile("" : "+a"(acc[y][z]));  // in the registers that the products use
            }
    };

    int32_t tile = blockIdx.x;
    if (tile >= tiles)
        return;
    open_tile();
#pragma unroll
    for (int s = 0; s < kRing; ++s) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            load_piece(s * kMidStage, j);
        load_done();
    }
    clear_acc();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(kWaitAll);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (tail && kb == 1)
        clear_tail(0);
    if (tail && kb <= 2)
        clear_tail(kMidStage);
    int64_t i0, j0;
    tile_at(tile, &i0, &j0);
    first_bytes(i0, j0);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        read_one(0, 0, i);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        read_scale(0, i, 0);
    __syncthreads();  // every wave has read the first group before another is loaded into its place
    uint32_t stage = 0;
    int32_t g = 0, two = 2 % kb;  // the group that is multiplied, and the one two stages on

    // Group g is multiplied from registers e while the next group's operands are read
    // into the other ones and the group kRing on is loaded into g's place.
    const auto step = [&](int e) {
        const uint32_t next = (stage + kMidStage) % (kRing * kMidStage);
        const bool last = g + 1 == kb;
        const int32_t gn = last ? 0 : g + 1;
        if (gn % 8 == 0) {
            word = word == (kMidWordRing - 1) * kMidWords ? 0 : word + kMidWords;
            if (last && tile + (int32_t)gridDim.x < tiles) {
                tile_at(tile + gridDim.x, &i0, &j0);
                first_bytes(i0, j0);
            }
        }
        bf16x8 b[4], a;
        Lowered low;
        bool far = false;
        if constexpr (kWide)
            far = lower_scales<true, kFormatA>(ca[e], cb[e], acc, low);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if constexpr (!kWide) {
                const int y = i >> 2, z = i & 3;
                acc[y][z] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    operand(f[e].b[z][0], f[e].b[z][1]), operand(f[e].a[y][0], f[e].a[y][1]), acc[y][z], ZR_E4M3,
                    kFormatA, 0, (int)cb[e][z], 0, (int)ca[e][y]);
                asm volatile("" : "+a"(acc[y][z]));
            } else {  // 8 codes of each lane, one row of tiles
                const int q = i >> 2, y = i & 3, h = q / 2, c = q % 2 * 2;
                if (y == 0)
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        b[z] = widen8<ZR_E4M3>(f[e].b[z][h][c], f[e].b[z][h][c + 1], __uint_as_float(cb[e][z] << 23));
                a = widen8<kFormatA>(f[e].a[y][h][c], f[e].a[y][h][c + 1], __uint_as_float(ca[e][y] << 23));
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    acc[y][z] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[z], a, acc[y][z], 0, 0, 0);
                    asm volatile("" : "+a"(acc[y][z]));
                }
            }
            if (i < 8) {
                read_one(next, e ^ 1, 2 * i);
                read_one(next, e ^ 1, 2 * i + 1);
                read_scale(e ^ 1, i, gn);
            } else {
                load_piece(stage, i - 8);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kWide) {
            if (far)
                raise_sums<true>(acc, low);
            pin(acc);
        }
        load_done();
        // two stages on has landed, in every wave, and the next one has been read by all
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(kWaitRing);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
#pragma unroll
        for (int x = 0; x < 4; ++x)  // whole words from here on, not bytes to be widened at every use
            asm volatile("" : "+v"(ca[e ^ 1][x]), "+v"(cb[e ^ 1][x]));
        if (tail && two + 1 == kb)
            clear_tail((stage + 2 * kMidStage) % (kRing * kMidStage));
        two = two + 1 == kb ? 0 : two + 1;
        stage = next;
        g = gn;
    };
    // Stores a finished tile; false after the last one.
    int64_t out_i, out_j;
    tile_at(tile, &out_i, &out_j);
    const auto finish = [&]() {
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                const int64_t i = out_i + wm + y * 16 + row, j = out_j + wn + z * 16 + quad * 4;
                if (i < p.m)
                    store_out(p, i, j, acc[y][z], p.n - j);
            }
        tile += gridDim.x;
        if (tile >= tiles)
            return false;
        out_i = i0;
        out_j = j0;
        clear_acc();
        return true;
    };
    for (;;) {
        step(0);
        if (g == 0 && !finish())
            break;
        step(1);
        if (g == 0 && !finish())
            break;
    }
    __builtin_amdgcn_s_waitcnt(kWaitAll);  // no load into LDS outlives the workgroup
}

// ------------------------------------------------ few tiles, a long summed axis --

// A workgroup computes 128 x 64 outputs with two teams of four waves, one for each half
// of the groups: a wave of a team computes 64 x 32, two waves to a SIMD, so that one
// multiplies while the other issues its loads.  Each team has a ring of three groups of
// both operands in LDS; at the end the teams' sums meet there, each team stores half.
// Against four waves alone: a single wave to a SIMD issues its ~110 instructions of a
// group one after another, 0.41 us for 0.11 us of products (333 x 4096 x 11008 with 128 x
// 128 outputs: 54 us); the teams take 40 us, now bound by the loads (24 us with the same
// loop that loads nothing; 29 us with operands in the last-level cache).  Bringing lines
// into the L2 ahead of the loads, shared out or not, made it slower (43, 52 us).
constexpr int kPairRows = 128, kPairCols = 64;
constexpr int kPairThreads = 512;
constexpr int kPairRing = 3;
constexpr int kPairStage = (kPairRows + kPairCols) * kGroup;  // LDS bytes of a group of both operands, A first
constexpr int kPairWords = 256 * 16;                          // of eight groups' scales
constexpr int kPairWait = 0x0076;  // s_waitcnt vmcnt(6) lgkmcnt(0): all but the last stage

template <int kFormatA, bool kWide>
__global__ __launch_bounds__(kPairThreads, 2) void matmul_pair_kernel(MatmulArgs p, int32_t tiles_m, int32_t tiles_n)
{
    __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kPairRing * kPairStage];
    __shared__ __attribute__((aligned(1024))) uint8_t words[2 * 2 * kPairWords];
    const int t = threadIdx.x & 255, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int team = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    const int wm = (wave >> 1) * 64, wn = (wave & 1) * 32, row = lane & 15, quad = lane >> 4;
    const int32_t tiles = tiles_m * tiles_n, kb = (int32_t)p.kb, half = (kb + 1) / 2;
    const int32_t first = team * half, count = team ? kb - half : half;
    const int tail = (int)(p.k % kGroup), tail_team = kb > 1, tail_at = kb > 1 ? kb - half - 1 : 0;
    typedef __attribute__((address_space(3))) uint8_t *lds_address;
    const uint32_t base = (uint32_t)team * (kPairRing * kPairStage), word_base = (uint32_t)team * (2 * kPairWords);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_address)lds + base + (uint32_t)wave * 1024;
    const uint32_t words0 = (uint32_t)(uintptr_t)(lds_address)words + word_base;

    // Scales: the 16 bytes from the word on that holds a row's first byte of eight
    // groups; words behind the array's last one read as zeros.
    const uint32_t low_a = (uint32_t)(uintptr_t)p.sa & 3, low_b = (uint32_t)(uintptr_t)p.sb & 3;
    const auto rsa = buffer(p.sa - low_a, (p.m * kb + low_a + 3) & ~3ll);
    const auto rsb = buffer(p.sb - low_b, ((((p.n - 1) >> p.b_shift) + 1) * kb + low_b + 3) & ~3ll);

    for (int32_t v = blockIdx.x; v < tiles; v += gridDim.x) {
        // one run of tiles per XCD, down the columns of tiles: they share their rows of B
        const int32_t x = v % kXcds, each = tiles / kXcds, more = tiles % kXcds;
        const int32_t tile = x * each + (x < more ? x : more) + v / kXcds;
        const int64_t i0 = (int64_t)(tile % tiles_m) * kPairRows, j0 = (int64_t)(tile / tiles_m) * kPairCols;

        // The loader.  Rows that do not exist are replaced by the last one, and so are
        // groups behind the team's last one, which nothing uses.
        const int here_a = (int)(p.m - i0 < kPairRows ? p.m - i0 : kPairRows);
        const int here_b = (int)(p.n - j0 < kPairCols ? p.n - j0 : kPairCols);
        const auto ra = buffer(p.a + i0 * p.lda, ((here_a - 1) * p.lda + p.k + 15) & ~15ll);
        const auto rb = buffer(p.b + j0 * p.ldb, ((here_b - 1) * p.ldb + p.k + 15) & ~15ll);
        uint32_t at[6];
#pragma unroll
        for (int j = 0; j < 6; ++j) {
            const int r = (j < 4 ? j : j - 4) * 32 + (t >> 3);
            at[j] = (j < 4 ? row_at(r, here_a, p.lda) : row_at(r, here_b, p.ldb)) + ((uint32_t)((t & 7) ^ (r >> 1 & 7)) << 4);
        }
        // waves 0 and 1 bring A's scales, wave 2 B's
        const uint32_t scale_row = wave < 2 ? (uint32_t)i0 + (uint32_t)(t < here_a ? t : here_a - 1)
                                            : (uint32_t)(j0 + (lane < here_b ? lane : here_b - 1)) >> p.b_shift;
        const uint32_t at_s = scale_row * (uint32_t)kb + (wave < 2 ? low_a : low_b) + (uint32_t)first;
        const auto group_at = [&](int32_t g) { return (first + (g < count ? g : count - 1)) * kGroup; };
        const auto load_piece = [&](uint32_t stage, int32_t g, int j) {
            load16_to_lds(j < 4 ? ra : rb, at[j], group_at(g), lds0 + stage, j * 4096);
        };
        const auto load_scales = [&](int32_t g) {  // of the eight groups from g on
            if (wave < 3)
                load16_to_lds(wave < 2 ? rsa : rsb, (at_s + (uint32_t)g) & ~3u, 0,
                              words0 + (uint32_t)(g & 8) * (kPairWords / 8) + (uint32_t)wave * 1024, 0);
        };
        // Zeros in place of what lies behind the rows' ends in the last group.
        const auto clear_tail = [&](uint32_t stage) {
            for (int q = t < kPairRows + kPairCols ? tail / 4 : kGroup / 4; q < kGroup / 4; ++q) {
                uint32_t *w = reinterpret_cast<uint32_t *>(lds + base + stage + staged(t, q / 4) + q % 4 * 4);
                *w = q == tail / 4 ? *w & ((1u << (8 * (tail % 4))) - 1u) : 0u;
            }
        };

        SplitGroup<4, 2> f[2];
        uint32_t ca[2][4], cb[2][2];
        f32x4 acc[4][2];
        // i-th of 12 reads of the operands of the group at `stage`
        const auto read_one = [&](uint32_t stage, int e, int i) {
            const bool b = i < 8 && i % 2 == 0;
            const int j = i < 8 ? i / 2 : i - 4, x = j / 2, piece = quad + j % 2 * 4;
            (b ? f[e].b[x] : f[e].a[x])[j % 2] = *reinterpret_cast<const u32x4 *>(
                lds + base + stage + staged((b ? kPairRows + wn : wm) + x * 16 + row, piece));
        };
        // this lane's bytes in eight groups' scales; rows 16 apart start at the same byte of a word
        const uint32_t ia = (uint32_t)i0 + wm + row, jb = (uint32_t)(j0 + wn + row) >> p.b_shift;
        const uint32_t first_a = word_base + (uint32_t)(wm + row) * 16 + ((ia * (uint32_t)kb + low_a + first) & 3);
        const uint32_t first_b = word_base + (uint32_t)(kPairRows + wn + row) * 16 + ((jb * (uint32_t)kb + low_b + first) & 3);
        const auto read_scale = [&](int e, int i, int32_t g) {  // i-th of 6
            const uint8_t *w = words + (uint32_t)(g & 8) * (kPairWords / 8) + (g & 7);
            if (i < 2)
                cb[e][i] = w[first_b + i * 256];
            else
                ca[e][i - 2] = w[first_a + (i - 2) * 256];
        };

#pragma unroll
        for (int s = 0; s < kPairRing; ++s) {
#pragma unroll
            for (int j = 0; j < 6; ++j)
                load_piece(s * kPairStage, s, j);
            if (s == 0)
                load_scales(0);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                acc[y][z] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                asm volatile("" : "+a"(acc[y][z]));  // in the registers that the products use
            }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(kWaitAll);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (tail && tail_at <= 1) {
            if (team == tail_team)
                clear_tail(tail_at * kPairStage);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 12; ++i)
            read_one(0, 0, i);
#pragma unroll
        for (int i = 0; i < 6; ++i)
            read_scale(0, i, 0);
        __syncthreads();  // every wave has read the first group before another is loaded into its place
        uint32_t stage = 0;
        int32_t g = 0;

        // Group g is multiplied from registers e while the next group's operands are read
        // into the other ones and the group kPairRing on is loaded into g's place.
        const auto step = [&](int e) {
            const uint32_t next = stage == (kPairRing - 1) * kPairStage ? 0 : stage + kPairStage;
            constexpr int kParts = kWide ? 16 : 8, kHalf = kParts / 2;
            bf16x8 b[2], a;
            Lowered low;
            bool far = false;
            if constexpr (kWide)
                far = lower_scales<true, kFormatA>(ca[e], cb[e], acc, low);
#pragma unroll
            for (int i = 0; i < kParts; ++i) {
                if constexpr (!kWide) {
                    const int y = i / 2, z = i % 2;
                    acc[y][z] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        operand(f[e].b[z][0], f[e].b[z][1]), operand(f[e].a[y][0], f[e].a[y][1]), acc[y][z], ZR_E4M3,
                        kFormatA, 0, (int)cb[e][z], 0, (int)ca[e][y]);
                    asm volatile("" : "+a"(acc[y][z]));
                } else {  // 8 codes of each lane, one row of tiles
                    const int q = i >> 2, y = i & 3, h = q / 2, c = q % 2 * 2;
                    if (y == 0)
#pragma unroll
                        for (int z = 0; z < 2; ++z)
                            b[z] = widen8<ZR_E4M3>(f[e].b[z][h][c], f[e].b[z][h][c + 1], __uint_as_float(cb[e][z] << 23));
                    a = widen8<kFormatA>(f[e].a[y][h][c], f[e].a[y][h][c + 1], __uint_as_float(ca[e][y] << 23));
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        acc[y][z] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[z], a, acc[y][z], 0, 0, 0);
                        asm volatile("" : "+a"(acc[y][z]));
                    }
                }
                if (i < kHalf) {
#pragma unroll
                    for (int x = i * 6 / kHalf; x < (i + 1) * 6 / kHalf; ++x)
                        load_piece(stage, g + kPairRing, x);
                }
                if (i == kHalf && (g + kPairRing) % 8 == 0)
                    load_scales(g + kPairRing);
#pragma unroll
                for (int x = i * 12 / kParts; x < (i + 1) * 12 / kParts; ++x)
                    read_one(next, e ^ 1, x);
#pragma unroll
                for (int x = i * 6 / kParts; x < (i + 1) * 6 / kParts; ++x)
                    read_scale(e ^ 1, x, g + 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (kWide) {
                if (far)
                    raise_sums<true>(acc, low);
                pin(acc);
            }
            // two stages on has landed, in every wave, and the next one has been read by all
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_waitcnt(kPairWait);
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
#pragma unroll
            for (int x = 0; x < 4; ++x) {  // whole words from here on, not bytes to be widened at every use
                asm volatile("" : "+v"(ca[e ^ 1][x]));
                if (x < 2)
                    asm volatile("" : "+v"(cb[e ^ 1][x]));
            }
            if (tail && tail_at == g + 2) {
                if (team == tail_team)
                    clear_tail(next == (kPairRing - 1) * kPairStage ? 0 : next + kPairStage);
                __syncthreads();
            }
            stage = next;
            ++g;
        };
        for (;;) {
            if (g >= count)
                break;
            step(0);
            if (g >= count)
                break;
            step(1);
        }
        if (count < half)  // the other team's last step
            __builtin_amdgcn_s_barrier();

        // The teams' sums: each hands half of its rows to the other.
        __builtin_amdgcn_s_waitcnt(kWaitAll);  // no load into LDS is under way
        __syncthreads();
        f32x4 *const swap = reinterpret_cast<f32x4 *>(lds) + wave * 64 + lane;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int z = 0; z < 2; ++z)
                swap[(team * 4 + y * 2 + z) * 256] = team ? acc[y][z] : acc[y + 2][z];
        __syncthreads();
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const f32x4 v4 = (team ? acc[y + 2][z] : acc[y][z]) + swap[((team ^ 1) * 4 + y * 2 + z) * 256];
                const int64_t i = i0 + wm + (y + team * 2) * 16 + row, j = j0 + wn + z * 16 + quad * 4;
                if (i < p.m)
                    store_out(p, i, j, v4, p.n - j);
            }
        __syncthreads();  // before the next tile's loads
    }
}

namespace {

template <int kFormatA, bool kWide, int MT, int NT, int kAhead>
zr_status split_run(const MatmulArgs &p, hipStream_t st)
{
    const int64_t tm = (p.m + 16 * MT - 1) / (16 * MT), tn = (p.n + 16 * NT - 1) / (16 * NT), tiles = tm * tn;
    // enough waves for every SIMD twice, none without a group
    int32_t split = kSplitWaves;
    while (split > 1 && (tiles * split / 2 >= kCus * kSplitWaves || p.kb < split))
        split /= 2;
    const int64_t slots = kSplitWaves / split, rounds = (tiles + slots - 1) / slots;
    return launch(matmul_split_kernel<kFormatA, kWide, MT, NT, kAhead>, grid_of(rounds), dim3(kSplitThreads), 0, st, p,
                  split, tm, rounds);
}

// Which kernel.  Times in us on MI355X, operands rotated through more than the caches:
//  - A split wave's tile is the smallest that leaves at most one workgroup to a compute
//    unit.  1 x 4096 x 4096: 16 x 16 outputs 6.6, 16 x 32 8.3, 32 x 32 8.9; 1 x 11008 x 4096
//    (m x n x k): 16.4, 15.2 and, with 16 x 64, 13.7; 32 x 11008 x 4096: 32 x 32 23, 32 x 64
//    18; 64 x 4096 x 4096: 32 x 32 12.5, 64 x 64 20.8.  At the upper end of 32 x 64 the two teams
//    would be faster (128 x 4096 x 4096: 16.5 against 13.5).
//  - More tiles than that go to the LDS kernels (250 x 4096 x 11008: 64 x 64 a wave 48, 128 x 64
//    and two teams 42; 17 x 32000 x 4096: 32 x 64 37, 128 x 128 34.5; 64 x 32000 x 4096: 62 and 39),
//    up to 16 rows excepted, which are bound by B's bytes either way (1 x 32000 x 4096:
//    16 x 32 26, 16 x 64 35).
//  - One round of 128 x 64 tiles goes to the two teams: 333 x 4096 x 4096 14.4 (128 x 128 by four
//    waves 21.3), with fp32 outputs 21 (39); 1000 x 1000 x 4000 14.9 (64 x 64 a wave 21.7).  Two
//    rounds of them lose to one of 128 x 128: 1000 x 4096 x 4096 29 and 24 (fp32 45 and 41).
//  - A round of 256 x 256 tiles costs 9/4 rounds of 128 x 128 (one round each, k = 4096: 52
//    and 24; 2048 x 4096 x 4096: 54 against 47 for two; 4096 x 4096 x 4096: 66 against 97 for four).
//    A last round of few tiles is where the rule is off by most: 1500 x 11008 x 4096, two
//    rounds of 256 x 256 for 258 tiles, takes 108 and would take 100 in five of 128 x 128.
// The LDS kernels load 16 bytes at a time and index a tile's rows in 32 bits; what does
// not meet that stays with the split waves.
template <int kFormatA, bool kWide>
zr_status matmul_run(const MatmulArgs &p, hipStream_t st)
{
    const auto tiles = [&](int64_t rows, int64_t cols) {
        return ((p.m + rows - 1) / rows) * ((p.n + cols - 1) / cols);
    };
    const auto rounds = [](int64_t n) { return (n + kCus - 1) / kCus; };
    const bool aligned = aligned_to(p.a, 16) && aligned_to(p.b, 16) && (p.lda % 16 == 0 || p.m == 1) &&
                         (p.ldb % 16 == 0 || p.n == 1) && p.lda < (1 << 23) && p.ldb < (1 << 23) &&
                         p.m * p.kb < (1ll << 31) && p.n * p.kb < (1ll << 31) && p.kb > 0;
    if (tiles(16, 16) <= kCus)
        return split_run<kFormatA, kWide, 1, 1, 2>(p, st);
    if (tiles(16, 32) <= kCus)
        return split_run<kFormatA, kWide, 1, 2, 2>(p, st);
    if (p.m <= 16)
        return tiles(16, 64) <= kCus ? split_run<kFormatA, kWide, 1, 4, 2>(p, st)
                                     : split_run<kFormatA, kWide, 1, 2, 2>(p, st);
    if (tiles(32, 32) <= kCus)
        return split_run<kFormatA, kWide, 2, 2, 2>(p, st);
    if (tiles(32, 64) <= kCus)
        return split_run<kFormatA, kWide, 2, 4, 2>(p, st);
    if (!aligned)
        return split_run<kFormatA, kWide, 4, 4, 1>(p, st);
    const int64_t pair = tiles(kPairRows, kPairCols);
    if (pair <= kCus)
        return launch(matmul_pair_kernel<kFormatA, kWide>, grid_of(pair), dim3(kPairThreads), 0, st, p,
                      (int32_t)((p.m + kPairRows - 1) / kPairRows), (int32_t)((p.n + kPairCols - 1) / kPairCols));
    const int64_t big = tiles(kBig, kBig), mid = tiles(kMid, kMid);
    if constexpr (!kWide) {
        if (p.kb > 1 && 9 * rounds(big) <= 4 * rounds(mid))
            return launch(matmul_big_kernel<kFormatA>, grid_of(big < kCus ? big : kCus), dim3(kBlock), 0, st, p,
                          (int32_t)((p.m + kBig - 1) / kBig), (int32_t)((p.n + kBig - 1) / kBig));
    }
    return launch(matmul_mid_kernel<kFormatA, kWide>, grid_of(mid < kCus ? mid : kCus), dim3(kBlock), 0, st, p,
                  (int32_t)((p.m + kMid - 1) / kMid), (int32_t)((p.n + kMid - 1) / kMid));
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
    if (k > (int64_t)kMostGroups * kGroup)
        return fail(ZR_EINVAL, "%s: k = %lld has too many groups", who, (long long)k);
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
