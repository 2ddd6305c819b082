// Root-mean-square norm with the residual's addition and 8-bit output, and its
// backward pass (gfx950).
//
// Forward, per row: h = T(x + residual), rstd = 1 / sqrt(mean h^2 + eps),
// y = h * rstd * weight, and codes of y with one E8M0 scale per 128 columns.
// Backward, with xh = h * rstd and g = dy * weight: dx = rstd * (g - xh * mean(g xh))
// + dh and dweight = sum over rows of dy * xh.
//
// Sums are fp32: a lane's elements in column order, then the lanes of a wave and
// the waves of a row in a fixed tree, so results depend only on the inputs, not
// on the grid or on addresses.  Both passes are bound by HBM.
#include "fp8.hpp"

namespace zr {

struct NormArgs {
    const uint16_t *x, *residual, *weight;
    int64_t ldx, ldr;
    int64_t rows, cols;
    float eps;
    uint16_t *h, *y;
    int64_t ldh, ldy;
    uint8_t *q, *scales;
    int64_t ldq;
    float *rstd;
};

// Eight elements of the stream h (fp32, already rounded to T).
template <typename T>
__device__ __forceinline__ u32x4 stream8(u32x4 x, u32x4 r)
{
    u32x4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        h[i] = T::pack(T::lo(x[i]) + T::lo(r[i]), T::hi(x[i]) + T::hi(r[i]));
    return h;
}

template <typename T>
__device__ __forceinline__ float squares8(u32x4 h, float sum)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = __builtin_fmaf(T::lo(h[i]), T::lo(h[i]), sum);
        sum = __builtin_fmaf(T::hi(h[i]), T::hi(h[i]), sum);
    }
    return sum;
}

__device__ __forceinline__ float rstd_of(float sum, int64_t cols, float eps)
{
    return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, (float)cols) + eps));
}

// y, codes and scales of eight columns from c on (n of them inside the row),
// held by a lane of the row of 16 lanes that holds the group.
template <typename T>
__device__ __forceinline__ void norm_outputs(const NormArgs &a, int64_t row, int64_t c, int64_t n, u32x4 h, u32x4 w,
                                             float rstd)
{
    float y[kVec];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = T::lo(h[i]) * rstd * T::lo(w[i]);
        y[2 * i + 1] = T::hi(h[i]) * rstd * T::hi(w[i]);
    }
    if (a.y) {
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = T::pack(y[2 * i], y[2 * i + 1]);
        store8<true>(a.y + row * a.ldy + c, o, n);
    }
    if (a.q) {
        uint32_t amax = 0;
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            amax = max_u32(amax, __float_as_uint(y[e]) & 0x7fffffffu);
        const uint32_t s = scale_byte<ZR_E4M3>(group_max(amax));
        const float inv = inverse_scale(s);
        store_codes8(a.q + row * a.ldq + c,
                               u32x2{codes4<ZR_E4M3>(y[0], y[1], y[2], y[3], inv, s),
                                     codes4<ZR_E4M3>(y[4], y[5], y[6], y[7], inv, s)}, n);
        if ((threadIdx.x & 15) == 0 && n > 0)
            a.scales[row * ((a.cols + kGroup - 1) / kGroup) + c / kGroup] = (uint8_t)s;
    }
}

// Sum over the workgroup's four waves of a value that wave_sum has spread over
// each wave; `slot` alternates so that one barrier per sum is enough.
__device__ __forceinline__ float block_sum(float v, float (*part)[4], int slot)
{
    if ((threadIdx.x & 63) == 0)
        part[slot][threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[slot][0] + part[slot][1]) + (part[slot][2] + part[slot][3]);
}

// Rows of any length: a workgroup per row, read twice (the second time from cache).  h is
// written in the second read, so that it may replace x or residual.  4096 x 20000 with
// residual, h, y and codes: 190 us, 3.9 TB/s.
template <typename T>
__global__ __launch_bounds__(kBlock) void norm_wide_kernel(NormArgs a)
{
    __shared__ float part[2][4];
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
        const uint16_t *x = a.x + row * a.ldx, *r = a.residual ? a.residual + row * a.ldr : nullptr;
        float sum = 0.0f;
        for (int64_t c = threadIdx.x * kVec; c < a.cols; c += kBlock * kVec) {
            u32x4 h = load8(x + c, a.cols - c);
            if (r)
                h = stream8<T>(h, load8(r + c, a.cols - c));
            sum = squares8<T>(h, sum);
        }
        const float rstd = rstd_of(block_sum(wave_sum(sum), part, slot), a.cols, a.eps);
        if (a.rstd && threadIdx.x == 0)
            a.rstd[row] = rstd;
        // whole rows of 16 lanes stay in the loop: they share a group's maximum
        for (int64_t c = threadIdx.x * kVec; c - (threadIdx.x & 15) * kVec < a.cols; c += kBlock * kVec) {
            const int64_t n = a.cols - c;
            u32x4 h = load8(x + c, n);
            if (r)
                h = stream8<T>(h, load8(r + c, n));
            if (a.h)
                store8<true>(a.h + row * a.ldh + c, h, n);
            norm_outputs<T>(a, row, c, n, h, load8(a.weight + c, n), rstd);
        }
    }
}

// Rows held in registers, read once: kWaves waves share a row, a lane holds NV vectors
// of 8 columns, each wave-wide access covers 512 consecutive columns (four groups).
// 16384 x 4096 with residual, h, y and codes: 105 us, 5.7 TB/s (without y 81 us); one row
// of 4096: 3.2 us, a launch and one round trip to memory.  With 4095 columns, where rows start
// at any element, the bytes from and to memory are the same to 3 %, but the vector cache is
// accessed 2.7 times as often and bounds: 167 us.
template <typename T, int NV, int kWaves>
__global__ __launch_bounds__(kWaves > 4 ? 64 * kWaves : kBlock) void norm_row_kernel(NormArgs a)
{
    constexpr int kThreads = kWaves > 4 ? 64 * kWaves : kBlock, kSlots = kThreads / (64 * kWaves);
    __shared__ float part[2][kThreads / 64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = wave / kWaves, w0 = wave % kWaves;
    int flip = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * kSlots; row0 < a.rows; row0 += (int64_t)gridDim.x * kSlots, flip ^= 1) {
        const int64_t row = row0 + slot;
        const bool live = row < a.rows;
        u32x4 h[NV], w[NV];
        int32_t n[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int32_t c = ((v * kWaves + w0) * 64 + lane) * kVec;
            n[v] = live ? (int32_t)a.cols - c : 0;
            h[v] = load8(a.x + row * a.ldx + c, n[v]);
        }
        if (a.residual) {
            u32x4 r[NV];
#pragma unroll
            for (int v = 0; v < NV; ++v)
                r[v] = load8(a.residual + row * a.ldr + ((v * kWaves + w0) * 64 + lane) * kVec, n[v]);
#pragma unroll
            for (int v = 0; v < NV; ++v)
                h[v] = stream8<T>(h[v], r[v]);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            w[v] = load8(a.weight + ((v * kWaves + w0) * 64 + lane) * kVec, n[v]);
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
            sum = squares8<T>(h[v], sum);
        sum = wave_sum(sum);
        if constexpr (kWaves > 1) {
            if (lane == 0)
                part[flip][wave] = sum;
            __syncthreads();
            sum = part[flip][slot * kWaves];
#pragma unroll
            for (int i = 1; i < kWaves; ++i)
                sum += part[flip][slot * kWaves + i];
        }
        const float rstd = rstd_of(sum, a.cols, a.eps);
        if (a.rstd && live && w0 == 0 && lane == 0)
            a.rstd[row] = rstd;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t c = ((v * kWaves + w0) * 64 + lane) * kVec;
            if (a.h)
                store8<true>(a.h + row * a.ldh + c, h[v], n[v]);
            norm_outputs<T>(a, row, c, n[v], h[v], w[v], rstd);
        }
    }
}

// ------------------------------------------------------------------ backward --

struct NormGradArgs {
    const uint16_t *dy, *h, *weight, *dh;
    const float *rstd;
    int64_t lddy, ldh, lddh;
    int64_t rows, cols;
    uint16_t *dx, *dweight;
    int64_t lddx;
    float *partial;  // [groups of rows][cols]
    int64_t parts;   // groups of rows: row r belongs to group r % parts
};

// sum of g * h over eight columns (the row's rstd is factored out)
template <typename T>
__device__ __forceinline__ float dots8(u32x4 dy, u32x4 w, u32x4 h, float sum)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sum = __builtin_fmaf(T::lo(dy[i]) * T::lo(w[i]), T::lo(h[i]), sum);
        sum = __builtin_fmaf(T::hi(dy[i]) * T::hi(w[i]), T::hi(h[i]), sum);
    }
    return sum;
}

// dx of eight columns: rstd * (g - h * k) + dh with k = rstd^2 * mean(g h).
template <typename T>
__device__ __forceinline__ u32x4 dx8(u32x4 dy, u32x4 w, u32x4 h, u32x4 dh, float rstd, float k)
{
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        o[i] = T::pack(__builtin_fmaf(__builtin_fmaf(-k, T::lo(h[i]), T::lo(dy[i]) * T::lo(w[i])), rstd, T::lo(dh[i])),
                       __builtin_fmaf(__builtin_fmaf(-k, T::hi(h[i]), T::hi(dy[i]) * T::hi(w[i])), rstd, T::hi(dh[i])));
    return o;
}

__device__ __forceinline__ float dx_factor(float dot, float rstd, int64_t cols)
{
    return __fdiv_rn(dot, (float)cols) * rstd * rstd;
}

// dx for rows of any length, read twice.  With the partial sums of the weight gradient,
// which read dy and h once more by columns, 4096 x 20000 with dh takes 260 us, 2.5 TB/s of
// what has to move.
template <typename T>
__global__ __launch_bounds__(kBlock) void norm_dx_wide_kernel(NormGradArgs a)
{
    __shared__ float part[2][4];
    int slot = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, slot ^= 1) {
        const uint16_t *dy = a.dy + row * a.lddy, *h = a.h + row * a.ldh;
        float sum = 0.0f;
        for (int64_t c = threadIdx.x * kVec; c < a.cols; c += kBlock * kVec)
            sum = dots8<T>(load8(dy + c, a.cols - c), load8(a.weight + c, a.cols - c),
                           load8(h + c, a.cols - c), sum);
        const float rstd = a.rstd[row];
        const float k = dx_factor(block_sum(wave_sum(sum), part, slot), rstd, a.cols);
        for (int64_t c = threadIdx.x * kVec; c < a.cols; c += kBlock * kVec) {
            const int64_t n = a.cols - c;
            const u32x4 dh = a.dh ? load8(a.dh + row * a.lddh + c, n) : u32x4{0, 0, 0, 0};
            store8<true>(a.dx + row * a.lddx + c,
                             dx8<T>(load8(dy + c, n), load8(a.weight + c, n),
                                    load8(h + c, n), dh, rstd, k), n);
        }
    }
}

// Partial weight gradients of one column and one group of rows per thread.
template <typename T>
__global__ __launch_bounds__(kBlock) void norm_dweight_partial_kernel(NormGradArgs a)
{
    const int64_t blocks = (a.cols + kBlock - 1) / kBlock;
    for (int64_t i = blockIdx.x; i < blocks * a.parts; i += gridDim.x) {
        const int64_t p = i / blocks, c = (i - p * blocks) * kBlock + threadIdx.x;
        if (c >= a.cols)
            continue;
        float sum = 0.0f;
        for (int64_t row = p; row < a.rows; row += a.parts)
            sum = __builtin_fmaf(widen<T>(a.dy[row * a.lddy + c]), widen<T>(a.h[row * a.ldh + c]) * a.rstd[row], sum);
        a.partial[p * a.cols + c] = sum;
    }
}

// Rows held in registers, read once, for dx and the weight gradient together: kWaves
// waves share a row, a workgroup takes kSlots rows at a time, every parts * kSlots'th,
// and reads the next rows before it reduces the present ones.  A lane sums the weight
// gradient of its columns over its rows; the slots meet in LDS, in slot order.
// 16384 x 4096 with dh: 104 us, 5.2 TB/s, the partial sums' own pass included; 8192 x 11008
// 153 us, 4.7 TB/s; 777 x 1000 10 us, two launches.  Fewer rounds to a workgroup overlap less, and
// the partial sums weigh more: 8192 x 1024 19.5 us, 3.4 TB/s.  Rows off 16 bytes are bound by the
// vector cache, as in the forward pass: 16384 x 4095 237 us, 4096 x 1257 24.
constexpr int kGradThreads = 512;

template <typename T, int NV, int kWaves>
__global__ __launch_bounds__(kGradThreads) void norm_grad_row_kernel(NormGradArgs a)
{
    constexpr int kSlots = kGradThreads / (64 * kWaves), kCols = NV * kWaves * 64 * kVec;
    constexpr bool kEarly = NV <= 2;  // two rows of 4 vectors to a lane are more than the registers hold
    __shared__ float part[2][kGradThreads / 64];
    __shared__ f32x4 sums[kSlots > 1 ? (kSlots - 1) * kCols / 4 : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = wave / kWaves, w0 = wave % kWaves;
    int32_t c[NV], n[NV];
    u32x4 w[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        c[v] = ((v * kWaves + w0) * 64 + lane) * kVec;
        n[v] = (int32_t)a.cols - c[v];
        w[v] = load8(a.weight + c[v], n[v]);
    }
    const int64_t stride = a.parts * kSlots;
    // alternates over all rounds, also from one group of rows to the next: where a row takes the
    // whole workgroup the barrier of a sum is the only one there is
    int flip = 0;
    for (int64_t p = blockIdx.x; p < a.parts; p += gridDim.x) {
        f32x4 dw[NV][2];
#pragma unroll
        for (int v = 0; v < NV; ++v)
            dw[v][0] = dw[v][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        u32x4 dy[NV], h[NV], dh[NV];
        float rstd = 0.0f;
        const auto load = [&](int64_t row) {
            const bool live = row < a.rows;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                dy[v] = load8(a.dy + row * a.lddy + c[v], live ? n[v] : 0);
                h[v] = load8(a.h + row * a.ldh + c[v], live ? n[v] : 0);
                dh[v] = a.dh ? load8(a.dh + row * a.lddh + c[v], live ? n[v] : 0) : u32x4{0, 0, 0, 0};
            }
            rstd = live ? a.rstd[row] : 0.0f;
        };
        // the same number of rounds in every slot
        load(p * kSlots + slot);
        for (int64_t row0 = p * kSlots; row0 < a.rows; row0 += stride, flip ^= 1) {
            const int64_t row = row0 + slot;
            float sum = 0.0f;
#pragma unroll
            for (int v = 0; v < NV; ++v)
                sum = dots8<T>(dy[v], w[v], h[v], sum);
            u32x4 o_dy[NV], o_h[NV], o_dh[NV];
            const float r = rstd;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                o_dy[v] = dy[v];
                o_h[v] = h[v];
                o_dh[v] = dh[v];
            }
            if constexpr (kEarly)
                load(row + stride);
            sum = wave_sum(sum);
            if constexpr (kWaves > 1) {
                if (lane == 0)
                    part[flip][wave] = sum;
                __syncthreads();
                sum = part[flip][slot * kWaves];
#pragma unroll
                for (int i = 1; i < kWaves; ++i)
                    sum += part[flip][slot * kWaves + i];
            }
            const float k = dx_factor(sum, r, a.cols);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float *d = reinterpret_cast<float *>(&dw[v][i / 2]) + i % 2 * 2;
                    d[0] = __builtin_fmaf(T::lo(o_dy[v][i]), T::lo(o_h[v][i]) * r, d[0]);
                    d[1] = __builtin_fmaf(T::hi(o_dy[v][i]), T::hi(o_h[v][i]) * r, d[1]);
                }
                if (row < a.rows)
                    store8<true>(a.dx + row * a.lddx + c[v], dx8<T>(o_dy[v], w[v], o_h[v], o_dh[v], r, k), n[v]);
            }
            if constexpr (!kEarly)
                load(row + stride);
        }
        if constexpr (kSlots > 1) {
            __syncthreads();
            if (slot > 0) {
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    sums[(slot - 1) * (kCols / 4) + c[v] / 4] = dw[v][0];
                    sums[(slot - 1) * (kCols / 4) + c[v] / 4 + 1] = dw[v][1];
                }
            }
            __syncthreads();
        }
        if (slot == 0) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
#pragma unroll
                for (int s = 1; s < kSlots; ++s) {
                    dw[v][0] += sums[(s - 1) * (kCols / 4) + c[v] / 4];
                    dw[v][1] += sums[(s - 1) * (kCols / 4) + c[v] / 4 + 1];
                }
#pragma unroll
                for (int e = 0; e < kVec; ++e)
                    if (e < n[v])
                        a.partial[p * a.cols + c[v] + e] = dw[v][e / 4][e % 4];
            }
        }
    }
}

// dweight from the partial sums: 32 columns (a line) to a workgroup, 16 threads to a
// column, each over every 16th partial sum; they meet in LDS in that order.
template <typename T>
__global__ __launch_bounds__(kGradThreads) void norm_dweight_kernel(NormGradArgs a)
{
    __shared__ float part[16][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    for (int64_t c0 = (int64_t)blockIdx.x * 32; c0 < a.cols; c0 += (int64_t)gridDim.x * 32) {
        const int64_t c = c0 + x;
        float sum = 0.0f;
        if (c < a.cols)
#pragma unroll 8
            for (int64_t p = y; p < a.parts; p += 16)
                sum += a.partial[p * a.cols + c];
        part[y][x] = sum;
        __syncthreads();
        if (y == 0 && c < a.cols) {
#pragma unroll
            for (int i = 1; i < 16; ++i)
                sum += part[i][x];
            a.dweight[c] = narrow<T>(sum);
        }
        __syncthreads();
    }
}

namespace {

template <typename T, int NV, int kWaves>
zr_status norm_rows(const NormArgs &a, hipStream_t st)
{
    constexpr int threads = kWaves > 4 ? 64 * kWaves : kBlock, slots = threads / (64 * kWaves);
    return launch(norm_row_kernel<T, NV, kWaves>, grid_of((a.rows + slots - 1) / slots), dim3(threads), 0, st, a);
}

// Up to 2048 columns one vector to a lane, up to 8192 two, so that 4 or 8 waves cover a
// row; longer rows take four, and from 16385 columns on a row no longer fits the registers
// of 8 waves.
template <typename T>
zr_status norm_run(const NormArgs &a, hipStream_t st)
{
    if (a.cols <= 512)
        return norm_rows<T, 1, 1>(a, st);
    if (a.cols <= 1024)
        return norm_rows<T, 1, 2>(a, st);
    if (a.cols <= 2048)
        return norm_rows<T, 1, 4>(a, st);
    if (a.cols <= 4096)
        return norm_rows<T, 2, 4>(a, st);
    if (a.cols <= 8192)
        return norm_rows<T, 2, 8>(a, st);
    if (a.cols <= 16384)
        return norm_rows<T, 4, 8>(a, st);
    return launch(norm_wide_kernel<T>, grid_of(a.rows), dim3(kBlock), 0, st, a);
}

template <typename T, int NV, int kWaves>
zr_status norm_grad_rows(NormGradArgs a, hipStream_t st)
{
    constexpr int slots = kGradThreads / (64 * kWaves);
    const int64_t rounds = (a.rows + slots - 1) / slots;
    a.parts = rounds < ZR_RMSNORM_PARTIALS ? rounds : ZR_RMSNORM_PARTIALS;
    const zr_status s = launch(norm_grad_row_kernel<T, NV, kWaves>, grid_of(a.parts), dim3(kGradThreads), 0, st, a);
    return s != ZR_OK ? s : launch(norm_dweight_kernel<T>, grid_of((a.cols + 31) / 32), dim3(kGradThreads), 0, st, a);
}

template <typename T>
zr_status norm_backward_run(NormGradArgs a, hipStream_t st)
{
    if (a.rows > 0 && a.cols <= 16384) {
        if (a.cols <= 512)
            return norm_grad_rows<T, 1, 1>(a, st);
        if (a.cols <= 1024)
            return norm_grad_rows<T, 2, 1>(a, st);
        if (a.cols <= 2048)
            return norm_grad_rows<T, 2, 2>(a, st);
        if (a.cols <= 4096)
            return norm_grad_rows<T, 2, 4>(a, st);
        if (a.cols <= 8192)
            return norm_grad_rows<T, 2, 8>(a, st);
        return norm_grad_rows<T, 4, 8>(a, st);
    }
    zr_status s = ZR_OK;
    a.parts = a.rows < ZR_RMSNORM_PARTIALS ? a.rows : ZR_RMSNORM_PARTIALS;
    if (a.rows > 0) {
        // dweight's partial sums first: dx may replace dy
        const int64_t blocks = (a.cols + kBlock - 1) / kBlock * a.parts;
        s = launch(norm_dweight_partial_kernel<T>, grid_of(blocks), dim3(kBlock), 0, st, a);
        if (s == ZR_OK)
            s = launch(norm_dx_wide_kernel<T>, grid_of(a.rows), dim3(kBlock), 0, st, a);
    }
    return s != ZR_OK ? s : launch(norm_dweight_kernel<T>, grid_of((a.cols + 31) / 32), dim3(kGradThreads), 0, st, a);
}

bool same_matrix(const void *p, int64_t ldp, const void *q, int64_t ldq) { return p == q && ldp == ldq; }

}  // namespace
}  // namespace zr

using namespace zr;

extern "C" zr_status zr_rmsnorm_fp8(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                                    zr_dtype dtype, int64_t rows, int64_t cols, double eps, void *h, int64_t ldh,
                                    void *y, int64_t ldy, uint8_t *q, int64_t ldq, uint8_t *scales, float *rstd,
                                    void *stream)
{
    clear_error();
    const char *who = "zr_rmsnorm_fp8";
    if (dtype != ZR_BF16 && dtype != ZR_F16)
        return fail(ZR_EINVAL, "%s: dtype = %d, must be ZR_BF16 or ZR_F16", who, dtype);
    if (rows < 0 || cols < 1)
        return fail(ZR_EINVAL, "%s: rows < 0 or cols < 1", who);
    if (!(eps >= 0.0) || !std::isfinite(eps) || !std::isfinite((float)eps))
        return fail(ZR_EINVAL, "%s: eps must be finite and >= 0", who);
    if ((!q) != (!scales))
        return fail(ZR_EINVAL, "%s: codes without scales or scales without codes", who);
    if (h && !residual)
        return fail(ZR_EINVAL, "%s: h without residual (it would equal x)", who);
    if (rows == 0)
        return ZR_OK;
    if (!x || !weight || (!y && !q))
        return fail(ZR_EINVAL, "%s: NULL x or weight, or neither y nor q", who);
    int64_t nx, nr = 0, nh = 0, ny = 0, nq = 0;
    if (!matrix_extent(rows, cols, ldx, 2, &nx) || (residual && !matrix_extent(rows, cols, ldr, 2, &nr)) ||
        (h && !matrix_extent(rows, cols, ldh, 2, &nh)) || (y && !matrix_extent(rows, cols, ldy, 2, &ny)) ||
        (q && !matrix_extent(rows, cols, ldq, 1, &nq)))
        return fail(ZR_EINVAL, "%s: row distance below cols, or a matrix past int64", who);
    if (!aligned_to(x, 2) || !aligned_to(residual, 2) || !aligned_to(weight, 2) || !aligned_to(h, 2) ||
        !aligned_to(y, 2) || !aligned_to(rstd, 4))
        return fail(ZR_EALIGN, "%s: 16-bit matrices must be 2-byte and rstd 4-byte aligned", who);
    {
        // outputs first; inputs may overlap one another, and h may be x or residual
        const void *p[8] = {h, y, q, scales, rstd, x, residual, weight};
        const int64_t b[8] = {nh, ny, nq, rows * ((cols + kGroup - 1) / kGroup), 4 * rows, nx, nr, 2 * cols};
        for (int i = 0; i < 5; ++i)
            for (int j = i + 1; j < 8; ++j) {
                const bool in_place = i == 0 && ((j == 5 && same_matrix(h, ldh, x, ldx)) ||
                                                 (j == 6 && same_matrix(h, ldh, residual, ldr)));
                if (p[i] && p[j] && !in_place && overlaps(p[i], b[i], p[j], b[j]))
                    return fail(ZR_EINVAL, "%s: an output overlaps another buffer", who);
            }
    }
    const NormArgs a{static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(residual),
                     static_cast<const uint16_t *>(weight), ldx, ldr, rows, cols, (float)eps,
                     static_cast<uint16_t *>(h), static_cast<uint16_t *>(y), ldh, ldy, q, scales, ldq, rstd};
    hipStream_t st = static_cast<hipStream_t>(stream);
    return dtype == ZR_BF16 ? norm_run<BF16>(a, st) : norm_run<F16>(a, st);
}

extern "C" zr_status zr_rmsnorm_backward(const void *dy, int64_t lddy, const void *h, int64_t ldh, const void *weight,
                                         const float *rstd, const void *dh, int64_t lddh, zr_dtype dtype,
                                         int64_t rows, int64_t cols, void *dx, int64_t lddx, void *dweight,
                                         float *workspace, void *stream)
{
    clear_error();
    const char *who = "zr_rmsnorm_backward";
    if (dtype != ZR_BF16 && dtype != ZR_F16)
        return fail(ZR_EINVAL, "%s: dtype = %d, must be ZR_BF16 or ZR_F16", who, dtype);
    if (rows < 0 || cols < 1)
        return fail(ZR_EINVAL, "%s: rows < 0 or cols < 1", who);
    if (!dweight || !workspace || (rows > 0 && (!dy || !h || !weight || !rstd || !dx)))
        return fail(ZR_EINVAL, "%s: NULL buffer", who);
    int64_t ndy = 0, nh = 0, ndh = 0, ndx = 0, nw;
    if (rows > 0 && (!matrix_extent(rows, cols, lddy, 2, &ndy) || !matrix_extent(rows, cols, ldh, 2, &nh) ||
                     (dh && !matrix_extent(rows, cols, lddh, 2, &ndh)) || !matrix_extent(rows, cols, lddx, 2, &ndx)))
        return fail(ZR_EINVAL, "%s: row distance below cols, or a matrix past int64", who);
    if (!matrix_extent(ZR_RMSNORM_PARTIALS, cols, cols, 4, &nw))
        return fail(ZR_EINVAL, "%s: workspace past int64", who);
    if (!aligned_to(dy, 2) || !aligned_to(h, 2) || !aligned_to(weight, 2) || !aligned_to(rstd, 4) ||
        !aligned_to(dh, 2) || !aligned_to(dx, 2) || !aligned_to(dweight, 2) || !aligned_to(workspace, 4))
        return fail(ZR_EALIGN, "%s: 16-bit matrices must be 2-byte, rstd and workspace 4-byte aligned", who);
    {
        const void *p[8] = {dx, dweight, workspace, dy, h, dh, weight, rstd};
        const int64_t b[8] = {ndx, 2 * cols, nw, ndy, nh, ndh, rows > 0 ? 2 * cols : 0, 4 * rows};
        for (int i = 0; i < 3; ++i)
            for (int j = i + 1; j < 8; ++j) {
                const bool in_place = i == 0 && ((j == 3 && same_matrix(dx, lddx, dy, lddy)) ||
                                                 (j == 5 && same_matrix(dx, lddx, dh, lddh)));
                if (p[i] && p[j] && !in_place && overlaps(p[i], b[i], p[j], b[j]))
                    return fail(ZR_EINVAL, "%s: an output overlaps another buffer", who);
            }
    }
    const NormGradArgs a{static_cast<const uint16_t *>(dy), static_cast<const uint16_t *>(h),
                         static_cast<const uint16_t *>(weight), static_cast<const uint16_t *>(dh), rstd, lddy, ldh,
                         lddh, rows, cols, static_cast<uint16_t *>(dx), static_cast<uint16_t *>(dweight), lddx,
                         workspace, 0};
    hipStream_t st = static_cast<hipStream_t>(stream);
    return dtype == ZR_BF16 ? norm_backward_run<BF16>(a, st) : norm_backward_run<F16>(a, st);
}
