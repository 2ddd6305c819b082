// Clipping by the global gradient norm (gfx950): the sum of squares of many tensors with
// norm and factor, tensors scaled in place, and AdamW on the clipped gradient.
//
//   S = sum of x^2,  norm = |grad_scale| sqrt(S) / loss scale,  factor = min(1, max_norm / (norm + eps))
//
// The tensors of a call travel as a table of descriptors in the kernel arguments (in
// batches); a wave finds the tensor of a tile by comparing the tiles' prefix
// sums all at once.  Squares are added in fp64: a 16-bit or fp32 value
// widens exactly, its square has at most 48 bits and never overflows, and the sum's error
// (about 1e-13 over 2^31 elements) is far below the fp32 norm's rounding, so that clipping
// decisions do not go by the order of the additions.
#include <algorithm>
#include <new>

#include "clip.hpp"
#include "fp16.hpp"
#include "fp8.hpp"

namespace zr {

// ------------------------------------------------------------ tensor lists ----

constexpr int kMaxPieces = 224;                  // 3584 bytes of kernel arguments
constexpr int kLookups = (kMaxPieces + 63) / 64;
constexpr int kTileVecs = 8;                     // 16-byte vectors of a tile to a lane
constexpr int kTileBytes = kTileVecs * 64 * 16;  // 8 KB: a wave's

struct PieceBatch {
    int32_t count;
    uint32_t tiles;
    uint32_t begin[kMaxPieces];  // prefix sums of tiles within the batch
    uint32_t last[kMaxPieces];   // bytes of the tensors' last tiles
    uintptr_t base[kMaxPieces];
};

// Where a tile lies: its first byte, how many of its bytes belong to the tensor, and
// whether it is the tensor's first.
struct TileAt {
    uintptr_t p;
    int32_t bytes;
    bool first;
};

// A wave's copy of the prefix sums, a tensor to a lane (64 a word): the tensor of a tile is
// found by comparing all of them at once.  The table is cold in every cache when a kernel
// starts, and a binary search would wait for memory at each of its eight steps: 290 small
// tensors scaled in two launches of 8 us each, so in two of 4.
struct Lookup {
    uint32_t begin[kLookups];

    __device__ __forceinline__ explicit Lookup(const PieceBatch &batch)
    {
        const int lane = threadIdx.x & 63;
#pragma unroll
        for (int i = 0; i < kLookups; ++i)
            begin[i] = lane + 64 * i < batch.count ? batch.begin[lane + 64 * i] : 0xffffffffu;
    }

    __device__ __forceinline__ TileAt at(const PieceBatch &batch, uint32_t tile) const
    {
        int t = -1;
#pragma unroll
        for (int i = 0; i < kLookups; ++i)
            t += __builtin_popcountll(__ballot(begin[i] <= tile));
        const uint32_t next = t + 1 < batch.count ? batch.begin[t + 1] : batch.tiles, index = tile - batch.begin[t];
        return {batch.base[t] + (uintptr_t)index * kTileBytes, tile + 1 == next ? (int32_t)batch.last[t] : kTileBytes,
                index == 0};
    }
};

// ------------------------------------------------------------------- norm ----

struct F32 {};

// Adds the squares of a vector's elements to four sums.
template <typename T>
__device__ __forceinline__ void add_squares(u32x4 w, double (&s)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, F32>::value) {
            const double x = (double)__uint_as_float(w[i]);
            s[i] = __builtin_fma(x, x, s[i]);
        } else {
            const double a = (double)T::lo(w[i]), b = (double)T::hi(w[i]);
            s[i] = __builtin_fma(a, a, s[i]);
            s[i] = __builtin_fma(b, b, s[i]);
        }
    }
}

// The first `bytes` bytes at p (0 for more), zeros behind them; p at any element.
template <typename T>
__device__ __forceinline__ u32x4 load_part(uintptr_t p, int32_t bytes)
{
    constexpr bool wide = std::is_same<T, F32>::value;
    if (bytes >= 16)
        return __builtin_nontemporal_load((global_ptr<const any_u32x4>)p);
    u32x4 w = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < (wide ? 4 : 8); ++e)
        if (e * (wide ? 4 : 2) < bytes) {
            if constexpr (wide)
                w[e] = load_global(reinterpret_cast<const uint32_t *>(p) + e);
            else
                w[e / 2] |= (uint32_t)load_global(reinterpret_cast<const uint16_t *>(p) + e) << (16 * (e % 2));
        }
    return w;
}

// A tile's vectors, a lane taking every 64th.
template <typename T>
__device__ __forceinline__ void load_tile(const TileAt &at, u32x4 (&w)[kTileVecs])
{
    const int lane = threadIdx.x & 63;
    if (at.bytes == kTileBytes) {
#pragma unroll
        for (int v = 0; v < kTileVecs; ++v)
            w[v] = __builtin_nontemporal_load((global_ptr<const any_u32x4>)(at.p + (v * 64 + lane) * 16));
    } else {
#pragma unroll
        for (int v = 0; v < kTileVecs; ++v) {
            const int32_t off = (v * 64 + lane) * 16;
            w[v] = load_part<T>(at.p + off, at.bytes - off);
        }
    }
}

// Sum of the squares of tiles `tile`, tile + step, ... of the batch.
template <typename T>
__device__ __forceinline__ double tiles_squares(const PieceBatch &batch, uint64_t tile, uint64_t step)
{
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    const Lookup lookup(batch);
    for (; tile < batch.tiles; tile += step) {
        u32x4 w[kTileVecs];
        load_tile<T>(lookup.at(batch, (uint32_t)tile), w);
#pragma unroll
        for (int v = 0; v < kTileVecs; ++v)
            add_squares<T>(w[v], s);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

// Sum over the workgroup, in a fixed tree; the value is thread 0's.
template <int kThreads>
__device__ __forceinline__ double block_sum(double a)
{
    __shared__ double part[kThreads / 64];
#pragma unroll
    for (int m = 1; m < 64; m *= 2)
        a += __shfl_xor(a, m, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = a;
    __syncthreads();
    a = part[0];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i)
        a += part[i];
    return a;
}

__device__ __forceinline__ void finish_norm(double sum, const NormFinish &f)
{
    if (f.accumulate)
        sum += f.clip->sum_squares;
    double norm = __builtin_fabs(f.grad_scale) * __builtin_sqrt(sum);
    if (f.ls) {
        norm = norm / (double)f.ls->scale;
        if (!__builtin_isfinite(sum))
            f.ls->found_inf = 1;
    }
    const double factor = f.max_norm / (norm + f.eps);
    f.clip->sum_squares = sum;
    f.clip->norm = (float)norm;
    f.clip->factor = factor > 1.0 || __builtin_isinf(f.max_norm) ? 1.0f : (float)factor;  // a NaN stays
}

// Bound by HBM's reads: 1.75e9 bf16 504 us, 6.9 TB/s; 8.1e8 fp32 in 36 tensors 465 us, 7.0 TB/s;
// bf16 tensors that start on an odd element 5.1 TB/s, since a tile's vectors stay where
// the element count puts them (the order of the sums may not go by addresses) and straddle
// lines.  A lane's eight loads go out together; fp64 costs two operations an element, hidden
// behind them.  65 tensors of 4096: 4.2 us, then 1.7 us for the sums of the sums.
//
// Partial sums, one to a workgroup: wave w of sum p takes the batch's tiles p * kWaves + w and
// every parts * kWaves'th behind it; the first `begun` sums continue those of the batches
// before.
constexpr int kWaves = kBlock / 64;
template <typename T>
__global__ __launch_bounds__(kBlock) void squares_kernel(PieceBatch batch, uint32_t parts, uint32_t begun, double *partial)
{
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint32_t p = blockIdx.x; p < parts; p += gridDim.x) {
        const double sum = block_sum<kBlock>(tiles_squares<T>(batch, (uint64_t)p * kWaves + wave, (uint64_t)parts * kWaves));
        if (threadIdx.x == 0)
            partial[p] = p < begun ? partial[p] + sum : sum;
    }
}

constexpr int kOneThreads = 1024, kFinishThreads = 256;

__global__ __launch_bounds__(kFinishThreads) void norm_finish_kernel(const double *partial, uint32_t parts, NormFinish f)
{
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < ZR_GRAD_NORM_PARTIALS / kFinishThreads; ++i)
        if (threadIdx.x + i * kFinishThreads < parts)
            a += partial[threadIdx.x + i * kFinishThreads];
    a = block_sum<kFinishThreads>(a);
    if (threadIdx.x == 0)
        finish_norm(a, f);
}

// A few tiles in one workgroup, norm and factor with them: one launch.
template <typename T>
__global__ __launch_bounds__(kOneThreads) void norm_one_kernel(PieceBatch batch, NormFinish f)
{
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const double sum = block_sum<kOneThreads>(tiles_squares<T>(batch, wave, kOneThreads / 64));
    if (threadIdx.x == 0)
        finish_norm(sum, f);
}

// Up to 32 tiles one workgroup takes 6.5 us and one launch, two launches 9 us of the host's time;
// past that the workgroup's fp64 arithmetic is longer (65 tiles 10 us).
constexpr int64_t kOneTiles = 32;

// ------------------------------------------------------------------ clipping ----

// One 16-byte vector times the factor, each element rounded once.
template <typename T>
__device__ __forceinline__ u32x4 scaled(u32x4 w, float factor)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, F32>::value)
            w[i] = __float_as_uint(__uint_as_float(w[i]) * factor);
        else
            w[i] = T::pack(T::lo(w[i]) * factor, T::hi(w[i]) * factor);
    }
    return w;
}

// Tiles start on 128-byte lines: a tensor's first tile begins up to 126 bytes before it
// and leaves what is there alone, as its last leaves what follows.  Bound by HBM: 4e8 fp16
// in place 265 us, 6.1 TB/s (tiles of a whole workgroup, every access with a check of its own,
// 371 us); at any address the same.  A factor of 1 ends the kernel before it reads an element:
// 7 us for the 4e8, the launch.
template <typename T>
__global__ __launch_bounds__(kBlock) void clip_kernel(PieceBatch batch, const zr_clip *clip)
{
    Lookup lookup(batch);
    float factor = clip->factor;
    // the table's loads wait together with the record's
    static_assert(kLookups == 4, "one operand to a word");
    asm volatile("" : "+v"(lookup.begin[0]), "+v"(lookup.begin[1]), "+v"(lookup.begin[2]), "+v"(lookup.begin[3]), "+s"(factor));
    if (factor == 1.0f)
        return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (uint64_t tile = (uint64_t)blockIdx.x * kWaves + wave; tile < batch.tiles; tile += (uint64_t)gridDim.x * kWaves) {
        const TileAt at = lookup.at(batch, (uint32_t)tile);
        const int32_t skip = at.first ? (int32_t)(at.p & 127) : 0;
        const uintptr_t line = at.p & ~(uintptr_t)127;
        if (skip == 0 && at.bytes == kTileBytes) {
            u32x4 *p = reinterpret_cast<u32x4 *>(line) + lane;
            u32x4 w[kTileVecs];
#pragma unroll
            for (int v = 0; v < kTileVecs; ++v)
                w[v] = load_stream(p + v * 64);
#pragma unroll
            for (int v = 0; v < kTileVecs; ++v)
                store_stream(p + v * 64, scaled<T>(w[v], factor));
            continue;
        }
        constexpr int size = std::is_same<T, F32>::value ? 4 : 2;
#pragma unroll 1
        for (int32_t off = lane * 16; off < at.bytes; off += 64 * 16) {
            if (off >= skip && off + 16 <= at.bytes) {
                u32x4 *p = reinterpret_cast<u32x4 *>(line + off);
                store_stream(p, scaled<T>(load_stream(p), factor));
                continue;
            }
            for (int32_t b = off < skip ? skip : off; b < off + 16 && b < at.bytes; b += size) {
                if constexpr (size == 4) {
                    const auto p = (global_ptr<float>)(line + b);
                    *p = *p * factor;
                } else {
                    const auto p = (global_ptr<uint16_t>)(line + b);
                    *p = narrow<T>(widen<T>(*p) * factor);
                }
            }
        }
    }
}

// --------------------------------------------------------------------- AdamW ----

// The gradient and copy types of the step: the conversions of zr_adamw_step and
// zr_adamw_step_f16.
struct StepBF16 {
    static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_bf16x2(lo, hi); }
};
struct StepF16 {
    static __device__ __forceinline__ float lo(uint32_t w) { return f16_lo(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return f16_hi(w); }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return pack_f16x2(lo, hi); }
};

template <typename T>
__device__ __forceinline__ double step_gradient(float g, double unscale, double scale)
{
    if constexpr (std::is_same<T, StepF16>::value)
        return (double)g * unscale * scale;
    return (double)g * scale;
}

template <typename T>
__device__ __forceinline__ void adamw_clip_one(const uint16_t *grad, float *master, float *m, float *v, uint16_t *param,
                                               int64_t j, double unscale, double scale, const AdamWScalars &s)
{
    float th = master[j], mm = m[j], vv = v[j];
    adamw_update(step_gradient<T>(T::lo(grad[j]), unscale, scale), th, mm, vv, s);
    master[j] = th;
    m[j] = mm;
    v[j] = vv;
    if (param)
        param[j] = (uint16_t)T::pack(th, 0.0f);
}

// The AdamW kernel of 4 elements to a lane (28 bytes an element, seven streams), its
// factor read from the record.  The record's load is issued before the data's and first
// used behind it: the empty asm takes both together.  1.05e8 elements, in turn with the kernel
// without a record on the same buffers (medians of a kernel trace): 474 us, 6.2 TB/s, beside 466 in
// bf16, 476 beside 475 in fp16; called on one set of buffers 467 beside 463, and 472 beside 469.
// Either kernel takes up to a quarter longer in its first fifty launches behind an idle time.
template <typename T, bool kParam>
__global__ __launch_bounds__(kBlock) void adamw_clip_vec_kernel(const uint16_t *grad, float *master, float *m, float *v,
                                                                uint16_t *param, int64_t numel, int64_t head,
                                                                int64_t groups, AdamWScalars s,
                                                                const zr_loss_scale *ls, const zr_clip *clip)
{
    constexpr bool kF16 = std::is_same<T, StepF16>::value;
    const u32x2 *g2 = reinterpret_cast<const u32x2 *>(grad + head);
    f32x4 *th4 = reinterpret_cast<f32x4 *>(master + head);
    f32x4 *m4 = reinterpret_cast<f32x4 *>(m + head);
    f32x4 *v4 = reinterpret_cast<f32x4 *>(v + head);
    u32x2 *p2 = kParam ? reinterpret_cast<u32x2 *>(param + head) : nullptr;
    const int32_t skip = kF16 ? ls->found_inf : 0;
    const float loss_scale = kF16 ? ls->scale : 1.0f, factor = clip->factor;

    for (int64_t i = first_tile<kAdamwOrder>() * kBlock + threadIdx.x; i < groups; i += grid_stride()) {
        u32x2 g = load_stream(g2 + i);
        f32x4 a = load_stream(th4 + i);
        f32x4 mm = load_stream(m4 + i);
        f32x4 vv = load_stream(v4 + i);
        int32_t sk = skip;
        float sc = loss_scale, fa = factor;
        asm volatile("" : "+v"(g), "+v"(a), "+v"(mm), "+v"(vv), "+s"(sk), "+s"(sc), "+s"(fa));
        if (kF16 && sk)  // the whole step is skipped: nothing is written
            return;
        const double unscale = kF16 ? 1.0 / (double)sc : 1.0, scale = s.grad_scale * (double)fa;
        const float gr[4] = {T::lo(g.x), T::hi(g.x), T::lo(g.y), T::hi(g.y)};
        float th[4] = {a.x, a.y, a.z, a.w};
        float mo[4] = {mm.x, mm.y, mm.z, mm.w};
        float vo[4] = {vv.x, vv.y, vv.z, vv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
            adamw_update(step_gradient<T>(gr[e], unscale, scale), th[e], mo[e], vo[e], s);
        store_stream(th4 + i, f32x4{th[0], th[1], th[2], th[3]});
        store_stream(m4 + i, f32x4{mo[0], mo[1], mo[2], mo[3]});
        store_stream(v4 + i, f32x4{vo[0], vo[1], vo[2], vo[3]});
        if (kParam)
            store_stream(p2 + i, u32x2{T::pack(th[0], th[1]), T::pack(th[2], th[3])});
    }
    if (blockIdx.x == 0 && !skip) {
        const int64_t tail_start = head + 4 * groups;
        const int64_t edge = head + (numel - tail_start);  // at most 63 + 3
        if ((int64_t)threadIdx.x < edge) {
            const int64_t j = (int64_t)threadIdx.x < head ? (int64_t)threadIdx.x : tail_start + (threadIdx.x - head);
            adamw_clip_one<T>(grad, master, m, v, kParam ? param : nullptr, j, kF16 ? 1.0 / (double)loss_scale : 1.0,
                              s.grad_scale * (double)factor, s);
        }
    }
}

// Where the buffers' 16-byte phases disagree: element by element, same bits.
template <typename T>
__global__ __launch_bounds__(kBlock) void adamw_clip_scalar_kernel(const uint16_t *grad, float *master, float *m, float *v,
                                                                   uint16_t *param, int64_t numel, AdamWScalars s,
                                                                   const zr_loss_scale *ls, const zr_clip *clip)
{
    constexpr bool kF16 = std::is_same<T, StepF16>::value;
    if (kF16 && ls->found_inf)
        return;
    const double unscale = kF16 ? 1.0 / (double)ls->scale : 1.0, scale = s.grad_scale * (double)clip->factor;
    for (int64_t j = global_tid(); j < numel; j += grid_stride())
        adamw_clip_one<T>(grad, master, m, v, param, j, unscale, scale, s);
}

constexpr size_t kAdamwClipLds = 32 * 1024;  // 5 workgroups per CU, as for zr_adamw_step

int clip_scalar_slots(ScalarSlot *out)
{
    out[0] = slot_of(adamw_clip_vec_kernel<StepBF16, true>);
    out[1] = slot_of(adamw_clip_vec_kernel<StepBF16, false>);
    out[2] = slot_of(adamw_clip_vec_kernel<StepF16, true>);
    out[3] = slot_of(adamw_clip_vec_kernel<StepF16, false>);
    out[4] = slot_of(adamw_clip_scalar_kernel<StepBF16>);
    out[5] = slot_of(adamw_clip_scalar_kernel<StepF16>);
    return 6;
}

int norm_finish_slots(ScalarSlot *out)
{
    out[0] = slot_of<NormFinish>(norm_finish_kernel);
    out[1] = slot_of<NormFinish>(norm_one_kernel<BF16>);
    out[2] = slot_of<NormFinish>(norm_one_kernel<F16>);
    out[3] = slot_of<NormFinish>(norm_one_kernel<F32>);
    return 4;
}

namespace {

zr_status check_clip(const char *who, const void *clip)
{
    if (!clip)
        return fail(ZR_EINVAL, "%s: clip record is NULL", who);
    if (!aligned_to(clip, 8))
        return fail(ZR_EALIGN, "%s: clip record must be 8-byte aligned", who);
    return ZR_OK;
}

constexpr int64_t kMostBytes = (int64_t)1 << 44;  // 2^31 tiles

// Checks a tensor list; buffers p[i] of b[i] bytes (NULL: none) must not overlap a tensor.
zr_status check_list(const char *who, const void *const *grads, const int64_t *numels, int32_t n, zr_dtype dtype,
                     const void *const *p, const int64_t *b, int count)
{
    if (dtype != ZR_BF16 && dtype != ZR_F16 && dtype != ZR_F32)
        return fail(ZR_EINVAL, "%s: dtype = %d, must be ZR_BF16, ZR_F16 or ZR_F32", who, dtype);
    if (n < 0 || (n > 0 && (!grads || !numels)))
        return fail(ZR_EINVAL, "%s: n < 0, or grads or numels is NULL", who);
    const int64_t size = dtype == ZR_F32 ? 4 : 2;
    for (int32_t t = 0; t < n; ++t) {
        if (numels[t] < 0 || (numels[t] > 0 && !grads[t]))
            return fail(ZR_EINVAL, "%s: numels[%d] < 0 or grads[%d] is NULL", who, t, t);
        if (numels[t] > kMostBytes / 4)  // no device holds as much
            return fail(ZR_EINVAL, "%s: numels[%d] past 2^42", who, t);
        if (!aligned_to(grads[t], size))
            return fail(ZR_EALIGN, "%s: grads[%d] must be %d-byte aligned", who, t, (int)size);
        for (int i = 0; i < count; ++i)
            if (p[i] && overlaps(grads[t], size * numels[t], p[i], b[i]))
                return fail(ZR_EINVAL, "%s: grads[%d] overlaps the record, the workspace or the loss-scale record", who,
                            t);
    }
    return ZR_OK;
}

// Calls run(batch) for the non-empty tensors, kMaxPieces at a time.  kInPlace (scaling, where
// neither order nor bounds of the tensors matter): a tensor that starts where the one before
// it ends goes on as one piece with it, as the tensors of a flat buffer do, and a piece's first
// tile starts on the 128-byte line that holds its first element (the table keeps the
// element's own address).
template <bool kInPlace, typename F>
zr_status for_batches(const void *const *grads, const int64_t *numels, int32_t n, int64_t size, F run)
{
    PieceBatch batch;
    batch.count = 0;
    batch.tiles = 0;
    const auto flush = [&]() -> zr_status {
        const zr_status s = batch.count > 0 ? run(batch) : ZR_OK;
        batch.count = 0;
        batch.tiles = 0;
        return s;
    };
    for (int32_t t = 0; t < n;) {
        if (numels[t] == 0) {
            ++t;
            continue;
        }
        const uintptr_t p = reinterpret_cast<uintptr_t>(grads[t]);
        int64_t bytes = size * numels[t++];
        if constexpr (kInPlace) {
            for (; t < n && bytes < kMostBytes &&
                   (numels[t] == 0 || reinterpret_cast<uintptr_t>(grads[t]) == p + (uintptr_t)bytes);
                 ++t)
                bytes += size * numels[t];
            bytes += (int64_t)(p & 127);
        }
        const int64_t tiles = (bytes + kTileBytes - 1) / kTileBytes;
        if (batch.count == kMaxPieces || batch.tiles + tiles > 0xfffffff0) {
            const zr_status s = flush();
            if (s != ZR_OK)
                return s;
        }
        batch.begin[batch.count] = batch.tiles;
        batch.last[batch.count] = (uint32_t)(bytes - (tiles - 1) * kTileBytes);
        batch.base[batch.count++] = p;
        batch.tiles += (uint32_t)tiles;
    }
    return flush();
}

template <typename T>
zr_status grad_norm_run(const void *const *grads, const int64_t *numels, int32_t n, int64_t size, double *partial,
                        const NormFinish &f, hipStream_t st)
{
    uint32_t parts = 0;
    bool done = false;
    int64_t tiles = 0;
    int32_t pieces = 0;
    for (int32_t t = 0; t < n; ++t) {
        tiles += (size * numels[t] + kTileBytes - 1) / kTileBytes;
        pieces += numels[t] > 0;
    }
    const bool one = tiles <= kOneTiles && pieces <= kMaxPieces && pieces > 0;
    zr_status s = for_batches<false>(grads, numels, n, size, [&](const PieceBatch &batch) -> zr_status {
        if (one) {
            done = true;
            return launch(norm_one_kernel<T>, dim3(1), dim3(kOneThreads), 0, st, batch, f);
        }
        const uint32_t mine = std::min<uint32_t>((batch.tiles + kWaves - 1) / kWaves, ZR_GRAD_NORM_PARTIALS);
        const zr_status r = launch(squares_kernel<T>, grid_of(mine), dim3(kBlock), 0, st, batch, mine, parts, partial);
        parts = std::max(parts, mine);
        return r;
    });
    if (s != ZR_OK || done)
        return s;
    return launch(norm_finish_kernel, dim3(1), dim3(kFinishThreads), 0, st, partial, parts, f);
}

template <typename T>
zr_status clip_run(const void *const *grads, const int64_t *numels, int32_t n, int64_t size, const zr_clip *clip,
                   hipStream_t st)
{
    return for_batches<true>(grads, numels, n, size, [&](const PieceBatch &batch) {
        return launch(clip_kernel<T>, grid_of(((int64_t)batch.tiles + kWaves - 1) / kWaves), dim3(kBlock), 0, st, batch, clip);
    });
}

// No two tensors may overlap: neighbours in the order of their addresses.  The usual
// list (pieces of a flat buffer) is in that order already.
zr_status check_disjoint(const char *who, const void *const *grads, const int64_t *numels, int32_t n, int64_t size)
{
    bool sorted = true;
    uintptr_t end = 0;
    for (int32_t t = 0; t < n && sorted; ++t)
        if (numels[t] > 0) {
            const uintptr_t p = reinterpret_cast<uintptr_t>(grads[t]);
            sorted = p >= end;
            end = p + (uintptr_t)(size * numels[t]);
        }
    if (sorted)
        return ZR_OK;
    auto *order = new (std::nothrow) int32_t[n];
    if (!order)
        return fail(ZR_ENOMEM, "%s: out of host memory", who);
    int32_t m = 0;
    for (int32_t t = 0; t < n; ++t)
        if (numels[t] > 0)
            order[m++] = t;
    std::sort(order, order + m, [&](int32_t a, int32_t b) { return grads[a] < grads[b]; });
    zr_status s = ZR_OK;
    for (int32_t i = 1; i < m && s == ZR_OK; ++i)
        if (overlaps(grads[order[i - 1]], size * numels[order[i - 1]], grads[order[i]], size * numels[order[i]]))
            s = fail(ZR_EINVAL, "%s: grads[%d] and grads[%d] overlap", who, order[i - 1], order[i]);
    delete[] order;
    return s;
}

template <typename T>
zr_status adamw_clip_run(const uint16_t *g, float *master, float *exp_avg, float *exp_avg_sq, uint16_t *p, int64_t numel,
                         const AdamWScalars &s, const zr_loss_scale *ls, const zr_clip *clip, hipStream_t st)
{
    const int64_t head = line_head32(master, g, numel);
    const bool vec = aligned_to(exp_avg + head, 16) && aligned_to(exp_avg_sq + head, 16) && aligned_to(g + head, 8) &&
                     (!p || aligned_to(p + head, 8));
    if (!vec)
        return launch(adamw_clip_scalar_kernel<T>, grid_of((numel + kBlock - 1) / kBlock), dim3(kBlock), 0, st, g, master,
                      exp_avg, exp_avg_sq, p, numel, s, ls, clip);
    const int64_t groups = (numel - head) / 4;
    const dim3 grid = order_grid<kAdamwOrder>((groups + kBlock - 1) / kBlock);
    if (p)
        return launch(adamw_clip_vec_kernel<T, true>, grid, dim3(kBlock), kAdamwClipLds, st, g, master, exp_avg,
                      exp_avg_sq, p, numel, head, groups, s, ls, clip);
    return launch(adamw_clip_vec_kernel<T, false>, grid, dim3(kBlock), kAdamwClipLds, st, g, master, exp_avg,
                  exp_avg_sq, p, numel, head, groups, s, ls, clip);
}

zr_status adamw_clip(const char *who, bool f16, const void *grad, float *master, float *exp_avg, float *exp_avg_sq,
                     void *param_out, int64_t numel, const zr_adamw_hparams *hp, const zr_loss_scale *ls,
                     const zr_clip *clip, void *stream)
{
    zr_status s = check_adamw_hparams(who, hp);
    if (s == ZR_OK && f16)
        s = check_ls(who, ls);
    if (s == ZR_OK)
        s = check_clip(who, clip);
    if (s != ZR_OK)
        return s;
    if (numel < 0)
        return fail(ZR_EINVAL, "%s: numel < 0", who);
    if (numel > 0 && (!grad || !master || !exp_avg || !exp_avg_sq))
        return fail(ZR_EINVAL, "%s: NULL buffer", who);
    if (!aligned_to(grad, 2) || !aligned_to(param_out, 2) || !aligned_to(master, 4) || !aligned_to(exp_avg, 4) ||
        !aligned_to(exp_avg_sq, 4))
        return fail(ZR_EALIGN, "%s: buffers must be naturally aligned (gradient and copy: 2 B, fp32: 4 B)", who);
    {
        const void *p[7] = {grad, master, exp_avg, exp_avg_sq, param_out, clip, ls};
        const int64_t b[7] = {2 * numel, 4 * numel, 4 * numel, 4 * numel, param_out ? 2 * numel : 0,
                              (int64_t)sizeof(zr_clip), ls ? (int64_t)sizeof(zr_loss_scale) : 0};
        int x, y;
        if (any_overlap(p, b, 7, &x, &y))
            return fail(ZR_EINVAL, "%s: buffers %d and %d overlap", who, x, y);
    }
    if (numel == 0)
        return ZR_OK;
    const auto g = static_cast<const uint16_t *>(grad);
    const auto p = static_cast<uint16_t *>(param_out);
    const auto st = static_cast<hipStream_t>(stream);
    const AdamWScalars a = adamw_scalars(*hp);
    return f16 ? adamw_clip_run<StepF16>(g, master, exp_avg, exp_avg_sq, p, numel, a, ls, clip, st)
               : adamw_clip_run<StepBF16>(g, master, exp_avg, exp_avg_sq, p, numel, a, ls, clip, st);
}

}  // namespace
}  // namespace zr

using namespace zr;

extern "C" zr_status zr_grad_norm(const void *const *grads, const int64_t *numels, int32_t n, zr_dtype dtype,
                                  const zr_clip_hparams *hp, int32_t accumulate, zr_loss_scale *ls, zr_clip *clip,
                                  double *workspace, void *stream)
{
    clear_error();
    const char *who = "zr_grad_norm";
    if (!hp)
        return fail(ZR_EINVAL, "%s: hp is NULL", who);
    if (!(hp->max_norm > 0.0))
        return fail(ZR_EINVAL, "%s: max_norm must be > 0", who);
    if (!(hp->eps >= 0.0) || !std::isfinite(hp->eps) || !std::isfinite(hp->grad_scale))
        return fail(ZR_EINVAL, "%s: eps must be finite and >= 0, grad_scale finite", who);
    if (accumulate != 0 && accumulate != 1)
        return fail(ZR_EINVAL, "%s: accumulate must be 0 or 1", who);
    zr_status s = check_clip(who, clip);
    if (s != ZR_OK)
        return s;
    if (!workspace)
        return fail(ZR_EINVAL, "%s: workspace is NULL", who);
    if (!aligned_to(workspace, 8) || !aligned_to(ls, 4))
        return fail(ZR_EALIGN, "%s: workspace must be 8-byte and the loss-scale record 4-byte aligned", who);
    const void *p[3] = {clip, workspace, ls};
    const int64_t b[3] = {(int64_t)sizeof(zr_clip), ZR_GRAD_NORM_PARTIALS * 8, (int64_t)sizeof(zr_loss_scale)};
    int x, y;
    if (any_overlap(p, b, 3, &x, &y))
        return fail(ZR_EINVAL, "%s: record, workspace and loss-scale record overlap", who);
    s = check_list(who, grads, numels, n, dtype, p, b, 3);
    if (s != ZR_OK)
        return s;
    const NormFinish f{hp->max_norm, hp->eps, hp->grad_scale, accumulate, ls, clip};
    const auto st = static_cast<hipStream_t>(stream);
    if (dtype == ZR_F32)
        return grad_norm_run<F32>(grads, numels, n, 4, workspace, f, st);
    return dtype == ZR_BF16 ? grad_norm_run<BF16>(grads, numels, n, 2, workspace, f, st)
                            : grad_norm_run<F16>(grads, numels, n, 2, workspace, f, st);
}

extern "C" zr_status zr_clip_grads(void *const *grads, const int64_t *numels, int32_t n, zr_dtype dtype,
                                   const zr_clip *clip, void *stream)
{
    clear_error();
    const char *who = "zr_clip_grads";
    zr_status s = check_clip(who, clip);
    if (s != ZR_OK)
        return s;
    const void *p[1] = {clip};
    const int64_t b[1] = {(int64_t)sizeof(zr_clip)};
    s = check_list(who, grads, numels, n, dtype, p, b, 1);
    const int64_t size = dtype == ZR_F32 ? 4 : 2;
    if (s == ZR_OK)
        s = check_disjoint(who, grads, numels, n, size);
    if (s != ZR_OK)
        return s;
    const auto st = static_cast<hipStream_t>(stream);
    if (dtype == ZR_F32)
        return clip_run<F32>(grads, numels, n, size, clip, st);
    return dtype == ZR_BF16 ? clip_run<BF16>(grads, numels, n, size, clip, st)
                            : clip_run<F16>(grads, numels, n, size, clip, st);
}

extern "C" zr_status zr_adamw_step_clip(const void *grad, float *master, float *exp_avg, float *exp_avg_sq,
                                        void *param_out, int64_t numel, const zr_adamw_hparams *hp, const zr_clip *clip,
                                        void *stream)
{
    clear_error();
    return adamw_clip("zr_adamw_step_clip", false, grad, master, exp_avg, exp_avg_sq, param_out, numel, hp, nullptr, clip,
                      stream);
}

extern "C" zr_status zr_adamw_step_clip_f16(const void *grad, float *master, float *exp_avg, float *exp_avg_sq,
                                            void *param_out, int64_t numel, const zr_adamw_hparams *hp,
                                            const zr_loss_scale *ls, const zr_clip *clip, void *stream)
{
    clear_error();
    return adamw_clip("zr_adamw_step_clip_f16", true, grad, master, exp_avg, exp_avg_sq, param_out, numel, hp, ls, clip,
                      stream);
}
