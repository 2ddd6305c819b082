// Norm of queries and keys for each head with the rotation by their positions, and its
// backward pass (gfx950).
//
// Forward, per token and head: y = x * rstd * w, then pairs (a, b) of y turned by
// angle = position * inv_freq.  Backward: the gradient turned back, then the norm's:
// dw = sum g xh, dx = rstd * (g w - xh * mean(g w xh)).
//
// A head's row lies in a group of kGroupLanes lanes, a lane holding a chunk of V pairs
// (2V elements) as V words, a pair to a word: both elements of a pair are in one lane,
// and turning takes no exchange.  Where the pairs are halves of the row apart, a lane
// loads V elements of either half and the words are put together by byte permutes; where
// they are neighbours the loaded words are the pairs.  A wave works on 64 / kGroupLanes
// heads of one token at a time, so that a token's sines and cosines, taken once by the
// wave (a lane to a pair) and handed over through LDS, serve all its heads.
#include "fp8.hpp"
#include "zr_rope.h"

namespace zr {

constexpr int kMaxPairs = ZR_MAX_HEAD_DIM / 2;

// One tensor's side of a call; heads 0: not there.
struct HeadRows {
    const uint16_t *x, *dy, *w;
    uint16_t *out;
    int64_t x_token, x_head, dy_token, dy_head, out_token, out_head;
    int32_t heads;
};

struct RopeArgs {
    HeadRows t[2];  // queries, keys
    int64_t tokens, position_stride;
    const int64_t *positions;
    const float *inv_freq;
    float *partial;
    int32_t dim, rot, interleaved, parts[2];
    float eps;
    uint8_t axis[kMaxPairs];
};

// A vector of V 16-bit elements at any element.
template <int V>
struct Vec;
template <>
struct Vec<8> {
    typedef any_u32x4 type;
};
template <>
struct Vec<4> {
    typedef any_u32x2 type;
};

// Where a lane's chunk lies in a row: the first elements of its two vectors.  `second` is
// false where the second (single-element chunks of an odd rest) is past the row.
struct Chunk {
    int32_t first, other;
    bool live, second, turned;
};

template <int V>
__device__ __forceinline__ Chunk chunk_of(int32_t c, const RopeArgs &a)
{
    const int32_t turned = a.rot / (2 * V);
    Chunk k;
    k.turned = c < turned;
    const bool halves = k.turned && !a.interleaved;
    k.first = halves ? V * c : 2 * V * c;
    k.other = halves ? a.rot / 2 + V * c : 2 * V * c + V;
    k.live = k.first < a.dim;
    k.second = k.other < a.dim;
    return k;
}

// A chunk as pairs, one to a word.
template <int V>
__device__ __forceinline__ void load_pairs(const uint16_t *row, const Chunk &k, bool live, int32_t interleaved,
                                           uint32_t (&w)[V])
{
    if constexpr (V == 1) {
        w[0] = 0;
        if (live) {
            w[0] = load_global(row + k.first);
            if (k.second)
                w[0] |= (uint32_t)load_global(row + k.other) << 16;
        }
    } else {
        typedef typename Vec<V>::type vec;
        vec p{}, q{};
        if (live) {
            p = *(global_ptr<const vec>)(row + k.first);
            q = *(global_ptr<const vec>)(row + k.other);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t halves = __builtin_amdgcn_perm(q[i / 2], p[i / 2], i % 2 ? 0x07060302 : 0x05040100);
            w[i] = interleaved ? (i < V / 2 ? p[i % (V / 2)] : q[i % (V / 2)]) : halves;
        }
    }
}

template <int V>
__device__ __forceinline__ void store_pairs(uint16_t *row, const Chunk &k, int32_t interleaved, const uint32_t (&w)[V])
{
    if constexpr (V == 1) {
        *(global_ptr<uint16_t>)(row + k.first) = (uint16_t)w[0];
        if (k.second)
            *(global_ptr<uint16_t>)(row + k.other) = (uint16_t)(w[0] >> 16);
    } else {
        typedef typename Vec<V>::type vec;
        vec p, q;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            p[i] = interleaved ? w[i] : __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x05040100);
            q[i] = interleaved ? w[V / 2 + i] : __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x07060302);
        }
        *(global_ptr<vec>)(row + k.first) = p;
        *(global_ptr<vec>)(row + k.other) = q;
    }
}

// Sum over each group of kLanes lanes, the same bits in all of them.
template <int kLanes>
__device__ __forceinline__ float lanes_sum(float a)
{
    const auto swap = [](float x, auto move) { return __uint_as_float(move(__float_as_uint(x))); };
    if constexpr (kLanes >= 2)
        a += swap(a, dpp_move<0xb1>);
    if constexpr (kLanes >= 4)
        a += swap(a, dpp_move<0x4e>);
    if constexpr (kLanes >= 8)
        a += swap(a, dpp_move<0x141>);
    if constexpr (kLanes >= 16)
        a += swap(a, dpp_move<0x140>);
    if constexpr (kLanes >= 32)
        a += __shfl_xor(a, 16, 64);
    if constexpr (kLanes >= 64)
        a += __shfl_xor(a, 32, 64);
    return a;
}

// LDS written by a wave's lanes is read by the same wave's others: no barrier between
// waves, only the order of the wave's own accesses.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Cosines and sines of a token's pairs, a pair to a lane at a time, in the wave's own LDS.
__device__ __forceinline__ void turn_pairs(const RopeArgs &a, int64_t token, float2 *turn)
{
    wave_fence();  // the token before has been read
    for (int32_t j = threadIdx.x & 63; j < a.rot / 2; j += 64) {
        const double position = (double)a.positions[(int64_t)a.axis[j] * a.position_stride + token];
        const double turns = position * (double)a.inv_freq[j] * 0.15915494309189535;  // 1 / (2 pi)
        float s, c;
        sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &c);
        turn[j] = float2{c, s};
    }
    wave_fence();
}

// A lane's own pairs' cosines and sines (1 and 0 outside the turned part, where they are
// not used).
template <int V>
__device__ __forceinline__ void read_turns(const float2 *turn, int32_t c, bool turned, float (&cs)[V], float (&sn)[V])
{
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 t = turned ? turn[c * V + e] : float2{1.0f, 0.0f};
        cs[e] = t.x;
        sn[e] = t.y;
    }
}

__device__ __forceinline__ float head_rstd(float squares, const RopeArgs &a)
{
    return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(squares, (float)a.dim) + a.eps));
}

constexpr int kRopeThreads = 256;

// kSteps: steps (of 64 / kLanes heads of one tensor each) that a wave takes of a token;
// kChunks: chunks of a row to a lane.
template <typename T, int V, int kLanes, int kChunks, int kSteps>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a, int32_t q_steps, int32_t steps, int32_t splits)
{
    __shared__ float2 turns[kRopeThreads / 64][kMaxPairs];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int32_t group = lane / kLanes;
    constexpr int kHeads = 64 / kLanes;
    Chunk k[kChunks];
    uint32_t w[2][kChunks][V];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        k[i] = chunk_of<V>(lane % kLanes + i * 64, a);
#pragma unroll
        for (int t = 0; t < 2; ++t)
            load_pairs<V>(a.t[t].w, k[i], k[i].live && a.t[t].w, a.interleaved, w[t][i]);
    }
    const int64_t units = a.tokens * splits;
    for (int64_t u = (int64_t)blockIdx.x * (kRopeThreads / 64) + wave; u < units;
         u += (int64_t)gridDim.x * (kRopeThreads / 64)) {
        const int64_t token = u / splits;
        const int32_t first = (int32_t)(u - token * splits) * kSteps;
        uint32_t x[kSteps][kChunks][V];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const HeadRows &t = a.t[first + s >= q_steps];
            const int32_t head = (first + s - (first + s >= q_steps ? q_steps : 0)) * kHeads + group;
            const bool live = first + s < steps && head < t.heads;
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                load_pairs<V>(t.x + token * t.x_token + head * t.x_head, k[i], live && k[i].live, a.interleaved, x[s][i]);
        }
        float cs[kChunks][V], sn[kChunks][V];
        if (a.rot > 0)
            turn_pairs(a, token, turns[wave]);
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            read_turns<V>(turns[wave], lane % kLanes + i * 64, k[i].turned, cs[i], sn[i]);
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int keys = first + s >= q_steps;
            const HeadRows &t = a.t[keys];
            const int32_t head = (first + s - (keys ? q_steps : 0)) * kHeads + group;
            const bool live = first + s < steps && head < t.heads;
            float rstd = 1.0f;
            if (t.w) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        sum = __builtin_fmaf(T::lo(x[s][i][e]), T::lo(x[s][i][e]), sum);
                        sum = __builtin_fmaf(T::hi(x[s][i][e]), T::hi(x[s][i][e]), sum);
                    }
                rstd = head_rstd(lanes_sum<kLanes>(sum), a);
            }
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                uint32_t o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float p = T::lo(x[s][i][e]), q = T::hi(x[s][i][e]);
                    if (t.w) {
                        const uint32_t we = keys ? w[1][i][e] : w[0][i][e];
                        p = p * rstd * T::lo(we);
                        q = q * rstd * T::hi(we);
                    }
                    const float pt = __builtin_fmaf(p, cs[i][e], -(q * sn[i][e]));
                    const float qt = __builtin_fmaf(q, cs[i][e], p * sn[i][e]);
                    o[e] = k[i].turned ? T::pack(pt, qt) : T::pack(p, q);
                }
                if (live && k[i].live)
                    store_pairs<V>(t.out + token * t.out_token + head * t.out_head, k[i], a.interleaved, o);
            }
        }
    }
}

// ------------------------------------------------------------------ backward --

constexpr int kRopeGradThreads = 512;

// Workgroups take parts: the first parts[0] queries', the others keys'; a wave of part p
// takes every parts * 8'th token with all its heads, and sums the weight gradient of its
// lanes' chunks over them.
template <typename T, int V, int kLanes, int kChunks>
__global__ __launch_bounds__(kRopeGradThreads) void rope_grad_kernel(RopeArgs a)
{
    constexpr int kWaves = kRopeGradThreads / 64, kHeads = 64 / kLanes;
    __shared__ float2 turns[kWaves][kMaxPairs];
    __shared__ float sums[kWaves][ZR_MAX_HEAD_DIM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Chunk k[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
        k[i] = chunk_of<V>(lane % kLanes + i * 64, a);
    for (int32_t part = blockIdx.x; part < a.parts[0] + a.parts[1]; part += gridDim.x) {
        const int keys = part >= a.parts[0];
        const HeadRows &t = a.t[keys];
        const int32_t p = part - (keys ? a.parts[0] : 0), parts = a.parts[keys];
        uint32_t w[kChunks][V];
        float acc[kChunks][2 * V];
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            load_pairs<V>(t.w, k[i], k[i].live && t.w, a.interleaved, w[i]);
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                acc[i][e] = 0.0f;
        }
        for (int64_t token = (int64_t)p * kWaves + wave; token < a.tokens; token += (int64_t)parts * kWaves) {
            float cs[kChunks][V], sn[kChunks][V];
            if (a.rot > 0)
                turn_pairs(a, token, turns[wave]);
#pragma unroll
            for (int i = 0; i < kChunks; ++i)
                read_turns<V>(turns[wave], lane % kLanes + i * 64, k[i].turned, cs[i], sn[i]);
            for (int32_t head = lane / kLanes; head - lane / kLanes < t.heads; head += kHeads) {
                const bool live = head < t.heads;
                uint32_t dy[kChunks][V], x[kChunks][V];
                float g[kChunks][2 * V], squares = 0.0f, dot = 0.0f;
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    load_pairs<V>(t.dy + token * t.dy_token + head * t.dy_head, k[i], live && k[i].live, a.interleaved, dy[i]);
                    load_pairs<V>(t.x + token * t.x_token + head * t.x_head, k[i], live && k[i].live && t.w, a.interleaved,
                                  x[i]);
                }
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float da = T::lo(dy[i][e]), db = T::hi(dy[i][e]);
                        g[i][2 * e] = k[i].turned ? __builtin_fmaf(da, cs[i][e], db * sn[i][e]) : da;
                        g[i][2 * e + 1] = k[i].turned ? __builtin_fmaf(db, cs[i][e], -(da * sn[i][e])) : db;
                        const float xa = T::lo(x[i][e]), xb = T::hi(x[i][e]);
                        squares = __builtin_fmaf(xa, xa, squares);
                        squares = __builtin_fmaf(xb, xb, squares);
                        dot = __builtin_fmaf(g[i][2 * e] * T::lo(w[i][e]), xa, dot);
                        dot = __builtin_fmaf(g[i][2 * e + 1] * T::hi(w[i][e]), xb, dot);
                    }
                if (t.w) {
                    squares = lanes_sum<kLanes>(squares);
                    dot = lanes_sum<kLanes>(dot);
                    const float rstd = head_rstd(squares, a);
                    const float along = __fdiv_rn(dot, (float)a.dim) * rstd * rstd;
#pragma unroll
                    for (int i = 0; i < kChunks; ++i)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float xa = T::lo(x[i][e]), xb = T::hi(x[i][e]);
                            float &ga = g[i][2 * e], &gb = g[i][2 * e + 1];
                            acc[i][2 * e] = __builtin_fmaf(ga, live ? xa * rstd : 0.0f, acc[i][2 * e]);
                            acc[i][2 * e + 1] = __builtin_fmaf(gb, live ? xb * rstd : 0.0f, acc[i][2 * e + 1]);
                            ga = __builtin_fmaf(-along, xa, ga * T::lo(w[i][e])) * rstd;
                            gb = __builtin_fmaf(-along, xb, gb * T::hi(w[i][e])) * rstd;
                        }
                }
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    uint32_t o[V];
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        o[e] = T::pack(g[i][2 * e], g[i][2 * e + 1]);
                    if (live && k[i].live)
                        store_pairs<V>(t.out + token * t.out_token + head * t.out_head, k[i], a.interleaved, o);
                }
            }
        }
        if (!t.w)
            continue;
        // the wave's groups, then the workgroup's waves, each in a fixed order
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) {
#pragma unroll
                for (int m = kLanes; m < 64; m *= 2)
                    acc[i][e] += __shfl_xor(acc[i][e], m, 64);
                const bool b = e & 1;
                const int32_t at = a.interleaved || V == 1 ? k[i].first + e : (b ? k[i].other : k[i].first) + e / 2;
                const int32_t column = V == 1 && b ? k[i].other : at;
                if (lane < kLanes && k[i].live && column < a.dim)
                    sums[wave][column] = acc[i][e];
            }
        __syncthreads();
        for (int32_t c = threadIdx.x; c < a.dim; c += kRopeGradThreads) {
            float sum = sums[0][c];
#pragma unroll
            for (int i = 1; i < kWaves; ++i)
                sum += sums[i][c];
            a.partial[(int64_t)part * a.dim + c] = sum;
        }
        __syncthreads();
    }
}

// Weight gradients from the partial sums: a workgroup takes 32 columns of one tensor, 16
// threads to a column, each every 16th partial sum; they meet in LDS in that order.
template <typename T>
__global__ __launch_bounds__(kRopeGradThreads) void rope_dweight_kernel(const float *partial, int32_t dim, int32_t q_parts,
                                                                        int32_t k_parts, uint16_t *dq, uint16_t *dk)
{
    __shared__ float part[16][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int32_t blocks = (dim + 31) / 32;
    for (int32_t b = blockIdx.x; b < 2 * blocks; b += gridDim.x) {
        const bool keys = b >= blocks;
        const int32_t c = (b - (keys ? blocks : 0)) * 32 + x;
        uint16_t *out = keys ? dk : dq;
        const int32_t begin = keys ? q_parts : 0, end = begin + (keys ? k_parts : q_parts);
        float sum = 0.0f;
        if (c < dim)
#pragma unroll 8
            for (int32_t p = begin + y; p < end; p += 16)
                sum += partial[(int64_t)p * dim + c];
        part[y][x] = sum;
        __syncthreads();
        if (y == 0 && c < dim && out) {
#pragma unroll
            for (int i = 1; i < 16; ++i)
                sum += part[i][x];
            out[c] = narrow<T>(sum);
        }
        __syncthreads();
    }
}

namespace {

// Address range of a tensor's rows in bytes; false where a stride is too small for rows
// not to overlap, or the range does not fit int64.
bool heads_extent(const zr_heads &h, int64_t tokens, int64_t dim, int64_t *bytes)
{
    int64_t n0 = tokens, s0 = h.token_stride, n1 = h.heads, s1 = h.head_stride;
    if (n1 > 1 && (n0 <= 1 || s1 < s0)) {
        std::swap(n0, n1);
        std::swap(s0, s1);
    }
    // (n0, s0) is the inner axis, if there is one
    int64_t span = dim, step;
    for (const auto &axis : {std::pair<int64_t, int64_t>{n0, s0}, {n1, s1}}) {
        if (axis.first <= 1)
            continue;
        if (axis.second < span || __builtin_mul_overflow(axis.first - 1, axis.second, &step) ||
            __builtin_add_overflow(span, step, &span))
            return false;
    }
    return !__builtin_mul_overflow(span, (int64_t)2, bytes);
}

struct Checked {
    const void *p;
    int64_t bytes, token_bytes, row_bytes;  // row: what one token's heads span; 0: not a row of heads
};

// Whether two buffers share bytes.  Heads of the same token distance that lie in ranges
// of the token's row that do not meet (queries and keys of one fused row) share none.
bool meet(const Checked &a, const Checked &b)
{
    if (!a.p || !b.p || !overlaps(a.p, a.bytes, b.p, b.bytes))
        return false;
    if (a.row_bytes == 0 || b.row_bytes == 0 || a.token_bytes != b.token_bytes)
        return true;
    const int64_t row = a.token_bytes;
    if (a.row_bytes > row || b.row_bytes > row)
        return true;
    int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % row;
    if (apart < 0)
        apart += row;
    return apart < a.row_bytes || apart + b.row_bytes > row;
}

zr_status check_heads(const char *who, const char *name, const zr_heads *h, int64_t tokens, int64_t dim, int64_t heads,
                      Checked *out)
{
    *out = {nullptr, 0, 0, 0};
    if (heads == 0 || tokens == 0)
        return ZR_OK;
    if (!h || !h->ptr)
        return fail(ZR_EINVAL, "%s: %s is NULL", who, name);
    if (h->heads != heads)
        return fail(ZR_EINVAL, "%s: %s has %lld heads, %lld needed", who, name, (long long)h->heads, (long long)heads);
    if (!aligned_to(h->ptr, 2))
        return fail(ZR_EALIGN, "%s: %s must be 2-byte aligned", who, name);
    int64_t bytes;
    if (h->token_stride < 0 || h->head_stride < 0 || !heads_extent(*h, tokens, dim, &bytes))
        return fail(ZR_EINVAL, "%s: rows of %s overlap, or reach past int64", who, name);
    const int64_t row = ((heads - 1) * h->head_stride + dim) * 2;  // no overflow: part of the extent
    *out = {h->ptr, bytes, h->token_stride * 2, tokens > 1 ? row : 0};
    return ZR_OK;
}

zr_status check_rope(const char *who, zr_dtype dtype, int64_t tokens, int64_t head_dim, double eps,
                     const int64_t *positions, int64_t position_stride, const zr_rope *rope, const zr_heads *q,
                     const zr_heads *k)
{
    if (dtype != ZR_BF16 && dtype != ZR_F16)
        return fail(ZR_EINVAL, "%s: dtype = %d, must be ZR_BF16 or ZR_F16", who, dtype);
    if (tokens < 0 || head_dim < 1 || head_dim > ZR_MAX_HEAD_DIM)
        return fail(ZR_EINVAL, "%s: tokens < 0 or head_dim outside [1, %d]", who, ZR_MAX_HEAD_DIM);
    if (!(eps >= 0.0) || !std::isfinite(eps) || !std::isfinite((float)eps))
        return fail(ZR_EINVAL, "%s: eps must be finite and >= 0", who);
    if ((q && (q->heads < 0 || q->heads > 65536)) || (k && (k->heads < 0 || k->heads > 65536)))
        return fail(ZR_EINVAL, "%s: heads outside [0, 65536]", who);
    if (!rope)
        return fail(ZR_EINVAL, "%s: rope is NULL", who);
    if (rope->rot_dim < 0 || rope->rot_dim > head_dim || rope->rot_dim % 2)
        return fail(ZR_EINVAL, "%s: rot_dim = %d, must be even and within [0, head_dim]", who, rope->rot_dim);
    if (rope->axes < 1 || rope->axes > ZR_MAX_ROPE_AXES)
        return fail(ZR_EINVAL, "%s: axes = %d outside [1, %d]", who, rope->axes, ZR_MAX_ROPE_AXES);
    if (rope->interleaved != 0 && rope->interleaved != 1)
        return fail(ZR_EINVAL, "%s: interleaved must be 0 or 1", who);
    if (rope->pair_axis)
        for (int32_t j = 0; j < rope->rot_dim / 2; ++j)
            if (rope->pair_axis[j] >= rope->axes)
                return fail(ZR_EINVAL, "%s: pair_axis[%d] = %d, the call has %d axes", who, j, rope->pair_axis[j],
                            rope->axes);
    if (rope->rot_dim > 0 && tokens > 0) {
        if (!positions || !rope->inv_freq)
            return fail(ZR_EINVAL, "%s: positions or inv_freq is NULL", who);
        if (!aligned_to(positions, 8) || !aligned_to(rope->inv_freq, 4))
            return fail(ZR_EALIGN, "%s: positions must be 8-byte and inv_freq 4-byte aligned", who);
        int64_t n;
        if (rope->axes > 1 && (position_stride < tokens ||
                               __builtin_mul_overflow((int64_t)rope->axes, position_stride, &n) || n > INT64_MAX / 8))
            return fail(ZR_EINVAL, "%s: position_stride below tokens, or positions past int64", who);
    }
    return ZR_OK;
}

void fill_args(RopeArgs *a, int64_t tokens, int64_t head_dim, double eps, const int64_t *positions,
               int64_t position_stride, const zr_rope *rope)
{
    a->tokens = tokens;
    a->position_stride = position_stride;
    a->positions = positions;
    a->inv_freq = rope->inv_freq;
    a->partial = nullptr;
    a->dim = (int32_t)head_dim;
    a->rot = rope->rot_dim;
    a->interleaved = rope->interleaved;
    a->parts[0] = a->parts[1] = 0;
    a->eps = (float)eps;
    for (int32_t j = 0; j < kMaxPairs; ++j)
        a->axis[j] = rope->pair_axis && j < rope->rot_dim / 2 ? rope->pair_axis[j] : 0;
}

template <typename T, int V, int kLanes, int kChunks>
zr_status rope_launch(const RopeArgs &a, hipStream_t st)
{
    constexpr int heads = 64 / kLanes, kSteps = 4;
    const int32_t q_steps = (a.t[0].heads + heads - 1) / heads, steps = q_steps + (a.t[1].heads + heads - 1) / heads;
    const int32_t splits = (steps + kSteps - 1) / kSteps;
    const int64_t units = a.tokens * splits;
    return launch(rope_kernel<T, V, kLanes, kChunks, kSteps>, grid_of((units + 3) / 4), dim3(kRopeThreads), 0, st, a,
                  q_steps, steps, splits);
}

template <typename T, int V, int kLanes, int kChunks>
zr_status rope_grad_launch(const RopeArgs &a, hipStream_t st)
{
    return launch(rope_grad_kernel<T, V, kLanes, kChunks>, grid_of(a.parts[0] + a.parts[1]), dim3(kRopeGradThreads), 0, st,
                  a);
}

// Calls F with the layout of a row: vectors of 8 or 4 elements where both halves of the
// turned part and the rest are whole chunks, else single elements.
template <typename T, template <typename, int, int, int> class F>
zr_status for_layout(const RopeArgs &a, hipStream_t st)
{
    const int32_t rest = a.dim - a.rot;
    if (a.rot % 16 == 0 && rest % 16 == 0) {
        if (a.dim <= 64)
            return F<T, 8, 4, 1>::run(a, st);
        if (a.dim <= 128)
            return F<T, 8, 8, 1>::run(a, st);
        if (a.dim <= 256)
            return F<T, 8, 16, 1>::run(a, st);
        return F<T, 8, 32, 1>::run(a, st);
    }
    if (a.rot % 8 == 0 && rest % 8 == 0) {
        if (a.dim <= 128)
            return F<T, 4, 16, 1>::run(a, st);
        return F<T, 4, 64, 1>::run(a, st);
    }
    if (a.dim <= 128)
        return F<T, 1, 64, 1>::run(a, st);
    return F<T, 1, 64, 4>::run(a, st);
}

template <typename T, int V, int kLanes, int kChunks>
struct Forward {
    static zr_status run(const RopeArgs &a, hipStream_t st) { return rope_launch<T, V, kLanes, kChunks>(a, st); }
};
template <typename T, int V, int kLanes, int kChunks>
struct Backward {
    static zr_status run(const RopeArgs &a, hipStream_t st) { return rope_grad_launch<T, V, kLanes, kChunks>(a, st); }
};

int64_t heads_of(const zr_heads *h) { return h ? h->heads : 0; }
bool same_heads(const zr_heads *a, const zr_heads *b)
{
    return a && b && a->ptr == b->ptr && a->token_stride == b->token_stride && a->head_stride == b->head_stride;
}

}  // namespace
}  // namespace zr

using namespace zr;

extern "C" zr_status zr_qk_norm_rope(const zr_heads *q, const zr_heads *k, const void *q_weight, const void *k_weight,
                                     zr_dtype dtype, int64_t tokens, int64_t head_dim, double eps,
                                     const int64_t *positions, int64_t position_stride, const zr_rope *rope,
                                     const zr_heads *q_out, const zr_heads *k_out, void *stream)
{
    clear_error();
    const char *who = "zr_qk_norm_rope";
    zr_status s = check_rope(who, dtype, tokens, head_dim, eps, positions, position_stride, rope, q, k);
    if (s != ZR_OK)
        return s;
    const int64_t hq = heads_of(q), hk = heads_of(k);
    if (tokens == 0 || (hq == 0 && hk == 0))
        return ZR_OK;
    if (!aligned_to(q_weight, 2) || !aligned_to(k_weight, 2))
        return fail(ZR_EALIGN, "%s: weights must be 2-byte aligned", who);
    Checked c[8];
    if ((s = check_heads(who, "q_out", q_out, tokens, head_dim, hq, &c[0])) != ZR_OK ||
        (s = check_heads(who, "k_out", k_out, tokens, head_dim, hk, &c[1])) != ZR_OK ||
        (s = check_heads(who, "q", q, tokens, head_dim, hq, &c[2])) != ZR_OK ||
        (s = check_heads(who, "k", k, tokens, head_dim, hk, &c[3])) != ZR_OK)
        return s;
    c[4] = {q_weight, 2 * head_dim, 0, 0};
    c[5] = {k_weight, 2 * head_dim, 0, 0};
    const bool turned = rope->rot_dim > 0;
    c[6] = {turned ? positions : nullptr, 8 * ((rope->axes - 1) * (rope->axes > 1 ? position_stride : 0) + tokens), 0, 0};
    c[7] = {turned ? rope->inv_freq : nullptr, 2 * rope->rot_dim, 0, 0};
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 8; ++j) {
            const bool in_place = (i == 0 && j == 2 && same_heads(q_out, q)) || (i == 1 && j == 3 && same_heads(k_out, k));
            if (!in_place && meet(c[i], c[j]))
                return fail(ZR_EINVAL, "%s: an output overlaps another buffer", who);
        }
    RopeArgs a;
    fill_args(&a, tokens, head_dim, eps, positions, position_stride, rope);
    const zr_heads none{nullptr, 0, 0, 0};
    const zr_heads *in[2] = {hq ? q : &none, hk ? k : &none}, *out[2] = {hq ? q_out : &none, hk ? k_out : &none};
    const void *w[2] = {q_weight, k_weight};
    for (int t = 0; t < 2; ++t)
        a.t[t] = {static_cast<const uint16_t *>(in[t]->ptr), nullptr, static_cast<const uint16_t *>(w[t]),
                  static_cast<uint16_t *>(out[t]->ptr), in[t]->token_stride, in[t]->head_stride, 0, 0,
                  out[t]->token_stride, out[t]->head_stride, (int32_t)in[t]->heads};
    const auto st = static_cast<hipStream_t>(stream);
    return dtype == ZR_BF16 ? for_layout<BF16, Forward>(a, st) : for_layout<F16, Forward>(a, st);
}

extern "C" zr_status zr_qk_norm_rope_backward(const zr_heads *dq, const zr_heads *dk, const zr_heads *q, const zr_heads *k,
                                              const void *q_weight, const void *k_weight, zr_dtype dtype, int64_t tokens,
                                              int64_t head_dim, double eps, const int64_t *positions,
                                              int64_t position_stride, const zr_rope *rope, const zr_heads *dq_in,
                                              const zr_heads *dk_in, void *dq_weight, void *dk_weight, float *workspace,
                                              void *stream)
{
    clear_error();
    const char *who = "zr_qk_norm_rope_backward";
    zr_status s = check_rope(who, dtype, tokens, head_dim, eps, positions, position_stride, rope, dq, dk);
    if (s != ZR_OK)
        return s;
    const int64_t hq = heads_of(dq), hk = heads_of(dk);
    if ((q_weight && !dq_weight) || (k_weight && !dk_weight) || ((q_weight || k_weight) && !workspace))
        return fail(ZR_EINVAL, "%s: a weight without its gradient's buffer or without workspace", who);
    if (!q_weight)
        dq_weight = nullptr;
    if (!k_weight)
        dk_weight = nullptr;
    if (!q_weight && !k_weight)
        workspace = nullptr;
    if (!aligned_to(q_weight, 2) || !aligned_to(k_weight, 2) || !aligned_to(dq_weight, 2) || !aligned_to(dk_weight, 2) ||
        !aligned_to(workspace, 4))
        return fail(ZR_EALIGN, "%s: weights and their gradients must be 2-byte, the workspace 4-byte aligned", who);
    Checked c[13];
    if ((s = check_heads(who, "dq_in", dq_in, tokens, head_dim, hq, &c[0])) != ZR_OK ||
        (s = check_heads(who, "dk_in", dk_in, tokens, head_dim, hk, &c[1])) != ZR_OK ||
        (s = check_heads(who, "dq", dq, tokens, head_dim, hq, &c[5])) != ZR_OK ||
        (s = check_heads(who, "dk", dk, tokens, head_dim, hk, &c[6])) != ZR_OK ||
        (s = check_heads(who, "q", q, tokens, head_dim, q_weight ? hq : 0, &c[7])) != ZR_OK ||
        (s = check_heads(who, "k", k, tokens, head_dim, k_weight ? hk : 0, &c[8])) != ZR_OK)
        return s;
    c[2] = {dq_weight, 2 * head_dim, 0, 0};
    c[3] = {dk_weight, 2 * head_dim, 0, 0};
    c[4] = {workspace, 4 * ZR_QK_PARTIALS * head_dim, 0, 0};
    c[9] = {q_weight, 2 * head_dim, 0, 0};
    c[10] = {k_weight, 2 * head_dim, 0, 0};
    const bool turned = rope->rot_dim > 0 && tokens > 0;
    c[11] = {turned ? positions : nullptr, 8 * ((rope->axes - 1) * (rope->axes > 1 ? position_stride : 0) + tokens), 0, 0};
    c[12] = {turned ? rope->inv_freq : nullptr, 2 * rope->rot_dim, 0, 0};
    for (int i = 0; i < 5; ++i)
        for (int j = i + 1; j < 13; ++j) {
            const bool in_place = (i == 0 && ((j == 5 && same_heads(dq_in, dq)) || (j == 7 && same_heads(dq_in, q)))) ||
                                  (i == 1 && ((j == 6 && same_heads(dk_in, dk)) || (j == 8 && same_heads(dk_in, k))));
            if (!in_place && meet(c[i], c[j]))
                return fail(ZR_EINVAL, "%s: an output overlaps another buffer", who);
        }
    RopeArgs a;
    fill_args(&a, tokens, head_dim, eps, positions, position_stride, rope);
    a.partial = workspace;
    const zr_heads none{nullptr, 0, 0, 0};
    const bool any = tokens > 0;
    const zr_heads *dy[2] = {hq && any ? dq : &none, hk && any ? dk : &none};
    const zr_heads *x[2] = {hq && any && q_weight ? q : &none, hk && any && k_weight ? k : &none};
    const zr_heads *out[2] = {hq && any ? dq_in : &none, hk && any ? dk_in : &none};
    const void *w[2] = {q_weight, k_weight};
    for (int t = 0; t < 2; ++t)
        a.t[t] = {static_cast<const uint16_t *>(x[t]->ptr), static_cast<const uint16_t *>(dy[t]->ptr),
                  static_cast<const uint16_t *>(w[t]), static_cast<uint16_t *>(out[t]->ptr), x[t]->token_stride,
                  x[t]->head_stride, dy[t]->token_stride, dy[t]->head_stride, out[t]->token_stride, out[t]->head_stride,
                  (int32_t)dy[t]->heads};
    // parts go to the tensors by their heads, at most one to 8 tokens
    const int64_t most = (tokens + 7) / 8, heads = a.t[0].heads + a.t[1].heads;
    for (int t = 0; t < 2; ++t)
        if (a.t[t].heads > 0) {
            int64_t share = ZR_QK_PARTIALS * a.t[t].heads / heads;
            share = share < 1 ? 1 : share > ZR_QK_PARTIALS - 1 && a.t[1 - t].heads > 0 ? ZR_QK_PARTIALS - 1 : share;
            a.parts[t] = (int32_t)(share < most ? share : most);
        }
    const auto st = static_cast<hipStream_t>(stream);
    if (a.parts[0] + a.parts[1] > 0) {
        s = dtype == ZR_BF16 ? for_layout<BF16, Backward>(a, st) : for_layout<F16, Backward>(a, st);
        if (s != ZR_OK)
            return s;
    }
    if (!dq_weight && !dk_weight)
        return ZR_OK;
    const dim3 grid = grid_of(2 * ((head_dim + 31) / 32)), block(kRopeGradThreads);
    const auto gq = static_cast<uint16_t *>(dq_weight), gk = static_cast<uint16_t *>(dk_weight);
    return dtype == ZR_BF16 ? launch(rope_dweight_kernel<BF16>, grid, block, 0, st, (const float *)workspace, a.dim, a.parts[0], a.parts[1], gq, gk)
                            : launch(rope_dweight_kernel<F16>, grid, block, 0, st, (const float *)workspace, a.dim, a.parts[0], a.parts[1], gq, gk);
}
