// Norm of queries and keys for each head with the rotation by their positions, and its
// backward pass (gfx950).
//
// Forward, per token and head: y = x * rstd * w, then pairs (a, b) of y turned by
// angle = position * inv_freq.  Backward: the gradient turned back, then the norm's:
// dw = sum g xh, dx = rstd * (g w - xh * mean(g w xh)).
//
// A head's row lies in a group of kLanes lanes, a lane holding a chunk of V pairs
// (2V elements) as V words, a pair to a word: both elements of a pair are in one lane,
// and turning takes no exchange.  Where the pairs are halves of the row apart, a lane
// loads V elements of either half and the words are put together by byte permutes; where
// they are neighbours the loaded words are the pairs.  A wave works on 64 / kLanes
// heads of one token at a time, so that a token's sines and cosines, taken once by the
// wave (a lane to a pair) and handed over through LDS, serve all its heads.
#include <algorithm>

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
    int32_t dim, rot, axes, interleaved;
    int32_t parts[2];  // units of a token (forward) or sums (backward) of each tensor
    int32_t per[2];    // steps of a unit
    float eps, inv_dim;
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
    typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2)));
};

// Chunks of V pairs that the turned part of a row has, and the rest behind it (in vectors, two
// to a chunk).  Pairs half the turned part apart take a vector of either half, neighbours
// vectors of the whole part.
template <int V>
__host__ __device__ __forceinline__ int32_t turned_chunks(int32_t rot, bool neighbours)
{
    return neighbours && V > 1 ? ((rot + V - 1) / V + 1) / 2 : (rot / 2 + V - 1) / V;
}
template <int V>
__host__ __device__ __forceinline__ int32_t rest_chunks(int32_t rest)
{
    return ((rest + V - 1) / V + 1) / 2;
}

// Where a lane's chunk lies in a row: two vectors of V elements, neighbouring lanes' side by
// side.  The last vector of a part ends where the part ends, and so may begin before
// the end of the one before it: its first `skip` elements are that one's.  They are worked out
// twice, with the same result, and counted once; a rest shorter than a vector begins
// among turned elements (`crosses`), which its lane must not store.  A chunk that the row does not
// have is moved to its first elements.
struct Chunk {
    int32_t first, other, skip_first, skip_other;
    bool live, turned, crosses;
};

template <int V>
__device__ __forceinline__ Chunk chunk_of(int32_t c, const RopeArgs &a)
{
    const int32_t rest = a.dim - a.rot, half = a.rot / 2, turned = turned_chunks<V>(a.rot, a.interleaved);
    Chunk k = {0, 0, V, V, false, false, false};
    // vector i of a part of n elements from `begin` on
    const auto vector = [](int32_t i, int32_t begin, int32_t n, int32_t &at, int32_t &skip) {
        const int32_t from = V * i < n - V ? V * i : n - V;
        at = begin + from;
        skip = V * i - from < V ? V * i - from : V;
    };
    if (c < turned) {
        k.live = k.turned = true;
        if (!a.interleaved) {
            vector(c, 0, half, k.first, k.skip_first);
            k.other = half + k.first;
            k.skip_other = k.skip_first;
        } else if (V == 1) {
            k.first = 2 * c;
            k.other = 2 * c + 1;
            k.skip_first = k.skip_other = 0;
        } else {
            vector(c, 0, a.rot, k.first, k.skip_first);
            vector(c + turned, 0, a.rot, k.other, k.skip_other);
        }
    } else if (c < turned + rest_chunks<V>(rest)) {
        k.live = true;
        k.crosses = rest < V;
        vector(c - turned, a.rot, rest, k.first, k.skip_first);
        vector(c - turned + rest_chunks<V>(rest), a.rot, rest, k.other, k.skip_other);
    }
    return k;
}

// A chunk's words, a pair to a word, are made of its two vectors' words p, q by byte
// permutes: words 2i and 2i + 1 are the low and the high halves of q[i] and p[i] where pairs
// are halves of the row apart, and p[i] and q[i] themselves where they are neighbours.  The
// same selectors turn the words back.
struct Selectors {
    uint32_t even, odd;

    __device__ __forceinline__ explicit Selectors(const RopeArgs &a)
        : even(a.interleaved ? 0x03020100u : 0x05040100u), odd(a.interleaved ? 0x07060504u : 0x07060302u)
    {
    }
};

// The pair in word e of a turned chunk.
template <int V>
__device__ __forceinline__ int32_t pair_of(const Chunk &k, int e, const RopeArgs &a)
{
    if (V > 1 && a.interleaved)
        return (e % 2 ? k.other : k.first) / 2 + e / 2;
    return V == 1 && a.interleaved ? k.first / 2 : k.first + e;
}

// The column of element b (0: first, 1: second) of word e, and whether the chunk counts it.
template <int V>
__device__ __forceinline__ int32_t column_of(const Chunk &k, int e, int b, const RopeArgs &a)
{
    if (V > 1 && a.interleaved)
        return (e % 2 ? k.other : k.first) + e / 2 * 2 + b;
    return (b ? k.other : k.first) + e;
}
template <int V>
__device__ __forceinline__ bool counts(const Chunk &k, int e, int b, const RopeArgs &a)
{
    if (V > 1 && a.interleaved)
        return e / 2 * 2 + b >= (e % 2 ? k.skip_other : k.skip_first);
    return e >= (b ? k.skip_other : k.skip_first);
}

// A lane's place in the rows of one buffer: the offsets of its chunks' two vectors from the
// first head of a step.
template <int V, int kChunks>
struct Offsets {
    int64_t head, first[kChunks], other[kChunks];

    __device__ __forceinline__ Offsets(const Chunk (&k)[kChunks], int32_t group, int64_t head_stride)
        : head(group * head_stride)
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            first[i] = head + k[i].first;
            other[i] = head + k[i].other;
        }
    }
};

// A row's chunks as they lie in memory.  Every lane loads: one whose chunk is not in the
// row (or whose head is not there) loads another's, which is not used, so that no load waits
// for a branch and none is used before all of them are on their way.
template <int V, int kChunks>
struct Loaded {
    typename Vec<V>::type p[kChunks], q[kChunks];

    // `step` points to the step's first head; where the lane's own head is not there (`back`)
    // it takes that one.
    __device__ __forceinline__ void load(const uint16_t *step, const Offsets<V, kChunks> &o, bool back)
    {
        typedef typename Vec<V>::type vec;
        const uint16_t *row = step - (back ? o.head : 0);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            p[i] = *(global_ptr<const vec>)(row + o.first[i]);
            q[i] = *(global_ptr<const vec>)(row + o.other[i]);
        }
    }

    __device__ __forceinline__ void pairs(int i, const Chunk &, const Selectors &sel, uint32_t (&w)[V]) const
    {
#pragma unroll
        for (int e = 0; e < V; ++e)
            w[e] = __builtin_amdgcn_perm(q[i][e / 2], p[i][e / 2], e % 2 ? sel.odd : sel.even);
    }
};

template <int kChunks>
struct Loaded<1, kChunks> {
    uint16_t p[kChunks], q[kChunks];

    __device__ __forceinline__ void load(const uint16_t *step, const Offsets<1, kChunks> &o, bool back)
    {
        const uint16_t *row = step - (back ? o.head : 0);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            p[i] = load_global(row + o.first[i]);
            q[i] = load_global(row + o.other[i]);
        }
    }

    __device__ __forceinline__ void pairs(int i, const Chunk &k, const Selectors &, uint32_t (&w)[1]) const
    {
        w[0] = p[i] | (k.skip_other == 0 ? (uint32_t)q[i] << 16 : 0);
    }
};

template <bool kRagged, int V, int kChunks>
__device__ __forceinline__ void store_pairs(uint16_t *step, const Offsets<V, kChunks> &o, int i, const Chunk &k,
                                            const Selectors &sel, const uint32_t (&w)[V])
{
    if constexpr (V == 1) {
        *(global_ptr<uint16_t>)(step + o.first[i]) = (uint16_t)w[0];
        if (k.skip_other == 0)
            *(global_ptr<uint16_t>)(step + o.other[i]) = (uint16_t)(w[0] >> 16);
    } else {
        typedef typename Vec<V>::type vec;
        vec p, q;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            p[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], sel.even);
            q[j] = __builtin_amdgcn_perm(w[2 * j + 1], w[2 * j], sel.odd);
        }
        if (kRagged && k.crosses) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (e >= k.skip_first)
                    *(global_ptr<uint16_t>)(step + o.first[i] + e) = (uint16_t)(p[e / 2] >> (16 * (e % 2)));
                if (e >= k.skip_other)
                    *(global_ptr<uint16_t>)(step + o.other[i] + e) = (uint16_t)(q[e / 2] >> (16 * (e % 2)));
            }
            return;
        }
        __builtin_nontemporal_store(p, (global_ptr<vec>)(step + o.first[i]));
        __builtin_nontemporal_store(q, (global_ptr<vec>)(step + o.other[i]));
    }
}

// Sum of u * v over the elements of a chunk that it counts; 0 for a chunk that is not there.
template <int V, bool kRagged>
__device__ __forceinline__ float dot_of(const Chunk &k, const RopeArgs &a, const float (&u)[2 * V], const float (&v)[2 * V])
{
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 2 * V; ++e) {
        const float next = __builtin_fmaf(u[e], v[e], sum);
        sum = !kRagged || counts<V>(k, e / 2, e % 2, a) ? next : sum;
    }
    return k.live ? sum : 0.0f;
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

// Cosines and sines of a token's pairs, a pair to a lane at a time (kPairs to a lane), in
// the wave's own LDS.  The frequencies stay in registers from token to token, positions are
// asked for ahead.
template <int kPairs>
struct Turns {
    double freq[kPairs];  // turns for a position of 1
    const int64_t *at[kPairs];
    int64_t position[kPairs];

    __device__ __forceinline__ explicit Turns(const RopeArgs &a)
    {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const int32_t j = (threadIdx.x & 63) + 64 * i;
            const bool live = j < a.rot / 2;
            freq[i] = live ? (double)a.inv_freq[j] * 0.15915494309189535 : 0.0;  // 1 / (2 pi)
            at[i] = a.positions + (a.axes > 1 && live ? (int64_t)a.axis[j] * a.position_stride : 0);
        }
    }

    __device__ __forceinline__ void ask(const RopeArgs &a, int64_t token)
    {
        if (a.rot > 0)
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                position[i] = load_global(at[i] + token);
    }

    __device__ __forceinline__ void write(const RopeArgs &a, float2 *turn) const
    {
        if (a.rot == 0)
            return;
        wave_fence();  // the token before has been read
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const double turns = (double)position[i] * freq[i];
            float s, c;
            sincospif(2.0f * (float)(turns - __builtin_rint(turns)), &s, &c);
            turn[(threadIdx.x & 63) + 64 * i] = float2{c, s};
        }
        wave_fence();
    }
};

// 1 / sqrt(mean + eps).  The hardware's reciprocal root is right to one unit in the last
// place for all but subnormal arguments, which only an eps near 0 lets through.
__device__ __forceinline__ float head_rstd(float squares, const RopeArgs &a)
{
    if (a.eps >= 0x1p-100f)
        return __builtin_amdgcn_rsqf(__builtin_fmaf(squares, a.inv_dim, a.eps));
    return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(squares, (float)a.dim) + a.eps));
}

// Pairs to a lane when a wave takes a token's sines: rows of kLanes lanes of kChunks
// chunks of V pairs.
template <int V, int kLanes, int kChunks>
constexpr int kPairsOf = (V * kLanes * kChunks + 63) / 64;

// What the waves of both passes share: one tensor's rows.  A step is 64 / kLanes heads of a
// token, a unit `per` steps of one token; backward, a wave takes every stride'th unit.
template <typename T, int V, int kLanes, int kChunks>
struct HeadWave {
    static constexpr int kHeads = 64 / kLanes;
    const RopeArgs &a;
    const HeadRows t;  // a copy: read from the arguments once, not at every step
    const Selectors sel;
    const int32_t group, steps, per, splits;
    const int64_t stride, units;
    const bool mixed;  // part of the row is not turned
    Chunk k[kChunks];
    float w[kChunks][2 * V];  // pairs, first and second element by turns; 1 without a weight

    // A place in the wave's work: a step of a unit, up to step `end`.
    struct Place {
        int64_t unit, token;
        int32_t step, end;
    };

    __device__ __forceinline__ HeadWave(const RopeArgs &args, int keys, int64_t stride_)
        : a(args), t(args.t[keys]), sel(args), group((threadIdx.x & 63) / kLanes), steps((t.heads + kHeads - 1) / kHeads),
          per(args.per[keys]), splits((steps + per - 1) / per), stride(stride_), units(args.tokens * splits),
          mixed(args.rot < args.dim)
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
            k[i] = chunk_of<V>((threadIdx.x & 63) % kLanes + i * 64, a);
        Loaded<V, kChunks> l = {};
        if (t.w)
            l.load(t.w, Offsets<V, kChunks>(k, 0, 0), false);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            uint32_t p[V];
            l.pairs(i, k[i], sel, p);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                w[i][2 * e] = t.w ? T::lo(p[e]) : 1.0f;
                w[i][2 * e + 1] = t.w ? T::hi(p[e]) : 1.0f;
            }
        }
    }

    __device__ __forceinline__ int64_t token_of(int64_t unit) const { return splits == 1 ? unit : unit / splits; }

    __device__ __forceinline__ Place place(int64_t unit) const
    {
        const int64_t token = token_of(unit);
        const int32_t step = (int32_t)(unit - token * splits) * per;
        return {unit, token, step, step + per < steps ? step + per : steps};
    }

    __device__ __forceinline__ Place next(const Place &p) const
    {
        return p.step + 1 < p.end ? Place{p.unit, p.token, p.step + 1, p.end} : place(p.unit + stride);
    }

    __device__ __forceinline__ bool has_head(const Place &p) const { return p.step * kHeads + group < t.heads; }

    __device__ __forceinline__ int64_t at(const Place &p, int64_t token_stride, int64_t head_stride) const
    {
        return p.token * token_stride + (int64_t)p.step * kHeads * head_stride;
    }

    // A lane's own pairs' cosines and sines (1 and 0 outside the turned part).
    __device__ __forceinline__ void read_turns(const float2 *turn, float (&cs)[kChunks][V], float (&sn)[kChunks][V]) const
    {
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 r = turn[k[i].turned ? pair_of<V>(k[i], e, a) : 0];
                cs[i][e] = r.x;
                sn[i][e] = r.y;
            }
            if (mixed)
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    cs[i][e] = k[i].turned ? cs[i][e] : 1.0f;
                    sn[i][e] = k[i].turned ? sn[i][e] : 0.0f;
                }
        }
    }
};

constexpr int kRopeThreads = 256;

// Workgroups go round four tokens at a time: parts[0] of them take the queries' units, parts[1]
// the keys', a wave one unit of at most kSteps steps of its token, so that a token's heads,
// which lie together in memory, are read together.  The loads of all steps go out before
// the sines are worked out.
// With the weight multiplied into the cosines and sines once for the unit, an element of a
// step costs three operations: out_a = (x_a rstd) (w_a cos) - (x_b rstd) (w_b sin).
// Bound by HBM where rows are whole vectors and batches large: 16384 tokens of 40 heads of 128
// 57.4 us, 5.8 TB/s (units of mixed queries and keys 63.6, keys' units behind all queries' 64,
// loads behind branches 70); by arithmetic where lanes are idle (72 elements, 9 of 16 lanes:
// 4.3 TB/s).  One token 4 us, a launch and two round trips to memory.
template <typename T, int V, int kLanes, int kChunks, bool kRagged, int kSteps>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a)
{
    constexpr int kWaves = kRopeThreads / 64;
    __shared__ float2 turns[kWaves][64 * kPairsOf<V, kLanes, kChunks>];
    typedef HeadWave<T, V, kLanes, kChunks> Wave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Turns<kPairsOf<V, kLanes, kChunks>> turn(a);
    const int32_t splits = a.parts[0] + a.parts[1];
    const int64_t blocks = (a.tokens + kWaves - 1) / kWaves * splits;
    for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {
        const int64_t four = block / splits;
        const int32_t split = (int32_t)(block - four * splits);
        const int keys = split >= a.parts[0];
        const Wave me(a, keys, 1);
        const HeadRows &t = me.t;
        const Offsets<V, kChunks> in(me.k, me.group, t.x_head), out(me.k, me.group, t.out_head);
        const int64_t token = four * kWaves + wave;
        if (token >= a.tokens)
            continue;
        turn.ask(a, token);
        const int32_t first = (split - (keys ? a.parts[0] : 0)) * me.per;
        const int32_t count = first + me.per < me.steps ? me.per : me.steps - first;
        typename Wave::Place p{0, token, first, 0};
        Loaded<V, kChunks> rows[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
            if (s < count) {
                p.step = first + s;
                rows[s].load(t.x + me.at(p, t.x_token, t.x_head), in, !me.has_head(p));
            }
        turn.write(a, turns[wave]);
        float ca[kChunks][V], sb[kChunks][V], cb[kChunks][V], sa[kChunks][V];
        me.read_turns(turns[wave], ca, sb);
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float wa = me.w[i][2 * e], wb = me.w[i][2 * e + 1];
                cb[i][e] = ca[i][e] * wb;
                sa[i][e] = sb[i][e] * wa;
                ca[i][e] *= wa;
                sb[i][e] *= wb;
            }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            if (s >= count)
                continue;
            p.step = first + s;
            float x[kChunks][2 * V];
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                uint32_t pair[V];
                rows[s].pairs(i, me.k[i], me.sel, pair);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[i][2 * e] = T::lo(pair[e]);
                    x[i][2 * e + 1] = T::hi(pair[e]);
                }
            }
            float rstd = 1.0f;
            if (t.w) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
                    sum += dot_of<V, kRagged>(me.k[i], a, x[i], x[i]);
                rstd = head_rstd(lanes_sum<kLanes>(sum), a);
            }
            uint16_t *to = t.out + me.at(p, t.out_token, t.out_head);
            const bool live = me.has_head(p);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                uint32_t o[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    float &xa = x[i][2 * e], &xb = x[i][2 * e + 1];
                    xa *= rstd;
                    xb *= rstd;
                    o[e] = T::pack(__builtin_fmaf(xa, ca[i][e], -(xb * sb[i][e])),
                                   __builtin_fmaf(xb, cb[i][e], xa * sa[i][e]));
                }
                if (me.mixed) {  // no infinity of a pair's other half in what is not turned
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const uint32_t straight = T::pack(x[i][2 * e] * ca[i][e], x[i][2 * e + 1] * cb[i][e]);
                        o[e] = me.k[i].turned ? o[e] : straight;
                    }
                }
                if (live && me.k[i].live)
                    store_pairs<kRagged, V, kChunks>(to, out, i, me.k[i], me.sel, o);
            }
        }
    }
}

// ------------------------------------------------------------------ backward --

constexpr int kRopeGradThreads = 256;

// Workgroups take sums: the first parts[0] the queries', the others the keys'; a wave of sum p
// takes every parts * 4'th unit and sums the weight gradient of its lanes' chunks over them.
// The next step's rows, of the next unit too, are asked for before the present ones are
// worked on; two steps ahead (107 us), or 12 waves to a compute unit for 8 (105), were slower.
// 16384 tokens of 40 heads of 128: 97 us, 5.2 TB/s, and 5 for the sums of the sums.
template <typename T, int V, int kLanes, int kChunks, bool kRagged>
__global__ __launch_bounds__(kRopeGradThreads) void rope_grad_kernel(RopeArgs a)
{
    constexpr int kWaves = kRopeGradThreads / 64;
    __shared__ float2 turns[kWaves][64 * kPairsOf<V, kLanes, kChunks>];
    __shared__ float sums[kWaves][2 * V * kLanes * kChunks];
    typedef HeadWave<T, V, kLanes, kChunks> Wave;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Turns<kPairsOf<V, kLanes, kChunks>> turn(a);
    for (int64_t part = blockIdx.x; part < a.parts[0] + a.parts[1]; part += gridDim.x) {
        const int keys = part >= a.parts[0];
        const Wave me(a, keys, (int64_t)a.parts[keys] * kWaves);
        const HeadRows &t = me.t;
        const Offsets<V, kChunks> in(me.k, me.group, t.x_head), grad(me.k, me.group, t.dy_head),
            out(me.k, me.group, t.out_head);
        float acc[kChunks][2 * V];
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e)
                acc[i][e] = 0.0f;
        Loaded<V, kChunks> dy = {}, xr = {};
        const auto ask = [&](const typename Wave::Place &p) {
            dy.load(t.dy + me.at(p, t.dy_token, t.dy_head), grad, !me.has_head(p));
            if (t.w)
                xr.load(t.x + me.at(p, t.x_token, t.x_head), in, !me.has_head(p));
        };
        typename Wave::Place p = me.place((part - (keys ? a.parts[0] : 0)) * kWaves + wave);
        if (p.unit < me.units) {
            turn.ask(a, p.token);
            ask(p);
        }
        float cs[kChunks][V], sn[kChunks][V];
        for (int64_t turned = -1; p.unit < me.units;) {
            if (p.unit != turned) {
                turned = p.unit;
                turn.write(a, turns[wave]);
                me.read_turns(turns[wave], cs, sn);
                if (p.unit + me.stride < me.units)
                    turn.ask(a, me.token_of(p.unit + me.stride));
            }
            float g[kChunks][2 * V], x[kChunks][2 * V];
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                uint32_t dw[V], xw[V];
                dy.pairs(i, me.k[i], me.sel, dw);
                xr.pairs(i, me.k[i], me.sel, xw);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float da = T::lo(dw[e]), db = T::hi(dw[e]);
                    g[i][2 * e] = __builtin_fmaf(da, cs[i][e], db * sn[i][e]);
                    g[i][2 * e + 1] = __builtin_fmaf(db, cs[i][e], -(da * sn[i][e]));
                    x[i][2 * e] = T::lo(xw[e]);
                    x[i][2 * e + 1] = T::hi(xw[e]);
                }
                if (me.mixed)  // no infinity of a pair's other half
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        g[i][2 * e] = me.k[i].turned ? g[i][2 * e] : T::lo(dw[e]);
                        g[i][2 * e + 1] = me.k[i].turned ? g[i][2 * e + 1] : T::hi(dw[e]);
                    }
            }
            const typename Wave::Place ahead = me.next(p);
            if (ahead.unit < me.units)
                ask(ahead);
            const bool live = me.has_head(p);
            if (t.w) {
                float squares = 0.0f;
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
                    squares += dot_of<V, kRagged>(me.k[i], a, x[i], x[i]);
                const float rstd = head_rstd(lanes_sum<kLanes>(squares), a);
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e)
                        x[i][e] *= rstd;
                if (live)  // one that is not there stands for the step's first head
#pragma unroll
                    for (int i = 0; i < kChunks; ++i)
#pragma unroll
                        for (int e = 0; e < 2 * V; ++e)
                            acc[i][e] = __builtin_fmaf(g[i][e], x[i][e], acc[i][e]);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e)
                        g[i][e] *= me.w[i][e];
                    dot += dot_of<V, kRagged>(me.k[i], a, g[i], x[i]);
                }
                const float along = lanes_sum<kLanes>(dot) * a.inv_dim;
#pragma unroll
                for (int i = 0; i < kChunks; ++i)
#pragma unroll
                    for (int e = 0; e < 2 * V; ++e)
                        g[i][e] = __builtin_fmaf(-along, x[i][e], g[i][e]) * rstd;
            }
            uint16_t *to = t.out + me.at(p, t.out_token, t.out_head);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                uint32_t o[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o[e] = T::pack(g[i][2 * e], g[i][2 * e + 1]);
                if (live && me.k[i].live)
                    store_pairs<kRagged, V, kChunks>(to, out, i, me.k[i], me.sel, o);
            }
            p = ahead;
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
                if (lane < kLanes && me.k[i].live && ((V > 1 && !kRagged) || counts<V>(me.k[i], e / 2, e % 2, a)))
                    sums[wave][column_of<V>(me.k[i], e / 2, e % 2, a)] = acc[i][e];
            }
        __syncthreads();
        for (int32_t c = threadIdx.x; c < a.dim; c += kRopeGradThreads) {
            float sum = sums[0][c];
#pragma unroll
            for (int i = 1; i < kWaves; ++i)
                sum += sums[i][c];
            a.partial[part * a.dim + c] = sum;
        }
        __syncthreads();
    }
}

// Partial sums that a call makes, at most: two workgroups to a compute unit.
constexpr int64_t kGradParts = 512;
static_assert(kGradParts <= ZR_QK_PARTIALS, "the workspace holds them");

constexpr int kDweightThreads = 512;

// Weight gradients from the partial sums: a workgroup takes 32 columns of one tensor, 16
// threads to a column, each every 16th partial sum; they meet in LDS in that order.
template <typename T>
__global__ __launch_bounds__(kDweightThreads) void rope_dweight_kernel(const float *partial, int32_t dim, int32_t q_parts,
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
    if (tokens < 0 || tokens > (int64_t)1 << 40 || head_dim < 1 || head_dim > ZR_MAX_HEAD_DIM)
        return fail(ZR_EINVAL, "%s: tokens outside [0, 2^40] or head_dim outside [1, %d]", who, ZR_MAX_HEAD_DIM);
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
        if (rope->axes > 1 && ((position_stride != 0 && position_stride < tokens) ||
                               __builtin_mul_overflow((int64_t)rope->axes, position_stride, &n) || n > INT64_MAX / 8))
            return fail(ZR_EINVAL, "%s: position_stride below tokens and not 0, or positions past int64", who);
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
    a->axes = rope->pair_axis ? rope->axes : 1;
    a->interleaved = rope->interleaved;
    a->parts[0] = a->parts[1] = 0;
    a->per[0] = a->per[1] = 1;
    a->eps = (float)eps;
    a->inv_dim = 1.0f / (float)head_dim;
    for (int32_t j = 0; j < kMaxPairs; ++j)
        a->axis[j] = rope->pair_axis && j < rope->rot_dim / 2 ? rope->pair_axis[j] : 0;
}

// Steps of a call up to which a wave takes one.  Replayed graphs, 32 + 8 heads of 128, one step to a
// wave and up to four: 160 steps 3.1 us and 4.0, 1280 3.5 and 4.1, 2050 3.8 and 4.2, 4000 4.5 and 4.7,
// 5120 4.9 and 4.7, 20480 12.4 and 9.1 (heads of 80 and of 64 the same): they cross between 4000
// and 5000.
constexpr int64_t kFewSteps = 2048;

template <typename T, int V, int kLanes, int kChunks, bool kRagged, int kSteps>
zr_status rope_steps(RopeArgs *a, hipStream_t st)
{
    constexpr int kHeads = 64 / kLanes, kWaves = kRopeThreads / 64;
    for (int t = 0; t < 2; ++t) {
        const int64_t steps = (a->t[t].heads + kHeads - 1) / kHeads, splits = (steps + kSteps - 1) / kSteps;
        a->per[t] = splits > 0 ? (int32_t)((steps + splits - 1) / splits) : 1;
        a->parts[t] = (int32_t)((steps + a->per[t] - 1) / a->per[t]);
    }
    const int64_t blocks = (a->tokens + kWaves - 1) / kWaves * (a->parts[0] + a->parts[1]);
    return launch(rope_kernel<T, V, kLanes, kChunks, kRagged, kSteps>, grid_of(blocks), dim3(kRopeThreads), 0, st, *a);
}

// Few tokens: a wave to a step, for latency.  Else a unit is a token's steps, four at most.
template <typename T, int V, int kLanes, int kChunks, bool kRagged>
zr_status rope_launch(RopeArgs *a, hipStream_t st)
{
    constexpr int kHeads = 64 / kLanes;
    const int64_t steps = (a->t[0].heads + kHeads - 1) / kHeads + (a->t[1].heads + kHeads - 1) / kHeads;
    return a->tokens * steps <= kFewSteps ? rope_steps<T, V, kLanes, kChunks, kRagged, 1>(a, st)
                                          : rope_steps<T, V, kLanes, kChunks, kRagged, 4>(a, st);
}

// Divides a backward pass among kGradParts workgroups of `waves` waves: per and parts of each
// tensor, for `steps` steps a token.  A unit costs its steps and half of one for its sines;
// every wave of a tensor takes the same number of units, and the most that any wave takes
// is as little as the workgroups allow (units of two steps where one does not give less).
void divide_backward(RopeArgs *a, const int64_t (&steps)[2], int64_t waves)
{
    int64_t best = 0;
    for (int32_t pair = 3; pair >= 0; --pair) {
        const int64_t per[2] = {1 + (pair & 1), 1 + (pair >> 1)};
        if ((per[0] > 1 && per[0] > steps[0]) || (per[1] > 1 && per[1] > steps[1]))
            continue;
        int64_t units[2], parts[2];
        for (int t = 0; t < 2; ++t)
            units[t] = a->tokens * ((steps[t] + per[t] - 1) / per[t]);
        // workgroups that waves with work for `most` half steps need
        const auto needed = [&](int64_t most) {
            for (int t = 0; t < 2; ++t) {
                const int64_t each = waves * (most / (2 * per[t] + 1));  // units of a workgroup
                parts[t] = units[t] == 0 ? 0 : each == 0 ? kGradParts + 1 : (units[t] + each - 1) / each;
            }
            return parts[0] + parts[1];
        };
        // from what an even division would give, up in steps of at most a 500th
        int64_t low = 1 + (units[0] * (2 * per[0] + 1) + units[1] * (2 * per[1] + 1)) / (kGradParts * waves);
        while (needed(low) > kGradParts && (best == 0 || low < best))
            low += 1 + low / 512;
        if (best == 0 || low < best) {
            best = low;
            needed(low);
            for (int t = 0; t < 2; ++t) {
                a->per[t] = (int32_t)per[t];
                a->parts[t] = (int32_t)parts[t];
            }
        }
    }
}

template <typename T, int V, int kLanes, int kChunks, bool kRagged>
zr_status rope_grad_launch(RopeArgs *a, hipStream_t st)
{
    constexpr int kHeads = 64 / kLanes;
    divide_backward(a, {(a->t[0].heads + kHeads - 1) / kHeads, (a->t[1].heads + kHeads - 1) / kHeads}, kRopeGradThreads / 64);
    return launch(rope_grad_kernel<T, V, kLanes, kChunks, kRagged>, grid_of(a->parts[0] + a->parts[1]),
                  dim3(kRopeGradThreads), 0, st, *a);
}

// Lanes for the chunks of a row, the least of 4 ... 64 (0: more than a wave has); 0 also where a
// vector is longer than what it has to lie in.
template <int V>
int32_t lanes_of(const RopeArgs &a)
{
    if (a.dim < V || (a.rot > 0 && (a.interleaved ? a.rot : a.rot / 2) < V))
        return 0;
    const int32_t chunks = turned_chunks<V>(a.rot, a.interleaved) + rest_chunks<V>(a.dim - a.rot);
    for (int32_t lanes = 4; lanes <= 64; lanes *= 2)
        if (chunks <= lanes)
            return lanes;
    return 0;
}

// Whether the last vector of a part begins before the end of the one before it.
template <int V>
bool ragged(const RopeArgs &a)
{
    return (a.interleaved ? a.rot % (2 * V) : a.rot / 2 % V) != 0 || (a.dim - a.rot) % (2 * V) != 0;
}

template <typename T, bool kForward, int V, int kLanes, int kChunks, bool kRagged>
zr_status layout_launch(RopeArgs *a, hipStream_t st)
{
    if constexpr (kForward)
        return rope_launch<T, V, kLanes, kChunks, kRagged>(a, st);
    else
        return rope_grad_launch<T, V, kLanes, kChunks, kRagged>(a, st);
}

template <typename T, bool kForward, int V, bool kRagged>
zr_status vector_launch(RopeArgs *a, int32_t lanes, hipStream_t st)
{
    switch (lanes) {
    case 4: return layout_launch<T, kForward, V, 4, 1, kRagged>(a, st);
    case 8: return layout_launch<T, kForward, V, 8, 1, kRagged>(a, st);
    case 16: return layout_launch<T, kForward, V, 16, 1, kRagged>(a, st);
    case 32: return layout_launch<T, kForward, V, 32, 1, kRagged>(a, st);
    default: break;
    }
    // 32 chunks of 8 pairs are the longest row: only a ragged one has 33
    constexpr int kMost = V == 8 && !kRagged ? 32 : 64;
    return layout_launch<T, kForward, V, kMost, 1, kRagged>(a, st);
}

constexpr int64_t kFewBackward = 4096;

// Forward, vectors of 4 elements leave room for 7 waves to a SIMD where those of 8 leave 4
// (replayed graphs: 5003 tokens of 24 heads of 96 13.4 us and 15.6; 16384 of 40 of 128 58.1 and 65.9).
// Backward, where sums stay in registers anyway, 8 take half as many steps (124 us with 4, 98 with 8),
// but where those are few, what counts is how long one takes, and the sums behind it (40 heads of
// 128, with 8 and with 4: 64 tokens 8.2 us and 6.7, 777 12.5 and 12.9, 2048 19.6 and 22.7).
// What those do not fit (65 chunks forward; parts shorter than a vector) takes the other
// kind, heads too short for both single elements: 16384 tokens of 40 heads of 128 of which 6
// elements are turned 129 us forward, 2.6 TB/s, and 376 backward; 4096 of 256, 90 and 158 (three sets
// of buffers in turn).
template <typename T, bool kForward>
zr_status for_layout(RopeArgs *a, hipStream_t st)
{
    const int32_t four = lanes_of<4>(*a), eight = lanes_of<8>(*a);
    if constexpr (kForward) {
        if (four)
            return ragged<4>(*a) ? vector_launch<T, true, 4, true>(a, four, st) : vector_launch<T, true, 4, false>(a, four, st);
        if (eight)
            return layout_launch<T, true, 8, 64, 1, true>(a, st);
    } else {
        // steps of 64 / lanes heads
        const bool few = eight && a->tokens <= kFewBackward &&
                         a->tokens * ((a->t[0].heads * eight + 63) / 64 + (a->t[1].heads * eight + 63) / 64) <= kFewBackward;
        if (eight && !(few && four))
            return ragged<8>(*a) ? vector_launch<T, false, 8, true>(a, eight, st) : vector_launch<T, false, 8, false>(a, eight, st);
        if (four)
            return vector_launch<T, false, 4, true>(a, four, st);
    }
    if (a->dim <= 128)
        return layout_launch<T, kForward, 1, 64, 1, false>(a, st);
    return layout_launch<T, kForward, 1, 64, 4, false>(a, st);
}

int64_t heads_of(const zr_heads *h) { return h ? h->heads : 0; }
// Whether two tensors' rows are the same ones: the distance along an axis of length 1 says nothing.
bool same_heads(const zr_heads *a, const zr_heads *b, int64_t tokens)
{
    return a && b && a->ptr == b->ptr && (tokens <= 1 || a->token_stride == b->token_stride) &&
           (a->heads <= 1 || a->head_stride == b->head_stride);
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
            const bool in_place = (i == 0 && j == 2 && same_heads(q_out, q, tokens)) ||
                                  (i == 1 && j == 3 && same_heads(k_out, k, tokens));
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
    return dtype == ZR_BF16 ? for_layout<BF16, true>(&a, st) : for_layout<F16, true>(&a, st);
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
            const bool in_place =
                (i == 0 && ((j == 5 && same_heads(dq_in, dq, tokens)) || (j == 7 && same_heads(dq_in, q, tokens)))) ||
                (i == 1 && ((j == 6 && same_heads(dk_in, dk, tokens)) || (j == 8 && same_heads(dk_in, k, tokens))));
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
    const auto st = static_cast<hipStream_t>(stream);
    if (a.t[0].heads + a.t[1].heads > 0) {
        s = dtype == ZR_BF16 ? for_layout<BF16, false>(&a, st) : for_layout<F16, false>(&a, st);
        if (s != ZR_OK)
            return s;
    }
    if (!dq_weight && !dk_weight)
        return ZR_OK;
    const dim3 grid = grid_of(2 * ((head_dim + 31) / 32)), block(kDweightThreads);
    const auto gq = static_cast<uint16_t *>(dq_weight), gk = static_cast<uint16_t *>(dk_weight);
    return dtype == ZR_BF16 ? launch(rope_dweight_kernel<BF16>, grid, block, 0, st, (const float *)workspace, a.dim, a.parts[0], a.parts[1], gq, gk)
                            : launch(rope_dweight_kernel<F16>, grid, block, 0, st, (const float *)workspace, a.dim, a.parts[0], a.parts[1], gq, gk);
}
