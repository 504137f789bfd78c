// mru_gated_tile.cuh -- tiles of the gated recurrence: how a tile of 64 tokens
// and 64 channels is brought on chip and how its carry is found.
#pragma once

#include "mru_ops.cuh"

namespace mru {
namespace gated {

using namespace ops;

constexpr int kTok = MRU_GATED_KEEP;     // tokens of a tile: a kept state per tile
constexpr int kWarps = 8;
constexpr int kStep = kTok / kWarps;     // tokens of a warp
constexpr int kThreads = 32 * kWarps;
constexpr int kFan = 8;                  // tiles of a group, groups of a block of the carry's tree

struct Args {
    int64_t B, L, D, ld, ldg;
    int64_t K;                           // tiles (kept states) per sequence, ceil(L / 64)
    float c;
    const void *x, *f, *i;
    mru_packed8 x8, f8, i8;              // forward: written; backward: read
    const float *lam, *h0;
    const uint8_t* reset;
    const int32_t* lens;
    // forward
    void* y;
    float *h_last, *states;
    // backward
    const void* dy;
    const float* dh_last;
    void *dx, *df, *di;
    float *dlam_part, *dh0;
    float *edge_h, *edge_d, *edge_q;     // 8-bit copies, a piece's first token: h_{t-1}, d and q d, [B, K, D] each
    // carry of the tiles of a sequence
    uint32_t* status;
    uint32_t* ticket;                    // next tile to draw
    uint32_t* abort;                     // a wait gave up
    uint64_t *a0, *a1, *c2;              // aggregates of tiles and of groups, carries into blocks
    uint32_t tiles, cols, cgs;           // tiles in all; columns (a tile's channels of a sequence); those per sequence
    uint32_t groups, blocks;             // groups and blocks per column
    uint64_t wait_ns;
    int32_t withhold;                    // testing: the first tile publishes nothing
};

__device__ __forceinline__ int64_t valid_tokens(const Args& g, int64_t b)
{
    if (!g.lens) return g.L;
    const int64_t n = g.lens[b];
    return n < 0 ? 0 : n < g.L ? n : g.L;
}

// a h where a = 0 forgets h whatever it is.
__device__ __forceinline__ float carry_in(float a, float h) { return a == 0.0f ? 0.0f : a * h; }

// Decay and input of a token; csp = c softplus(lam), NEAR: csp <= 0.5.
template <int GATE, bool NEAR = false>
__device__ __forceinline__ void gates(float x, float f, float i, float csp, float& a, float& b)
{
    if constexpr (GATE == MRU_GATE_DECAY) {
        a = f;
        b = x;
    } else if constexpr (GATE == MRU_GATE_SIGMOID) {
        float na;
        sigmoid2(f, a, na);
        b = na * x;
    } else {
        float m;                                      // a - 1
        exp_expm1_neg<NEAR>(-csp * sigmoid(f), a, m);
        b = root(-m * (1.0f + a)) * sigmoid(i) * x;   // 1 - a^2 = -m (1 + a)
    }
}

// The states of a lane's C channels, and the map h -> P h + H of a run of
// tokens on them.
template <int C>
struct Vec {
    float v[C];
};
template <int C>
struct Map {
    float P[C], H[C];
    __device__ __forceinline__ static Map of(float p)
    {
        Map m;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            m.P[c] = p;
            m.H[c] = 0.0f;
        }
        return m;
    }
    // this one after `first`
    __device__ __forceinline__ Map after(const Map& first) const
    {
        Map m;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            m.P[c] = P[c] * first.P[c];
            m.H[c] = carry_in(P[c], first.H[c]) + H[c];
        }
        return m;
    }
    __device__ __forceinline__ Vec<C> operator()(const Vec<C>& h) const
    {
        Vec<C> r;
#pragma unroll
        for (int c = 0; c < C; ++c) r.v[c] = carry_in(P[c], h.v[c]) + H[c];
        return r;
    }
};
// A row of maps in shared memory, (P, H, P, H) of two channels to 16 bytes.
template <int C>
struct MapRow {
    float4 q[C / 2][32];
    __device__ __forceinline__ void put(int lane, const Map<C>& m)
    {
#pragma unroll
        for (int k = 0; k < C / 2; ++k)
            q[k][lane] = make_float4(m.P[2 * k], m.H[2 * k], m.P[2 * k + 1], m.H[2 * k + 1]);
    }
    __device__ __forceinline__ Map<C> get(int lane) const
    {
        Map<C> m;
#pragma unroll
        for (int k = 0; k < C / 2; ++k) {
            const float4 v = q[k][lane];
            m.P[2 * k] = v.x;
            m.H[2 * k] = v.y;
            m.P[2 * k + 1] = v.z;
            m.H[2 * k + 1] = v.w;
        }
        return m;
    }
};

// ------------------------------------------------------------------ tiles ---

// Place of a tile, worked out by one thread for its block.  `order` counts
// along the scan (from the last tile in the backward).
struct Tile {
    uint32_t ticket, col, order;
    int32_t tokens, channels, valid;     // in the tile: tokens and channels there are, tokens that are not padding
    int64_t row, b;                      // first token's row, sequence
    int64_t d0, k;                       // first channel, index of its kept state
    int32_t last;                        // nothing is carried out of it
};

template <int C, bool REVERSE>
__device__ __forceinline__ void find_tile(const Args& g, uint32_t ticket, Tile& t)
{
    t.ticket = ticket;
    if (ticket >= g.tiles) return;
    const uint32_t order = ticket / g.cols, col = ticket - order * g.cols, b = col / g.cgs;
    const int64_t t0 = (REVERSE ? g.K - 1 - (int64_t)order : (int64_t)order) * kTok;
    const int64_t d0 = (int64_t)(col - b * g.cgs) * (32 * C), left = valid_tokens(g, b) - t0;
    t.order = order;
    t.col = col;
    t.tokens = (int32_t)(g.L - t0 < kTok ? g.L - t0 : kTok);
    t.channels = (int32_t)(g.D - d0 < 32 * C ? g.D - d0 : 32 * C);
    t.valid = left <= 0 ? 0 : left < kTok ? (int32_t)left : kTok;
    t.row = b * g.L + t0;
    t.b = b;
    t.d0 = d0;
    t.k = b * g.K + t0 / kTok;
    t.last = order + 1 == (uint32_t)g.K;
}

// Draws the next tile, in the order of the scan.  A tile waits only for tiles
// drawn before it, and a block works through its tiles in the order drawn, so
// the earliest unfinished tile never waits.
__device__ __forceinline__ uint32_t draw(const Args& g, uint32_t before)
{
    return g.ticket ? atomicAdd(g.ticket, 1u) : before + gridDim.x;
}

// A warp's tokens that are not padding, and which of them start anew.
__device__ __forceinline__ void warp_masks(const Args& g, const Tile& t, int w, int lane, int& n, uint32_t& resets)
{
    n = min(max(t.valid - w * kStep, 0), kStep);
    resets = 0;
    if (g.reset) resets = __ballot_sync(~0u, lane < n && g.reset[t.row + w * kStep + lane] != 0);
}

// ------------------------------------------------------------------ carry ---
//
// Tiles publish their maps, the last tile of 8 the composition of the group,
// and the last of 64 (a block) the state itself, so that a tile's carry is one
// block carry and at most 7 groups and 7 tiles, all in a fixed order: the same
// bits on every run, and a chain of one hop per 64 tiles.  A pair (P, H) of a
// channel is one 64-bit word, complemented so that zeroed memory reads as "not
// there yet" (no pair is all ones: such a NaN is published as another NaN):
// word and flag arrive together, which saves a fence before the flag and a
// round trip after it.

__device__ __forceinline__ uint64_t pair_word(float P, float H)
{
    uint32_t p = __float_as_uint(P);
    if (p == 0xffffffffu) p = 0x7fffffffu;
    return ~(((uint64_t)p << 32) | __float_as_uint(H));
}

template <int C>
__device__ __forceinline__ uint64_t* tile_words(const Args& g, const Tile& t, uint32_t order)
{
    return g.a0 + ((uint64_t)t.col * (uint64_t)g.K + order) * (32 * C);
}
template <int C>
__device__ __forceinline__ uint64_t* group_words(const Args& g, const Tile& t, uint32_t group)
{
    return g.a1 + ((uint64_t)t.col * g.groups + group) * (32 * C);
}
template <int C>
__device__ __forceinline__ uint64_t* block_words(const Args& g, const Tile& t, uint32_t block)
{
    return g.c2 + ((uint64_t)t.col * g.blocks + block) * (32 * C);
}

// Words [2 k, lane, 2]: 16 bytes of a lane next to its neighbours'.
template <int C>
__device__ __forceinline__ void publish(uint64_t* at, int lane, const Map<C>& m)
{
#pragma unroll
    for (int k = 0; k < C / 2; ++k)
        asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(at + 64 * k + 2 * lane),
                     "l"(pair_word(m.P[2 * k], m.H[2 * k])), "l"(pair_word(m.P[2 * k + 1], m.H[2 * k + 1]))
                     : "memory");
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

template <int C>
__device__ __forceinline__ bool peek(const uint64_t* at, int lane, uint64_t (&u)[C])
{
    bool there = true;
#pragma unroll
    for (int k = 0; k < C / 2; ++k)
        asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];"
                     : "=l"(u[2 * k]), "=l"(u[2 * k + 1])
                     : "l"(at + 64 * k + 2 * lane)
                     : "memory");
#pragma unroll
    for (int c = 0; c < C; ++c) there = there && u[c] != 0;
    return there;
}
template <int C>
__device__ __forceinline__ Map<C> map_of(const uint64_t (&u)[C])
{
    Map<C> m;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        m.P[c] = __uint_as_float((uint32_t)(~u[c] >> 32));
        m.H[c] = __uint_as_float((uint32_t)~u[c]);
    }
    return m;
}

// Waits for two published maps (either may be absent: the identity), for a
// limited time, and composes them, `one` first.
template <int C>
__device__ __forceinline__ Map<C> await(const Args& g, const uint64_t* one, const uint64_t* two, int lane)
{
    uint64_t u[C], v[C], t0 = 0;
    for (int n = 0;; ++n) {
        const bool a = !one || peek<C>(one, lane, u), b = !two || peek<C>(two, lane, v);
        if (__all_sync(~0u, a && b)) break;
        if ((n & 63) == 63) {
            uint32_t stop;
            asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(stop) : "l"(g.abort) : "memory");
            const uint64_t t = now_ns();
            if (t0 == 0) t0 = t;
            bool out = false;
            if (lane == 0 && t - t0 > g.wait_ns) {
                atomicOr(g.status, (uint32_t)STATUS_TIMEOUT);
                atomicExch(g.abort, 1u);
                out = true;
            }
            if (__any_sync(~0u, out || stop)) return Map<C>::of(1.0f);
        }
    }
    if (!one) return Map<C>::of(1.0f);
    const Map<C> first = map_of<C>(u);
    return two ? map_of<C>(v).after(first) : first;
}

// What a tile's carry is made of, in shared memory: [0 .. 3] the block's carry
// in and the block's groups before this one, [4 .. 7] the tiles before in the
// group; two to an entry, so that [0] is the carry in and group 0, [1] groups 1
// and 2, and so on.
template <int C>
struct Entries {
    MapRow<C> e[8];

    // Warp w fetches entry w.  `start` is the state before the first tile (h0,
    // or the last state's gradient).
    __device__ __forceinline__ void fetch(const Args& g, const Tile& t, int w, int lane, const float* start)
    {
        const uint32_t block = t.order / (kFan * kFan), group = t.order / kFan % kFan, j = t.order % kFan;
        if (w >= 4) {
            const uint32_t k = 2 * (w - 4);
            if (k < j) {
                const uint64_t* at = tile_words<C>(g, t, t.order - j + k);
                e[w].put(lane, await<C>(g, at, k + 1 < j ? at + 32 * C : nullptr, lane));
            }
        } else if (w == 0 && block == 0) {
            Map<C> m = Map<C>::of(0.0f);
            if (start) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (C * lane + c < t.channels) m.H[c] = start[t.b * g.D + t.d0 + C * lane + c];
            }
            e[0].put(lane, group ? await<C>(g, group_words<C>(g, t, 0), nullptr, lane).after(m) : m);
        } else if (2u * w <= group) {
            const uint64_t* at = group_words<C>(g, t, block * kFan + 2 * w);
            e[w].put(lane, await<C>(g, w ? at - 32 * C : block_words<C>(g, t, block), 2u * w < group ? at : nullptr, lane));
        }
    }
    __device__ __forceinline__ Vec<C> carry(const Tile& t, int lane) const
    {
        const uint32_t group = t.order / kFan % kFan, j = t.order % kFan;
        const Map<C> first = e[0].get(lane);
        Vec<C> h;
#pragma unroll
        for (int c = 0; c < C; ++c) h.v[c] = first.H[c];
        for (uint32_t k = 1; 2 * k <= group; ++k) h = e[k].get(lane)(h);
        for (uint32_t k = 0; 2 * k < j; ++k) h = e[4 + k].get(lane)(h);
        return h;
    }
    // After the carry is known: the group's map (last tile of a group) and the
    // next block's carry (last tile of a block), by one warp.
    __device__ __forceinline__ void publish_up(const Args& g, const Tile& t, int lane, const Map<C>& own,
                                               const Vec<C>& carry) const
    {
        if (t.last || t.order % kFan != kFan - 1) return;
        const uint32_t group = t.order / kFan;
        Map<C> m;
        if (group % kFan != kFan - 1) {
            m = e[4].get(lane);
            for (int k = 5; k < 8; ++k) m = e[k].get(lane).after(m);
            publish<C>(group_words<C>(g, t, group), lane, own.after(m));
        } else {
            const Vec<C> h = own(carry);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                m.P[c] = 0.0f;
                m.H[c] = h.v[c];
            }
            publish<C>(block_words<C>(g, t, group / kFan + 1), lane, m);
        }
    }
};

// ------------------------------------------------------- loads and stores ---

__device__ __forceinline__ void cp_async(void* smem, const void* gmem, int bytes16)
{
    const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(gmem), "r"(bytes16) : "memory");
}
__device__ __forceinline__ void cp_async4(void* smem, const void* gmem, int bytes4)
{
    const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(s), "l"(gmem), "r"(bytes4) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile of one input into shared memory [64][32 C], zeros past the last token
// or channel.  VEC: rows start on 16 bytes; else element by element.
template <typename T, int C, bool VEC>
__device__ __forceinline__ void load_tile(const Tile& t, const void* from, int64_t ld, T* to)
{
    constexpr int kCh = 32 * C;
    const T* src = (const T*)from + t.row * ld + t.d0;
    if constexpr (VEC) {
        constexpr int per = 16 / sizeof(T), chunks = kCh / per, rows = kThreads / chunks;
        const int row = threadIdx.x / chunks, c = threadIdx.x % chunks * per;
        const T* at = src + row * ld + c;
        T* put = to + row * kCh + c;
        const int bytes = c >= t.channels ? 0 : t.channels - c >= per ? 16 : (t.channels - c) * (int)sizeof(T);
        const int64_t jump = rows * ld;
#pragma unroll
        for (int k = 0; k < kTok / rows; ++k) {
            const bool in = row + k * rows < t.tokens && bytes > 0;
            cp_async(put + k * rows * kCh, in ? at : src, in ? bytes : 0);
            at += jump;
        }
    } else {
        for (int k = threadIdx.x; k < kTok * kCh; k += kThreads) {
            const int row = k / kCh, c = k % kCh;
            const bool in = row < t.tokens && c < t.channels;
            const T* at = in ? src + row * ld + c : src;
            if constexpr (sizeof(T) == 4) cp_async4(to + k, at, in ? 4 : 0);
            else to[k] = in ? *at : from_f32<T>(0.0f);
        }
    }
}

// C adjacent channels of a row.
template <int C>
__device__ __forceinline__ Vec<C> read_row(const float* p)
{
    Vec<C> r;
    if constexpr (C == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        r.v[0] = v.x; r.v[1] = v.y; r.v[2] = v.z; r.v[3] = v.w;
    } else {
        const float2 v = *reinterpret_cast<const float2*>(p);
        r.v[0] = v.x; r.v[1] = v.y;
    }
    return r;
}
template <int C>
__device__ __forceinline__ Vec<C> read_row(const __nv_bfloat16* p)
{
    Vec<C> r;
    uint32_t u[C / 2];
    if constexpr (C == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        u[0] = v.x; u[1] = v.y;
    } else {
        u[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int k = 0; k < C / 2; ++k) {
        r.v[2 * k] = __uint_as_float(u[k] << 16);
        r.v[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
    return r;
}

// Whether rows of C channels can be written in one piece, and how many
// channels of the lane there are otherwise.
struct Put {
    bool whole;
    int channels;
};
template <int C>
__device__ __forceinline__ void write_row(float* p, const Vec<C>& r, const Put& put)
{
    if (put.whole) {
        if constexpr (C == 4) *reinterpret_cast<float4*>(p) = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
        else *reinterpret_cast<float2*>(p) = make_float2(r.v[0], r.v[1]);
        return;
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (c < put.channels) p[c] = r.v[c];
}
template <int C>
__device__ __forceinline__ void write_row(__nv_bfloat16* p, const Vec<C>& r, const Put& put)
{
    if (put.whole) {
        uint32_t u[C / 2];
#pragma unroll
        for (int k = 0; k < C / 2; ++k) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(r.v[2 * k], r.v[2 * k + 1]);
            u[k] = *reinterpret_cast<const uint32_t*>(&h);
        }
        if constexpr (C == 4) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
        else *reinterpret_cast<uint32_t*>(p) = u[0];
        return;
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (c < put.channels) p[c] = __float2bfloat16_rn(r.v[c]);
}
// fp32 rows of one value per channel ([B, D] arrays).
template <int C>
__device__ __forceinline__ void write_state(float* p, const Vec<C>& r, int channels)
{
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (c < channels) p[c] = r.v[c];
}

}  // namespace gated
}  // namespace mru
