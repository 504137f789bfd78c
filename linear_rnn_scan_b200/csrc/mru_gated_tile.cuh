// mru_gated_tile.cuh -- tiles of the gated recurrence: how a tile of 64 tokens
// and 64 channels is brought on chip and how its carry is found.
#pragma once

#include "mru_ops.cuh"

namespace mru {
namespace gated {

using namespace ops;

constexpr int kTok = MRU_GATED_KEEP;     // tokens of a tile: a kept state per tile
constexpr int kCh = 64;                  // channels of a tile: two to a lane
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
    uint32_t tiles, cols, cgs;           // tiles in all; columns (64 channels of a sequence); those per sequence
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
        const float sf = __fdividef(1.0f, 1.0f + __expf(-f)), si = __fdividef(1.0f, 1.0f + __expf(-i));
        float m, u;                                   // a - 1; sqrt(1 - a^2), 1 - a^2 = -m (1 + a)
        exp_expm1_neg<NEAR>(-csp * sf, a, m);
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(u) : "f"(-m * (1.0f + a)));
        b = u * si * x;
    }
}

// ------------------------------------------------------------------ carry ---
//
// The map of a run of tokens is h -> P h + H.  Tiles publish theirs, the last
// tile of 8 the composition of the group, and the last of 64 (a block) the
// state itself, so that a tile's carry is one block carry and at most 7 groups
// and 7 tiles, all in a fixed order: the same bits on every run, and a chain
// of one hop per 64 tiles.  A pair (P, H) of a channel is one 64-bit word,
// complemented so that zeroed memory reads as "not there yet" (no pair is all
// ones: such a NaN is published as another NaN): word and flag arrive
// together, which saves a fence before the flag and a round trip after it.

__device__ __forceinline__ uint64_t pair_word(float P, float H)
{
    uint32_t p = __float_as_uint(P);
    if (p == 0xffffffffu) p = 0x7fffffffu;
    return ~(((uint64_t)p << 32) | __float_as_uint(H));
}

// Two channels of a lane: word 2 lane, 2 lane + 1 of the tile's 64.
__device__ __forceinline__ void publish(uint64_t* at, int lane, float4 v)
{
    asm volatile("st.relaxed.gpu.global.v2.b64 [%0], {%1, %2};" ::"l"(at + 2 * lane), "l"(pair_word(v.x, v.y)),
                 "l"(pair_word(v.z, v.w))
                 : "memory");
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Waits for a published pair of the lane's channels, for a limited time.
__device__ __forceinline__ float4 await(const Args& g, const uint64_t* at, int lane)
{
    uint64_t u, v, t0 = 0;
    for (int n = 0;; ++n) {
        asm volatile("ld.relaxed.gpu.global.v2.b64 {%0, %1}, [%2];" : "=l"(u), "=l"(v) : "l"(at + 2 * lane) : "memory");
        if (__all_sync(~0u, u != 0 && v != 0)) break;
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
            if (__any_sync(~0u, out || stop)) return make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        }
    }
    u = ~u;
    v = ~v;
    return make_float4(__uint_as_float((uint32_t)(u >> 32)), __uint_as_float((uint32_t)u),
                       __uint_as_float((uint32_t)(v >> 32)), __uint_as_float((uint32_t)v));
}

// The later map after the earlier one, two channels.
__device__ __forceinline__ float4 after(float4 later, float4 first)
{
    return make_float4(later.x * first.x, carry_in(later.x, first.y) + later.y, later.z * first.z,
                       carry_in(later.z, first.w) + later.w);
}
__device__ __forceinline__ float2 apply(float4 m, float2 h)
{
    return make_float2(carry_in(m.x, h.x) + m.y, carry_in(m.z, h.y) + m.w);
}

// Place of a tile: `order` counts along the scan (from the last tile in the
// backward).
struct Tile {
    uint32_t col, order;
    int64_t b, d0, t0;
    bool last;                           // nothing is carried out of it
};
template <bool REVERSE>
__device__ __forceinline__ Tile tile_of(const Args& g, uint32_t ticket)
{
    Tile t;
    t.order = ticket / g.cols;
    t.col = ticket - t.order * g.cols;
    const uint32_t b = t.col / g.cgs;
    t.b = b;
    t.d0 = (int64_t)(t.col - b * g.cgs) * kCh;
    t.t0 = (REVERSE ? g.K - 1 - (int64_t)t.order : (int64_t)t.order) * kTok;
    t.last = t.order + 1 == (uint32_t)g.K;
    return t;
}
__device__ __forceinline__ uint64_t* tile_words(const Args& g, const Tile& t, uint32_t order)
{
    return g.a0 + ((uint64_t)t.col * (uint64_t)g.K + order) * kCh;
}
__device__ __forceinline__ uint64_t* group_words(const Args& g, const Tile& t, uint32_t group)
{
    return g.a1 + ((uint64_t)t.col * g.groups + group) * kCh;
}
__device__ __forceinline__ uint64_t* block_words(const Args& g, const Tile& t, uint32_t block)
{
    return g.c2 + ((uint64_t)t.col * g.blocks + block) * kCh;
}

// Fetches what a tile's carry is made of into ent: [0] the block's carry in,
// [1 .. 7] groups, [8 .. 14] tiles; warp w fetches w and 8 + w.  `start` is the
// state before the first tile (h0, or the last state's gradient).
__device__ __forceinline__ void fetch_carry(const Args& g, const Tile& t, int w, int lane, const float* start,
                                            float4 (*ent)[32])
{
    const uint32_t block = t.order / (kFan * kFan), group = t.order / kFan % kFan, j = t.order % kFan;
    if (w == 0) {
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (block) {
            v = await(g, block_words(g, t, block), lane);
        } else if (start) {
            const int64_t d = t.d0 + 2 * lane;
            if (d < g.D) v.y = start[t.b * g.D + d];
            if (d + 1 < g.D) v.w = start[t.b * g.D + d + 1];
        }
        ent[0][lane] = v;
    } else if ((uint32_t)w <= group) {
        ent[w][lane] = await(g, group_words(g, t, block * kFan + w - 1), lane);
    }
    if ((uint32_t)w < j) ent[kFan + w][lane] = await(g, tile_words(g, t, t.order - j + w), lane);
}

__device__ __forceinline__ float2 carry_of(const Tile& t, int lane, const float4 (*ent)[32])
{
    const uint32_t group = t.order / kFan % kFan, j = t.order % kFan;
    float2 h = make_float2(ent[0][lane].y, ent[0][lane].w);
    for (uint32_t k = 1; k <= group; ++k) h = apply(ent[k][lane], h);
    for (uint32_t k = 0; k < j; ++k) h = apply(ent[kFan + k][lane], h);
    return h;
}

// After the carry is known: the group's map (last tile of a group) and the
// next block's carry (last tile of a block), by one warp.
__device__ __forceinline__ void publish_up(const Args& g, const Tile& t, int lane, float4 own, float2 carry,
                                           const float4 (*ent)[32])
{
    if (t.last || t.order % kFan != kFan - 1) return;
    const uint32_t group = t.order / kFan;
    if (group % kFan != kFan - 1) {
        float4 m = ent[kFan][lane];
        for (int k = 1; k < kFan - 1; ++k) m = after(ent[kFan + k][lane], m);
        publish(group_words(g, t, group), lane, after(own, m));
    } else {
        const float2 h = apply(own, carry);
        publish(block_words(g, t, group / kFan + 1), lane, make_float4(0.0f, h.x, 0.0f, h.y));
    }
}

// ------------------------------------------------------------------ loads ---

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

// A tile of one input into shared memory [64][64], zeros past the last token
// or channel.  VEC: rows start on 16 bytes; else element by element.
template <typename T, bool VEC>
__device__ __forceinline__ void load_tile(const Args& g, const Tile& t, const void* from, int64_t ld, T* to)
{
    const T* src = (const T*)from + t.b * g.L * ld;
    if constexpr (VEC) {
        constexpr int per = 16 / sizeof(T), chunks = kCh / per;
#pragma unroll
        for (int k = threadIdx.x; k < kTok * chunks; k += kThreads) {
            const int row = k / chunks, c = k % chunks * per;
            const int64_t tok = t.t0 + row, left = g.D - t.d0 - c;
            const bool in = tok < g.L && left > 0;
            const int bytes = !in ? 0 : left >= per ? 16 : (int)left * (int)sizeof(T);
            cp_async(to + row * kCh + c, in ? src + tok * ld + t.d0 + c : src, bytes);
        }
    } else {
        for (int k = threadIdx.x; k < kTok * kCh; k += kThreads) {
            const int row = k / kCh, c = k % kCh;
            const int64_t tok = t.t0 + row;
            const bool in = tok < g.L && t.d0 + c < g.D;
            const T* at = in ? src + tok * ld + t.d0 + c : src;
            if constexpr (sizeof(T) == 4) cp_async4(to + k, at, in ? 4 : 0);
            else to[k] = in ? *at : from_f32<T>(0.0f);
        }
    }
}

__device__ __forceinline__ float2 pair_at(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 pair_at(const __nv_bfloat16* p)
{
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Two adjacent channels of a row (d the first; `wide`: the pair is aligned and
// both are there).
__device__ __forceinline__ void put_pair(float* p, float2 v, bool wide, bool one, bool two)
{
    if (wide) { *reinterpret_cast<float2*>(p) = v; return; }
    if (one) p[0] = v.x;
    if (two) p[1] = v.y;
}
__device__ __forceinline__ void put_pair(__nv_bfloat16* p, float2 v, bool wide, bool one, bool two)
{
    if (wide) { *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y); return; }
    if (one) p[0] = __float2bfloat16_rn(v.x);
    if (two) p[1] = __float2bfloat16_rn(v.y);
}

}  // namespace gated
}  // namespace mru
