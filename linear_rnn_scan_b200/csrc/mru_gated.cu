// mru_gated.cu -- gated linear recurrence: h_t = a_t h_{t-1} + b_t per channel,
// its backward, and their entry points.
#include <string.h>

#include <atomic>

#include "mru_gated_tile.cuh"

namespace mru {
namespace {

using namespace gated;

constexpr int kKeep = MRU_GATED_KEEP;

// Inputs of a gate.
constexpr int inputs_of(int gate) { return gate == MRU_GATE_LRU ? 3 : 2; }

// The testing hook's limit in ms for the next launch (0: none).
std::atomic<int> g_stall_ms{0};

// ------------------------------------------------------- short sequences ---

// One token's inputs of one channel.
template <typename T, int GATE, bool PACKED>
__device__ __forceinline__ void load_token(const Args& g, int64_t row, int64_t d, float& x, float& f, float& i)
{
    i = 0.0f;
    if constexpr (PACKED) {
        const int64_t e = row * g.D + d, r = row * ((g.D + 63) / 64) + d / 64;
        x = (float)g.x8.q[e] * g.x8.scale[r];
        f = (float)g.f8.q[e] * g.f8.scale[r];
        if (GATE == MRU_GATE_LRU) i = (float)g.i8.q[e] * g.i8.scale[r];
    } else {
        const int64_t e = row * g.ld + d;
        x = to_f32(((const T*)g.x)[e]);
        f = to_f32(((const T*)g.f)[e]);
        if (GATE == MRU_GATE_LRU) i = to_f32(((const T*)g.i)[e]);
    }
}

// What a token's gradient d is multiplied with: dx = cx d, df = cf d, di = ci d
// and, for lam, q d.  a: the decay, p = h_{t-1}.
template <int GATE, bool NEAR = false>
__device__ __forceinline__ void gradient_factors(float x, float f, float i, float csp, float p, float& a, float& b,
                                                 float& cx, float& cf, float& ci, float& q)
{
    ci = q = 0.0f;
    if constexpr (GATE == MRU_GATE_DECAY) {
        a = f;
        b = x;
        cx = 1.0f;
        cf = p;
    } else if constexpr (GATE == MRU_GATE_SIGMOID) {
        sigmoid2(f, a, cx);
        b = cx * x;
        cf = a * cx * (p - x);
    } else {
        float sf, nf, si, ni, m;
        sigmoid2(f, sf, nf);
        sigmoid2(i, si, ni);
        const float la = -csp * sf;
        exp_expm1_neg<NEAR>(la, a, m);
        const float v = -m * (1.0f + a);                   // 1 - a^2
        const float r = v > 0.0f ? inv_root(v) : 0.0f;     // la / u tends to 0 with u
        const float sx = si * x, u = v * r;
        cx = u * si;
        b = u * sx;
        ci = b * ni;
        q = la * a * (p - sx * a * r);
        cf = q * nf;
    }
}

constexpr int kShort = 8;                // tokens up to which a thread takes a channel alone

// A thread per channel, token after token.
template <typename T, int GATE>
__global__ void __launch_bounds__(128) k_gated_short(Args g)
{
    const int64_t ch = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (ch == 0 && g.status) *g.status = 0;
    if (ch >= g.B * g.D) return;
    const int64_t b = ch / g.D, d = ch - b * g.D, len = valid_tokens(g, b);
    const float csp = GATE == MRU_GATE_LRU ? g.c * softplus(g.lam[d]) : 0.0f;
    float h = g.h0 ? g.h0[ch] : 0.0f;
    if (g.states && g.L > 0) g.states[ch] = h;
    for (int64_t t = 0; t < g.L; ++t) {
        const int64_t row = b * g.L + t;
        float out = 0.0f;
        if (t < len) {
            float x, f, i, a, u;
            load_token<T, GATE, false>(g, row, d, x, f, i);
            gates<GATE>(x, f, i, csp, a, u);
            if (g.reset && g.reset[row]) h = 0.0f;
            h = out = carry_in(a, h) + u;
        }
        ((T*)g.y)[row * g.D + d] = from_f32<T>(out);
    }
    if (g.h_last) g.h_last[ch] = h;
}

template <typename T, int GATE, bool PACKED>
__global__ void __launch_bounds__(128) k_gated_short_bwd(Args g)
{
    const int64_t ch = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (ch == 0 && g.status) *g.status = 0;
    if (ch >= g.B * g.D) return;
    const int64_t b = ch / g.D, d = ch - b * g.D, len = valid_tokens(g, b);
    const float csp = GATE == MRU_GATE_LRU ? g.c * softplus(g.lam[d]) : 0.0f;
    float e = g.dh_last ? g.dh_last[ch] : 0.0f;            // gradient of the state after a token
    float h = g.L > 0 ? g.states[ch] : 0.0f, dlam = 0.0f;
    float a[kShort], cx[kShort], cf[kShort], ci[kShort], q[kShort];
#pragma unroll
    for (int t = 0; t < kShort; ++t) {
        a[t] = 1.0f;
        cx[t] = cf[t] = ci[t] = q[t] = 0.0f;
        if (t >= len) continue;
        const int64_t row = b * g.L + t;
        const bool reset = g.reset && g.reset[row];
        float x, f, i, u;
        load_token<T, GATE, PACKED>(g, row, d, x, f, i);
        if (reset) h = 0.0f;
        gradient_factors<GATE>(x, f, i, csp, h, a[t], u, cx[t], cf[t], ci[t], q[t]);
        h = carry_in(a[t], h) + u;
        if (reset) a[t] = 0.0f;
    }
#pragma unroll
    for (int t = kShort - 1; t >= 0; --t) {
        if (t >= g.L) continue;
        const int64_t row = b * g.L + t, at = row * g.ldg + d;
        const float dt = t < len ? e + to_f32(((const T*)g.dy)[row * g.D + d]) : 0.0f;
        ((T*)g.dx)[at] = from_f32<T>(cx[t] * dt);
        ((T*)g.df)[at] = from_f32<T>(cf[t] * dt);
        if (GATE == MRU_GATE_LRU) {
            ((T*)g.di)[at] = from_f32<T>(ci[t] * dt);
            dlam = fmaf(q[t], dt, dlam);
        }
        if (t < len) e = carry_in(a[t], dt);
    }
    if (g.dh0) g.dh0[ch] = e;
    if (GATE == MRU_GATE_LRU && g.dlam_part) g.dlam_part[ch] = dlam;
}

// ---------------------------------------------------------------- forward ---

// Channels of a lane: tiles of 128 channels in bf16's forward, of 64 elsewhere.
constexpr int fwd_channels(size_t elem) { return elem == 2 ? 4 : 2; }
constexpr int kBwdC = 2;

template <int C>
struct TileMem {
    MapRow<C> agg[kWarps];               // the warps' maps
    Entries<C> ent;
    float csp[32 * C];                   // c softplus(lam) of the tile's channels
    Tile tile[3];                        // this one, the next, the one after
};

template <int C>
__device__ __forceinline__ Vec<C> csp_of(const float* csp, int lane)
{
    return read_row<C>(csp + C * lane);
}

template <int C>
__device__ __forceinline__ bool all_near(const Vec<C>& csp)
{
    bool near = true;
#pragma unroll
    for (int c = 0; c < C; ++c) near = near && csp.v[c] <= 0.5f;
    return __all_sync(~0u, near);
}

// 8-bit copies of a warp's tokens.  A run of 64 channels is 64 / C lanes of a
// row; the largest magnitudes of all runs (input, token, half) are found first
// and a lane takes the factors of one or two of them for all.
template <typename T, int C, int NIN>
__device__ __forceinline__ void pack_rows(const Args& g, const Tile& t, int w, int lane, const T* stage, bool wide8)
{
    constexpr int kCh = 32 * C, HALVES = kCh / 64, RUNS = NIN * kStep * HALVES, SETS = (RUNS + 31) / 32;
    uint32_t mine[SETS];
#pragma unroll
    for (int k = 0; k < SETS; ++k) mine[k] = 0;
#pragma unroll
    for (int n = 0; n < NIN; ++n)
#pragma unroll
        for (int s = 0; s < kStep; ++s) {
            const Vec<C> v = read_row<C>(stage + (n * kTok + w * kStep + s) * kCh + C * lane);
            uint32_t m = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) m = max(m, mag_bits(v.v[c]));
#pragma unroll
            for (int h = 0; h < HALVES; ++h) {
                const int run = (n * kStep + s) * HALVES + h;
                const uint32_t r = __reduce_max_sync(~0u, lane * HALVES / 32 == h ? m : 0u);
                if (lane == run % 32) mine[run / 32] = r;
            }
        }
    float inv[SETS];
    const int64_t row0 = t.row + w * kStep, runs = (g.D + 63) / 64;
    const int left = t.tokens - w * kStep;
#pragma unroll
    for (int k = 0; k < SETS; ++k) {
        float scale;
        pack8_factors(__uint_as_float(mine[k]), inv[k], scale);
        const int run = 32 * k + lane, h = run % HALVES, s = run / HALVES % kStep, n = run / HALVES / kStep;
        if (n < NIN && s < left && h * 64 < t.channels) {
            float* to = n == 0 ? g.x8.scale : n == 1 ? g.f8.scale : g.i8.scale;
            to[(row0 + s) * runs + t.d0 / 64 + h] = scale;
        }
    }
    const int channels = t.channels - C * lane;
#pragma unroll
    for (int n = 0; n < NIN; ++n) {
        int8_t* at = (n == 0 ? g.x8.q : n == 1 ? g.f8.q : g.i8.q) + row0 * g.D + t.d0 + C * lane;
#pragma unroll
        for (int s = 0; s < kStep; ++s, at += g.D) {
            const int run = (n * kStep + s) * HALVES;
            float k = __shfl_sync(~0u, inv[run / 32], run % 32);
            if (HALVES == 2) {
                const float k1 = __shfl_sync(~0u, inv[run / 32], run % 32 + 1);
                if (lane >= 16) k = k1;
            }
            if (s >= left) continue;
            const Vec<C> v = read_row<C>(stage + (n * kTok + w * kStep + s) * kCh + C * lane);
            uint32_t q = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) q |= (uint32_t)pack8_q(v.v[c], k) << (8 * c);
            if (wide8) {
                if (channels > 0) {
                    if constexpr (C == 4) *reinterpret_cast<uint32_t*>(at) = q;
                    else *reinterpret_cast<uint16_t*>(at) = (uint16_t)q;
                }
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (c < channels) at[c] = (int8_t)(q >> (8 * c));
            }
        }
    }
}

// The decays and inputs of a warp's tokens and their map.  SPECIAL: padding
// (nothing happens) or resets (the state before counts as zero).
template <typename T, int C, int GATE, bool SPECIAL, bool NEAR>
__device__ __forceinline__ Map<C> local_map(const T* at, const Vec<C>& csp, int n, uint32_t resets,
                                            Vec<C> (&a)[kStep], Vec<C> (&b)[kStep])
{
    constexpr int kCh = 32 * C, kIn = kTok * kCh;
    Map<C> m = Map<C>::of(1.0f);
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
        if (SPECIAL && s >= n) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                a[s].v[c] = 1.0f;
                b[s].v[c] = 0.0f;
            }
            continue;
        }
        const Vec<C> x = read_row<C>(at + s * kCh), f = read_row<C>(at + kIn + s * kCh);
        Vec<C> i = x;
        if (GATE == MRU_GATE_LRU) i = read_row<C>(at + 2 * kIn + s * kCh);
        if (SPECIAL && (resets >> s & 1)) m = Map<C>::of(0.0f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            gates<GATE, NEAR>(x.v[c], f.v[c], i.v[c], csp.v[c], a[s].v[c], b[s].v[c]);
            m.P[c] *= a[s].v[c];
            m.H[c] = GATE == MRU_GATE_DECAY ? carry_in(a[s].v[c], m.H[c]) + b[s].v[c]
                                            : fmaf(a[s].v[c], m.H[c], b[s].v[c]);
        }
    }
    return m;
}

template <typename T, int C, int GATE, bool SPECIAL>
__device__ __forceinline__ void run_states(T* y, int64_t D, int left, Vec<C> h, int n, uint32_t resets,
                                           const Vec<C> (&a)[kStep], const Vec<C> (&b)[kStep], const Put& put)
{
#pragma unroll
    for (int s = 0; s < kStep; ++s, y += D) {
        if (SPECIAL && (resets >> s & 1)) h = Vec<C>{};
#pragma unroll
        for (int c = 0; c < C; ++c)
            h.v[c] = GATE == MRU_GATE_DECAY ? carry_in(a[s].v[c], h.v[c]) + b[s].v[c]
                                            : fmaf(a[s].v[c], h.v[c], b[s].v[c]);
        Vec<C> out = h;
        if (SPECIAL && s >= n) out = Vec<C>{};
        if (!SPECIAL || s < left) write_row<C>(y, out, put);
    }
}

template <typename T, int C, int GATE>
constexpr size_t forward_stage_bytes()
{
    return (size_t)inputs_of(GATE) * kTok * 32 * C * sizeof(T);
}

template <typename T, int C, int GATE, bool VEC>
__device__ __forceinline__ void load_inputs(const Args& g, const Tile& t, T* to)
{
    constexpr int kIn = kTok * 32 * C;
    load_tile<T, C, VEC>(t, g.x, g.ld, to);
    load_tile<T, C, VEC>(t, g.f, g.ld, to + kIn);
    if (GATE == MRU_GATE_LRU) load_tile<T, C, VEC>(t, g.i, g.ld, to + 2 * kIn);
}

// Forward: every input is read once and every output written once.  Blocks
// stay and draw tiles in the order of the scan; the next tile's inputs are on
// their way while one is worked on.  Per tile: each warp maps its 8 tokens,
// the maps meet in shared memory, the tile's map is published, the carry is
// fetched (by then the tiles before have published theirs), and the states
// are run again from it over decays and inputs that stayed in registers.
template <typename T, int C, int GATE, bool VEC, bool PACK>
__global__ void __launch_bounds__(kThreads, C == 4 ? 2 : 3) k_gated_tile(Args g)
{
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ TileMem<C> mem;
    constexpr int NIN = inputs_of(GATE), kCh = 32 * C, kElems = NIN * kTok * kCh;
    constexpr bool lru = GATE == MRU_GATE_LRU;
    T* stage = reinterpret_cast<T*>(stages);
    const int tid = threadIdx.x, lane = tid & 31, w = tid / 32;
    const bool whole = g.D % C == 0 && aligned(g.y, C * sizeof(T));
    const bool wide8 = PACK && g.D % C == 0 && aligned(g.x8.q, C) && aligned(g.f8.q, C) && (!lru || aligned(g.i8.q, C));
    if (tid == 0) {
        const uint32_t first = g.ticket ? atomicAdd(g.ticket, 1u) : blockIdx.x;
        find_tile<C, false>(g, first, mem.tile[0]);
        find_tile<C, false>(g, draw(g, first), mem.tile[1]);
        if (!g.ticket && blockIdx.x == 0 && g.status) *g.status = 0;
    }
    __syncthreads();
    if (mem.tile[0].ticket < g.tiles) {
        const Tile& t = mem.tile[0];
        load_inputs<T, C, GATE, VEC>(g, t, stage);
        if (lru && tid < kCh) mem.csp[tid] = tid < t.channels ? g.c * softplus(g.lam[t.d0 + tid]) : 0.0f;
    }
    cp_commit();
    for (int st = 0, now = 0; mem.tile[now].ticket < g.tiles; st ^= 1) {
        const int then = now == 2 ? 0 : now + 1, later = then == 2 ? 0 : then + 1;
        const Tile& t = mem.tile[now];
        uint32_t drawn = 0;
        float lam = 0.0f;
        if (tid == 0) drawn = draw(g, mem.tile[then].ticket);
        if (mem.tile[then].ticket < g.tiles) {
            const Tile& u = mem.tile[then];
            load_inputs<T, C, GATE, VEC>(g, u, stage + (st ^ 1) * kElems);
            if (lru && tid < u.channels) lam = g.lam[u.d0 + tid];
        }
        cp_commit();
        int n;
        uint32_t resets;
        warp_masks(g, t, w, lane, n, resets);
        cp_wait<1>();
        __syncthreads();
        const T* in = stage + st * kElems;
        if constexpr (PACK) pack_rows<T, C, NIN>(g, t, w, lane, in, wide8);
        Vec<C> csp = {};
        if (lru) csp = csp_of<C>(mem.csp, lane);
        const bool special = n < kStep || resets;
        Vec<C> a[kStep], b[kStep];
        const T* rows = in + w * kStep * kCh + C * lane;
        Map<C> own;
        if (special) own = local_map<T, C, GATE, true, false>(rows, csp, n, resets, a, b);
        else if (lru && all_near<C>(csp)) own = local_map<T, C, GATE, false, lru>(rows, csp, n, resets, a, b);
        else own = local_map<T, C, GATE, false, false>(rows, csp, n, resets, a, b);
        mem.agg[w].put(lane, own);
        __syncthreads();
        Map<C> pre = Map<C>::of(1.0f);
        for (int v = 0; v < w; ++v) pre = mem.agg[v].get(lane).after(pre);
        if (w == kWarps - 1) {
            own = own.after(pre);                          // the tile's map
            if (!t.last && !(g.withhold && t.ticket == 0)) publish<C>(tile_words<C>(g, t, t.order), lane, own);
        }
        mem.ent.fetch(g, t, w, lane, g.h0);
        if (tid == 0) find_tile<C, false>(g, drawn, mem.tile[later]);
        __syncthreads();
        const Vec<C> carry = mem.ent.carry(t, lane);
        const int channels = t.channels - C * lane;
        if (w == kWarps - 1) {
            mem.ent.publish_up(g, t, lane, own, carry);
            if (t.last && g.h_last) write_state<C>(g.h_last + t.b * g.D + t.d0 + C * lane, own(carry), channels);
        }
        if (w == 0 && g.states) write_state<C>(g.states + t.k * g.D + t.d0 + C * lane, carry, channels);
        T* y = (T*)g.y + (t.row + w * kStep) * g.D + t.d0 + C * lane;
        const Put put = {whole && channels > 0, channels};
        const int left = t.tokens - w * kStep;
        if (special) run_states<T, C, GATE, true>(y, g.D, left, pre(carry), n, resets, a, b, put);
        else run_states<T, C, GATE, false>(y, g.D, left, pre(carry), n, resets, a, b, put);
        if (lru && tid < kCh) mem.csp[tid] = g.c * softplus(lam);
        now = then;
    }
}

// --------------------------------------------------------------- backward ---

template <int C>
struct BackMem {
    MapRow<C> agg[kWarps];               // the warps' maps of states
    MapRow<C> back[kWarps];              // and of gradients
    Entries<C> ent;
    float dlam[kWarps][32 * C];
    float csp[32 * C];
    float state[2][32 * C];              // the kept state before the tile
    float scale[2][3][kTok];             // 8-bit copies: the scale of a token's run
    Tile tile[3];
};

template <typename T, int C, int GATE, bool PACKED>
constexpr size_t backward_stage_bytes()
{
    return (size_t)kTok * 32 * C * (inputs_of(GATE) * (PACKED ? 1 : sizeof(T)) + sizeof(T));
}
// Two stages where two blocks of them fit an SM's 227 KB, else one.
template <typename T, int C, int GATE, bool PACKED>
constexpr int backward_stages()
{
    return backward_stage_bytes<T, C, GATE, PACKED>() <= 48 * 1024 ? 2 : 1;
}

template <typename T, int C, int GATE, bool VEC, bool PACKED>
__device__ __forceinline__ void load_back(const Args& g, const Tile& t, unsigned char* stage, BackMem<C>& mem, int st)
{
    static_assert(!PACKED || C == 2, "a tile's row is one run of 64 channels");
    constexpr int NIN = inputs_of(GATE), kCh = 32 * C;
    T* dy = reinterpret_cast<T*>(stage);
    load_tile<T, C, VEC>(t, g.dy, g.D, dy);
    const int tid = threadIdx.x;
    if constexpr (PACKED) {
        int8_t* q = reinterpret_cast<int8_t*>(dy + kTok * kCh);
        const int64_t runs = g.cgs;
#pragma unroll
        for (int n = 0; n < NIN; ++n) {
            const mru_packed8& h = n == 0 ? g.x8 : n == 1 ? g.f8 : g.i8;
            const int8_t* src = h.q + t.row * g.D + t.d0;
            if constexpr (VEC) {
                constexpr int chunks = kCh / 16;
                for (int k = tid; k < kTok * chunks; k += kThreads) {
                    const int row = k / chunks, c = k % chunks * 16;
                    const bool in = row < t.tokens && c < t.channels;
                    cp_async(q + (n * kTok + row) * kCh + c, in ? src + row * g.D + c : h.q, in ? 16 : 0);
                }
            } else {
                for (int k = tid; k < kTok * kCh; k += kThreads) {
                    const int row = k / kCh, c = k % kCh;
                    q[n * kTok * kCh + k] = row < t.tokens && c < t.channels ? src[row * g.D + c] : (int8_t)0;
                }
            }
            if (tid < kTok) {
                const bool in = tid < t.tokens;
                cp_async4(&mem.scale[st][n][tid], in ? h.scale + (t.row + tid) * runs + t.d0 / 64 : h.scale, in ? 4 : 0);
            }
        }
    } else {
        load_inputs<T, C, GATE, VEC>(g, t, dy + kTok * kCh);
    }
    if (tid < kCh) {
        const bool in = tid < t.channels;
        cp_async4(&mem.state[st][tid], in ? g.states + t.k * g.D + t.d0 + tid : g.states, in ? 4 : 0);
    }
}

// A lane's channels of a token's input n, from the stage.
template <typename T, int C, bool PACKED>
__device__ __forceinline__ Vec<C> input_row(const unsigned char* stage, const float (&scale)[3][kTok], int n, int row,
                                            int lane)
{
    constexpr int kCh = 32 * C;
    const unsigned char* in = stage + kTok * kCh * sizeof(T);
    if constexpr (PACKED) {
        const char2 q = *reinterpret_cast<const char2*>(in + (n * kTok + row) * kCh + C * lane);
        const float k = scale[n][row];
        return Vec<C>{(float)(signed char)q.x * k, (float)(signed char)q.y * k};
    } else {
        return read_row<C>(reinterpret_cast<const T*>(in) + (n * kTok + row) * kCh + C * lane);
    }
}

// The map of a warp's tokens; a and, for the sigmoid gate, cx = 1 - a stay.
template <typename T, int C, int GATE, bool PACKED, bool NEAR>
__device__ __forceinline__ Map<C> back_map(const unsigned char* stage, const float (&scale)[3][kTok], int w, int lane,
                                           const Vec<C>& csp, int n, uint32_t resets, Vec<C> (&a)[kStep],
                                           Vec<C> (&cx)[kStep])
{
    Map<C> m = Map<C>::of(1.0f);
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            a[s].v[c] = 1.0f;
            cx[s].v[c] = 0.0f;
        }
        if (s >= n) continue;
        const int row = w * kStep + s;
        const Vec<C> x = input_row<T, C, PACKED>(stage, scale, 0, row, lane);
        const Vec<C> f = input_row<T, C, PACKED>(stage, scale, 1, row, lane);
        Vec<C> i = x;
        if (GATE == MRU_GATE_LRU) i = input_row<T, C, PACKED>(stage, scale, 2, row, lane);
        if (resets >> s & 1) m = Map<C>::of(0.0f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float b;
            if (GATE == MRU_GATE_SIGMOID) {
                sigmoid2(f.v[c], a[s].v[c], cx[s].v[c]);
                b = cx[s].v[c] * x.v[c];
            } else {
                gates<GATE, NEAR>(x.v[c], f.v[c], i.v[c], csp.v[c], a[s].v[c], b);
            }
            m.P[c] *= a[s].v[c];
            m.H[c] = carry_in(a[s].v[c], m.H[c]) + b;
        }
    }
    return m;
}

// A warp's tokens: states from h, the factors of the gradients, and the map of
// gradients e -> P e + E from the token after the last to before the first.
// dl: sum q d and sum q dd/de (for lam) at e = 0, without the first token where
// it is a piece's edge (k_gated_edge counts it).  h: the state after the last.
template <typename T, int C, int GATE, bool PACKED, bool NEAR>
__device__ __forceinline__ Map<C> back_factors(const unsigned char* stage, const float (&scale)[3][kTok], int w,
                                               int lane, const Vec<C>& csp, Vec<C>& h, int n, uint32_t resets,
                                               bool edge, Vec<C> (&a)[kStep], Vec<C> (&cx)[kStep],
                                               Vec<C> (&cf)[kStep], Vec<C> (&ci)[kStep], Vec<C>& dl0, Vec<C>& dl1)
{
    constexpr int kCh = 32 * C;
    Vec<C> q[kStep];
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
        cf[s] = ci[s] = q[s] = Vec<C>{};
        if (s >= n) continue;
        const int row = w * kStep + s;
        const Vec<C> x = input_row<T, C, PACKED>(stage, scale, 0, row, lane);
        Vec<C> f = x, i = x;
        if (GATE == MRU_GATE_LRU) {
            f = input_row<T, C, PACKED>(stage, scale, 1, row, lane);
            i = input_row<T, C, PACKED>(stage, scale, 2, row, lane);
        }
        const bool reset = resets >> s & 1;
        if (reset) h = Vec<C>{};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float b;
            if (GATE == MRU_GATE_DECAY) {
                b = x.v[c];
                cf[s].v[c] = h.v[c];
            } else if (GATE == MRU_GATE_SIGMOID) {
                b = cx[s].v[c] * x.v[c];
                cf[s].v[c] = a[s].v[c] * cx[s].v[c] * (h.v[c] - x.v[c]);
            } else {
                gradient_factors<GATE, NEAR>(x.v[c], f.v[c], i.v[c], csp.v[c], h.v[c], a[s].v[c], b, cx[s].v[c],
                                             cf[s].v[c], ci[s].v[c], q[s].v[c]);
            }
            h.v[c] = carry_in(a[s].v[c], h.v[c]) + b;
            if (reset) a[s].v[c] = 0.0f;
        }
    }
    if (PACKED && edge) q[0] = Vec<C>{};
    Map<C> m = Map<C>::of(1.0f);
    dl0 = dl1 = Vec<C>{};
#pragma unroll
    for (int s = kStep - 1; s >= 0; --s) {
        if (s >= n) continue;
        const Vec<C> dy = read_row<C>(reinterpret_cast<const T*>(stage) + (w * kStep + s) * kCh + C * lane);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float d = m.H[c] + dy.v[c];
            if (GATE == MRU_GATE_LRU) {
                dl0.v[c] = fmaf(q[s].v[c], d, dl0.v[c]);
                dl1.v[c] = fmaf(q[s].v[c], m.P[c], dl1.v[c]);
            }
            m.P[c] *= a[s].v[c];
            m.H[c] = carry_in(a[s].v[c], d);
        }
    }
    return m;
}

// Backward, tiles from the last to the first: the states of the tile again
// from its kept state, the factors of the gradients, then the gradient's own
// recurrence with its carry from the later tiles, as the forward's.
template <typename T, int C, int GATE, bool VEC, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2) k_gated_tile_bwd(Args g)
{
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ BackMem<C> mem;
    constexpr int kCh = 32 * C;
    constexpr size_t kBytes = backward_stage_bytes<T, C, GATE, PACKED>();
    constexpr int STAGES = backward_stages<T, C, GATE, PACKED>();
    constexpr bool lru = GATE == MRU_GATE_LRU;
    const int tid = threadIdx.x, lane = tid & 31, w = tid / 32;
    const bool whole = g.D % C == 0 && g.ldg % C == 0 && aligned(g.dx, C * sizeof(T)) && aligned(g.df, C * sizeof(T)) &&
                       (!lru || aligned(g.di, C * sizeof(T)));
    if (tid == 0) {
        const uint32_t first = g.ticket ? atomicAdd(g.ticket, 1u) : blockIdx.x;
        find_tile<C, true>(g, first, mem.tile[0]);
        find_tile<C, true>(g, draw(g, first), mem.tile[1]);
        if (!g.ticket && blockIdx.x == 0 && g.status) *g.status = 0;
    }
    __syncthreads();
    if (mem.tile[0].ticket < g.tiles) {
        const Tile& t = mem.tile[0];
        if (STAGES == 2) load_back<T, C, GATE, VEC, PACKED>(g, t, stages, mem, 0);
        if (lru && tid < kCh) mem.csp[tid] = tid < t.channels ? g.c * softplus(g.lam[t.d0 + tid]) : 0.0f;
    }
    cp_commit();
    for (int st = 0, now = 0; mem.tile[now].ticket < g.tiles; st ^= 1) {
        const int then = now == 2 ? 0 : now + 1, later = then == 2 ? 0 : then + 1;
        const Tile& t = mem.tile[now];
        unsigned char* stage = stages + (STAGES == 2 ? st * kBytes : 0);
        uint32_t drawn = 0;
        float lam = 0.0f;
        if (tid == 0) drawn = draw(g, mem.tile[then].ticket);
        if (STAGES == 1) load_back<T, C, GATE, VEC, PACKED>(g, t, stage, mem, st);
        if (mem.tile[then].ticket < g.tiles) {
            const Tile& u = mem.tile[then];
            if (STAGES == 2) load_back<T, C, GATE, VEC, PACKED>(g, u, stages + (st ^ 1) * kBytes, mem, st ^ 1);
            if (lru && tid < u.channels) lam = g.lam[u.d0 + tid];
        }
        cp_commit();
        int n;
        uint32_t resets;
        warp_masks(g, t, w, lane, n, resets);
        cp_wait<STAGES - 1>();
        __syncthreads();
        Vec<C> csp = {};
        if (lru) csp = csp_of<C>(mem.csp, lane);
        const bool near = lru && all_near<C>(csp);
        Vec<C> a[kStep], cx[kStep], cf[kStep], ci[kStep];
        mem.agg[w].put(lane, near ? back_map<T, C, GATE, PACKED, lru>(stage, mem.scale[st], w, lane, csp, n, resets, a, cx)
                                  : back_map<T, C, GATE, PACKED, false>(stage, mem.scale[st], w, lane, csp, n, resets, a,
                                                                        cx));
        __syncthreads();
        Vec<C> h = read_row<C>(&mem.state[st][C * lane]), dl0, dl1;
        for (int v = 0; v < w; ++v) h = mem.agg[v].get(lane)(h);
        const bool edge = PACKED && w == 0 && t.k % g.K > 0;
        Map<C> own = near ? back_factors<T, C, GATE, PACKED, lru>(stage, mem.scale[st], w, lane, csp, h, n, resets, edge,
                                                                  a, cx, cf, ci, dl0, dl1)
                          : back_factors<T, C, GATE, PACKED, false>(stage, mem.scale[st], w, lane, csp, h, n, resets,
                                                                    edge, a, cx, cf, ci, dl0, dl1);
        mem.back[w].put(lane, own);
        __syncthreads();
        Map<C> post = Map<C>::of(1.0f);
        for (int v = kWarps - 1; v > w; --v) post = mem.back[v].get(lane).after(post);
        if (w == 0) {
            own = own.after(post);                         // the tile's map
            if (!t.last && !(g.withhold && t.ticket == 0)) publish<C>(tile_words<C>(g, t, t.order), lane, own);
        }
        mem.ent.fetch(g, t, w, lane, g.dh_last);
        if (tid == 0) find_tile<C, true>(g, drawn, mem.tile[later]);
        __syncthreads();
        const Vec<C> carry = mem.ent.carry(t, lane);
        const int channels = t.channels - C * lane;
        if (w == 0) {
            mem.ent.publish_up(g, t, lane, own, carry);
            if (t.last && g.dh0) write_state<C>(g.dh0 + t.b * g.D + t.d0 + C * lane, own(carry), channels);
        }
        if (PACKED && g.edge_h && w == kWarps - 1 && t.order > 0)
            write_state<C>(g.edge_h + (t.k + 1) * g.D + t.d0 + C * lane, h, channels);
        Vec<C> e = post(carry);
        if (lru) {
#pragma unroll
            for (int c = 0; c < C; ++c) mem.dlam[w][C * lane + c] = fmaf(dl1.v[c], e.v[c], dl0.v[c]);
        }
        const int left = t.tokens - w * kStep;
        const Put put = {whole && channels > 0, channels};
        int64_t at = (t.row + w * kStep + kStep - 1) * g.ldg + t.d0 + C * lane;
#pragma unroll
        for (int s = kStep - 1; s >= 0; --s, at -= g.ldg) {
            if (s >= left) continue;
            Vec<C> d = {};
            if (s < n) {
                d = read_row<C>(reinterpret_cast<const T*>(stage) + (w * kStep + s) * kCh + C * lane);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    d.v[c] += e.v[c];
                    e.v[c] = carry_in(a[s].v[c], d.v[c]);
                }
            }
            if (PACKED && s == 0 && edge) write_state<C>(g.edge_d + t.k * g.D + t.d0 + C * lane, d, channels);
            Vec<C> o;
            if (GATE == MRU_GATE_DECAY) {
                write_row<C>((T*)g.dx + at, d, put);
            } else {
#pragma unroll
                for (int c = 0; c < C; ++c) o.v[c] = cx[s].v[c] * d.v[c];
                write_row<C>((T*)g.dx + at, o, put);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) o.v[c] = cf[s].v[c] * d.v[c];
            write_row<C>((T*)g.df + at, o, put);
            if (lru) {
#pragma unroll
                for (int c = 0; c < C; ++c) o.v[c] = ci[s].v[c] * d.v[c];
                write_row<C>((T*)g.di + at, o, put);
            }
        }
        if (lru && tid < kCh) mem.csp[tid] = g.c * softplus(lam);
        __syncthreads();                                   // the stage may be filled again
        if (lru && g.dlam_part && tid < t.channels) {
            float s = 0.0f;
            for (int v = 0; v < kWarps; ++v) s += mem.dlam[v][tid];
            g.dlam_part[t.k * g.D + t.d0 + tid] = s;
        }
        now = then;
    }
}

// With 8-bit copies the states run in pieces of 64 tokens from the kept states,
// and the state before a piece's first token is the last of the piece before,
// whose tile comes later in the backward: the first tokens' df (and q d for
// lam) are written here, from d and that state.
template <typename T, int GATE>
__global__ void __launch_bounds__(128) k_gated_edge(Args g)
{
    const int64_t n = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (n >= g.B * (g.K - 1) * g.D) return;
    const int64_t bk = n / g.D, d = n - bk * g.D, b = bk / (g.K - 1), k = bk - b * (g.K - 1) + 1;
    const int64_t at = (b * g.K + k) * g.D + d, t = k * kTok, row = b * g.L + t;
    float q = 0.0f;
    if (t < valid_tokens(g, b)) {
        const float csp = GATE == MRU_GATE_LRU ? g.c * softplus(g.lam[d]) : 0.0f;
        const float p = g.reset && g.reset[row] ? 0.0f : g.edge_h[at], dt = g.edge_d[at];
        float x, f, i, a, u, cx, cf, ci;
        load_token<T, GATE, true>(g, row, d, x, f, i);
        gradient_factors<GATE>(x, f, i, csp, p, a, u, cx, cf, ci, q);
        ((T*)g.df)[row * g.ldg + d] = from_f32<T>(cf * dt);
        q *= dt;
    }
    if (GATE == MRU_GATE_LRU && g.dlam_part) g.edge_q[at] = q;
}

// dlam = s(lam) / softplus(lam) times the sum of the tiles' sums (in fp64, in
// a fixed order: 8 threads to a channel, then one).
__global__ void __launch_bounds__(256) k_gated_dlam(int64_t parts, int64_t K, int64_t D, const float* __restrict__ part,
                                                    const float* __restrict__ edge, const float* __restrict__ lam,
                                                    float* __restrict__ dlam)
{
    __shared__ double sums[8][33];
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t d = (int64_t)blockIdx.x * 32 + x;
    double s = 0.0;
    if (d < D)
        for (int64_t p = y; p < parts; p += 8) {
            s += (double)part[p * D + d];
            if (edge && p % K) s += (double)edge[p * D + d];
        }
    sums[y][x] = s;
    __syncthreads();
    if (y || d >= D) return;
    for (int k = 1; k < 8; ++k) s += sums[k][x];
    dlam[d] = (float)(s * (double)softplus_slope_ratio(lam[d]));
}

mru_status check_problem(const mru_gated_problem* p)
{
    if (!p || p->B < 0 || p->L < 0 || p->D < 0 || p->ld < 0 || p->ld_grad < 0) return MRU_ERR_INVALID_ARG;
    if ((p->ld != 0 && p->ld < p->D) || (p->ld_grad != 0 && p->ld_grad < p->D)) return MRU_ERR_INVALID_ARG;
    if (p->dtype != MRU_F32 && p->dtype != MRU_BF16) return MRU_ERR_INVALID_ARG;
    if (p->gate < MRU_GATE_DECAY || p->gate > MRU_GATE_LRU) return MRU_ERR_INVALID_ARG;
    if (p->gate == MRU_GATE_LRU && !(p->c > 0.0f && p->c <= 3.402823466e+38f)) return MRU_ERR_INVALID_ARG;
    int64_t ld = p->ld > p->ld_grad ? p->ld : p->ld_grad;
    if (ld < p->D) ld = p->D;
    if (p->B > (int64_t)1 << 31 || p->L > (int64_t)1 << 31 || ld > (int64_t)1 << 31 ||
        !product_within(p->B * (p->L > 0 ? p->L : 1), ld, (int64_t)1 << 50))
        return MRU_ERR_UNSUPPORTED;
    // one index per 64 channels and 64 tokens
    if (!product_within(p->B * (p->D / 64 + 1), p->L / 64 + 1, (int64_t)1 << 30)) return MRU_ERR_UNSUPPORTED;
    return MRU_OK;
}

Args make_args(const mru_gated_problem& p, const mru_gated_inputs& in)
{
    Args g;
    memset(&g, 0, sizeof g);
    g.B = p.B; g.L = p.L; g.D = p.D; g.ld = p.ld ? p.ld : p.D; g.ldg = p.ld_grad ? p.ld_grad : p.D; g.K = div_up(p.L, kKeep);
    g.c = p.c;
    g.x = in.x; g.f = in.f; g.i = in.i;
    g.lam = in.lam; g.h0 = in.h0; g.reset = in.reset; g.lens = in.lens;
    return g;
}

// Checks of the parameters that both directions share.
bool common_inputs_ok(const mru_gated_problem& p, const mru_gated_inputs& in)
{
    const bool lru = p.gate == MRU_GATE_LRU;
    if (lru ? (p.D > 0 && !in.lam) : (in.lam != nullptr)) return false;
    return aligned(in.lam, 4) && aligned(in.h0, 4) && aligned(in.lens, 4);
}

bool packed_ok(const mru_packed8& v) { return !v.q || (v.scale && aligned(v.scale, 4)); }

template <typename F>
cudaError_t by_type(int32_t dtype, int32_t gate, F&& f)
{
    if (dtype == MRU_BF16) {
        if (gate == MRU_GATE_DECAY) return f.template operator()<__nv_bfloat16, MRU_GATE_DECAY>();
        if (gate == MRU_GATE_SIGMOID) return f.template operator()<__nv_bfloat16, MRU_GATE_SIGMOID>();
        return f.template operator()<__nv_bfloat16, MRU_GATE_LRU>();
    }
    if (gate == MRU_GATE_DECAY) return f.template operator()<float, MRU_GATE_DECAY>();
    if (gate == MRU_GATE_SIGMOID) return f.template operator()<float, MRU_GATE_SIGMOID>();
    return f.template operator()<float, MRU_GATE_LRU>();
}

// Workspace: the status word, a control block (ticket, abort flag), the words
// of the tiles' carries, then the tiles' sums for dlam.  Everything up to
// `zeroed` starts at zero.
struct Layout {
    size_t a0, a1, c2, zeroed, part, edge, bytes;
    uint32_t tiles, cols, cgs, groups, blocks;
};
constexpr size_t kControl = 256;
Layout layout(const mru_gated_problem& p, bool backward)
{
    const int64_t kCh = 32 * (backward ? kBwdC : fwd_channels(elem_size(p.dtype)));
    Layout W;
    memset(&W, 0, sizeof W);
    const int64_t K = div_up(p.L, kKeep);
    W.cgs = (uint32_t)div_up(p.D, kCh);
    W.cols = (uint32_t)(p.B * W.cgs);
    W.tiles = (uint32_t)(W.cols * K);
    W.groups = (uint32_t)div_up(K, kFan);
    W.blocks = (uint32_t)div_up(K, kFan * kFan);
    size_t off = 2 * kControl;
    const size_t words = (size_t)W.cols * kCh * sizeof(uint64_t);
    if (K > 1) {
        W.a0 = off; off += words * (size_t)K;
        W.a1 = off; off += words * W.groups;
        W.c2 = off; off += words * W.blocks;
    }
    W.zeroed = K > 1 ? off : sizeof(uint32_t);
    if (backward && p.gate == MRU_GATE_LRU) {
        W.part = off;
        off += align256((size_t)p.B * (size_t)(K > 0 ? K : 1) * (size_t)p.D * sizeof(float));
    }
    if (backward && K > 1) {
        W.edge = off;
        off += 3 * align256((size_t)p.B * (size_t)K * (size_t)p.D * sizeof(float));
    }
    W.bytes = off;
    return W;
}

void place(Args& g, const Layout& W, void* ws)
{
    char* base = reinterpret_cast<char*>(ws);
    g.status = reinterpret_cast<uint32_t*>(base);
    if (g.K > 1) {
        g.ticket = reinterpret_cast<uint32_t*>(base + kControl);
        g.abort = g.ticket + 1;
        g.a0 = reinterpret_cast<uint64_t*>(base + W.a0);
        g.a1 = reinterpret_cast<uint64_t*>(base + W.a1);
        g.c2 = reinterpret_cast<uint64_t*>(base + W.c2);
    }
    g.tiles = W.tiles;
    g.cols = W.cols;
    g.cgs = W.cgs;
    g.groups = W.groups;
    g.blocks = W.blocks;
    g.wait_ns = 2000000000ull;
}

// The testing hook: this launch's first tile publishes nothing.
void take_stall(Args& g)
{
    if (g.K < 2) return;
    const int ms = g_stall_ms.exchange(0);
    if (ms > 0) {
        g.withhold = 1;
        g.wait_ns = (uint64_t)ms * 1000000ull;
    }
}

// Blocks of a kernel that fit an SM, found once per device.
struct Fits {
    std::atomic<int> on[32];
};

// Blocks that stay: as many as fit the card.
template <typename K>
cudaError_t launch_tiles(K kernel, Fits& fits, const Args& g, size_t smem, cudaStream_t s)
{
    int device = 0;
    const cudaError_t got = cudaGetDevice(&device);
    if (got != cudaSuccess) return got;
    const bool kept = device < 32;
    int per = kept ? fits.on[device].load(std::memory_order_relaxed) : 0;
    if (per == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, smem);
        if (e != cudaSuccess) return e;
        if (per < 1) return cudaErrorInvalidConfiguration;
        if (kept) fits.on[device].store(per, std::memory_order_relaxed);
    }
    const uint32_t most = 148u * (uint32_t)per;
    kernel<<<g.tiles < most ? g.tiles : most, kThreads, smem, s>>>(g);
    return cudaGetLastError();
}

struct Forward {
    const Args& g;
    bool vec, pack;
    cudaStream_t s;
    template <typename T, int GATE>
    cudaError_t operator()() const
    {
        if (g.L <= kShort) {
            k_gated_short<T, GATE><<<(unsigned)div_up(g.B * g.D, 128), 128, 0, s>>>(g);
            return cudaGetLastError();
        }
        constexpr int C = fwd_channels(sizeof(T));
        constexpr size_t smem = 2 * forward_stage_bytes<T, C, GATE>();
        static Fits fits[4];
        if (vec)
            return pack ? launch_tiles(k_gated_tile<T, C, GATE, true, true>, fits[0], g, smem, s)
                        : launch_tiles(k_gated_tile<T, C, GATE, true, false>, fits[1], g, smem, s);
        return pack ? launch_tiles(k_gated_tile<T, C, GATE, false, true>, fits[2], g, smem, s)
                    : launch_tiles(k_gated_tile<T, C, GATE, false, false>, fits[3], g, smem, s);
    }
};

struct Backward {
    const Args& g;
    bool vec, packed;
    cudaStream_t s;
    template <typename T, int GATE, bool PACKED>
    cudaError_t go() const
    {
        if (g.L <= kShort) {
            k_gated_short_bwd<T, GATE, PACKED><<<(unsigned)div_up(g.B * g.D, 128), 128, 0, s>>>(g);
            return cudaGetLastError();
        }
        constexpr int C = kBwdC;
        constexpr size_t smem = backward_stages<T, C, GATE, PACKED>() * backward_stage_bytes<T, C, GATE, PACKED>();
        static Fits fits[2];
        const cudaError_t e = vec ? launch_tiles(k_gated_tile_bwd<T, C, GATE, true, PACKED>, fits[0], g, smem, s)
                                  : launch_tiles(k_gated_tile_bwd<T, C, GATE, false, PACKED>, fits[1], g, smem, s);
        if (e != cudaSuccess || !g.edge_h) return e;
        k_gated_edge<T, GATE><<<(unsigned)div_up(g.B * (g.K - 1) * g.D, 128), 128, 0, s>>>(g);
        return cudaGetLastError();
    }
    template <typename T, int GATE>
    cudaError_t operator()() const
    {
        return packed ? go<T, GATE, true>() : go<T, GATE, false>();
    }
};

}  // namespace
}  // namespace mru

using namespace mru;

extern "C" {

size_t mru_gated_workspace_size(const mru_gated_problem* p)
{
    return check_problem(p) == MRU_OK ? layout(*p, false).bytes : 0;
}

size_t mru_gated_backward_workspace_size(const mru_gated_problem* p)
{
    return check_problem(p) == MRU_OK ? layout(*p, true).bytes : 0;
}

mru_status mru_gated_scan(const mru_gated_problem* p, const mru_gated_inputs* in, void* y, float* h_last,
                          const mru_gated_saved* saved, void* ws, size_t ws_bytes, void* stream)
{
    mru_status st = check_problem(p);
    if (st != MRU_OK) return st;
    const bool waits = p->L > kKeep;                                 // else the workspace may be left out
    if (!in || (waits && !ws) || !aligned(ws, 16) || !common_inputs_ok(*p, *in)) return MRU_ERR_INVALID_ARG;
    const size_t es = elem_size(p->dtype);
    const bool lru = p->gate == MRU_GATE_LRU, any = p->B * p->D > 0, tokens = any && p->L > 0;
    if (lru ? (tokens && !in->i) : (in->i != nullptr)) return MRU_ERR_INVALID_ARG;
    if (tokens && (!in->x || !in->f || !y)) return MRU_ERR_INVALID_ARG;
    if (!aligned(in->x, es) || !aligned(in->f, es) || !aligned(in->i, es) || !aligned(y, es) || !aligned(h_last, 4))
        return MRU_ERR_INVALID_ARG;
    bool pack = false;
    if (saved) {
        pack = saved->x.q != nullptr;
        if (tokens && !saved->states) return MRU_ERR_INVALID_ARG;
        if (pack != (saved->f.q != nullptr) || (pack && lru) != (saved->i.q != nullptr)) return MRU_ERR_INVALID_ARG;
        if (!packed_ok(saved->x) || !packed_ok(saved->f) || !packed_ok(saved->i) || !aligned(saved->states, 4))
            return MRU_ERR_INVALID_ARG;
    }
    Args g = make_args(*p, *in);
    const int64_t rows = g.B * g.L;
    const size_t state = (size_t)(g.B * g.D) * 4, width = (size_t)g.D * es, pitch = (size_t)g.ld * es;
    Buffers b;
    for (const void* v : {g.x, g.f, g.i}) b.in_rows(v, rows, width, pitch);
    b.in(g.lam, (size_t)g.D * 4);
    b.in(g.h0, state);
    b.in(g.reset, (size_t)rows);
    b.in(g.lens, (size_t)g.B * 4);
    b.out(y, (size_t)rows * width);
    b.out(h_last, state);
    b.out(ws, ws ? ws_bytes : 0);
    if (saved) {
        b.out(saved->states, (size_t)(g.B * g.K * g.D) * 4);
        for (const mru_packed8* v : {&saved->x, &saved->f, &saved->i}) {
            if (!v->q) continue;
            b.out(v->q, (size_t)(rows * g.D));
            b.out(v->scale, (size_t)(rows * div_up(g.D, 64)) * 4);
        }
    }
    if (b.clash()) return MRU_ERR_INVALID_ARG;
    const Layout W = layout(*p, false);
    if (ws && ws_bytes < W.bytes) return MRU_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (ws && (!any || g.K > 1)) e = cudaMemsetAsync(ws, 0, W.zeroed, s);   // else the kernel clears the status word
    if (e != cudaSuccess || !any) return cuda_status(e);
    place(g, W, ws);
    take_stall(g);
    g.y = y;
    g.h_last = h_last;
    g.states = saved ? saved->states : nullptr;
    const bool here = pack && p->L > kShort;                        // copies in the same pass
    if (here) { g.x8 = saved->x; g.f8 = saved->f; g.i8 = saved->i; }
    const bool vec = pitch % 16 == 0 && aligned(g.x, 16) && aligned(g.f, 16) && aligned(g.i, 16);
    e = by_type(p->dtype, p->gate, Forward{g, vec, here, s});
    if (e != cudaSuccess || !pack || !tokens || here) return cuda_status(e);
    e = launch_pack8(rows, g.D, g.ld, p->dtype, g.x, saved->x, s);
    if (e == cudaSuccess) e = launch_pack8(rows, g.D, g.ld, p->dtype, g.f, saved->f, s);
    if (e == cudaSuccess && lru) e = launch_pack8(rows, g.D, g.ld, p->dtype, g.i, saved->i, s);
    return cuda_status(e);
}

mru_status mru_gated_scan_backward(const mru_gated_problem* p, const mru_gated_inputs* in,
                                   const mru_gated_saved* saved, const void* dy, const float* dh_last, void* dx,
                                   void* df, void* di, float* dlam, float* dh0, void* ws, size_t ws_bytes,
                                   void* stream)
{
    mru_status st = check_problem(p);
    if (st != MRU_OK) return st;
    if (!in || !saved || !ws || !aligned(ws, 16) || !common_inputs_ok(*p, *in)) return MRU_ERR_INVALID_ARG;
    const size_t es = elem_size(p->dtype);
    const bool lru = p->gate == MRU_GATE_LRU, any = p->B * p->D > 0, tokens = any && p->L > 0;
    const bool packed = saved->x.q != nullptr;
    if (packed != (saved->f.q != nullptr) || (packed && lru) != (saved->i.q != nullptr)) return MRU_ERR_INVALID_ARG;
    if (!packed_ok(saved->x) || !packed_ok(saved->f) || !packed_ok(saved->i) || !aligned(saved->states, 4))
        return MRU_ERR_INVALID_ARG;
    if (tokens && (!saved->states || !dy || !dx || !df || (lru && !di))) return MRU_ERR_INVALID_ARG;
    if (tokens && !packed && (!in->x || !in->f || (lru && !in->i))) return MRU_ERR_INVALID_ARG;
    if (!lru && (di || dlam || in->i)) return MRU_ERR_INVALID_ARG;
    for (const void* v : {in->x, in->f, in->i, dy, (const void*)dx, (const void*)df, (const void*)di})
        if (!aligned(v, es)) return MRU_ERR_INVALID_ARG;
    if (!aligned(dh_last, 4) || !aligned(dlam, 4) || !aligned(dh0, 4)) return MRU_ERR_INVALID_ARG;
    Args g = make_args(*p, *in);
    const int64_t rows = g.B * g.L;
    const size_t state = (size_t)(g.B * g.D) * 4, width = (size_t)g.D * es, pitch = (size_t)g.ld * es;
    Buffers b;
    if (packed) {
        g.x = g.f = g.i = nullptr;
        for (const mru_packed8* v : {&saved->x, &saved->f, &saved->i}) {
            if (!v->q) continue;
            b.in(v->q, (size_t)(rows * g.D));
            b.in(v->scale, (size_t)(rows * div_up(g.D, 64)) * 4);
        }
    }
    for (const void* v : {g.x, g.f, g.i}) b.in_rows(v, rows, width, pitch);
    b.in(g.lam, (size_t)g.D * 4);
    b.in(g.reset, (size_t)rows);
    b.in(g.lens, (size_t)g.B * 4);
    b.in(saved->states, (size_t)(g.B * g.K * g.D) * 4);
    b.in(dy, (size_t)rows * width);
    b.in(dh_last, state);
    for (const void* v : {(const void*)dx, (const void*)df, (const void*)di}) b.out_rows(v, rows, width, (size_t)g.ldg * es);
    b.out(dlam, (size_t)g.D * 4);
    b.out(dh0, state);
    b.out(ws, ws_bytes);
    if (b.clash()) return MRU_ERR_INVALID_ARG;
    const Layout W = layout(*p, true);
    if (ws_bytes < W.bytes) return MRU_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (!any || g.K > 1) e = cudaMemsetAsync(ws, 0, W.zeroed, s);   // else the kernel clears the status word
    if (e == cudaSuccess && !any && dlam && g.D > 0) e = cudaMemsetAsync(dlam, 0, (size_t)g.D * 4, s);
    if (e != cudaSuccess || !any) return cuda_status(e);
    g.x8 = saved->x; g.f8 = saved->f; g.i8 = saved->i;
    g.states = saved->states;
    g.dy = dy; g.dh_last = dh_last;
    g.dx = dx; g.df = df; g.di = di; g.dh0 = dh0;
    place(g, W, ws);
    take_stall(g);
    g.dlam_part = dlam ? reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + W.part) : nullptr;
    if (packed && g.K > 1) {
        const size_t one = align256((size_t)(g.B * g.K * g.D) * sizeof(float));
        char* edge = reinterpret_cast<char*>(ws) + W.edge;
        g.edge_h = reinterpret_cast<float*>(edge);
        g.edge_d = reinterpret_cast<float*>(edge + one);
        g.edge_q = reinterpret_cast<float*>(edge + 2 * one);
    }
    bool vec = width % 16 == 0 && aligned(dy, 16);
    if (packed)
        vec = vec && g.D % 16 == 0 && aligned(saved->x.q, 16) && aligned(saved->f.q, 16) && aligned(saved->i.q, 16);
    else
        vec = vec && pitch % 16 == 0 && aligned(g.x, 16) && aligned(g.f, 16) && aligned(g.i, 16);
    e = by_type(p->dtype, p->gate, Backward{g, vec, packed, s});
    if (e == cudaSuccess && dlam) {
        const int64_t parts = g.B * (g.K > 0 ? g.K : 1);
        k_gated_dlam<<<(unsigned)div_up(g.D, 32), 256, 0, s>>>(parts, g.K > 0 ? g.K : 1, g.D, g.dlam_part, g.edge_q, g.lam,
                                                                  dlam);
        e = cudaGetLastError();
    }
    return cuda_status(e);
}

void mru_debug_stall_next_gated(int32_t ms) { g_stall_ms.store(ms > 0 ? ms : 0); }

}  // extern "C"
