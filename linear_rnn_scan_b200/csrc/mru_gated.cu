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
        const float r = v > 0.0f ? rsqrtf(v) : 0.0f;       // la / u tends to 0 with u
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
    if (ch == 0) *g.status = 0;
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
    if (ch == 0) *g.status = 0;
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

// ------------------------------------------------------------------ tiles ---

// Shared memory of a tile kernel beside its stages.
struct TileMem {
    float4 agg[kWarps][32];              // a warp's map, two channels to a lane
    float4 ent[2 * kFan][32];            // what the carry is made of
    float csp[2][kCh];
    uint32_t next[2];
};

// Draws tiles in the order of the scan.  A tile waits only for tiles drawn
// before it, and a block works through its tiles in the order drawn, so the
// earliest unfinished tile never waits.
__device__ __forceinline__ uint32_t draw(const Args& g, uint32_t before)
{
    return g.ticket ? atomicAdd(g.ticket, 1u) : before + gridDim.x;
}

// Tokens of a warp that are not padding, and which of them start anew.
__device__ __forceinline__ void warp_masks(const Args& g, const Tile& t, int w, int lane, int& n, uint32_t& resets)
{
    const int64_t at = t.t0 + w * kStep, left = valid_tokens(g, t.b) - at;
    n = left <= 0 ? 0 : left < kStep ? (int)left : kStep;
    resets = 0;
    if (g.reset) resets = __ballot_sync(~0u, lane < n && g.reset[t.b * g.L + at + lane] != 0);
}

// 8-bit copies of a warp's tokens: a run of 64 channels is the warp's row, so
// a lane takes the factors of one run (token and input) for all.
template <typename T, int NIN>
__device__ __forceinline__ void pack_rows(const Args& g, const Tile& t, int w, int lane, const T* stage, bool wide8)
{
    uint32_t mine = 0;
#pragma unroll
    for (int n = 0; n < NIN; ++n)
#pragma unroll
        for (int s = 0; s < kStep; ++s) {
            const float2 v = pair_at(stage + (n * kTok + w * kStep + s) * kCh + 2 * lane);
            const uint32_t m = __reduce_max_sync(~0u, max(mag_bits(v.x), mag_bits(v.y)));
            if (lane == n * kStep + s) mine = m;
        }
    float inv, scale;
    pack8_factors(__uint_as_float(mine), inv, scale);
    const int64_t row0 = t.b * g.L + t.t0 + w * kStep, runs = g.cgs;
    const int64_t left = g.L - t.t0 - w * kStep;
    if (lane < NIN * kStep && lane % kStep < left) {
        float* to = lane < kStep ? g.x8.scale : lane < 2 * kStep ? g.f8.scale : g.i8.scale;
        to[(row0 + lane % kStep) * runs + t.d0 / kCh] = scale;
    }
    const int64_t d = t.d0 + 2 * lane;
#pragma unroll
    for (int n = 0; n < NIN; ++n) {
        int8_t* to = n == 0 ? g.x8.q : n == 1 ? g.f8.q : g.i8.q;
#pragma unroll
        for (int s = 0; s < kStep; ++s) {
            const float k = __shfl_sync(~0u, inv, n * kStep + s);
            if (s >= left) continue;
            const float2 v = pair_at(stage + (n * kTok + w * kStep + s) * kCh + 2 * lane);
            const int q0 = pack8_q(v.x, k), q1 = pack8_q(v.y, k);
            int8_t* at = to + (row0 + s) * g.D + d;
            if (wide8) {
                if (d < g.D) *reinterpret_cast<char2*>(at) = make_char2((char)q0, (char)q1);
            } else {
                if (d < g.D) at[0] = (int8_t)q0;
                if (d + 1 < g.D) at[1] = (int8_t)q1;
            }
        }
    }
}

// The decays and inputs of a warp's tokens and their map.  SPECIAL: padding
// (nothing happens) or resets (the state before counts as zero).
template <typename T, int GATE, bool SPECIAL, bool NEAR>
__device__ __forceinline__ float4 local_map(const T* stage, int w, int lane, float2 csp, int n, uint32_t resets,
                                            float2 (&a)[kStep], float2 (&b)[kStep])
{
    float4 m = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
        const T* at = stage + (w * kStep + s) * kCh + 2 * lane;
        if (SPECIAL && s >= n) {
            a[s] = make_float2(1.0f, 1.0f);
            b[s] = make_float2(0.0f, 0.0f);
            continue;
        }
        const float2 x = pair_at(at), f = pair_at(at + kTok * kCh);
        const float2 i = GATE == MRU_GATE_LRU ? pair_at(at + 2 * kTok * kCh) : make_float2(0.0f, 0.0f);
        gates<GATE, NEAR>(x.x, f.x, i.x, csp.x, a[s].x, b[s].x);
        gates<GATE, NEAR>(x.y, f.y, i.y, csp.y, a[s].y, b[s].y);
        if (SPECIAL && (resets >> s & 1)) m = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        m.x *= a[s].x;
        m.z *= a[s].y;
        if (GATE == MRU_GATE_DECAY) {
            m.y = carry_in(a[s].x, m.y) + b[s].x;
            m.w = carry_in(a[s].y, m.w) + b[s].y;
        } else {
            m.y = fmaf(a[s].x, m.y, b[s].x);
            m.w = fmaf(a[s].y, m.w, b[s].y);
        }
    }
    return m;
}

template <typename T, int GATE, bool SPECIAL>
__device__ __forceinline__ void run_states(const Args& g, const Tile& t, int w, int lane, float2 h, int n,
                                           uint32_t resets, const float2 (&a)[kStep], const float2 (&b)[kStep],
                                           bool wide)
{
    const int64_t d = t.d0 + 2 * lane, left = g.L - t.t0 - w * kStep;
    T* y = (T*)g.y + (t.b * g.L + t.t0 + w * kStep) * g.D + d;
    const bool one = d < g.D, two = d + 1 < g.D;
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
        if (SPECIAL && (resets >> s & 1)) h = make_float2(0.0f, 0.0f);
        if (GATE == MRU_GATE_DECAY) {
            h.x = carry_in(a[s].x, h.x) + b[s].x;
            h.y = carry_in(a[s].y, h.y) + b[s].y;
        } else {
            h.x = fmaf(a[s].x, h.x, b[s].x);
            h.y = fmaf(a[s].y, h.y, b[s].y);
        }
        const float2 out = SPECIAL && s >= n ? make_float2(0.0f, 0.0f) : h;
        if (!SPECIAL || s < left) put_pair(y + s * g.D, out, wide && one, one, two);
    }
}

template <typename T, int GATE>
constexpr size_t forward_stage_bytes()
{
    return (size_t)inputs_of(GATE) * kTok * kCh * sizeof(T);
}

template <typename T, int GATE, bool VEC>
__device__ __forceinline__ void load_inputs(const Args& g, const Tile& t, T* to)
{
    load_tile<T, VEC>(g, t, g.x, g.ld, to);
    load_tile<T, VEC>(g, t, g.f, g.ld, to + kTok * kCh);
    if (GATE == MRU_GATE_LRU) load_tile<T, VEC>(g, t, g.i, g.ld, to + 2 * kTok * kCh);
}

// Forward: every input is read once and every output written once.  Blocks
// stay and draw tiles in the order of the scan; the next tile's inputs are on
// their way while one is worked on.  Per tile: each warp maps its 8 tokens,
// the maps meet in shared memory, the tile's map is published, the carry is
// fetched (by then the tiles before have published theirs), and the states
// are run again from it over decays and inputs that stayed in registers.
template <typename T, int GATE, bool VEC, bool PACK>
__global__ void __launch_bounds__(kThreads, 3) k_gated_tile(Args g)
{
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ TileMem mem;
    constexpr int NIN = inputs_of(GATE), kElems = NIN * kTok * kCh;
    T* stage = reinterpret_cast<T*>(stages);
    const int tid = threadIdx.x, lane = tid & 31, w = tid / 32;
    const bool wide = g.D % 2 == 0 && aligned(g.y, 2 * sizeof(T));
    const bool wide8 = PACK && g.D % 2 == 0 && aligned(g.x8.q, 2) && aligned(g.f8.q, 2) &&
                       (GATE != MRU_GATE_LRU || aligned(g.i8.q, 2));
    if (tid == 0) {
        const uint32_t first = g.ticket ? atomicAdd(g.ticket, 1u) : blockIdx.x;
        mem.next[0] = first;
        mem.next[1] = draw(g, first);
        if (!g.ticket && blockIdx.x == 0) *g.status = 0;
    }
    __syncthreads();
    uint32_t cur = mem.next[0], nxt = mem.next[1];
    if (cur < g.tiles) {
        const Tile t = tile_of<false>(g, cur);
        load_inputs<T, GATE, VEC>(g, t, stage);
        if (GATE == MRU_GATE_LRU && tid < kCh)
            mem.csp[0][tid] = t.d0 + tid < g.D ? g.c * softplus(g.lam[t.d0 + tid]) : 0.0f;
    }
    cp_commit();
    for (int st = 0; cur < g.tiles; st ^= 1) {
        uint32_t drawn = 0;
        if (tid == 0) drawn = draw(g, nxt);
        float lam = 0.0f;
        if (nxt < g.tiles) {
            const Tile t = tile_of<false>(g, nxt);
            load_inputs<T, GATE, VEC>(g, t, stage + (st ^ 1) * kElems);
            if (GATE == MRU_GATE_LRU && tid < kCh && t.d0 + tid < g.D) lam = g.lam[t.d0 + tid];
        }
        cp_commit();
        const Tile t = tile_of<false>(g, cur);
        int n;
        uint32_t resets;
        warp_masks(g, t, w, lane, n, resets);
        cp_wait<1>();
        __syncthreads();
        const T* in = stage + st * kElems;
        if constexpr (PACK) pack_rows<T, NIN>(g, t, w, lane, in, wide8);
        float2 csp = make_float2(0.0f, 0.0f);
        if (GATE == MRU_GATE_LRU) csp = *reinterpret_cast<const float2*>(&mem.csp[st][2 * lane]);
        const bool near = GATE == MRU_GATE_LRU && __all_sync(~0u, csp.x <= 0.5f && csp.y <= 0.5f);
        const bool special = n < kStep || resets;
        float2 a[kStep], b[kStep];
        float4 own;
        if (special) own = local_map<T, GATE, true, false>(in, w, lane, csp, n, resets, a, b);
        else if (near) own = local_map<T, GATE, false, GATE == MRU_GATE_LRU>(in, w, lane, csp, n, resets, a, b);
        else own = local_map<T, GATE, false, false>(in, w, lane, csp, n, resets, a, b);
        mem.agg[w][lane] = own;
        __syncthreads();
        float4 pre = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        for (int v = 0; v < w; ++v) pre = after(mem.agg[v][lane], pre);
        if (w == kWarps - 1) {
            own = after(own, pre);                         // the tile's map
            if (!t.last && !(g.withhold && cur == 0)) publish(tile_words(g, t, t.order), lane, own);
        }
        fetch_carry(g, t, w, lane, g.h0, mem.ent);
        if (tid == 0) mem.next[0] = drawn;
        __syncthreads();
        const float2 carry = carry_of(t, lane, mem.ent);
        const int64_t d = t.d0 + 2 * lane;
        if (w == kWarps - 1) {
            publish_up(g, t, lane, own, carry, mem.ent);
            if (t.last && g.h_last) {
                const float2 h = apply(own, carry);
                if (d < g.D) g.h_last[t.b * g.D + d] = h.x;
                if (d + 1 < g.D) g.h_last[t.b * g.D + d + 1] = h.y;
            }
        }
        if (w == 0 && g.states) {
            float* to = g.states + (t.b * g.K + t.order) * g.D + d;
            if (d < g.D) to[0] = carry.x;
            if (d + 1 < g.D) to[1] = carry.y;
        }
        const float2 h = apply(pre, carry);
        if (special) run_states<T, GATE, true>(g, t, w, lane, h, n, resets, a, b, wide);
        else run_states<T, GATE, false>(g, t, w, lane, h, n, resets, a, b, wide);
        if (GATE == MRU_GATE_LRU && tid < kCh) mem.csp[st ^ 1][tid] = g.c * softplus(lam);
        cur = nxt;
        nxt = mem.next[0];
    }
}

// Shared memory of the backward beside its stages.
struct BackMem {
    float4 agg[kWarps][32];              // a warp's map of states
    float4 back[kWarps][32];             // and of gradients
    float4 ent[2 * kFan][32];
    float2 dlam[kWarps][32];
    float csp[2][kCh];
    float state[2][kCh];                 // the kept state before the tile
    float scale[2][3][kTok];             // 8-bit copies: the scale of a token's run
    uint32_t next[2];
};

template <typename T, int GATE, bool PACKED>
constexpr size_t backward_stage_bytes()
{
    return (size_t)kTok * kCh * (inputs_of(GATE) * (PACKED ? 1 : sizeof(T)) + sizeof(T));
}
// Two stages where three blocks of them fit an SM's 227 KB, else one.
template <typename T, int GATE, bool PACKED>
constexpr int backward_stages()
{
    return backward_stage_bytes<T, GATE, PACKED>() <= 36 * 1024 ? 2 : 1;
}

template <typename T, int GATE, bool VEC, bool PACKED>
__device__ __forceinline__ void load_back(const Args& g, const Tile& t, unsigned char* stage, BackMem& mem, int st)
{
    constexpr int NIN = inputs_of(GATE);
    T* dy = reinterpret_cast<T*>(stage);
    load_tile<T, VEC>(g, t, g.dy, g.D, dy);
    const int tid = threadIdx.x;
    if constexpr (PACKED) {
        int8_t* q = reinterpret_cast<int8_t*>(dy + kTok * kCh);
#pragma unroll
        for (int n = 0; n < NIN; ++n) {
            const mru_packed8& h = n == 0 ? g.x8 : n == 1 ? g.f8 : g.i8;
            const int8_t* src = h.q + t.b * g.L * g.D;
            if constexpr (VEC) {
                const int row = tid / 4, c = tid % 4 * 16;
                const bool in = t.t0 + row < g.L && t.d0 + c < g.D;
                cp_async(q + n * kTok * kCh + row * kCh + c, in ? src + (t.t0 + row) * g.D + t.d0 + c : src, in ? 16 : 0);
            } else {
                for (int k = tid; k < kTok * kCh; k += kThreads) {
                    const int row = k / kCh, c = k % kCh;
                    const bool in = t.t0 + row < g.L && t.d0 + c < g.D;
                    q[n * kTok * kCh + k] = in ? src[(t.t0 + row) * g.D + t.d0 + c] : (int8_t)0;
                }
            }
            if (tid < kTok) {
                const bool in = t.t0 + tid < g.L;
                const float* at = h.scale + (in ? (t.b * g.L + t.t0 + tid) * (int64_t)g.cgs + t.d0 / kCh : 0);
                cp_async4(&mem.scale[st][n][tid], at, in ? 4 : 0);
            }
        }
    } else {
        load_inputs<T, GATE, VEC>(g, t, dy + kTok * kCh);
    }
    if (tid < kCh) {
        const bool in = t.d0 + tid < g.D;
        const float* at = g.states + (in ? (t.b * g.K + t.t0 / kTok) * g.D + t.d0 + tid : 0);
        cp_async4(&mem.state[st][tid], at, in ? 4 : 0);
    }
}

// Two channels of a token's input n, from the stage.
template <typename T, bool PACKED>
__device__ __forceinline__ float2 input_pair(const unsigned char* stage, const float (&scale)[3][kTok], int n, int row,
                                             int lane)
{
    const unsigned char* in = stage + kTok * kCh * sizeof(T);
    if constexpr (PACKED) {
        const char2 q = *reinterpret_cast<const char2*>(in + (n * kTok + row) * kCh + 2 * lane);
        const float k = scale[n][row];
        return make_float2((float)(signed char)q.x * k, (float)(signed char)q.y * k);
    } else {
        return pair_at(reinterpret_cast<const T*>(in) + (n * kTok + row) * kCh + 2 * lane);
    }
}

template <typename T, int GATE, bool PACKED, bool NEAR>
__device__ __forceinline__ float4 back_map(const unsigned char* stage, const float (&scale)[3][kTok], int w, int lane,
                                           float2 csp, int n, uint32_t resets)
{
    float4 m = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
        if (s >= n) continue;
        const int row = w * kStep + s;
        const float2 x = input_pair<T, PACKED>(stage, scale, 0, row, lane);
        const float2 f = input_pair<T, PACKED>(stage, scale, 1, row, lane);
        const float2 i = GATE == MRU_GATE_LRU ? input_pair<T, PACKED>(stage, scale, 2, row, lane) : make_float2(0.0f, 0.0f);
        float2 a, b;
        gates<GATE, NEAR>(x.x, f.x, i.x, csp.x, a.x, b.x);
        gates<GATE, NEAR>(x.y, f.y, i.y, csp.y, a.y, b.y);
        if (resets >> s & 1) m = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        m = make_float4(m.x * a.x, carry_in(a.x, m.y) + b.x, m.z * a.y, carry_in(a.y, m.w) + b.y);
    }
    return m;
}

// A warp's tokens: states from h, the factors of the gradients, and the map of
// gradients e -> P e + E from the token after the last to before the first.
// dl: sum q d and sum q dd/de (for lam) at e = 0, without the first token where
// it is a piece's edge (k_gated_edge counts it).  h: the state after the last.
template <typename T, int GATE, bool PACKED, bool NEAR>
__device__ __forceinline__ float4 back_factors(const unsigned char* stage, const float (&scale)[3][kTok], int w,
                                               int lane, float2 csp, float2& h, int n, uint32_t resets, bool edge,
                                               float2 (&a)[kStep], float2 (&cx)[kStep], float2 (&cf)[kStep],
                                               float2 (&ci)[kStep], float4& dl)
{
    float2 q[kStep];
#pragma unroll
    for (int s = 0; s < kStep; ++s) {
        a[s] = make_float2(1.0f, 1.0f);
        cx[s] = cf[s] = ci[s] = q[s] = make_float2(0.0f, 0.0f);
        if (s >= n) continue;
        const int row = w * kStep + s;
        const float2 x = input_pair<T, PACKED>(stage, scale, 0, row, lane);
        const float2 f = input_pair<T, PACKED>(stage, scale, 1, row, lane);
        const float2 i = GATE == MRU_GATE_LRU ? input_pair<T, PACKED>(stage, scale, 2, row, lane) : make_float2(0.0f, 0.0f);
        const bool reset = resets >> s & 1;
        if (reset) h = make_float2(0.0f, 0.0f);
        float2 b;
        gradient_factors<GATE, NEAR>(x.x, f.x, i.x, csp.x, h.x, a[s].x, b.x, cx[s].x, cf[s].x, ci[s].x, q[s].x);
        gradient_factors<GATE, NEAR>(x.y, f.y, i.y, csp.y, h.y, a[s].y, b.y, cx[s].y, cf[s].y, ci[s].y, q[s].y);
        h.x = carry_in(a[s].x, h.x) + b.x;
        h.y = carry_in(a[s].y, h.y) + b.y;
        if (reset) a[s] = make_float2(0.0f, 0.0f);
    }
    if (PACKED && edge) q[0] = make_float2(0.0f, 0.0f);
    float4 m = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
    dl = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int s = kStep - 1; s >= 0; --s) {
        if (s >= n) continue;
        const float2 dy = pair_at(reinterpret_cast<const T*>(stage) + (w * kStep + s) * kCh + 2 * lane);
        const float2 d = make_float2(m.y + dy.x, m.w + dy.y);
        if (GATE == MRU_GATE_LRU) {
            dl.x = fmaf(q[s].x, d.x, dl.x);
            dl.y = fmaf(q[s].x, m.x, dl.y);
            dl.z = fmaf(q[s].y, d.y, dl.z);
            dl.w = fmaf(q[s].y, m.z, dl.w);
        }
        m = make_float4(m.x * a[s].x, carry_in(a[s].x, d.x), m.z * a[s].y, carry_in(a[s].y, d.y));
    }
    return m;
}

// Backward, tiles from the last to the first: the states of the tile again
// from its kept state, the factors of the gradients, then the gradient's own
// recurrence with its carry from the later tiles, as the forward's.
template <typename T, int GATE, bool VEC, bool PACKED>
__global__ void __launch_bounds__(kThreads, 2) k_gated_tile_bwd(Args g)
{
    extern __shared__ __align__(16) unsigned char stages[];
    __shared__ BackMem mem;
    constexpr size_t kBytes = backward_stage_bytes<T, GATE, PACKED>();
    constexpr int STAGES = backward_stages<T, GATE, PACKED>();
    constexpr bool lru = GATE == MRU_GATE_LRU;
    const int tid = threadIdx.x, lane = tid & 31, w = tid / 32;
    const bool wide = g.D % 2 == 0 && g.ldg % 2 == 0 && aligned(g.dx, 2 * sizeof(T)) && aligned(g.df, 2 * sizeof(T)) &&
                      (!lru || aligned(g.di, 2 * sizeof(T)));
    if (tid == 0) {
        const uint32_t first = g.ticket ? atomicAdd(g.ticket, 1u) : blockIdx.x;
        mem.next[0] = first;
        mem.next[1] = draw(g, first);
        if (!g.ticket && blockIdx.x == 0) *g.status = 0;
    }
    __syncthreads();
    uint32_t cur = mem.next[0], nxt = mem.next[1];
    if (cur < g.tiles) {
        const Tile t = tile_of<true>(g, cur);
        if (STAGES == 2) load_back<T, GATE, VEC, PACKED>(g, t, stages, mem, 0);
        if (lru && tid < kCh) mem.csp[0][tid] = t.d0 + tid < g.D ? g.c * softplus(g.lam[t.d0 + tid]) : 0.0f;
    }
    cp_commit();
    for (int st = 0; cur < g.tiles; st ^= 1) {
        unsigned char* stage = stages + (STAGES == 2 ? st * kBytes : 0);
        uint32_t drawn = 0;
        if (tid == 0) drawn = draw(g, nxt);
        float lam = 0.0f;
        const Tile t = tile_of<true>(g, cur);
        if (STAGES == 1) load_back<T, GATE, VEC, PACKED>(g, t, stage, mem, st);
        if (nxt < g.tiles) {
            const Tile u = tile_of<true>(g, nxt);
            if (STAGES == 2) load_back<T, GATE, VEC, PACKED>(g, u, stages + (st ^ 1) * kBytes, mem, st ^ 1);
            if (lru && tid < kCh && u.d0 + tid < g.D) lam = g.lam[u.d0 + tid];
        }
        cp_commit();
        int n;
        uint32_t resets;
        warp_masks(g, t, w, lane, n, resets);
        cp_wait<STAGES - 1>();
        __syncthreads();
        float2 csp = make_float2(0.0f, 0.0f);
        if (lru) csp = *reinterpret_cast<const float2*>(&mem.csp[st][2 * lane]);
        const bool near = lru && __all_sync(~0u, csp.x <= 0.5f && csp.y <= 0.5f);
        mem.agg[w][lane] = near ? back_map<T, GATE, PACKED, lru>(stage, mem.scale[st], w, lane, csp, n, resets)
                                : back_map<T, GATE, PACKED, false>(stage, mem.scale[st], w, lane, csp, n, resets);
        __syncthreads();
        float2 h = *reinterpret_cast<const float2*>(&mem.state[st][2 * lane]);
        for (int v = 0; v < w; ++v) h = apply(mem.agg[v][lane], h);
        float2 a[kStep], cx[kStep], cf[kStep], ci[kStep];
        float4 dl;
        const bool edge = PACKED && w == 0 && t.t0 > 0;
        float4 own = near ? back_factors<T, GATE, PACKED, lru>(stage, mem.scale[st], w, lane, csp, h, n, resets, edge,
                                                               a, cx, cf, ci, dl)
                          : back_factors<T, GATE, PACKED, false>(stage, mem.scale[st], w, lane, csp, h, n, resets, edge,
                                                                 a, cx, cf, ci, dl);
        mem.back[w][lane] = own;
        __syncthreads();
        float4 post = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
        for (int v = kWarps - 1; v > w; --v) post = after(mem.back[v][lane], post);
        if (w == 0) {
            own = after(own, post);                        // the tile's map
            if (!t.last && !(g.withhold && cur == 0)) publish(tile_words(g, t, t.order), lane, own);
        }
        fetch_carry(g, t, w, lane, g.dh_last, mem.ent);
        if (tid == 0) mem.next[0] = drawn;
        __syncthreads();
        const float2 carry = carry_of(t, lane, mem.ent);
        const int64_t d0 = t.d0 + 2 * lane;
        const bool one = d0 < g.D, two = d0 + 1 < g.D;
        if (w == 0) {
            publish_up(g, t, lane, own, carry, mem.ent);
            if (t.last && g.dh0) {
                const float2 e = apply(own, carry);
                if (one) g.dh0[t.b * g.D + d0] = e.x;
                if (two) g.dh0[t.b * g.D + d0 + 1] = e.y;
            }
        }
        if (PACKED && g.edge_h && w == kWarps - 1 && t.order > 0) {
            float* to = g.edge_h + (t.b * g.K + t.t0 / kTok + 1) * g.D + d0;
            if (one) to[0] = h.x;
            if (two) to[1] = h.y;
        }
        float2 e = apply(post, carry);
        if (lru) mem.dlam[w][lane] = make_float2(fmaf(dl.y, e.x, dl.x), fmaf(dl.w, e.y, dl.z));
        const int64_t at = (t.b * g.L + t.t0 + w * kStep) * g.ldg + d0, left = g.L - t.t0 - w * kStep;
#pragma unroll
        for (int s = kStep - 1; s >= 0; --s) {
            if (s >= left) continue;
            float2 d = make_float2(0.0f, 0.0f);
            if (s < n) {
                const float2 dy = pair_at(reinterpret_cast<const T*>(stage) + (w * kStep + s) * kCh + 2 * lane);
                d = make_float2(e.x + dy.x, e.y + dy.y);
                e = make_float2(carry_in(a[s].x, d.x), carry_in(a[s].y, d.y));
            }
            if (s == 0 && edge) {
                float* to = g.edge_d + (t.b * g.K + t.t0 / kTok) * g.D + d0;
                if (one) to[0] = d.x;
                if (two) to[1] = d.y;
            }
            put_pair((T*)g.dx + at + s * g.ldg, make_float2(cx[s].x * d.x, cx[s].y * d.y), wide && one, one, two);
            put_pair((T*)g.df + at + s * g.ldg, make_float2(cf[s].x * d.x, cf[s].y * d.y), wide && one, one, two);
            if (lru)
                put_pair((T*)g.di + at + s * g.ldg, make_float2(ci[s].x * d.x, ci[s].y * d.y), wide && one, one, two);
        }
        if (lru && tid < kCh) mem.csp[st ^ 1][tid] = g.c * softplus(lam);
        cur = nxt;
        nxt = mem.next[0];
        __syncthreads();                                   // the stage may be filled again
        if (lru && g.dlam_part && tid < kCh && t.d0 + tid < g.D) {
            float s = 0.0f;
            for (int v = 0; v < kWarps; ++v) s += reinterpret_cast<const float*>(mem.dlam[v])[tid];
            g.dlam_part[(t.b * g.K + t.t0 / kTok) * g.D + t.d0 + tid] = s;
        }
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
        constexpr size_t smem = 2 * forward_stage_bytes<T, GATE>();
        static Fits fits[4];
        if (vec)
            return pack ? launch_tiles(k_gated_tile<T, GATE, true, true>, fits[0], g, smem, s)
                        : launch_tiles(k_gated_tile<T, GATE, true, false>, fits[1], g, smem, s);
        return pack ? launch_tiles(k_gated_tile<T, GATE, false, true>, fits[2], g, smem, s)
                    : launch_tiles(k_gated_tile<T, GATE, false, false>, fits[3], g, smem, s);
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
        constexpr size_t smem = backward_stages<T, GATE, PACKED>() * backward_stage_bytes<T, GATE, PACKED>();
        static Fits fits[2];
        const cudaError_t e = vec ? launch_tiles(k_gated_tile_bwd<T, GATE, true, PACKED>, fits[0], g, smem, s)
                                  : launch_tiles(k_gated_tile_bwd<T, GATE, false, PACKED>, fits[1], g, smem, s);
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
    if (!in || !ws || !aligned(ws, 16) || !common_inputs_ok(*p, *in)) return MRU_ERR_INVALID_ARG;
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
    b.out(ws, ws_bytes);
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
    if (ws_bytes < W.bytes) return MRU_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (!any || g.K > 1) e = cudaMemsetAsync(ws, 0, W.zeroed, s);   // else the kernel clears the status word
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
