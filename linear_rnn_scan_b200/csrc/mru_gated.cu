// mru_gated.cu -- gated linear recurrence: h_t = a_t h_{t-1} + b_t per channel,
// its backward, and their entry points.
#include <string.h>

#include "mru_ops.cuh"

namespace mru {
namespace {

using namespace ops;

constexpr int kKeep = MRU_GATED_KEEP;

struct Args {
    int64_t B, L, D, ld, ldg, K;     // K: kept states per sequence, ceil(L / 64)
    float c;
    const void *x, *f, *i;
    mru_packed8 x8, f8, i8;
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
    float *dlam_part, *dh0;          // dlam_part [B, D]: a sequence's sum of q
};

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

// Decay and input of a token; csp = c softplus(lam).
template <int GATE>
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
        float sf, nf, si, ni;
        sigmoid2(f, sf, nf);
        sigmoid2(i, si, ni);
        float m;                                      // a - 1
        exp_expm1_neg(-csp * sf, a, m);
        b = sqrtf(-m * (1.0f + a)) * si * x;          // 1 - a^2 = -m (1 + a)
    }
}

// a h where a = 0 forgets h whatever it is.
__device__ __forceinline__ float carry_in(float a, float h) { return a == 0.0f ? 0.0f : a * h; }

__device__ __forceinline__ int64_t valid_tokens(const Args& g, int64_t b)
{
    if (!g.lens) return g.L;
    const int64_t n = g.lens[b];
    return n < 0 ? 0 : n < g.L ? n : g.L;
}

// A thread per channel, token after token.
template <typename T, int GATE>
__global__ void __launch_bounds__(64) k_gated_serial(Args g)
{
    const int64_t ch = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (ch >= g.B * g.D) return;
    const int64_t b = ch / g.D, d = ch - b * g.D, len = valid_tokens(g, b);
    const float csp = GATE == MRU_GATE_LRU ? g.c * softplus(g.lam[d]) : 0.0f;
    float h = g.h0 ? g.h0[ch] : 0.0f;
    for (int64_t t = 0; t < g.L; ++t) {
        const int64_t row = b * g.L + t;
        if (g.states && t % kKeep == 0) g.states[(b * g.K + t / kKeep) * g.D + d] = h;
        float out = 0.0f;
        if (t < len) {
            float x, f, i, a, u;
            load_token<T, GATE, false>(g, row, d, x, f, i);
            gates<GATE>(x, f, i, csp, a, u);
            if (g.reset && g.reset[row]) a = 0.0f;
            h = out = carry_in(a, h) + u;
        }
        ((T*)g.y)[row * g.D + d] = from_f32<T>(out);
    }
    if (g.h_last) g.h_last[ch] = h;
}

template <typename T, int GATE, bool PACKED>
__global__ void __launch_bounds__(64) k_gated_serial_bwd(Args g)
{
    const int64_t ch = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (ch >= g.B * g.D) return;
    const int64_t b = ch / g.D, d = ch - b * g.D, len = valid_tokens(g, b);
    const float csp = GATE == MRU_GATE_LRU ? g.c * softplus(g.lam[d]) : 0.0f;
    float delta = g.dh_last ? g.dh_last[ch] : 0.0f;   // gradient of the state after token t
    float dlam = 0.0f;
    float prev[kKeep];
    for (int64_t k = g.K - 1; k >= 0; --k) {
        const int n = (int)(g.L - k * kKeep < kKeep ? g.L - k * kKeep : kKeep);
        float h = g.states[(b * g.K + k) * g.D + d];
        for (int j = 0; j < n; ++j) {
            prev[j] = h;
            const int64_t t = k * kKeep + j, row = b * g.L + t;
            if (t >= len) continue;
            float x, f, i, a, u;
            load_token<T, GATE, PACKED>(g, row, d, x, f, i);
            gates<GATE>(x, f, i, csp, a, u);
            if (g.reset && g.reset[row]) { a = 0.0f; prev[j] = 0.0f; }
            h = carry_in(a, h) + u;
        }
        for (int j = n - 1; j >= 0; --j) {
            const int64_t t = k * kKeep + j, row = b * g.L + t, e = row * g.ldg + d;
            float gx = 0.0f, gf = 0.0f, gi = 0.0f;
            if (t < len) {
                float x, f, i, a, u;
                load_token<T, GATE, PACKED>(g, row, d, x, f, i);
                gates<GATE>(x, f, i, csp, a, u);
                delta += to_f32(((const T*)g.dy)[row * g.D + d]);
                if constexpr (GATE == MRU_GATE_DECAY) {
                    gx = delta;
                    gf = delta * prev[j];
                } else if constexpr (GATE == MRU_GATE_SIGMOID) {
                    float s, na;
                    sigmoid2(f, s, na);
                    gx = na * delta;
                    gf = s * na * (prev[j] - x) * delta;
                } else {
                    float sf, nf, si, ni;
                    sigmoid2(f, sf, nf);
                    sigmoid2(i, si, ni);
                    const float la = -csp * sf;
                    float av, m;
                    exp_expm1_neg(la, av, m);
                    const float v = -m * (1.0f + av);
                    const float r = v > 0.0f ? rsqrtf(v) : 0.0f, beta = v * r;
                    const float q = delta * la * (av * prev[j] - si * x * av * av * r);
                    gx = delta * beta * si;
                    gi = delta * beta * x * si * ni;
                    gf = q * nf;
                    dlam += q;
                }
                if (g.reset && g.reset[row]) a = 0.0f;
                delta = carry_in(a, delta);
            }
            ((T*)g.dx)[e] = from_f32<T>(gx);
            ((T*)g.df)[e] = from_f32<T>(gf);
            if (GATE == MRU_GATE_LRU) ((T*)g.di)[e] = from_f32<T>(gi);
        }
    }
    if (g.dh0) g.dh0[ch] = delta;
    if (GATE == MRU_GATE_LRU && g.dlam_part) g.dlam_part[ch] = dlam;
}

// dlam = s(lam) / softplus(lam) times the sum of the sequences' sums.
__global__ void __launch_bounds__(128) k_gated_dlam(int64_t parts, int64_t D, const float* __restrict__ part,
                                                    const float* __restrict__ lam, float* __restrict__ dlam)
{
    const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (d >= D) return;
    double s = 0.0;
    for (int64_t p = 0; p < parts; ++p) s += (double)part[p * D + d];
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

struct Forward {
    const Args& g;
    cudaStream_t s;
    template <typename T, int GATE>
    cudaError_t operator()() const
    {
        k_gated_serial<T, GATE><<<(unsigned)div_up(g.B * g.D, 64), 64, 0, s>>>(g);
        return cudaGetLastError();
    }
};

struct Backward {
    const Args& g;
    bool packed;
    cudaStream_t s;
    template <typename T, int GATE>
    cudaError_t operator()() const
    {
        const unsigned grid = (unsigned)div_up(g.B * g.D, 64);
        if (packed)
            k_gated_serial_bwd<T, GATE, true><<<grid, 64, 0, s>>>(g);
        else
            k_gated_serial_bwd<T, GATE, false><<<grid, 64, 0, s>>>(g);
        return cudaGetLastError();
    }
};

}  // namespace
}  // namespace mru

using namespace mru;

extern "C" {

size_t mru_gated_workspace_size(const mru_gated_problem* p)
{
    if (check_problem(p) != MRU_OK) return 0;
    return 256;
}

size_t mru_gated_backward_workspace_size(const mru_gated_problem* p)
{
    if (check_problem(p) != MRU_OK) return 0;
    return 256 + align256((size_t)p->B * (size_t)p->D * 4);
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
    if (ws_bytes < mru_gated_workspace_size(p)) return MRU_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(uint32_t), s);
    if (e != cudaSuccess || !any) return cuda_status(e);
    g.y = y;
    g.h_last = h_last;
    g.states = saved ? saved->states : nullptr;
    if ((e = by_type(p->dtype, p->gate, Forward{g, s})) != cudaSuccess || !pack || !tokens) return cuda_status(e);
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
    if (ws_bytes < mru_gated_backward_workspace_size(p)) return MRU_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(uint32_t), s);
    if (e == cudaSuccess && !any && dlam && g.D > 0) e = cudaMemsetAsync(dlam, 0, (size_t)g.D * 4, s);
    if (e != cudaSuccess || !any) return cuda_status(e);
    g.x8 = saved->x; g.f8 = saved->f; g.i8 = saved->i;
    g.states = saved->states;
    g.dy = dy; g.dh_last = dh_last;
    g.dx = dx; g.df = df; g.di = di; g.dh0 = dh0;
    g.dlam_part = dlam ? reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + 256) : nullptr;
    e = by_type(p->dtype, p->gate, Backward{g, packed, s});
    if (e == cudaSuccess && dlam) {
        k_gated_dlam<<<(unsigned)div_up(g.D, 128), 128, 0, s>>>(g.B, g.D, g.dlam_part, g.lam, dlam);
        e = cudaGetLastError();
    }
    return cuda_status(e);
}

}  // extern "C"
