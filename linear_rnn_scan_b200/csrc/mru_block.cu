// mru_block.cu -- the ends of a block, row by row: r' = r + rs s act(g) N(y),
// z = N(r'), and the backward with the parameters' sums over rows.
//
// A row is held in registers, 8 columns to a thread, from its one read to its
// one write; its sums go through shuffles, then shared memory, then (rows
// wider than 4096) the distributed shared memory of a cluster of CTAs.
#include <cooperative_groups.h>
#include <string.h>

#include "mru_ops.cuh"

namespace cg = cooperative_groups;

namespace mru {
namespace {

using namespace ops;

constexpr int kMaxD = 16384;
constexpr int kCtaCols = 4096;             // 512 threads of 8 columns
constexpr int kMaxCluster = kMaxD / kCtaCols;

struct BArgs {
    int64_t rows, ldy, ldg, lddy, lddg;
    int32_t D, norm, act, cluster;
    float eps, rs;
    mru_block_params prm;
    const void *r, *y, *g;                 // forward: r; backward: the stored r'
    mru_packed8 r8, y8, g8;
    void *r_out, *z;                       // forward
    const void *dro, *dz;                  // backward
    void *dr, *dy, *dg;
    float* part;                           // [5][parts][D]: dw_y, ds, dw_z, db_y, db_z
    int32_t parts;
    bool has_y, has_z;
};

// The columns of a thread: 8 in a row (VEC), or 8 a team apart.
template <bool VEC>
struct Cols {
    int c0, step, D;             // D is also the row pitch of the 8-bit copies
    __device__ __forceinline__ int at(int e) const { return VEC ? c0 + e : c0 + e * step; }
    __device__ __forceinline__ bool ok(int e) const { return VEC ? c0 < D : at(e) < D; }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, const Cols<VEC>& c, float (&v)[8])
{
    if constexpr (VEC) {
        if (c.c0 >= c.D) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
        } else if constexpr (sizeof(T) == 2) {
            const uint4 w = *reinterpret_cast<const uint4*>(row + c.c0);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            const float4 a = *reinterpret_cast<const float4*>(row + c.c0);
            const float4 b = *reinterpret_cast<const float4*>(row + c.c0 + 4);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c.ok(e) ? to_f32(row[c.at(e)]) : 0.0f;
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, const Cols<VEC>& c, const float (&v)[8])
{
    if constexpr (VEC) {
        if (c.c0 >= c.D) return;
        if constexpr (sizeof(T) == 2) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                u[e] = *reinterpret_cast<const uint32_t*>(&p);
            }
            *reinterpret_cast<uint4*>(row + c.c0) = make_uint4(u[0], u[1], u[2], u[3]);
        } else {
            *reinterpret_cast<float4*>(row + c.c0) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(row + c.c0 + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c.ok(e)) row[c.at(e)] = from_f32<T>(v[e]);
    }
}

template <bool VEC>
__device__ __forceinline__ void load_param(const float* p, float none, const Cols<VEC>& c, float (&v)[8])
{
    if (p) {
        load8<float, VEC>(p, c, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = none;
    }
}

// The values 8 bits hold, from 8 of them and their run's scale.
__device__ __forceinline__ void held8(uint2 q, float s, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = (float)(int8_t)(q.x >> (8 * e)) * s;
        v[4 + e] = (float)(int8_t)(q.y >> (8 * e)) * s;
    }
}

// A row of values held in 8 bits, column by column.
__device__ __forceinline__ void load_packed(const mru_packed8& h, int64_t row, const Cols<false>& c, float (&v)[8])
{
    const int8_t* q = h.q + row * c.D;
    const float* sc = h.scale + row * ((c.D + 63) / 64);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = c.ok(e) ? (float)q[c.at(e)] * sc[c.at(e) / 64] : 0.0f;
}

// Rows on their way: every thread copies its own columns of the coming rows
// into its own slots of shared memory and later reads them back itself, so
// that no barrier is needed; the memory's latency is covered by the rows in
// flight, not by resident warps (whose registers hold whole rows).
template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* gmem)
{
    const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s), "l"(gmem), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Bytes of 8 columns of one input in a stage, and stages of `inputs` plain
// ones and `held` 8-bit ones (with their scales): up to 4 in 160 KB for 512
// threads.
template <typename T>
constexpr int plane_bytes() { return 8 * (int)sizeof(T); }
template <typename T>
constexpr int stage_bytes(int inputs, int held) { return inputs * plane_bytes<T>() + held * 12; }
template <typename T>
constexpr int stages_of(int inputs, int held)
{
    const int n = 160 * 1024 / (512 * stage_bytes<T>(inputs, held));
    return n > 4 ? 4 : n < 2 ? 2 : n;
}

// A thread's slots of one input: plane `at` (bytes per thread before it).
template <typename T>
struct Slot {
    unsigned char* base;                   // the stage
    __device__ __forceinline__ unsigned char* piece(int at, int k) const
    {
        return base + (size_t)(at + 16 * k) * blockDim.x + 16 * threadIdx.x;
    }
    __device__ __forceinline__ void fill(int at, const T* from) const
    {
#pragma unroll
        for (int k = 0; k < plane_bytes<T>() / 16; ++k) copy_async<16>(piece(at, k), (const char*)from + 16 * k);
    }
    __device__ __forceinline__ void read(int at, float (&v)[8]) const
    {
        if constexpr (sizeof(T) == 2) {
            const uint4 w = *reinterpret_cast<const uint4*>(piece(at, 0));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            const float4 a = *reinterpret_cast<const float4*>(piece(at, 0));
            const float4 b = *reinterpret_cast<const float4*>(piece(at, 1));
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
            v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        }
    }
    // 8-bit values: 8 bytes, then the scale
    __device__ __forceinline__ void fill8(int at, const mru_packed8& h, int64_t row, int c0, int D) const
    {
        copy_async<8>(base + (size_t)at * blockDim.x + 8 * threadIdx.x, h.q + row * D + c0);
        copy_async<4>(base + (size_t)(at + 8) * blockDim.x + 4 * threadIdx.x, h.scale + row * ((D + 63) / 64) + c0 / 64);
    }
    __device__ __forceinline__ void read8(int at, float (&v)[8]) const
    {
        held8(*reinterpret_cast<const uint2*>(base + (size_t)at * blockDim.x + 8 * threadIdx.x),
              *reinterpret_cast<const float*>(base + (size_t)(at + 8) * blockDim.x + 4 * threadIdx.x), v);
    }
};

// Writes a row's 8-bit copy (VEC: a run of 64 channels is 8 lanes in a row).
__device__ __forceinline__ void store_packed(const mru_packed8& h, int64_t row, const Cols<true>& c, const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, mag_bits(v[e]));
#pragma unroll
    for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
    if (c.c0 >= c.D) return;
    float inv, sc;
    pack8_factors(__uint_as_float(m), inv, sc);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e / 4] |= (uint32_t)(pack8_q(v[e], inv) & 0xff) << (8 * (e % 4));
    *reinterpret_cast<uint2*>(h.q + row * c.D + c.c0) = make_uint2(w[0], w[1]);
    if (c.c0 % 64 == 0) h.scale[row * ((c.D + 63) / 64) + c.c0 / 64] = sc;
}

// Sums over a row's team, the same bits in every thread.  TEAM > 0: lanes of a
// warp; 0: the CTA, and its cluster where there is one.  Buffers alternate, so
// that one barrier serves a reduction: a buffer is written again only after
// the next reduction's barrier, which every reader has reached.
struct ReduceMem {
    float4 warp[2][4][4];                  // [sum][warps by fours]; warps that are not there stay 0
    float4 cta[2][4];                      // [sum], a CTA of the cluster to a component
};

__device__ __forceinline__ void clear(ReduceMem& m)
{
    float* f = reinterpret_cast<float*>(&m);
    for (int k = threadIdx.x; k < (int)(sizeof(ReduceMem) / 4); k += blockDim.x) f[k] = 0.0f;
    __syncthreads();
}

// N sums of a warp: halves of it take over half of the sums each, so that 4
// sums take 6 shuffles.  Returns the lane's sum; lane 32 / N * k holds sum k.
template <int N>
__device__ __forceinline__ float warp_sums(const float (&v)[N], int lane)
{
    float r;
    if constexpr (N == 4) {
        const bool hi = lane & 16, up = lane & 8;
        const float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(~0u, hi ? v[0] : v[2], 16);
        const float b = (hi ? v[3] : v[1]) + __shfl_xor_sync(~0u, hi ? v[1] : v[3], 16);
        r = (up ? b : a) + __shfl_xor_sync(~0u, up ? a : b, 8);
    } else if constexpr (N == 2) {
        const bool hi = lane & 16;
        r = (hi ? v[1] : v[0]) + __shfl_xor_sync(~0u, hi ? v[0] : v[1], 16);
        r += __shfl_xor_sync(~0u, r, 8);
    } else {
        static_assert(N == 1, "1, 2 or 4 sums");
        r = v[0] + __shfl_xor_sync(~0u, v[0], 16);
        r += __shfl_xor_sync(~0u, r, 8);
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) r += __shfl_xor_sync(~0u, r, o);
    return r;
}

template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], ReduceMem& m, int cluster, int& phase)
{
    if constexpr (TEAM > 0) {
#pragma unroll
        for (int o = TEAM / 2; o; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(~0u, v[k], o);
    } else {
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
        const float r = warp_sums(v, lane);
        if (lane % (32 / N) == 0) reinterpret_cast<float*>(&m.warp[phase][lane * N / 32][0])[warp] = r;
        __syncthreads();
        const int fours = (int)(blockDim.x + 127) / 128;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float4 q = m.warp[phase][k][0];
            for (int w = 1; w < fours; ++w) {
                const float4 t = m.warp[phase][k][w];
                q = make_float4(q.x + t.x, q.y + t.y, q.z + t.z, q.w + t.w);
            }
            v[k] = (q.x + q.y) + (q.z + q.w);
        }
        if (cluster > 1) {
            cg::cluster_group cl = cg::this_cluster();
            const unsigned rank = cl.block_rank();
            if ((int)threadIdx.x < cluster) {
                float* to = cl.map_shared_rank(reinterpret_cast<float*>(&m.cta[phase][0]), threadIdx.x);
#pragma unroll
                for (int k = 0; k < N; ++k) to[4 * k + rank] = v[k];
            }
            cl.sync();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float4 q = m.cta[phase][k];
                v[k] = (q.x + q.y) + (q.z + q.w);
            }
        }
        phase ^= 1;
    }
}

// g becomes act(g), and da its derivative where it is asked for.
template <bool DERIVATIVE>
__device__ __forceinline__ void activation(int act, float (&g)[8], float (&da)[8])
{
    if (act == MRU_ACT_SILU) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float c = logit(g[e]);
            if constexpr (DERIVATIVE) {
                float s, ns;
                sigmoid2(c, s, ns);
                da[e] = s * fmaf(c, ns, 1.0f);
                g[e] = c * s;
            } else {
                g[e] = c * sigmoid(c);
            }
        }
    } else if (act == MRU_ACT_SIGMOID) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float s, ns;
            sigmoid2(g[e], s, ns);
            if constexpr (DERIVATIVE) da[e] = s * ns;
            g[e] = s;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            g[e] = 1.0f;
            if constexpr (DERIVATIVE) da[e] = 0.0f;
        }
    }
}

// v - mean (layer norm) and 1 / sqrt(mean square + eps) of a row.
template <int TEAM, bool VEC>
__device__ __forceinline__ float normalise(const BArgs& p, const Cols<VEC>& c, float (&v)[8], ReduceMem& m, int& phase)
{
    const float inv_d = 1.0f / (float)p.D;
    float s[1];
    if (p.norm == MRU_NORM_LAYER) {
        s[0] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[e];
        team_sum<TEAM>(s, m, p.cluster, phase);
        const float mean = s[0] * inv_d;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c.ok(e) ? v[e] - mean : 0.0f;
    }
    s[0] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = fmaf(v[e], v[e], s[0]);
    team_sum<TEAM>(s, m, p.cluster, phase);
    return inv_root(fmaf(s[0], inv_d, p.eps));
}

// The thread's place: team (row within the CTA's rows) and columns.
template <int TEAM, bool VEC>
__device__ __forceinline__ Cols<VEC> place(const BArgs& p, int64_t& row, int64_t& step)
{
    Cols<VEC> c;
    c.D = p.D;
    if constexpr (TEAM > 0) {
        const int teams = blockDim.x / TEAM;
        row = (int64_t)blockIdx.x * teams + threadIdx.x / TEAM;
        step = (int64_t)gridDim.x * teams;
        c.step = TEAM;
        c.c0 = (threadIdx.x % TEAM) * (VEC ? 8 : 1);
    } else {
        row = blockIdx.x / p.cluster;
        step = gridDim.x / p.cluster;
        c.step = blockDim.x;
        c.c0 = (blockIdx.x % p.cluster) * blockDim.x * 8 + threadIdx.x * (VEC ? 8 : 1);
    }
    return c;
}

template <typename T, int TEAM, bool VEC, bool PACK>
__global__ void __launch_bounds__(TEAM ? 256 : 512, TEAM ? 4 : 2) k_block(BArgs p)
{
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ ReduceMem mem;
    constexpr int STAGES = stages_of<T>(3, 0), PLANE = plane_bytes<T>();
    int phase = 0;
    if (TEAM == 0) clear(mem);
    int64_t row, step;
    const Cols<VEC> c = place<TEAM, VEC>(p, row, step);
    // teams of a warp take their shuffles together: rows past the end go through the motions
    const int64_t last = TEAM ? (p.rows + step - 1) / step * step : p.rows;
    const bool gate = p.has_y && p.act != MRU_ACT_NONE;
    auto slot = [&](int k) { return Slot<T>{ring + (size_t)k * 3 * PLANE * blockDim.x}; };
    auto fill = [&](int64_t to, int k) {
        if (to < p.rows && c.c0 < p.D) {
            const Slot<T> s = slot(k);
            s.fill(0, (const T*)p.r + to * p.D + c.c0);
            if (p.has_y) s.fill(PLANE, (const T*)p.y + to * p.ldy + c.c0);
            if (gate) s.fill(2 * PLANE, (const T*)p.g + to * p.ldg + c.c0);
        }
        copy_commit();
    };
    int stage = 0;
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < STAGES - 1; ++k) fill(row + k * step, k);
    }
    for (; row < last; row += step) {
        const bool live = row < p.rows;
        const int64_t rr = live ? row : 0;
        Cols<VEC> cc = c;
        if (!live) cc.D = 0;
        const Cols<VEC> pc = live ? c : Cols<VEC>{c.D, c.step, c.D};   // the 8-bit copies' columns
        float r[8], y[8], g[8];
        if constexpr (VEC) {
            fill(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
            copy_wait<STAGES - 1>();
            if (cc.c0 < cc.D) {
                const Slot<T> s = slot(stage);
                s.read(0, r);
                if (p.has_y) s.read(PLANE, y);
                if (gate) s.read(2 * PLANE, g);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = y[e] = g[e] = 0.0f;
            }
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        } else {
            load8<T, VEC>((const T*)p.r + rr * p.D, cc, r);
            if (p.has_y) load8<T, VEC>((const T*)p.y + rr * p.ldy, cc, y);
            if (gate) load8<T, VEC>((const T*)p.g + rr * p.ldg, cc, g);
        }
        if (p.has_y) {
            float w[8], b[8];
            if constexpr (PACK && VEC) {
                store_packed(p.y8, rr, pc, y);
                if (gate) store_packed(p.g8, rr, pc, g);
            }
            const float rstd = normalise<TEAM, VEC>(p, cc, y, mem, phase);
            load_param<VEC>(p.prm.w_y, 1.0f, cc, w);
            load_param<VEC>(p.prm.b_y, 0.0f, cc, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e] * rstd, w[e], b[e]);
            load_param<VEC>(p.prm.s, 1.0f, cc, w);
            activation<false>(p.act, g, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                r[e] = fmaf(p.rs * w[e] * g[e], y[e], r[e]);
                if (!VEC && !cc.ok(e)) r[e] = 0.0f;
            }
            if (VEC && cc.c0 >= cc.D) {
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = 0.0f;
            }
            store8<T, VEC>((T*)p.r_out + rr * p.D, cc, r);
        }
        if constexpr (PACK && VEC) {
            float h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = to_f32(from_f32<T>(r[e]));
            store_packed(p.r8, rr, pc, h);
        }
        if (p.has_z) {
            float w[8], b[8];
            const float rstd = normalise<TEAM, VEC>(p, cc, r, mem, phase);
            load_param<VEC>(p.prm.w_z, 1.0f, cc, w);
            load_param<VEC>(p.prm.b_z, 0.0f, cc, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = fmaf(r[e] * rstd, w[e], b[e]);
            store8<T, VEC>((T*)p.z + rr * p.D, cc, r);
        }
    }
    if (TEAM == 0 && p.cluster > 1) cg::this_cluster().sync();     // peers may still write this CTA's sums
}

// A CTA's (cluster's) sums over its rows of one parameter's gradient.
template <int TEAM, bool VEC>
__device__ __forceinline__ void write_part(const BArgs& p, const Cols<VEC>& c, int which, const float (&acc)[8],
                                           float* sums)
{
    float* to = p.part + ((int64_t)which * p.parts + blockIdx.x / p.cluster) * p.D;
    if constexpr (TEAM > 0) {
        const int teams = blockDim.x / TEAM, cols = TEAM * 8;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sums[(threadIdx.x / TEAM) * cols + (threadIdx.x % TEAM) * 8 + e] = acc[e];
        __syncthreads();
        for (int k = threadIdx.x; k < cols && k < p.D; k += blockDim.x) {
            float s = 0.0f;
            for (int t = 0; t < teams; ++t) s += sums[t * cols + k];
            to[k] = s;
        }
    } else {
        store8<float, false>(to, Cols<false>{c.c0, VEC ? 1 : c.step, p.D}, acc);
    }
}

// FULL: layer norm, or sums for the biases.
template <typename T, int TEAM, bool VEC, bool PACKED, bool FULL>
__global__ void __launch_bounds__(TEAM ? 256 : 512) k_block_bwd(BArgs p)
{
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ ReduceMem mem;
    __shared__ float sums[TEAM ? 2048 : 1];
    constexpr int STAGES = stages_of<T>(PACKED ? 2 : 5, PACKED ? 3 : 0), PLANE = plane_bytes<T>();
    constexpr int STAGE = stage_bytes<T>(PACKED ? 2 : 5, PACKED ? 3 : 0);
    constexpr int R8 = 2 * PLANE, NEXT = PACKED ? 12 : PLANE;      // planes: dr', dz, r', y, g
    int phase = 0;
    if (TEAM == 0) clear(mem);
    int64_t row, step;
    const Cols<VEC> c = place<TEAM, VEC>(p, row, step);
    const int64_t last = TEAM ? (p.rows + step - 1) / step * step : p.rows;
    const float inv_d = 1.0f / (float)p.D;
    const bool layer = FULL && p.norm == MRU_NORM_LAYER;
    float dwy[8], ds[8], dwz[8], dby[8], dbz[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dwy[e] = ds[e] = dwz[e] = dby[e] = dbz[e] = 0.0f;
    const bool gate = p.has_y && p.act != MRU_ACT_NONE;
    auto slot = [&](int k) { return Slot<T>{ring + (size_t)k * STAGE * blockDim.x}; };
    auto fill = [&](int64_t to, int k) {
        if (to < p.rows && c.c0 < p.D) {
            const Slot<T> s = slot(k);
            if (p.dro) s.fill(0, (const T*)p.dro + to * p.D + c.c0);
            if (p.has_z) s.fill(PLANE, (const T*)p.dz + to * p.D + c.c0);
            if constexpr (PACKED) {
                if (p.has_z) s.fill8(R8, p.r8, to, c.c0, p.D);
                if (p.has_y) s.fill8(R8 + NEXT, p.y8, to, c.c0, p.D);
                if (gate) s.fill8(R8 + 2 * NEXT, p.g8, to, c.c0, p.D);
            } else {
                if (p.has_z) s.fill(R8, (const T*)p.r + to * p.D + c.c0);
                if (p.has_y) s.fill(R8 + NEXT, (const T*)p.y + to * p.ldy + c.c0);
                if (gate) s.fill(R8 + 2 * NEXT, (const T*)p.g + to * p.ldg + c.c0);
            }
        }
        copy_commit();
    };
    int stage = 0;
    if constexpr (VEC) {
#pragma unroll
        for (int k = 0; k < STAGES - 1; ++k) fill(row + k * step, k);
    }
    for (; row < last; row += step) {
        const bool live = row < p.rows;
        const int64_t rr = live ? row : 0;
        Cols<VEC> cc = c;
        if (!live) cc.D = 0;
        float e_[8], u[8], r[8], y[8], g[8], dz[8], w[8];
        if constexpr (VEC) {
            fill(row + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
            copy_wait<STAGES - 1>();
            const Slot<T> s = slot(stage);
            if (p.dro) s.read(0, e_);
            if (p.has_z) {
                s.read(PLANE, dz);
                if constexpr (PACKED) s.read8(R8, r);
                else s.read(R8, r);
            }
            if (p.has_y) {
                if constexpr (PACKED) s.read8(R8 + NEXT, y);
                else s.read(R8 + NEXT, y);
            }
            if (gate) {
                if constexpr (PACKED) s.read8(R8 + 2 * NEXT, g);
                else s.read(R8 + 2 * NEXT, g);
            }
            if (cc.c0 >= cc.D) {
#pragma unroll
                for (int e = 0; e < 8; ++e) e_[e] = dz[e] = r[e] = y[e] = g[e] = 0.0f;
            }
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        } else {
            if (p.dro) load8<T, VEC>((const T*)p.dro + rr * p.D, cc, e_);
            if (p.has_z) {
                load8<T, VEC>((const T*)p.dz + rr * p.D, cc, dz);
                if constexpr (PACKED) load_packed(p.r8, rr, cc, r);
                else load8<T, VEC>((const T*)p.r + rr * p.D, cc, r);
            }
            if (p.has_y) {
                if constexpr (PACKED) load_packed(p.y8, rr, cc, y);
                else load8<T, VEC>((const T*)p.y + rr * p.ldy, cc, y);
            }
            if (gate) {
                if constexpr (PACKED) load_packed(p.g8, rr, cc, g);
                else load8<T, VEC>((const T*)p.g + rr * p.ldg, cc, g);
            }
        }
        load_param<VEC>(p.prm.w_z, 1.0f, cc, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!p.dro) e_[e] = 0.0f;
            if (!p.has_z) dz[e] = r[e] = 0.0f;
            if (!p.has_y) y[e] = 0.0f;
            u[e] = dz[e] * w[e];
        }
        if (layer) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0] += r[e];
                s[1] += y[e];
            }
            team_sum<TEAM>(s, mem, p.cluster, phase);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                r[e] = cc.ok(e) ? r[e] - s[0] * inv_d : 0.0f;
                y[e] = cc.ok(e) ? y[e] - s[1] * inv_d : 0.0f;
            }
        }
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};             // r r, u r, y y, u
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[0] = fmaf(r[e], r[e], s[0]);
            s[1] = fmaf(u[e], r[e], s[1]);
            s[2] = fmaf(y[e], y[e], s[2]);
            if (FULL) s[3] += u[e];
        }
        team_sum<TEAM>(s, mem, p.cluster, phase);
        // a row past the end adds nothing to the sums, whatever eps is
        const float rstd_y = live ? inv_root(fmaf(s[2], inv_d, p.eps)) : 0.0f;
        if (p.has_z) {
            const float rstd = live ? inv_root(fmaf(s[0], inv_d, p.eps)) : 0.0f;
            const float c1 = rstd * s[1] * inv_d, c0 = layer ? s[3] * inv_d : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float hat = r[e] * rstd;
                e_[e] = fmaf(rstd, u[e] - c0 - hat * c1, e_[e]);
                dwz[e] = fmaf(dz[e], hat, dwz[e]);
                if (FULL) dbz[e] += dz[e];
            }
        }
        if (p.dr) store8<T, VEC>((T*)p.dr + rr * p.D, cc, e_);
        if (!p.has_y) continue;
        float b[8], sc[8];
        load_param<VEC>(p.prm.w_y, 1.0f, cc, w);
        load_param<VEC>(p.prm.b_y, 0.0f, cc, b);
        load_param<VEC>(p.prm.s, 1.0f, cc, sc);
        float t[2] = {0.0f, 0.0f};                         // q yhat, q
        activation<true>(p.act, g, dz);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float hat = y[e] * rstd_y, n = fmaf(hat, w[e], b[e]);
            const float re = !FULL || cc.ok(e) ? p.rs * e_[e] : 0.0f, dm = re * sc[e], dn = dm * g[e];
            ds[e] = fmaf(re * g[e], n, ds[e]);
            dwy[e] = fmaf(dn, hat, dwy[e]);
            if (FULL) dby[e] += dn;
            g[e] = dm * n * dz[e];
            u[e] = dn * w[e];
            y[e] = hat;
            t[0] = fmaf(u[e], hat, t[0]);
            if (FULL) t[1] += u[e];
        }
        if (p.dg) store8<T, VEC>((T*)p.dg + rr * p.lddg, cc, g);
        team_sum<TEAM>(t, mem, p.cluster, phase);
        const float t1 = t[0] * inv_d, t0 = layer ? t[1] * inv_d : 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = rstd_y * (u[e] - t0 - y[e] * t1);
        store8<T, VEC>((T*)p.dy + rr * p.lddy, cc, u);
    }
    write_part<TEAM, VEC>(p, c, 0, dwy, sums);
    write_part<TEAM, VEC>(p, c, 1, ds, sums);
    write_part<TEAM, VEC>(p, c, 2, dwz, sums);
    if (FULL) {
        write_part<TEAM, VEC>(p, c, 3, dby, sums);
        write_part<TEAM, VEC>(p, c, 4, dbz, sums);
    }
    if (TEAM == 0 && p.cluster > 1) cg::this_cluster().sync();
}

struct GradOut {
    float* to[5];
};

// The parameters' gradients from the CTAs' sums, in the order of the CTAs.
__global__ void __launch_bounds__(256) k_block_grads(int32_t D, int32_t parts, const float* __restrict__ part, GradOut out)
{
    float* to = out.to[blockIdx.y];
    if (!to) return;
    __shared__ float s[8][33];
    const int d = blockIdx.x * 32 + threadIdx.x % 32, k = threadIdx.x / 32;
    const float* from = part + (int64_t)blockIdx.y * parts * D;
    float v = 0.0f;
    if (d < D)
        for (int p = k; p < parts; p += 8) v += from[(int64_t)p * D + d];
    s[k][threadIdx.x % 32] = v;
    __syncthreads();
    if (k == 0 && d < D) {
        for (int j = 1; j < 8; ++j) v += s[j][threadIdx.x % 32];
        to[d] = v;
    }
}

// ------------------------------------------------------------------ host ---

struct Shape {
    int team, cluster, threads;
    unsigned grid;
};

// Teams: 8 lanes up to 64 columns, a warp up to 256, else a CTA of as many
// warps as the columns need and beyond 4096 columns a cluster of 2 or 4.
Shape shape_of(int64_t rows, int64_t D, bool vec, int per_sm)
{
    Shape s;
    s.team = !vec ? 0 : D <= 64 ? 8 : D <= 256 ? 32 : 0;
    s.cluster = 1;
    int64_t units;
    if (s.team) {
        s.threads = 256;
        units = div_up(rows, 256 / s.team);
    } else {
        while (s.cluster * kCtaCols < D) s.cluster *= 2;
        s.threads = (int)(div_up(div_up(D, 8 * s.cluster), 32) * 32);
        units = rows;
    }
    int64_t most = (int64_t)148 * per_sm;
    if (!s.team) most = most * (512 / s.threads > 4 ? 4 : 512 / s.threads) / s.cluster;
    s.grid = (unsigned)((units < most ? units : most) * s.cluster);
    return s;
}

// `per_thread`: bytes of shared memory of a thread's rows on their way.
template <typename K>
cudaError_t launch(K kernel, const Shape& sh, const BArgs& p, int per_thread, cudaStream_t s)
{
    const size_t smem = (size_t)per_thread * (size_t)sh.threads;
    if (smem > 32 * 1024) {                                        // with the static part, beyond the default 48 KB
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(sh.grid);
    cfg.blockDim = dim3((unsigned)sh.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)sh.cluster;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = sh.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t run_forward(const Shape& sh, const BArgs& p, bool vec, bool pack, cudaStream_t s)
{
    constexpr int ring = stages_of<T>(3, 0) * stage_bytes<T>(3, 0);
    if (!vec) return launch(k_block<T, 0, false, false>, sh, p, 0, s);
    if (sh.team == 8) return launch(pack ? k_block<T, 8, true, true> : k_block<T, 8, true, false>, sh, p, ring, s);
    if (sh.team == 32) return launch(pack ? k_block<T, 32, true, true> : k_block<T, 32, true, false>, sh, p, ring, s);
    return launch(pack ? k_block<T, 0, true, true> : k_block<T, 0, true, false>, sh, p, ring, s);
}

template <typename T, bool PACKED, bool FULL>
cudaError_t run_backward(const Shape& sh, const BArgs& p, bool vec, cudaStream_t s)
{
    constexpr int plain = PACKED ? 2 : 5, held = PACKED ? 3 : 0;
    constexpr int ring = stages_of<T>(plain, held) * stage_bytes<T>(plain, held);
    if (!vec) return launch(k_block_bwd<T, 0, false, PACKED, FULL>, sh, p, 0, s);
    if (sh.team == 8) return launch(k_block_bwd<T, 8, true, PACKED, FULL>, sh, p, ring, s);
    if (sh.team == 32) return launch(k_block_bwd<T, 32, true, PACKED, FULL>, sh, p, ring, s);
    return launch(k_block_bwd<T, 0, true, PACKED, FULL>, sh, p, ring, s);
}

constexpr int kBwdPerSm = 1, kFwdPerSm = 2;

mru_status check_problem(const mru_block_problem* p)
{
    if (!p || p->rows < 0 || p->D < 0 ) return MRU_ERR_INVALID_ARG;
    for (int64_t ld : {p->ld_y, p->ld_g, p->ld_dy, p->ld_dg})
        if (ld && ld < p->D) return MRU_ERR_INVALID_ARG;
    if (p->dtype != MRU_F32 && p->dtype != MRU_BF16) return MRU_ERR_INVALID_ARG;
    if (p->norm != MRU_NORM_RMS && p->norm != MRU_NORM_LAYER) return MRU_ERR_INVALID_ARG;
    if (p->act < MRU_ACT_NONE || p->act > MRU_ACT_SIGMOID || !(p->eps >= 0.0f)) return MRU_ERR_INVALID_ARG;
    if (p->D > kMaxD) return MRU_ERR_UNSUPPORTED;
    const int64_t most = (int64_t)1 << 50;
    for (int64_t ld : {p->D, p->ld_y, p->ld_g, p->ld_dy, p->ld_dg})
        if (!product_within(p->rows, ld, most)) return MRU_ERR_UNSUPPORTED;
    return MRU_OK;
}

BArgs make_args(const mru_block_problem& p, const mru_block_params* prm)
{
    BArgs a;
    memset(&a, 0, sizeof a);
    a.rows = p.rows; a.D = (int32_t)p.D;
    a.ldy = p.ld_y ? p.ld_y : p.D;
    a.ldg = p.ld_g ? p.ld_g : p.D;
    a.lddy = p.ld_dy ? p.ld_dy : p.D;
    a.lddg = p.ld_dg ? p.ld_dg : p.D;
    a.norm = p.norm; a.act = p.act; a.eps = p.eps; a.rs = p.res_scale;
    if (prm) a.prm = *prm;
    return a;
}

bool params_aligned(const mru_block_params& q, size_t a)
{
    return aligned(q.w_y, a) && aligned(q.b_y, a) && aligned(q.s, a) && aligned(q.w_z, a) && aligned(q.b_z, a);
}

bool packed_given(const mru_packed8& v, bool want) { return (v.q != nullptr) == want && (!want || (v.scale && aligned(v.scale, 4))); }

}  // namespace
}  // namespace mru

using namespace mru;

extern "C" {

mru_status mru_block_norm(const mru_block_problem* p, const mru_block_params* prm, const void* r, const void* y,
                          const void* g, void* r_out, void* z, const mru_block_saved* saved, void* stream)
{
    const mru_status st = check_problem(p);
    if (st != MRU_OK) return st;
    const size_t es = elem_size(p->dtype);
    const bool any = p->rows > 0 && p->D > 0, has_y = y != nullptr, has_z = z != nullptr;
    BArgs a = make_args(*p, prm);
    if (!any) return MRU_OK;
    const bool gate = has_y && p->act != MRU_ACT_NONE;
    if (!r || has_y != (r_out != nullptr) || (!has_y && !has_z) || gate != (g != nullptr)) return MRU_ERR_INVALID_ARG;
    for (const void* v : {r, y, g, (const void*)r_out, (const void*)z})
        if (!aligned(v, es)) return MRU_ERR_INVALID_ARG;
    if (!params_aligned(a.prm, 4)) return MRU_ERR_INVALID_ARG;
    if (saved && (!packed_given(saved->r, true) || !packed_given(saved->y, has_y) || !packed_given(saved->g, gate)))
        return MRU_ERR_INVALID_ARG;
    const size_t D = (size_t)p->D, all = (size_t)p->rows * D;
    Buffers b;
    b.in(r, all * es);
    b.in_rows(y, p->rows, D * es, (size_t)a.ldy * es);
    b.in_rows(g, p->rows, D * es, (size_t)a.ldg * es);
    for (const float* v : {a.prm.w_y, a.prm.b_y, a.prm.s, a.prm.w_z, a.prm.b_z}) b.in(v, D * 4);
    b.out(r_out, all * es);
    b.out(z, all * es);
    if (saved)
        for (const mru_packed8* v : {&saved->r, &saved->y, &saved->g})
            if (v->q) {
                b.out(v->q, all);
                b.out(v->scale, (size_t)(p->rows * div_up(p->D, 64)) * 4);
            }
    if (b.clash()) return MRU_ERR_INVALID_ARG;
    // 8 columns to an access: whole runs, everything 16-byte aligned
    bool vec = p->D % 8 == 0 && (a.ldy * es) % 16 == 0 && (a.ldg * es) % 16 == 0 && params_aligned(a.prm, 16);
    for (const void* v : {r, y, g, (const void*)r_out, (const void*)z}) vec = vec && aligned(v, 16);
    if (saved) vec = vec && aligned(saved->r.q, 8) && aligned(saved->y.q, 8) && aligned(saved->g.q, 8);
    a.r = r; a.y = y; a.g = g; a.r_out = r_out; a.z = z;
    a.has_y = has_y; a.has_z = has_z;
    if (saved) { a.r8 = saved->r; a.y8 = saved->y; a.g8 = saved->g; }
    const Shape sh = shape_of(p->rows, p->D, vec, kFwdPerSm);
    a.cluster = sh.cluster;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = p->dtype == MRU_BF16 ? run_forward<__nv_bfloat16>(sh, a, vec, saved != nullptr, s)
                                         : run_forward<float>(sh, a, vec, saved != nullptr, s);
    if (e == cudaSuccess && saved && !vec) {
        e = launch_pack8(p->rows, p->D, p->D, p->dtype, has_y ? r_out : r, saved->r, s);
        if (e == cudaSuccess && has_y) e = launch_pack8(p->rows, p->D, a.ldy, p->dtype, y, saved->y, s);
        if (e == cudaSuccess && gate) e = launch_pack8(p->rows, p->D, a.ldg, p->dtype, g, saved->g, s);
    }
    return cuda_status(e);
}

size_t mru_block_backward_workspace_size(const mru_block_problem* p)
{
    if (check_problem(p) != MRU_OK) return 0;
    if (p->rows == 0 || p->D == 0) return 256;
    // the larger of the two column layouts
    size_t parts = 0;
    for (bool vec : {false, true}) {
        const Shape sh = shape_of(p->rows, p->D, vec, kBwdPerSm);
        const size_t n = sh.grid / (size_t)sh.cluster;
        if (n > parts) parts = n;
    }
    return 256 + align256(5 * parts * (size_t)p->D * 4);
}

mru_status mru_block_norm_backward(const mru_block_problem* p, const mru_block_params* prm, const void* r_out,
                                   const void* y, const void* g, const mru_block_saved* saved, const void* dr_out,
                                   const void* dz, void* dr, void* dy, void* dg, const mru_block_grads* grads,
                                   void* ws, size_t ws_bytes, void* stream)
{
    const mru_status st = check_problem(p);
    if (st != MRU_OK) return st;
    if (!ws || !aligned(ws, 16)) return MRU_ERR_INVALID_ARG;
    const size_t es = elem_size(p->dtype);
    const bool any = p->rows > 0 && p->D > 0;
    BArgs a = make_args(*p, prm);
    mru_block_grads gr;
    memset(&gr, 0, sizeof gr);
    if (grads) gr = *grads;
    const size_t D = (size_t)p->D, all = (size_t)p->rows * D;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    for (const float* v : {gr.dw_y, gr.db_y, gr.ds, gr.dw_z, gr.db_z})
        if (!aligned(v, 4)) return MRU_ERR_INVALID_ARG;
    if (!any) {
        if (ws_bytes < mru_block_backward_workspace_size(p)) return MRU_ERR_WORKSPACE;
        cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(uint32_t), s);
        for (float* v : {gr.dw_y, gr.db_y, gr.ds, gr.dw_z, gr.db_z})
            if (e == cudaSuccess && v && D > 0) e = cudaMemsetAsync(v, 0, D * 4, s);
        return cuda_status(e);
    }
    const bool has_z = dz != nullptr, has_y = saved ? saved->y.q != nullptr : y != nullptr;
    const bool gate = has_y && p->act != MRU_ACT_NONE;
    if ((!dr_out && !dz) || (has_y && !dy) || gate != (dg != nullptr) || (!has_y && dy)) return MRU_ERR_INVALID_ARG;
    if (!has_y && !has_z) return MRU_ERR_INVALID_ARG;
    if (saved) {
        if (!packed_given(saved->r, true) || !packed_given(saved->y, has_y) || !packed_given(saved->g, gate))
            return MRU_ERR_INVALID_ARG;
        r_out = y = g = nullptr;
    } else {
        if ((has_z && !r_out) || gate != (g != nullptr)) return MRU_ERR_INVALID_ARG;
        if (!has_z) r_out = nullptr;
    }
    for (const void* v : {r_out, y, g, dr_out, dz, (const void*)dr, (const void*)dy, (const void*)dg})
        if (!aligned(v, es)) return MRU_ERR_INVALID_ARG;
    if (!params_aligned(a.prm, 4)) return MRU_ERR_INVALID_ARG;
    Buffers b;
    b.in(r_out, all * es);
    b.in_rows(y, p->rows, D * es, (size_t)a.ldy * es);
    b.in_rows(g, p->rows, D * es, (size_t)a.ldg * es);
    if (saved)
        for (const mru_packed8* v : {&saved->r, &saved->y, &saved->g})
            if (v->q) {
                b.in(v->q, all);
                b.in(v->scale, (size_t)(p->rows * div_up(p->D, 64)) * 4);
            }
    for (const float* v : {a.prm.w_y, a.prm.b_y, a.prm.s, a.prm.w_z}) b.in(v, D * 4);
    b.in(dr_out, all * es);
    b.in(dz, all * es);
    b.out(dr, all * es);
    b.out_rows(dy, p->rows, D * es, (size_t)a.lddy * es);
    b.out_rows(dg, p->rows, D * es, (size_t)a.lddg * es);
    for (float* v : {gr.dw_y, gr.db_y, gr.ds, gr.dw_z, gr.db_z}) b.out(v, D * 4);
    b.out(ws, ws_bytes);
    if (b.clash()) return MRU_ERR_INVALID_ARG;
    if (ws_bytes < mru_block_backward_workspace_size(p)) return MRU_ERR_WORKSPACE;
    bool vec = p->D % 8 == 0 && (a.ldy * es) % 16 == 0 && (a.ldg * es) % 16 == 0 &&
               (a.lddy * es) % 16 == 0 && (a.lddg * es) % 16 == 0 && params_aligned(a.prm, 16);
    for (const void* v : {r_out, y, g, dr_out, dz, (const void*)dr, (const void*)dy, (const void*)dg})
        vec = vec && aligned(v, 16);
    if (saved) vec = vec && aligned(saved->r.q, 8) && aligned(saved->y.q, 8) && aligned(saved->g.q, 8);
    a.r = r_out; a.y = y; a.g = g;
    if (saved) { a.r8 = saved->r; a.y8 = saved->y; a.g8 = saved->g; }
    a.dro = dr_out; a.dz = dz; a.dr = dr; a.dy = dy; a.dg = dg;
    a.has_y = has_y; a.has_z = has_z;
    a.part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + 256);
    const Shape sh = shape_of(p->rows, p->D, vec, kBwdPerSm);
    a.cluster = sh.cluster;
    a.parts = (int32_t)(sh.grid / (unsigned)sh.cluster);
    cudaError_t e = cudaMemsetAsync(ws, 0, sizeof(uint32_t), s);
    if (e != cudaSuccess) return MRU_ERR_CUDA;
    const bool full = p->norm == MRU_NORM_LAYER || gr.db_y || gr.db_z, packed = saved != nullptr;
    if (p->dtype == MRU_BF16)
        e = packed ? (full ? run_backward<__nv_bfloat16, true, true>(sh, a, vec, s)
                           : run_backward<__nv_bfloat16, true, false>(sh, a, vec, s))
                   : (full ? run_backward<__nv_bfloat16, false, true>(sh, a, vec, s)
                           : run_backward<__nv_bfloat16, false, false>(sh, a, vec, s));
    else
        e = packed ? (full ? run_backward<float, true, true>(sh, a, vec, s)
                           : run_backward<float, true, false>(sh, a, vec, s))
                   : (full ? run_backward<float, false, true>(sh, a, vec, s)
                           : run_backward<float, false, false>(sh, a, vec, s));
    if (e != cudaSuccess) return MRU_ERR_CUDA;
    if (gr.dw_y || gr.db_y || gr.ds || gr.dw_z || gr.db_z) {
        const GradOut out = {{gr.dw_y, gr.ds, gr.dw_z, gr.db_y, gr.db_z}};
        k_block_grads<<<dim3((unsigned)div_up(p->D, 32), 5), 256, 0, s>>>(a.D, a.parts, a.part, out);
        e = cudaGetLastError();
    }
    return cuda_status(e);
}

}  // extern "C"
