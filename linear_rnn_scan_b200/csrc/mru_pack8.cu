// mru_pack8.cu -- activations to and from 8 bits with a scale per run of 64
// channels of a row.
#include "mru_ops.cuh"

namespace mru {
namespace {

using namespace ops;

// A warp per run: lanes hold channels lane and lane + 32.
template <typename T>
__global__ void __launch_bounds__(256) k_pack8(int64_t rows, int64_t D, int64_t ld, const T* __restrict__ x,
                                               int8_t* __restrict__ q, float* __restrict__ scale)
{
    const int lane = threadIdx.x & 31;
    const int64_t runs = (D + 63) / 64, nw = (int64_t)gridDim.x * (blockDim.x / 32);
    for (int64_t w = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32; w < rows * runs; w += nw) {
        const int64_t row = w / runs, g = w - row * runs;
        const int64_t d0 = g * 64 + lane, d1 = d0 + 32;
        const float v0 = d0 < D ? to_f32(x[row * ld + d0]) : 0.0f;
        const float v1 = d1 < D ? to_f32(x[row * ld + d1]) : 0.0f;
        const uint32_t m = __reduce_max_sync(~0u, max(mag_bits(v0), mag_bits(v1)));
        float inv, sc;
        pack8_factors(__uint_as_float(m), inv, sc);
        if (d0 < D) q[row * D + d0] = (int8_t)pack8_q(v0, inv);
        if (d1 < D) q[row * D + d1] = (int8_t)pack8_q(v1, inv);
        if (lane == 0) scale[w] = sc;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) k_unpack8(int64_t rows, int64_t D, int64_t ld, const int8_t* __restrict__ q,
                                                 const float* __restrict__ scale, T* __restrict__ x)
{
    const int64_t runs = (D + 63) / 64, n = rows * D, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += step) {
        const int64_t row = e / D, d = e - row * D;
        x[row * ld + d] = from_f32<T>((float)q[e] * scale[row * runs + d / 64]);
    }
}

unsigned grid_for(int64_t blocks) { return (unsigned)(blocks < 148 * 16 ? blocks : 148 * 16); }

mru_status check(int64_t rows, int64_t D, int64_t& ld, int32_t dtype, const void* x, const mru_packed8* h, bool packs)
{
    if (rows < 0 || D < 0 || (dtype != MRU_F32 && dtype != MRU_BF16) || !h) return MRU_ERR_INVALID_ARG;
    if (ld == 0) ld = D;
    if (ld < D) return MRU_ERR_INVALID_ARG;
    if (!product_within(rows, ld, (int64_t)1 << 58)) return MRU_ERR_UNSUPPORTED;
    if (rows == 0 || D == 0) return MRU_OK;
    const size_t es = elem_size(dtype);
    if (!x || !h->q || !h->scale || !aligned(x, es) || !aligned(h->scale, 4)) return MRU_ERR_INVALID_ARG;
    Buffers b;
    b.add(x, rows, (size_t)D * es, (size_t)ld * es, !packs);
    b.add(h->q, 1, (size_t)(rows * D), (size_t)(rows * D), packs);
    b.add(h->scale, 1, (size_t)(rows * div_up(D, 64)) * 4, (size_t)(rows * div_up(D, 64)) * 4, packs);
    return b.clash() ? MRU_ERR_INVALID_ARG : MRU_OK;
}

}  // namespace

cudaError_t launch_pack8(int64_t rows, int64_t D, int64_t ld, int32_t dtype, const void* x, const mru_packed8& out,
                         cudaStream_t s)
{
    const unsigned grid = grid_for(div_up(rows * div_up(D, 64), 8));
    if (dtype == MRU_BF16)
        k_pack8<<<grid, 256, 0, s>>>(rows, D, ld, (const __nv_bfloat16*)x, out.q, out.scale);
    else
        k_pack8<<<grid, 256, 0, s>>>(rows, D, ld, (const float*)x, out.q, out.scale);
    return cudaGetLastError();
}

}  // namespace mru

using namespace mru;

extern "C" {

mru_status mru_pack8(int64_t rows, int64_t D, int64_t ld, int32_t dtype, const void* x, const mru_packed8* out,
                     void* stream)
{
    const mru_status st = check(rows, D, ld, dtype, x, out, true);
    if (st != MRU_OK || rows == 0 || D == 0) return st;
    return ops::cuda_status(launch_pack8(rows, D, ld, dtype, x, *out, reinterpret_cast<cudaStream_t>(stream)));
}

mru_status mru_unpack8(int64_t rows, int64_t D, int64_t ld, int32_t dtype, const mru_packed8* in, void* x,
                       void* stream)
{
    const mru_status st = check(rows, D, ld, dtype, x, in, false);
    if (st != MRU_OK || rows == 0 || D == 0) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = grid_for(ops::div_up(rows * D, 256));
    if (dtype == MRU_BF16)
        k_unpack8<<<grid, 256, 0, s>>>(rows, D, ld, in->q, in->scale, (__nv_bfloat16*)x);
    else
        k_unpack8<<<grid, 256, 0, s>>>(rows, D, ld, in->q, in->scale, (float*)x);
    return ops::cuda_status(cudaGetLastError());
}

}  // extern "C"
