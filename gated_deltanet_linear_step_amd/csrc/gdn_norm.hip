// gdn_norm.hip -- RMS norm of rows with the residual's addition in front and, if
// asked for, an 8-bit output with a scale per row, on gfx950:
//     h = x + residual            (f32; stored rounded as the next residual)
//     y = h (mean h^2 + eps)^(-1/2) weight
//     scale = max |y| / 127,  q = y (127 / max |y|) rounded to nearest even
// HBM bound: each row is read once, and its outputs written once. One workgroup per
// row; sums in f32.

#include "gdn_device.h"
#include "gdn_kernels.h"

namespace gdn {
namespace {

constexpr int kNormThreads = 256;

// The largest |y| below which a row is stored as zeros with scale 0: 127 / max |y|
// would leave f32's range soon after.
constexpr float kQuantFloor = 0x1p-100f;

__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1)
        x = fmaxf(x, __shfl_xor(x, m, 64));
    return x;
}

__device__ __forceinline__ float norm_input(const NormParams &p, int64_t row, int i)
{
    float h = load_act(p.x, row * p.x_stride + i, p.dt);
    if (p.residual)
        h += load_act(p.residual, row * p.residual_stride + i, p.dt);
    return h;
}

__global__ __launch_bounds__(kNormThreads) void norm_rows_kernel(const NormParams p)
{
    __shared__ float part[3][kNormThreads / 64];
    const int64_t row = blockIdx.x;
    float ss = 0.f;
    for (int i = threadIdx.x; i < p.hidden; i += kNormThreads) {
        const float h = norm_input(p, row, i);
        ss = fmaf(h, h, ss);
    }
    ss = group_sum<64>(ss);
    if ((threadIdx.x & 63) == 0)
        part[0][threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = 0.f;
    for (int w = 0; w < kNormThreads / 64; ++w)
        ss += part[0][w];
    const float rs = 1.f / sqrtf(ss / (float)p.hidden + p.eps);
    float top = 0.f, bad = 0.f;
    for (int i = threadIdx.x; i < p.hidden; i += kNormThreads) {
        const float y = norm_input(p, row, i) * rs * p.weight[i];
        top = fmaxf(top, fabsf(y));
        bad = __builtin_isfinite(y) ? bad : 1.f;
    }
    top = wave_max(top);
    bad = wave_max(bad);
    if ((threadIdx.x & 63) == 0) {
        part[1][threadIdx.x >> 6] = top;
        part[2][threadIdx.x >> 6] = bad;
    }
    __syncthreads();
    for (int w = 0; w < kNormThreads / 64; ++w) {
        top = fmaxf(top, part[1][w]);
        bad = fmaxf(bad, part[2][w]);
    }
    const bool zero = !(top >= kQuantFloor) || bad != 0.f;
    const float inv = zero ? 0.f : 127.f / top;
    if (p.out_scale && threadIdx.x == 0)
        p.out_scale[row] = bad != 0.f ? __builtin_nanf("") : (zero ? 0.f : top / 127.f);
    for (int i = threadIdx.x; i < p.hidden; i += kNormThreads) {
        const float h = norm_input(p, row, i);
        if (p.residual_out)
            store_act(p.residual_out, row * p.residual_out_stride + i, p.dt, h);
        const float y = h * rs * p.weight[i];
        if (p.out)
            store_act(p.out, row * p.out_stride + i, p.out_dt, y);
        if (p.out_q)
            p.out_q[row * p.out_q_stride + i] = (int8_t)(zero ? 0.f : rintf(y * inv));
    }
}

}  // namespace

hipError_t launch_norm(const NormParams &p, hipStream_t s)
{
    norm_rows_kernel<<<p.rows, kNormThreads, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace gdn
