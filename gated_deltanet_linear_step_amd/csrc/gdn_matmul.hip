// gdn_matmul.hip -- product of 8-bit integers with a scale per row of each side:
//     out[m][n] = (sum_k a[m][k] w[n][k]) a_scale[m] w_scale[n]
// on v_mfma_i32_16x16x64_i8 (gfx950). The sums are 32-bit integers, exact for
// K <= 131071 (|a w| <= 2^14); the scales multiply them in f32 and the result is
// rounded once. Both operands are row-major with k innermost, so a lane's 16
// consecutive bytes are 16 k-values of one row for either operand, and any one
// order of k serves both.

#include "gdn_device.h"
#include "gdn_kernels.h"

namespace gdn {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Simple form: a workgroup of 4 waves owns 64 x 64 outputs, a wave 32 x 32 as
// 2 x 2 tiles, operands straight from global memory. Rows past M or N read the
// last row and store nothing.
__global__ __launch_bounds__(256) void matmul_simple_kernel(const MatmulParams p)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
    const int nt = (p.N + 63) / 64;
    const int m0 = blockIdx.x / nt * 64 + (wave >> 1) * 32, n0 = blockIdx.x % nt * 64 + (wave & 1) * 32;
    i32x4 acc[2][2] = {};
    const int8_t *ap[2], *wp[2];
    for (int i = 0; i < 2; ++i) {
        ap[i] = p.a + (int64_t)min(m0 + 16 * i + li, p.M - 1) * p.a_stride;
        wp[i] = p.w + (int64_t)min(n0 + 16 * i + li, p.N - 1) * p.w_stride;
    }
    for (int k0 = 0; k0 < p.K; k0 += 64) {
        const int k = k0 + 16 * lg;
        i32x4 av[2] = {}, wv[2] = {};
        if (k < p.K)
            for (int i = 0; i < 2; ++i) {
                av[i] = *reinterpret_cast<const i32x4 *>(ap[i] + k);
                wv[i] = *reinterpret_cast<const i32x4 *>(wp[i] + k);
            }
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av[i], wv[j], acc[i][j], 0, 0, 0);
    }
    for (int i = 0; i < 2; ++i)
        for (int r = 0; r < 4; ++r) {
            const int m = m0 + 16 * i + 4 * lg + r;
            if (m >= p.M)
                continue;
            const float sa = p.a_scale[m];
            for (int j = 0; j < 2; ++j) {
                const int n = n0 + 16 * j + li;
                if (n < p.N)
                    store_act(p.out, (int64_t)m * p.out_stride + n, p.out_dt,
                              (float)acc[i][j][r] * sa * p.w_scale[n]);
            }
        }
}

}  // namespace

hipError_t launch_matmul(const MatmulParams &p, hipStream_t s)
{
    matmul_simple_kernel<<<((p.N + 63) / 64) * ((p.M + 63) / 64), 256, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace gdn
