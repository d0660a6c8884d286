// gdn_matmul.hip -- product of 8-bit integers with a scale per row of each side:
//     out[m][n] = (sum_k a[m][k] w[n][k]) a_scale[m] w_scale[n]
// on the int8 matrix instructions of gfx950. The sums are 32-bit integers, exact for
// K <= 131071 (|a w| <= 2^14); the scales multiply them in f32 and the result is
// rounded once. Both operands are row-major with k innermost, so a lane's 16
// consecutive bytes are 16 k-values of one row for either operand, and any one
// order of k serves both. The matrix instruction takes w as its rows and a as its
// columns: a lane then holds four consecutive n of one m and stores them together.
//
// Two kernels:
//  * tile_kernel -- M above kSkinnyRows: BM x BN outputs a workgroup through LDS,
//    128 bytes of k at a time, double buffered.
//  * skinny_kernel -- a few rows: bound by the weights, which stream through once.

#include "gdn_device.h"
#include "gdn_kernels.h"

namespace gdn {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// A buffer of `bytes` from a scalar base: loads past its end give 0.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const int8_t *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, bytes, 0x00020000);
}

__device__ __forceinline__ i32x4 load16(Buffer b, uint32_t off)
{
    return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
}

// N consecutive outputs of which the first `valid` exist, aligned to one element.
template <int N>
__device__ __forceinline__ void store_row(void *out, int64_t at, int dt, const float (&x)[N], int valid)
{
    if (valid < N) {
        for (int i = 0; i < valid; ++i)
            store_act(out, at + i, dt, x[i]);
        return;
    }
    if (dt == DT_F32) {
        struct __attribute__((packed, aligned(4))) Words {
            float v[N];
        } w;
#pragma unroll
        for (int i = 0; i < N; ++i)
            w.v[i] = x[i];
        *reinterpret_cast<Words *>(static_cast<float *>(out) + at) = w;
    } else {
        struct __attribute__((packed, aligned(2))) Words {
            uint16_t v[N];
        } w;
#pragma unroll
        for (int i = 0; i < N; ++i)
            w.v[i] = dt == DT_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)x[i]) : __builtin_bit_cast(uint16_t, (_Float16)x[i]);
        *reinterpret_cast<Words *>(static_cast<uint16_t *>(out) + at) = w;
    }
}

// ---- tiles --------------------------------------------------------------------

constexpr int BK = 128;  // bytes of k per stage: an LDS row, 8 blocks of 16

// LDS stage: rows of BK bytes, their 16-byte blocks swizzled by row so that the 16
// rows one read serves at a time (pitch 128 bytes: half the banks) use every bank.
__device__ __forceinline__ int stage_at(int row, int block) { return row * BK + 16 * (block ^ (row & 7)); }

// WGM x WGN waves, each (BM / WGM) x (BN / WGN) outputs as 32 x 32 tiles.
template <int BM, int BN, int WGM, int WGN, int WAVES>
__global__ __launch_bounds__(64 * WGM * WGN, WAVES) void tile_kernel(const MatmulParams p)
{
    constexpr int THREADS = 64 * WGM * WGN, TM = BM / WGM / 32, TN = BN / WGN / 32;
    constexpr int UA = BM * 8 / THREADS, UW = BN * 8 / THREADS, STEP = THREADS / 8;
    constexpr int STAGE = (BM + BN) * BK;
    // epilogue: a wave's 32 rows of its BN / WGN columns, in f32
    constexpr int EP = BN / WGN * 4 + 16, EPI = WGM * WGN * 32 * EP;
    __shared__ __align__(16) unsigned char lds[2 * STAGE > EPI ? 2 * STAGE : EPI];

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave % WGM, wn = wave / WGM;

    // Workgroups go to the 8 XCDs in turn: give each XCD (with an L2 of its own) a run of
    // neighbouring tiles, 8 tiles of m deep.
    const int nm = (p.M + BM - 1) / BM, nn = (p.N + BN - 1) / BN, tiles = nm * nn;
    const int xcd = blockIdx.x % 8, q = tiles / 8, rem = tiles % 8;
    const int at = xcd * q + min(xcd, rem) + blockIdx.x / 8;
    constexpr int DEEP = 8;
    const int group = at / (DEEP * nn), in_group = at % (DEEP * nn), deep = min(nm - group * DEEP, DEEP);
    const int m0 = (group * DEEP + in_group % deep) * BM, n0 = in_group / deep * BN;

    const uint32_t as = (uint32_t)p.a_stride, ws = (uint32_t)p.w_stride;
    const int8_t *ab = p.a + (int64_t)m0 * p.a_stride, *wb = p.w + (int64_t)n0 * p.w_stride;
    const uint32_t a_bytes = (uint32_t)(min(p.M - m0, BM) - 1) * as + p.K;
    const uint32_t w_bytes = (uint32_t)(min(p.N - n0, BN) - 1) * ws + p.K;
    const int row = tid / 8, block = tid % 8;
    i32x4 ra[UA], rw[UW];
    auto fetch = [&](int k0) {
        const Buffer ba = buffer_of(ab + k0, a_bytes - k0), bw = buffer_of(wb + k0, w_bytes - k0);
        // past K an offset past every buffer's end: 0
        const uint32_t c = k0 + 16 * block < p.K ? 16 * block : 0xf0000000u;
#pragma unroll
        for (int i = 0; i < UA; ++i)
            ra[i] = load16(ba, max((row + i * STEP) * as + c, c));
#pragma unroll
        for (int i = 0; i < UW; ++i)
            rw[i] = load16(bw, max((row + i * STEP) * ws + c, c));
    };
    auto stage = [&](unsigned char *s) {
#pragma unroll
        for (int i = 0; i < UA; ++i)
            *reinterpret_cast<i32x4 *>(s + stage_at(row + i * STEP, block)) = ra[i];
#pragma unroll
        for (int i = 0; i < UW; ++i)
            *reinterpret_cast<i32x4 *>(s + BM * BK + stage_at(row + i * STEP, block)) = rw[i];
    };

    i32x16 acc[TN][TM] = {};
    fetch(0);
    stage(lds);
    __syncthreads();
    for (int k0 = 0, buf = 0; k0 < p.K; k0 += BK, buf ^= 1) {
        const bool more = k0 + BK < p.K;
        if (more)
            fetch(k0 + BK);
        const unsigned char *s = lds + buf * STAGE;
#pragma unroll
        for (int ks = 0; ks < BK / 32; ++ks) {
            i32x4 fa[TM], fw[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i)
                fa[i] = *reinterpret_cast<const i32x4 *>(s + stage_at(wm * TM * 32 + 32 * i + l32, 2 * ks + half));
#pragma unroll
            for (int j = 0; j < TN; ++j)
                fw[j] = *reinterpret_cast<const i32x4 *>(s + BM * BK + stage_at(wn * TN * 32 + 32 * j + l32, 2 * ks + half));
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[j], fa[i], acc[j][i], 0, 0, 0);
        }
        if (more)
            stage(lds + (buf ^ 1) * STAGE);
        __syncthreads();
    }

    // Epilogue, 32 rows of m at a time through the wave's own LDS: a lane holds n = 8 g + 4 half + e of row l32
    unsigned char *mine = lds + wave * 32 * EP;
    constexpr int PER = BN / WGN / 8, ROWS = 64 / PER;  // lanes per row of 8 outputs each, rows per pass
    const int er = lane / PER, ec = lane % PER * 8;
    const int nb = n0 + wn * TN * 32, valid = p.N - nb - ec;
    float sw[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        sw[e] = e < valid ? p.w_scale[nb + ec + e] : 0.f;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int mb = m0 + (wm * TM + i) * 32;
        const float sa = mb + l32 < p.M ? p.a_scale[mb + l32] : 0.f;
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float4 v;
                v.x = (float)acc[j][i][4 * g] * sa;
                v.y = (float)acc[j][i][4 * g + 1] * sa;
                v.z = (float)acc[j][i][4 * g + 2] * sa;
                v.w = (float)acc[j][i][4 * g + 3] * sa;
                *reinterpret_cast<float4 *>(mine + l32 * EP + 4 * (32 * j + 8 * g + 4 * half)) = v;
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int r = 0; r < 32; r += ROWS) {
            const float4 a = *reinterpret_cast<const float4 *>(mine + (r + er) * EP + 4 * ec);
            const float4 b = *reinterpret_cast<const float4 *>(mine + (r + er) * EP + 4 * ec + 16);
            const float x[8] = {a.x * sw[0], a.y * sw[1], a.z * sw[2], a.w * sw[3],
                                b.x * sw[4], b.y * sw[5], b.z * sw[6], b.w * sw[7]};
            const int m = mb + r + er;
            if (m < p.M && valid > 0)
                store_row<8>(p.out, (int64_t)m * p.out_stride + nb + ec, p.out_dt, x, min(valid, 8));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

template <int BM, int BN, int WGM, int WGN, int WAVES>
hipError_t launch_tiles(const MatmulParams &p, hipStream_t s)
{
    const int64_t tiles = (int64_t)((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN);
    tile_kernel<BM, BN, WGM, WGN, WAVES><<<(unsigned)tiles, 64 * WGM * WGN, 0, s>>>(p);
    return hipGetLastError();
}

// ---- a few rows ---------------------------------------------------------------

constexpr int kSkinnyRows = 64, kSkinnyWaves = 8;

// 16 MT rows by 16 NT columns a workgroup; its waves take 256 bytes of k in turn, straight from global memory (a
// weight is read by one lane, once), and add up their sums through LDS.
template <int MT, int NT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(const MatmulParams p)
{
    constexpr int STEPS = 4;
    __shared__ i32x4 part[kSkinnyWaves][MT * NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16 * NT;
    const int8_t *wr[NT], *ar[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        wr[j] = p.w + (int64_t)min(n0 + 16 * j + li, p.N - 1) * p.w_stride;
#pragma unroll
    for (int i = 0; i < MT; ++i)
        ar[i] = p.a + (int64_t)min(16 * i + li, p.M - 1) * p.a_stride;
    i32x4 acc[MT][NT] = {};
    for (int k0 = wave * 64 * STEPS; k0 < p.K; k0 += kSkinnyWaves * 64 * STEPS) {
        i32x4 fw[STEPS][NT], fa[STEPS][MT];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + 64 * s + 16 * lg;
            const bool in = k < p.K;
            const int kc = in ? k : 0;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fw[s][j] = *reinterpret_cast<const i32x4 *>(wr[j] + kc);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                fa[s][i] = *reinterpret_cast<const i32x4 *>(ar[i] + kc);
                fa[s][i] = in ? fa[s][i] : i32x4{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[s][j], fa[s][i], acc[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            part[wave][i * NT + j][lane] = acc[i][j];
    __syncthreads();
    // wave x adds up tile x: a lane holds columns 4 lg .. + 3 of row li
    for (int x = wave; x < MT * NT; x += kSkinnyWaves) {
        i32x4 sum = part[0][x][lane];
#pragma unroll
        for (int w = 1; w < kSkinnyWaves; ++w)
            sum += part[w][x][lane];
        const int m = 16 * (x / NT) + li, n = n0 + 16 * (x % NT) + 4 * lg, valid = min(p.N - n, 4);
        if (m < p.M && valid > 0) {
            const float sa = p.a_scale[m];
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = (float)sum[e] * sa * p.w_scale[n + min(e, valid - 1)];
            store_row<4>(p.out, (int64_t)m * p.out_stride + n, p.out_dt, y, valid);
        }
    }
}

template <int MT>
hipError_t launch_skinny(const MatmulParams &p, hipStream_t s)
{
    // two column tiles share each read of a, where that leaves a workgroup for every CU
    if (p.N >= 256 * 32)
        skinny_kernel<MT, 2><<<(p.N + 31) / 32, 64 * kSkinnyWaves, 0, s>>>(p);
    else
        skinny_kernel<MT, 1><<<(p.N + 15) / 16, 64 * kSkinnyWaves, 0, s>>>(p);
    return hipGetLastError();
}

int64_t tiles_of(const MatmulParams &p, int bm, int bn)
{
    return (int64_t)((p.M + bm - 1) / bm) * ((p.N + bn - 1) / bn);
}

}  // namespace

hipError_t launch_matmul(const MatmulParams &p, hipStream_t s)
{
    if (p.M <= 16)
        return launch_skinny<1>(p, s);
    if (p.M <= 32)
        return launch_skinny<2>(p, s);
    if (p.M <= kSkinnyRows)
        return launch_skinny<4>(p, s);
    if (tiles_of(p, 256, 256) >= 200)
        return launch_tiles<256, 256, 2, 4, 2>(p, s);
    if (tiles_of(p, 128, 128) >= 300)
        return launch_tiles<128, 128, 2, 2, 2>(p, s);
    return launch_tiles<64, 128, 1, 4, 2>(p, s);
}

}  // namespace gdn
