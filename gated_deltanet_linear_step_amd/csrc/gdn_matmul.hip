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
//    128 bytes of k (a stage) at a time, double buffered, with two or three more stages on
//    their way in registers. Bound by the LDS: a stage of 256 x 256 moves 192 KB out of
//    it and 64 KB in for 2048 clocks of products. 4096^3: 67-69 us, 1980-2050 TOPS (a
//    library's int8 product reaches 2078 at 8192^3); 8192 x 8192 x 2048: 148-160 us, where storing the
//    128 MB of bf16 outputs adds about 20 us that no product covers.
//  * skinny_kernel -- a few rows: bound by the weights, which stream through once
//    (1 x 8192 x 2048: 4.7 us).

#include "gdn_device.h"
#include "gdn_ops.h"

namespace gdn {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

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

// WGM x WGN waves, each (BM / WGM) x (BN / WGN) outputs as 32 x 32 tiles; KG groups of them, each every KG-th stage
// of k, whose sums are added at the end. D stages (of every group) are on their way in registers.
template <int BM, int BN, int WGM, int WGN, int WAVES, int D, int KG>
__global__ __launch_bounds__(64 * WGM * WGN * KG, WAVES) void tile_kernel(const MatmulParams p)
{
    constexpr int THREADS = 64 * WGM * WGN * KG, TM = BM / WGM / 32, TN = BN / WGN / 32;
    constexpr int KB = BK * KG, STEP = THREADS / (8 * KG), UA = BM / STEP, UW = BN / STEP;
    constexpr int PLANE = (BM + BN) * BK, STAGE = PLANE * KG;
    // epilogue: a wave's 32 rows of its BN / WGN columns, in f32
    constexpr int EP = BN / WGN * 4 + 16, EPI = WGM * WGN * 32 * EP;
    __shared__ __align__(64) unsigned char lds[2 * STAGE > EPI ? 2 * STAGE : EPI];
    // the tile's scales of a and w, fetched behind the first stages: after the products a round trip to memory for
    // them would stand alone
    __shared__ __align__(16) float scales[BM + BN];
    static_assert(BM + BN <= THREADS && 64 % (BN / WGN / 8) == 0, "a scale for a thread, whole rows for a wave's stores");

    const int tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), kg = wave / (WGM * WGN);
    const int wm = wave % WGM, wn = wave / WGM % WGN;

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
    const int row = tid / (8 * KG), block = tid % (8 * KG);
    // Loads and writes of one stage, in BK / 32 parts that go between the products of a stage: the L1 delivers 64
    // bytes a clock, so that a wave issuing a whole stage's loads at once stands still until most have left.
    constexpr int U = UA + UW, KS = BK / 32, PART = (U + KS - 1) / KS;
    static_assert(D >= 2, "the stage that goes to the LDS is not the one being fetched");
    i32x4 regs[D][U];
    uint32_t off[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
        off[i] = i < UA ? (row + i * STEP) * as : (row + (i - UA) * STEP) * ws;
    auto fetch = [&](int k0, i32x4 (&r)[U], int part) {
        // behind the last stage nothing is read, but the loads stay, so that the loop has no branch and each
        // wait counts exactly the loads issued since
        const bool in = k0 < p.K;
        const Buffer ba = buffer_of(ab + k0, in ? a_bytes - k0 : 0), bw = buffer_of(wb + k0, in ? w_bytes - k0 : 0);
        // past K an offset past every buffer's end: 0
        const uint32_t c = k0 + 16 * block < p.K ? 16 * block : 0xf0000000u;
#pragma unroll
        for (int i = part * PART; i < U && i < (part + 1) * PART; ++i)
            r[i] = load16(i < UA ? ba : bw, max(off[i] + c, c));
    };
    auto stage = [&](unsigned char *s, const i32x4 (&r)[U], int part) {
#pragma unroll
        for (int i = part * PART; i < U && i < (part + 1) * PART; ++i)
            *reinterpret_cast<i32x4 *>(s + block / 8 * PLANE + (i < UA ? stage_at(row + i * STEP, block % 8)
                                                                       : BM * BK + stage_at(row + (i - UA) * STEP, block % 8))) = r[i];
    };

    i32x16 acc[TN][TM] = {};
    i32x4 f[2][TM + TN];
    auto read = [&](const unsigned char *s, int ks, i32x4 (&f)[TM + TN]) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            f[i] = *reinterpret_cast<const i32x4 *>(s + stage_at(wm * TM * 32 + 32 * i + l32, 2 * ks + half));
#pragma unroll
        for (int j = 0; j < TN; ++j)
            f[TM + j] = *reinterpret_cast<const i32x4 *>(s + BM * BK + stage_at(wn * TN * 32 + 32 * j + l32, 2 * ks + half));
    };
    // One stage: each step's operands are read during the step before it
    auto step = [&](int buf, int d, int k0, bool load, const i32x4 (&next)[U]) {
        const unsigned char *s = lds + buf * STAGE + kg * PLANE;
        read(s, 0, f[0]);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if (ks + 1 < KS)
                read(s, ks + 1, f[(ks + 1) & 1]);
            if (load)
                fetch(k0, regs[d], ks);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f[ks & 1][TM + j], f[ks & 1][i], acc[j][i], 0, 0, 0);
            stage(lds + (buf ^ 1) * STAGE, next, ks);
            __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
    };
    // D stages of k in registers on their way to the LDS, besides the two in it
    const int stages = (p.K + KB - 1) / KB;
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int part = 0; part < KS; ++part)
            fetch(d * KB, regs[d], part);
    const float scale = tid < BM ? p.a_scale[min(m0 + tid, p.M - 1)] : p.w_scale[min(n0 + min(tid - BM, BN - 1), p.N - 1)];
#pragma unroll
    for (int part = 0; part < KS; ++part)
        stage(lds, regs[0], part);
    __syncthreads();
    int buf = 0, k0 = D * KB;
    for (int g = 0; g < stages / D; ++g) {
#pragma unroll
        for (int d = 0; d < D; ++d, k0 += KB) {
            step(buf, d, k0, true, regs[(d + 1) % D]);
            buf ^= 1;
        }
    }
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
        if (d < stages % D) {
            step(buf, d, 0, false, regs[d + 1]);
            buf ^= 1;
        }

    if (tid < BM + BN)
        scales[tid] = scale;
    if constexpr (KG == 1)
        __syncthreads();

    // With KG > 1 the other groups of waves hand their sums over, behind the epilogue's part of the LDS
    if constexpr (KG > 1) {
        constexpr int WAVES1 = WGM * WGN;
        static_assert(TM == 1 && TN == 1 && EPI % 64 == 0 && EPI + (KG - 1) * WAVES1 * 4096 <= 2 * STAGE, "one tile a wave");
        i32x16 *sums = reinterpret_cast<i32x16 *>(lds + EPI) + wave % WAVES1 * 64 + lane;
        if (kg > 0)
            sums[(kg - 1) * WAVES1 * 64] = acc[0][0];
        __syncthreads();
        if (kg > 0)
            return;
#pragma unroll
        for (int g = 0; g < KG - 1; ++g)
            acc[0][0] += sums[g * WAVES1 * 64];
    }

    // Epilogue, 32 rows of m at a time through the wave's own LDS: a lane holds n = 8 g + 4 half + e of row l32
    unsigned char *mine = lds + wave * 32 * EP;
    constexpr int PER = BN / WGN / 8, ROWS = 64 / PER;  // lanes per row of 8 outputs each, rows per pass
    const int er = lane / PER, ec = lane % PER * 8;
    const int nb = n0 + wn * TN * 32, valid = p.N - nb - ec;
    float sw[8];
    __builtin_memcpy(sw, &scales[BM + wn * TN * 32 + ec], sizeof(sw));
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int mb = m0 + (wm * TM + i) * 32;
        const float sa = scales[(wm * TM + i) * 32 + l32];
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

template <int BM, int BN, int WGM, int WGN, int WAVES, int D, int KG = 1>
struct Tiles {
    static constexpr int kRows = BM, kCols = BN, kThreads = 64 * WGM * WGN * KG;
    static hipError_t launch(const MatmulParams &p, unsigned workgroups, hipStream_t s)
    {
        tile_kernel<BM, BN, WGM, WGN, WAVES, D, KG><<<workgroups, kThreads, 0, s>>>(p);
        return hipGetLastError();
    }
};

// ---- a few rows ---------------------------------------------------------------

constexpr int kSkinnyRows = 16, kSkinnyWaves = 8;

// 16 rows by 16 NT columns a workgroup; its waves take 256 bytes of k in turn, straight from global memory (a
// weight is read by one lane, once), and add up their sums through LDS.
template <int NT>
__global__ __launch_bounds__(64 * kSkinnyWaves) void skinny_kernel(const MatmulParams p)
{
    constexpr int STEPS = 4;
    __shared__ i32x4 part[kSkinnyWaves][NT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
    const int n0 = blockIdx.x * 16 * NT;
    const int8_t *wr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
        wr[j] = p.w + (int64_t)min(n0 + 16 * j + li, p.N - 1) * p.w_stride;
    const int8_t *ar = p.a + (int64_t)min(li, p.M - 1) * p.a_stride;
    // the scales of the tile that this wave adds up at the end, fetched with the first operands
    const int n = n0 + 16 * min(wave, NT - 1) + 4 * lg;
    const float sa = p.a_scale[min(li, p.M - 1)];
    float sw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        sw[e] = p.w_scale[min(n + e, p.N - 1)];
    i32x4 acc[NT] = {};
    for (int k0 = wave * 64 * STEPS; k0 < p.K; k0 += kSkinnyWaves * 64 * STEPS) {
        i32x4 fw[STEPS][NT], fa[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + 64 * s + 16 * lg;
            const bool in = k < p.K;
            const int kc = in ? k : 0;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                fw[s][j] = *reinterpret_cast<const i32x4 *>(wr[j] + kc);
            fa[s] = *reinterpret_cast<const i32x4 *>(ar + kc);
            fa[s] = in ? fa[s] : i32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[s][j], fa[s], acc[j], 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
        part[wave][j][lane] = acc[j];
    __syncthreads();
    // wave x adds up tile x: a lane holds columns 4 lg .. + 3 of row li
    if (wave < NT) {
        i32x4 sum = part[0][wave][lane];
#pragma unroll
        for (int w = 1; w < kSkinnyWaves; ++w)
            sum += part[w][wave][lane];
        const int valid = min(p.N - n, 4);
        if (li < p.M && valid > 0) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                y[e] = (float)sum[e] * sa * sw[e];
            store_row<4>(p.out, (int64_t)li * p.out_stride + n, p.out_dt, y, valid);
        }
    }
}

template <int NT>
struct Skinny {
    static constexpr int kRows = kSkinnyRows, kCols = 16 * NT, kThreads = 64 * kSkinnyWaves;
    static hipError_t launch(const MatmulParams &p, unsigned workgroups, hipStream_t s)
    {
        skinny_kernel<NT><<<workgroups, kThreads, 0, s>>>(p);
        return hipGetLastError();
    }
};

constexpr int64_t kMostTiles = 1 << 23;  // a launch holds fewer than 2^32 threads, 512 of them a tile at most

// Microseconds that a CU takes for a stage (BK bytes of k) of its tiles, as measured at K = 4096: `alone` for a
// workgroup by itself, `each` for each of several that share or follow one another on the CU.
double stage_cost(int64_t tiles, double alone, double each)
{
    const int64_t per_cu = (tiles + 255) / 256;
    return per_cu <= 1 ? alone : (double)per_cu * each;
}

// A kernel of the choice: its outputs a workgroup, threads, and cost of a stage.
struct Kernel {
    int rows, cols, threads;
    double alone, each;
    hipError_t (*launch)(const MatmulParams &, unsigned, hipStream_t);
};
template <class T>
constexpr Kernel kernel(double alone = 0, double each = 0)
{
    return Kernel{T::kRows, T::kCols, T::kThreads, alone, each, T::launch};
}
int64_t workgroups(const Kernel &k, int M, int N)
{
    return (((int64_t)M + k.rows - 1) / k.rows) * (((int64_t)N + k.cols - 1) / k.cols);
}

constexpr Kernel kSkinny[] = {kernel<Skinny<1>>(), kernel<Skinny<2>>()};
constexpr Kernel kTiles[] = {kernel<Tiles<256, 256, 2, 4, 2, 2>>(1.42, 1.42), kernel<Tiles<128, 128, 2, 2, 2, 2>>(0.63, 0.66),
                             kernel<Tiles<64, 128, 1, 4, 2, 2>>(0.49, 0.41),  kernel<Tiles<64, 64, 2, 2, 2, 3>>(0.33, 0.28),
                             kernel<Tiles<64, 32, 2, 1, 1, 2, 2>>(0.22, 0.21), kernel<Tiles<32, 32, 1, 1, 1, 2, 4>>(0.15, 0.17)};

const Kernel &choose(int M, int N)
{
    // M x 8192 x 2048, us (skinny, tiles): M = 1 4.8 5.5, 16 5.3 5.7; M x 2048 x 4096: 1 4.3 6.0, 16 5.6 5.9. A second
    // block of 16 rows costs the skinny kernel as much again: 32 6.5 5.9, 7.5 6.1.
    // Two column tiles share each read of a, where that leaves a workgroup for every CU.
    if (M <= kSkinnyRows && workgroups(kSkinny[0], M, N) < kMostTiles)
        return kSkinny[N >= 256 * 32];
    // A larger tile reads each operand from the LDS fewer times, but a stage of it takes a lone workgroup longer:
    // the tile whose slowest CU is done first. The smallest two deal k out to groups of waves besides (2 and 4).
    // M x N x K, us (256 x 256, 128 x 128, 64 x 128, 64 x 64, 64 x 32, 32 x 32):
    //   4096 x 4096 x 4096  67  81  100 121  -  -        100 x 8192 x 2048  26  12  9.0  7.2  8.0  11
    //   2048 x 4096 x 2048  31  24  28  34   -  -         64 x 8192 x 2048  25  12  8.9  7.1  6.0  7.0
    //   1001 x 2050 x 4112  50  23  27  28   29 36       128 x 2048 x 4096  45  19  14   11   8.0  6.4
    //   1001 x 2048 x 4096  46  20  15  18   21 29        64 x 2048 x 4096  43  19  14   11   7.7  6.1
    const Kernel *best = nullptr;
    double least = 0;
    for (const Kernel &k : kTiles) {
        const int64_t tiles = workgroups(k, M, N);
        const double cost = stage_cost(tiles, k.alone, k.each);
        if (!best || (cost < least && tiles < kMostTiles)) {
            best = &k;
            least = cost;
        }
    }
    return *best;
}

}  // namespace

MatmulPlan matmul_plan(int M, int N)
{
    const Kernel &k = choose(M, N);
    return MatmulPlan{(int)workgroups(k, M, N), k.threads};
}

hipError_t launch_matmul(const MatmulParams &p, hipStream_t s)
{
    const Kernel &k = choose(p.M, p.N);
    return k.launch(p, (unsigned)workgroups(k, p.M, p.N), s);
}

}  // namespace gdn
