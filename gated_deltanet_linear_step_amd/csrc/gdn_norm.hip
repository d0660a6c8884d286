// gdn_norm.hip -- RMS norm of rows with the residual's addition in front and, if
// asked for, an 8-bit output with a scale per row, on gfx950:
//     h = x + residual            (f32; stored rounded as the next residual)
//     y = h (mean h^2 + eps)^(-1/2) weight
//     scale = max |y| / 127,  q = y (127 / max |y|) rounded to nearest even
// HBM bound: each row is read once, and its outputs written once.
//
// row_kernel holds a row in the registers of one workgroup (one wave up to 512
// elements, 16 waves up to 16384), 8 consecutive elements of it to a thread's vector.
// A workgroup takes several rows, with the weights kept in registers -- read again
// for every row they would be more L2 traffic than the 16-bit rows themselves -- and
// the next row's loads in flight while the current one is reduced. Vectors need no
// alignment beyond the element's (the hardware splits them), so odd widths and
// strides take the same path; a width's last hidden % 8 elements go one to a thread.
// loop_kernel takes wider rows (and those of less than 8) in passes over memory, an element to a lane.
// Sums and maxima are f32, in a fixed order: lanes, DPP tree, waves.
// 8192 x 4096 bf16, residual in and out, 16- and 8-bit rows out: 56-58 us, 5.2 TB/s (a large
// copy reaches 5.0). 1537 x 5003 f16: 9.3-9.8 us, 3.1-3.3 TB/s; 64 x 2048: 3.5 us, a launch and
// one round trip to memory. loop_kernel, 2048 x 20480 bf16 with residual and 8-bit rows: 358 us,
// 0.8 TB/s: bound by its single-element loads and their conversions, three times over the row. It is kept
// that simple because the widths of model layers are row_kernel's.

#include "gdn_device.h"
#include "gdn_ops.h"

#include <algorithm>

namespace gdn {
namespace {

// The largest |y| below which a row is stored as zeros with scale 0: 127 / max |y|
// would leave f32's range soon after.
constexpr float kQuantFloor = 0x1p-100f;

// Largest of 64 lanes' words.
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
#define GDN_DPP_MAX(CTRL) x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false))
    GDN_DPP_MAX(0xB1);
    GDN_DPP_MAX(0x4E);
    GDN_DPP_MAX(0x141);
    GDN_DPP_MAX(0x140);
#undef GDN_DPP_MAX
    x = max(x, (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, 0x401F));
    return max(x, (uint32_t)__shfl_xor((int)x, 32, 64));
}

// What the 8-bit output of a row needs from the bits of its largest |y|. As words, the
// absolute values order like themselves, infinity above them and NaN above that.
struct Quant {
    float inv, scale;
};
__device__ __forceinline__ Quant quant_of(uint32_t top_bits)
{
    const float top = __uint_as_float(top_bits);
    if (top_bits >= 0x7f800000u)
        return Quant{0.f, __builtin_nanf("")};
    if (top < kQuantFloor)
        return Quant{0.f, 0.f};
    return Quant{127.f / top, top / 127.f};
}
// (a row without a finite scale is stored as zeros, whatever y is)
__device__ __forceinline__ int quant(float y, Quant q) { return q.inv == 0.f ? 0 : (int)rintf(y * q.inv); }

// Eight consecutive elements, aligned to one.
template <int DT>
struct Vec8 {
    uint32_t w[DT == DT_F32 ? 8 : 4];
};
template <int DT>
__device__ __forceinline__ Vec8<DT> load_vec8(const void *p, int64_t idx)
{
    struct __attribute__((packed, aligned(DT == DT_F32 ? 4 : 2))) Bits {
        Vec8<DT> v;
    };
    return reinterpret_cast<const Bits *>(static_cast<const char *>(p) + idx * (DT == DT_F32 ? 4 : 2))->v;
}
template <int DT>
__device__ __forceinline__ float element(const Vec8<DT> &v, int e)
{
    if constexpr (DT == DT_F32)
        return __uint_as_float(v.w[e]);
    else {
        const uint32_t h = e & 1 ? v.w[e / 2] >> 16 : v.w[e / 2] & 0xffffu;
        return DT == DT_BF16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h);
    }
}
template <int DT>
__device__ __forceinline__ void store_vec8_t(void *p, int64_t idx, const float (&x)[8])
{
    struct __attribute__((packed, aligned(DT == DT_F32 ? 4 : 2))) Bits {
        Vec8<DT> v;
    } b;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (DT == DT_F32)
            b.v.w[e] = __float_as_uint(x[e]);
        else {
            const uint16_t h = DT == DT_BF16 ? __builtin_bit_cast(uint16_t, (__bf16)x[e])
                                             : __builtin_bit_cast(uint16_t, (_Float16)x[e]);
            if (e & 1)
                b.v.w[e / 2] |= (uint32_t)h << 16;
            else
                b.v.w[e / 2] = h;
        }
    }
    *reinterpret_cast<Bits *>(static_cast<char *>(p) + idx * (DT == DT_F32 ? 4 : 2)) = b;
}
__device__ __forceinline__ void store_vec8(void *p, int64_t idx, int dt, const float (&x)[8])
{
    if (dt == DT_F32)
        store_vec8_t<DT_F32>(p, idx, x);
    else if (dt == DT_BF16)
        store_vec8_t<DT_BF16>(p, idx, x);
    else
        store_vec8_t<DT_F16>(p, idx, x);
}

// V vectors of 8 to each of a workgroup's threads, MOST of them or, where that is 256, whole waves up to it: rows of
// 8 up to 8 V elements a thread (and the tail). Loads are never
// conditional -- a thread without a vector loads the last one, and counts it in no sum and no maximum (its owner may
// have stored residual_out over it by then) -- so that all of a row's are in flight together.
template <int DT, int V, int MOST, bool RES>
__global__ __launch_bounds__(MOST) void row_kernel(const NormParams p)
{
    constexpr int WAVES = MOST / 64;
    __shared__ float sums[2][WAVES];
    __shared__ uint32_t tops[2][WAVES];
    const int tid = threadIdx.x, wave = tid >> 6, NT = MOST == 256 ? blockDim.x : MOST;
    // the slots of waves that this row has no use for
    if (MOST == 256 && tid < WAVES && tid >= NT / 64) {
        sums[0][tid] = sums[1][tid] = 0.f;
        tops[0][tid] = tops[1][tid] = 0u;
    }
    const int whole = p.hidden / 8, tail = p.hidden % 8;
    const bool tails = tid < tail;
    const int ti = whole * 8 + tid, tc = min(ti, p.hidden - 1);  // this thread's element of the tail

    Vec8<DT> x[V], r[V];
    uint32_t xt, rt = 0;
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int64_t u = 8 * min(v * NT + tid, whole - 1);
            x[v] = load_vec8<DT>(p.x, row * p.x_stride + u);
            if constexpr (RES)
                r[v] = load_vec8<DT>(p.residual, row * p.residual_stride + u);
        }
        xt = load_raw1<DT>(p.x, row * p.x_stride + tc);
        if constexpr (RES)
            rt = load_raw1<DT>(p.residual, row * p.residual_stride + tc);
    };
    fetch(blockIdx.x);
    Vec8<DT_F32> w[V];
    float wt = p.weight[tc];
#pragma unroll
    for (int v = 0; v < V; ++v)
        w[v] = load_vec8<DT_F32>(p.weight, 8 * min(v * NT + tid, whole - 1));
    wt = tails ? wt : 0.f;

    int par = 0;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
        float h[V][8], ht = raw1_to_f32<DT>(xt);
        if constexpr (RES)
            ht += raw1_to_f32<DT>(rt);
        float ss = tails ? ht * ht : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float sv = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[v][e] = element<DT>(x[v], e);
                if constexpr (RES)
                    h[v][e] += element<DT>(r[v], e);
                sv = fmaf(h[v][e], h[v][e], sv);
            }
            ss += v * NT + tid < whole ? sv : 0.f;
        }
        if (row + gridDim.x < p.rows)
            fetch(row + gridDim.x);
        if (p.residual_out) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v * NT + tid < whole)
                    store_vec8_t<DT>(p.residual_out, row * p.residual_out_stride + 8 * (v * NT + tid), h[v]);
            if (tails)
                store_act(p.residual_out, row * p.residual_out_stride + ti, DT, ht);
        }
        ss = group_sum<64>(ss);
        if constexpr (WAVES > 1) {
            // two slots in turn: a wave writes a slot again only past a barrier that all have reached after
            // reading it
            if ((tid & 63) == 0)
                sums[par][wave] = ss;
            __syncthreads();
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < WAVES; ++i)
                ss += sums[par][i];
        }
        const float rs = 1.f / sqrtf(ss / (float)p.hidden + p.eps);
        uint32_t top = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            uint32_t tv = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[v][e] = h[v][e] * rs * __uint_as_float(w[v].w[e]);
                tv = max(tv, __float_as_uint(h[v][e]) & 0x7fffffffu);
            }
            top = max(top, v * NT + tid < whole ? tv : 0u);
        }
        ht = tails ? ht * rs * wt : 0.f;
        top = max(top, __float_as_uint(ht) & 0x7fffffffu);
        if (p.out) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v * NT + tid < whole)
                    store_vec8(p.out, row * p.out_stride + 8 * (v * NT + tid), p.out_dt, h[v]);
            if (tails)
                store_act(p.out, row * p.out_stride + ti, p.out_dt, ht);
        }
        if (p.out_q) {
            top = wave_max(top);
            if constexpr (WAVES > 1) {
                if ((tid & 63) == 0)
                    tops[par][wave] = top;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < WAVES; ++i)
                    top = max(top, tops[par][i]);
            }
            const Quant q = quant_of(top);
            if (tid == 0)
                p.out_scale[row] = q.scale;
            int8_t *o = p.out_q + row * p.out_q_stride;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v * NT + tid < whole) {
                    struct __attribute__((packed)) Bytes {
                        uint32_t b[2];
                    } b = {{0, 0}};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        b.b[e / 4] |= (uint32_t)(quant(h[v][e], q) & 0xff) << (8 * (e % 4));
                    *reinterpret_cast<Bytes *>(o + 8 * (v * NT + tid)) = b;
                }
            if (tails)
                o[ti] = (int8_t)quant(ht, q);
        }
    }
}

constexpr int kLoopThreads = 1024;

__device__ __forceinline__ float norm_input(const NormParams &p, int64_t row, int i)
{
    float h = load_act(p.x, row * p.x_stride + i, p.dt);
    if (p.residual)
        h += load_act(p.residual, row * p.residual_stride + i, p.dt);
    return h;
}

// Rows of any width, three passes over memory. h is formed again in each: the last pass writes residual_out and
// out, which may be an input's own buffer, element by element after reading it.
__global__ __launch_bounds__(kLoopThreads) void loop_kernel(const NormParams p)
{
    constexpr int WAVES = kLoopThreads / 64;
    __shared__ float sums[WAVES];
    __shared__ uint32_t tops[WAVES];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float ss = 0.f;
        for (int i = threadIdx.x; i < p.hidden; i += kLoopThreads) {
            const float h = norm_input(p, row, i);
            ss = fmaf(h, h, ss);
        }
        ss = group_sum<64>(ss);
        if ((threadIdx.x & 63) == 0)
            sums[threadIdx.x >> 6] = ss;
        __syncthreads();
        ss = 0.f;
        for (int w = 0; w < WAVES; ++w)
            ss += sums[w];
        const float rs = 1.f / sqrtf(ss / (float)p.hidden + p.eps);
        Quant q{0.f, 0.f};
        if (p.out_q) {
            uint32_t top = 0;
            for (int i = threadIdx.x; i < p.hidden; i += kLoopThreads)
                top = max(top, __float_as_uint(norm_input(p, row, i) * rs * p.weight[i]) & 0x7fffffffu);
            top = wave_max(top);
            if ((threadIdx.x & 63) == 0)
                tops[threadIdx.x >> 6] = top;
            __syncthreads();
            for (int w = 0; w < WAVES; ++w)
                top = max(top, tops[w]);
            q = quant_of(top);
            if (threadIdx.x == 0)
                p.out_scale[row] = q.scale;
        }
        for (int i = threadIdx.x; i < p.hidden; i += kLoopThreads) {
            const float h = norm_input(p, row, i);
            if (p.residual_out)
                store_act(p.residual_out, row * p.residual_out_stride + i, p.dt, h);
            const float y = h * rs * p.weight[i];
            if (p.out)
                store_act(p.out, row * p.out_stride + i, p.out_dt, y);
            if (p.out_q)
                p.out_q[row * p.out_q_stride + i] = (int8_t)quant(y, q);
        }
        __syncthreads();  // the sums and tops are read
    }
}

template <int DT, int V, int MOST>
hipError_t launch_rows_t(const NormParams &p, hipStream_t s)
{
    // Up to four waves, as many as the row fills (4096 x 2560 bf16 13.9 us, 15.3 with four; 4096 x 1000 5.5, 6.6);
    // more are eight or sixteen (five to seven share the four SIMDs unevenly: 4096 x 5120 32.4 us with eight, 35.0 with
    // five).
    const int NT = MOST > 256 ? MOST : 64 * ((p.hidden / 8 + 64 * V - 1) / (64 * V));
    // as many workgroups as the card holds at 2048 threads a CU; each takes every grid-th row
    const int grid = std::min(p.rows, 256 * (2048 / NT));
    if (p.residual)
        row_kernel<DT, V, MOST, true><<<grid, NT, 0, s>>>(p);
    else
        row_kernel<DT, V, MOST, false><<<grid, NT, 0, s>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_rows(const NormParams &p, hipStream_t s)
{
    if (p.hidden < 8 * 64 + 8)
        return launch_rows_t<DT, 1, 64>(p, s);
    if (p.hidden < 8 * 256 + 8)
        return launch_rows_t<DT, 1, 256>(p, s);
    if (p.hidden < 16 * 256 + 8)
        return launch_rows_t<DT, 2, 256>(p, s);
    if (p.hidden < 16 * 512 + 8)
        return launch_rows_t<DT, 2, 512>(p, s);
    return launch_rows_t<DT, 2, 1024>(p, s);
}

constexpr int kRowMost = 16 * 1024 + 8;  // four vectors a thread would spill

}  // namespace

hipError_t launch_norm(const NormParams &p, hipStream_t s)
{
    if (p.hidden < 8 || p.hidden >= kRowMost) {
        loop_kernel<<<std::min(p.rows, 512), kLoopThreads, 0, s>>>(p);  // two a CU; each takes every grid-th row
        return hipGetLastError();
    }
    switch (p.dt) {
    case DT_F32: return launch_rows<DT_F32>(p, s);
    case DT_F16: return launch_rows<DT_F16>(p, s);
    default: return launch_rows<DT_BF16>(p, s);
    }
}

}  // namespace gdn
