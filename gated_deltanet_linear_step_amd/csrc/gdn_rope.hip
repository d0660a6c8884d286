// gdn_rope.hip -- rotary positions on gfx950: a pair (a, b) of a head at position p, with
// the pair's frequency w, becomes (a c - b s, b c + a s), c = m cos(p w), s = m sin(p w).
//
// A workgroup turns one token: its rotary_dim / 2 angles are formed once, in 64 bits (at
// position 10^6 an f32 angle is off by up to 0.03), reduced there to an eighth of a turn, and
// shared by every head through LDS as f32 cosines and sines. Then q and k are read once
// and written once, k and v where the cache's pages are; heads' other elements are copied
// on the way. Bound by bytes for prompts, by latency for a decode step: 8192 tokens, 32 + 8 heads of 128 onto pages 39 us
// (5.1 TB/s, the rate of a large copy); 64 tokens 4.4 us.

#include "gdn_device.h"
#include "gdn_attn.h"

#include <type_traits>

namespace gdn {
namespace {

constexpr int kThreads = 256, kMostPairs = 512;

// c, s = m cos, m sin of the angle p w.
__device__ __forceinline__ float2 turn_of(int p, double w, float m)
{
    const double turns = (double)p * w * 0.15915494309189533577;  // 1 / (2 pi)
    const double quarters = rint(4.0 * turns);
    // half turns of what is left: at most 1/4, where f32 resolves 2^-27
    const float rest = (float)(2.0 * (turns - 0.25 * quarters));
    // quarters mod 4, also past 32 bits
    const int n = (int)(quarters - 4.0 * floor(0.25 * quarters));
    float s, c;
    sincospif(rest, &s, &c);
    const float x = n & 1 ? s : c, y = n & 1 ? c : s;
    return make_float2(m * (n == 1 || n == 2 ? -x : x), m * (n >= 2 ? -y : y));
}

// N elements of 16 or 32 bits, as their bits
template <int DT, int N>
struct Run {
    using Bits = std::conditional_t<DT == DT_F32, uint32_t, uint16_t>;
    typedef Bits Vec __attribute__((ext_vector_type(N)));
    Vec w;
    __device__ __forceinline__ void load(const void *p, int64_t at)
    {
        w = *reinterpret_cast<const Vec *>(static_cast<const Bits *>(p) + at);
    }
    __device__ __forceinline__ void store(void *p, int64_t at) const
    {
        *reinterpret_cast<Vec *>(static_cast<Bits *>(p) + at) = w;
    }
    __device__ __forceinline__ float get(int i) const { return raw1_to_f32<DT>(w[i]); }
    __device__ __forceinline__ void set(int i, float x)
    {
        if constexpr (DT == DT_F32)
            w[i] = __float_as_uint(x);
        else if constexpr (DT == DT_BF16)
            w[i] = __builtin_bit_cast(uint16_t, (__bf16)x);
        else
            w[i] = __builtin_bit_cast(uint16_t, (_Float16)x);
    }
};

// V elements of either half of a pair run at a time: whole 16 bytes where sizes, strides and pointers allow it, else one.
template <int DT, int V, int LAYOUT>
__global__ __launch_bounds__(kThreads) void rope_kernel(const RopeParams p)
{
    __shared__ float2 turns[kMostPairs];
    const int t = blockIdx.x, half = p.rot / 2;
    const int pos = p.positions[t];
    for (int i = threadIdx.x; i < half; i += kThreads)
        turns[i] = turn_of(pos, p.w[i], p.magnitude);
    int64_t slot = -1;
    if (p.k_pages) {
        slot = p.slots[t];
        if (slot >= p.num_slots)
            slot = -1;
    }
    __syncthreads();

    const int per_head = (p.D + 2 * V - 1) / (2 * V);
    const int heads = (p.q ? p.Hq : 0) + (p.k ? p.Hkv : 0) + (p.v ? p.Hkv : 0);
    for (int u = threadIdx.x; u < heads * per_head; u += kThreads) {
        int h = u / per_head;
        const int e = (u - h * per_head) * 2 * V;  // first element
        const void *from;
        void *to;
        int64_t in, out;
        bool turn = e < p.rot;
        const bool is_q = p.q && h < p.Hq;
        h -= !is_q && p.q ? p.Hq : 0;
        if (is_q) {
            from = p.q, to = p.q_out;
            in = t * p.q_stride + (int64_t)h * p.D;
            out = t * p.q_out_stride + (int64_t)h * p.D;
        } else {
            const bool is_k = h < p.Hkv;
            h -= is_k ? 0 : p.Hkv;
            turn = turn && is_k;
            from = is_k ? p.k : p.v;
            in = t * (is_k ? p.k_stride : p.v_stride) + (int64_t)h * p.D;
            if (p.k_pages) {
                if (slot < 0)
                    continue;
                to = is_k ? p.k_pages : p.v_pages;
                const int64_t size = (int64_t)1 << p.page_shift;
                out = (slot >> p.page_shift) * p.page_stride + (h * size + (slot & (size - 1))) * p.D;
            } else {
                to = p.k_out;
                out = t * p.k_out_stride + (int64_t)h * p.D;
            }
        }
        // a run's two parts: the pairs' first and second elements, or just neighbours
        const int first = turn && LAYOUT == 0 ? e / 2 : e, second = turn && LAYOUT == 0 ? e / 2 + half : e + V;
        const bool both = V > 1 || second < p.D;
        Run<DT, V> a, b;
        a.load(from, in + first);
        b.load(from, in + (both ? second : first));
        if (turn) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // interleaved: pairs lie side by side within a part, V > 1, or across the two
                const int j = LAYOUT == 0 ? i : i / 2;
                if (LAYOUT == 0 || V == 1) {
                    const float2 r = turns[e / 2 + j];
                    const float x = a.get(i), y = b.get(i);
                    a.set(i, x * r.x - y * r.y);
                    b.set(i, y * r.x + x * r.y);
                } else if (i % 2 == 0) {
                    const float2 r = turns[e / 2 + j], r2 = turns[e / 2 + V / 2 + j];
                    const float x = a.get(i), y = a.get(i + 1), x2 = b.get(i), y2 = b.get(i + 1);
                    a.set(i, x * r.x - y * r.y);
                    a.set(i + 1, y * r.x + x * r.y);
                    b.set(i, x2 * r2.x - y2 * r2.y);
                    b.set(i + 1, y2 * r2.x + x2 * r2.y);
                }
            }
        }
        a.store(to, out + first);
        if (both)
            b.store(to, out + second);
    }
}

template <int DT, int V>
hipError_t launch(const RopeParams &p, hipStream_t s)
{
    if (p.layout == 0)
        rope_kernel<DT, V, 0><<<p.tokens, kThreads, 0, s>>>(p);
    else
        rope_kernel<DT, V, 1><<<p.tokens, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(const RopeParams &p, hipStream_t s)
{
    constexpr int V = DT == DT_F32 ? 4 : 8, B = DT == DT_F32 ? 4 : 2;
    bool wide = p.rot % (2 * V) == 0 && p.D % (2 * V) == 0;
    for (const void *x : {p.q, p.k, p.v, (const void *)p.q_out, (const void *)p.k_out, (const void *)p.k_pages, (const void *)p.v_pages})
        wide = wide && reinterpret_cast<uintptr_t>(x) % (V * B) == 0;
    for (int64_t x : {p.q ? p.q_stride : 0, p.k ? p.k_stride : 0, p.v ? p.v_stride : 0, p.q ? p.q_out_stride : 0,
                      p.k && !p.k_pages ? p.k_out_stride : 0, p.k_pages ? p.page_stride : 0})
        wide = wide && x % V == 0;
    return wide ? launch<DT, V>(p, s) : launch<DT, 1>(p, s);
}

}  // namespace

hipError_t launch_rope(const RopeParams &p, hipStream_t s)
{
    return p.dt == DT_F32 ? launch_dt<DT_F32>(p, s) : p.dt == DT_F16 ? launch_dt<DT_F16>(p, s) : launch_dt<DT_BF16>(p, s);
}

}  // namespace gdn
