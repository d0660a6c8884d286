// gdn_attn_decode.h -- softmax attention of a few queries of each sequence against its pages on gfx950 (instantiated per
// dtype by gdn_attn_bf16.hip and gdn_attn_f16.hip).
//
// A workgroup takes a run of one sequence's keys for one key head; the query heads that read it and the
// tokens of the step are its up to 16 NR rows. Bound by the bytes of the keys and values, each read
// once: 16 rows use the matrix instructions at a few percent.
//
//  * A wave walks every WAVES-th 32 keys of the run by itself, with a running maximum and sum of its own; nothing waits for
//    another wave before the end, where the waves' results are joined through the LDS.
//  * K and V of 32 keys go from memory straight to the wave's LDS, the next K while V is multiplied and the next V while K is:
//    one buffer of each is enough, no copy needs a register, and every wait counts exactly the copies behind it.
//  * The pages of the whole run are looked up at once, a 16-key group a lane.
//  * S^T = K Q^T (v_mfma_f32_16x16x32): a lane holds one row's scores; as they lie, the exponentials of two 16-key tiles are the
//    operand of O^T += V^T P^T, whose V^T comes from transposing LDS reads. Blocks of 16 bytes are permuted within
//    a row by the address that a lane copies from, so that reads of 16 rows fall into different banks (V's transposing ones of
//    128 wide heads still conflict, in 57 % of the LDS's active clocks; the kernel waits for memory meanwhile).
//  * P is rounded to the 16 bits of V as in the prompts' kernel.
// 64 sequences of 128 to 8192 keys, 32 heads over 8 of 128, bf16: 200 us and 5 to join the runs, 5.4 TB/s (a large copy
// reaches 5.1, the last-level cache holds part of the keys); one of 32768 keys, 16 heads over 2 of 256: 16 and 5 us.
#pragma once

#include "gdn_attn_prefill.h"

namespace gdn {
namespace attn {

template <int D>
struct DecodeGeo {
    static constexpr int KEYS = 32, NB = D / 8, PITCH = 2 * D;
    static constexpr int HALF = KEYS * PITCH, STAGE = 2 * HALF;         // K, then V
    static constexpr int WAVES = 4;                                     // 8 to 32 KB each
    static constexpr int COPIES = NB / 4;                               // of 16 bytes a lane: 16 keys of K or of V
    static_assert(KEYS * WAVES == kDecodeRound && 2 * kDecodeRounds <= 64, "64 lanes hold the pages of a run");
    // Where block b of a V row lies: the blocks 2 b, 2 b + 1 of 8 rows cover all banks
    __device__ __forceinline__ static int v_at(int row, int b)
    {
        return row * PITCH + 16 * (b ^ (2 * (D == 64 ? (row >> 1) & 3 : D == 96 ? (row >> 2) & 1 : row & 7)));
    }
};

// Maximum and sum over the four lanes 16 apart
__device__ __forceinline__ float rows_max(float x)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float rows_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

template <int DT, int D, int NR>
__device__ __forceinline__ void decode_run(const AttnDecodeParams &p)
{
    using G_ = Geo<D>;
    using DG = DecodeGeo<D>;
    using T = Type16<DT>;
    constexpr int KC = D / 32, TV = D / 16, WAVES = DG::WAVES, THREADS = 64 * WAVES;
    constexpr int STAGES = WAVES * DG::STAGE, RESULTS = WAVES * 16 * NR * D * 4;
    __shared__ __align__(1024) unsigned char lds[STAGES > RESULTS ? STAGES : RESULTS];
    __shared__ float2 stats[WAVES][16 * NR];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int li = lane & 15, lg = lane >> 4;
    const int G = p.a.Hq / p.a.Hkv, rows = p.T * G;
    const int kvh = blockIdx.x % p.a.Hkv, rest = blockIdx.x / p.a.Hkv;
    const int split = rest % p.splits, b = rest / p.splits;
    const int len = min(max(p.lens[b], 0), p.max_len);
    const int begin = split * p.split_keys, end = min(len, begin + p.split_keys);

    // The wave's steps of 32 keys; lane l holds the page of 16-key group l % 2 of step l / 2, -1 where it is none
    const int keys0 = begin + wave * DG::KEYS;
    const int steps = keys0 < end ? (end - keys0 + DG::KEYS * WAVES - 1) / (DG::KEYS * WAVES) : 0;
    int pages = 0;
    if (steps > 0) {
        const int key = min(keys0 + (lane >> 1) * DG::KEYS * WAVES + 16 * (lane & 1), end - 1);
        pages = p.a.kv.table[b * p.a.kv.table_stride + (key >> p.a.kv.page_shift)];
        pages = pages < 0 || pages >= p.a.kv.num_pages ? -1 : pages;
    }

    u32x4 q[NR][KC];
    int seen[NR];  // own keys that the lane's row sees
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const int row = min(16 * r + li, rows - 1), token = row / G, head = kvh * G + row - token * G;
        seen[r] = len - p.T + 1 + token;
        const unsigned char *from = static_cast<const unsigned char *>(p.a.q) + 2 * ((int64_t)(b * p.T + token) * p.a.q_stride + (int64_t)head * D + 8 * lg);
#pragma unroll
        for (int c = 0; c < KC; ++c)
            q[r][c] = *reinterpret_cast<const u32x4 *>(from + 64 * c);
    }
    const int all_see = len - p.T + 1;

    uint32_t k_off[DG::COPIES], v_off[DG::COPIES];
#pragma unroll
    for (int i = 0; i < DG::COPIES; ++i) {
        const int at = 64 * i + lane, r = at / DG::NB, x = at % DG::NB;
        k_off[i] = G_::k_at(r, x);
        v_off[i] = DG::v_at(r, x);
    }
    const unsigned char *const kb = static_cast<const unsigned char *>(p.a.kv.k), *const vb = static_cast<const unsigned char *>(p.a.kv.v);
    const int64_t head_at = ((int64_t)kvh << p.a.kv.page_shift) * D;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void *)lds + wave * DG::STAGE;
    auto fetch = [&](int step, bool is_v) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            // keys behind the last one, and those of no page, are some other rows of the pool: they are masked
            const int page = max(0, __builtin_amdgcn_readlane(pages, 2 * step + t));
            const int in_page = (keys0 + step * DG::KEYS * WAVES + 16 * t) & ((1 << p.a.kv.page_shift) - 1);
            const int64_t at = head_at + (int64_t)in_page * D;
            const unsigned char *from = is_v ? vb + 2 * (page * p.a.kv.v_stride + at) : kb + 2 * (page * p.a.kv.k_stride + at);
#pragma unroll
            for (int i = 0; i < DG::COPIES; ++i)
                copy16(from, is_v ? v_off[i] : k_off[i], lds0 + (is_v ? DG::HALF : 0) + t * (DG::HALF / 2) + 1024 * i);
        }
    };

    // the queries and pages are here before the copies start, so that waits below count copies alone
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < KC; ++c)
            asm volatile("" : "+v"(q[r][c]));
    asm volatile("" : "+v"(pages));

    const float scale = base2(p.a.scale);
    f32x4 o[NR][TV] = {};
    float top[NR], sum[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        top[r] = kNone;
        sum[r] = 0.f;
    }
    const uint32_t kt = lds0, vt = lds0 + DG::HALF;
    constexpr int HALF_COPIES = 2 * DG::COPIES;
    if (steps > 0) {
        fetch(0, false);
        fetch(0, true);
    }
    for (int step = 0; step < steps; ++step) {
        const int k0 = keys0 + step * DG::KEYS * WAVES;
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(HALF_COPIES) : "memory");  // K is here, V behind it
        int none = 0;  // 16-key groups without a page
        none |= __builtin_amdgcn_readlane(pages, 2 * step) < 0 ? 1 : 0;
        none |= __builtin_amdgcn_readlane(pages, 2 * step + 1) < 0 ? 2 : 0;
        const bool masked = k0 + DG::KEYS > min(all_see, end) || none != 0;

        f32x4 s[NR][2] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                const u32x4 k = lds_read16(kt + G_::k_at(16 * t + li, 4 * c + lg));
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    s[r][t] = T::mfma16(k, q[r][c], s[r][t]);
            }
        if (masked) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = k0 + 16 * t + 4 * lg + i;
                        s[r][t][i] = key < min(seen[r], end) && !(none >> t & 1) ? s[r][t][i] : kNone;
                    }
        }
        // K has been read: the next one
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (step + 1 < steps)
            fetch(step + 1, false);
        u32x4 pf[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float most = s[r][0][0];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    most = fmaxf(most, s[r][t][i]);
            most = rows_max(most);
            if (__ballot((most - top[r]) * scale > 8.f) != 0) {  // as in the prompts' kernel
                const float up = fmaxf(top[r], most), f = up == kNone ? 1.f : exp2_f((top[r] - up) * scale);
                top[r] = up;
                sum[r] *= f;
#pragma unroll
                for (int j = 0; j < TV; ++j)
                    o[r][j] *= f;
            }
            const float base = top[r] == kNone ? 0.f : top[r];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float x = exp2_f(fmaf(s[r][t][i] - base, scale, T::kLift)), y = exp2_f(fmaf(s[r][t][i + 1] - base, scale, T::kLift));
                    sum[r] += x;
                    sum[r] += y;
                    pf[r][2 * t + i / 2] = pack2<DT>(x, y);
                }
        }
        if (step + 1 < steps)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(HALF_COPIES) : "memory");  // V is here, the next K behind it
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const int tr_row = 4 * lg + (li >> 2);
        auto v_of = [&](int j) {
            const uint32_t at = vt + DG::v_at(tr_row, 2 * j + ((li & 3) >> 1)) + 8 * (li & 1);
            const u32x2 x = lds_read_tr(at), y = lds_read_tr(at + 16 * DG::PITCH);
            return u32x4{x.x, x.y, y.x, y.y};
        };
        bool plain = true;
        if (masked) {
            // as in the prompts' kernel: what is not finite is left out where it is not seen, and makes a NaN where it is
            uint32_t bad = 0;
            for (int at = 16 * lane; at < DG::HALF; at += 1024) {
                const u32x4 w = lds_read16(vt + at);
                bad |= not_finite<DT>(w.x) | not_finite<DT>(w.y) | not_finite<DT>(w.z) | not_finite<DT>(w.w);
            }
            if (__ballot(bad != 0) != 0) {
                const uint32_t one = pack2<DT>(1.f, 1.f);
                u32x4 sees[NR];
#pragma unroll
                for (int r = 0; r < NR; ++r)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int key = k0 + 16 * (w / 2) + 4 * lg + 2 * (w % 2), upto = none >> (w / 2) & 1 ? 0 : min(seen[r], end);
                        sees[r][w] = (key < upto ? one & 0xffffu : 0u) | (key + 1 < upto ? one & 0xffff0000u : 0u);
                    }
#pragma unroll
                for (int j = 0; j < TV; ++j) {
                    u32x4 v = v_of(j), wrong;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        wrong[w] = (not_finite<DT>(v[w]) >> 15) * 0xffffu & one;
                        v[w] = finite_part<DT>(v[w]);
                    }
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        o[r][j] = T::mfma16(v, pf[r], o[r][j]);
                        const f32x4 hit = T::mfma16(wrong, sees[r], f32x4{});
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[r][j][i] = hit[i] > 0.f ? __builtin_nanf("") : o[r][j][i];
                    }
                }
                plain = false;
            }
        }
        if (plain) {
#pragma unroll
            for (int j = 0; j < TV; ++j) {
                const u32x4 v = v_of(j);
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    o[r][j] = T::mfma16(v, pf[r], o[r][j]);
            }
        }
        // V has been read: the next one
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        if (step + 1 < steps)
            fetch(step + 1, true);
    }

    // The waves' results, [wave][row][D], over the stages
    float *const results = reinterpret_cast<float *>(lds);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        sum[r] = rows_sum(sum[r]);
        if (lg == 0)
            stats[wave][16 * r + li] = make_float2(top[r], sum[r]);
#pragma unroll
        for (int j = 0; j < TV; ++j)
            *reinterpret_cast<f32x4 *>(results + ((wave * NR + r) * 16 + li) * D + 16 * j + 4 * lg) = o[r][j];
    }
    __syncthreads();
    constexpr int LANES = D / 4;  // of a row
    for (int at = threadIdx.x; at < rows * LANES; at += THREADS) {
        const int row = at / LANES, d = 4 * (at % LANES);
        float most = kNone, total = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            most = fmaxf(most, stats[w][row].x);
        const float base = most == kNone ? 0.f : most;
        f32x4 x = {};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float f = exp2_f((stats[w][row].x - base) * scale);
            total += f * stats[w][row].y;
            x += f * *reinterpret_cast<const f32x4 *>(results + (w * NR * 16 + row) * D + d);
        }
        const int token = row / G, head = kvh * G + row - token * G;
        const int64_t to = (int64_t)(b * p.T + token) * p.a.Hq + head;
        if (p.a.slots > 0) {
            const int64_t slot = to * p.a.slots + p.first_slot + split;
            if (d == 0)
                p.a.stat[slot] = make_float2(most, total);
            if (total != 0.f)  // (a NaN too)
                *reinterpret_cast<f32x4 *>(p.a.part + slot * D + d) = x;
        } else {
            const float inv = total == 0.f ? 0.f : 1.f / total;
            uint16_t *out = static_cast<uint16_t *>(p.a.out) + (int64_t)(b * p.T + token) * p.a.out_stride + (int64_t)head * D + d;
            *reinterpret_cast<u32x2 *>(out) = u32x2{pack_outputs<DT>(x.x * inv, x.y * inv), pack_outputs<DT>(x.z * inv, x.w * inv)};
            if (p.a.lse && d == 0)
                p.a.lse[to] = log_sum<DT>(most, p.a.scale, total);
        }
    }
}

template <int DT, int D, int NR>
__global__ __launch_bounds__(64 * DecodeGeo<D>::WAVES, 1) void decode_kernel(const AttnDecodeParams p)
{
    decode_run<DT, D, NR>(p);
}

template <int DT, int D>
hipError_t launch_decode_d(const AttnDecodeParams &p, unsigned grid, hipStream_t s)
{
    constexpr int THREADS = 64 * DecodeGeo<D>::WAVES;
    const int rows = p.T * (p.a.Hq / p.a.Hkv);
    if (rows <= 16)
        decode_kernel<DT, D, 1><<<grid, THREADS, 0, s>>>(p);
    else
        decode_kernel<DT, D, 2><<<grid, THREADS, 0, s>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_decode(const AttnDecodeParams &p, unsigned grid, hipStream_t s)
{
    switch (p.a.D) {
    case 64: return launch_decode_d<DT, 64>(p, grid, s);
    case 96: return launch_decode_d<DT, 96>(p, grid, s);
    case 128: return launch_decode_d<DT, 128>(p, grid, s);
    default: return launch_decode_d<DT, 256>(p, grid, s);
    }
}

}  // namespace attn
}  // namespace gdn
