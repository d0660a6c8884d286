// gdn_attn_prefill.h -- softmax attention of blocks of queries on gfx950 (instantiated per dtype by
// gdn_attn_bf16.hip and gdn_attn_f16.hip).
//
// The queries of one key head -- all the query heads that read it, token after token -- are
// the rows of one matrix, so that a block of 128 rows shares each key and value whatever
// the grouping. A workgroup of four waves walks the keys in tiles; a wave holds 32 rows.
//
//  * Scores are formed transposed, S^T = K Q^T (v_mfma_f32_32x32x16): a lane then holds one row's scores, 16 keys of a
//    tile of 32, and the row's maximum and sum need one exchange, with the lane 32 away.
//  * As they lie, the exponentials are the operand of O^T += V^T P^T: the product's slot 8 h + e is key 4 h + e (e < 4) or
//    8 + 4 h + e - 4 of 16, and V^T is read in that order by transposing LDS reads. Nothing passes between lanes.
//  * The running maximum moves only where a row's scores pass it by more than 2^8: sums and outputs are rescaled a few
//    times at a row's start and hardly ever after. Exponentials are then at most 2^8, which f32 and either 16-bit type hold
//    with the same relative error.
//  * K and V tiles go from memory straight to the LDS, a tile ahead. Their 16-byte blocks are permuted within a row by
//    the address that a lane fetches from, so that reads of 16 rows fall into different banks.
//  * P is rounded to the 16 bits of V, 2^-9 (bf16) or 2^-12 of each term; its sum is of the unrounded ones.
#pragma once

#include "gdn_attn_device.h"

namespace gdn {
namespace attn {

constexpr int kRows = 32, kWaves = 4, kBlock = kRows * kWaves, kThreads = 64 * kWaves;

template <int D>
struct Geo {
    static constexpr int KT = D <= 128 ? 64 : 32;   // keys of a tile
    static constexpr int NB = D / 8;                // 16-byte blocks of a row
    static constexpr int PITCH = 2 * D, TILE = KT * PITCH;
    static constexpr int ROWS = KT / kWaves;        // rows of a tile that a wave fetches, within one page
    static constexpr int FETCH = ROWS * NB / 64;    // 16-byte fetches of a lane
    // Where block b of a row lies. K: 16 rows' blocks b cover all banks; V: the blocks 4 b .. 4 b + 3 of 4 rows do.
    __device__ __forceinline__ static int k_at(int row, int b)
    {
        return row * PITCH + 16 * (D == 64 ? b ^ ((row >> 1) & 7) : D == 96 ? b ^ ((row >> 2) & 3) : b ^ (row & 15));
    }
    __device__ __forceinline__ static int v_swizzle(int row)
    {
        return D == 64 ? 4 * ((row >> 1) & 1) : D == 96 ? 0 : 4 * (row & 3);
    }
    __device__ __forceinline__ static int v_at(int row, int b) { return row * PITCH + 16 * (b ^ v_swizzle(row)); }
    // Blocks 2 c + x of a row, and 4 c + x of V, from where blocks x lie: the permutation is an exclusive or of a few bits
    __device__ __forceinline__ static uint32_t k_next(uint32_t at, int c)
    {
        constexpr int M = D == 64 ? 4 : D == 96 ? 2 : 8;
        return (at ^ (32 * (c % M))) + 32 * M * (c / M);
    }
    __device__ __forceinline__ static uint32_t v_next(uint32_t at, int c)
    {
        constexpr int M = D == 64 ? 2 : D == 96 ? 1 : 4;
        return (at ^ (64 * (c % M))) + 64 * M * (c / M);
    }
};

// First block of 128 rows that the sequences before cu[s] leave to sequence s (some blocks stay empty)
__host__ __device__ __forceinline__ int block_base(const int32_t *cu, int s, int G)
{
    return (int)((int64_t)cu[s] * G / kBlock) + s;
}

template <int DT, int D, bool PAGED>
__device__ __forceinline__ void prefill_block(const AttnPrefillParams &p)
{
    using G_ = Geo<D>;
    using T = Type16<DT>;
    constexpr int KT = G_::KT, NB = G_::NB, KC = D / 16, TV = D / 32, TS = KT / 32;
    __shared__ __align__(1024) unsigned char lds[4 * G_::TILE];  // K, K, V, V

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    const int G = p.a.Hq / p.a.Hkv;

    // Work: a key head, a run of keys, a block of rows; the last blocks, which see most keys, first
    const int kvh = blockIdx.x % p.a.Hkv, rest = blockIdx.x / p.a.Hkv;
    const int split = rest % p.splits;
    const int blocks_all = gridDim.x / (p.a.Hkv * p.splits);
    int block = rest / p.splits;
    // (of one round of workgroups, two on a CU, the second half goes the other way, so that a CU has one of either kind)
    block = p.one_round && block >= blocks_all / 2 ? block - blocks_all / 2 : blocks_all - 1 - block;
    int seq = 0, row0, len, nk;
    int64_t key0 = 0;
    if (p.cu_q) {
        int lo = 0, hi = p.N - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (block_base(p.cu_q, mid, G) <= block)
                lo = mid;
            else
                hi = mid - 1;
        }
        seq = lo;
        block -= block_base(p.cu_q, seq, G);
        row0 = p.cu_q[seq];
        len = p.cu_q[seq + 1] - row0;
        key0 = p.cu_k[seq];
        nk = p.cu_k[seq + 1] - (int)key0;
    } else {
        const int blocks = (int)(((int64_t)p.T * G + kBlock - 1) / kBlock);
        seq = block / blocks;
        block %= blocks;
        row0 = seq * p.T;
        len = p.T;
        nk = p.lens ? min(max(p.lens[seq], 0), p.max_keys) : p.max_keys;
    }
    const bool causal = p.cu_q || p.lens;
    const int rows = len * G, m0 = block * kBlock;
    if (m0 >= rows)
        return;
    // keys that token i sees: nk - len + 1 + i of the causal ones
    const int ahead = causal ? nk - len + 1 : nk, step = causal ? 1 : 0;
    const int wrow = m0 + wave * kRows;  // this wave's first row
    const int row = min(wrow + col, rows - 1);
    const int token = row / G, head = kvh * G + row - token * G;
    const int seen = min(nk, ahead + step * token);
    const int wave_least = ahead + step * (min(wrow, rows - 1) / G);
    const int wave_most = wrow < rows ? ahead + step * ((min(wrow + kRows, rows) - 1) / G) : 0;
    const int block_most = max(0, min(nk, ahead + step * ((min(m0 + kBlock, rows) - 1) / G)));
    const int tiles = (block_most + KT - 1) / KT;
    const int first = (int)min((int64_t)split * p.split_tiles, (int64_t)tiles), last = min(tiles - first, p.split_tiles) + first;

    // What a lane fetches of each tile: FETCH blocks of the wave's ROWS rows
    const unsigned char *const kb = static_cast<const unsigned char *>(p.a.kv.k), *const vb = static_cast<const unsigned char *>(p.a.kv.v);
    const int32_t *const table = p.a.kv.table + (PAGED ? seq * p.a.kv.table_stride : 0);
    // bytes from row to row: below 2^25, and 16 rows are fetched from one address
    const uint32_t k_row = 2 * (PAGED ? D : (uint32_t)p.a.kv.k_stride), v_row = 2 * (PAGED ? D : (uint32_t)p.a.kv.v_stride);
    const int64_t head_at = PAGED ? ((int64_t)kvh << p.a.kv.page_shift) * D : (int64_t)kvh * D;
    uint32_t k_off[G_::FETCH], v_off[G_::FETCH];
#pragma unroll
    for (int i = 0; i < G_::FETCH; ++i) {
        const int at = 64 * i + lane, r = at / NB, r_tile = wave * G_::ROWS + r, b = at % NB;
        k_off[i] = r * k_row + G_::k_at(r_tile, b) - r_tile * G_::PITCH;
        v_off[i] = r * v_row + G_::v_at(r_tile, b) - r_tile * G_::PITCH;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void *)lds, lds_at = lds0 + wave * G_::ROWS * G_::PITCH;
    // On pages: the lanes hold the table's entries for the 64 groups of 16 keys of so many tiles. They are asked for as a whole,
    // before the first of those tiles is: a wait for an entry is one for every copy on its way too.
    constexpr int GROUPS = KT / 16, HELD = 64 / GROUPS;
    int entries = 0, none = 0;  // none: groups of the tile fetched last that have no page
    auto fetch = [&](int tile, int buf) {
        int k0 = tile * KT + wave * G_::ROWS;
        const uint32_t to = lds_at + buf * G_::TILE;
        const unsigned char *k_from, *v_from;
        if constexpr (PAGED) {
            const int held = (tile - first) % HELD * GROUPS;
            if (held == 0) {
                entries = table[(int)min((int64_t)tile * KT + 16 * lane, (int64_t)nk - 1) >> p.a.kv.page_shift];
                asm volatile("" : "+v"(entries));
            }
            none = (int)(__ballot(entries < 0 || entries >= p.a.kv.num_pages) >> held) & ((1 << GROUPS) - 1);
            // keys behind the last one, and those of no page, are some other rows of the pool: they are masked
            const int entry = __builtin_amdgcn_readlane(entries, held + wave * G_::ROWS / 16);
            const int page = entry < 0 || entry >= p.a.kv.num_pages ? 0 : entry;
            const int64_t in_page = head_at + (int64_t)(k0 & ((1 << p.a.kv.page_shift) - 1)) * D;
            k_from = kb + 2 * (page * p.a.kv.k_stride + in_page);
            v_from = vb + 2 * (page * p.a.kv.v_stride + in_page);
        } else {
            k0 = min(k0, nk - 1);
            k_from = kb + 2 * ((key0 + k0) * p.a.kv.k_stride + head_at);
            v_from = vb + 2 * ((key0 + k0) * p.a.kv.v_stride + head_at);
            if (k0 + G_::ROWS > nk) {  // no row behind the last key
#pragma unroll
                for (int i = 0; i < G_::FETCH; ++i) {
                    const uint32_t over = max(0, (64 * i + opaque(lane)) / NB - (nk - 1 - k0));
                    copy16(k_from, k_off[i] - over * k_row, to + 1024 * i);
                    copy16(v_from, v_off[i] - over * v_row, to + 1024 * i + 2 * G_::TILE);
                }
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < G_::FETCH; ++i) {
            copy16(k_from, k_off[i], to + 1024 * i);
            copy16(v_from, v_off[i], to + 1024 * i + 2 * G_::TILE);
        }
    };

    u32x4 q[KC];
    {
        const unsigned char *from = static_cast<const unsigned char *>(p.a.q) + 2 * ((int64_t)(row0 + token) * p.a.q_stride + (int64_t)head * D + 8 * half);
#pragma unroll
        for (int c = 0; c < KC; ++c)
            q[c] = *reinterpret_cast<const u32x4 *>(from + 32 * c);
        // here, not in the loop, where the wait would be for the tile on its way too
#pragma unroll
        for (int c = 0; c < KC; ++c)
            asm volatile("" : "+v"(q[c]));
    }
    const float scale = p.a.scale * 1.4426950408889634f;  // exponentials in base 2
    f32x16 o[TV] = {};
    float top = kNone, sum = 0.f;

    // Of the two waves of a SIMD one goes first wherever both could: equals would use the matrix unit at the same time, and
    // then the vector unit, and neither beside the other
    if (__builtin_amdgcn_s_getreg(4 | 3 << 11) & 1)  // the wave's slot
        __builtin_amdgcn_s_setprio(1);

    if (first < last)
        fetch(first, 0);
    for (int tile = first; tile < last; ++tile) {
        const int buf = (tile - first) & 1, k0 = tile * KT, none_here = none;
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's part of the tile has landed
        __syncthreads();                                  // and everyone's; the other buffer is no longer read
        if (tile + 1 < last)
            fetch(tile + 1, buf ^ 1);
        if (k0 >= wave_most)
            continue;

        // the LDS addresses of a tile are formed as they are needed (D = 256 has no registers for them)
        const uint32_t kt = lds0 + buf * G_::TILE, vt = lds0 + (2 + buf) * G_::TILE;
        const uint32_t k_at = opaque(kt + G_::k_at(col, half));
        f32x16 s[TS] = {};
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int c = 0; c < KC; ++c)
                s[t] = T::mfma32(lds_read16(G_::k_next(k_at, c) + 32 * t * G_::PITCH), q[c], s[t]);

        // some row of the wave does not see all of the tile
        const bool masked = k0 + KT > wave_least || k0 + KT > nk || none_here != 0;
        if (masked) {
#pragma unroll
            for (int t = 0; t < TS; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = 32 * t + 8 * (i / 4) + 4 * half + i % 4;
                    s[t][i] = k0 + key < seen && !(none_here >> (key / 16) & 1) ? s[t][i] : kNone;
                }
        }
        float most = s[0][0];
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                most = fmaxf(most, s[t][i]);
        most = half_max(most) * scale;
        if (__ballot(most > top + 8.f) != 0) {
            const float up = fmaxf(top, most), f = up == kNone ? 1.f : exp2_f(top - up);
            top = up;
            sum *= f;
#pragma unroll
            for (int t = 0; t < TV; ++t)
                o[t] *= f;
        }
        const float base = top == kNone ? 0.f : top;
        u32x4 pf[KT / 16];
#pragma unroll
        for (int t = 0; t < TS; ++t)
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float a = exp2_f(fmaf(s[t][i], scale, -base)), b = exp2_f(fmaf(s[t][i + 1], scale, -base));
                sum += a;
                sum += b;
                pf[2 * t + i / 8][i % 8 / 2] = pack2<DT>(a, b);
            }

        // V^T, 32 dv from 32 tv on and the 16 keys of step st, in P's order
        const uint32_t v_at = opaque(vt + G_::v_at(4 * half + ((lane & 15) >> 2), 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) + 8 * (lane & 1));
        auto v_of = [&](int tv, int st) {
            const uint32_t at = G_::v_next(v_at, tv) + 16 * st * G_::PITCH;
            const u32x2 x = lds_read_tr(at), y = lds_read_tr(at + 8 * G_::PITCH);
            return u32x4{x.x, x.y, y.x, y.y};
        };
        if (masked) {
            // 0 times what is not finite in a masked place must not reach a row: those values are left out, and
            // a row that sees one of them becomes NaN
            uint32_t bad = 0;
            for (int at = 16 * lane; at < G_::TILE; at += 1024) {
                const u32x4 w = lds_read16(vt + at);
                bad |= not_finite<DT>(w.x) | not_finite<DT>(w.y) | not_finite<DT>(w.z) | not_finite<DT>(w.w);
            }
            if (__ballot(bad != 0) != 0) {
                const uint32_t one = pack2<DT>(1.f, 1.f);
                u32x4 sees[KT / 16];
#pragma unroll
                for (int st = 0; st < KT / 16; ++st)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int key = 16 * st + 8 * (w / 2) + 4 * half + 2 * (w % 2);
                        const bool page = !(none_here >> st & 1);
                        sees[st][w] = (page && k0 + key < seen ? one & 0xffffu : 0u) | (page && k0 + key + 1 < seen ? one & 0xffff0000u : 0u);
                    }
#pragma unroll
                for (int tv = 0; tv < TV; ++tv) {
                    f32x16 hit = {};
#pragma unroll
                    for (int st = 0; st < KT / 16; ++st) {
                        u32x4 v = v_of(tv, st), wrong;
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            wrong[w] = (not_finite<DT>(v[w]) >> 15) * 0xffffu & one;
                            v[w] = finite_part<DT>(v[w]);
                        }
                        o[tv] = T::mfma32(v, pf[st], o[tv]);
                        hit = T::mfma32(wrong, sees[st], hit);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[tv][i] = hit[i] > 0.f ? __builtin_nanf("") : o[tv][i];
                }
                continue;
            }
        }
#pragma unroll
        for (int st = 0; st < KT / 16; ++st)
#pragma unroll
            for (int tv = 0; tv < TV; ++tv)
                o[tv] = T::mfma32(v_of(tv, st), pf[st], o[tv]);
    }

    sum = half_sum(sum);
    const int end_row = wrow + opaque(col);
    if (end_row >= rows)
        return;
    const int end_token = end_row / G, end_head = kvh * G + end_row - end_token * G;
    const int64_t at = (int64_t)(row0 + end_token) * p.a.Hq + end_head;
    if (p.a.slots > 0) {
        const int64_t slot = at * p.a.slots + p.first_slot + split;
        if (half == 0)
            p.a.stat[slot] = make_float2(top, sum);
        if (first >= last)
            return;
        float *to = p.a.part + slot * D;
#pragma unroll
        for (int tv = 0; tv < TV; ++tv)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<float4 *>(to + 32 * tv + 8 * g + 4 * half) =
                    make_float4(o[tv][4 * g], o[tv][4 * g + 1], o[tv][4 * g + 2], o[tv][4 * g + 3]);
        return;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t *to = static_cast<uint16_t *>(p.a.out) + (int64_t)(row0 + end_token) * p.a.out_stride + (int64_t)end_head * D;
#pragma unroll
    for (int tv = 0; tv < TV; ++tv)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const u32x2 w = {pack2<DT>(o[tv][4 * g] * inv, o[tv][4 * g + 1] * inv), pack2<DT>(o[tv][4 * g + 2] * inv, o[tv][4 * g + 3] * inv)};
            *reinterpret_cast<u32x2 *>(to + 32 * tv + 8 * g + 4 * half) = w;
        }
    if (p.a.lse && half == 0)
        p.a.lse[at] = sum == 0.f ? kNone : (top + __log2f(sum)) * 0.69314718055994531f;
}

template <int DT, int D, bool PAGED>
__global__ __launch_bounds__(kThreads, 2) void prefill_kernel(const AttnPrefillParams p)
{
    prefill_block<DT, D, PAGED>(p);
}

template <int DT, int D>
hipError_t launch_d(const AttnPrefillParams &p, unsigned grid, hipStream_t s)
{
    if (p.a.kv.page_shift >= 0)
        prefill_kernel<DT, D, true><<<grid, kThreads, 0, s>>>(p);
    else
        prefill_kernel<DT, D, false><<<grid, kThreads, 0, s>>>(p);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_prefill(const AttnPrefillParams &p, unsigned grid, hipStream_t s)
{
    switch (p.a.D) {
    case 64: return launch_d<DT, 64>(p, grid, s);
    case 96: return launch_d<DT, 96>(p, grid, s);
    case 128: return launch_d<DT, 128>(p, grid, s);
    default: return launch_d<DT, 256>(p, grid, s);
    }
}

}  // namespace attn
}  // namespace gdn
