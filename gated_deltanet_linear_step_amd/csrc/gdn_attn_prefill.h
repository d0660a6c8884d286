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
//    times at a row's start and hardly ever after. Exponentials are then at most 2^8, of f16 2^15 (Type16: kLift).
//  * K and V tiles go from memory straight to the LDS, one to two tiles ahead, two buffers for K and three for V: one barrier
//    a tile. Their 16-byte blocks are permuted within a row by the address that a lane fetches from, so that
//    reads fall into different banks.
//  * Tiles that every row of the block sees run in a loop of their own without masks. It goes 32 keys at a time: the next
//    scores are formed beside the exponentials of these, and the next maximum beside the products with V. Tiles with masked
//    places (the diagonal, the last keys, missing pages) are apart.
//  * P is rounded to the 16 bits of V, by up to 2^-8 (bf16) or 2^-11 (f16, of weights from 2^-21 of the row's largest on; below by
//    up to 2^-32 of that) of each term, as much as the outputs' own rounding; its sum is of the unrounded ones.
//
// Eight prompts of 30,208 tokens, 32 heads over 8 of 128, bf16: 1286 to 1345 us on different cards, 980 to 1020 TFLOP/s (a library's
// product of 8192^3 reaches 1356); 16384 tokens, 16 heads over 2 of 256: 1880 to 1955 us, 1125 to 1170; 4096 such tokens: 178 to
// 183, of which 21 to 23 join parts.
// Bound by the matrix unit and the vector instructions, which hardly overlap: of 128 wide heads' clocks the one is busy in 51 %, the
// other issues in 51 %, with no LDS conflicts, although two waves share a SIMD; the card runs at 1.6 to 1.9 GHz meanwhile. Wave
// priorities, operands read 4 to 8 products ahead and the scheduler's own order of the exponentials made no difference (594 to
// 605 us at 8192 tokens); without the exponentials the same takes 5 % less, without the products of the scores 28 %.
#pragma once

#include "gdn_attn_device.h"

namespace gdn {
namespace attn {

constexpr int kRows = 32, kWaves = 4, kThreads = 64 * kWaves;
static_assert(kBlock == kRows * kWaves, "the rows of a workgroup");

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

template <int DT, int D, bool PAGED>
__device__ __forceinline__ void prefill_block(const AttnPrefillParams &p)
{
    using G_ = Geo<D>;
    using T = Type16<DT>;
    constexpr int KT = G_::KT, NB = G_::NB, KC = D / 16, TV = D / 32, HALVES = KT / 32;
    __shared__ __align__(1024) unsigned char lds[5 * G_::TILE];  // K twice, V three times

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, col = lane & 31;
    const int G = p.a.Hq / p.a.Hkv;

    // Work: a key head, a block of rows, a run of keys. The last blocks, which see most keys, come first. Where there are blocks
    // for every CU, second runs, shorter than first ones, come last; where there are fewer, the runs of a block side by
    // side (128 queries behind 16256 keys, 16 heads over 4: 38 us; the blocks of a run side by side: 48).
    const int kvh = blockIdx.x % p.a.Hkv, rest = blockIdx.x / p.a.Hkv;
    const bool last_runs = p.blocks * p.a.Hkv >= kCus;
    const int split = last_runs ? rest / p.blocks : rest % p.splits, order = last_runs ? rest % p.blocks : rest / p.splits;
    // (of one round of workgroups, two on a CU, the second half goes the other way, so that a CU has one of either kind)
    int block = p.one_round && order >= p.blocks / 2 ? order - p.blocks / 2 : p.blocks - 1 - order;
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
    const int wave_most = wrow < rows ? ahead + step * ((min(wrow + kRows, rows) - 1) / G) : 0;
    const int block_most = max(0, min(nk, ahead + step * ((min(m0 + kBlock, rows) - 1) / G)));
    const int tiles = (block_most + KT - 1) / KT;
    const int first = (int)min((int64_t)split * p.split_tiles, (int64_t)tiles), last = min(tiles - first, p.split_tiles) + first;
    // a block whose keys are one run has nothing to join
    const bool whole = p.whole && tiles <= p.split_tiles;
    if (whole && split > 0)
        return;

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
    int entries = 0;
    // Where a wave's rows of a tile come from, found before the tile's turn
    struct From {
        const unsigned char *k, *v;
        int none;  // groups of the tile that have no page, a bit each
        int over;  // rows of the wave behind the last key (packed rows: none of them is read)
    };
    auto locate = [&](int tile) {
        int k0 = tile * KT + wave * G_::ROWS;
        From from{kb, vb, 0, 0};
        if constexpr (PAGED) {
            const int held = (tile - first) % HELD * GROUPS;
            if (held == 0) {
                entries = table[(int)min((int64_t)tile * KT + 16 * lane, (int64_t)nk - 1) >> p.a.kv.page_shift];
                asm volatile("" : "+v"(entries));
            }
            from.none = (int)(__ballot(entries < 0 || entries >= p.a.kv.num_pages) >> held) & ((1 << GROUPS) - 1);
            // keys behind the last one, and those of no page, are some other rows of the pool: they are masked
            const int entry = __builtin_amdgcn_readlane(entries, held + wave * G_::ROWS / 16);
            const int page = entry < 0 || entry >= p.a.kv.num_pages ? 0 : entry;
            const int64_t in_page = head_at + (int64_t)(k0 & ((1 << p.a.kv.page_shift) - 1)) * D;
            from.k += 2 * (page * p.a.kv.k_stride + in_page);
            from.v += 2 * (page * p.a.kv.v_stride + in_page);
        } else {
            k0 = min(k0, nk - 1);
            from.k += 2 * ((key0 + k0) * p.a.kv.k_stride + head_at);
            from.v += 2 * ((key0 + k0) * p.a.kv.v_stride + head_at);
            from.over = max(0, k0 + G_::ROWS - nk);
        }
        return from;
    };
    auto fetch = [&](const From &from, int k_buf, int v_buf) {
        const uint32_t k_to = lds_at + k_buf * G_::TILE, v_to = lds_at + (2 + v_buf) * G_::TILE;
        if (!PAGED && from.over > 0) {
#pragma unroll
            for (int i = 0; i < G_::FETCH; ++i) {
                const uint32_t over = max(0, (64 * i + opaque(lane)) / NB - (G_::ROWS - 1 - from.over));
                copy16(from.k, k_off[i] - over * k_row, k_to + 1024 * i);
                copy16(from.v, v_off[i] - over * v_row, v_to + 1024 * i);
            }
            return;
        }
        copy16_runs(from.k, k_off, k_to);
        copy16_runs(from.v, v_off, v_to);
    };

    u32x4 q[KC];
    {
        const unsigned char *from = static_cast<const unsigned char *>(p.a.q) + 2 * ((int64_t)(row0 + token) * p.a.q_stride + (int64_t)head * D + 8 * half);
#pragma unroll
        for (int c = 0; c < KC; ++c)
            q[c] = *reinterpret_cast<const u32x4 *>(from + 32 * c);
    }
    const float scale = base2(p.a.scale);
    f32x16 o[TV] = {};
    // The sum of the weights, those of up to 16 tiles apart: one sum of all would lose what is below 2^-25 of it and drift by the rounding of
    // each (2^20 weights of 0.67: 0.35 % off, now 2e-5).
    float top = kNone, sum = 0.f, recent = 0.f;
    float base = -T::kLift;  // exponentials are 2^(scale s - base)
    bool far = false;  // of any row of the wave: kFar

    auto largest = [&](const f32x16 &s) {
        float x = fmaxf(s[0], s[1]);
#pragma unroll
        for (int i = 2; i < 16; i += 2)
            x = fmaxf(fmaxf(x, s[i]), s[i + 1]);
        return x;
    };
    // Takes the largest of the 32 scores s into the running maximum where it passes that by 8 in base 2
    auto rescale = [&](float most, f32x16 &s) {
        most = half_max(most);
        if (__ballot((most - top) * scale > 8.f) != 0) {
            const float up = fmaxf(top, most), f = up == kNone ? 1.f : exp2_f((top - up) * scale);
            top = up;
            base = up == kNone ? 0.f : up * scale;
            far = __ballot(fabsf(base) > kFar) != 0;
            base = (far ? 0.f : base) - T::kLift;
            sum *= f;
            recent *= f;
#pragma unroll
            for (int t = 0; t < TV; ++t)
                o[t] *= f;
        }
        if (far)
            s -= top == kNone ? 0.f : top;
    };
    auto scores = [&](f32x16 &s, uint32_t kt) {
        const uint32_t k_at = opaque(kt + G_::k_at(col, half));
        s = f32x16{};
#pragma unroll
        for (int c = 0; c < KC; ++c)
            s = T::mfma32(lds_read16(G_::k_next(k_at, c)), q[c], s);
    };
    // V^T, 32 dv from 32 tv on and the 16 keys of st, in P's order
    const int v_lane = G_::v_at(4 * half + ((lane & 15) >> 2), 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) + 8 * (lane & 1);
    auto v_of = [&](uint32_t v_at, int tv, int st) {
        const uint32_t at = G_::v_next(v_at, tv) + 16 * st * G_::PITCH;
        const u32x2 x = lds_read_tr(at), y = lds_read_tr(at + 8 * G_::PITCH);
        return u32x4{x.x, x.y, y.x, y.y};
    };

    // 32 keys that every row of the block sees, with scores s and values at vt. The scores `next` of the next 32 keys, which
    // lie at next_kt, are formed while the exponentials of these are, a product and what fits beside it in turn (the
    // scheduler would put the products first), and their largest is found beside the products with V. LDS reads run ahead of
    // the products, the first ones of a step (kf) of the step before.
    // D = 256 has no registers for two sets of scores: the next ones are formed at the end, in the same place.
    constexpr bool AHEAD = D <= 128;
    constexpr int READ = 3;  // operands read ahead
    u32x4 kf[KC];
    auto read_k = [&](uint32_t kt) {
        const uint32_t k_at = opaque(kt + G_::k_at(col, half));
#pragma unroll
        for (int c = 0; c < READ; ++c)
            kf[c] = lds_read16(G_::k_next(k_at, c));
    };
    // read_on: the keys after the next are here, at then_kt. go_on: the next keys are attended to by a call of this (scores of keys
    // that a row does not see must not move its maximum)
    auto attend = [&](f32x16 &s, f32x16 &next, uint32_t vt, uint32_t next_kt, bool read_on, uint32_t then_kt, bool go_on) {
        u32x4 pf[2];
        const uint32_t v_at = opaque(vt + v_lane);
        if constexpr (AHEAD) {
            constexpr int N = 2 * TV;
            const uint32_t k_at = opaque(next_kt + G_::k_at(col, half));
            u32x4 vf[N];
            float e[16];
            next = f32x16{};
#pragma unroll
            for (int c = 0; c <= KC; ++c) {
                if (c + READ < KC)
                    kf[c + READ] = lds_read16(G_::k_next(k_at, c + READ));
                else if (c < KC)
                    vf[c + READ - KC] = v_of(v_at, (c + READ - KC) % TV, (c + READ - KC) / TV);
                if (c < KC)
                    next = T::mfma32(kf[c], q[c], next);
                // a share of the eight pairs of exponentials, and what follows from those of the product before
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (c < KC && i * KC / 8 == c) {
                        e[2 * i] = exp2_f(fmaf(s[2 * i], scale, -base));
                        e[2 * i + 1] = exp2_f(fmaf(s[2 * i + 1], scale, -base));
                    }
                    if (i * KC / 8 + 1 == c) {
                        recent += e[2 * i];
                        recent += e[2 * i + 1];
                        pf[i / 4][i % 4] = pack2<DT>(e[2 * i], e[2 * i + 1]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            const uint32_t then_at = opaque(then_kt + G_::k_at(col, half));
            float most = fmaxf(next[0], next[1]);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (i + READ < N)
                    vf[i + READ] = v_of(v_at, (i + READ) % TV, (i + READ) / TV);
                else if (read_on)
                    kf[i + READ - N] = lds_read16(G_::k_next(then_at, i + READ - N));
                o[i % TV] = T::mfma32(vf[i], pf[i / TV], o[i % TV]);
#pragma unroll
                for (int x = 1; x < 8; ++x)
                    if (i == min(x * N / 8 + 1, N - 1))
                        most = fmaxf(fmaxf(most, next[2 * x]), next[2 * x + 1]);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (go_on)
                rescale(most, next);
        } else {
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float x = exp2_f(fmaf(s[i], scale, -base)), y = exp2_f(fmaf(s[i + 1], scale, -base));
                recent += x;
                recent += y;
                pf[i / 8][i % 8 / 2] = pack2<DT>(x, y);
            }
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int tv = 0; tv < TV; ++tv)
                    o[tv] = T::mfma32(v_of(v_at, tv, st), pf[st], o[tv]);
            scores(next, next_kt);
            if (go_on)
                rescale(largest(next), next);
        }
    };

    // 32 keys from k0 on, of which a row may not see some; `none`: two bits, the groups of 16 without a page.
    auto attend_masked = [&](int k0, int none, uint32_t kt, uint32_t vt) {
        // 0 times what is not finite in a masked place must not reach a row: those values are left out, and
        // a row that sees one of them becomes NaN
        uint32_t bad = 0;
        const auto look = [&](int at) {
            const u32x4 w = lds_read16(vt + at + 16 * lane);
            bad |= not_finite<DT>(w.x) | not_finite<DT>(w.y) | not_finite<DT>(w.z) | not_finite<DT>(w.w);
        };
        if constexpr (AHEAD) {  // beside the products of the scores (D = 256 has no registers for that)
#pragma unroll
            for (int at = 0; at < 32 * G_::PITCH; at += 1024)
                look(at);
        }
        f32x16 s;
        scores(s, kt);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int key = 8 * (i / 4) + 4 * half + i % 4;
            s[i] = k0 + key < seen && !(none >> (i / 8) & 1) ? s[i] : kNone;
        }
        rescale(largest(s), s);
        u32x4 pf[2];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const float x = exp2_f(fmaf(s[i], scale, -base)), y = exp2_f(fmaf(s[i + 1], scale, -base));
            recent += x;
            recent += y;
            pf[i / 8][i % 8 / 2] = pack2<DT>(x, y);
        }
        if constexpr (!AHEAD) {
#pragma unroll 1
            for (int at = 0; at < 32 * G_::PITCH; at += 1024)
                look(at);
        }
        const uint32_t v_at = opaque(vt + v_lane);
        const bool finite = __ballot(bad != 0) == 0;
        if constexpr (AHEAD)  // (two ways to the sums take more registers than D = 256 has)
            if (finite) {
#pragma unroll
                for (int st = 0; st < 2; ++st)
#pragma unroll
                    for (int tv = 0; tv < TV; ++tv)
                        o[tv] = T::mfma32(v_of(v_at, tv, st), pf[st], o[tv]);
                return;
            }
        u32x4 sees[2];
        const uint32_t one = pack2<DT>(1.f, 1.f);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            const int key = k0 + 8 * (i / 4) + 4 * half + i % 4, upto = none >> (i / 8) & 1 ? 0 : seen;
            sees[i / 8][i % 8 / 2] = (key < upto ? one & 0xffffu : 0u) | (key + 1 < upto ? one & 0xffff0000u : 0u);
        }
#pragma unroll
        for (int tv = 0; tv < TV; ++tv) {
            f32x16 hit = {};
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                u32x4 v = v_of(v_at, tv, st), wrong;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    wrong[w] = (not_finite<DT>(v[w]) >> 15) * 0xffffu;
                    v[w] &= ~wrong[w];
                    wrong[w] &= one;
                }
                o[tv] = T::mfma32(v, pf[st], o[tv]);
                if (!finite)
                    hit = T::mfma32(wrong, sees[st], hit);
            }
            if (!finite) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[tv][i] = hit[i] > 0.f ? __builtin_nanf("") : o[tv][i];
            }
        }
    };

    // K and V of a tile are here at the end of the tile before (with D = 256 of the one before that, K being read a tile ahead). At
    // a tile's last 32 keys its K is no longer read, nor is V of the tile before: the tile after the next takes their places.
    int none = 0, next_none = 0, v_buf = 0;
    if (first < last) {
        const From from = locate(first);
        fetch(from, 0, 0);
        none = from.none;
        if (first + 1 < last) {
            const From second = locate(first + 1);
            fetch(second, 1, 1);
            next_none = second.none;
        }
        // the queries too: a wait for them in the loop would be one for the tile on its way
#pragma unroll
        for (int c = 0; c < KC; ++c)
            asm volatile("" : "+v"(q[c]));
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
    // read_on: the next step's first operands are read as soon as the tile is here, at kt
    auto turn = [&](int tile, bool read_on, uint32_t kt) {
        if (((tile - first) & 15) == 15) {
            sum += recent;
            recent = 0.f;
        }
        From from{kb, vb, 0, 0};
        if (tile + 2 < last)
            from = locate(tile + 2);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's part of the next tile has landed
        __syncthreads();                                  // and everyone's
        if (read_on)
            read_k(kt);
        if (tile + 2 < last)
            fetch(from, (tile - first) & 1, v_buf == 0 ? 2 : v_buf - 1);
        none = next_none;
        next_none = from.none;
        v_buf = v_buf == 2 ? 0 : v_buf + 1;
    };
    // tiles that every row of the block sees, up to a page that is none; the same for every wave
    const int block_least = min(nk, ahead + step * (m0 / G)), full = min(last, max(0, block_least) / KT);
    int tile = first;
    if (tile < full && none == 0) {
        f32x16 s[HALVES];
        static_assert(AHEAD == (HALVES == 2), "two sets of scores, or one");
        scores(s[0], lds0);
        rescale(largest(s[0]), s[0]);
        if constexpr (AHEAD)
            read_k(lds0 + 32 * G_::PITCH);
        do {
            const uint32_t kt = lds0 + ((tile - first) & 1) * G_::TILE, vt = lds0 + (2 + v_buf) * G_::TILE;
            const uint32_t next_kt = lds0 + ((tile + 1 - first) & 1) * G_::TILE;
            if constexpr (HALVES == 2)
                attend(s[0], s[1], vt, kt + 32 * G_::PITCH, false, 0, true);
            turn(tile, AHEAD, next_kt);
            attend(s[HALVES - 1], s[0], vt + (KT - 32) * G_::PITCH, next_kt, true, next_kt + 32 * G_::PITCH,
                   tile + 1 < full && none == 0);
            ++tile;
        } while (tile < full && none == 0);
    }
    for (; tile < last; ++tile) {
        const uint32_t kt = lds0 + ((tile - first) & 1) * G_::TILE, vt = lds0 + (2 + v_buf) * G_::TILE;
#pragma unroll 1
        for (int h = 0; h < HALVES; ++h)
            if (tile * KT + 32 * h < wave_most)
                attend_masked(tile * KT + 32 * h, none >> 2 * h, kt + 32 * h * G_::PITCH, vt + 32 * h * G_::PITCH);
        turn(tile, false, 0);
    }

    sum = half_sum(sum + recent);
    const int end_row = wrow + opaque(col);
    if (end_row >= rows)
        return;
    const int end_token = end_row / G, end_head = kvh * G + end_row - end_token * G;
    const int64_t at = (int64_t)(row0 + end_token) * p.a.Hq + end_head;
    if (whole && p.a.slots > 0 && half == 0)
        p.a.stat[at * p.a.slots] = make_float2(kNone, kJoined);
    if (p.a.slots > 0 && !whole) {
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
            const u32x2 w = {pack_outputs<DT>(o[tv][4 * g] * inv, o[tv][4 * g + 1] * inv),
                             pack_outputs<DT>(o[tv][4 * g + 2] * inv, o[tv][4 * g + 3] * inv)};
            *reinterpret_cast<u32x2 *>(to + 32 * tv + 8 * g + 4 * half) = w;
        }
    if (p.a.lse && half == 0)
        p.a.lse[at] = log_sum<DT>(top, p.a.scale, sum);
}

// Waves of a SIMD: what the LDS holds, but of 64 wide heads three (168 registers), not four.
template <int DT, int D, bool PAGED>
__global__ __launch_bounds__(kThreads, D == 64 ? 3 : 2) void prefill_kernel(const AttnPrefillParams p)
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
