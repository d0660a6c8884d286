// gdn_attn.hip -- softmax attention: how calls are split into launches, and the join of
// partial results.
//
// Where a call has few rows, a row's keys are split into runs that go to workgroups of
// their own. Each leaves its outputs relative to its own maximum m, with m and the sum l:
//     o = sum_s e^(scale (m_s - M)) o_s / sum_s e^(scale (m_s - M)) l_s,   M = max_s m_s
// joins them. A run without keys has l = 0 and no outputs.

#include "gdn_attn_device.h"

#include <algorithm>

namespace gdn {
namespace {

using namespace attn;

// Four of a row's outputs, from element d on
template <int DT>
__device__ __forceinline__ void store_joined(const AttnParams &p, int64_t row, int d, f32x4 o, float most, float total)
{
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int64_t token = row / p.Hq, head = row - token * p.Hq;
    uint16_t *to = static_cast<uint16_t *>(p.out) + token * p.out_stride + head * p.D + d;
    *reinterpret_cast<u32x2 *>(to) = u32x2{pack_outputs<DT>(o.x * inv, o.y * inv), pack_outputs<DT>(o.z * inv, o.w * inv)};
    if (p.lse && d == 0)
        p.lse[row] = log_sum<DT>(most, p.scale, total);
}

// Up to 64 runs: a wave joins a row (a query and head). A lane looks at one run's maximum and sum; then D / 4 lanes
// share a run's outputs, D <= 128 several runs side by side, all loads of eight turns in flight together.
template <int DT, int D>
__global__ __launch_bounds__(256) void join_few_kernel(const AttnParams p, int64_t rows)
{
    constexpr int LANES = D / 4, GROUPS = 64 / LANES, TURNS = 8;
    const int lane = threadIdx.x & 63, group = lane / LANES, d = 4 * (lane % LANES);
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), first = row * p.slots;
    if (row >= rows)
        return;
    const float2 st = lane < p.slots ? p.stat[first + lane] : make_float2(kNone, 0.f);
    if (__shfl(st.y, 0, 64) == kJoined)
        return;
    float most = st.y == 0.f ? kNone : st.x;
#pragma unroll
    for (int x = 32; x; x >>= 1)
        most = fmaxf(most, __shfl_xor(most, x, 64));
    // a run without keys left its outputs as they were: -1; one whose factor f32 holds as 0 counts, for what is not finite in it
    // (no mask of runs shifted by a lane's own number here: gdn_attn_device.h, on 64-bit shifts)
    const float f = st.y == 0.f ? -1.f : exp2_f((st.x - most) * base2(p.scale));
    float total = f * st.y;
#pragma unroll
    for (int x = 32; x; x >>= 1)
        total += __shfl_xor(total, x, 64);
    f32x4 o = {};
    for (int s0 = 0; s0 < p.slots; s0 += GROUPS * TURNS) {
        f32x4 v[TURNS];
        float w[TURNS];
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
            const int s = s0 + i * GROUPS + group;
            w[i] = __shfl(f, s & 63, 64);
            if (group >= GROUPS || s >= p.slots)
                w[i] = -1.f;
            // in place of what is left out the first run's are read
            v[i] = *reinterpret_cast<const f32x4 *>(p.part + (first + (w[i] < 0.f ? 0 : s)) * D + d);
        }
#pragma unroll
        for (int i = 0; i < TURNS; ++i)
            o += w[i] < 0.f ? f32x4{} : w[i] * v[i];
    }
    if constexpr (GROUPS > 1) {
#pragma unroll
        for (int g = 1; g < GROUPS; g *= 2) {
            // from the upper half of the groups (of 96 wide rows: lanes 24 on)
            const int from = (lane + g * LANES) & 63;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] += __shfl(o[i], from, 64);
        }
    }
    if (group == 0)
        store_joined<DT>(p, row, d, o, most, total);
}

constexpr int kJoinThreads = 256, kJoinWidth = 32, kJoinRuns = kJoinThreads / (kJoinWidth / 4);

// A workgroup joins 32 of a row's (a query and head) D outputs: 8 lanes share a run's, 32 runs are read at a time.
template <int DT>
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const AttnParams p)
{
    __shared__ float4 sums[kJoinThreads];
    __shared__ float tops[kJoinThreads / 64], totals[kJoinThreads];
    const int parts = p.D / kJoinWidth, lane = threadIdx.x % 8, group = threadIdx.x / 8;
    const int64_t row = blockIdx.x / parts, first = row * p.slots;
    const int d = blockIdx.x % parts * kJoinWidth + 4 * lane;
    float most = kNone;
    for (int s = threadIdx.x; s < p.slots; s += kJoinThreads) {
        const float2 st = p.stat[first + s];
        most = fmaxf(most, st.y == 0.f ? kNone : st.x);
    }
#pragma unroll
    for (int x = 32; x; x >>= 1)
        most = fmaxf(most, __shfl_xor(most, x, 64));
    if ((threadIdx.x & 63) == 0)
        tops[threadIdx.x >> 6] = most;
    __syncthreads();
    most = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    f32x4 o = {};
    float total = 0.f;
    for (int s = group; s < p.slots; s += kJoinRuns) {
        const float2 st = p.stat[first + s];
        if (st.y == 0.f)
            continue;
        const float f = exp2_f((st.x - most) * base2(p.scale));
        total += f * st.y;
        o += f * *reinterpret_cast<const f32x4 *>(p.part + (first + s) * p.D + d);
    }
    // the wave's eight runs, then the four waves
#pragma unroll
    for (int x = 8; x < 64; x *= 2) {
        total += __shfl_xor(total, x, 64);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] += __shfl_xor(o[i], x, 64);
    }
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) < 8) {
        sums[8 * wave + lane] = make_float4(o.x, o.y, o.z, o.w);
        totals[8 * wave + lane] = total;
    }
    __syncthreads();
    if (threadIdx.x >= 8)
        return;
#pragma unroll
    for (int w = 1; w < kJoinThreads / 64; ++w) {
        const float4 v = sums[8 * w + lane];
        total += totals[8 * w + lane];
        o += f32x4{v.x, v.y, v.z, v.w};
    }
    store_joined<DT>(p, row, d, o, most, total);
}

template <int DT>
hipError_t join_few(const AttnParams &p, int64_t rows, unsigned grid, hipStream_t s)
{
    switch (p.D) {
    case 64: join_few_kernel<DT, 64><<<grid, 256, 0, s>>>(p, rows); break;
    case 96: join_few_kernel<DT, 96><<<grid, 256, 0, s>>>(p, rows); break;
    case 128: join_few_kernel<DT, 128><<<grid, 256, 0, s>>>(p, rows); break;
    default: join_few_kernel<DT, 256><<<grid, 256, 0, s>>>(p, rows); break;
    }
    return hipGetLastError();
}

}  // namespace

int64_t attn_prefill_blocks(int Hq, int Hkv, int N, int64_t total, bool packed)
{
    const int64_t G = Hq / Hkv;
    // packed: an upper bound, of which up to one a sequence stays empty
    const int64_t blocks = packed ? total * G / kBlock + N : N * ((total / std::max(N, 1) * G + kBlock - 1) / kBlock);
    return blocks * Hkv;
}

bool attn_supported(int D) { return D == 64 || D == 96 || D == 128 || D == 256; }

int attn_prefill_most_splits(int Hq, int Hkv, int64_t total)
{
    const int64_t G = Hq / Hkv, blocks = std::max<int64_t>(1, (total * G + kBlock - 1) / kBlock) * Hkv;
    return blocks > 2 * kCus ? 1 : blocks >= kCus ? 2 : (int)std::min<int64_t>(1024 / blocks, 32);
}

void attn_prefill_splits(int Hq, int Hkv, int D, int N, int64_t total, const int32_t *cu_q, const int32_t *cu_k, int keys, int *splits,
                         int *split_tiles)
{
    const int most = attn_prefill_most_splits(Hq, Hkv, total), KT = D <= 128 ? 64 : 32;
    const int64_t G = Hq / Hkv;
    *splits = 1;
    *split_tiles = 1 << 30;
    if (most == 1)
        return;
    // f(tiles, block) for every block of rows, numbered as the kernel does
    const auto blocks = [&](auto f) {
        for (int s = 0; s < N; ++s) {
            const int64_t len = cu_q ? cu_q[s + 1] - cu_q[s] : total, nk = cu_q ? cu_k[s + 1] - cu_k[s] : keys;
            int64_t block = cu_q ? block_base(cu_q, s, (int)G) : 0;
            for (int64_t row = 0; row < len * G; row += kBlock, ++block) {
                const int64_t token = (std::min(row + kBlock, len * G) - 1) / G;
                f((std::clamp<int64_t>(cu_q ? nk - len + 1 + token : nk, 0, nk) + KT - 1) / KT, block);
            }
        }
    };
    int64_t all = 0, longest = 0, count = 0;
    blocks([&](int64_t tiles, int64_t) {
        all += tiles * Hkv;
        count += Hkv;
        longest = std::max(longest, tiles);
    });
    constexpr int64_t kSlots = 2 * kCus;  // two workgroups on a CU
    int64_t each = std::max<int64_t>({(all + kSlots - 1) / kSlots, 4, (longest + most - 1) / most});
    if (count >= kCus) {
        // Blocks for every CU, but of all lengths: a long one would be left alone on its CU, at about 0.6 of the rate of two. Cut at
        // the average, their ends go where short ones were; it pays where that is more than writing and joining parts takes.
        // Heads of 256 (us, uncut / cut): 2048 tokens, 32 heads over 4, 109 / 113; 4096, 16 over 2, 199 / 172; behind 16384, 1126 / 1104;
        // 2048 behind 14336 725 / 488. Narrower ones gain less by a tile, and are cut where the longest has 64 tiles more. Of 128, 16
        // heads over 2: 4096 tokens (31 more) 89 / 104, behind 16384 (31) 583 / 607, 8 x 300 behind 8000 (54) 222 / 232, 8 over 1 of
        // 8192 (63) 168 / 169; 2048 behind 14336 (135) 299 / 279, 8 x 300 behind up to 16000 (200) 288 / 212; a prefix of 16000 for
        // 1200 queries, 32 over 8 (101) 536 / 502. Heads of 96 turn at the same lengths (72 / 92, 186 / 194, 135 / 151; 244 / 233, 237 /
        // 181, 438 / 400), those of 64 a little sooner (31: 69 / 87, 46: 117 / 120, 54: 180 / 148, 59: 89 / 86, 101: 372 / 284; but 63: 119 / 134).
        bool pays = longest - each >= (D == 64 ? 50 : 64);
        if (D == 256) {
            int64_t cut = 0;
            blocks([&](int64_t tiles, int64_t) { cut += tiles > each ? Hkv : 0; });
            // microseconds: 1.25 a tile, 8 a launch, 4.5e6 bytes of parts written and read
            pays = 0.7 * 1.25 * (longest - each) > 8 + cut * 2.0 * kBlock * D * 4 * 2 / 4.5e6;
        }
        if (!pays)
            return;
    } else {
        // Fewer: runs of one length, as many as one round of workgroups holds on every XCD (they go to the 8 in turn, those
        // that have no keys too)
        const int64_t numbered = attn_prefill_blocks(Hq, Hkv, N, total, cu_q != nullptr) / Hkv;
        while (each < longest) {
            const int64_t runs = (longest + each - 1) / each;
            int64_t on[8] = {}, most_on = 0;
            blocks([&](int64_t tiles, int64_t block) {
                for (int64_t run = 0; run * each < tiles; ++run)
                    for (int h = 0; h < Hkv; ++h)
                        most_on = std::max(most_on, ++on[(((numbered - 1 - block) * runs + run) * Hkv + h) % 8]);
            });
            if (most_on <= kSlots / 8)
                break;
            each = (longest + runs - 2) / (runs - 1);  // one run less of the longest
        }
    }
    if (longest > each) {
        *splits = (int)((longest + each - 1) / each);
        *split_tiles = (int)each;
    }
}

hipError_t launch_attn_prefill(const AttnPrefillParams &given, hipStream_t s)
{
    AttnPrefillParams p = given;
    p.blocks = (int)(attn_prefill_blocks(p.a.Hq, p.a.Hkv, p.N, p.total, p.cu_q != nullptr) / p.a.Hkv);
    const int64_t grid = (int64_t)p.blocks * p.a.Hkv * p.splits;
    // without the blocks that stay empty: one a sequence
    p.one_round = p.splits == 1 && (int64_t)(p.blocks - (p.cu_q ? p.N : 0)) * p.a.Hkv <= 2 * kCus;
    return p.a.dt == DT_BF16 ? launch_attn_prefill_bf16(p, (unsigned)grid, s) : launch_attn_prefill_f16(p, (unsigned)grid, s);
}

namespace {

// Up to this many rows of a sequence and key head the decode kernel takes; more are blocks of rows like a prompt's
constexpr int kDecodeRows = 32;
bool few_rows(int Hq, int Hkv, int T) { return (int64_t)T * (Hq / Hkv) <= kDecodeRows; }

}  // namespace

int64_t attn_decode_blocks(int Hq, int Hkv, int D, int B, int T)
{
    return few_rows(Hq, Hkv, T) ? (int64_t)B * Hkv : attn_prefill_blocks(Hq, Hkv, B, (int64_t)B * T, false);
}

void attn_decode_splits(int Hq, int Hkv, int D, int B, int T, int max_len, int *splits, int *split_keys)
{
    const int64_t blocks = attn_decode_blocks(Hq, Hkv, D, B, T);
    if (!few_rows(Hq, Hkv, T)) {
        const int KT = D <= 128 ? 64 : 32;
        const int64_t tiles = (std::max(max_len, 1) + KT - 1) / KT, want = std::clamp<int64_t>(2 * kCus / blocks, 1, 64);
        *split_keys = (int)std::clamp<int64_t>((tiles + want - 1) / want, 4, kMostKeys / KT);
        *splits = (int)((tiles + *split_keys - 1) / *split_keys);
        return;
    }
    // Runs of a whole number of rounds of the waves: as many workgroups as fill the card once, and at most 1024 keys each, so that
    // sequences of all lengths even out (64 of 128 to 8192 keys, 32 heads over 8 of 128: 202 us). Where a long bound would make
    // more than 64 runs of that, longer ones, up to what the lanes hold pages for.
    constexpr int64_t round = kDecodeRound, most = kDecodeRounds;
    const int64_t rounds = (std::max(max_len, 1) + round - 1) / round;
    const int64_t want = std::clamp<int64_t>((D == 256 ? kCus : 2 * kCus) / std::max<int64_t>(blocks, 1), 1, rounds);
    const int64_t even = std::min<int64_t>((rounds + want - 1) / want, 1024 / round);
    const int64_t each = std::min(std::max(even, want > 64 ? even : (rounds + 63) / 64), most);
    *split_keys = (int)(each * round);
    *splits = (int)((rounds + each - 1) / each);
}

hipError_t launch_attn_decode(const AttnDecodeParams &p, hipStream_t s)
{
    if (few_rows(p.a.Hq, p.a.Hkv, p.T)) {
        const unsigned grid = (unsigned)((int64_t)p.B * p.a.Hkv * p.splits);
        return p.a.dt == DT_BF16 ? launch_attn_decode_bf16(p, grid, s) : launch_attn_decode_f16(p, grid, s);
    }
    AttnPrefillParams f{};
    f.a = p.a;
    f.N = p.B;
    f.T = p.T;
    f.total = p.B * p.T;
    f.lens = p.lens;
    f.max_keys = p.max_len;
    f.splits = p.splits;
    f.split_tiles = p.split_keys;
    f.first_slot = p.first_slot;
    return launch_attn_prefill(f, s);
}

int64_t attn_join_blocks(int D, int slots, int64_t rows) { return slots <= 64 ? (rows + 3) / 4 : rows * (D / kJoinWidth); }

hipError_t launch_attn_join(const AttnParams &p, int64_t rows, hipStream_t s)
{
    const unsigned grid = (unsigned)attn_join_blocks(p.D, p.slots, rows);
    if (p.slots <= 64)
        return p.dt == DT_BF16 ? join_few<DT_BF16>(p, rows, grid, s) : join_few<DT_F16>(p, rows, grid, s);
    if (p.dt == DT_BF16)
        join_kernel<DT_BF16><<<grid, kJoinThreads, 0, s>>>(p);
    else
        join_kernel<DT_F16><<<grid, kJoinThreads, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace gdn
