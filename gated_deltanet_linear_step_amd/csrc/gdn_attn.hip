// gdn_attn.hip -- softmax attention: how calls are split into launches, and the join of
// partial results.
//
// Where a call has few rows, a row's keys are split into runs that go to workgroups of
// their own. Each leaves its outputs relative to its own maximum m, with m and the sum l:
//     o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,   M = max_s m_s
// joins them. A run without keys has l = 0 and no outputs.

#include "gdn_attn_device.h"

#include <algorithm>

namespace gdn {
namespace {

using namespace attn;

// A workgroup per row (query and head); D / 4 lanes share a run's outputs, the workgroup's other lanes take other runs.
template <int DT>
__global__ void join_kernel(const AttnParams p)
{
    __shared__ float4 sums[256];
    __shared__ float totals[256];
    const int lanes = p.D / 4, groups = blockDim.x / lanes, group = threadIdx.x / lanes, lane = threadIdx.x % lanes;
    const int64_t row = blockIdx.x, first = row * p.slots;
    float most = kNone;
    for (int s = 0; s < p.slots; ++s)
        most = fmaxf(most, p.stat[first + s].y == 0.f ? kNone : p.stat[first + s].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    if (group < groups)
        for (int s = group; s < p.slots; s += groups) {
            const float2 st = p.stat[first + s];
            if (st.y == 0.f)
                continue;
            const float f = exp2_f(st.x - most);
            const float4 v = *reinterpret_cast<const float4 *>(p.part + (first + s) * p.D + 4 * lane);
            total += f * st.y;
            o.x += f * v.x;
            o.y += f * v.y;
            o.z += f * v.z;
            o.w += f * v.w;
        }
    sums[threadIdx.x] = o;
    totals[threadIdx.x] = total;
    __syncthreads();
    if (group != 0)
        return;
    for (int g = 1; g < groups; ++g) {
        const float4 v = sums[g * lanes + lane];
        total += totals[g * lanes + lane];
        o.x += v.x;
        o.y += v.y;
        o.z += v.z;
        o.w += v.w;
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int64_t token = row / p.Hq, head = row - token * p.Hq;
    uint16_t *to = static_cast<uint16_t *>(p.out) + token * p.out_stride + head * p.D + 4 * lane;
    *reinterpret_cast<u32x2 *>(to) = u32x2{pack2<DT>(o.x * inv, o.y * inv), pack2<DT>(o.z * inv, o.w * inv)};
    if (p.lse && lane == 0)
        p.lse[row] = total == 0.f ? kNone : (most + __log2f(total)) * 0.69314718055994531f;
}

constexpr int kBlock = 128;  // rows of a workgroup of the prefill kernel
constexpr int kCus = 256;

}  // namespace

bool attn_supported(int D) { return D == 64 || D == 96 || D == 128 || D == 256; }

int attn_prefill_splits(int Hq, int Hkv, int64_t total, int64_t max_keys)
{
    // at least this many workgroups where there are keys enough: two for each CU
    const int64_t G = Hq / Hkv, blocks = std::max<int64_t>(1, (total * G + kBlock - 1) / kBlock) * Hkv;
    const int64_t most = std::max<int64_t>(1, max_keys / 256);
    return (int)std::clamp<int64_t>(512 / blocks, 1, std::min<int64_t>(most, 32));
}

int64_t attn_prefill_blocks(int Hq, int Hkv, int N, int64_t total, bool packed)
{
    const int64_t G = Hq / Hkv;
    // packed: an upper bound, of which up to one a sequence stays empty
    return (packed ? total * G / kBlock + N : N * ((total / std::max(N, 1) * G + kBlock - 1) / kBlock)) * Hkv;
}

hipError_t launch_attn_prefill(const AttnPrefillParams &given, hipStream_t s)
{
    AttnPrefillParams p = given;
    const int64_t blocks = attn_prefill_blocks(p.a.Hq, p.a.Hkv, p.N, p.total, p.cu_q != nullptr) * p.splits;
    // without the blocks that stay empty: one a sequence
    const int64_t empty = p.cu_q ? (int64_t)p.N * p.a.Hkv * p.splits : 0;
    p.one_round = blocks - empty <= 2 * kCus;
    return p.a.dt == DT_BF16 ? launch_attn_prefill_bf16(p, (unsigned)blocks, s) : launch_attn_prefill_f16(p, (unsigned)blocks, s);
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
        *splits = (int)std::clamp<int64_t>(1024 / blocks, 1, std::min<int64_t>(std::max(1, max_len / 256), 64));
        *split_keys = 0;
        return;
    }
    // Runs of a whole number of rounds of the waves, as many workgroups as keep every CU busy, at most what the lanes hold pages
    // for
    const int waves = D == 64 ? 4 : D == 256 ? 1 : 2, round = 32 * waves;
    const int64_t rounds = (std::max(max_len, 1) + round - 1) / round;
    const int64_t want = std::clamp<int64_t>(1024 / std::max<int64_t>(blocks, 1), 1, rounds);
    const int64_t each = std::min<int64_t>((rounds + want - 1) / want, std::max(1, 1024 / round));
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
    f.first_slot = p.first_slot;
    return launch_attn_prefill(f, s);
}

hipError_t launch_attn_join(const AttnParams &p, int64_t rows, hipStream_t s)
{
    const int threads = p.slots <= 8 ? 64 : 256;
    if (p.dt == DT_BF16)
        join_kernel<DT_BF16><<<(unsigned)rows, threads, 0, s>>>(p);
    else
        join_kernel<DT_F16><<<(unsigned)rows, threads, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace gdn
