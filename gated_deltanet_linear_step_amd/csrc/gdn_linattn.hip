// gdn_linattn.hip -- decayed linear attention on gfx950: per v-head, with a state
// S[dv][dk] (f32, key index innermost) and a log decay g_t,
//     S <- exp(g_t) S + v_t k_t^T,   o_t = scale (S q_t).
// The decay is one rate per head (GDN_HEAD_DECAY) or one value per token and head.
//
// recur_kernel runs the recurrence token by token: the decode step.
//  * HBM bound: 0.5 flop per state byte. Every state row is loaded into VGPRs once
//    per call, carried through the call's tokens and stored once.
//  * Rows are independent (there is no delta rule to couple them), so a head's rows
//    are split over workgroups as finely as the batch needs.
//  * LPR lanes hold a row as float4 pieces, 16-byte loads of contiguous runs; the
//    row's dot with q reduces over LPR <= 16 lanes on DPP alone. Lane r of a row
//    group stores the output of the group's row r, so a wave's rows leave in one
//    store instruction.
//  * The next token's k, q, v and decay are loaded while the current one runs.
// B=64, 32 heads of 128 x 128, one token: 48.7 us, 5.5 TB/s of state (a large copy reaches
// 5.0, the last-level cache holds part of the states); one sequence of 48 heads: 3.7 us.

#include "gdn_device.h"
#include "gdn_ops.h"
#include "gdn_linattn_chunk.h"

#include <algorithm>
#include <type_traits>

namespace gdn {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool NT>
__device__ __forceinline__ float4 load_row4(const float *p)
{
    f32x4 v;
    if constexpr (NT)
        v = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
    else
        v = *reinterpret_cast<const f32x4 *>(p);
    return make_float4(v.x, v.y, v.z, v.w);
}

template <bool NT>
__device__ __forceinline__ void store_row4(float *p, float4 s)
{
    f32x4 v = {s.x, s.y, s.z, s.w};
    if constexpr (NT)
        __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(p));
    else
        *reinterpret_cast<f32x4 *>(p) = v;
}

// ---- the recurrence ----------------------------------------------------------

constexpr int kRecurWaves = 4;

// Lanes per state row: 16 lanes of one or more float4 pieces; 8 where a row has
// too few pieces for 16 (dk = 32) or they do not divide (dk = 96).
constexpr int recur_lpr(int dk) { return dk % 64 == 0 ? 16 : 8; }

// Rows a workgroup of R rows per lane group covers.
constexpr int recur_rows(int dk, int r) { return kRecurWaves * r * (64 / recur_lpr(dk)); }

template <int DK, int QT, int R>
struct RecurToken {
    static constexpr int P = DK / (4 * recur_lpr(DK));
    Raw4<QT> k[P], q[P];
    uint32_t v[R];
    float g;
};

template <int DK, int QT, int R>
__device__ __forceinline__ void load_recur_token(RecurToken<DK, QT, R> &t, const LinattnParams &p,
                                                 int64_t row, int h, int kh, int col, const int *vrow)
{
    constexpr int LPR = recur_lpr(DK);
    const ActInputs &in = p.in;
#pragma unroll
    for (int m = 0; m < t.P; ++m) {
        const int64_t c = (int64_t)kh * DK + col + 4 * LPR * m;
        t.k[m] = load_raw4<QT>(in.k, row * in.k_stride + c);
        t.q[m] = load_raw4<QT>(in.q, row * in.q_stride + c);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        t.v[i] = load_raw1<QT>(in.v, row * in.v_stride + (int64_t)h * p.hc.dv + vrow[i]);
    if (!(p.hc.flags & F_HEAD_DECAY))
        t.g = in.g[row * p.hc.Hv + h + vgpr_zero()];
}

// One workgroup per (sequence, v-head, recur_rows rows). R rows per lane group.
template <int DK, int QT, int R, bool NT>
__global__ __launch_bounds__(64 * kRecurWaves) void recur_kernel(const LinattnParams p)
{
    constexpr int LPR = recur_lpr(DK), P = DK / (4 * LPR), ROWS = recur_rows(DK, R);
    const int slices = (p.hc.dv + ROWS - 1) / ROWS;
    const int slice = blockIdx.x % slices;
    const int h = (blockIdx.x / slices) % p.hc.Hv;
    const int b = blockIdx.x / slices / p.hc.Hv;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane % LPR, grp = lane / LPR;
    const int col = 4 * r;

    int64_t row0 = (int64_t)b * p.T;
    int T = p.T;
    if (p.cu) {
        row0 = p.cu[b];
        T = p.cu[b + 1] - p.cu[b];
    }
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.num_slots || T <= 0)
        return;

    // the group's R rows; rows past dv repeat the last one and store nothing
    const int first = slice * ROWS + (wave * (64 / LPR) + grp) * R;
    int vrow[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        vrow[i] = min(first + i, p.hc.dv - 1);
    const int kh = k_head_of(p.hc.head_map, h, p.hc.Hk, p.hc.Hv);
    RecurToken<DK, QT, R> tok;
    load_recur_token<DK, QT, R>(tok, p, row0, h, kh, col, vrow);

    float *sb = p.state + ((int64_t)slot * p.hc.Hv + h) * p.hc.dv * DK;
    float4 S[R][P];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int m = 0; m < P; ++m)
            S[i][m] = load_row4<NT>(sb + (int64_t)vrow[i] * DK + col + 4 * LPR * m);

    if (p.hc.flags & F_HEAD_DECAY) {
        const float d = p.in.decay_param[h];
        tok.g = p.hc.decay_kind == 0 ? -expf(d) : d;
    }
    for (int t = 0; t < T; ++t) {
        const RecurToken<DK, QT, R> cur = tok;
        if (t + 1 < T)
            load_recur_token<DK, QT, R>(tok, p, row0 + t + 1, h, kh, col, vrow);
        const float a = expf(cur.g);
        float o[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
            o[i] = 0.f;
#pragma unroll
        for (int m = 0; m < P; ++m) {
            const float4 k = raw4_to_f32<QT>(cur.k[m]), q = raw4_to_f32<QT>(cur.q[m]);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float v = raw1_to_f32<QT>(cur.v[i]);
                float4 &s = S[i][m];
                s.x = fmaf(v, k.x, a * s.x);
                s.y = fmaf(v, k.y, a * s.y);
                s.z = fmaf(v, k.z, a * s.z);
                s.w = fmaf(v, k.w, a * s.w);
                o[i] += dot4(s, q);
            }
        }
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float sum = group_sum<LPR>(o[i]);
            mine = r == i ? sum : mine;
        }
        if (r < R && first + r < p.hc.dv)
            store_act(p.out, ((row0 + t) * p.hc.Hv + h) * p.hc.dv + first + r, p.out_dt, p.hc.scale * mine);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (first + i < p.hc.dv) {
#pragma unroll
            for (int m = 0; m < P; ++m)
                store_row4<NT>(sb + (int64_t)vrow[i] * DK + col + 4 * LPR * m, S[i][m]);
        }
}

template <int DK, int QT, int R, bool NT>
hipError_t launch_recur_t(const LinattnParams &p, hipStream_t s)
{
    const int slices = (p.hc.dv + recur_rows(DK, R) - 1) / recur_rows(DK, R);
    recur_kernel<DK, QT, R, NT><<<dim3((unsigned)((int64_t)p.N * p.hc.Hv * slices)), 64 * kRecurWaves, 0, s>>>(p);
    return hipGetLastError();
}

template <int DK, int QT>
hipError_t launch_recur_q(const LinattnParams &p, hipStream_t s)
{
    // Rows per lane group. One token: 2 (B=64 x 32 heads of 128 x 128: 48.7 us, 50.3 with 4, 54.1 with 8; 8
    // sequences 7.2, 7.5, 7.1). Several tokens: 4, which share each token's k, q and decay (B=64, T=8: 68 us, 76
    // with 2), unless that leaves CUs idle: then 1 (B=1, T=8: 6.1 us, 7.4 with 4).
    const bool nt = p.hc.flags & F_STREAM_STATE;
    if (p.T == 1)
        return nt ? launch_recur_t<DK, QT, 2, true>(p, s) : launch_recur_t<DK, QT, 2, false>(p, s);
    if ((int64_t)p.N * p.hc.Hv * p.hc.dv < 256 * recur_rows(DK, 4))
        return launch_recur_t<DK, QT, 1, false>(p, s);
    return nt ? launch_recur_t<DK, QT, 4, true>(p, s) : launch_recur_t<DK, QT, 4, false>(p, s);
}

template <int DK>
hipError_t launch_recur_d(const LinattnParams &p, hipStream_t s)
{
    switch (p.in.qkv_dt) {
    case DT_F32: return launch_recur_q<DK, DT_F32>(p, s);
    case DT_F16: return launch_recur_q<DK, DT_F16>(p, s);
    default: return launch_recur_q<DK, DT_BF16>(p, s);
    }
}

hipError_t launch_recur(const LinattnParams &p, hipStream_t s)
{
    switch (p.hc.dk) {
    case 32: return launch_recur_d<32>(p, s);
    case 64: return launch_recur_d<64>(p, s);
    case 96: return launch_recur_d<96>(p, s);
    case 128: return launch_recur_d<128>(p, s);
    default: return launch_recur_d<256>(p, s);
    }
}

}  // namespace

bool linattn_supported(int dk, int dv) { return decode_supported(dk, dv); }

// Whether a launch over the sequences' heads holds fewer than 2^32 threads: the recurrence with two rows to a lane
// group (with one it has few workgroups); the chunk kernels have no more for the same states.
bool linattn_grid_fits(int N, int Hv, int dk, int dv)
{
    return (int64_t)N * Hv * ((dv + recur_rows(dk, 2) - 1) / recur_rows(dk, 2)) * 64 * kRecurWaves < (int64_t)1 << 32;
}

hipError_t launch_linattn_decode(const LinattnParams &p, hipStream_t s) { return launch_recur(p, s); }

// ---- the chunked prefill (kernels: gdn_linattn_chunk.h) ------------------------

namespace {

using linattn::Cut;

// Segments are a multiple of 64 tokens (whole chunks of 64 or 32), at least kMinSegment, and not more in a call than
// about kSegments over all heads (and a head's parts of 128 dv rows): every one but a sequence's last costs a pass
// over its keys and values and its state written and read twice.
constexpr int kMinSegment = 128, kSegments = 1024;
constexpr int kShortest = 8;  // sequences up to this long go token by token

int parts_of(int dv) { return dv > 128 ? dv / 128 : 1; }

int least_segment(int Hv, int dv, int64_t total)
{
    const int64_t heads = (int64_t)Hv * parts_of(dv), per = (total * heads + kSegments - 1) / kSegments;
    return (int)std::max<int64_t>(kMinSegment, (per + 63) / 64 * 64);
}

// States between segments a call may need, per head: a sequence of several segments is longer than one of them,
// so it has at most len / L + 1/2 states. Grows with total.
int64_t segment_slots(int Hv, int dv, int64_t total)
{
    const int64_t most = std::min<int64_t>(total / kMinSegment, kSegments / ((int64_t)Hv * parts_of(dv)) + 1);
    return most + (most + 1) / 2;
}

struct Counts {
    int64_t first, between, last;
    int longest_single;
};
Counts count_segments(const int32_t *cu, int N, Cut cut)
{
    Counts c{N, 0, 0, 0};  // an empty sequence counts for a first segment, which ends at once
    for (int i = 0; i < N; ++i) {
        const int len = cu[i + 1] - cu[i], segs = cut.segments(len);
        if (segs == 1)
            c.longest_single = std::max(c.longest_single, len);
        c.between += segs > 2 ? segs - 2 : 0;
        c.last += segs > 1;
    }
    return c;
}

// The segment length whose launches end first, of a few lengths from the least one on. In units of a token's time in a
// segment without outputs (29 ns at 128 x 128; with outputs twice that), as measured for bf16 heads of 128 x 128 and an estimate
// for others, where a CU may hold one workgroup and a state fewer bytes: a launch takes its longest
// segment times its rounds, a state between segments 1.55, the second launch and the running sum 250. The host walks the
// offsets for each length: with many sequences, which fill the card by themselves, one is taken unseen.
// us with segments of 128, 256, 512: 4096 tokens x 32 heads 108 85 90, 2048 x 32 58 57 83, 1024 x 16 34 48 79,
// 4096 x 8 43 52 81; 700 tokens x 16 heads of 256 x 256: 55 71 107.
constexpr int kFewSequences = 64, kManySequencesSegment = 256;
// Rounds of n workgroups on 256 CUs that hold two each; two that share a CU take 1.4 times as long as one alone.
double rounds(int64_t n)
{
    const int64_t rest = n % 512;
    return n / 512 * 1.4 + (rest == 0 ? 0.0 : rest <= 256 ? 1.0 : 1.4);
}
Cut choose_cut(const int32_t *cu, int N, int Hv, int dv, int64_t total)
{
    int least = least_segment(Hv, dv, total);
    if (N > kFewSequences)
        least = std::max(least, kManySequencesSegment);
    const int64_t heads = (int64_t)Hv * parts_of(dv);
    Cut best{};
    double best_cost = 0;
    for (int i = 0; i < (N <= kFewSequences ? 8 : 1); ++i) {
        const int L = least + 64 * i * ((least + 511) / 512);
        const Cut cut{L, (L / 2 + 63) / 64 * 64};
        const Counts c = count_segments(cu, N, cut);
        const double longest = std::max(c.last ? (double)L : 0.0, 2.0 * c.longest_single);
        const double cost = longest * rounds((c.first + c.between) * heads) + 2.0 * L * rounds((c.between + c.last) * heads) +
                            1.55 * (double)(c.between * heads) + (c.last ? 250 : 0);
        if (i == 0 || cost < best_cost) {
            best = cut;
            best_cost = cost;
        }
    }
    return best;
}

// Entering states: a sequence's slot s (state after its segment s, entered with zero
// from s = 1 on) becomes the state after segment s. HBM bound, one float4 a thread; the
// loads of later segments do not wait for the running sum. The grid covers `seqs` sequences at a time.
__global__ __launch_bounds__(256) void scan_kernel(const LinattnParams p, int vecs, int seqs)
{
    const int blocks = vecs / 256;  // vecs = dk dv / 4 is a multiple of 256 for every head shape
    const int at = blockIdx.x % blocks * 256 + threadIdx.x, h = blockIdx.x / blocks % p.hc.Hv;
    const Cut cut{p.seg_tokens, p.seg_first_tokens};
    for (int64_t seq = blockIdx.x / blocks / p.hc.Hv; seq < p.N; seq += seqs) {
        const int segs = cut.segments(p.cu[seq + 1] - p.cu[seq]);
        if (segs < 3)
            continue;
        const int64_t step = (int64_t)p.hc.Hv * vecs;
        const int64_t slot = (int64_t)linattn::slots_before(p.cu, cut, (int)seq) * p.hc.Hv + h;
        float4 *x = reinterpret_cast<float4 *>(p.seg_state) + slot * vecs + at;
        const float *d = p.seg_decay + slot;
        float4 run = *x;
        // eight segments' loads at a time, in front of their stores; the rest by fours (more would be loads for nothing)
        auto batch = [&](int s0, auto count) {
            constexpr int n = decltype(count)::value;
            float4 add[n];
            float a[n];
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const int s = min(s0 + i, segs - 2);
                add[i] = x[s * step];
                a[i] = d[(int64_t)s * p.hc.Hv];
            }
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float e = expf(a[i]);
                run = make_float4(fmaf(e, run.x, add[i].x), fmaf(e, run.y, add[i].y), fmaf(e, run.z, add[i].z), fmaf(e, run.w, add[i].w));
                if (s0 + i < segs - 1)
                    x[(s0 + i) * step] = run;
            }
        };
        int s = 1;
        for (; s + 8 < segs; s += 8)
            batch(s, std::integral_constant<int, 8>());
        for (; s + 1 < segs; s += 4)
            batch(s, std::integral_constant<int, 4>());
    }
}

hipError_t launch_chunk_dt(const LinattnParams &p, int64_t segments, bool second, hipStream_t s)
{
    switch (p.in.qkv_dt) {
    case DT_F32: return launch_linattn_chunk_f32(p, segments, second, s);
    case DT_F16: return launch_linattn_chunk_f16(p, segments, second, s);
    default: return launch_linattn_chunk_bf16(p, segments, second, s);
    }
}

}  // namespace

size_t linattn_prefill_workspace_bytes(int, int Hv, int dk, int dv, int, int64_t total)
{
    return 256 + (size_t)segment_slots(Hv, dv, total) * Hv * (4 * (size_t)dk * dv + 4);
}

hipError_t launch_linattn_prefill(const LinattnParams &given, const int32_t *cu, hipStream_t s)
{
    LinattnParams p = given;
    // A chunk costs the same however few tokens are in it. 8 sequences x 32 heads of 128 x 128, us (recurrence,
    // chunks): 4 tokens 10.4 14.5, 8 13.5 14.4, 16 20 14.4; 64 sequences: 8 68 77, 16 101 78.
    if (p.T <= kShortest)
        return launch_recur(p, s);
    const Cut cut = choose_cut(cu, p.N, p.hc.Hv, p.hc.dv, p.total);
    const Counts c = count_segments(cu, p.N, cut);
    p.seg_tokens = cut.L;
    p.seg_first_tokens = cut.L0;
    p.segs_first = (int)c.first;
    p.segs_between = (int)c.between;
    p.seg_state = static_cast<float *>(p.workspace);
    p.seg_decay = p.seg_state + segment_slots(p.hc.Hv, p.hc.dv, p.total) * p.hc.Hv * p.hc.dk * p.hc.dv;
    hipError_t e = launch_chunk_dt(p, c.first + c.between, false, s);
    if (e != hipSuccess || c.last == 0)
        return e;
    if (c.between > 0) {
        // (few sequences have states between segments; a grid of 2^20 workgroups is plenty)
        const int vecs = p.hc.dk * p.hc.dv / 4, per_seq = p.hc.Hv * (vecs / 256);
        const int seqs = std::min(p.N, std::max(1, (1 << 20) / per_seq));
        scan_kernel<<<(unsigned)((int64_t)seqs * per_seq), 256, 0, s>>>(p, vecs, seqs);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return launch_chunk_dt(p, c.between + c.last, true, s);
}

}  // namespace gdn
