// gdn_linattn_chunk.h -- chunked prefill of the decayed linear attention on gfx950
// (instantiated per input dtype by gdn_linattn_bf16.hip, _f16.hip, _f32.hip).
//
// Per chunk of C tokens of one v-head, with the log decays' prefix sums G_t and the
// entering state S:
//     O  = scale (diag(e^G) Q S^T + (tril(Q K^T) . e^(G_t - G_j)) V)
//     S <- e^G_last S + (diag(e^(G_last - G_j)) V)^T K
//
// A workgroup walks the chunks of one segment (a run of consecutive chunks of one
// sequence) of one v-head, the head's state in MFMA accumulators. Long sequences are
// split into segments so that few rows still fill the card:
//   1. chunk_kernel, first launch: every sequence's first segment, complete (from the
//      given state, which the last segment overwrites in the second launch); every later
//      segment but the last, its contribution to the state alone, as if it entered with
//      zero.
//   2. scan_kernel: entering states by a running sum over each sequence's segments.
//   3. chunk_kernel, second launch: the later segments, complete.
// A call whose sequences all have one segment is the first launch alone.
//
// Products are on v_mfma_f32_16x16x32_bf16. An operand that is not bf16 is a sum of
// bf16 parts: f16 two, and f32 -- inputs, the state, P and the decayed V -- three, which
// leave nothing (of f32 values below 2^-109, less than 2^-133, where bf16 ends). The
// leading part is cut off, not rounded, so that it cannot overflow: it leaves less than
// 2^-7 of its power of two. The second is rounded and leaves at most 2^-16, of either sign.
// Products of parts whose orders, counted from 0, add up to more than 2 are left out:
// with bf16 inputs there are none; of two f32 factors two of up to 2^-23 each, 2^-22
// of the product at most; of f32 and f16 one of them. So scores, outputs and states are
// f32 sums of products exact to 2^-22 or better whatever the output's type: 16-bit
// outputs are the f32 ones, rounded once.
//
// Layouts. A 16x16x32 operand's lane (li, lg) = (lane % 16, lane / 16) holds eight
// k-values of row li; the accumulator's lane holds column li of rows 4 lg + r.
//  * S is accumulated as D[dk][dv] = K^T V: two row tiles (32 dk) are then, as they
//    lie, an operand over dk whose slot 8 lg + e is index 4 lg + e (e < 4) or
//    16 + 4 lg + e - 4, and Q is read in that order: S never leaves its registers.
//  * K^T and V^T operands are transposing LDS reads (ds_read_b64_tr_b16) of the
//    row-major K and V tiles; P's columns and the weights are stored in their token order.
//  * P is formed transposed, D[j][t], so that a lane holds four consecutive j of one
//    t and stores them in pairs; it is shared through LDS because the waves split dv.
//  * O is formed as D[dv][t]. A wave's NT tiles take its dv rows in groups of four in
//    turn (row 4 g + i of tile v is row 4 NT g + 4 v + i of the wave's), so that a lane
//    holds 4 NT consecutive dv of one t.
// LDS pitches are an odd number of 16-byte blocks: 16 rows of a column, or 16
// 32-byte row pieces of a transposing read, fall into different banks.
//
// 4096 tokens, 32 heads of 128 x 128, bf16: 90 us (launches of 34, 12 and 51); 8 sequences of 30,208 tokens in all:
// 364-382 (with P and the state in two parts in the outputs of 16 bits 84 and 323, but 2^-15 of a term off, always towards
// zero). 4096 tokens in f16 113, in f32 173. Bound by matrix and vector instructions: the 1920 products of the two
// chunks that a CU works on at a time take 7.7 K clocks; the rest is splitting into parts, decays and LDS reads.
#pragma once

#include "gdn_device.h"
#include "gdn_ops.h"

namespace gdn {
namespace linattn {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// bf16 parts of an f32 value, and the order up to which products of parts are taken
constexpr int kParts = 3, kOrder = 2;
// bf16 parts of an input of dtype QT
constexpr int input_parts(int qt) { return qt == DT_BF16 ? 1 : qt == DT_F16 ? 2 : 3; }

// A workgroup covers DV of a head's dv rows (all of them up to 128; two workgroups share
// a head of 256), NT tiles of 16 to a wave: two where the registers allow it, which halve the LDS reads of K^T, Q
// and P against one.
template <int DK, int DV, int QT>
struct Geo {
    static constexpr int IP = input_parts(QT);
    static constexpr int NT = DV == 128 && DK <= 128 ? 2 : 1;
    static constexpr int W = DV / (16 * NT);
    static constexpr int THREADS = 64 * W;
    static constexpr int PK = DK * 2 + 16, PV = DV * 2 + 16;  // row pitches, bytes
    static constexpr int lds(int c)
    {
        return IP * c * (2 * PK + PV) + kParts * c * (2 * c + 16) + 20 * c + c * (c - 16) / 8 + 32;
    }
    // Tokens per chunk: 64, or 32 where two workgroups then fit a CU's 160 KB and registers (4096 tokens, 32 heads,
    // us with 64 and 32: f16 128 x 128 134 113, 96 x 96 104 88, 64 x 64 71 56; f32 64 x 64 85 66, 128 x 64 119 93, 96 x 96,
    // where registers leave one workgroup, 126 133) or where 64 do not fit at all
    static constexpr int kLds = 160 * 1024;
    static constexpr bool PAIR = 2 * lds(64) > kLds && 2 * lds(32) <= kLds && (W <= 4 || (W <= 6 && QT != DT_F32));
    static constexpr int C = PAIR || lds(64) > kLds ? 32 : 64;
};
constexpr int rows_per_workgroup(int dv) { return dv > 128 ? 128 : dv; }

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Cuts the leading bf16 off x: returns its bits (upper half of a word) and leaves the
// rest in x (NaN of an infinity).
__device__ __forceinline__ uint32_t cut(float &x)
{
    const uint32_t h = __float_as_uint(x) & 0xffff0000u;
    x -= __uint_as_float(h);
    return h;
}

// Rounds lo and hi to bf16 (to nearest even): returns their bits as one word, lo's below hi's, and leaves the rests.
__device__ __forceinline__ uint32_t round2(float &lo, float &hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const uint32_t w = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
    lo -= __uint_as_float(w << 16);
    hi -= __uint_as_float(w & 0xffff0000u);
    return w;
}

// The upper halves of two words as one: lo's below hi's.
__device__ __forceinline__ uint32_t pack_hi(uint32_t lo, uint32_t hi)
{
    return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

// Eight values as PARTS operands of eight bf16 (the last part has what is left, which fits).
template <int PARTS>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&out)[PARTS])
{
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        r[e] = x[e];
#pragma unroll
    for (int s = 0; s < PARTS; ++s) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (s == PARTS - 1) {
                w[e] = pack_hi(__float_as_uint(r[2 * e]), __float_as_uint(r[2 * e + 1]));
            } else if (s > 0) {
                w[e] = round2(r[2 * e], r[2 * e + 1]);
            } else {
                const uint32_t lo = cut(r[2 * e]), hi = cut(r[2 * e + 1]);
                w[e] = pack_hi(lo, hi);
            }
        }
        __builtin_memcpy(&out[s], w, 16);
    }
}

// The value of parts, from the last on: the first two alone may be a rounding above f32's largest number.
template <int PARTS>
__device__ __forceinline__ float join(const bf16x8 (&p)[PARTS], int e)
{
    float x = (float)p[PARTS - 1][e];
#pragma unroll
    for (int s = PARTS - 2; s >= 0; --s)
        x += (float)p[s][e];
    return x;
}

// Eight consecutive activations as loaded, and as bf16 parts.
template <int QT>
struct Raw8 {
    uint32_t w[QT == DT_F32 ? 8 : 4];
};

// A buffer of `bytes` from a scalar base: one 32-bit lane offset addresses it, loads past its end give 0 and
// stores there are dropped.
typedef __amdgpu_buffer_rsrc_t Buffer;
__device__ __forceinline__ Buffer buffer_of(const void *base, uint32_t bytes)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}

template <int QT>
__device__ __forceinline__ Raw8<QT> load_raw8(Buffer b, uint32_t off)
{
    Raw8<QT> r;
#pragma unroll
    for (int i = 0; i < (QT == DT_F32 ? 2 : 1); ++i) {
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(b, off + 16 * i, 0, 0);
        __builtin_memcpy(r.w + 4 * i, &v, 16);
    }
    return r;
}

template <int QT>
__device__ __forceinline__ void raw8_parts(const Raw8<QT> &r, bf16x8 (&out)[input_parts(QT)])
{
    if constexpr (QT == DT_BF16) {
        __builtin_memcpy(&out[0], r.w, 16);
    } else {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = QT == DT_F32 ? __uint_as_float(r.w[e % (sizeof(r.w) / 4)])
                                : f16_bits_to_f32(e & 1 ? r.w[e / 2] >> 16 : r.w[e / 2] & 0xffffu);
        split8<input_parts(QT)>(x, out);
    }
}

// A tile of C rows of D elements on its way from global memory to the LDS parts. A
// thread's units (8 elements) are STEP rows apart.
template <int QT, int C, int D, int THREADS>
struct Tile {
    static constexpr int U = C * D / 8, N = U / THREADS, STEP = THREADS * 8 / D, PITCH = D * 2 + 16;
    static constexpr int ES = QT == DT_F32 ? 4 : 2;
    static_assert(U % THREADS == 0 && THREADS * 8 % D == 0, "units split evenly over the threads, whole rows apart");
    Raw8<QT> r[N];

    // rows [0, n) of the tile at `base`, rows `stride` bytes apart (below 2^26: the host checks, so that a
    // tile's offsets fit 32 bits); those past them are 0, and all of them where n <= 0
    struct From {
        Buffer b;
        uint32_t off, step;
    };
    static __device__ __forceinline__ From from(const char *base, uint32_t stride, int n, int tid)
    {
        return From{buffer_of(base, n > 0 ? (uint32_t)(min(n, C) - 1) * stride + D * ES : 0),
                    tid / (D / 8) * stride + tid % (D / 8) * 8 * ES, STEP * stride};
    }
    // the units that fall to part `part` of `parts`
    __device__ __forceinline__ void load(const From &f, int part = 0, int parts = 1)
    {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * parts / N == part)
                r[i] = load_raw8<QT>(f.b, f.off + i * f.step);
    }
    __device__ __forceinline__ void store(unsigned char *lds, int tid) const
    {
        const int row = tid / (D / 8), c = tid % (D / 8) * 8;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            bf16x8 part[input_parts(QT)];
            raw8_parts<QT>(r[i], part);
#pragma unroll
            for (int s = 0; s < input_parts(QT); ++s)
                *reinterpret_cast<bf16x8 *>(lds + s * C * PITCH + (row + i * STEP) * PITCH + 2 * c) = part[s];
        }
    }
};

// N consecutive outputs (4 or 8) at a byte offset, as 16- or 8-byte stores (the host checks the alignment).
template <bool F32, int N>
__device__ __forceinline__ void store_out(Buffer b, uint32_t off, int dt, const float (&x)[N])
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            u32x4 w;
            __builtin_memcpy(&w, x + i, 16);
            __builtin_amdgcn_raw_buffer_store_b128(w, b, off + 4 * i, 0, 0);
        }
    } else {
        uint16_t y[N];
        if (dt == DT_BF16) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                y[i] = __builtin_bit_cast(uint16_t, (__bf16)x[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                y[i] = __builtin_bit_cast(uint16_t, (_Float16)x[i]);
        }
        if constexpr (N == 8) {
            u32x4 w;
            __builtin_memcpy(&w, y, 16);
            __builtin_amdgcn_raw_buffer_store_b128(w, b, off, 0, 0);
        } else {
            u32x2 w;
            __builtin_memcpy(&w, y, 8);
            __builtin_amdgcn_raw_buffer_store_b64(w, b, off, 0, 0);
        }
    }
}

__device__ __forceinline__ bf16x8 lds8(const unsigned char *p) { return *reinterpret_cast<const bf16x8 *>(p); }

// Eight k-values of one row in the accumulator pair's slot order: 4 at p, 4 at p + 16 elements.
__device__ __forceinline__ bf16x8 lds4x2(const unsigned char *p)
{
    uint2 w[2] = {*reinterpret_cast<const uint2 *>(p), *reinterpret_cast<const uint2 *>(p + 32)};
    bf16x8 v;
    __builtin_memcpy(&v, w, 16);
    return v;
}

// Token j of a chunk as a k-value of an operand: the 32 tokens of a product go to its slots 8 lg + e so that
// lane group lg's four rows of a transposing read (e < 4, and 16 on for e >= 4) are two apart and the groups
// that the LDS serves together, 0 with 1 and 2 with 3, cover 8 even or 8 odd rows: rows one 16-byte block
// past a multiple of all banks apart then fall into different banks (consecutive rows overlap by half).
__device__ __forceinline__ int token_of(int lg, int e) { return 8 * (lg & 1) + (lg >> 1) + 2 * (e & 3) + 4 * (e & 4); }
__device__ __forceinline__ int slot_of(int j)
{
    return (j & ~31) + 8 * (((j >> 3) & 1) + 2 * (j & 1)) + ((j >> 1) & 3) + ((j >> 2) & 4);
}

// Transposed operand of a row-major bf16 tile: rows row0 + token_of(lg, e) of column c0 + gap (li / 4) + li % 4.
// A transposing read hands lane i of 16 column i of the four rows whose 16 columns, in groups of four, the lanes
// point at.
__device__ __forceinline__ bf16x8 lds_tr8(unsigned char *tile, int pitch, int row0, int c0, int gap, int li, int lg)
{
    unsigned char *p = tile + (row0 + token_of(lg, li >> 2)) * pitch + 2 * (c0 + gap * (li & 3));
    s16x4 w[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p),
                  __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 16 * pitch))};
    bf16x8 v;
    __builtin_memcpy(&v, w, 16);
    return v;
}

// Log decays at most as low as this count as exp = 0 (f32 reaches 0 at -104); a finite
// bound keeps differences of prefix sums finite. In f64 the sums still resolve 2^-30 of
// a small decay beside it.
constexpr double kLowest = -1e4;

// How a sequence of `len` tokens is cut: one segment up to L tokens, else L0 tokens and then L at a time. (Only
// the first segment is walked with its outputs in the first launch; that takes twice as long as the others' states.)
struct Cut {
    int L, L0;
    __host__ __device__ int segments(int len) const { return len <= L ? (len > 0 ? 1 : 0) : 2 + (len - L0 - 1) / L; }
};

__device__ __forceinline__ float lane_value(float x, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ int lane_sum(int x)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(x, d, 64);
        x += lane >= d ? o : 0;
    }
    return x;
}

// The states between segments of the sequences before `seq`.
__device__ __forceinline__ int slots_before(const int32_t *cu, Cut cut, int seq)
{
    int slots = 0;
    for (int s0 = 0; s0 < seq; s0 += 64) {
        const int s = s0 + (threadIdx.x & 63);
        const int n = s < seq ? cut.segments(cu[s + 1] - cu[s]) : 0;
        slots += __builtin_amdgcn_readlane(lane_sum(n > 1 ? n - 1 : 0), 63);
    }
    return slots;
}

// Segments are dealt out longest first, by kind: every sequence's first, those between, the last of several.
enum SegmentKind { kFirst, kBetween, kLast };
struct Segment {
    int seq, seg, segs, start, len;
    int slot0;  // of the sequence's states after its segments but the last
};
// Segment `idx` of a kind; len 0 if there is none. Every sequence counts for one of the first kind, so that many
// short sequences need no search; else every lane counts for one of 64 sequences at a time.
__device__ __forceinline__ Segment find_segment(const int32_t *cu, int N, Cut cut, int kind, int idx)
{
    if (kind == kFirst) {
        const int start = cu[idx], len = cu[idx + 1] - start, segs = cut.segments(len);
        return Segment{idx, 0, segs, start, segs > 1 ? cut.L0 : len, segs > 1 ? slots_before(cu, cut, idx) : 0};
    }
    const int lane = threadIdx.x & 63;
    int before = 0, slots_upto_here = 0;
    for (int s0 = 0; s0 < N; s0 += 64) {
        const int s = s0 + lane;
        const int start = s < N ? cu[s] : 0, len = s < N ? cu[s + 1] - start : 0;
        const int segs = cut.segments(len), slots = max(segs - 1, 0);
        const int cnt = kind == kBetween ? max(segs - 2, 0) : min(slots, 1);
        const int upto = lane_sum(cnt), slots_upto = lane_sum(slots);
        const uint64_t hit = __ballot(idx >= before + upto - cnt && idx < before + upto);
        if (hit) {
            // scalar reads: what follows from the segment stays in scalar registers
            const int src = __builtin_ctzll(hit);
            Segment r;
            r.seq = s0 + src;
            r.segs = __builtin_amdgcn_readlane(segs, src);
            const int nth = idx - before - __builtin_amdgcn_readlane(upto - cnt, src);
            r.seg = kind == kBetween ? 1 + nth : r.segs - 1;
            const int from = cut.L0 + (r.seg - 1) * cut.L;
            r.start = __builtin_amdgcn_readlane(start, src) + from;
            r.len = min(cut.L, __builtin_amdgcn_readlane(len, src) - from);
            r.slot0 = slots_upto_here + __builtin_amdgcn_readlane(slots_upto - slots, src);
            return r;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
        slots_upto_here += __builtin_amdgcn_readlane(slots_upto, 63);
    }
    return Segment{0, 0, 0, 0, 0, 0};
}

template <int DK, int DV, int QT, bool F32OUT>
struct Walk {
    using G = Geo<DK, DV, QT>;
    static constexpr int IP = G::IP, C = G::C, NT = G::NT, W = G::W, THREADS = G::THREADS;
    static constexpr int PK = G::PK, PV = G::PV, PP = 2 * C + 16;
    static constexpr int OP = kParts;
    static constexpr int KT = DK / 16, KS = DK / 32, TT = C / 16, JS = C / 32;

    struct __align__(16) Lds {
        unsigned char q[IP * C * PK], k[IP * C * PK], v[IP * C * PV], p[OP * C * PP];
        float2 g[C];        // prefix sums of the log decays in base 2, as the sum of two f32
        // e^(G_t - G_j) of the tiles left of the diagonal, as the product of a row's and a column's factor about the
        // row tile's first token r: e^(G_t - G_r) and scale e^(G_r - G_j)
        float row[C], col[8 * TT * (TT - 1)];  // row tile i's 16 i columns from col_at(i) on
        float eg[C], w[C];  // scale e^G_t and e^(G_last - G_t)
        float decay;        // e^G_last
        double last;        // G_last
    };

    static constexpr int col_at(int i) { return 8 * i * (i - 1); }

    // waves per SIMD that the registers leave room for: those of two workgroups, where their LDS fits
    static constexpr int WAVES = 2 * sizeof(Lds) <= 160 * 1024 && W == 4 ? 2 : 1;

    // x of the lane that DPP control CTRL names, 0 where there is none or the row is masked out
    template <int CTRL, int ROWS>
    static __device__ __forceinline__ double dpp_f64(double x)
    {
        int w[2];
        __builtin_memcpy(w, &x, 8);
        w[0] = __builtin_amdgcn_update_dpp(0, w[0], CTRL, ROWS, 0xF, false);
        w[1] = __builtin_amdgcn_update_dpp(0, w[1], CTRL, ROWS, 0xF, false);
        __builtin_memcpy(&x, w, 8);
        return x;
    }
    // Prefix sum of the lanes' log decays, in f64: within rows of 16 lanes (row_shr 1, 2, 4, 8), then a row's
    // total to the next (row_bcast 15) and the first half's to the second (row_bcast 31)
    static __device__ __forceinline__ double prefix(double g)
    {
        double s = g < kLowest ? kLowest : g;
        s += dpp_f64<0x111, 0xF>(s);
        s += dpp_f64<0x112, 0xF>(s);
        s += dpp_f64<0x114, 0xF>(s);
        s += dpp_f64<0x118, 0xF>(s);
        s += dpp_f64<0x142, 0xA>(s);
        s += dpp_f64<0x143, 0xC>(s);
        return s;
    }

    // Walks the segment's chunks from the state at `in` (NULL: zero) and stores the state after them at
    // `out_state` (unless NULL); OUT: with the tokens' outputs. Returns the segment's summed log decay. in, out_state and
    // dvh are those of the workgroup's DV rows, the first of which is row dvh of the head.
    template <bool OUT>
    static __device__ __forceinline__ double run(Lds &l, const LinattnParams &p, const Segment sg, int h, int dvh,
                                                 const float *in, float *out_state)
    {
        int tid = threadIdx.x;
        int lane = tid & 63, li = lane & 15, lg = lane >> 4;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int kh = k_head_of(p.hc.head_map, h, p.hc.Hk, p.hc.Hv);
        const int dv0 = wave * 16 * NT;
        const int row0 = dv0 + 4 * NT * (li >> 2) + (li & 3);  // the lane's state row of tile 0; tile v's is 4 v on
        const bool head_decay = p.hc.flags & F_HEAD_DECAY;
        double rate = 0.0;
        if (head_decay) {
            const float d = p.in.decay_param[h];
            rate = p.hc.decay_kind == 0 ? -expf(d) : d;
        }

        f32x4 S[KT][NT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int v = 0; v < NT; ++v)
                S[kt][v] = in ? *reinterpret_cast<const f32x4 *>(in + (row0 + 4 * v) * DK + 16 * kt + 4 * lg)
                              : f32x4{0.f, 0.f, 0.f, 0.f};

        // The next chunk's rows are fetched a tile at a time between the current one's products
        Tile<QT, C, DK, THREADS> tq, tk;
        Tile<QT, C, DV, THREADS> tv;
        constexpr int ES = Tile<QT, C, DK, THREADS>::ES;
        const uint32_t qs = (uint32_t)(p.in.q_stride * ES), ks_ = (uint32_t)(p.in.k_stride * ES), vs = (uint32_t)(p.in.v_stride * ES);
        const char *qp = static_cast<const char *>(p.in.q) + (sg.start * p.in.q_stride + (int64_t)kh * DK) * ES;
        const char *kp = static_cast<const char *>(p.in.k) + (sg.start * p.in.k_stride + (int64_t)kh * DK) * ES;
        const char *vp = static_cast<const char *>(p.in.v) + (sg.start * p.in.v_stride + (int64_t)h * p.hc.dv + dvh) * ES;
        double tg = 0.0, last = 0.0;
        float graw = 0.f, te = 0.f, tw = 0.f, trow = 0.f, tcol[TT - 1];
        float2 g2 = {0.f, 0.f};
        using TK = Tile<QT, C, DK, THREADS>;
        using TV = Tile<QT, C, DV, THREADS>;
        auto from_q = [&](int c0) { return TK::from(qp + (int64_t)c0 * qs, qs, sg.len - c0, tid); };
        auto from_k = [&](int c0) { return TK::from(kp + (int64_t)c0 * ks_, ks_, sg.len - c0, tid); };
        auto from_v = [&](int c0) { return TV::from(vp + (int64_t)c0 * vs, vs, sg.len - c0, tid); };
        auto fetch_g = [&](int c0) {
            if (wave == W - 1 && !head_decay)
                graw = p.in.g[((int64_t)sg.start + c0 + min(lane, sg.len - c0 - 1)) * p.hc.Hv + h];
        };
        // the last wave turns the fetched decays into the chunk's decay rows before the others need them
        auto scan = [&](int c0) {
            if (wave == W - 1) {
                tg = prefix(lane < sg.len - c0 && lane < C ? (head_decay ? rate : (double)graw) : 0.0);
                int w[2];
                __builtin_memcpy(w, &tg, 8);
                w[0] = __builtin_amdgcn_readlane(w[0], C - 1);
                w[1] = __builtin_amdgcn_readlane(w[1], C - 1);
                __builtin_memcpy(&last, w, 8);
                te = expf((float)tg);
                tw = lane < sg.len - c0 ? expf((float)(last - tg)) : 0.f;
                if constexpr (OUT) {
                    constexpr double kLog2e = 1.4426950408889634;
                    const float hi = (float)(tg * kLog2e);
                    g2 = make_float2(hi, (float)(tg * kLog2e - hi));
                    trow = 1.f;
#pragma unroll
                    for (int i = 1; i < TT; ++i) {
                        const float rx = lane_value(g2.x, 16 * i), ry = lane_value(g2.y, 16 * i);
                        const float d = (rx - g2.x) + (ry - g2.y);
                        if (i == (lane >> 4))
                            trow = __builtin_amdgcn_exp2f(-d);
                        tcol[i - 1] = p.hc.scale * __builtin_amdgcn_exp2f(d);  // read left of row tile i only
                    }
                    if (lane < 16) {
                        const float rx = lane_value(g2.x, 0), ry = lane_value(g2.y, 0);
                        trow = __builtin_amdgcn_exp2f((g2.x - rx) + (g2.y - ry));
                    }
                }
            }
        };
        auto stage = [&] {
            tk.store(l.k, tid);
            tv.store(l.v, tid);
            if (wave == W - 1 && lane < C) {
                if constexpr (OUT) {
                    l.g[lane] = g2;
                    l.row[lane] = trow;
#pragma unroll
                    for (int i = 1; i < TT; ++i)
                        if (lane < 16 * i)
                            l.col[col_at(i) + lane] = tcol[i - 1];
                }
                l.eg[lane] = p.hc.scale * te;
                l.w[slot_of(lane)] = tw;
                if (lane == C - 1) {
                    l.decay = te;
                    l.last = last;
                }
            }
        };
        if constexpr (OUT) {
            // the P tiles right of the diagonal that the 32-wide products reach: tokens 16 .. 31 of the
            // product's, slots 8 lg + 4 .. + 7
            for (int u = threadIdx.x; u < OP * (TT / 2) * 16 * 4; u += THREADS) {
                const int s = u / (TT / 2 * 64), it = u / 64 % (TT / 2) * 2, row = u / 4 % 16, g = u % 4;
                *reinterpret_cast<uint2 *>(l.p + s * C * PP + (16 * it + row) * PP + 2 * (16 * it + 8 * g + 4)) = make_uint2(0, 0);
            }
        }
        fetch_g(0);
        tk.load(from_k(0));
        if constexpr (OUT)
            tq.load(from_q(0));
        tv.load(from_v(0));
        scan(0);
        if constexpr (OUT)
            tq.store(l.q, tid);
        stage();
        __syncthreads();

        double total = 0.0;
        for (int c0 = 0; c0 < sg.len; c0 += C) {
            const bool more = c0 + C < sg.len;
            // the lane's LDS and buffer offsets are formed anew in each chunk: kept across the loop, some forty
            // of them push the tiles into scratch, whose reloads wait for the fetches in flight
            asm volatile("" : "+v"(tid));
            lane = tid & 63;
            li = lane & 15;
            lg = lane >> 4;
            f32x4 O[OUT ? TT : 1][NT];
            if constexpr (OUT) {
                // P = tril(Q K^T) . e^(G_t - G_j), the 16 x 16 tiles (it, jt) on and below the diagonal dealt to
                // the waves, and O = scale diag(e^G) Q S^T
                constexpr int TILES = TT * (TT + 1) / 2, MINE = (TILES + W - 1) / W;
                constexpr bool MERGED = TT == 4 && W == 4;
                f32x4 a[MINE];
                int it[MINE], jt[MINE];
                if constexpr (MERGED) {
                    // Both in one loop over dk, on the same Q operands (Q and K in the state's slot order). Wave w
                    // takes tiles (1, w), (2, w), (3, w); the two of these that wave 2 and 3 have above the diagonal
                    // leave room for (0, 0) at wave 2 and for the decays at wave 3, whose one tile is (3, 3).
                    it[0] = wave == 2 ? 0 : 1;
                    it[1] = 2;
                    it[2] = 3;
                    jt[0] = wave == 2 ? 0 : wave;
                    jt[1] = jt[2] = wave;
                } else {
#pragma unroll
                    for (int m = 0; m < MINE; ++m) {
                        const int idx = min(wave + m * W, TILES - 1);  // one too many repeats the last tile
                        it[m] = 0;
#pragma unroll
                        for (int i = 1; i < TT; ++i)
                            it[m] += idx >= i * (i + 1) / 2 ? 1 : 0;
                        jt[m] = idx - it[m] * (it[m] + 1) / 2;
                    }
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                        for (int m = 0; m < MINE; ++m)
#pragma unroll
                            for (int x = 0; x < IP; ++x)
#pragma unroll
                                for (int y = 0; y < IP; ++y)
                                    if (x + y <= kOrder)
                                        a[m] = mfma(lds8(l.k + x * C * PK + (16 * jt[m] + li) * PK + 64 * ks + 16 * lg),
                                                    lds8(l.q + y * C * PK + (16 * it[m] + li) * PK + 64 * ks + 16 * lg),
                                                    ks + x + y == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : a[m]);
                        if (ks % 2)
                            __builtin_amdgcn_sched_barrier(0);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
                // the next chunk's k and q rows are fetched between these products, its v rows between P's
                if (more)
                    fetch_g(c0 + C);
                const typename TK::From fk = from_k(c0 + C), fq = from_q(c0 + C);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    tk.load(fk, ks, KS);
                    tq.load(fq, ks, KS);
                    bf16x8 sp[NT][OP];
#pragma unroll
                    for (int v = 0; v < NT; ++v) {
                        const f32x4 s0 = S[2 * ks][v], s1 = S[2 * ks + 1][v];
                        const float x[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
                        split8<OP>(x, sp[v]);
                    }
                    bf16x8 q[TT][IP];
#pragma unroll
                    for (int i = 0; i < TT; ++i)
#pragma unroll
                        for (int y = 0; y < IP; ++y)
                            q[i][y] = lds4x2(l.q + y * C * PK + (16 * i + li) * PK + 64 * ks + 8 * lg);
                    if constexpr (MERGED) {
#pragma unroll
                        for (int x = 0; x < IP; ++x) {
                            const unsigned char *kp = l.k + x * C * PK + li * PK + 64 * ks + 8 * lg;
                            const bf16x8 k0 = lds4x2(kp + 16 * jt[0] * PK), k1 = lds4x2(kp + 16 * jt[1] * PK);
#pragma unroll
                            for (int y = 0; y < IP; ++y)
                                if (x + y <= kOrder) {
                                    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
                                    a[0] = mfma(k0, wave == 2 ? q[0][y] : q[1][y], ks + x + y == 0 ? zero : a[0]);
                                    a[1] = mfma(k1, q[2][y], ks + x + y == 0 ? zero : a[1]);
                                    a[2] = mfma(k1, q[3][y], ks + x + y == 0 ? zero : a[2]);
                                }
                        }
                    }
#pragma unroll
                    for (int i = 0; i < TT; ++i)
#pragma unroll
                        for (int y = 0; y < IP; ++y)
#pragma unroll
                            for (int v = 0; v < NT; ++v)
#pragma unroll
                                for (int s = 0; s < OP; ++s)
                                    if (s + y <= kOrder)
                                        O[i][v] = mfma(sp[v][s], q[i][y], ks + y + s == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : O[i][v]);
                    __builtin_amdgcn_sched_barrier(0);  // or every step's reads are issued first, into spills
                }
#pragma unroll
                for (int m = 0; m < MINE; ++m) {
                    if (MERGED && jt[m] > it[m])
                        continue;
                    const int t = 16 * it[m] + li, j0 = 16 * jt[m] + 4 * lg;
                    float x[4];
                    if (jt[m] < it[m]) {
                        const float row = l.row[t];
                        const f32x4 col = *reinterpret_cast<const f32x4 *>(&l.col[col_at(it[m]) + j0]);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            x[r] = a[m][r] * (row * col[r]);
                    } else {
                        const float2 gt = l.g[t];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float2 gj = l.g[j0 + r];
                            x[r] = a[m][r] * (p.hc.scale * __builtin_amdgcn_exp2f((gt.x - gj.x) + (gt.y - gj.y)));
                            asm volatile("" : "+v"(x[r]));  // taken for every lane: no branch around each exponential
                            x[r] = j0 + r <= t ? x[r] : 0.f;
                        }
                    }
                    // tokens 4 lg .. + 3 of the tile: two pairs of neighbouring slots
                    unsigned char *at = l.p + t * PP + 2 * slot_of(j0);
#pragma unroll
                    for (int s = 0; s < OP; ++s) {
                        uint32_t even, odd;
                        if (s == 1) {
                            even = round2(x[0], x[2]);
                            odd = round2(x[1], x[3]);
                        } else {
                            even = pack_hi(__float_as_uint(x[0]), __float_as_uint(x[2]));
                            odd = pack_hi(__float_as_uint(x[1]), __float_as_uint(x[3]));
                        }
                        if (s == 0) {
                            cut(x[0]);
                            cut(x[1]);
                            cut(x[2]);
                            cut(x[3]);
                        }
                        *reinterpret_cast<uint32_t *>(at + s * C * PP) = even;
                        *reinterpret_cast<uint32_t *>(at + s * C * PP + 32) = odd;
                    }
                }
#pragma unroll
                for (int i = 0; i < TT; ++i) {
                    const float e = l.eg[16 * i + li];
#pragma unroll
                    for (int v = 0; v < NT; ++v)
                        O[i][v] *= e;
                }
                if (more)
                    scan(c0 + C);
                __syncthreads();  // P is whole, and the chunk's q rows are no longer read
                if (more)
                    tq.store(l.q, tid);
            } else if (more) {
                fetch_g(c0 + C);
                tk.load(from_k(c0 + C));
                tv.load(from_v(c0 + C));
            }
            // V^T operands: dv as the row, tokens as k
            bf16x8 vt[JS][NT][IP];
#pragma unroll
            for (int js = 0; js < JS; ++js)
#pragma unroll
                for (int v = 0; v < NT; ++v)
#pragma unroll
                    for (int x = 0; x < IP; ++x)
                        vt[js][v][x] = lds_tr8(l.v + x * C * PV, PV, 32 * js, dv0 + 4 * v, 4 * NT, li, lg);
            if constexpr (OUT) {
                const typename TV::From fv = from_v(c0 + C);
                // a V that is not finite: 0 times it, right of the diagonal, is not 0
                typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
                u16x2 top = {0, 0};
#pragma unroll
                for (int js = 0; js < JS; ++js)
#pragma unroll
                    for (int v = 0; v < NT; ++v) {
                        u16x2 w[4];
                        __builtin_memcpy(w, &vt[js][v][0], 16);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            top = __builtin_elementwise_max(top, w[e] & (uint16_t)0x7fff);
                    }
                if (__ballot(top[0] >= 0x7f80 || top[1] >= 0x7f80) == 0) {
                    tv.load(fv);
#pragma unroll
                    for (int it = 0; it < TT; ++it)
#pragma unroll
                        for (int js = 0; js <= it / 2; ++js)
#pragma unroll
                            for (int s = 0; s < OP; ++s) {
                                const bf16x8 pt = lds8(l.p + s * C * PP + (16 * it + li) * PP + 64 * js + 16 * lg);
#pragma unroll
                                for (int v = 0; v < NT; ++v)
#pragma unroll
                                    for (int x = 0; x < IP; ++x)
                                        if (s + x <= kOrder)
                                            O[it][v] = mfma(vt[js][v][x], pt, O[it][v]);
                            }
                } else {
                    tv.load(fv);
                    // term by term, the tokens up to t alone
                    for (int j = 0; j < C; ++j)
#pragma unroll
                        for (int it = 0; it < TT; ++it)
                            if (j <= 16 * it + li) {
                                float pj = 0.f;
#pragma unroll
                                for (int s = OP - 1; s >= 0; --s)
                                    pj += bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(
                                        l.p + s * C * PP + (16 * it + li) * PP + 2 * slot_of(j)));
#pragma unroll
                                for (int v = 0; v < NT; ++v)
#pragma unroll
                                    for (int r = 0; r < 4; ++r) {
                                        float x = 0.f;
#pragma unroll
                                        for (int y = IP - 1; y >= 0; --y)
                                            x += bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(
                                                l.v + y * C * PV + j * PV + 2 * (dv0 + 4 * NT * lg + 4 * v + r)));
                                        O[it][v][r] = fmaf(pj, x, O[it][v][r]);
                                    }
                            }
                }
                constexpr int OES = F32OUT ? 4 : 2;
                const uint32_t os = (uint32_t)(p.hc.Hv * p.hc.dv) * OES;
                const Buffer ob = buffer_of(static_cast<char *>(p.out) +
                                                (((int64_t)sg.start + c0) * p.hc.Hv + h) * p.hc.dv * OES,
                                            (uint32_t)(min(sg.len - c0, C) - 1) * os + p.hc.dv * OES);
#pragma unroll
                for (int it = 0; it < TT; ++it) {
                    float x[4 * NT];
#pragma unroll
                    for (int e = 0; e < 4 * NT; ++e)
                        x[e] = O[it][e / 4][e % 4];
                    store_out<F32OUT>(ob, (16 * it + li) * os + (dvh + dv0 + 4 * NT * lg) * OES, p.out_dt, x);
                }
            }
            // S <- e^G_last S + K^T diag(w) V
            const float dec = l.decay;
            total += l.last;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int v = 0; v < NT; ++v)
                    S[kt][v] *= dec;
#pragma unroll
            for (int js = 0; js < JS; ++js) {
                const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&l.w[32 * js + 8 * lg]);
                const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&l.w[32 * js + 8 * lg + 4]);
                bf16x8 vd[NT][kParts];
#pragma unroll
                for (int v = 0; v < NT; ++v) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = join<IP>(vt[js][v], e) * (e < 4 ? w0[e & 3] : w1[e & 3]);
                    split8<kParts>(x, vd[v]);
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int y = 0; y < IP; ++y) {
                        const bf16x8 k = lds_tr8(l.k + y * C * PK, PK, 32 * js, 16 * kt, 4, li, lg);
#pragma unroll
                        for (int v = 0; v < NT; ++v)
#pragma unroll
                            for (int s = 0; s < kParts; ++s)
                                if (s + y <= kOrder)
                                    S[kt][v] = mfma(k, vd[v][s], S[kt][v]);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (!OUT) {
                if (more)
                    scan(c0 + C);
            }
            __syncthreads();  // every wave is done with the chunk's tiles
            if (more) {
                stage();
                __syncthreads();
            }
        }
        if (!out_state)
            return total;
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int v = 0; v < NT; ++v)
                *reinterpret_cast<f32x4 *>(out_state + (row0 + 4 * v) * DK + 16 * kt + 4 * lg) = S[kt][v];
        return total;
    }
};

// Blocks: segments (the launch's first kind, then its second), then heads, then a head's parts of DV rows.
template <int DK, int DV, int QT, bool F32OUT, bool SECOND>
__global__ __launch_bounds__((Geo<DK, DV, QT>::THREADS), (Walk<DK, DV, QT, F32OUT>::WAVES)) void chunk_kernel(const LinattnParams p)
{
    using Wk = Walk<DK, DV, QT, F32OUT>;
    __shared__ typename Wk::Lds l;
    const int parts = p.hc.dv / DV, dvh = blockIdx.x % parts * DV;
    const int h = blockIdx.x / parts % p.hc.Hv;
    const int idx = blockIdx.x / parts / p.hc.Hv, one = SECOND ? p.segs_between : p.segs_first;
    const Cut cut{p.seg_tokens, p.seg_first_tokens};
    const Segment sg = find_segment(p.cu, p.N, cut, idx < one ? (SECOND ? kBetween : kFirst) : (SECOND ? kLast : kBetween),
                                    idx < one ? idx : idx - one);
    if (sg.len <= 0)
        return;
    const int64_t size = (int64_t)DK * p.hc.dv, skip = (int64_t)DK * dvh;
    float *state = p.state + ((int64_t)sg.seq * p.hc.Hv + h) * size + skip;
    const int64_t slot = (int64_t)(sg.slot0 + sg.seg) * p.hc.Hv + h;
    const bool last = sg.seg == sg.segs - 1;
    float *after = last ? state : p.seg_state + slot * size + skip;
    if constexpr (SECOND) {
        // (the states between segments are read in this launch, not written)
        Wk::template run<true>(l, p, sg, h, dvh, p.seg_state + (slot - p.hc.Hv) * size + skip, last ? state : nullptr);
    } else if (sg.seg == 0) {
        Wk::template run<true>(l, p, sg, h, dvh, state, after);
    } else {
        const double g = Wk::template run<false>(l, p, sg, h, dvh, nullptr, after);
        if (threadIdx.x == 0 && dvh == 0)
            p.seg_decay[slot] = (float)g;
    }
}

template <int DK, int DV, int QT, bool F32OUT>
hipError_t launch_chunk(const LinattnParams &p, int64_t segments, bool second, hipStream_t s)
{
    constexpr int threads = Geo<DK, DV, QT>::THREADS;
    const unsigned blocks = (unsigned)(segments * p.hc.Hv * (p.hc.dv / DV));
    if (second)
        chunk_kernel<DK, DV, QT, F32OUT, true><<<blocks, threads, 0, s>>>(p);
    else
        chunk_kernel<DK, DV, QT, F32OUT, false><<<blocks, threads, 0, s>>>(p);
    return hipGetLastError();
}

template <int QT>
hipError_t launch_chunk_for(const LinattnParams &p, int64_t segments, bool second, hipStream_t s)
{
    const int dk = p.hc.dk, dv = rows_per_workgroup(p.hc.dv);
#define GDN_CHUNK(DK, DV)                                                             \
    if (dk == DK && dv == DV)                                                         \
        return p.out_dt == DT_F32 ? launch_chunk<DK, DV, QT, true>(p, segments, second, s) \
                                  : launch_chunk<DK, DV, QT, false>(p, segments, second, s);
    GDN_CHUNK(32, 32)
    GDN_CHUNK(64, 64)
    GDN_CHUNK(96, 96)
    GDN_CHUNK(128, 128)
    GDN_CHUNK(64, 128)
    GDN_CHUNK(128, 64)
    GDN_CHUNK(256, 128)
#undef GDN_CHUNK
    return hipErrorInvalidValue;
}

}  // namespace linattn
}  // namespace gdn
