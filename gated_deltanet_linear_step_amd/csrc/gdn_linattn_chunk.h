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
//      given state); every later segment but the last, its contribution to the state
//      alone, as if it entered with zero.
//   2. scan_kernel: entering states by a running sum over each sequence's segments.
//   3. chunk_kernel, second launch: the later segments, complete.
// A call whose sequences all have one segment is the first launch alone.
//
// Products are on v_mfma_f32_16x16x32_bf16. An operand that is not bf16 is a sum of
// bf16 parts: f16 two (exact), f32 three (exact). Parts are cut off, not rounded, so
// that no part overflows; what three leave of an f32 is zero, two leave 2^-16. Products
// of parts whose orders add up to more than LIM are left out. The state's update keeps
// 2^-24 (three parts of the decayed V, LIM 2) whatever the types: states are f32. The
// outputs keep as much for f32 outputs; for 16-bit ones P and the state are taken as
// two parts, 2^-16, two hundred times finer than the output's own rounding.
//
// Layouts. A 16x16x32 operand's lane (li, lg) = (lane % 16, lane / 16) holds eight
// k-values of row li; the accumulator's lane holds column li of rows 4 lg + r.
//  * S is accumulated as D[dk][dv] = K^T V: two row tiles (32 dk) are then, as they
//    lie, an operand over dk whose slot 8 lg + e is index 4 lg + e (e < 4) or
//    16 + 4 lg + e - 4, and Q is read in that order: S never leaves its registers.
//  * K^T and V^T operands are transposing LDS reads (ds_read_b64_tr_b16) of the
//    row-major K and V tiles.
//  * P is formed transposed, D[j][t], so that a lane holds four consecutive j of one
//    t and stores them as one LDS word pair; it is shared through LDS because the
//    waves split dv.
//  * O is formed as D[dv][t]: a lane stores four consecutive dv.
// LDS pitches are an odd number of 16-byte blocks: 16 rows of a column, or 16
// 32-byte row pieces of a transposing read, fall into different banks.
#pragma once

#include "gdn_device.h"
#include "gdn_kernels.h"

namespace gdn {
namespace linattn {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// bf16 parts of an input of dtype QT
constexpr int input_parts(int qt) { return qt == DT_BF16 ? 1 : qt == DT_F16 ? 2 : 3; }

template <int DK, int DV, int QT>
struct Geo {
    static constexpr int IP = input_parts(QT);
    // dv tiles per wave and waves: 32 dv rows a wave halve the LDS reads of K^T, Q and
    // P against 16; at dk = 256 the 16-row state alone takes the registers of it
    static constexpr int NT = (DV >= 128 && !(DK == 256 && DV == 128)) ? 2 : 1;
    static constexpr int W = DV / (16 * NT);
    static constexpr int THREADS = 64 * W;
    static constexpr int PK = DK * 2 + 16, PV = DV * 2 + 16;  // row pitches, bytes
    static constexpr int lds(int c)
    {
        return IP * c * (2 * PK + PV) + 3 * c * (2 * c + 16) + 16 * c;
    }
    static constexpr int C = lds(64) <= 160 * 1024 ? 64 : 32;
};

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Cuts the leading bf16 off x: returns its bits (upper half of a word) and leaves the
// rest in x. Nothing is left of an infinity, so that its parts add up to it.
__device__ __forceinline__ uint32_t cut(float &x)
{
    const uint32_t h = __float_as_uint(x) & 0xffff0000u;
    const float rest = x - __uint_as_float(h);
    x = __builtin_isinf(x) ? 0.f : rest;
    return h;
}

// Eight values as PARTS operands of eight bf16.
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
            const uint32_t lo = cut(r[2 * e]), hi = cut(r[2 * e + 1]);
            w[e] = (lo >> 16) | hi;
        }
        __builtin_memcpy(&out[s], w, 16);
    }
}

template <int PARTS>
__device__ __forceinline__ float join(const bf16x8 (&p)[PARTS], int e)
{
    float x = (float)p[0][e];
#pragma unroll
    for (int s = 1; s < PARTS; ++s)
        x += (float)p[s][e];
    return x;
}

// Eight consecutive activations as loaded, and as bf16 parts.
template <int QT>
struct Raw8 {
    uint32_t w[QT == DT_F32 ? 8 : 4];
};

// Activations are aligned to 4 elements (the host checks): 8 bytes of 16-bit ones.
template <int QT>
__device__ __forceinline__ Raw8<QT> load_raw8(const void *p, int64_t idx)
{
    struct __attribute__((packed, aligned(8))) Words {
        uint32_t w[4];
    };
    Raw8<QT> r;
    const char *b = static_cast<const char *>(p) + idx * (QT == DT_F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < (QT == DT_F32 ? 2 : 1); ++i) {
        const Words v = *reinterpret_cast<const Words *>(b + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            r.w[4 * i + e] = v.w[e];
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

// A tile of C rows of D elements on its way from global memory to the LDS parts.
template <int QT, int C, int D, int THREADS>
struct Tile {
    static constexpr int U = C * D / 8, N = (U + THREADS - 1) / THREADS, PITCH = D * 2 + 16;
    Raw8<QT> r[N];

    // rows [0, n) of the tile at element base `at`; the others are zero
    __device__ __forceinline__ void load(const void *p, int64_t at, int64_t stride, int n)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = i * THREADS + threadIdx.x, row = u / (D / 8), c = u % (D / 8) * 8;
            r[i] = Raw8<QT>{};
            if ((U % THREADS == 0 || u < U) && row < n)
                r[i] = load_raw8<QT>(p, at + row * stride + c);
        }
    }
    __device__ __forceinline__ void store(unsigned char *lds) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = i * THREADS + threadIdx.x, row = u / (D / 8), c = u % (D / 8) * 8;
            if (U % THREADS == 0 || u < U) {
                bf16x8 part[input_parts(QT)];
                raw8_parts<QT>(r[i], part);
#pragma unroll
                for (int s = 0; s < input_parts(QT); ++s)
                    *reinterpret_cast<bf16x8 *>(lds + s * C * PITCH + row * PITCH + 2 * c) = part[s];
            }
        }
    }
};

__device__ __forceinline__ bf16x8 lds8(const unsigned char *p) { return *reinterpret_cast<const bf16x8 *>(p); }

// Eight k-values of one row in the accumulator pair's slot order: 4 at p, 4 at p + 16 elements.
__device__ __forceinline__ bf16x8 lds4x2(const unsigned char *p)
{
    uint2 w[2] = {*reinterpret_cast<const uint2 *>(p), *reinterpret_cast<const uint2 *>(p + 32)};
    bf16x8 v;
    __builtin_memcpy(&v, w, 16);
    return v;
}

// Transposed operand: column c0 + li of rows row0 + 8 lg .. + 7 of a row-major bf16 tile. A transposing
// read hands lane i of 16 column i of the four rows whose 16 columns the lanes point at.
__device__ __forceinline__ bf16x8 lds_tr8(unsigned char *tile, int pitch, int row0, int c0, int li, int lg)
{
    unsigned char *p = tile + (row0 + 8 * lg + (li >> 2)) * pitch + 2 * (c0 + 4 * (li & 3));
    s16x4 w[2] = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p),
                  __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + 4 * pitch))};
    bf16x8 v;
    __builtin_memcpy(&v, w, 16);
    return v;
}

// Log decays at most as low as this count as exp = 0 (f32 reaches 0 at -104); a finite
// bound keeps differences of prefix sums finite. In f64 the sums still resolve 2^-30 of
// a small decay beside it.
constexpr double kLowest = -1e4;

// Segment `idx` of a launch: which sequence, which of its segments, its tokens. Every
// lane scans 64 sequences' counts at once.
struct Segment {
    int seq, seg, segs, start, len;
};
__device__ __forceinline__ Segment find_segment(const int32_t *cu, int N, int idx, int tokens, bool second)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int s0 = 0; s0 < N; s0 += 64) {
        const int s = s0 + lane;
        const int start = s < N ? cu[s] : 0, len = s < N ? cu[s + 1] - start : 0;
        const int segs = (len + tokens - 1) / tokens;
        const int cnt = second ? max(segs - 1, 0) : segs > 1 ? segs - 1 : segs;
        int upto = cnt;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d, 64);
            upto += lane >= d ? o : 0;
        }
        const uint64_t hit = __ballot(idx >= before + upto - cnt && idx < before + upto);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            Segment r;
            r.seq = s0 + src;
            r.segs = __shfl(segs, src, 64);
            r.seg = idx - before - __shfl(upto - cnt, src, 64) + (second ? 1 : 0);
            r.start = __shfl(start, src, 64) + r.seg * tokens;
            r.len = min(tokens, __shfl(len, src, 64) - r.seg * tokens);
            return r;
        }
        before += __shfl(upto, 63, 64);
    }
    return Segment{-1, 0, 0, 0, 0};
}

// Workspace slot of a sequence's segment 0 state (segments but the last have one):
// distinct, since a sequence of n tokens has at most n / tokens of them.
__device__ __forceinline__ int first_slot(const int32_t *cu, int seq, int tokens) { return cu[seq] / tokens; }

template <int DK, int DV, int QT, bool F32OUT>
struct Walk {
    using G = Geo<DK, DV, QT>;
    static constexpr int IP = G::IP, C = G::C, NT = G::NT, W = G::W, THREADS = G::THREADS;
    static constexpr int PK = G::PK, PV = G::PV, PP = 2 * C + 16;
    static constexpr int OP = F32OUT ? 3 : 2, LIM = F32OUT ? 2 : 1;  // parts of P and S in the outputs
    static constexpr int KT = DK / 16, KS = DK / 32, TT = C / 16, JS = C / 32;

    struct __align__(16) Lds {
        unsigned char q[IP * C * PK], k[IP * C * PK], v[IP * C * PV], p[OP * C * PP];
        double g[C];        // prefix sums of the log decays
        float eg[C], w[C];  // e^G_t and e^(G_last - G_t)
    };

    // The chunk's decay rows, by one wave (C <= 64 lanes).
    static __device__ __forceinline__ void decays(Lds &l, double g)
    {
        const int lane = threadIdx.x & 63;
        double s = g < kLowest ? kLowest : g;
#pragma unroll
        for (int d = 1; d < C; d <<= 1) {
            const double o = __shfl_up(s, d, 64);
            s += lane >= d ? o : 0.0;
        }
        const double last = __shfl(s, C - 1, 64);
        if (lane < C) {
            l.g[lane] = s;
            l.eg[lane] = expf((float)s);
            l.w[lane] = expf((float)(last - s));
        }
    }

    // Walks the segment's chunks from the state at `in` (NULL: zero) and stores the state after them at
    // `out_state`; OUT: with the tokens' outputs. Returns the segment's summed log decay.
    template <bool OUT>
    static __device__ __forceinline__ double run(Lds &l, const LinattnParams &p, const Segment sg, int h, const float *in,
                                                 float *out_state)
    {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, li = lane & 15, lg = lane >> 4;
        const int kh = k_head_of(p.hc.head_map, h, p.hc.Hk, p.hc.Hv);
        const int dv0 = wave * 16 * NT;
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
                S[kt][v] = in ? *reinterpret_cast<const f32x4 *>(in + (int64_t)(dv0 + 16 * v + li) * DK + 16 * kt + 4 * lg)
                              : f32x4{0.f, 0.f, 0.f, 0.f};

        Tile<QT, C, DK, THREADS> tq, tk;
        Tile<QT, C, DV, THREADS> tv;
        double tg = 0.0;
        auto fetch = [&](int c0) {
            const int n = sg.len - c0;
            const int64_t row = (int64_t)sg.start + c0;
            if constexpr (OUT)
                tq.load(p.in.q, row * p.in.q_stride + (int64_t)kh * DK, p.in.q_stride, n);
            tk.load(p.in.k, row * p.in.k_stride + (int64_t)kh * DK, p.in.k_stride, n);
            tv.load(p.in.v, row * p.in.v_stride + (int64_t)h * DV, p.in.v_stride, n);
            if (wave == 0)
                tg = lane < n && lane < C ? (head_decay ? rate : (double)p.in.g[(row + lane) * p.hc.Hv + h]) : 0.0;
        };
        auto stage = [&] {
            if constexpr (OUT)
                tq.store(l.q);
            tk.store(l.k);
            tv.store(l.v);
            if (wave == 0)
                decays(l, tg);
        };
        if constexpr (OUT) {
            // the P tiles right of the diagonal that the 32-wide products reach
            for (int u = threadIdx.x; u < OP * (TT / 2) * 16 * 2; u += THREADS) {
                const int s = u / (TT / 2 * 32), it = u / 32 % (TT / 2) * 2, row = u / 2 % 16, half = u % 2;
                *reinterpret_cast<uint4 *>(l.p + s * C * PP + (16 * it + row) * PP + 2 * (16 * it + 16 + 8 * half)) =
                    make_uint4(0, 0, 0, 0);
            }
        }
        fetch(0);
        stage();
        __syncthreads();

        double total = 0.0;
        for (int c0 = 0; c0 < sg.len; c0 += C) {
            if (c0 + C < sg.len)
                fetch(c0 + C);
            f32x4 O[OUT ? TT : 1][NT];
            if constexpr (OUT) {
                // P = tril(Q K^T) . e^(G_t - G_j), tiles on and below the diagonal dealt to the waves
                for (int idx = wave; idx < TT * (TT + 1) / 2; idx += W) {
                    int it = 0;
#pragma unroll
                    for (int i = 1; i < TT; ++i)
                        it += idx >= i * (i + 1) / 2 ? 1 : 0;
                    const int jt = idx - it * (it + 1) / 2;
                    f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int x = 0; x < IP; ++x)
#pragma unroll
                            for (int y = 0; y < IP; ++y)
                                if (x + y <= LIM)
                                    a = mfma(lds8(l.k + x * C * PK + (16 * jt + li) * PK + 64 * ks + 16 * lg),
                                             lds8(l.q + y * C * PK + (16 * it + li) * PK + 64 * ks + 16 * lg), a);
                    const int t = 16 * it + li;
                    const double gt = l.g[t];
                    float x[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int j = 16 * jt + 4 * lg + r;
                        x[r] = j <= t ? a[r] * __expf((float)(gt - l.g[j])) : 0.f;
                    }
#pragma unroll
                    for (int s = 0; s < OP; ++s) {
                        const uint32_t b0 = cut(x[0]), b1 = cut(x[1]), b2 = cut(x[2]), b3 = cut(x[3]);
                        *reinterpret_cast<uint2 *>(l.p + s * C * PP + t * PP + 2 * (16 * jt + 4 * lg)) =
                            make_uint2((b0 >> 16) | b1, (b2 >> 16) | b3);
                    }
                }
                // O = diag(e^G) Q S^T
#pragma unroll
                for (int it = 0; it < TT; ++it)
#pragma unroll
                    for (int v = 0; v < NT; ++v)
                        O[it][v] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    bf16x8 sp[NT][OP];
#pragma unroll
                    for (int v = 0; v < NT; ++v) {
                        const f32x4 a = S[2 * ks][v], b = S[2 * ks + 1][v];
                        const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
                        split8<OP>(x, sp[v]);
                    }
#pragma unroll
                    for (int it = 0; it < TT; ++it)
#pragma unroll
                        for (int y = 0; y < IP; ++y) {
                            const bf16x8 q = lds4x2(l.q + y * C * PK + (16 * it + li) * PK + 64 * ks + 8 * lg);
#pragma unroll
                            for (int v = 0; v < NT; ++v)
#pragma unroll
                                for (int s = 0; s < OP; ++s)
                                    if (s + y <= LIM)
                                        O[it][v] = mfma(sp[v][s], q, O[it][v]);
                        }
                }
#pragma unroll
                for (int it = 0; it < TT; ++it) {
                    const float e = l.eg[16 * it + li];
#pragma unroll
                    for (int v = 0; v < NT; ++v)
                        O[it][v] *= e;
                }
            }
            // V^T operands: dv as the row, tokens as k
            bf16x8 vt[JS][NT][IP];
#pragma unroll
            for (int js = 0; js < JS; ++js)
#pragma unroll
                for (int v = 0; v < NT; ++v)
#pragma unroll
                    for (int x = 0; x < IP; ++x)
                        vt[js][v][x] = lds_tr8(l.v + x * C * PV, PV, 32 * js, dv0 + 16 * v, li, lg);
            if constexpr (OUT) {
                __syncthreads();  // P is whole
                bool bad = false;  // a V that is not finite: 0 times it, right of the diagonal, is not 0
#pragma unroll
                for (int js = 0; js < JS; ++js)
#pragma unroll
                    for (int v = 0; v < NT; ++v) {
                        uint32_t w[4];
                        __builtin_memcpy(w, &vt[js][v][0], 16);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            bad |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
                    }
                if (__ballot(bad) == 0) {
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
                                        if (s + x <= LIM)
                                            O[it][v] = mfma(vt[js][v][x], pt, O[it][v]);
                            }
                } else {
                    // term by term, the tokens up to t alone
                    for (int j = 0; j < C; ++j)
#pragma unroll
                        for (int it = 0; it < TT; ++it)
                            if (j <= 16 * it + li) {
                                float pj = 0.f;
#pragma unroll
                                for (int s = OP - 1; s >= 0; --s)
                                    pj += bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(
                                        l.p + s * C * PP + (16 * it + li) * PP + 2 * j));
#pragma unroll
                                for (int v = 0; v < NT; ++v)
#pragma unroll
                                    for (int r = 0; r < 4; ++r) {
                                        float x = 0.f;
#pragma unroll
                                        for (int y = IP - 1; y >= 0; --y)
                                            x += bf16_bits_to_f32(*reinterpret_cast<const uint16_t *>(
                                                l.v + y * C * PV + j * PV + 2 * (dv0 + 16 * v + 4 * lg + r)));
                                        O[it][v][r] = fmaf(pj, x, O[it][v][r]);
                                    }
                            }
                }
#pragma unroll
                for (int it = 0; it < TT; ++it) {
                    const int t = c0 + 16 * it + li;
                    if (t < sg.len) {
#pragma unroll
                        for (int v = 0; v < NT; ++v) {
                            const int64_t at = (((int64_t)sg.start + t) * p.hc.Hv + h) * DV + dv0 + 16 * v + 4 * lg;
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                store_act(p.out, at + r, p.out_dt, p.hc.scale * O[it][v][r]);
                        }
                    }
                }
            }
            // S <- e^G_last S + K^T diag(w) V
            const float dec = l.eg[C - 1];
            total += l.g[C - 1];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                for (int v = 0; v < NT; ++v)
                    S[kt][v] *= dec;
#pragma unroll
            for (int js = 0; js < JS; ++js) {
                const f32x4 w0 = *reinterpret_cast<const f32x4 *>(&l.w[32 * js + 8 * lg]);
                const f32x4 w1 = *reinterpret_cast<const f32x4 *>(&l.w[32 * js + 8 * lg + 4]);
                bf16x8 vd[NT][3];
#pragma unroll
                for (int v = 0; v < NT; ++v) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = join<IP>(vt[js][v], e) * (e < 4 ? w0[e & 3] : w1[e & 3]);
                    split8<3>(x, vd[v]);
                }
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int x = 0; x < IP; ++x) {
                        const bf16x8 k = lds_tr8(l.k + x * C * PK, PK, 32 * js, 16 * kt, li, lg);
#pragma unroll
                        for (int v = 0; v < NT; ++v)
#pragma unroll
                            for (int s = 0; s < 3; ++s)
                                if (s + x <= 2)
                                    S[kt][v] = mfma(k, vd[v][s], S[kt][v]);
                    }
            }
            __syncthreads();  // every wave is done with the chunk's tiles
            if (c0 + C < sg.len) {
                stage();
                __syncthreads();
            }
        }
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int v = 0; v < NT; ++v)
                *reinterpret_cast<f32x4 *>(out_state + (int64_t)(dv0 + 16 * v + li) * DK + 16 * kt + 4 * lg) = S[kt][v];
        return total;
    }
};

// Blocks: segment-major, heads fastest.
template <int DK, int DV, int QT, bool F32OUT, bool SECOND>
__global__ __launch_bounds__((Geo<DK, DV, QT>::THREADS), 1) void chunk_kernel(const LinattnParams p)
{
    using Wk = Walk<DK, DV, QT, F32OUT>;
    __shared__ typename Wk::Lds l;
    const int h = blockIdx.x % p.hc.Hv;
    const Segment sg = find_segment(p.cu, p.N, blockIdx.x / p.hc.Hv, p.seg_tokens, SECOND);
    if (sg.seq < 0)
        return;
    const int64_t size = (int64_t)DK * DV;
    float *state = p.state + ((int64_t)sg.seq * p.hc.Hv + h) * size;
    const bool last = sg.seg == sg.segs - 1;
    const int64_t slot = last && !sg.seg ? 0 : ((int64_t)first_slot(p.cu, sg.seq, p.seg_tokens) + sg.seg) * p.hc.Hv + h;
    float *after = last ? state : p.seg_state + slot * size;
    if constexpr (SECOND) {
        Wk::template run<true>(l, p, sg, h, p.seg_state + (slot - p.hc.Hv) * size, after);
    } else if (sg.seg == 0) {
        Wk::template run<true>(l, p, sg, h, state, after);
    } else {
        const double g = Wk::template run<false>(l, p, sg, h, nullptr, after);
        if (threadIdx.x == 0)
            p.seg_decay[slot] = (float)g;
    }
}

template <int DK, int DV, int QT, bool F32OUT>
hipError_t launch_chunk(const LinattnParams &p, int blocks, bool second, hipStream_t s)
{
    constexpr int threads = Geo<DK, DV, QT>::THREADS;
    if (second)
        chunk_kernel<DK, DV, QT, F32OUT, true><<<blocks, threads, 0, s>>>(p);
    else
        chunk_kernel<DK, DV, QT, F32OUT, false><<<blocks, threads, 0, s>>>(p);
    return hipGetLastError();
}

template <int QT>
hipError_t launch_chunk_for(const LinattnParams &p, int blocks, bool second, hipStream_t s)
{
#define GDN_CHUNK(DK, DV)                                                       \
    if (p.hc.dk == DK && p.hc.dv == DV)                                         \
        return p.out_dt == DT_F32 ? launch_chunk<DK, DV, QT, true>(p, blocks, second, s) \
                                  : launch_chunk<DK, DV, QT, false>(p, blocks, second, s);
    GDN_CHUNK(32, 32)
    GDN_CHUNK(64, 64)
    GDN_CHUNK(96, 96)
    GDN_CHUNK(128, 128)
    GDN_CHUNK(64, 128)
    GDN_CHUNK(128, 64)
    GDN_CHUNK(128, 256)
    GDN_CHUNK(256, 128)
    GDN_CHUNK(256, 256)
#undef GDN_CHUNK
    return hipErrorInvalidValue;
}

// Tokens per chunk of a head shape
template <int QT>
int chunk_tokens_for(int dk, int dv)
{
#define GDN_CHUNK(DK, DV)         \
    if (dk == DK && dv == DV)     \
        return Geo<DK, DV, QT>::C;
    GDN_CHUNK(32, 32)
    GDN_CHUNK(64, 64)
    GDN_CHUNK(96, 96)
    GDN_CHUNK(128, 128)
    GDN_CHUNK(64, 128)
    GDN_CHUNK(128, 64)
    GDN_CHUNK(128, 256)
    GDN_CHUNK(256, 128)
#undef GDN_CHUNK
    return Geo<256, 256, QT>::C;
}

}  // namespace linattn
}  // namespace gdn
