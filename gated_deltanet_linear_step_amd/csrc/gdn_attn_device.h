// gdn_attn_device.h -- what the attention kernels of gfx950 share: 16-bit types and their matrix instructions,
// transposing LDS reads, 16-byte copies to the LDS, page lookups and the softmax in base 2.
#pragma once

#include "gdn_device.h"
#include "gdn_attn.h"

// 64-bit shifts by an amount in a VGPR (v_lshlrev_b64, v_lshrrev_b64, v_ashrrev_i64): where that is the last register that a wave is
// allotted (of allotments of 8), stores of waves beside it have held foreign registers here, a few rows in 30,000. The same code with
// one register more is right. The compiler avoids that register on gfx90a, not on gfx950: tests/test_kernel_code.py looks for it.

namespace gdn {
namespace attn {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) void lds_void;

constexpr int kBlock = 128;  // rows of a workgroup of the prompts' kernel

// First block of 128 rows that the sequences before cu[s] leave to sequence s (some blocks stay empty)
__host__ __device__ __forceinline__ int block_base(const int32_t *cu, int s, int G)
{
    return (int)((int64_t)cu[s] * G / kBlock) + s;
}

// exp2 of a masked score, and the running maximum before any key
constexpr float kNone = -__builtin_inff();
// in place of the first run's sum: the outputs are there, nothing is joined
constexpr float kJoined = -1.f;

// kLift: weights are 2^kLift times what they are beside the row's largest, so that f16 keeps their accuracy down to 2^-21 of that and
// drops them below 2^-32 (bf16 has f32's exponents). With a maximum that is passed by up to 2^8, at most 2^15.
template <int DT>
struct Type16;
template <>
struct Type16<DT_BF16> {
    typedef __bf16 T8 __attribute__((ext_vector_type(8)));
    typedef __bf16 T2 __attribute__((ext_vector_type(2)));
    static constexpr uint32_t kExponents = 0x7f807f80u, kLow = 0x00800080u;
    static constexpr int kLift = 0;
    __device__ __forceinline__ static f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(T8, a), __builtin_bit_cast(T8, b), c, 0, 0, 0);
    }
    __device__ __forceinline__ static f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(T8, a), __builtin_bit_cast(T8, b), c, 0, 0, 0);
    }
};
template <>
struct Type16<DT_F16> {
    typedef _Float16 T8 __attribute__((ext_vector_type(8)));
    typedef _Float16 T2 __attribute__((ext_vector_type(2)));
    static constexpr uint32_t kExponents = 0x7c007c00u, kLow = 0x04000400u;
    static constexpr int kLift = 7;
    __device__ __forceinline__ static f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(T8, a), __builtin_bit_cast(T8, b), c, 0, 0, 0);
    }
    __device__ __forceinline__ static f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(T8, a), __builtin_bit_cast(T8, b), c, 0, 0, 0);
    }
};

// Two f32 rounded to the type, lo's bits below hi's
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), typename Type16<DT>::T2));
}

// Two outputs of a row. Averages of finite f16 values are at most the type's largest, which the rounding of their weights may pass by up
// to half a step, to where it would become an infinity: they stop there.
template <int DT>
__device__ __forceinline__ uint32_t pack_outputs(float lo, float hi)
{
    const auto average = [](float x) {
        return DT == DT_F16 && fabsf(x) < __builtin_inff() ? fminf(fmaxf(x, -65504.f), 65504.f) : x;
    };
    return pack2<DT>(average(lo), average(hi));
}

// The top bits of the halves of w that are infinite or NaN
template <int DT>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    return ((w & Type16<DT>::kExponents) + Type16<DT>::kLow) & 0x80008000u;
}

// w with the halves that are infinite or NaN made 0
template <int DT>
__device__ __forceinline__ uint32_t finite_part(uint32_t w)
{
    const uint32_t bad = not_finite<DT>(w) >> 15;
    return w & ~(bad * 0xffffu);
}

// 16 bytes at an LDS address, and a transposing read: a lane's four elements are column i (of lane i of 16) of the four rows
// whose 16 columns, in groups of four, the lanes point at
__device__ __forceinline__ u32x4 lds_read16(uint32_t at) { return *(const lds_u32x4 *)(uintptr_t)at; }
__device__ __forceinline__ u32x2 lds_read_tr(uint32_t at)
{
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)at));
}

// A value of which the compiler knows nothing: what is computed from it late is not kept in registers from early on
__device__ __forceinline__ int opaque(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

// Copies 16 bytes a lane from base + off to the LDS, lane l's to byte `to` + 16 l, without waiting. Written out because
// the compiler lets every transposing LDS read wait for all such copies, those to another buffer too: whoever
// reads what was copied waits for it (vmcnt) itself. (m0 is reserved: the compiler keeps nothing in it
// and sets it right before each use of its own, and refuses it as a clobber.)
__device__ __forceinline__ void copy16(const unsigned char *base, uint32_t off, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(off), "s"(base)
                 : "memory");
}

// The same for N runs of 1024 bytes, one after another from byte `to` on: off[i] is the offset of the i-th, at least 1024 i.
// (An instruction's own offset counts in memory and in the LDS.)
template <int N>
__device__ __forceinline__ void copy16_runs(const unsigned char *base, const uint32_t (&off)[N], uint32_t to)
{
    static_assert(N >= 2 && N <= 4, "offsets below 4096");
    if constexpr (N == 2)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %3\n\t"
                     "global_load_lds_dwordx4 %2, %3 offset:1024"
                     :
                     : "s"(to), "v"(off[0]), "v"(off[1] - 1024), "s"(base)
                     : "memory");
    else if constexpr (N == 3)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %4\n\t"
                     "global_load_lds_dwordx4 %2, %4 offset:1024\n\tglobal_load_lds_dwordx4 %3, %4 offset:2048"
                     :
                     : "s"(to), "v"(off[0]), "v"(off[1] - 1024), "v"(off[2] - 2048), "s"(base)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %5\n\t"
                     "global_load_lds_dwordx4 %2, %5 offset:1024\n\tglobal_load_lds_dwordx4 %3, %5 offset:2048\n\t"
                     "global_load_lds_dwordx4 %4, %5 offset:%6"
                     :
                     : "s"(to), "v"(off[0]), "v"(off[1] - 1024), "v"(off[2] - 2048), "v"(off[3] - 3 * 1024), "s"(base),
                       "n"(3 * 1024)
                     : "memory");
}

// Maximum and sum over a lane and the one 32 away (the swap leaves the lower half's values in one word, the upper half's
// in the other)
__device__ __forceinline__ float half_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Scores' factor for exponentials in base 2
__device__ __forceinline__ float base2(float scale) { return scale * 1.4426950408889634f; }

// Exponents in base 2 are formed as scale s - base in one instruction, with base the rounded product of scale and the row's
// maximum (less kLift). What that rounding left out raises every weight of a row alike: by less than 2^-15 of itself while |base| <= 2^8,
// but without bound beyond (at 2^36, by 2^4096 or to nothing). Rows past that take the maximum from the scores first.
constexpr float kFar = 256.f;

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }

// ln of the sum of e^(scale s), from the sum of the weights relative to the score `top`
template <int DT>
__device__ __forceinline__ float log_sum(float top, float scale, float sum)
{
    constexpr float one = 1 << Type16<DT>::kLift;
    return sum == 0.f ? kNone : (top * base2(scale) + __log2f(sum * (1.f / one))) * 0.69314718055994531f;
}

}  // namespace attn
}  // namespace gdn
