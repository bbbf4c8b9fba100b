// E4M3 codes with block scales: conversion, the matrix instruction and the
// asynchronous copy to LDS that the FP8 kernels share.
#pragma once

#include <type_traits>

#include "common.h"

namespace moe {

constexpr int FP8_BLOCK = FP8_K;              // elements of K under one scale
constexpr float FP8_MAX = 448.0f;             // largest E4M3 value
constexpr float FP8_TINY = 7.888609e-31f;     // 2^-100, smallest block maximum a scale is made from

// Two values rounded to bf16 (to nearest even, by the conversion instruction).
__device__ __forceinline__ uint32_t cvt_bf2(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, bf16x2));
}

// Divisor of one block: codes are round-to-nearest-even of 448 x / top.  The
// product by 448 comes first and the quotient is refined to the correctly
// rounded one for every quotient that fp32 can hold (one residual step on
// the hardware reciprocal; the residual is exact): a quotient half way
// between two codes then stays half way, as it does for many ratios of two
// bf16 values, and rounds to the even code as the definition says.  A
// multiplication by a rounded 448 / top moved 1 in 2000 codes of bf16 data by
// one step.  Blocks above 2^100 are scaled down so that the product by 448
// stays finite.
struct Fp8Block {
    float pre, top, rcp, scale;
};

__device__ __forceinline__ Fp8Block fp8_block(float amax)
{
    Fp8Block b;
    const float m = fmaxf(amax, FP8_TINY);
    const bool big = m > 1.2676506e30f;  // 2^100
    b.pre = big ? FP8_MAX * 5.421011e-20f : FP8_MAX;  // 448 (* 2^-64)
    b.top = big ? m * 5.421011e-20f : m;
    b.rcp = __builtin_amdgcn_rcpf(b.top);
    b.scale = m / FP8_MAX;
    return b;
}

__device__ __forceinline__ float fp8_quot(float x, const Fp8Block &b)
{
    const float n = x * b.pre;
    const float q = n * b.rcp;
    return fmaf(fmaf(-q, b.top, n), b.rcp, q);
}

// Codes of four values, the first in the lowest byte.
__device__ __forceinline__ uint32_t fp8x4(float x0, float x1, float x2, float x3, const Fp8Block &b)
{
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_quot(x0, b), fp8_quot(x1, b), 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(fp8_quot(x2, b), fp8_quot(x3, b), v, true);
    return (uint32_t)v;
}

// Staging rows of the FP8 experts' outputs: half precision under one exponent
// byte for each 8 columns, the largest of their finite values scaled to
// [2^14, 2^15).  2^-11 relative where bf16 rows, of the same size, are 2^-8
// off: the sum over a token's slots then adds no error that shows next to the
// rounding of y to bf16 (with bf16 rows it was as large again).  Infinities and
// NaN stay what they are.
constexpr uint32_t STAGE_MIN_EXP = 15;  // keeps both factors normal

__device__ __forceinline__ uint32_t stage_exponent(float v)
{
    const uint32_t e = (__float_as_uint(v) >> 23) & 0xFF;
    return e == 0xFF ? 0 : e;
}

// 2^(141 - e) and 2^(e - 141) of a biased exponent e.
__device__ __forceinline__ float stage_pack(uint32_t e) { return __uint_as_float((268 - e) << 23); }
__device__ __forceinline__ float stage_unpack(uint32_t e) { return __uint_as_float((e - 14) << 23); }

__device__ __forceinline__ uint32_t cvt_half2(float a, float b)
{
    typedef _Float16 half2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, half2));
}

// Largest value over each row of 16 lanes, in all of them (row rotations).
__device__ __forceinline__ float row16_max(float v)
{
    auto rot = [](float x, auto ctrl) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value,
                                                          0xf, 0xf, true));
    };
    v = fmaxf(v, rot(v, std::integral_constant<int, 0x128>{}));
    v = fmaxf(v, rot(v, std::integral_constant<int, 0x124>{}));
    v = fmaxf(v, rot(v, std::integral_constant<int, 0x122>{}));
    v = fmaxf(v, rot(v, std::integral_constant<int, 0x121>{}));
    return v;
}

// Fragments of 16 rows x 128 K (A) and 128 K x 16 columns (B) of E4M3 codes:
// lane l holds 32 codes of row (column) l % 16, which 32 of the 128 is free as
// long as both operands hold the same ones; products onto zero,
// C[4 * (l / 16) + i][l % 16].
//
// The FP8 matrix instructions (this one and the 16x16x32 form alike) add the
// products of 8 consecutive K in a narrow window: each is cut, towards zero,
// to multiples of 2^-13 of the largest one's power of two (measured bit by
// bit); the sums of eight are then added in fp32.  On normally distributed
// codes that is 1.5e-5 of the result (2-norm), far below a bf16 rounding, and
// too much for an fp32 result and for gate and up: h is rounded to 3 bits of
// mantissa, so that an error of its sums moves every code whose quotient is as
// near to a midpoint by a step, 6 to 12% of the value (T=1, H=2048, k=8, I=768: 14
// of 6144 codes, y off by more than 0.005 of its size in 4% of the tokens and by 0.010
// at most of 256 tokens, with exact sums by 0.0018).  So results and staging rows that are
// rounded to bf16 or half precision take the FP8 instruction, fp32 results and
// the sums of gate and up the bf16 one on the same codes: every product is exact
// there and the sum is fp32's, at half the instruction's rate.
typedef intx8 Fp8Raw;  // the codes as they are read: one register tuple, as the instruction takes it

__device__ __forceinline__ Fp8Raw fp8_raw(uint4 lo, uint4 hi)
{
    return Fp8Raw{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

template <bool EXACT>
struct Fp8Frag;

template <>
struct Fp8Frag<false> {
    intx8 v;
    __device__ __forceinline__ Fp8Frag(Fp8Raw r) : v(r) {}
};

__device__ __forceinline__ floatx4 mfma_fp8(const Fp8Frag<false> &a, const Fp8Frag<false> &b)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, floatx4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

template <>
struct Fp8Frag<true> {
    bf16x8 v[4];
    __device__ __forceinline__ Fp8Frag(Fp8Raw w)
    {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bf16x2 p = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * q + j], 1.0f, false);
                const bf16x2 u = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * q + j], 1.0f, true);
                v[q][4 * j] = p[0], v[q][4 * j + 1] = p[1];
                v[q][4 * j + 2] = u[0], v[q][4 * j + 3] = u[1];
            }
    }
};

__device__ __forceinline__ floatx4 mfma_fp8(const Fp8Frag<true> &a, const Fp8Frag<true> &b)
{
    floatx4 c{0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        c = mfma16(a.v[q], b.v[q], c);
    return c;
}

// Asynchronous copy from memory to LDS: 16 (4) bytes per lane from `base` +
// the lane's byte offset to `lds` + 16 (4) * lane; `base` and `lds` are uniform
// in the wave.  Written as instructions because the compiler, which cannot
// tell what such a copy overwrites, waits for all of them before every LDS
// read; the kernels wait themselves (dma_wait_barrier).  There is no register
// result, so nothing the compiler tracks changes behind its back; its own
// waits count these copies too and can only become stricter for it.  Every
// copy is waited for before the wave ends, since its LDS may belong to another
// workgroup afterwards.
__device__ __forceinline__ void dma16(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off),
                 "s"(base)
                 : "memory", "m0");
}

__device__ __forceinline__ void dma4(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off),
                 "s"(base)
                 : "memory", "m0");
}

// Waits until at most N of this wave's memory operations are outstanding and
// all its LDS operations are done, then for the workgroup.
template <int N>
__device__ __forceinline__ void dma_wait_barrier()
{
    static_assert(N >= 0 && N < 64, "the counter holds 6 bits");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Waits for this wave's LDS operations, then for the workgroup; copies and
// loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void *p)
{
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void *)p;
}

}  // namespace moe
