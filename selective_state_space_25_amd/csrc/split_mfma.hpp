// split_mfma.hpp -- fp32-grade matrix products on the bf16 matrix cores.
//
// An fp32 value is held as the sum of up to three bfloat16 values, each the
// rounding of what the ones before it leave (8 significant bits a plane, 24
// in all), so a product of two such sums is a handful of bf16 MFMAs that
// accumulate in fp32.  Keeping the plane pairs (a, b) with a + b < 3 leaves
// out terms near 2^-25 of the product: the result is as exact as an fp32
// product, at 6 (both sides fp32) or 3 (one side bf16, which is one plane)
// of the 16 MFMAs that the same product takes at the fp32 rate.  bf16 planes
// keep fp32's range; an infinity leaves NaN in its lower planes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.hpp"

namespace selscan {
namespace smm {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// v_mfma_f32_16x16x32_bf16.  Lane l = 16 g + i: operand A holds row i,
// operand B column i, k = 8 g .. 8 g + 7 of either; C holds rows
// 4 g .. 4 g + 3 of column i.
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// c += A B over one k-step of 32, the sides split in NA and NB planes, plane
// pairs with a + b < LIM, small terms first.
template <int LIM, int NA, int NB>
__device__ __forceinline__ f32x4 mm(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int s = LIM - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) c = mfma(a[i], b[s - i], c);
    return c;
}

// M such products step by step: an MFMA that adds to the sum of the one
// before waits out its latency (several times its issue slot), so products
// that are independent take turns.  a(m), b(m): planes of product m.
template <int LIM, int NA, int NB, int M, typename FA, typename FB>
__device__ __forceinline__ void mm_turns(FA a, FB b, f32x4 (&c)[M]) {
#pragma unroll
    for (int s = LIM - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) {
#pragma unroll
                for (int m = 0; m < M; ++m) c[m] = mfma(a(m)[i], b(m)[s - i], c[m]);
            }
}

// The 12 plane products of two k-steps of fp32 by fp32, four chains of three.
__device__ __forceinline__ f32x4 mm_pair(const bf16x8 (&a)[2][3], const bf16x8 (&b)[2][3]) {
    f32x4 c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 2; ++k) c[k] = mfma(a[k][1], b[k][1], c[k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) c[2 + k] = mfma(a[k][0], b[k][2], c[2 + k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) c[k] = mfma(a[k][2], b[k][0], c[k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) c[2 + k] = mfma(a[k][0], b[k][1], c[2 + k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) c[k] = mfma(a[k][1], b[k][0], c[k]);
#pragma unroll
    for (int k = 0; k < 2; ++k) c[2 + k] = mfma(a[k][0], b[k][0], c[2 + k]);
    return (c[0] + c[1]) + (c[2] + c[3]);
}

// Pairs e, e + 1 of two values into word `e` of NP planes (a plane is one
// operand, four words of two bf16 each).
template <int NP>
__device__ __forceinline__ void split2(float a, float b, u32x4 (&p)[NP], int e) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint32_t w = pack_bf16x2(a, b);
        p[i][e] = w;
        if (i + 1 < NP) {
            a -= bf16lo(w);
            b -= bf16hi(w);
        }
    }
}

template <int NP>
__device__ __forceinline__ void as_operand(const u32x4 (&w)[NP], bf16x8 (&p)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) p[i] = __builtin_bit_cast(bf16x8, w[i]);
}

// Eight values (two groups of four) into NP planes.
template <int NP>
__device__ __forceinline__ void split8(f32x4 lo, f32x4 hi, bf16x8 (&p)[NP]) {
    u32x4 w[NP];
    split2<NP>(lo[0], lo[1], w, 0);
    split2<NP>(lo[2], lo[3], w, 1);
    split2<NP>(hi[0], hi[1], w, 2);
    split2<NP>(hi[2], hi[3], w, 3);
    as_operand(w, p);
}

__device__ __forceinline__ bf16x8 ld8(const uint16_t* p) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ bf16x8 cat(s16x4 a, s16x4 b) {
    const s16x8 r = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, r);
}

// Transposing LDS load: within 16 lanes, lane a passes the address of 4
// consecutive elements of row r0 + a / 4 (columns c0 + 4 (a % 4) ..); lane i
// receives rows r0 .. r0 + 3 of column c0 + i.
__device__ __forceinline__ s16x4 ld_tr(const uint16_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p));
}

// Operand with k running down the rows of m (row stride rs): rows
// r0 .. r0 + 31, columns c0 .. c0 + 15.
__device__ __forceinline__ bf16x8 ld_down(const uint16_t* m, int rs, int r0, int c0, int lane) {
    const int g = lane >> 4, a = lane & 15;
    const uint16_t* p = m + (r0 + 8 * g + (a >> 2)) * rs + c0 + 4 * (a & 3);
    return cat(ld_tr(p), ld_tr(p + 4 * rs));
}

// Four consecutive values into NP planes of 4 bf16 each.
template <int NP>
__device__ __forceinline__ void split4(f32x4 r, uint2 (&p)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        p[i] = make_uint2(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]));
        if (i + 1 < NP) {
            r[0] -= bf16lo(p[i].x);
            r[1] -= bf16hi(p[i].x);
            r[2] -= bf16lo(p[i].y);
            r[3] -= bf16hi(p[i].y);
        }
    }
}

}  // namespace smm
}  // namespace selscan
