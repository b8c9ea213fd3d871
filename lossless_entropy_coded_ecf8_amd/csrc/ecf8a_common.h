// ecf8a_common.h -- what the kernels beside a compressed weight share: the
// 16x16x32 matrix instruction of both 16-bit types, 16-byte moves, the split
// of a float32 into two bfloat16, and host-side checks.
//
// Layout of the matrix instruction (64 lanes, c = lane % 16, g = lane / 16):
// operand A holds row c, operand B column c, each lane the eight reduction
// slots 8g .. 8g + 7; the result holds column c, rows 4g .. 4g + 3.  A sum does
// not depend on which reduction index sits in which slot as long as A and B
// agree, and the kernels use that freedom to keep every load 16 bytes wide.
#ifndef ECF8A_COMMON_H
#define ECF8A_COMMON_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ecf8a.h"

namespace ecf8a {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kBf16 = ECF8A_BF16, kFp16 = ECF8A_FP16, kE4m3 = ECF8A_E4M3;

__device__ __forceinline__ f32x4 mfma_bf16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int TYPE>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
{
    if constexpr (TYPE == kBf16) return mfma_bf16(a, b, c);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 16 bytes.  ALIGNED: on a 16-byte border; else anywhere (the card takes 16-byte
// accesses at any address, lines apart at the cost of a second line).
typedef u32x4 __attribute__((aligned(1))) u32x4_any;

template <bool ALIGNED>
__device__ __forceinline__ u32x4 load16(const void* p)
{
    if constexpr (ALIGNED) return *static_cast<const u32x4*>(p);
    return *static_cast<const u32x4_any*>(p);
}

// Aligned: past the caches, for results that this library does not read again.
template <bool ALIGNED>
__device__ __forceinline__ void store16(void* p, u32x4 v)
{
    if constexpr (ALIGNED) __builtin_nontemporal_store(v, static_cast<u32x4*>(p));
    else *static_cast<u32x4_any*>(p) = v;
}

// The two values of a dword of 16-bit type.
template <int TYPE>
__device__ __forceinline__ f32x2 unpack2(uint32_t v)
{
    if constexpr (TYPE == kBf16)
        return f32x2{__builtin_bit_cast(float, v << 16), __builtin_bit_cast(float, v & 0xFFFF0000u)};
    const f16x2 h = __builtin_bit_cast(f16x2, v);
    return f32x2{(float)h[0], (float)h[1]};
}

// Rounds two float32 to a dword of 16-bit type (round to nearest even).
template <int TYPE>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if constexpr (TYPE == kBf16) return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
}

template <int TYPE>
__device__ __forceinline__ float load1(const uint16_t* p)
{
    if constexpr (TYPE == kBf16) return __builtin_bit_cast(float, (uint32_t)*p << 16);
    return (float)__builtin_bit_cast(_Float16, *p);
}

template <int TYPE>
__device__ __forceinline__ uint16_t round1(float v)
{
    return (uint16_t)pack2<TYPE>(v, 0.0f);
}

// A float32 as the sum of two bfloat16, for the matrix instruction: hi is v
// rounded, lo the rest rounded, together within 2^-16 of v (a bfloat16 alone:
// 2^-8).  A float16 value (11 significant bits) is held exactly.  Where hi is
// infinite or NaN, lo is 0, so that products keep what hi makes of them.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo)
{
    hi = pack2<kBf16>(a, b);
    const f32x2 h = unpack2<kBf16>(hi);
    const float la = a - h[0], lb = b - h[1];
    lo = pack2<kBf16>(__builtin_fabsf(la) < 3.0e38f ? la : 0.0f, __builtin_fabsf(lb) < 3.0e38f ? lb : 0.0f);
}

// Eight float32 as two bfloat16 operands.
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, u32x4& hi, u32x4& lo)
{
    uint32_t h[4], l[4];
    split2(a[0], a[1], h[0], l[0]);
    split2(a[2], a[3], h[1], l[1]);
    split2(b[0], b[1], h[2], l[2]);
    split2(b[2], b[3], h[3], l[3]);
    hi = u32x4{h[0], h[1], h[2], h[3]};
    lo = u32x4{l[0], l[1], l[2], l[3]};
}

// Eight float16 as two bfloat16 operands.
__device__ __forceinline__ void split8_f16(u32x4 v, u32x4& hi, u32x4& lo)
{
    const f32x2 a = unpack2<kFp16>(v[0]), b = unpack2<kFp16>(v[1]), c = unpack2<kFp16>(v[2]), d = unpack2<kFp16>(v[3]);
    split8(f32x4{a[0], a[1], b[0], b[1]}, f32x4{c[0], c[1], d[0], d[1]}, hi, lo);
}

// A bfloat16 operand with 0 in place of infinities and NaN: for the product with a
// lower half, which may be 0 or of the other sign and would make a NaN of what the
// upper half's product says rightly.
__device__ __forceinline__ u32x4 finite(u32x4 v)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if ((v[i] & 0x7F80u) == 0x7F80u) v[i] &= 0xFFFF0000u;
        if ((v[i] & 0x7F800000u) == 0x7F800000u) v[i] &= 0xFFFFu;
    }
    return v;
}

// Whether a result of the wave is not finite: then, and only then, infinities may
// have met lower halves, and the products are done again with `finite` in place.
template <int N>
__device__ __forceinline__ bool any_not_finite(const f32x4* acc)
{
    float test = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) test = __builtin_fmaf(acc[j][i], 0.0f, test);
    return __ballot(test != test) != 0;
}

// Eight rows of eight 16-bit columns, one row in each w[q], turned into one
// operand for each column: t[j] holds column j of rows 0 .. 7.
__device__ __forceinline__ void transpose8(const u32x4 w[8], u32x4 t[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t sel = (j & 1) ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int p = 0; p < 4; ++p)
            t[j][p] = __builtin_amdgcn_perm(w[2 * p + 1][j >> 1], w[2 * p][j >> 1], sel);
    }
}

inline bool aligned(const void* p, uint64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

inline uint64_t round_up(uint64_t v, uint64_t unit) { return (v + unit - 1) / unit * unit; }

inline int launch_status() { return hipGetLastError() == hipSuccess ? ECF8_OK : ECF8_ERR_HIP; }

}  // namespace ecf8a

#endif
