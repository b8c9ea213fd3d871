// ecf8x_common.h -- what the kernels of 4-bit weights and of experts share:
// sizes of the stored form, widening, and the sum of shares.
//
// A lane that holds 16 bytes of a 4-bit row holds one block of 32 values with
// one scale, four operands of the 16x16x32 instruction; 16 bytes of an E4M3 row
// are two.  Which values sit in which reduction slot is free as long as both
// operands agree, so a lane group g takes the 16-byte chunks 4 (u + g) .. + 3 of
// a row: 64 contiguous bytes, and for 4 bits one aligned dword of scales.
#ifndef ECF8X_COMMON_H
#define ECF8X_COMMON_H

#include "ecf8a_common.h"
#include "ecf8x.h"

namespace ecf8x {

using namespace ecf8a;

constexpr int kMx4 = ECF8X_MX4;

typedef int i32x8 __attribute__((ext_vector_type(8)));

inline uint64_t padded(uint64_t cols) { return round_up(cols, ECF8X_PITCH); }

// The float that a scale byte stands for, as the conversions take it: they read
// the exponent field alone (0 is 2^-127, 255 NaN), so that neighbouring bytes may
// come along.  Byte `at` of a dword, and the low byte.
__device__ __forceinline__ float scale_at(uint32_t dword, int at)
{
    return __builtin_bit_cast(float, at == 3 ? dword >> 1 : dword << (23 - 8 * at));
}

__device__ __forceinline__ float scale_of(uint32_t low) { return scale_at(low, 0); }

// Eight codes of a dword, times the scale, as one bfloat16 operand.  Exact.
__device__ __forceinline__ u32x4 widen4(uint32_t codes, float scale)
{
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3))};
}

// Eight codes of a dword as they are, without their scale, as one float16 operand.
__device__ __forceinline__ u32x4 widen4_f16(uint32_t codes)
{
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3))};
}

// The value of a scale, 2^-127 and NaN included: the code of 1 under it.
__device__ __forceinline__ float value_of(float scale) { return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(2u, scale, 0)[0]; }

__device__ __forceinline__ f32x4 mfma_f16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// The value of lane LANE of every 16.
template <int LANE>
__device__ __forceinline__ float of_lane(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x150 + LANE, 0xF, 0xF, true));
}

// Four rows' sums of one block, times the block's scales, which lanes 4 N .. 4 N + 3 of every 16 hold: each lane then converts
// one row's scale for the others, where it would convert those of all.
template <int N>
__device__ __forceinline__ f32x4 add_scaled(f32x4 acc, f32x4 block, float scale)
{
    return f32x4{__builtin_fmaf(of_lane<4 * N>(scale), block[0], acc[0]), __builtin_fmaf(of_lane<4 * N + 1>(scale), block[1], acc[1]),
                 __builtin_fmaf(of_lane<4 * N + 2>(scale), block[2], acc[2]), __builtin_fmaf(of_lane<4 * N + 3>(scale), block[3], acc[3])};
}

// Two float32 as the sums of three bfloat16, for the matrix instruction: hi is the value rounded, mid the rest rounded, low
// what is left of 24 bits, eight of them: exact down to bfloat16's smallest step, 2^-133.  Where hi is infinite or NaN the
// others are 0.
__device__ __forceinline__ void split3(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& low)
{
    hi = pack2<kBf16>(a, b);
    const f32x2 h = unpack2<kBf16>(hi);
    const float ra = __builtin_fabsf(a - h[0]) < 3.0e38f ? a - h[0] : 0.0f, rb = __builtin_fabsf(b - h[1]) < 3.0e38f ? b - h[1] : 0.0f;
    mid = pack2<kBf16>(ra, rb);
    const f32x2 m = unpack2<kBf16>(mid);
    low = pack2<kBf16>(ra - m[0], rb - m[1]);
}

// Eight E4M3 bytes as one operand of a 16-bit type.  Exact.
template <int TYPE>
__device__ __forceinline__ u32x4 widen8(uint32_t a, uint32_t b)
{
    if constexpr (TYPE == kBf16)
        return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true))};
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true))};
}

// The scaled product of two 4-bit operands of 128 values; byte OP of a and b scales.
template <int OP>
__device__ __forceinline__ f32x4 mfma_mx4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb)
{
    const i32x8 x{(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0}, y{(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, OP, (int)sa, OP, (int)sb);
}

// Stores the first `count` of four values in a 16-bit type, eight bytes at any
// address where all are wanted.  (Value by value where rows have an odd length:
// 1024 x 13821 x 5120 from 4 bits took 78 us where this takes 67.)
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

template <int TYPE>
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v, int count)
{
    if (count >= 4) {
        *reinterpret_cast<u32x2_any*>(p) = u32x2_any{pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3])};
        return;
    }
#pragma unroll
    for (int i = 0; i < 3; ++i)
        if (i < count) p[i] = round1<TYPE>(v[i]);
}

// Sums `shares` planes [share][rows][pitch] in order, adds the bias and rounds.
// pitch: cols rounded up to 4.
template <int TYPE>
__global__ __launch_bounds__(256) void join_kernel(const float* planes, int64_t rows, int cols, int pitch, int shares,
                                                   const uint16_t* bias, uint16_t* out, int64_t ld)
{
    const int64_t plane = rows * pitch, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= plane) return;
    f32x4 s{0, 0, 0, 0};
    for (int p = 0; p < shares; p += 8) {                     // eight loads in flight, added in order
        f32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const f32x4*>(planes + min(p + j, shares - 1) * plane + i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (p + j < shares) s += v[j];
    }
    const int64_t t = i / pitch;
    const int c = (int)(i - t * pitch);
    if (bias) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < cols) s[j] += load1<TYPE>(bias + c + j);
    }
    store4<TYPE>(out + t * ld + c, s, cols - c);
}

}  // namespace ecf8x

#endif
