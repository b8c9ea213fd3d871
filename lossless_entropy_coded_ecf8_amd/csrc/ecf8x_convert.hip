// ecf8x_convert.hip -- values to microscaled 4-bit floating point and back.
//
// Memory bounds both.  A lane takes eight values, four lanes one block of 32:
// the block's largest magnitude is found by two exchanges between them, every
// load is a whole run of a wave's lanes, and a lane stores its codes as one
// dword.  The largest magnitude is compared as an integer, so that infinities
// and NaN are larger than every number.  Rows without a gap and aligned ones need
// no kernel of their own: one with 16-byte loads known to be aligned, over one long
// row, took as long (28672 x 8192 bfloat16: 107 us and 106).
//
// Measured: 28672 x 8192 bfloat16 quantised in 104 us, 595 MB read and written at
// 5.7 TB/s; E4M3 of the same size in 63, and back to bfloat16 in 84.
#include "ecf8x_common.h"

namespace {

using namespace ecf8x;

constexpr int kFp32 = ECF8A_FP32, kThreads = 256, kUnits = 4;      // units of eight values a lane, in flight together

struct ConvertArgs {
    const void* x;
    void* out;
    const float* x_scale;
    uint8_t *codes, *scales;
    const uint8_t *codes_in, *scales_in;
    int64_t ld;
    uint32_t units_row, units_in, total;     // units of a stored row, of them before the last value; units of this launch
};

// Eight values as they are stored, and as float32.
template <int TYPE>
struct Unit {
    static constexpr int WORDS = TYPE == kFp32 ? 8 : TYPE == kE4m3 ? 2 : 4;
    uint32_t raw[WORDS];

    __device__ __forceinline__ void load(const void* x, int64_t at)
    {
        const char* p = static_cast<const char*>(x) + at * WORDS / 2;
        if constexpr (WORDS == 2) {
            __builtin_memcpy(raw, p, 8);
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const u32x4 d = load16<false>(p + 4 * i);
#pragma unroll
                for (int j = 0; j < 4; ++j) raw[i + j] = d[j];
            }
        }
    }

    // mask: 0 makes them zeros, whatever the factor is.
    __device__ __forceinline__ void widen(uint32_t mask, float factor, float v[8]) const
    {
        factor = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, factor) & mask);
#pragma unroll
        for (int i = 0; i < WORDS; ++i) {
            const uint32_t d = raw[i] & mask;
            if constexpr (TYPE == kFp32) {
                v[i] = __builtin_bit_cast(float, d);
            } else if constexpr (TYPE == kE4m3) {
                const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(d, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(d, true);
                v[4 * i] = lo[0] * factor, v[4 * i + 1] = lo[1] * factor, v[4 * i + 2] = hi[0] * factor, v[4 * i + 3] = hi[1] * factor;
            } else {
                const f32x2 p = unpack2<TYPE>(d);
                v[2 * i] = p[0], v[2 * i + 1] = p[1];
            }
        }
    }
};

__device__ __forceinline__ uint32_t of_block(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));       // lane ^ 1
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));    // lane ^ 2
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void quantize_kernel(ConvertArgs A)
{
    const float factor = TYPE == kE4m3 && A.x_scale ? *A.x_scale : 1.0f;
    // Units past the end or in the padding load the first one: a branch would make each wait for its own load.
    Unit<TYPE> x[kUnits];
    uint32_t unit[kUnits], mask[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = unit[i] = (blockIdx.x * kUnits + i) * (uint32_t)kThreads + threadIdx.x;
        const uint32_t row = u / A.units_row, col = u - row * A.units_row;
        const bool in = u < A.total && col < A.units_in;
        mask[i] = in ? ~0u : 0;
        x[i].load(A.x, in ? (int64_t)row * A.ld + col * 8 : 0);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        float v[8];
        x[i].widen(mask[i], factor, v);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
        const uint32_t e = of_block(m) >> 23;
        const uint32_t s = e == 255 ? 255 : max(e, 2u) - 2;
        const float scale = scale_of(s);
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], scale, 3);
        if (s == 255) c = 0;
        if (unit[i] < A.total) {
            reinterpret_cast<uint32_t*>(A.codes)[unit[i]] = c;
            if ((unit[i] & 3) == 0) A.scales[unit[i] >> 2] = (uint8_t)s;
        }
    }
}

// A lane writes 16 bytes, so that a wave's run has no gaps: eight values of 16 bits, four of float32.  (Eight of these in two
// stores: 28672 x 8192 in 278 us, past the cache 399, and so 158, 6.7 TB/s.)
template <int TYPE>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(ConvertArgs A)
{
    constexpr int HALF = TYPE == kFp32;                       // lanes of a unit, less one
    uint32_t c[kUnits], s[kUnits];
    const uint32_t first = blockIdx.x * kUnits * (uint32_t)kThreads + threadIdx.x, total = A.total << HALF;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = first + i * kThreads;
        c[i] = s[i] = 0;
        if (u < total) {
            if constexpr (HALF) c[i] = reinterpret_cast<const uint16_t*>(A.codes_in)[u];
            else c[i] = reinterpret_cast<const uint32_t*>(A.codes_in)[u];
            s[i] = A.scales_in[u >> (2 + HALF)];
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = first + i * kThreads, row = (u >> HALF) / A.units_row, col = (u >> HALF) - row * A.units_row;
        if (u >= total || col >= A.units_in) continue;
        const int64_t at = (int64_t)row * A.ld + col * 8 + (HALF ? 4 * (u & 1) : 0);
        const float scale = scale_of(s[i]);
        if constexpr (TYPE == kBf16) {
            store16<true>(static_cast<uint16_t*>(A.out) + at, widen4(c[i], scale));
        } else {
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 1);
            if constexpr (HALF) {
                store16<true>(static_cast<float*>(A.out) + at, __builtin_bit_cast(u32x4, f32x4{a[0], a[1], b[0], b[1]}));
            } else {
                const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 2), f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 3);
                store16<true>(static_cast<uint16_t*>(A.out) + at,
                              u32x4{pack2<kFp16>(a[0], a[1]), pack2<kFp16>(b[0], b[1]), pack2<kFp16>(d[0], d[1]), pack2<kFp16>(f[0], f[1])});
            }
        }
    }
}

int bytes_of(uint32_t type) { return type == ECF8A_FP32 ? 4 : type == ECF8A_E4M3 ? 1 : 2; }

bool sizes_ok(uint64_t rows, uint64_t cols)
{
    return rows <= ECF8X_MAX_ROWS && cols >= ECF8X_BLOCK && cols <= ECF8A_MAX_FEATURES && cols % ECF8X_BLOCK == 0;
}

// Units, and halves of them, are counted in 32 bits: so many rows go into one launch.
uint64_t rows_of_launch(uint64_t units_row) { return (1ull << 30) / units_row; }

uint32_t grid_of(uint64_t units) { return (uint32_t)((units + kThreads * kUnits - 1) / (kThreads * kUnits)); }

}  // namespace

extern "C" int ecf8x_quantize(const void* x, uint64_t ld_x, uint32_t type, const float* x_scale, uint64_t rows, uint64_t cols,
                              uint8_t* codes, uint8_t* scales, void* hip_stream)
{
    if (type != ECF8A_BF16 && type != ECF8A_FP16 && type != ECF8A_FP32 && type != ECF8A_E4M3) return ECF8_ERR_UNSUPPORTED;
    if (!sizes_ok(rows, cols)) return ECF8_ERR_SIZE;
    if (rows == 0) return ECF8_OK;
    const uint64_t size = bytes_of(type), units_row = padded(cols) / 8;
    if (!x || !codes || !scales || !aligned(x, size) || !aligned(codes, 16) || !aligned(scales, 4) || (x_scale && type != ECF8A_E4M3) ||
        !aligned(x_scale, 4))
        return ECF8_ERR_ARG;
    if (rows > 1 && (ld_x < cols || ld_x > (1ull << 40))) return ECF8_ERR_SIZE;
    if (rows == 1) ld_x = cols;
    for (uint64_t r = 0; r < rows; r += rows_of_launch(units_row)) {
        const uint64_t part = rows - r < rows_of_launch(units_row) ? rows - r : rows_of_launch(units_row);
        ConvertArgs A{};
        A.x = static_cast<const char*>(x) + r * ld_x * size;
        A.x_scale = x_scale;
        A.codes = codes + r * units_row * 4;
        A.scales = scales + r * units_row / 4;
        A.ld = (int64_t)ld_x;
        A.units_row = (uint32_t)units_row;
        A.units_in = (uint32_t)(cols / 8);
        A.total = (uint32_t)(part * units_row);
        const uint32_t grid = grid_of(A.total);
        hipStream_t st = static_cast<hipStream_t>(hip_stream);
        if (type == ECF8A_BF16) quantize_kernel<kBf16><<<grid, kThreads, 0, st>>>(A);
        else if (type == ECF8A_FP16) quantize_kernel<kFp16><<<grid, kThreads, 0, st>>>(A);
        else if (type == ECF8A_FP32) quantize_kernel<kFp32><<<grid, kThreads, 0, st>>>(A);
        else quantize_kernel<kE4m3><<<grid, kThreads, 0, st>>>(A);
        const int rc = launch_status();
        if (rc != ECF8_OK) return rc;
    }
    return ECF8_OK;
}

extern "C" int ecf8x_dequantize(const uint8_t* codes, const uint8_t* scales, uint64_t rows, uint64_t cols, uint32_t type, void* out,
                                uint64_t ld_out, void* hip_stream)
{
    if (type != ECF8A_BF16 && type != ECF8A_FP16 && type != ECF8A_FP32) return ECF8_ERR_UNSUPPORTED;
    if (!sizes_ok(rows, cols)) return ECF8_ERR_SIZE;
    if (rows == 0) return ECF8_OK;
    if (rows == 1) ld_out = cols;
    if (!codes || !scales || !out || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(out, 16) || ld_out % 8) return ECF8_ERR_ARG;
    if (ld_out < cols || ld_out > (1ull << 40)) return ECF8_ERR_SIZE;
    const uint64_t units_row = padded(cols) / 8;
    for (uint64_t r = 0; r < rows; r += rows_of_launch(units_row)) {
        const uint64_t part = rows - r < rows_of_launch(units_row) ? rows - r : rows_of_launch(units_row);
        ConvertArgs A{};
        A.codes_in = codes + r * units_row * 4;
        A.scales_in = scales + r * units_row / 4;
        A.out = static_cast<char*>(out) + r * ld_out * bytes_of(type);
        A.ld = (int64_t)ld_out;
        A.units_row = (uint32_t)units_row;
        A.units_in = (uint32_t)(cols / 8);
        A.total = (uint32_t)(part * units_row);
        const uint32_t grid = grid_of((uint64_t)A.total << (type == ECF8A_FP32));
        hipStream_t st = static_cast<hipStream_t>(hip_stream);
        if (type == ECF8A_BF16) dequantize_kernel<kBf16><<<grid, kThreads, 0, st>>>(A);
        else if (type == ECF8A_FP16) dequantize_kernel<kFp16><<<grid, kThreads, 0, st>>>(A);
        else dequantize_kernel<kFp32><<<grid, kThreads, 0, st>>>(A);
        const int rc = launch_status();
        if (rc != ECF8_OK) return rc;
    }
    return ECF8_OK;
}
