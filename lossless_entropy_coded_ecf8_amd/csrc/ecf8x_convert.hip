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
// Measured: 28672 x 8192 bfloat16 quantised in 106 us, 595 MB read and written at
// 5.6 TB/s; E4M3 of the same size in 69, and back to bfloat16 in 84.
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

// The eight values of unit u of a row.
template <int TYPE>
__device__ __forceinline__ void load8(const void* x, int64_t at, float factor, float v[8])
{
    if constexpr (TYPE == kFp32) {
        const char* p = static_cast<const char*>(x) + 4 * at;
        const f32x4 a = __builtin_bit_cast(f32x4, load16<false>(p)), b = __builtin_bit_cast(f32x4, load16<false>(p + 16));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
    } else if constexpr (TYPE == kE4m3) {
        const char* p = static_cast<const char*>(x) + at;
        uint32_t d[2];
        __builtin_memcpy(d, p, 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(d[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(d[i], true);
            v[4 * i] = lo[0] * factor, v[4 * i + 1] = lo[1] * factor, v[4 * i + 2] = hi[0] * factor, v[4 * i + 3] = hi[1] * factor;
        }
    } else {
        const u32x4 d = load16<false>(static_cast<const char*>(x) + 2 * at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f32x2 p = unpack2<TYPE>(d[i]);
            v[2 * i] = p[0], v[2 * i + 1] = p[1];
        }
    }
}

__device__ __forceinline__ uint32_t of_block(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));       // lane ^ 1
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));    // lane ^ 2
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void quantize_kernel(ConvertArgs A)
{
    const float factor = TYPE == kE4m3 && A.x_scale ? *A.x_scale : 1.0f;
    float v[kUnits][8];
    uint32_t unit[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = unit[i] = (blockIdx.x * kUnits + i) * (uint32_t)kThreads + threadIdx.x;
        const uint32_t row = u / A.units_row, col = u - row * A.units_row;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
        if (u < A.total && col < A.units_in) load8<TYPE>(A.x, (int64_t)row * A.ld + col * 8, factor, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(uint32_t, v[i][j]) & 0x7FFFFFFFu);
        const uint32_t e = of_block(m) >> 23;
        const uint32_t s = e == 255 ? 255 : max(e, 2u) - 2;
        const float scale = scale_of(s);
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[i][0], v[i][1], scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[i][2], v[i][3], scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[i][4], v[i][5], scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[i][6], v[i][7], scale, 3);
        if (s == 255) c = 0;
        if (unit[i] < A.total) {
            reinterpret_cast<uint32_t*>(A.codes)[unit[i]] = c;
            if ((unit[i] & 3) == 0) A.scales[unit[i] >> 2] = (uint8_t)s;
        }
    }
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(ConvertArgs A)
{
    uint32_t unit[kUnits], c[kUnits], s[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = unit[i] = (blockIdx.x * kUnits + i) * (uint32_t)kThreads + threadIdx.x;
        c[i] = s[i] = 0;
        if (u < A.total) {
            c[i] = reinterpret_cast<const uint32_t*>(A.codes_in)[u];
            s[i] = A.scales_in[u >> 2];
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const uint32_t u = unit[i], row = u / A.units_row, col = u - row * A.units_row;
        if (u >= A.total || col >= A.units_in) continue;
        const int64_t at = (int64_t)row * A.ld + col * 8;
        const float scale = scale_of(s[i]);
        if constexpr (TYPE == kBf16) {
            store16<true>(static_cast<uint16_t*>(A.out) + at, widen4(c[i], scale));
        } else {
            const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 1),
                        d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 2), f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], scale, 3);
            if constexpr (TYPE == kFp32) {
                float* p = static_cast<float*>(A.out) + at;
                store16<true>(p, __builtin_bit_cast(u32x4, f32x4{a[0], a[1], b[0], b[1]}));
                store16<true>(p + 4, __builtin_bit_cast(u32x4, f32x4{d[0], d[1], f[0], f[1]}));
            } else {
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

// Units are counted in 32 bits: so many rows go into one launch.
uint64_t rows_of_launch(uint64_t units_row) { return (1ull << 31) / units_row; }

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
        const uint32_t grid = grid_of(A.total);
        hipStream_t st = static_cast<hipStream_t>(hip_stream);
        if (type == ECF8A_BF16) dequantize_kernel<kBf16><<<grid, kThreads, 0, st>>>(A);
        else if (type == ECF8A_FP16) dequantize_kernel<kFp16><<<grid, kThreads, 0, st>>>(A);
        else dequantize_kernel<kFp32><<<grid, kThreads, 0, st>>>(A);
        const int rc = launch_status();
        if (rc != ECF8_OK) return rc;
    }
    return ECF8_OK;
}
