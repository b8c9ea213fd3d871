// ecf8a_linear.hip -- the gradient a frozen E4M3 weight passes to its input:
// dx = w_scale * dy w, dy (T x N) in a 16-bit type, w (N x K) E4M3 bytes.
//
// Each E4M3 value is exact in bfloat16 and in float16, so the weight is widened
// in registers and the 16-bit matrix instruction gives exact products, summed
// in float32 over N; w_scale is applied to the sum, which is rounded once.
#include "ecf8a_common.h"

namespace {

using namespace ecf8a;

constexpr int kThreads = 256;
constexpr int kTileT = 128, kTileK = 128;
constexpr int kWaveT = 64, kWaveK = 64;

struct GradArgs {
    const uint16_t* dy;
    int64_t ld_dy;
    const uint8_t* w;
    const float* w_scale;
    uint16_t* dx;
    int64_t ld_dx;
    float* planes;           // [share][tokens][in_features]; nullptr: one share, written to dx
    int64_t tokens;
    int n, k, share;         // share: reduction length of one of gridDim.z shares, a multiple of 32
};

// Two E4M3 bytes of a dword (the lower or the upper pair) widened.
template <int TYPE, bool UPPER>
__device__ __forceinline__ uint32_t widen2(uint32_t b)
{
    if constexpr (TYPE == kBf16)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, UPPER));
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, UPPER));
}

// Four rows of four bytes turned: out[j] holds column j's four rows.
__device__ __forceinline__ void transpose4(const uint32_t r[4], uint32_t out[4])
{
    const uint32_t a = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), b = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
    const uint32_t c = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u), d = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
    out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
    out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
    out[2] = __builtin_amdgcn_perm(d, b, 0x05040100u);
    out[3] = __builtin_amdgcn_perm(d, b, 0x07060302u);
}

// One workgroup: 128 tokens by 128 columns, a wave 64 by 64, operands straight
// from memory.  A lane's four columns are consecutive, so a weight row is read
// four bytes at a time; eight rows are turned into one operand per column.
template <int TYPE>
__global__ __launch_bounds__(kThreads) void input_grad_kernel(GradArgs A)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.y * kTileT + (wave >> 1) * kWaveT;
    const int k0 = blockIdx.x * kTileK + (wave & 1) * kWaveK + 4 * c;
    const int kc = k0 < A.k ? k0 : 0;
    const uint16_t* row[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int64_t t = t0 + m * 16 + c;
        row[m] = A.dy + (t < A.tokens ? t : A.tokens - 1) * A.ld_dy;
    }
    f32x4 acc[4][4] = {};
    const int n0 = blockIdx.z * A.share, n1 = min(A.n, n0 + A.share);
    for (int n = n0 + 8 * g; n - 8 * g < n1; n += 32) {
        const bool in = n < A.n;                              // A.n is a multiple of 16: eight values are in or out
        const int ns = in ? n : 0;
        u32x4 a[4];
        uint32_t w[8], lo[4], hi[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            a[m] = *reinterpret_cast<const u32x4*>(row[m] + ns);
            if (!in) a[m] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            w[q] = *reinterpret_cast<const uint32_t*>(A.w + (int64_t)(ns + q) * A.k + kc);
            if (!in) w[q] = 0;
        }
        transpose4(w, lo);
        transpose4(w + 4, hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const u32x4 b{widen2<TYPE, false>(lo[j]), widen2<TYPE, true>(lo[j]), widen2<TYPE, false>(hi[j]), widen2<TYPE, true>(hi[j])};
#pragma unroll
            for (int m = 0; m < 4; ++m) acc[m][j] = mfma<TYPE>(a[m], b, acc[m][j]);
        }
    }
    if (k0 >= A.k) return;
    const float scale = *A.w_scale;
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t t = t0 + m * 16 + 4 * g + i;
            if (t >= A.tokens) continue;
            const f32x4 v{acc[m][0][i], acc[m][1][i], acc[m][2][i], acc[m][3][i]};
            if (A.planes) {
                *reinterpret_cast<f32x4*>(A.planes + ((int64_t)blockIdx.z * A.tokens + t) * A.k + k0) = v;
            } else {
                uint32_t* p = reinterpret_cast<uint32_t*>(A.dx + t * A.ld_dx + k0);
                p[0] = pack2<TYPE>(v[0] * scale, v[1] * scale);
                p[1] = pack2<TYPE>(v[2] * scale, v[3] * scale);
            }
        }
}

// Sums the shares in order, scales and rounds.
template <int TYPE>
__global__ __launch_bounds__(kThreads) void grad_join_kernel(GradArgs A, int shares)
{
    const int64_t plane = A.tokens * A.k, i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (i >= plane) return;
    f32x4 s = *reinterpret_cast<const f32x4*>(A.planes + i);
    for (int p = 1; p < shares; ++p) s += *reinterpret_cast<const f32x4*>(A.planes + p * plane + i);
    const float scale = *A.w_scale;
    const int64_t t = i / A.k;
    uint32_t* p = reinterpret_cast<uint32_t*>(A.dx + t * A.ld_dx + (i - t * A.k));
    p[0] = pack2<TYPE>(s[0] * scale, s[1] * scale);
    p[1] = pack2<TYPE>(s[2] * scale, s[3] * scale);
}

// Shares that the reduction is cut into where the output has too few tiles to
// fill the card, each of at least 256 rows of the weight.
uint32_t shares_of(uint64_t tokens, uint64_t n, uint64_t k)
{
    const uint64_t tiles = ((tokens + kTileT - 1) / kTileT) * ((k + kTileK - 1) / kTileK);
    uint64_t s = tiles ? 768 / tiles : 1;
    if (s > n / 256) s = n / 256;
    return (uint32_t)(s < 1 ? 1 : s > 32 ? 32 : s);
}

bool sizes_ok(uint64_t tokens, uint64_t n, uint64_t k)
{
    return tokens <= ECF8A_MAX_TOKENS && n >= 16 && n <= ECF8A_MAX_FEATURES && n % 16 == 0 && k >= 16 &&
           k <= ECF8A_MAX_FEATURES && k % 16 == 0 && (tokens + kTileT - 1) / kTileT <= 65535;
}

}  // namespace

extern "C" uint64_t ecf8a_input_grad_bytes(uint64_t tokens, uint64_t out_features, uint64_t in_features)
{
    if (!sizes_ok(tokens, out_features, in_features)) return 0;
    const uint64_t s = shares_of(tokens, out_features, in_features);
    return s > 1 ? round_up(4 * s * tokens * in_features, 256) : 0;
}

extern "C" int ecf8a_input_grad(const void* dy, uint64_t ld_dy, uint64_t tokens, uint64_t out_features, const uint8_t* w,
                                uint64_t in_features, const float* w_scale, uint32_t type, void* dx, uint64_t ld_dx,
                                void* workspace, uint64_t workspace_bytes, void* hip_stream)
{
    if (type != ECF8A_BF16 && type != ECF8A_FP16) return ECF8_ERR_UNSUPPORTED;
    if (!sizes_ok(tokens, out_features, in_features)) return ECF8_ERR_SIZE;
    if (tokens == 0) return ECF8_OK;
    if (!dy || !w || !w_scale || !dx || !aligned(dy, 16) || !aligned(w, 16) || !aligned(w_scale, 4) || !aligned(dx, 16) ||
        (tokens > 1 && (ld_dy % 8 || ld_dx % 8)))
        return ECF8_ERR_ARG;
    if (ld_dy < out_features || ld_dx < in_features) return ECF8_ERR_SIZE;
    const uint64_t need = ecf8a_input_grad_bytes(tokens, out_features, in_features);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return ECF8_ERR_WORKSPACE;
    const uint32_t shares = shares_of(tokens, out_features, in_features);
    GradArgs A{static_cast<const uint16_t*>(dy), (int64_t)ld_dy, w, w_scale, static_cast<uint16_t*>(dx), (int64_t)ld_dx,
               shares > 1 ? static_cast<float*>(workspace) : nullptr, (int64_t)tokens, (int)out_features, (int)in_features,
               (int)round_up((out_features + shares - 1) / shares, 32)};
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    const dim3 grid((uint32_t)((in_features + kTileK - 1) / kTileK), (uint32_t)((tokens + kTileT - 1) / kTileT), shares);
    if (type == ECF8A_BF16) input_grad_kernel<kBf16><<<grid, kThreads, 0, st>>>(A);
    else input_grad_kernel<kFp16><<<grid, kThreads, 0, st>>>(A);
    if (shares > 1) {
        const dim3 join((uint32_t)((tokens * in_features / 4 + kThreads - 1) / kThreads));
        if (type == ECF8A_BF16) grad_join_kernel<kBf16><<<join, kThreads, 0, st>>>(A, (int)shares);
        else grad_join_kernel<kFp16><<<join, kThreads, 0, st>>>(A, (int)shares);
    }
    return launch_status();
}
