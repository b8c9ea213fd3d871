// ecf8a_linear.hip -- the gradient a frozen E4M3 weight passes to its input:
// dx = w_scale * dy w, dy (T x N) in a 16-bit type, w (N x K) E4M3 bytes.
//
// Each E4M3 value is exact in bfloat16 and in float16, so the weight is widened
// in registers and the 16-bit matrix instruction gives exact products, summed
// in float32 over N; w_scale is applied to the sum, which is rounded once.
#include "ecf8a_common.h"

namespace {

using namespace ecf8a;

constexpr int kThreads = 512;              // eight waves
constexpr int kJoinThreads = 256;

struct GradArgs {
    const uint16_t* dy;
    int64_t ld_dy;
    const uint8_t* w;
    const float* w_scale;
    uint16_t* dx;
    int64_t ld_dx;
    float* planes;           // [share][tokens][in_features]; nullptr: one share, written to dx
    int64_t tokens;
    int n, k, share;         // share: reduction length of one of gridDim.y shares, a multiple of 128
    int tiles_m, tiles_n;
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

typedef __attribute__((address_space(1))) const void GlobalMem;
typedef __attribute__((address_space(3))) void LdsMem;

// One workgroup: BM tokens by BN columns of dx, eight waves in WM rows of WN,
// the reduction BK rows of the weight at a time through two LDS buffers.
//
// dy goes from memory to LDS without passing registers, 16 bytes a lane.  The
// weight passes registers once: a thread takes eight rows of four bytes, turns
// them, widens them, and leaves one 16-byte operand for each of four columns, so
// each byte is converted once for all eight waves.  Both tiles are rows of
// 16-byte units along the reduction; unit u of row r sits at u ^ swizzle(r), and
// sixteen lanes that read one unit of sixteen rows (or write it) meet different
// banks.
//
// The weight is operand A and dy operand B, so a lane's results belong to one
// token; the matrix instruction's rows are dealt to columns so that they are
// 4 NF consecutive ones, stored 16 bytes at a time.
template <int TYPE, int BM, int BN, int BK, int WM, int WN>
struct Tile {
    static constexpr int MF = BM / WM / 16, NF = BN / WN / 16, CH = BK / 8;
    static constexpr int kA = BM * CH, kB = BN * CH;           // 16-byte units of the two tiles
    static constexpr int kUnitsA = (kA + kThreads - 1) / kThreads, kUnitsB = (CH * BN / 4 + kThreads - 1) / kThreads;
    static_assert(WM * WN == kThreads / 64 && MF >= 1 && NF >= 2, "eight waves");
    static_assert(kA % 64 == 0 && (CH * BN / 4) % 64 == 0, "whole waves stage");

    static __device__ __forceinline__ int swizzle_b(int col) { return (col ^ (col >> 3)) & 7; }

    // dy's tile, straight to LDS.  Tokens past the last read the last one's row.
    static __device__ __forceinline__ void stage_a(const GradArgs& A, int64_t t0, int n, u32x4* lds)
    {
#pragma unroll
        for (int i = 0; i < kUnitsA; ++i) {
            const int first = i * kThreads + (threadIdx.x & ~63), u = first + (threadIdx.x & 63);
            if (kA % kThreads && first >= kA) break;
            const int row = u / CH, ch = (u % CH) ^ (row & 7);
            const int64_t t = min(t0 + row, A.tokens - 1);
            __builtin_amdgcn_global_load_lds((GlobalMem*)(A.dy + t * A.ld_dy + n + 8 * ch), (LdsMem*)(lds + first), 16, 0, 0);
        }
    }

    // The same where the reduction ends inside the tile: zeros past n1.
    static __device__ __forceinline__ void stage_a_tail(const GradArgs& A, int64_t t0, int n, int n1, u32x4* lds)
    {
        for (int u = threadIdx.x; u < kA; u += kThreads) {
            const int row = u / CH, ch = (u % CH) ^ (row & 7);
            const int64_t t = min(t0 + row, A.tokens - 1);
            u32x4 v{0, 0, 0, 0};
            if (n + 8 * ch < n1) v = *reinterpret_cast<const u32x4*>(A.dy + t * A.ld_dy + n + 8 * ch);
            lds[u] = v;
        }
    }

    // The weight's bytes for this thread: rows n + 8 oct .. + 7, columns 4 quad .. + 3 (TAIL: zeros past n1; a whole
    // tile is not looked at between its loads and its use, so that they stay in flight).
    template <bool TAIL>
    static __device__ __forceinline__ void load_b(const GradArgs& A, int k0, int n, int n1, uint32_t (*w)[8])
    {
#pragma unroll
        for (int i = 0; i < kUnitsB; ++i) {
            const int u = i * kThreads + threadIdx.x, quad = u % (BN / 4), oct = u / (BN / 4);
            const int col = k0 + 4 * quad < A.k ? k0 + 4 * quad : 0;
            const bool in = oct < CH && (!TAIL || n + 8 * oct < n1);
            const uint8_t* p = A.w + (int64_t)(in ? n + 8 * oct : 0) * A.k + col;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                w[i][q] = *reinterpret_cast<const uint32_t*>(p + (int64_t)q * A.k);
                if (TAIL && !in) w[i][q] = 0;
            }
        }
    }

    static __device__ __forceinline__ void store_b(const uint32_t (*w)[8], u32x4* lds)
    {
#pragma unroll
        for (int i = 0; i < kUnitsB; ++i) {
            const int u = i * kThreads + threadIdx.x, quad = u % (BN / 4), oct = u / (BN / 4);
            if ((CH * BN / 4) % kThreads && oct >= CH) break;
            uint32_t lo[4], hi[4];
            transpose4(w[i], lo);
            transpose4(w[i] + 4, hi);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                lds[(4 * quad + j) * CH + (oct ^ swizzle_b(4 * quad + j))] =
                    u32x4{widen2<TYPE, false>(lo[j]), widen2<TYPE, true>(lo[j]), widen2<TYPE, false>(hi[j]), widen2<TYPE, true>(hi[j])};
        }
    }

    static __device__ __forceinline__ void multiply(const u32x4* la, const u32x4* lb, int wm, int wn, f32x4 (*acc)[NF])
    {
        const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk) {
            u32x4 a[MF], b[NF];
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                const int row = wm * (BM / WM) + m * 16 + c;
                a[m] = la[row * CH + ((kk * 4 + g) ^ (row & 7))];
            }
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                const int col = wn * (BN / WN) + (c >> 2) * (4 * NF) + n * 4 + (c & 3);
                b[n] = lb[col * CH + ((kk * 4 + g) ^ swizzle_b(col))];
            }
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
                for (int n = 0; n < NF; ++n) acc[m][n] = mfma<TYPE>(b[n], a[m], acc[m][n]);
        }
    }
};

template <int TYPE, int BM, int BN, int BK, int WM, int WN>
__global__ __launch_bounds__(kThreads) void input_grad_kernel(GradArgs A)
{
    typedef Tile<TYPE, BM, BN, BK, WM, WN> S;
    extern __shared__ u32x4 lds[];
    u32x4* const la = lds;
    u32x4* const lb = lds + 2 * S::kA;
    const int wave = threadIdx.x >> 6, wm = wave / WN, wn = wave % WN;
    // Workgroups go to the eight dies in turn; each die gets a run of tiles, in
    // columns of eight tiles down the tokens, so that its cache sees the same rows
    // of dy and columns of the weight again.
    const int total = A.tiles_m * A.tiles_n;
    int id = blockIdx.x;
    if (total % 8 == 0) id = (id % 8) * (total / 8) + id / 8;
    const int band = id / (8 * A.tiles_n), rows = min(8, A.tiles_m - band * 8), in_band = id - band * 8 * A.tiles_n;
    const int tm = band * 8 + in_band % rows, tn = in_band / rows;
    const int64_t t0 = (int64_t)tm * BM;
    const int k0 = tn * BN;
    const int n0 = blockIdx.y * A.share, n1 = min(A.n, n0 + A.share), steps = (n1 - n0) / BK;
    f32x4 acc[S::MF][S::NF] = {};
    uint32_t w[S::kUnitsB][8];
    if (steps > 0) {
        S::stage_a(A, t0, n0, la);
        S::template load_b<false>(A, k0, n0, n1, w);
        S::store_b(w, lb);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
    for (int s = 0; s < steps; ++s) {
        const int cur = s & 1;
        if (s + 1 < steps) {
            S::stage_a(A, t0, n0 + (s + 1) * BK, la + (cur ^ 1) * S::kA);
            S::template load_b<false>(A, k0, n0 + (s + 1) * BK, n1, w);
        }
        S::multiply(la + cur * S::kA, lb + cur * S::kB, wm, wn, acc);
        if (s + 1 < steps) S::store_b(w, lb + (cur ^ 1) * S::kB);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
    }
    if (n0 + steps * BK < n1) {
        S::stage_a_tail(A, t0, n0 + steps * BK, n1, la);
        S::template load_b<true>(A, k0, n0 + steps * BK, n1, w);
        S::store_b(w, lb);
        __syncthreads();
        S::multiply(la, lb, wm, wn, acc);
    }
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int col = k0 + wn * (BN / WN) + g * (4 * S::NF);
    if (col >= A.k) return;                                   // K and 4 NF: multiples of 8, so groups of eight are in or out
    const float scale = *A.w_scale;
#pragma unroll
    for (int m = 0; m < S::MF; ++m) {
        const int64_t t = t0 + wm * (BM / WM) + m * 16 + c;
        if (t >= A.tokens) continue;
#pragma unroll
        for (int n = 0; n < S::NF; n += 2) {
            if (col + 4 * n >= A.k) continue;
            const f32x4 v0 = acc[m][n], v1 = acc[m][n + 1];
            if (A.planes) {
                float* p = A.planes + ((int64_t)blockIdx.y * A.tokens + t) * A.k + col + 4 * n;
                *reinterpret_cast<f32x4*>(p) = v0;
                *reinterpret_cast<f32x4*>(p + 4) = v1;
            } else {
                *reinterpret_cast<u32x4*>(A.dx + t * A.ld_dx + col + 4 * n) =
                    u32x4{pack2<TYPE>(v0[0] * scale, v0[1] * scale), pack2<TYPE>(v0[2] * scale, v0[3] * scale),
                          pack2<TYPE>(v1[0] * scale, v1[1] * scale), pack2<TYPE>(v1[2] * scale, v1[3] * scale)};
            }
        }
    }
}

// Sums the shares in order, scales and rounds.
template <int TYPE>
__global__ __launch_bounds__(kJoinThreads) void grad_join_kernel(GradArgs A, int shares)
{
    const int64_t plane = A.tokens * A.k, i = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (i >= plane) return;
    f32x4 s = *reinterpret_cast<const f32x4*>(A.planes + i);
    for (int p = 1; p < shares; ++p) s += *reinterpret_cast<const f32x4*>(A.planes + p * plane + i);
    const float scale = *A.w_scale;
    const int64_t t = i / A.k;
    uint32_t* p = reinterpret_cast<uint32_t*>(A.dx + t * A.ld_dx + (i - t * A.k));
    p[0] = pack2<TYPE>(s[0] * scale, s[1] * scale);
    p[1] = pack2<TYPE>(s[2] * scale, s[3] * scale);
}

// The tile for a size, and the shares that the reduction is cut into where too
// few tiles are left to fill the card.
struct Shape {
    int bm, bn;
    uint32_t shares;
};

Shape shape_of(uint64_t tokens, uint64_t n, uint64_t k)
{
    const auto tiles = [&](uint64_t m, uint64_t c) { return ((tokens + m - 1) / m) * ((k + c - 1) / c); };
    if (tokens > 64 && tiles(256, 256) >= 192) return Shape{256, 256, 1};
    const int bm = tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128;
    const uint64_t t = tiles(bm, 128);
    uint64_t s = t ? 512 / t : 1;
    if (s > n / 512) s = n / 512;
    return Shape{bm, 128, (uint32_t)(s < 1 ? 1 : s > 32 ? 32 : s)};
}

bool sizes_ok(uint64_t tokens, uint64_t n, uint64_t k)
{
    return tokens <= ECF8A_MAX_TOKENS && n >= 16 && n <= ECF8A_MAX_FEATURES && n % 16 == 0 && k >= 16 &&
           k <= ECF8A_MAX_FEATURES && k % 16 == 0;
}

template <int TYPE, int BM, int BN, int BK, int WM, int WN>
int launch(GradArgs A, uint32_t shares, hipStream_t st)
{
    typedef Tile<TYPE, BM, BN, BK, WM, WN> S;
    constexpr int bytes = 2 * (S::kA + S::kB) * 16;
    auto* kernel = input_grad_kernel<TYPE, BM, BN, BK, WM, WN>;
    if (bytes > 65536 &&
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
        return ECF8_ERR_HIP;
    A.tiles_m = (int)((A.tokens + BM - 1) / BM);
    A.tiles_n = (A.k + BN - 1) / BN;
    kernel<<<dim3((uint32_t)A.tiles_m * A.tiles_n, shares), kThreads, bytes, st>>>(A);
    return launch_status();
}

template <int TYPE>
int run(const GradArgs& A, const Shape& s, hipStream_t st)
{
    int rc;
    if (s.bm == 256) rc = launch<TYPE, 256, 256, 64, 2, 4>(A, 1, st);
    else if (s.bm == 128) rc = launch<TYPE, 128, 128, 128, 2, 4>(A, s.shares, st);
    else if (s.bm == 64) rc = launch<TYPE, 64, 128, 128, 2, 4>(A, s.shares, st);
    else rc = launch<TYPE, 32, 128, 128, 2, 4>(A, s.shares, st);
    if (rc != ECF8_OK || s.shares < 2) return rc;
    const uint32_t join = (uint32_t)((A.tokens * A.k / 4 + kJoinThreads - 1) / kJoinThreads);
    grad_join_kernel<TYPE><<<join, kJoinThreads, 0, st>>>(A, (int)s.shares);
    return launch_status();
}

}  // namespace

extern "C" uint64_t ecf8a_input_grad_bytes(uint64_t tokens, uint64_t out_features, uint64_t in_features)
{
    if (!sizes_ok(tokens, out_features, in_features)) return 0;
    const uint64_t s = shape_of(tokens, out_features, in_features).shares;
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
    const Shape s = shape_of(tokens, out_features, in_features);
    const GradArgs A{static_cast<const uint16_t*>(dy), (int64_t)ld_dy, w, w_scale, static_cast<uint16_t*>(dx), (int64_t)ld_dx,
                     s.shares > 1 ? static_cast<float*>(workspace) : nullptr, (int64_t)tokens, (int)out_features,
                     (int)in_features, (int)round_up((out_features + s.shares - 1) / s.shares, 128), 0, 0};
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    return type == ECF8A_BF16 ? run<kBf16>(A, s, st) : run<kFp16>(A, s, st);
}
