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
    int n, k, share;         // share: reduction length of one of gridDim.y shares, a multiple of 64
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

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void LdsMem;
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 LdsPair;

// Every offset used with it is inside the operand, so the range is left open.
__device__ __forceinline__ Rsrc buffer_of(const void* p)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, -1, 0x00020000);
}

// One workgroup: BM tokens by BN columns of dx, eight waves in WM rows of WN,
// the reduction BK rows of the weight at a time.
//
// Both tiles go from memory to LDS without passing registers, 16 bytes a lane,
// into STAGES buffers: while step s is multiplied, step s + STAGES - 1 is sent
// for and those between are on their way (about 1.5 us for a tile of 128 by 128,
// three times what its products take).  dy's tile is kept by token, 8 values of the
// reduction in a unit, one matrix operand's share of a lane.  The weight's is
// kept as it lies in memory, by row, and is turned by the transposing LDS read:
// each group of 16 lanes reads 8 rows of 16 columns and each lane gets one
// column's 8 rows, still E4M3, which four conversions widen.
//
// The weight is operand A and dy operand B, so a lane's results belong to one
// token, four consecutive columns of each operand.
//
// Banks.  Unit u of dy's row r sits at u ^ (r & 7), unit u of the weight's row r
// at u ^ turn(r): the lanes that a read serves at once take one unit of 16
// consecutive rows, and these cover the banks evenly.
template <int TYPE, int BM, int BN, int BK, int WM, int WN, int STAGES>
struct Tile {
    static constexpr int MF = BM / WM / 16, CH = BK / 8, BU = BN / 16;
    static constexpr int kA = BM * CH, kB = BK * BU;           // 16-byte units of the two tiles
    static constexpr int kUnitsA = (kA + kThreads - 1) / kThreads, kUnitsB = (kB + kThreads - 1) / kThreads;
    static constexpr int kLds = STAGES * 16 * (kA + kB);
    // Loads that may be under way at the end of a step: those of all stages but the next one's.
    static constexpr int kAhead = (STAGES - 2) * (kA / kThreads + kB / kThreads);
    static_assert(STAGES >= 3 && kLds <= 160 * 1024 && kAhead < 64, "LDS and the load counter");
    static_assert(WM * WN == kThreads / 64 && MF >= 1 && BN / WN == 64, "eight waves of 64 columns");
    static_assert(kA % 64 == 0 && kB % 64 == 0 && (BU == 8 || BU == 16), "whole waves stage");

    static __device__ __forceinline__ int turn(int row) { return BU == 16 ? row & 15 : (row ^ (row >> 3)) & 7; }

    // What a lane sends for lies at the same place of every step's tile: byte offsets from the tile's corner, found
    // once.  Tokens past the last read the last one's row, columns past the last the tile's first; neither reaches a
    // result that is stored.
    struct Places {
        uint32_t a[kUnitsA], b[kUnitsB];
    };

    static __device__ __forceinline__ Places places(const GradArgs& A, int64_t t0, int k0)
    {
        Places at;
#pragma unroll
        for (int i = 0; i < kUnitsA; ++i) {
            const int u = i * kThreads + threadIdx.x, row = u / CH, ch = (u % CH) ^ (row & 7);
            at.a[i] = 2 * ((uint32_t)min((int64_t)row, A.tokens - 1 - t0) * (uint32_t)A.ld_dy + 8 * ch);
        }
#pragma unroll
        for (int i = 0; i < kUnitsB; ++i) {
            const int u = i * kThreads + threadIdx.x, row = u / BU, col = 16 * ((u % BU) ^ turn(row));
            at.b[i] = (uint32_t)row * A.k + (k0 + col < A.k ? col : 0);
        }
        return at;
    }

    // Both tiles of one step, straight to LDS.  Buffer loads: the compiler takes a global load to LDS for one that
    // touches both memories and waits for all of them at every LDS read.
    static __device__ __forceinline__ void stage(const GradArgs& A, const Places& at, int64_t t0, int k0, int n, u32x4* la, u32x4* lb)
    {
        const Rsrc ra = buffer_of(A.dy + t0 * A.ld_dy), rb = buffer_of(A.w + (int64_t)n * A.k + k0);
#pragma unroll
        for (int i = 0; i < kUnitsA; ++i) {
            const int first = i * kThreads + (threadIdx.x & ~63);
            if (kA % kThreads && first >= kA) break;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LdsMem*)(la + first), 16, at.a[i], 2 * n, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kUnitsB; ++i) {
            const int first = i * kThreads + (threadIdx.x & ~63);
            if (kB % kThreads && first >= kB) break;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LdsMem*)(lb + first), 16, at.b[i], 0, 0, 0);
        }
    }

    // The same where the reduction ends inside the tile: zeros past n1.
    static __device__ __forceinline__ void stage_tail(const GradArgs& A, int64_t t0, int k0, int n, int n1, u32x4* la, u32x4* lb)
    {
        for (int u = threadIdx.x; u < kA; u += kThreads) {
            const int row = u / CH, ch = (u % CH) ^ (row & 7);
            const int64_t t = min(t0 + row, A.tokens - 1);
            u32x4 v{0, 0, 0, 0};
            if (n + 8 * ch < n1) v = *reinterpret_cast<const u32x4*>(A.dy + t * A.ld_dy + n + 8 * ch);
            la[u] = v;
        }
        for (int u = threadIdx.x; u < kB; u += kThreads) {
            const int row = u / BU, col = k0 + 16 * ((u % BU) ^ turn(row));
            u32x4 v{0, 0, 0, 0};
            if (n + row < n1 && col < A.k) v = *reinterpret_cast<const u32x4*>(A.w + (int64_t)(n + row) * A.k + col);
            lb[u] = v;
        }
    }

    // Operands are read one group of products ahead of their use.
    static __device__ __forceinline__ void multiply(const u32x4* la, const u32x4* lb, int wm, int wn, f32x4 (*acc)[4])
    {
        constexpr int KK = BK / 32, PER = MF < 2 ? 1 : 2, GROUPS = KK * MF / PER;
        const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4, row0 = wm * (BM / WM) + c;
        const int src = 8 * g + (c >> 1);                     // the weight's row that this lane reads for its group
        u32x4 a[2][PER], b[4];
        i32x2 raw[4];
        const auto read_b = [&](int kk) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int row = kk * 32 + src;
                const char* p = reinterpret_cast<const char*>(lb + row * BU + ((wn * 4 + n) ^ turn(row))) + 8 * (c & 1);
                raw[n] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((LdsPair*)p);
            }
        };
        read_b(0);
#pragma unroll
        for (int p = 0; p < PER; ++p) a[0][p] = la[(row0 + p * 16) * CH + (g ^ (c & 7))];
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int m = i * PER % MF;
            if (m == 0) {
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    b[n] = u32x4{widen2<TYPE, false>(raw[n][0]), widen2<TYPE, true>(raw[n][0]),
                                 widen2<TYPE, false>(raw[n][1]), widen2<TYPE, true>(raw[n][1])};
            }
            if (i + 1 < GROUPS) {
                const int k2 = (i + 1) * PER / MF, m2 = (i + 1) * PER % MF;
                if (m2 == 0) read_b(k2);
#pragma unroll
                for (int p = 0; p < PER; ++p) a[(i + 1) & 1][p] = la[(row0 + (m2 + p) * 16) * CH + ((k2 * 4 + g) ^ (c & 7))];
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int p = 0; p < PER; ++p)
#pragma unroll
                for (int n = 0; n < 4; ++n) acc[m + p][n] = mfma<TYPE>(b[n], a[i & 1][p], acc[m + p][n]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The buffers are told apart by __restrict__: else every LDS read waits for the loads to LDS in flight.
    static __device__ __forceinline__ void stage_and_multiply(const GradArgs& A, const Places& at, int64_t t0, int k0, int n,
                                                              u32x4* __restrict__ to_a, u32x4* __restrict__ to_b,
                                                              const u32x4* __restrict__ la, const u32x4* __restrict__ lb,
                                                              int wm, int wn, f32x4 (*acc)[4])
    {
        stage(A, at, t0, k0, n, to_a, to_b);
        __builtin_amdgcn_sched_barrier(0);                    // loads leave before the products that hide them
        multiply(la, lb, wm, wn, acc);
    }
};

// All but the newest LOADS loads have arrived, and every LDS access is done, in
// every wave of the workgroup.
template <int LOADS>
__device__ __forceinline__ void wait_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LOADS) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int TYPE, int BM, int BN, int BK, int WM, int WN, int STAGES>
__global__ __launch_bounds__(kThreads) void input_grad_kernel(GradArgs A)
{
    typedef Tile<TYPE, BM, BN, BK, WM, WN, STAGES> S;
    extern __shared__ u32x4 lds[];
    u32x4* const la = lds;
    u32x4* const lb = lds + STAGES * S::kA;
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
    const int n0 = blockIdx.y * A.share, n1 = min(A.n, n0 + A.share), steps = n1 > n0 ? (n1 - n0) / BK : 0;
    f32x4 acc[S::MF][4] = {};
    // At the end of step s the tiles of step s + 1 have to be there, and only those
    // of the steps behind it may be under way: kAhead loads (a wave that sent one
    // more waits for it as well).  Steps past the last are replaced by the last, so
    // that this count holds in every step.
    const typename S::Places at = S::places(A, t0, k0);
    if (steps > 0) {
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) S::stage(A, at, t0, k0, n0 + min(s, steps - 1) * BK, la + s * S::kA, lb + s * S::kB);
        wait_and_meet<S::kAhead>();
    }
    int use = 0, fill = STAGES - 1;                           // the buffers of steps s and s + STAGES - 1
    for (int s = 0; s < steps; ++s) {
        S::stage_and_multiply(A, at, t0, k0, n0 + min(s + STAGES - 1, steps - 1) * BK, la + fill * S::kA, lb + fill * S::kB,
                              la + use * S::kA, lb + use * S::kB, wm, wn, acc);
        wait_and_meet<S::kAhead>();
        use = use == STAGES - 1 ? 0 : use + 1;
        fill = fill == STAGES - 1 ? 0 : fill + 1;
    }
    if (n0 + steps * BK < n1) {
        wait_and_meet<0>();
        S::stage_tail(A, t0, k0, n0 + steps * BK, n1, la, lb);
        wait_and_meet<0>();
        S::multiply(la, lb, wm, wn, acc);
    }
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const float scale = *A.w_scale;
#pragma unroll
    for (int m = 0; m < S::MF; ++m) {
        const int64_t t = t0 + wm * (BM / WM) + m * 16 + c;
        if (t >= A.tokens) continue;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int col = k0 + wn * 64 + n * 16 + 4 * g;    // K is a multiple of 16: an operand's columns are in or out
            if (col >= A.k) continue;
            const f32x4 v = acc[m][n];
            if (A.planes) *reinterpret_cast<f32x4*>(A.planes + ((int64_t)blockIdx.y * A.tokens + t) * A.k + col) = v;
            else
                *reinterpret_cast<uint2*>(A.dx + t * A.ld_dx + col) =
                    make_uint2(pack2<TYPE>(v[0] * scale, v[1] * scale), pack2<TYPE>(v[2] * scale, v[3] * scale));
        }
    }
    // Loads to LDS that no step used are still under way: they land before the workgroup ends.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Sums the shares in order, scales and rounds.
template <int TYPE>
__global__ __launch_bounds__(kJoinThreads) void grad_join_kernel(GradArgs A, int shares)
{
    const int64_t plane = A.tokens * A.k, i = ((int64_t)blockIdx.x * kJoinThreads + threadIdx.x) * 4;
    if (i >= plane) return;
    f32x4 s{0, 0, 0, 0};
    for (int p = 0; p < shares; p += 8) {                     // eight loads in flight, added in order
        f32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const f32x4*>(A.planes + min(p + j, shares - 1) * plane + i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (p + j < shares) s += v[j];
    }
    const float scale = *A.w_scale;
    const int64_t t = i / A.k;
    uint32_t* p = reinterpret_cast<uint32_t*>(A.dx + t * A.ld_dx + (i - t * A.k));
    p[0] = pack2<TYPE>(s[0] * scale, s[1] * scale);
    p[1] = pack2<TYPE>(s[2] * scale, s[3] * scale);
}

// The tile for a size, and the shares that the reduction is cut into where too
// few tiles are left to fill the card: whichever of them the step times below
// make shortest.
struct Shape {
    int bm, bn;
    uint32_t shares;
};

// Measured on MI355X (bfloat16): microseconds of one step (64 rows of the weight)
// of a workgroup alone on its compute unit, and of two side by side (the largest
// two tiles leave no LDS for a second one).  Larger tiles take less from LDS and
// memory for each product; smaller ones fill 256 compute units from fewer tokens.
// 2048 x 4096 x 4096: 67 us in tiles of 128 x 256, 73 in 128 x 128, 100 in 256 x
// 256, which win at 4096 tokens with 109 against 122.  Joining shares costs a
// launch and their traffic: 1001 x 4096 x 4096 takes 40 us unsplit in 128 x 128,
// 44 in 128 x 256 with two shares.  24 x 14336 x 4096: 16.5 us with 16 shares, 17.7
// with 8, 19.5 with 28.  (Whole calls, one after the other.)
struct Cost {
    int bm, bn;
    double one, two;
};
constexpr Cost kCosts[] = {{256, 256, 1.65, 0.0}, {128, 256, 1.0, 0.0}, {128, 128, 0.7, 1.1}, {64, 256, 0.7, 1.1}, {32, 256, 0.8, 1.6}};

Shape shape_of(uint64_t tokens, uint64_t n, uint64_t k)
{
    Shape best{32, 256, 1};
    double least = -1.0;
    for (const Cost& c : kCosts) {
        if (c.bm > 32 && (uint64_t)c.bm / 2 >= tokens) continue;      // over half of the rows would be padding
        const uint64_t tiles = ((tokens + c.bm - 1) / c.bm) * ((k + c.bn - 1) / c.bn);
        for (uint32_t s = 1; s <= 16 && (s == 1 || n / s >= 256); ++s) {
            const uint64_t groups = tiles * s, slots = c.two > 0.0 ? 512 : 256, whole = groups / slots, rest = groups % slots;
            const double full = c.two > 0.0 ? c.two : c.one;
            const double turns = whole * full + (rest == 0 ? 0.0 : rest <= 256 ? c.one : full);
            const double us = turns * ((n + s - 1) / s + 63) / 64 + (s > 1 ? 4.0 + 8.0 * s * tokens * k / 5e6 : 0.0);
            if (least < 0.0 || us < least) {
                least = us;
                best = Shape{c.bm, c.bn, s};
            }
        }
    }
    return best;
}

bool sizes_ok(uint64_t tokens, uint64_t n, uint64_t k)
{
    return tokens <= ECF8A_MAX_TOKENS && n >= 16 && n <= ECF8A_MAX_FEATURES && n % 16 == 0 && k >= 16 &&
           k <= ECF8A_MAX_FEATURES && k % 16 == 0;
}

template <int TYPE, int BM, int BN, int BK, int WM, int WN, int STAGES>
int launch(GradArgs A, uint32_t shares, hipStream_t st)
{
    typedef Tile<TYPE, BM, BN, BK, WM, WN, STAGES> S;
    constexpr int bytes = S::kLds;
    auto* kernel = input_grad_kernel<TYPE, BM, BN, BK, WM, WN, STAGES>;
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
    if (s.bm == 256) rc = launch<TYPE, 256, 256, 64, 2, 4, 3>(A, s.shares, st);
    else if (s.bm == 128 && s.bn == 256) rc = launch<TYPE, 128, 256, 64, 2, 4, 3>(A, s.shares, st);
    else if (s.bm == 128) rc = launch<TYPE, 128, 128, 64, 4, 2, 3>(A, s.shares, st);
    else if (s.bm == 64) rc = launch<TYPE, 64, 256, 64, 2, 4, 3>(A, s.shares, st);
    else rc = launch<TYPE, 32, 256, 64, 2, 4, 3>(A, s.shares, st);
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
    if (ld_dy < out_features || ld_dx < in_features || ld_dy > (1u << 22)) return ECF8_ERR_SIZE;  // a tile's rows: 32-bit offsets
    const uint64_t need = ecf8a_input_grad_bytes(tokens, out_features, in_features);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return ECF8_ERR_WORKSPACE;
    const Shape s = shape_of(tokens, out_features, in_features);
    const GradArgs A{static_cast<const uint16_t*>(dy), (int64_t)ld_dy, w, w_scale, static_cast<uint16_t*>(dx), (int64_t)ld_dx,
                     s.shares > 1 ? static_cast<float*>(workspace) : nullptr, (int64_t)tokens, (int)out_features,
                     (int)in_features, (int)round_up((out_features + s.shares - 1) / s.shares, 64), 0, 0};
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    return type == ECF8A_BF16 ? run<kBf16>(A, s, st) : run<kFp16>(A, s, st);
}
