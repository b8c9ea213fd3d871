// ecf8x_grad.hip -- the gradient that a frozen 4-bit weight passes to its input:
// dx = dy w, dy (T x N) in a 16-bit type, w (N x K) in microscaled 4 bits.
//
// The reduction runs down the weight's columns, and a block's power of two
// changes from row to row, so that an operand of eight rows has eight scales.
// Each 16 bytes of codes (a block, under one scale) are therefore widened once
// per workgroup, on their way to LDS, and the operands are turned there by the
// transposing LDS read.  Widened values are exact bfloat16; float16 dy is split
// into two bfloat16 (exact).  Sums in float32, rounded once.
//
// Magnitudes of 2^128 and more, which quantisation never stores, widen to
// infinity.  A lower half of 0, or of the other sign, would make a NaN of that
// one, so that beside float16 dy weights are widened with an eighth of their
// scale, and the sums taken eight times.  (Scales of 2^-125 and less, which have no
// eighth, count as 2^-124 there: what they add to a sum, under 2^-80, is far below
// float16's smallest step.)
#include "ecf8x_stream.h"
#include "ecf8x_tiles.h"

namespace {

using namespace ecf8x;

constexpr int kThreads = 512, kStep = 64;

struct Args {
    const uint16_t* dy;
    int64_t ld_dy;
    const uint8_t *w, *w_scales;
    uint16_t* dx;
    int64_t ld_dx;
    float* sums;                // [share][tile that was left][BM][BN]
    int64_t tokens;
    int n, k, kp;
    Tiling tiling;              // shares of a multiple of 64
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 LdsQuad;

// One workgroup: BM tokens by BN columns of dx, eight waves in WM rows of WN, 64
// rows of the weight at a time.  The weight's codes are loaded to registers AHEAD
// steps early, widened and stored one step early, into two buffers.  bfloat16 dy
// goes straight to LDS, STAGES - 1 steps early; float16 dy is loaded like the codes,
// split into two bfloat16 and stored one step early, so that each value is split
// once per workgroup.
//
// What bounds it: the matrix instructions, 1.5 us a step of 256 x 256 at the rate of a large library product, and beside them
// 256 KB that go to and from LDS (4096 x 13824 x 5120: 445 us, 1300 TFLOP/s; float16, in tiles of 128 x 256 with twice the
// products and two planes of dy, 880).  With few tokens, the begin and end of short shares (77 x 14336 x 4096 in float16:
// 33 us, 14 steps of 1.4 us in tiles of 96 x 256).
//
// Banks.  Unit u (16 bytes) of dy's row r sits at u ^ (r & 7).  Unit u of the
// widened row r sits at u ^ turn(r): the transposing read takes two units of
// four rows in each lane group, and the 16 units that half a wave touches lie in
// different banks; so do those that 16 lanes store, since lanes of the second
// half of a row store their units in another order.
template <int TYPE, int BM, int BN, int WM, int WN, int STAGES, int AHEAD>
struct Tile {
    static constexpr bool SPLIT = TYPE == kFp16;
    static constexpr int MF = BM / WM / 16, NF = BN / WN / 16;
    static constexpr int BU = BN / 8;                          // 16-byte units of a widened row
    static constexpr int kA = BM * 8, kB = kStep * BU;         // of a plane of dy's tile, of the widened tile
    static constexpr int kWaveA = kA / 8, kUnitsA = (kWaveA + 63) / 64;    // a wave sends for the same number as any other, the last with part of its lanes
    static constexpr int kRaw = kStep * BN / 32;               // 16-byte units of codes
    static constexpr int kBuffers = SPLIT ? 4 : STAGES;        // split: two planes, two steps
    static constexpr int kLds = 16 * (kBuffers * kA + 2 * kB);
    // Loads that may be under way at the end of a step: those of all steps behind the next one's dy, codes included.
    static constexpr int kAhead = (STAGES - 2) * (kUnitsA + 2);
    static_assert(STAGES >= 2 && kLds <= 160 * 1024 && kAhead < 64, "LDS and the load counter");
    static_assert(WM * WN == kThreads / 64 && MF >= 1 && NF >= 1 && kRaw <= kThreads && kRaw % 64 == 0, "eight waves");
    static_assert(kUnitsA <= 4 && kWaveA % 16 == 0, "quarters");

    static __device__ __forceinline__ int turn(int row) { return 2 * ((row & 3) | (row >> 1 & 4)) | (row >> 2 & 1); }

    // Unit i that this lane sends for; lanes past its share of a wave repeat others'.
    static __device__ __forceinline__ int lanes_of(int i) { return kWaveA - 64 * i < 64 ? kWaveA - 64 * i : 64; }

    static __device__ __forceinline__ int unit_a(int i) { return wave_id() * kWaveA + i * 64 + (int)(threadIdx.x & 63) % lanes_of(i); }

    struct Places {
        uint32_t a[kUnitsA];
        uint32_t codes, scale;                                 // of this thread's block in the first row of the tile's first step
        int row;                                               // of a step, that this thread widens
    };

    static __device__ __forceinline__ Places places(const Args& A, int64_t t0, int k0)
    {
        Places at;
#pragma unroll
        for (int i = 0; i < kUnitsA; ++i) {
            const int u = unit_a(i), row = u >> 3;
            at.a[i] = 2 * ((uint32_t)min((int64_t)row, A.tokens - 1 - t0) * (uint32_t)A.ld_dy + 8 * ((u & 7) ^ (row & 7)));
        }
        const int u = threadIdx.x % kRaw, col = k0 + 32 * (u % (BN / 32));
        at.row = u / (BN / 32);
        at.codes = (col < A.kp ? col : 0) / 2;                 // past the last column: results that are not stored
        at.scale = at.codes / 16;
        return at;
    }

    // Unit i of the kUnitsA that a wave sends for.
    static __device__ __forceinline__ void stage_unit(const Args& A, const Places& at, int64_t t0, int n, int i, u32x4* la)
    {
        const int wave = wave_id();
        if (lanes_of(i) == 64 || (int)(threadIdx.x & 63) < lanes_of(i))
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(A.dy + t0 * A.ld_dy), (LdsMem*)(la + wave * kWaveA + i * 64), 16, at.a[i], 2 * n, 0, 0);
    }

    static __device__ __forceinline__ void stage(const Args& A, const Places& at, int64_t t0, int n, u32x4* la)
    {
#pragma unroll
        for (int i = 0; i < kUnitsA; ++i) stage_unit(A, at, t0, n, i, la);
    }

    // What a thread loads early: a block of codes with its scale, and float16 dy.
    struct Early {
        u32x4 codes;
        uint32_t scale;
        u32x4 dy[SPLIT ? kUnitsA : 1];
    };

    // Every lane loads, so that every wave has as many loads under way: rows past n1 read the last one, dy's steps past
    // its last whole one that one (`whole`; none: no dy).
    static __device__ __forceinline__ void fetch(const Args& A, const Places& at, int64_t t0, int n, int n1, int whole, Early& e)
    {
        const int64_t row = max(0, min(n + at.row, n1 - 1));
        e.codes = *reinterpret_cast<const u32x4*>(A.w + row * (A.kp / 2) + at.codes);
        e.scale = A.w_scales[row * (A.kp / 32) + at.scale];
        if constexpr (SPLIT) {
            if (whole >= 0) {
                const char* p = reinterpret_cast<const char*>(A.dy + t0 * A.ld_dy + min(n, whole));
#pragma unroll
                for (int i = 0; i < kUnitsA; ++i) e.dy[i] = *reinterpret_cast<const u32x4*>(p + at.a[i]);
            }
        }
    }

    // The scale byte that a block is widened with; `in`: 0 for rows past the last, which are zero.
    static __device__ __forceinline__ uint32_t scale_byte(uint32_t scale, uint32_t in)
    {
        if constexpr (SPLIT) scale = scale == 255 ? 255 : max(scale, 3u) - 3;
        return scale & in;
    }

    static __device__ __forceinline__ void put_split(u32x4 v, int u, u32x4* la)
    {
        u32x4 hi, lo;
        split8_f16(v, hi, lo);
        la[u] = hi;
        la[kA + u] = lo;
    }

    // Stores a quarter of what was loaded for the step whose first row is n; rows past n1 are zero.
    static __device__ __forceinline__ void store(int i, const Places& at, int n, int n1, const Early& e, u32x4* la, u32x4* lb)
    {
        if (kRaw == kThreads || threadIdx.x < kRaw) {
            const int j = threadIdx.x % (BN / 32), swap = j >> 2 & 1;
            // Masks: no branch between the products, no register chosen by a number that only the lane knows.
            const uint32_t in = n + at.row < n1 ? ~0u : 0, other = -(uint32_t)swap;
            lb[at.row * BU + ((4 * j + (i ^ swap)) ^ turn(at.row))] = widen4(((e.codes[i ^ 1] & other) | (e.codes[i] & ~other)) & in, scale_of(scale_byte(e.scale, in)));
        }
        if constexpr (SPLIT) {
#pragma unroll
            for (int d = 0; d < kUnitsA; ++d)
                if (d % 4 == i && (lanes_of(d) == 64 || (int)(threadIdx.x & 63) < lanes_of(d))) put_split(e.dy[d], unit_a(d), la);
        }
    }

    // dy's tile where the reduction ends inside the step: zeros past n1.
    static __device__ __forceinline__ void stage_tail(const Args& A, int64_t t0, int n, int n1, u32x4* la)
    {
        for (int u = threadIdx.x; u < kA; u += kThreads) {
            const int row = u >> 3, first = n + 8 * ((u & 7) ^ (row & 7));
            const uint16_t* p = A.dy + min(t0 + row, A.tokens - 1) * A.ld_dy + first;
            u32x4 v{0, 0, 0, 0};
            if (first + 8 <= n1) v = *reinterpret_cast<const u32x4*>(p);
            else
                for (int i = 0; first + i < n1; ++i) v[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
            if constexpr (SPLIT) put_split(v, u, la);
            else la[u] = v;
        }
    }

    // The products of a step, token fragments PER at a time: the operands of a group are read while the group before is
    // multiplied.  between(i): what else there is to do, a quarter before each of the first groups; its VALU and LDS work
    // then goes beside the other wave's products.  (All of it ahead of them: 2.0 us a step of 256 x 256; so: 1.6.)
    template <class Between>
    static __device__ __forceinline__ void multiply(const u32x4* la, const u32x4* lb, int wm, int wn, f32x4 (*acc)[NF], Between between)
    {
        constexpr int PER = MF % 2 ? 1 : 2, GROUPS = 2 * MF / PER;
        const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4, row0 = wm * (BM / WM) + c;
        u32x4 a[2][PER], low[2][SPLIT ? PER : 1], b[2][NF];
        const auto read_b = [&](int kk) {
#pragma unroll
            for (int n = 0; n < NF; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = 32 * kk + 8 * g + 4 * h + (c >> 2), u = (wn * (BN / WN) + 16 * n) / 8 + (c >> 1 & 1);
                    const char* p = reinterpret_cast<const char*>(lb + row * BU + (u ^ turn(row))) + 8 * (c & 1);
                    const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsQuad*)p));
                    b[kk][n][2 * h] = v.x, b[kk][n][2 * h + 1] = v.y;
                }
        };
        const auto read_a = [&](int i) {
#pragma unroll
            for (int p = 0; p < PER; ++p) {
                const int kk = i * PER / MF, m = i * PER % MF + p, u = (row0 + 16 * m) * 8 + ((4 * kk + g) ^ (c & 7));
                a[i & 1][p] = la[u];
                if constexpr (SPLIT) low[i & 1][p] = la[kA + u];
            }
        };
        read_b(0);
        read_a(0);
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
            const int kk = i * PER / MF, m = i * PER % MF;
            if (i + 1 < GROUPS) {
                if ((i + 1) * PER % MF == 0) read_b(kk + 1);
                read_a(i + 1);
            }
            if (GROUPS >= 4 ? i < 4 : true) {
#pragma unroll
                for (int q = 0; q < (GROUPS >= 4 ? 1 : 4 / GROUPS); ++q) between(i * (GROUPS >= 4 ? 1 : 4 / GROUPS) + q);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int p = 0; p < PER; ++p) {
#pragma unroll
                for (int n = 0; n < NF; ++n) acc[m + p][n] = mfma_bf16(b[kk][n], a[i & 1][p], acc[m + p][n]);
                if constexpr (SPLIT) {
#pragma unroll
                    for (int n = 0; n < NF; ++n) acc[m + p][n] = mfma_bf16(b[kk][n], low[i & 1][p], acc[m + p][n]);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // The buffers are told apart by __restrict__: else every LDS read waits for the loads to LDS in flight.
    static __device__ __forceinline__ void step(const Args& A, const Places& at, int64_t t0, int n, int later, int n1, int whole, const Early& next,
                                                Early& early, u32x4* __restrict__ to_a, u32x4* __restrict__ to_b, const u32x4* __restrict__ la,
                                                const u32x4* __restrict__ lb, int wm, int wn, bool real, f32x4 (*acc)[NF])
    {
        fetch(A, at, t0, n + AHEAD * kStep, n1, whole, early);
        __builtin_amdgcn_sched_barrier(0);                    // loads leave before the products that hide them
        if (real)
            multiply(la, lb, wm, wn, acc, [&](int i) {
                if (!SPLIT && i < kUnitsA) stage_unit(A, at, t0, later, i, to_a);
                store(i, at, n + kStep, n1, next, to_a, to_b);
            });
    }
};

template <int TYPE, int BM, int BN, int WM, int WN, int STAGES, int AHEAD>
__global__ __launch_bounds__(kThreads) void grad_kernel(Args A)
{
    typedef Tile<TYPE, BM, BN, WM, WN, STAGES, AHEAD> S;
    extern __shared__ u32x4 lds[];
    u32x4* const la = lds;
    u32x4* const lb = lds + S::kBuffers * S::kA;
    const int wave = wave_id(), wm = wave / WN, wn = wave % WN;
    const Part part = part_of(A.tiling, blockIdx.x);
    const int64_t t0 = (int64_t)part.tm * BM;
    const int k0 = part.tn * BN;
    const int n0 = part.share * A.tiling.length, n1 = part.at < 0 ? A.n : min(A.n, n0 + A.tiling.length), steps = n1 > n0 ? (n1 - n0) / kStep : 0;
    const int whole = steps > 0 ? n0 + (steps - 1) * kStep : -1;     // dy's last whole step
    f32x4 acc[S::MF][S::NF] = {};
    const typename S::Places at = S::places(A, t0, k0);
    typename S::Early early[AHEAD];                           // of step s at s % AHEAD
#pragma unroll
    for (int s = 0; s < AHEAD; ++s) S::fetch(A, at, t0, n0 + s * kStep, n1, whole, early[s]);
    if constexpr (!S::SPLIT) {
        if (steps > 0) {
#pragma unroll
            for (int s = 0; s < STAGES - 1; ++s) S::stage(A, at, t0, n0 + min(s, steps - 1) * kStep, la + s * S::kA);
        }
    }
    // Where no float16 dy was loaded: into the other buffer, which nothing reads.
#pragma unroll
    for (int i = 0; i < 4; ++i) S::store(i, at, n0, n1, early[0], S::SPLIT && steps == 0 ? la + 2 * S::kA : la, lb);
    wait_and_meet<0>();
    // In step s the codes (and float16 dy) of step s + 1 are stored, those of step s + AHEAD sent for, and bfloat16 dy's
    // tile of step s + STAGES - 1 (the last one again past the end).
    int use = 0, fill = S::SPLIT ? 1 : STAGES - 1;
    constexpr int kPlanes = S::SPLIT ? 2 : 1, kTurn = S::SPLIT ? 2 : STAGES;
    // Whole turns of AHEAD steps: a turn that is left inside makes the compiler copy what is being loaded, and wait for it.
    for (int s0 = 0; s0 < steps; s0 += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int s = s0 + i;
            S::step(A, at, t0, n0 + s * kStep, n0 + min(s + STAGES - 1, steps - 1) * kStep, n1, whole, early[(i + 1) % AHEAD], early[i],
                    la + fill * kPlanes * S::kA, lb + (s + 1 & 1) * S::kB, la + use * kPlanes * S::kA, lb + (s & 1) * S::kB, wm, wn, s < steps, acc);
            if constexpr (S::SPLIT) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
            } else {
                wait_and_meet<S::kAhead>();
            }
            use = use == kTurn - 1 ? 0 : use + 1;
            fill = fill == kTurn - 1 ? 0 : fill + 1;
        }
    }
    if (n0 + steps * kStep < n1) {
        wait_and_meet<0>();
        S::fetch(A, at, t0, n0 + steps * kStep, n1, -1, early[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) S::store(i, at, n0 + steps * kStep, n1, early[0], la + (S::SPLIT ? 2 * S::kA : 0), lb);
        S::stage_tail(A, t0, n0 + steps * kStep, n1, la);     // (float16 dy: stale values went to the other buffer)
        wait_and_meet<0>();
        S::multiply(la, lb, wm, wn, acc, [](int) {});
    }
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < S::MF; ++m) {
        const int64_t t = t0 + wm * (BM / WM) + m * 16 + c;
        if (t >= A.tokens) continue;
#pragma unroll
        for (int n = 0; n < S::NF; ++n) {
            const int col = k0 + wn * (BN / WN) + n * 16 + 4 * g;   // K is a multiple of 32: an operand's columns are in or out
            if (col >= A.k) continue;
            if constexpr (S::SPLIT) acc[m][n] *= 8.0f;
            if (part.at >= 0) *reinterpret_cast<f32x4*>(A.sums + ((int64_t)part.at * BM + (t - t0)) * BN + (col - k0)) = acc[m][n];
            else store4<TYPE>(A.dx + t * A.ld_dx + col, acc[m][n], 4);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");          // loads to LDS that no step used land before the workgroup ends
}

// Measured on MI355X: microseconds of a step (64 rows of the weight) of a workgroup alone on its compute unit, and of two
// side by side (0: no LDS for a second one).  Shares cost their sums' traffic and the launch that joins them: 77 x 14336 x
// 4096 in bfloat16 takes 24 + 5 us with 16 shares; 4096 x 13824 x 5120 530 us with all tiles in three shares, 455 with the 64
// that are left of 320 in four (now 445).  96 rows: 77 tokens 28 us in tiles of 128, 26 so,
// 192 tokens 42 and 38.  float16 has twice the products, and no tiles of 256
// tokens, whose two planes leave no room for a second buffer.
constexpr Cost kCosts[] = {{256, 256, 1.55, 0.0}, {128, 256, 0.95, 0.0}, {128, 128, 0.68, 1.36}, {96, 256, 0.85, 0.0}, {64, 256, 0.72, 0.0}, {32, 256, 0.61, 0.0}};
constexpr Cost kCostsSplit[] = {{128, 256, 1.67, 0.0}, {128, 128, 1.19, 2.36}, {96, 256, 1.41, 0.0}, {64, 256, 1.04, 0.0}, {32, 256, 0.81, 0.0}};

Tiling tiles_of(uint64_t tokens, uint64_t n, uint64_t k, bool split)
{
    return split ? tiling_of(kCostsSplit, 5, tokens, k, n, kStep, kStep, 256, 32) : tiling_of(kCosts, 6, tokens, k, n, kStep, kStep, 256, 32);
}

bool sizes_ok(uint64_t tokens, uint64_t n, uint64_t k)
{
    return tokens <= ECF8A_MAX_TOKENS && n >= 1 && n <= ECF8A_MAX_FEATURES && k >= ECF8X_BLOCK && k <= ECF8A_MAX_FEATURES &&
           k % ECF8X_BLOCK == 0;
}

template <int TYPE, int BM, int BN, int WM, int WN, int STAGES, int AHEAD>
int launch(const Args& A, hipStream_t st)
{
    constexpr int bytes = Tile<TYPE, BM, BN, WM, WN, STAGES, AHEAD>::kLds;
    auto* kernel = grad_kernel<TYPE, BM, BN, WM, WN, STAGES, AHEAD>;
    if (bytes > 65536 &&
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
        return ECF8_ERR_HIP;
    kernel<<<groups_of(A.tiling), kThreads, bytes, st>>>(A);
    return launch_status();
}

// The tiles that tiles_of chose: of 256 tokens for bfloat16 alone (kCostsSplit has none).
template <int TYPE>
int run_tiles(const Args& A, hipStream_t st)
{
    const int bm = A.tiling.bm, bn = A.tiling.bn;
    if constexpr (TYPE == kBf16) {
        if (bm == 256) return launch<TYPE, 256, 256, 2, 4, 3, 2>(A, st);
    }
    if (bm == 128 && bn == 256) return launch<TYPE, 128, 256, 2, 4, 5, 4>(A, st);
    if (bm == 128) return launch<TYPE, 128, 128, 4, 2, 3, 4>(A, st);
    if (bm == 96) return launch<TYPE, 96, 256, 2, 4, 5, 4>(A, st);
    if (bm == 64) return launch<TYPE, 64, 256, 2, 4, 6, 4>(A, st);
    return launch<TYPE, 32, 256, 2, 4, 6, 4>(A, st);
}

template <int TYPE>
int run(const Args& A, hipStream_t st)
{
    const Tiling& s = A.tiling;
    const int rc = run_tiles<TYPE>(A, st);
    if (rc != ECF8_OK || s.rest == 0) return rc;
    return join_tiles<TYPE>(A.sums, s, A.tokens, A.k, nullptr, A.dx, A.ld_dx, st);
}

}  // namespace

extern "C" uint64_t ecf8x_input_grad_bytes(uint64_t tokens, uint64_t out_features, uint64_t in_features, uint32_t type)
{
    if (!sizes_ok(tokens, out_features, in_features)) return 0;
    if (tokens == 0) return 0;
    return sums_of(tiles_of(tokens, out_features, in_features, type == ECF8A_FP16));
}

extern "C" int ecf8x_input_grad(const void* dy, uint64_t ld_dy, uint32_t type, uint64_t tokens, uint64_t out_features, uint64_t in_features,
                                const ecf8x_matrix* w, void* dx, uint64_t ld_dx, void* workspace, uint64_t workspace_bytes,
                                void* hip_stream)
{
    if (type != ECF8A_BF16 && type != ECF8A_FP16) return ECF8_ERR_UNSUPPORTED;
    if (!sizes_ok(tokens, out_features, in_features)) return ECF8_ERR_SIZE;
    if (tokens == 0) return ECF8_OK;
    if (tokens == 1) ld_dy = out_features, ld_dx = in_features;
    if (!dy || !w || !w->codes || !w->scales || !dx || !aligned(dy, 16) || !aligned(w->codes, 16) || !aligned(w->scales, 4) ||
        !aligned(dx, 16) || (tokens > 1 && (ld_dy % 8 || ld_dx % 8)))
        return ECF8_ERR_ARG;
    if (ld_dy < out_features || ld_dx < in_features || ld_dy > (1u << 22) || ld_dx > (1ull << 40)) return ECF8_ERR_SIZE;
    const uint64_t need = ecf8x_input_grad_bytes(tokens, out_features, in_features, type);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return ECF8_ERR_WORKSPACE;
    const Args A{static_cast<const uint16_t*>(dy), (int64_t)ld_dy, w->codes, w->scales, static_cast<uint16_t*>(dx), (int64_t)ld_dx,
                 static_cast<float*>(workspace), (int64_t)tokens, (int)out_features, (int)in_features, (int)padded(in_features),
                 tiles_of(tokens, out_features, in_features, type == ECF8A_FP16)};
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    return type == ECF8A_BF16 ? run<kBf16>(A, st) : run<kFp16>(A, st);
}
