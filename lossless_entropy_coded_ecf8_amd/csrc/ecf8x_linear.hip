// ecf8x_linear.hip -- y = x w^T + bias with w (N x K) in microscaled 4 bits and
// x in a 16-bit type or in the same 4 bits.
//
// Sixteen-bit x: each code times its power of two is exact in bfloat16, so the
// weight is widened in registers and the 16-bit matrix instruction gives exact
// products, summed in float32.  A block's power of two need not fit float16, so
// with float16 x an instruction takes one block of 32 unscaled, and its float32
// result is scaled as it is added.  Four-bit x: the scaled matrix instruction takes
// codes and scale bytes as they are stored.
#include "ecf8x_offsets.h"
#include "ecf8x_stream.h"
#include "ecf8x_tiles.h"

namespace {

using namespace ecf8x;

constexpr int kThreads = 512, kWaves = 8;      // of tile_kernel

struct Args {
    const void* x;              // 16-bit rows, ld_x elements apart, or codes
    const uint8_t* x_scales;
    int64_t ld_x;
    const uint8_t *w, *w_scales;
    const uint16_t* bias;
    uint16_t* y;
    int64_t ld_y;
    float* sums;                // few tokens: [share][token][pitch], nullptr where there is one share; else [share][tile that was left][BM][BN]
    int64_t tokens;
    int n, k, kp;               // kp: k rounded up to 128
    int pitch, share;           // few tokens: n rounded up to 4; length of one of gridDim.y shares, a multiple of 1024
    Tiling tiling;              // more: shares of a multiple of 256
};

template <int OUT>
__device__ __forceinline__ void finish(const Args& A, int64_t t, int n, f32x4 v)
{
    if (A.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < A.n) v[i] += load1<OUT>(A.bias + n + i);
    }
    store4<OUT>(A.y + t * A.ld_y + n, v, A.n - n);
}

// ------------------------------------------------------------ few tokens

// A share of the reduction is a multiple of 1024 values, so that it begins with a step.
//
// Up to about 16 tokens the stream of weights bounds it (28672 x 8192, 125 MB: one bfloat16 token 26 us, 4.8 TB/s; 16 of 4
// bits 27), past them what each workgroup stages of the tokens beside its weights, 25 to 30 bytes a nanosecond and compute
// unit together (45 float16 tokens 46 us, 40 of 4 bits 34).  Few rows (4096 x 4096: 6.6 us) are a chain of four steps.
template <int XT, int OUT, int MF, int RG, int TR>
__global__ __launch_bounds__(kThreads) void few_kernel(Args A)
{
    typedef Stream<kMx4, XT, MF, RG, TR> S;
    extern __shared__ __attribute__((aligned(16))) char few_lds[];
    const int lane = threadIdx.x & 63, wave = wave_id(), c = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * S::R, row_bytes = A.kp / 2, row_scales = A.kp / 32;
    const int first = min(n0 + 16 * S::fragment(wave), A.n - 1);       // rows past the last reach no result that is stored
    const int cols = XT == kMx4 ? A.kp : A.k, k0 = blockIdx.y * A.share, count = max(0, min(cols - k0, A.share));
    const typename S::Rows rows{A.w + (int64_t)first * row_bytes + k0 / 2, A.w_scales + (int64_t)first * row_scales + k0 / 32, A.n - 1 - first};
    const char* x = static_cast<const char*>(A.x) + (XT == kMx4 ? k0 / 2 : 2 * k0);
    const uint8_t* x_scales = A.x_scales + (XT == kMx4 ? k0 / 32 : 0);
    const typename S::Places at = S::places(rows, row_bytes, row_scales, x, x_scales, 0, [&](int i) {
        const uint32_t t = (uint32_t)min((int64_t)i, A.tokens - 1);
        return XT == kMx4 ? t : 2 * t * (uint32_t)A.ld_x;
    });
    f32x4 acc[S::RF][MF] = {};
    S::run(rows, at, x, x_scales, count, few_lds, acc);
    if (wave >= RG) return;
#pragma unroll
    for (int f = 0; f < S::RF; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int n = n0 + 16 * (wave * S::RF + f) + 4 * g, t = 16 * m + c;
            if (t >= A.tokens || n >= A.n) continue;
            if (A.sums) *reinterpret_cast<f32x4*>(A.sums + ((int64_t)blockIdx.y * A.tokens + t) * A.pitch + n) = acc[f][m];
            else finish<OUT>(A, t, n, acc[f][m]);
        }
}

// ------------------------------------------------------------ many tokens

// One workgroup: BM tokens by BN outputs, eight waves in WM rows of WN, the
// reduction in steps: 64 values of 16 bits (128 bytes of an x row, 32 of a weight
// row), or of 4 bits 128 (64 bytes of each) or 256.  Runs of 64 bytes come to LDS at
// 61 bytes a nanosecond and compute unit, of 128 at 100: the larger tiles take 256
// (4096 x 28672 x 8192: 560 us in steps of 128 through four buffers, 530 so).
//
// Tiles go from memory to LDS without passing registers into STAGES buffers:
// while step s is multiplied, step s + STAGES - 1 is sent for, between the products
// (all ahead of them: bfloat16 1440 us for 1370).  With bfloat16 x lane group g takes
// units 2g and 2g + 1 of an x row and the same values of a weight row, so that it meets
// 8 contiguous bytes of codes, under one scale; with 4-bit x unit g of either; float16,
// which takes one block at a time, unit g of its four.
//
// Banks: place p of row r sits at p ^ turn(r); weight rows of 32 bytes lie as they
// are.
//
// What bounds it, in tiles of 256 x 256 (4096 x 28672 x 8192): bfloat16 1370 us, 1400 TFLOP/s, the matrix instructions,
// 66% busy at the 1.8 GHz that the power limit leaves; 4 bits 530 us, 3630 TFLOP/s, 43% busy at 1.9, beside as many
// cycles of LDS.  In float16 the scaling of each block's sums, four multiply-adds for each product instruction (4096 x
// 13824 x 5120: 628 us, bfloat16 450).  Where there are few tiles, the units that have none (331 x 13821 x 5120 of 4 bits:
// 37 us, 162 tiles of 128 x 256).
//
// Scales: a dword of every row comes with the step (16-bit x: the four blocks that two
// steps share).  It asks the cache for as many lines as the codes do, so for the large
// tiles of 4-bit x they come in groups of 512 values instead, 16 bytes of a row, two
// groups ahead: each step sends for some rows' next but one group (4096 x 28672 x 8192
// gained 7%; 512 x 4096 x 4096, in tiles of 128 x 128: 18 -> 21, so not there; 16-bit
// x gained nothing).
template <int XT, int BM, int BN, int WM, int WN, int STAGES, int LENGTH>
struct Tile {
    static constexpr bool MX = XT == kMx4;
    static constexpr int MF = BM / WM / 16, NF = BN / WN / 16, STEP = LENGTH;
    static constexpr int AU = MX ? STEP / 32 : 8, BU = MX ? AU : 2;     // 16-byte units of a row's step: x, weight
    static constexpr int kA = BM * AU, kB = BN * BU;            // 16-byte units of the two tiles
    static constexpr bool GROUPED = MX && BN == 256;
    static constexpr int GROUP = 512 / STEP;                   // steps of a group of scales
    static constexpr int kRowsX = MX ? BM : 0, kRows = kRowsX + BN;    // rows of scales: tokens', then outputs'
    static constexpr int kWaveA = kA / 8, kWaveB = kB / 8, kUnitsA = (kWaveA + 63) / 64, kUnitsB = kWaveB < 64 ? 1 : kB / kThreads;
    static constexpr int kStage = 16 * (kA + kB) + (GROUPED ? 0 : 4 * kRows);                    // bytes
    static constexpr int kLds = STAGES * kStage + (GROUPED ? 3 * 16 * kRows : 0);
    // Loads that may be under way at the end of a step, the same in every wave, some with part of its lanes: those of all
    // steps behind the next one; of groups of scales those sent for since its tiles, at least one step's.
    static constexpr int kTiles = kUnitsA + kUnitsB, kScales = 1 + MX;
    static constexpr int kAhead = GROUPED ? (STAGES - 2) * kTiles + (STAGES > 2) * kScales : (STAGES - 2) * (kTiles + kScales);
    static_assert(STAGES >= 2 && (!GROUPED || STAGES <= GROUP + 2) && kLds <= 160 * 1024 && kAhead < 64 && kStage % 16 == 0, "LDS and the load counter");
    static_assert(kWaveA % 16 == 0 && (kWaveB < 64 || kWaveB % 64 == 0), "waves stage alike");
    static_assert(GROUPED ? BN % (8 * GROUP) == 0 && kRowsX % (8 * GROUP) == 0 : BN <= 512 && kRowsX <= 512, "so for the scales");
    static_assert(WM * WN == kWaves && (MX ? MF % 2 == 0 : MF >= 1) && NF >= 1, "eight waves");

    // The unit of a row that lies at place p of its eight (before the turn by the row): places are numbered so that
    // lane group g reads g and 4 + g, which the lanes of one cycle spread over all banks.
    static __device__ __forceinline__ int unit_at(int p) { return XT != kBf16 ? p : (p & 3) << 1 | p >> 2; }

    static __device__ __forceinline__ int turn(int row) { return AU == 4 ? 0x78 >> (row >> 1 & 6) & 3 : row & 7; }

    // Parts in which the rows' scales are sent for, and the rows of a wave and part.
    static constexpr int PARTS = GROUPED ? GROUP : 1, kPartX = kRowsX / (8 * PARTS), kPartW = BN / (8 * PARTS);

    // Byte offsets from the tile's corner of what a lane sends for.  Rows past the last read the last one's; they reach
    // no result that is stored.
    struct Places {
        uint32_t a[kUnitsA], b[kUnitsB], sx[PARTS], sw[PARTS];
        Rsrc x_scales, w_scales;
    };

    // Lanes of a wave that send for its unit i of x.
    static __device__ __forceinline__ int lanes_of(int i) { return kWaveA - 64 * i < 64 ? kWaveA - 64 * i : 64; }

    static __device__ __forceinline__ Places places(const Args& A, int64_t t0, int n0)
    {
        Places at;
        const uint32_t pitch_x = MX ? A.kp / 2 : 2 * (uint32_t)A.ld_x, pitch_w = A.kp / 2;
        const int lane = threadIdx.x & 63, wave = wave_id();
#pragma unroll
        for (int i = 0; i < kUnitsA; ++i) {
            const int u = wave * kWaveA + i * 64 + lane % lanes_of(i), row = u / AU;
            at.a[i] = (uint32_t)min((int64_t)row, A.tokens - 1 - t0) * pitch_x + 16 * unit_at((u % AU) ^ turn(row));
        }
#pragma unroll
        for (int i = 0; i < kUnitsB; ++i) {
            const int u = kWaveB < 64 ? wave * kWaveB + lane % kWaveB : wave * kWaveB + i * 64 + lane, row = u / BU;
            at.b[i] = (uint32_t)min(row, A.n - 1 - n0) * pitch_w + 16 * (MX ? u % BU ^ turn(row) : u & 1);
        }
        const bool small = GROUPED && A.kp < 512;
        const uint32_t pitch = small ? 0 : A.kp / 32;
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            at.sx[p] = MX ? scale_offset(p, wave, lane, kPartX, A.tokens - t0, pitch) : 0;
            at.sw[p] = scale_offset(p, wave, lane, kPartW, A.n - n0, pitch);
        }
        at.w_scales = buffer_of(small ? A.w : A.w_scales + (int64_t)n0 * (A.kp / 32));
        if constexpr (MX) at.x_scales = buffer_of(small ? A.w : A.x_scales + t0 * (A.kp / 32));
        return at;
    }

    // The first dword of a row's scales in group `group` of a share that begins at k0: 16 bytes of the row, the last ones
    // where it ends before.  (Rows of fewer than 16 bytes: see small_scales.)
    static __device__ __forceinline__ int first_of(const Args& A, int k0, int group) { return min(k0 / 128 + 4 * group, A.kp / 128 - 4); }

    // Part `part` of GROUP of the rows' scales, `dword` of each on.  Where rows are shorter than a group there is nothing to
    // send for; the same loads then read codes, which nobody looks at.
    static __device__ __forceinline__ void stage_group(const Args& A, const Places& at, int dword, int part, u32x4* to)
    {
        const int lane = threadIdx.x & 63, wave = wave_id(), from = A.kp < 512 ? 0 : 4 * dword;
        uint32_t x = at.sx[0], w = at.sw[0];
#pragma unroll
        for (int p = 1; p < PARTS; ++p)
            if (part == p) x = at.sx[p], w = at.sw[p];
        if (lane < kPartX) __builtin_amdgcn_raw_ptr_buffer_load_lds(at.x_scales, (LdsMem*)(to + scale_row(part, wave, 0, kPartX)), 16, x, from, 0, 0);
        if (lane < kPartW) __builtin_amdgcn_raw_ptr_buffer_load_lds(at.w_scales, (LdsMem*)(to + kRowsX + scale_row(part, wave, 0, kPartW)), 16, w, from, 0, 0);
    }

    // Rows of fewer than 16 bytes of scales: all of them, as group 0.
    static __device__ __forceinline__ void small_scales(const Args& A, int64_t t0, int n0, u32x4* scales)
    {
        uint32_t* to = reinterpret_cast<uint32_t*>(scales);
        const int dwords = A.kp / 128;
        for (int r = threadIdx.x; r < kRows; r += kThreads) {
            const uint8_t* row = r < kRowsX ? A.x_scales + min(t0 + r, A.tokens - 1) * (A.kp / 32) : A.w_scales + (int64_t)min(n0 + r - kRowsX, A.n - 1) * (A.kp / 32);
            for (int i = 0; i < dwords; ++i) to[4 * r + i] = reinterpret_cast<const uint32_t*>(row)[i];
        }
    }

    // One step's tiles, straight to LDS, in kParts parts; scales that come with the step go with the first.
    static constexpr int kParts = kUnitsA + kUnitsB;
    static constexpr int kKeep = 0x386;                       // of the scheduler: vector and scalar arithmetic and LDS may pass, loads and products not

    // Where step s of a share from k0 to k1 begins.  Rows of 4 bits are stored in whole 128 values: where half a step of 256 is
    // left it begins earlier, and its first half is left out.
    static __device__ __forceinline__ int start_of(int k0, int k1, int s) { return MX ? min(k0 + s * STEP, k1 - STEP) : k0 + s * STEP; }

    static __device__ __forceinline__ void stage_part(const Args& A, const Places& at, int64_t t0, int n0, int k, int part, u32x4* buf)
    {
        u32x4 *la = buf, *lb = buf + kA;
        uint32_t* ls = reinterpret_cast<uint32_t*>(lb + kB);
        const int lane = threadIdx.x & 63, wave = wave_id();
        if constexpr (!GROUPED) {
            if (part == 0) {
                if (MX && lane < kPartX) __builtin_amdgcn_raw_ptr_buffer_load_lds(at.x_scales, (LdsMem*)(ls + wave * kPartX), 4, at.sx[0], (k / 128) * 4, 0, 0);
                if (lane < kPartW) __builtin_amdgcn_raw_ptr_buffer_load_lds(at.w_scales, (LdsMem*)(ls + kRowsX + wave * kPartW), 4, at.sw[0], (k / 128) * 4, 0, 0);
            }
        }
        if (part < kUnitsB) {
            const Rsrc rb = buffer_of(A.w + (int64_t)n0 * (A.kp / 2));
            if (kWaveB >= 64 || lane < kWaveB)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LdsMem*)(lb + wave * kWaveB + part * 64), 16, at.b[part], k / 2, 0, 0);
        } else {
            const Rsrc ra = MX ? buffer_of(static_cast<const uint8_t*>(A.x) + t0 * (A.kp / 2)) : buffer_of(static_cast<const uint16_t*>(A.x) + t0 * A.ld_x);
            const int i = part - kUnitsB;
            if (lanes_of(i) == 64 || lane < lanes_of(i))
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LdsMem*)(la + wave * kWaveA + i * 64), 16, at.a[i], MX ? k / 2 : 2 * k, 0, 0);
        }
    }

    static __device__ __forceinline__ void stage(const Args& A, const Places& at, int64_t t0, int n0, int k, u32x4* buf)
    {
#pragma unroll
        for (int p = 0; p < kParts; ++p) stage_part(A, at, t0, n0, k, p, buf);
    }

    // The same where a reduction of 16-bit x ends inside the step: zeros past k1, a multiple of 32.  (Rows of 4 bits are
    // stored in whole steps.)
    static __device__ __forceinline__ void stage_tail(const Args& A, int64_t t0, int n0, int k, int k1, u32x4* buf)
    {
        u32x4 *la = buf, *lb = buf + kA;
        for (int u = threadIdx.x; u < kA; u += kThreads) {
            const int row = u / AU, unit = unit_at((u % AU) ^ turn(row));
            u32x4 v{0, 0, 0, 0};
            if (k + 8 * unit < k1) v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(A.x) + min(t0 + row, A.tokens - 1) * A.ld_x + k + 8 * unit);
            la[u] = v;
        }
        for (int u = threadIdx.x; u < kB; u += kThreads) {
            const int row = u / BU, unit = u % BU;
            u32x4 v{0, 0, 0, 0};
            if (k + 32 * unit < k1) v = *reinterpret_cast<const u32x4*>(A.w + (int64_t)min(n0 + row, A.n - 1) * (A.kp / 2) + k / 2 + 16 * unit);
            lb[u] = v;
        }
        uint32_t* ls = reinterpret_cast<uint32_t*>(lb + kB);
        for (int u = threadIdx.x; u < BN; u += kThreads)
            ls[u] = *reinterpret_cast<const uint32_t*>(A.w_scales + (int64_t)min(n0 + u, A.n - 1) * (A.kp / 32) + (k / 128) * 4);
    }

    // ls: the step's dword of the first row's scales, where they come in groups; odd: whether the step is the second of the
    // two that share one (16-bit x).  between(p): what else there is to do, kParts parts of it spread over the products: a wave
    // waits where it sends for more than the memory pipe has taken, and the pipe's time for a step is half of the step's.
    // FROM: 1 leaves the first half of a step of 256 values out.
    template <int FROM, class Between>
    static __device__ __forceinline__ void multiply(const u32x4* buf, const uint32_t* ls, int wm, int wn, int odd, f32x4 (*acc)[NF], Between between)
    {
        const auto spread = [&](int slot, int slots) {
#pragma unroll
            for (int p = 0; p < kParts; ++p)
                if (p * slots / kParts == slot) between(p);
        };
        const u32x4 *la = buf, *lb = buf + kA;
        constexpr int EACH = GROUPED ? 4 : 1;                  // dwords from row to row
        if constexpr (!GROUPED) ls = reinterpret_cast<const uint32_t*>(lb + kB);
        const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
        const int row0 = wm * (BM / WM) + c, col0 = wn * (BN / WN) + c;
        if constexpr (MX) {
            // Token operands are read two fragments ahead of their use, weights a fragment a group before the half of the step
            // that takes them.
            constexpr int HALF = MF / 2, GROUPS = (STEP / 128 - FROM) * HALF;
            u32x4 a[2][2], b[2][NF];
            uint32_t sa[2][2], sb[2][NF];
            // Sixteen rows on a unit's place is the same: one address, and constants from it.
            const auto read_a = [&](int i) {
                const int h = FROM + i / HALF, m = 2 * (i % HALF);
                const u32x4* from = la + row0 * AU + ((4 * h + g) ^ turn(row0));
                const uint32_t* scale = ls + EACH * row0 + h - FROM;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    a[i & 1][p] = from[16 * (m + p) * AU];
                    sa[i & 1][p] = scale[EACH * 16 * (m + p)] >> (8 * g);
                }
            };
            const auto read_b = [&](int h, int n) {
                b[h & 1][n] = (lb + col0 * BU + ((4 * h + g) ^ turn(col0)))[16 * n * BU];
                sb[h & 1][n] = (ls + EACH * (BM + col0) + h - FROM)[EACH * 16 * n] >> (8 * g);
            };
#pragma unroll
            for (int n = 0; n < NF; ++n) read_b(FROM, n);
            read_a(0);
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) {
                const int h = FROM + i / HALF, m = 2 * (i % HALF);
                if (i + 1 < GROUPS) read_a(i + 1);
                if (i + HALF < GROUPS) {
#pragma unroll
                    for (int n = 0; n < NF; ++n)
                        if (n * HALF / NF == i % HALF) read_b(h + 1, n);
                }
                if (i < HALF) spread(i, HALF);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int n = 0; n < NF; ++n) acc[m + p][n] = mfma_mx4<0>(b[h & 1][n], a[i & 1][p], acc[m + p][n], sb[h & 1][n], sa[i & 1][p]);
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
            // Lane group g: bfloat16, values 16 g .. 16 g + 15 of the step, 8 in each of two operands; float16, values
            // 8 g .. 8 g + 7 of each of its two blocks, whose sums are scaled as they are added.
            constexpr bool BLOCKS = XT == kFp16;
            uint32_t raw[NF][2];
            float scale[NF];
            const int sh = 16 * odd + 8 * (g >> 1);
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                const int row = col0 + 16 * n;
                if constexpr (BLOCKS) {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) raw[n][kk] = reinterpret_cast<const uint32_t*>(lb)[row * 8 + 4 * kk + g];
                } else {
                    const uint2 v = reinterpret_cast<const uint2*>(lb)[row * 4 + g];
                    raw[n][0] = v.x, raw[n][1] = v.y;
                    scale[n] = scale_of(ls[row] >> sh);
                }
            }
            // float16: lane 4 n + i of a group has the scales of row 4 g + i of fragment n.
            static_assert(!BLOCKS || NF == 4, "sixteen rows of a group");
            const uint32_t mine = BLOCKS ? ls[wn * (BN / WN) + 16 * (c >> 2) + 4 * g + (c & 3)] >> (16 * odd) : 0;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                u32x4 b[NF];
                const float by = BLOCKS ? value_of(scale_of(mine >> (8 * kk))) : 0.0f;
                const u32x4* from_a = la + row0 * AU + ((4 * kk + g) ^ turn(row0));
#pragma unroll
                for (int n = 0; n < NF; ++n) {
                    if constexpr (BLOCKS) b[n] = widen4_f16(raw[n][kk]);
                    else b[n] = widen4(raw[n][kk], scale[n]);
                }
                // float16: the sums of one group of tokens are added while the next group's are made.
                f32x4 sums[BLOCKS ? 2 : 1][NF];
#pragma unroll
                for (int m = 0; m < MF + BLOCKS; ++m) {
                    if (m < MF) {
                        if constexpr (BLOCKS) __builtin_amdgcn_sched_barrier(kKeep);
                        spread(kk * MF + m, 2 * MF);
                        if constexpr (BLOCKS) __builtin_amdgcn_sched_barrier(kKeep);
                        const u32x4 a = from_a[16 * m * AU];
#pragma unroll
                        for (int n = 0; n < NF; ++n) {
                            if constexpr (BLOCKS) sums[m & 1][n] = mfma_f16(b[n], a, f32x4{0, 0, 0, 0});
                            else acc[m][n] = mfma_bf16(b[n], a, acc[m][n]);
                        }
                    }
                    if constexpr (BLOCKS) {
                        __builtin_amdgcn_sched_barrier(0);
                        if (m > 0) {
                            acc[m - 1][0] = add_scaled<0>(acc[m - 1][0], sums[~m & 1][0], by);
                            acc[m - 1][1] = add_scaled<1>(acc[m - 1][1], sums[~m & 1][1], by);
                            acc[m - 1][2] = add_scaled<2>(acc[m - 1][2], sums[~m & 1][2], by);
                            acc[m - 1][3] = add_scaled<3>(acc[m - 1][3], sums[~m & 1][3], by);
                        }
                    }
                }
            }
        }
    }

    // One step.  The buffers are told apart by __restrict__: else every LDS read waits for the loads to LDS in flight.
    static __device__ __forceinline__ void stage_and_multiply(const Args& A, const Places& at, int64_t t0, int n0, int later, int dword, int part,
                                                              u32x4* __restrict__ to, u32x4* __restrict__ to_scales, const u32x4* __restrict__ from,
                                                              const uint32_t* __restrict__ ls, int wm, int wn, int odd, f32x4 (*acc)[NF])
    {
        multiply<0>(from, ls, wm, wn, odd, acc, [&](int p) {
            if (GROUPED && p == 0) stage_group(A, at, dword, part, to_scales);
            stage_part(A, at, t0, n0, later, p, to);
        });
        // The products belong here: without a use of their sums the compiler puts them behind the barrier that follows, where
        // all waves multiply at once and none reads (4 bits: 571 us for 560, float16 gains 2%).  Of bfloat16 it moves the last
        // few only, which is as well.
#pragma unroll
        for (int m = 0; m < (MX || XT == kFp16 ? MF : 0); ++m)
#pragma unroll
            for (int n = 0; n < NF; ++n) asm volatile("" : "+v"(acc[m][n]));
    }

    // Where the dword of a group's first step lies.
    static __device__ __forceinline__ const uint32_t* scales_of(const Args& A, int k0, int group, const u32x4* scales)
    {
        const int skip = A.kp < 512 ? 0 : k0 / 128 + 4 * group - first_of(A, k0, group);
        return reinterpret_cast<const uint32_t*>(scales + group % 3 * kRows) + skip;
    }
};

template <int XT, int OUT, int BM, int BN, int WM, int WN, int STAGES, int LENGTH>
__global__ __launch_bounds__(kThreads) void tile_kernel(Args A)
{
    typedef Tile<XT, BM, BN, WM, WN, STAGES, LENGTH> S;
    extern __shared__ u32x4 lds[];
    const int wave = wave_id(), wm = wave / WN, wn = wave % WN;
    const Part part = part_of(A.tiling, blockIdx.x);
    const int64_t t0 = (int64_t)part.tm * BM;
    const int n0 = part.tn * BN;
    const int end = XT == kMx4 ? A.kp : A.k, k0 = part.share * A.tiling.length, k1 = part.at < 0 ? end : min(end, k0 + A.tiling.length);
    const int steps = k1 > k0 ? (k1 - k0) / S::STEP : 0;
    const int sent = steps + (S::MX && k0 + steps * S::STEP < k1);      // and half a step
    f32x4 acc[S::MF][S::NF] = {};
    const typename S::Places at = S::places(A, t0, n0);
    constexpr int kUnits = S::kStage / 16;
    u32x4* const scales = lds + STAGES * kUnits;              // of GROUPED tiles
    if (S::GROUPED && k1 > k0) {
        if (A.kp < 512) S::small_scales(A, t0, n0, scales);
        else
#pragma unroll
            for (int i = 0; i < S::GROUP; ++i) S::stage_group(A, at, S::first_of(A, k0, 0), i, scales);
    }
    if (sent > 0) {
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            S::stage(A, at, t0, n0, S::start_of(k0, k1, min(s, sent - 1)), lds + s * kUnits);
            if (S::GROUPED && s == 0) {
#pragma unroll
                for (int i = 0; i < S::GROUP; ++i) S::stage_group(A, at, S::first_of(A, k0, 1), i, scales + S::kRows);
            }
        }
        wait_and_meet<S::kAhead>();
    }
    // At the end of step s the tiles of step s + 1 have to be there, and only what the
    // steps behind the one that sent for them did send for may be under way.  Steps past
    // the last are replaced by the last, so that this count holds in every step.
    int use = 0, fill = STAGES - 1;                           // the buffers of steps s and s + STAGES - 1
    int group = 0, turn = 0, dword = S::first_of(A, k0, 2);   // the step's group, its place in it; where the next but one begins
    u32x4* to_scales = scales + 2 * S::kRows;
    const uint32_t* ls = S::scales_of(A, k0, 0, scales);
    for (int s = 0; s < steps; ++s) {
        S::stage_and_multiply(A, at, t0, n0, S::start_of(k0, k1, min(s + STAGES - 1, sent - 1)), dword, turn, lds + fill * kUnits, to_scales,
                              lds + use * kUnits, ls, wm, wn, s & 1, acc);
        wait_and_meet<S::kAhead>();
        use = use == STAGES - 1 ? 0 : use + 1;
        fill = fill == STAGES - 1 ? 0 : fill + 1;
        ls += S::MX ? S::STEP / 128 : 0;
        if (S::GROUPED && ++turn == S::GROUP) {
            turn = 0;
            ++group;
            dword = S::first_of(A, k0, group + 2);
            to_scales = scales + (group + 2) % 3 * S::kRows;
            ls = S::scales_of(A, k0, group, scales);
        }
    }
    if constexpr (S::MX) {
        if constexpr (S::STEP > 128)
            if (sent > steps) S::template multiply<1>(lds + use * kUnits, ls, wm, wn, 0, acc, [](int) {});
    } else {
        if (k0 + steps * S::STEP < k1) {
            wait_and_meet<0>();
            S::stage_tail(A, t0, n0, k0 + steps * S::STEP, k1, lds);
            wait_and_meet<0>();
            S::template multiply<0>(lds, ls, wm, wn, steps & 1, acc, [](int) {});
        }
    }
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < S::MF; ++m) {
        const int64_t t = t0 + wm * (BM / WM) + m * 16 + c;
        if (t >= A.tokens) continue;
#pragma unroll
        for (int n = 0; n < S::NF; ++n) {
            const int col = n0 + wn * (BN / WN) + n * 16 + 4 * g;
            if (col >= A.n) continue;
            if (part.at >= 0) *reinterpret_cast<f32x4*>(A.sums + ((int64_t)part.at * BM + (t - t0)) * BN + (col - n0)) = acc[m][n];
            else finish<OUT>(A, t, col, acc[m][n]);
        }
    }
    // Loads to LDS that no step used are still under way: they land before the workgroup ends.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ------------------------------------------------------------ choice

// Tokens of few_kernel, which widens each code for up to 64 tokens, and tiles of 128 for 128.  64 x 28672 x 8192 in
// bfloat16, float16 and 4 bits: 47, 53 and 38 us, in tiles 70, 88 and 44; 64 x 4096 x 4096: 15, 15 and 14, in tiles 17, 24
// and 13.  (Past 64 an operand's accumulators leave no registers to read ahead with.)
constexpr uint64_t kFew = 64;

// Microseconds of a step of a workgroup, measured over 8192 values (64 a step, of 4 bits 128): of one alone on its
// compute unit and of two side by side (0: no LDS for a second one, or no gain: two of 128 x 256 in bfloat16 1.54, as one of
// 256 x 256).  Of 96 rows: 77 x 14336 x 4096 in bfloat16 26 us in tiles of 128, 25 so, 192 x 28672 x 8192 120 and 106.
// Those of 128 x 128 hold where weights come from memory, in runs of 32 bytes; from a cache a step takes 0.57, in float16
// 0.75, but choosing by that made 128 x 14336 x 4096 in float16 42 us for 37.
constexpr Cost kCostsBf16[] = {{256, 256, 1.52, 0.0}, {128, 256, 0.93, 0.0}, {128, 128, 0.62, 1.10}, {96, 256, 0.81, 0.0}};
constexpr Cost kCostsFp16[] = {{256, 256, 2.17, 0.0}, {128, 256, 1.37, 0.0}, {128, 128, 1.15, 2.28}, {96, 256, 1.28, 0.0}};
// (The first two are of steps of 256 values: a stored row has to have as many.)
constexpr Cost kCostsMx[] = {{256, 256, 1.16, 0.0}, {128, 256, 0.74, 0.0}, {128, 128, 0.62, 1.18}};

template <int XT>
Tiling tiles_of(uint64_t tokens, uint64_t n, uint64_t k)
{
    if (XT != kMx4) return tiling_of(XT == kBf16 ? kCostsBf16 : kCostsFp16, 4, tokens, n, k, 64, 256, 1024, 128);
    return k > 128 ? tiling_of(kCostsMx, 3, tokens, n, k, 128, 256, 1024, 128) : tiling_of(kCostsMx + 2, 1, tokens, n, k, 128, 256, 1024, 128);
}

struct Few {
    int rows;
    uint32_t shares;
};

// Few tokens.  Rows of a workgroup: as many as leave every compute unit one (two, where two fit: up to four tokens of 16
// bits, 16 of 4), 128, 64 or 32.  28672 x 8192: one bfloat16 token 30, 26 and 35 us, 16 of 4 bits 31 and 27, 24 of bfloat16
// 35 and 40; 4096 x 4096, one token: 8.7, 7.8 and 6.6.
// Shares of the reduction, where even the fewest rows leave compute units without one: if they save as many steps as the
// joining launch costs, 2 to 2.5 us.  A step takes 0.5 to 1.1 us with 16-bit tokens, 0.4 with 4 bits: 8 x 4096 x 4096 in
// float16 11.0 us whole and 8.5 in four shares, 32 in 4 bits 8.6 and 9.1; one token (four steps) 6.6 and 7.8.
Few few_of(uint64_t tokens, uint64_t n, uint64_t k, bool mx)
{
    const int least = tokens <= 4 ? 32 : tokens <= 32 ? 64 : 128;
    const bool two = tokens <= 4 || (mx && tokens <= 16);
    int rows = 128;
    while (rows > least && (n + rows - 1) / rows < (two && rows > 64 ? 256 : 192)) rows /= 2;
    const uint64_t groups = (n + rows - 1) / rows, steps = (k + 32768 / rows - 1) / (32768 / rows);
    uint32_t shares = 1;
    while (shares < 8 && groups * shares <= 128 && steps / (2 * shares) * (32768 / rows) >= 1024) shares *= 2;
    return Few{rows, steps - steps / shares >= (mx ? 8 : 5) ? shares : 1};
}

bool sizes_ok(uint64_t tokens, uint64_t n, uint64_t k)
{
    return tokens <= ECF8A_MAX_TOKENS && n >= 1 && n <= ECF8A_MAX_FEATURES && k >= ECF8X_BLOCK && k <= ECF8A_MAX_FEATURES &&
           k % ECF8X_BLOCK == 0;
}

template <int XT, int OUT, int MF, int RG, int TR = 16 * MF>
int launch_few(const Args& A, uint32_t shares, hipStream_t st)
{
    typedef Stream<kMx4, XT, MF, RG, TR> S;
    auto* kernel = few_kernel<XT, OUT, MF, RG, TR>;
    if (S::kLds > 65536 &&
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds) != hipSuccess)
        return ECF8_ERR_HIP;
    kernel<<<dim3((A.n + S::R - 1) / S::R, shares), S::kThreads, S::kLds, st>>>(A);
    return launch_status();
}

template <int XT, int OUT>
int run_few(const Args& A, const Few& s, hipStream_t st)
{
    // Token rows of a stage: 16 for each fragment, but four where there are no more and they are not the small part of it
    // (28672 x 8192, four tokens of bfloat16 26 us and with 16 rows 30, float16 30 and 36; 4 bits 25 either way).
    if (A.tokens <= 4) {
        constexpr int TR = XT == kMx4 ? 16 : 4;
        if (s.rows == 128) return launch_few<XT, OUT, 1, 4, TR>(A, s.shares, st);
        return s.rows == 64 ? launch_few<XT, OUT, 1, 2, TR>(A, s.shares, st) : launch_few<XT, OUT, 1, 1, TR>(A, s.shares, st);
    }
    if (A.tokens <= 16) return s.rows == 128 ? launch_few<XT, OUT, 1, 4>(A, s.shares, st) : launch_few<XT, OUT, 1, 2>(A, s.shares, st);
    if (A.tokens <= 32) return s.rows == 128 ? launch_few<XT, OUT, 2, 4>(A, s.shares, st) : launch_few<XT, OUT, 2, 2>(A, s.shares, st);
    return A.tokens <= 48 ? launch_few<XT, OUT, 3, 4>(A, s.shares, st) : launch_few<XT, OUT, 4, 4>(A, s.shares, st);
}

template <int XT, int OUT, int BM, int BN, int WM, int WN, int STAGES, int LENGTH>
int launch_tile(const Args& A, hipStream_t st)
{
    constexpr int bytes = Tile<XT, BM, BN, WM, WN, STAGES, LENGTH>::kLds;
    auto* kernel = tile_kernel<XT, OUT, BM, BN, WM, WN, STAGES, LENGTH>;
    if (bytes > 65536 &&
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes) != hipSuccess)
        return ECF8_ERR_HIP;
    kernel<<<groups_of(A.tiling), kThreads, bytes, st>>>(A);
    return launch_status();
}

// The tiles that tiles_of chose.
template <int XT, int OUT>
int run_tiles(const Args& A, hipStream_t st)
{
    const int bm = A.tiling.bm, bn = A.tiling.bn;
    if constexpr (XT == kMx4) {
        if (bm == 256) return launch_tile<XT, OUT, 256, 256, 2, 4, 2, 256>(A, st);
        if (bn == 256) return launch_tile<XT, OUT, 128, 256, 2, 4, 2, 256>(A, st);
        return launch_tile<XT, OUT, 128, 128, 2, 4, 4, 128>(A, st);
    } else {
        if (bm == 256) return launch_tile<XT, OUT, 256, 256, 2, 4, 3, 64>(A, st);
        if (bm == 96) return launch_tile<XT, OUT, 96, 256, 2, 4, 3, 64>(A, st);
        if (bn == 256) return launch_tile<XT, OUT, 128, 256, 2, 4, 3, 64>(A, st);
        return launch_tile<XT, OUT, 128, 128, 4, 2, 3, 64>(A, st);
    }
}

template <int XT, int OUT>
int run(Args A, float* workspace, hipStream_t st)
{
    constexpr bool MX = XT == kMx4;
    if (A.tokens <= (int64_t)kFew) {
        const Few s = few_of(A.tokens, A.n, A.k, MX);
        A.pitch = (A.n + 3) / 4 * 4;
        A.share = (int)round_up((A.k + s.shares - 1) / s.shares, 1024);
        A.sums = s.shares > 1 ? workspace : nullptr;
        const int rc = run_few<XT, OUT>(A, s, st);
        if (rc != ECF8_OK || s.shares < 2) return rc;
        const uint64_t units = (uint64_t)A.tokens * A.pitch / 4;
        join_kernel<OUT><<<(uint32_t)((units + 255) / 256), 256, 0, st>>>(A.sums, A.tokens, A.n, A.pitch, (int)s.shares, A.bias, A.y, A.ld_y);
        return launch_status();
    }
    A.sums = workspace;
    A.tiling = tiles_of<XT>(A.tokens, A.n, A.k);
    const Tiling& s = A.tiling;
    const int rc = run_tiles<XT, OUT>(A, st);
    if (rc != ECF8_OK || s.rest == 0) return rc;
    return join_tiles<OUT>(A.sums, s, A.tokens, A.n, A.bias, A.y, A.ld_y, st);
}

}  // namespace

extern "C" uint64_t ecf8x_linear_bytes(uint64_t tokens, uint64_t out_features, uint64_t in_features, uint32_t x_type)
{
    if (!sizes_ok(tokens, out_features, in_features)) return 0;
    const bool mx = x_type == ECF8X_MX4;
    if (tokens > kFew)
        return sums_of(mx ? tiles_of<kMx4>(tokens, out_features, in_features)
                          : x_type == ECF8A_FP16 ? tiles_of<kFp16>(tokens, out_features, in_features) : tiles_of<kBf16>(tokens, out_features, in_features));
    const uint64_t s = few_of(tokens, out_features, in_features, mx).shares;
    return s > 1 ? round_up(4 * s * tokens * round_up(out_features, 4), 256) : 0;
}

extern "C" int ecf8x_linear(const void* x, const uint8_t* x_scales, uint64_t ld_x, uint32_t x_type, uint64_t tokens, uint64_t out_features,
                            uint64_t in_features, const ecf8x_matrix* w, const void* bias, uint32_t y_type, void* y, uint64_t ld_y,
                            void* workspace, uint64_t workspace_bytes, void* hip_stream)
{
    const bool mx = x_type == ECF8X_MX4;
    if ((y_type != ECF8A_BF16 && y_type != ECF8A_FP16) || (!mx && x_type != y_type)) return ECF8_ERR_UNSUPPORTED;
    if (!sizes_ok(tokens, out_features, in_features)) return ECF8_ERR_SIZE;
    if (tokens == 0) return ECF8_OK;
    if (tokens == 1) ld_x = in_features, ld_y = out_features;
    if (!x || !w || !w->codes || !w->scales || !y || !aligned(x, 16) || !aligned(w->codes, 16) || !aligned(w->scales, 4) || !aligned(y, 2) ||
        !aligned(bias, 2) || (mx ? !x_scales || !aligned(x_scales, 4) : x_scales != nullptr || (tokens > 1 && ld_x % 8)))
        return ECF8_ERR_ARG;
    if ((!mx && (ld_x < in_features || ld_x > (1u << 22))) || ld_y < out_features || ld_y > (1ull << 40)) return ECF8_ERR_SIZE;
    const uint64_t need = ecf8x_linear_bytes(tokens, out_features, in_features, x_type);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return ECF8_ERR_WORKSPACE;
    Args A{};
    A.x = x;
    A.x_scales = x_scales;
    A.ld_x = (int64_t)ld_x;
    A.w = w->codes;
    A.w_scales = w->scales;
    A.bias = static_cast<const uint16_t*>(bias);
    A.y = static_cast<uint16_t*>(y);
    A.ld_y = (int64_t)ld_y;
    A.tokens = (int64_t)tokens;
    A.n = (int)out_features;
    A.k = (int)in_features;
    A.kp = (int)padded(in_features);
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    const bool b = y_type == ECF8A_BF16;
    float* ws = static_cast<float*>(workspace);
    if (mx) return b ? run<kMx4, kBf16>(A, ws, st) : run<kMx4, kFp16>(A, ws, st);
    return b ? run<kBf16, kBf16>(A, ws, st) : run<kFp16, kFp16>(A, ws, st);
}
