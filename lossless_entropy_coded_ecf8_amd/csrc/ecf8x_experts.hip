// ecf8x_experts.hip -- a mixture-of-experts layer for a few tokens: the choice
// of experts, and the gated products of those that were chosen.
//
// What bounds the products is reading the chosen experts' weights: once for every 8
// of an expert's pairs, or 16 or 32, as the pairs an expert of the whole batch has on
// average (the second product of small 4-bit layers: 4).  Batches that are far from
// even read them more often than that average needs: 8 of 256 experts, the same for all
// tokens, E4M3: 8 tokens 68 us, 16 127, 64 496.  Two
// kernels: gate and up with the activation (h of every pair of a token and an
// expert), then down and the weighted sum over a token's experts.  Weights are
// widened exactly; rows of the weight are operand A, the tokens of one expert
// operand B of the matrix instruction.  h keeps float32's 24 bits, as three
// bfloat16 that add up to it; where an expert has four pairs at most, its parts
// are columns of one operand, and the third costs no instruction.  (Two parts, 16
// bits, took 5% less time with eight pairs an expert and more, and as long with fewer, but left
// twice as many results a step off as sums of float32 do.)
//
// Measured: one token, 8 of 256 experts of 7168 x 2048 (352 MB of E4M3) 38 and 24 us,
// 5.6 TB/s; 64 tokens, 8 of the 256 in 4 bits (5.2 GB) 1,040 us together, 5.0 TB/s.
#include "ecf8x_stream.h"

namespace {

using namespace ecf8x;

constexpr int kFp32 = ECF8A_FP32, kThreads = 512;
constexpr int kHalf = 72;                 // KB of LDS with which two workgroups fit a compute unit
constexpr int kPairs = ECF8X_MAX_PAIRS, kExperts = ECF8X_MAX_EXPERTS;

// ---------------------------------------------------------------- choice

struct RouteArgs {
    const void* logits;
    int64_t ld, tokens;
    int32_t* ids;
    float* weights;
    int experts, top, score, normalise;
    float scale;
};

// A logit as an integer in the same order: NaN the largest, 0 for -inf, which is never chosen, and for no expert at all.
__device__ __forceinline__ uint32_t key_of(float v)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);            // -0 is 0
    if (v != v) return 0xFFFFFFFFu;
    if (b == 0xFF800000u) return 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Within 16 lanes by moves between neighbours, then across the four rows.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));       // lane ^ 1
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));       // lane ^ 2
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));      // 8 lanes mirrored
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));      // 16 lanes mirrored
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16), c = __builtin_amdgcn_readlane(v, 32),
                   d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// One wave a token; lane l holds experts l, 64 + l, ...: PER of them.  A round finds the largest logit that is left, and
// the lowest expert that has it.  (Keys of 64 bits that hold both, exchanged through LDS: 14 us where this takes 9, 8192
// tokens, 8 of 256.)  What bounds it is the rounds, one after another: 8 of 256 for one token take 4.2 us, for 8192 8.7
// (8.4 MB read, at 1 TB/s), 8 of 1024 20.
// PER: 1, 4 or 16, the fewest that hold the experts: 64 of them for 8192 tokens 5.6, 8.0 and 18 us, 256 8.7 and 19.
template <int TYPE, int PER>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs A)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= A.tokens) return;
    uint32_t key[PER];
    float logit[PER];                                         // all under way before the first is looked at
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t at = t * A.ld + min(64 * i + lane, A.experts - 1);
        if constexpr (TYPE == kFp32) logit[i] = static_cast<const float*>(A.logits)[at];
        else logit[i] = load1<TYPE>(static_cast<const uint16_t*>(A.logits) + at);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) key[i] = 64 * i + lane < A.experts ? key_of(logit[i]) : 0;
    float all = 0.0f, most = 0.0f;
    uint32_t mine = 0;                                        // the choice that this lane holds: lane j the j-th
    int id = -1;
    for (int j = 0; j < A.top; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) best = max(best, key[i]);
        best = wave_max(best);
        if (j == 0 && best) {
            most = value_of(best);
            if (!A.normalise && A.score == ECF8X_SOFTMAX) {
#pragma unroll
                for (int i = 0; i < PER; ++i) all += key[i] ? expf(value_of(key[i]) - most) : 0.0f;
                all = wave_sum(all);
            }
        }
        if (best == 0) break;
        int expert = -1;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint64_t has = expert < 0 ? __ballot(key[i] == best) : 0;
            if (has) {
                expert = 64 * i + __ffsll((unsigned long long)has) - 1;
                if (lane == (expert & 63)) key[i] = 0;
            }
        }
        if (lane == j) mine = best, id = expert;
    }
    const float v = value_of(mine);
    // Sigmoids that are normalised may share a factor: exp(-most) keeps those of large negative logits from vanishing.
    float p = 0.0f;
    if (mine) {
        if (A.score == ECF8X_SOFTMAX) p = expf(v - most);
        else p = A.normalise && most < 0.0f ? expf(v - most) / (1.0f + expf(v)) : 1.0f / (1.0f + expf(-v));
    }
    const float sum = A.normalise ? wave_sum(p) : A.score == ECF8X_SOFTMAX ? all : 1.0f;
    if (lane < A.top) {
        A.ids[t * A.top + lane] = id;
        A.weights[t * A.top + lane] = mine ? A.scale * (p / sum) : 0.0f;
    }
}

// -------------------------------------------------------------- products

struct Matrix {
    const uint8_t *codes, *scales;
    const float* factors;
};

struct MoeArgs {
    const uint16_t* x;
    int64_t ld_x;
    Matrix gate, up, down;
    const int32_t* ids;
    const float* weights;
    uint16_t* h;                // [pair][3][inner]: three bfloat16, which add up to the float32 value
    uint16_t* y;
    int64_t ld_y;
    float* part;                // [pair][features]
    uint32_t* counters;         // of the second kernel's tiles: workgroups that have ended
    int tokens, top, pairs, features, inner, experts, tiles;
};

// The pairs of one expert, in LDS.  Their order is free: a pair's results do not
// depend on its column.
struct Group {
    uint32_t chosen[kExperts / 32];                           // a bit for each expert that some pair names
    uint32_t count;
    uint16_t pair[kPairs];
};

// The chosen expert of rank r, in the order of their numbers, and its pairs: the
// number of chosen experts, expert -1 where there are no more than r.
__device__ __forceinline__ int find(const MoeArgs& A, Group& G, int r, int& expert)
{
    const int tid = threadIdx.x, lane = tid & 63;
    if (tid < kExperts / 32) G.chosen[tid] = 0;
    if (tid == 0) G.count = 0;
    int id = -1;
    if (tid < A.pairs) id = A.ids[tid];
    const bool is = id >= 0 && id < A.experts;
    __syncthreads();
    if (is) atomicOr(&G.chosen[id >> 5], 1u << (id & 31));
    __syncthreads();
    // Every wave finds the r-th bit for itself.
    uint32_t word = lane < kExperts / 32 ? G.chosen[lane] : 0;
    const int own = __popc(word);
    int upto = own;
#pragma unroll
    for (int d = 1; d < kExperts / 32; d <<= 1) {
        const int o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    const int chosen = __shfl(upto, kExperts / 32 - 1);
    expert = -1;
    if (r < chosen) {
        const int at = __ffsll((unsigned long long)__ballot(lane < kExperts / 32 && upto > r)) - 1;
        word = __shfl(word, at);
        for (int skip = r - __shfl(upto - own, at); skip > 0; --skip) word &= word - 1;
        expert = 32 * at + __ffs(word) - 1;
    }
    if (is && id == expert) G.pair[atomicAdd(&G.count, 1u)] = (uint16_t)tid;
    __syncthreads();
    return chosen;
}

// Bytes and scale bytes of a stored row.
template <int W>
__device__ __forceinline__ uint32_t row_bytes(int cols) { return W == kMx4 ? (cols + 127) / 128 * 64 : cols; }

__device__ __forceinline__ uint32_t row_scales(int cols) { return (cols + 127) / 128 * 4; }

// h of an expert's pairs p0 .. p0 + TR - 1, for as many rows of gate as of up:
// fragment 0 of a row group of the one, fragment 1 of the other.
template <class S, int W, int MF, int RG, int TR>
__device__ __forceinline__ void gate_up(const MoeArgs& A, const Group& G, int e, int p0, char* lds)
{
    const int lane = threadIdx.x & 63, wave = wave_id(), c = lane & 15, g = lane >> 4, count = G.count;
    const int i0 = blockIdx.x * (S::R / 2), frag = S::fragment(wave), first = min(i0 + 16 * (frag / 2), A.inner - 1);
    const Matrix& w = frag & 1 ? A.up : A.gate;
    const int64_t row = (int64_t)e * A.inner + first;         // rows past the last reach no result that is stored
    const typename S::Rows rows{w.codes + row * row_bytes<W>(A.features), w.scales + row * row_scales(A.features), A.inner - 1 - first};
    const typename S::Places at = S::places(rows, row_bytes<W>(A.features), row_scales(A.features), A.x, nullptr, 0, [&](int i) {
        return (uint32_t)(G.pair[min(p0 + i, count - 1)] / A.top) * (uint32_t)A.ld_x * 2;
    });
    f32x4 acc[2][MF] = {};
    if (p0) __syncthreads();                                  // the sums of the pairs before are read
    S::run(rows, at, A.x, nullptr, A.features, lds, acc);
    if (wave >= RG) return;
    const float fa = A.gate.factors ? A.gate.factors[e] : 1.0f, fb = A.up.factors ? A.up.factors[e] : 1.0f;
#pragma unroll
    for (int m = 0; m < MF; ++m) {
        const int p = p0 + 16 * m + c, i = i0 + 16 * wave + 4 * g;
        if (p >= count || 16 * m + c >= TR || i >= A.inner) continue;
        f32x4 h;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v = acc[0][m][q] * fa;
            h[q] = v / (1.0f + expf(-v)) * (acc[1][m][q] * fb);
        }
        uint32_t part[3][2];
        split3(h[0], h[1], part[0][0], part[1][0], part[2][0]);
        split3(h[2], h[3], part[0][1], part[1][1], part[2][1]);
        uint16_t* out = A.h + (int64_t)G.pair[p] * 3 * A.inner + i;          // inner is a multiple of 16
#pragma unroll
        for (int j = 0; j < 3; ++j) *reinterpret_cast<uint2*>(out + j * A.inner) = make_uint2(part[j][0], part[j][1]);
    }
}

template <int W, int TYPE, int MF, int RG>
__global__ __launch_bounds__(kThreads) void gate_up_kernel(MoeArgs A)
{
    __shared__ Group G;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    if (blockIdx.x == 0 && blockIdx.y == 0)                   // nothing counts in the second kernel before this one ends
        for (int i = threadIdx.x; i < A.tiles; i += kThreads) A.counters[i] = 0;
    int e;
    find(A, G, blockIdx.y, e);
    if (e < 0) return;
    const int count = G.count;
    if constexpr (MF == 0) {
        if (count <= 4) gate_up<Stream<W, TYPE, 1, RG, 4, kHalf>, W, 1, RG, 4>(A, G, e, 0, lds);
        else
            for (int p0 = 0; p0 < count; p0 += 8) gate_up<Stream<W, TYPE, 1, RG, 8, kHalf>, W, 1, RG, 8>(A, G, e, p0, lds);
    } else {
        for (int p0 = 0; p0 < count; p0 += 16 * MF) gate_up<Stream<W, TYPE, MF, RG>, W, MF, RG, 16 * MF>(A, G, e, p0, lds);
    }
}

// Sums that workgroups on other dies read: written through the die's own cache, and
// read past it.  (Plain stores and a release fence, which writes that whole cache
// back, took 114 us where the whole kernel takes 25 so: one token, 8 experts, 117 MB of weights.)
constexpr int kPastDie = 16;

__device__ __forceinline__ void put(Rsrc r, uint32_t at, f32x4 v)
{
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, at, 0, kPastDie);
}

__device__ __forceinline__ f32x4 get(Rsrc r, uint32_t at)
{
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kPastDie));
}

// The sums of an expert's pairs p0 .. p0 + TR - 1 for R features.
template <class S, int W, int MF, int RG, int TR>
__device__ __forceinline__ void down(const MoeArgs& A, const Group& G, Rsrc part, int e, int p0, char* lds)
{
    const int lane = threadIdx.x & 63, wave = wave_id(), c = lane & 15, g = lane >> 4, count = G.count;
    const int k0 = blockIdx.x * S::R, first = min(k0 + 16 * S::fragment(wave), A.features - 1);
    const int64_t row = (int64_t)e * A.features + first;
    const typename S::Rows rows{A.down.codes + row * row_bytes<W>(A.inner), A.down.scales + row * row_scales(A.inner), A.features - 1 - first};
    const float factor = A.down.factors ? A.down.factors[e] : 1.0f;
    const typename S::Places at = S::places(rows, row_bytes<W>(A.inner), row_scales(A.inner), A.h, nullptr, 2 * A.inner, [&](int i) {
        return (uint32_t)G.pair[min(p0 + i, count - 1)] * 6 * (uint32_t)A.inner;
    });
    f32x4 acc[S::RF][MF] = {};
    if (p0) __syncthreads();
    S::run(rows, at, A.h, nullptr, A.inner, lds, acc);
    if (wave >= RG) return;
#pragma unroll
    for (int f = 0; f < S::RF; ++f)
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            const int p = p0 + 16 * m + c, k = k0 + 16 * (wave * S::RF + f) + 4 * g;
            if (p < count && 16 * m + c < TR && k < A.features)       // features are a multiple of 16
                put(part, 4 * (G.pair[p] * (uint32_t)A.features + k), acc[f][m] * factor);
        }
}

// y: a workgroup takes R features of one expert and leaves its pairs' sums in the
// workspace; the last one of these features to end adds them up, a token's in the
// order of its choices, whichever workgroup that is.
template <int W, int TYPE, int MF, int RG>
__global__ __launch_bounds__(kThreads) void down_kernel(MoeArgs A)
{
    typedef Stream<W, kThree, MF ? MF : 1, RG> S;
    __shared__ Group G;
    __shared__ uint32_t ended;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    int e;
    const int chosen = find(A, G, blockIdx.y, e), k0 = blockIdx.x * S::R, count = G.count;
    const Rsrc part = buffer_of(A.part);
    if (e < 0 && (chosen || blockIdx.y)) return;              // where no token has an expert one workgroup clears y
    if (chosen) {
        if constexpr (MF == 0) {
            constexpr int TR = W == kMx4 && RG == 2 ? 4 : 8;   // (half of the LDS has no room for two stages of eight there)
            if (count <= 4) down<Stream<W, kThree, 1, RG, 4, kHalf>, W, 1, RG, 4>(A, G, part, e, 0, lds);
            else
                for (int p0 = 0; p0 < count; p0 += TR) down<Stream<W, kThree, 1, RG, TR, kHalf>, W, 1, RG, TR>(A, G, part, e, p0, lds);
        } else {
            for (int p0 = 0; p0 < count; p0 += 16 * MF) down<S, W, MF, RG, 16 * MF>(A, G, part, e, p0, lds);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // every wave's sums are where other dies see them
        __syncthreads();
        if (threadIdx.x == 0) ended = __hip_atomic_fetch_add(A.counters + blockIdx.x, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if ((int)ended != chosen - 1) return;
        asm volatile("" ::: "memory");
    }
    constexpr int kQuads = S::R / 4;
    for (int i = threadIdx.x; i < A.tokens * kQuads; i += kThreads) {
        const int t = i / kQuads, k = k0 + 4 * (i % kQuads);
        if (k >= A.features) continue;
        f32x4 y{0, 0, 0, 0};
        for (int j = 0; j < A.top; ++j) {
            const int pair = t * A.top + j, id = A.ids[pair];
            if (id < 0 || id >= A.experts) continue;
            y += get(part, 4 * (pair * (uint32_t)A.features + k)) * A.weights[pair];
        }
        store4<TYPE>(A.y + t * A.ld_y + k, y, 4);
    }
}

template <int TYPE>
void route(const RouteArgs& A, hipStream_t st)
{
    const uint32_t grid = (uint32_t)((A.tokens + 3) / 4);
    if (A.experts <= 64) route_kernel<TYPE, 1><<<grid, 256, 0, st>>>(A);
    else if (A.experts <= 256) route_kernel<TYPE, 4><<<grid, 256, 0, st>>>(A);
    else route_kernel<TYPE, 16><<<grid, 256, 0, st>>>(A);
}

template <class Kernel>
int allow(Kernel* kernel, int bytes)
{
    return bytes <= 65536 || hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes) == hipSuccess
               ? ECF8_OK
               : ECF8_ERR_HIP;
}

// Features of a workgroup of the second kernel: the fewest that any choice below has.
constexpr uint64_t kLeastRows = 64;

template <int W, int TYPE, int MF, int RG>
int moe(MoeArgs A, hipStream_t st)
{
    constexpr int R = 32 * RG, rows = R / 2;                  // features of a workgroup of the second kernel, rows of gate of the first
    int first, second;                                        // LDS
    if constexpr (MF == 0) first = second = kHalf * 1024;
    else first = Stream<W, TYPE, MF, RG>::kLds, second = Stream<W, kThree, MF, RG>::kLds;
    const int most = A.pairs < A.experts ? A.pairs : A.experts;
    A.tiles = (A.features + R - 1) / R;
    if (allow(gate_up_kernel<W, TYPE, MF, RG>, first) != ECF8_OK || allow(down_kernel<W, TYPE, MF, RG>, second) != ECF8_OK) return ECF8_ERR_HIP;
    gate_up_kernel<W, TYPE, MF, RG><<<dim3((A.inner + rows - 1) / rows, most), kThreads, first, st>>>(A);
    const int rc = launch_status();
    if (rc != ECF8_OK) return rc;
    down_kernel<W, TYPE, MF, RG><<<dim3(A.tiles, most), kThreads, second, st>>>(A);
    return launch_status();
}

template <int W, int TYPE>
int moe(const MoeArgs& A, hipStream_t st)
{
    // Token rows of a stage, by how many an expert meets on average, up to the most that any can.  Microseconds of both
    // launches, experts x features x inner:
    //   4 or 8 rows (two workgroups a compute unit) or 16: 128 x 4096 x 1024, 4 pairs an expert: 4-bit weights 226 and 298,
    //     E4M3 297 and 297; 2 an expert: 182 and 255, 245 and 254; 8 an expert (64 x 2048 x 1408): 154 and 147, 178 and 131;
    //   16 or 32: 64 x 2048 x 1408, 8 an expert: E4M3 131 and 144; 8 x 4096 x 2048, 16 an expert of 64 tokens: 99 and 62.
    // With so few chosen experts that 128 features a workgroup would not give every compute unit one, 64: 8 experts of
    // 4096 x 1024 for one token 31 and 33 us (4 bits: 24 and 29); 32 of 2048 x 1408: 57 and 51.
    const int most = A.pairs < A.experts ? A.pairs : A.experts;
    const bool small = (A.features + 127) / 128 * most <= 256;
    if (A.pairs <= (W == kMx4 || small ? 4 : 2) * A.experts) return small ? moe<W, TYPE, 0, 2>(A, st) : moe<W, TYPE, 0, 4>(A, st);
    if (A.tokens <= 16 || A.pairs <= 8 * A.experts) return moe<W, TYPE, 1, 4>(A, st);
    return moe<W, TYPE, 2, 4>(A, st);
}

bool layer_ok(const ecf8x_experts& L)
{
    const uint64_t unit = L.type == ECF8X_MX4 ? 32 : 16;
    return L.features >= unit && L.inner >= unit && L.features % unit == 0 && L.inner % unit == 0 && L.features <= 65536 && L.inner <= 65536 &&
           L.experts >= 1 && L.experts <= ECF8X_MAX_EXPERTS;
}

bool matrix_ok(const ecf8x_matrix& m, bool mx)
{
    return m.codes && aligned(m.codes, 16) && (mx ? m.scales && aligned(m.scales, 4) && !m.factors : !m.scales && aligned(m.factors, 4));
}

}  // namespace

extern "C" int ecf8x_route(const void* logits, uint64_t ld, uint32_t type, uint64_t tokens, uint32_t experts, uint32_t top, uint32_t score,
                           uint32_t normalise, float scale, int32_t* ids, float* weights, void* hip_stream)
{
    if ((type != ECF8A_FP32 && type != ECF8A_BF16 && type != ECF8A_FP16) || score > ECF8X_SIGMOID) return ECF8_ERR_UNSUPPORTED;
    if (tokens > ECF8A_MAX_TOKENS || experts < 1 || experts > ECF8X_MAX_EXPERTS || top < 1 || top > experts || top > ECF8X_MAX_TOP)
        return ECF8_ERR_SIZE;
    if (tokens == 0) return ECF8_OK;
    if (tokens == 1) ld = experts;
    if (!logits || !ids || !weights || !aligned(logits, type == ECF8A_FP32 ? 4 : 2) || !aligned(ids, 4) || !aligned(weights, 4)) return ECF8_ERR_ARG;
    if (ld < experts || ld > (1ull << 36)) return ECF8_ERR_SIZE;
    const RouteArgs A{logits, (int64_t)ld, (int64_t)tokens, ids, weights, (int)experts, (int)top, (int)score, normalise != 0, scale};
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    if (type == ECF8A_FP32) route<kFp32>(A, st);
    else if (type == ECF8A_BF16) route<kBf16>(A, st);
    else route<kFp16>(A, st);
    return launch_status();
}

extern "C" uint64_t ecf8x_moe_bytes(uint64_t tokens, uint32_t top, const ecf8x_experts* layer)
{
    if (!layer || !layer_ok(*layer) || top > ECF8X_MAX_TOP || tokens > ECF8X_MAX_PAIRS || tokens * top > ECF8X_MAX_PAIRS) return 0;
    // h, the pairs' sums, the counters
    return round_up(tokens * top * 6 * layer->inner, 256) + round_up(tokens * top * 4 * layer->features, 256) +
           round_up(4 * ((layer->features + kLeastRows - 1) / kLeastRows), 256);
}

extern "C" int ecf8x_moe(const void* x, uint64_t ld_x, uint32_t type, uint64_t tokens, uint32_t top, const int32_t* ids, const float* weights,
                         const ecf8x_experts* layer, void* y, uint64_t ld_y, void* workspace, uint64_t workspace_bytes, void* hip_stream)
{
    if (!layer) return ECF8_ERR_ARG;
    const bool mx = layer->type == ECF8X_MX4;
    if ((type != ECF8A_BF16 && type != ECF8A_FP16) || (!mx && layer->type != ECF8A_E4M3)) return ECF8_ERR_UNSUPPORTED;
    if (!layer_ok(*layer) || top < 1 || top > ECF8X_MAX_TOP || tokens > ECF8X_MAX_PAIRS || tokens * top > ECF8X_MAX_PAIRS) return ECF8_ERR_SIZE;
    if (tokens == 0) return ECF8_OK;
    if (tokens == 1) ld_x = ld_y = layer->features;
    if (!x || !y || !ids || !weights || !aligned(x, 16) || !aligned(y, 2) || !aligned(ids, 4) || !aligned(weights, 4) || (tokens > 1 && ld_x % 8) ||
        !matrix_ok(layer->gate, mx) || !matrix_ok(layer->up, mx) || !matrix_ok(layer->down, mx))
        return ECF8_ERR_ARG;
    if (ld_x < layer->features || ld_y < layer->features || ld_x > (1u << 21) || ld_y > (1ull << 40)) return ECF8_ERR_SIZE;   // 512 rows: 32-bit offsets
    const uint64_t need = ecf8x_moe_bytes(tokens, top, layer);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return ECF8_ERR_WORKSPACE;
    MoeArgs A{};
    A.x = static_cast<const uint16_t*>(x);
    A.ld_x = (int64_t)ld_x;
    const auto matrix = [](const ecf8x_matrix& m) { return Matrix{m.codes, m.scales, m.factors}; };
    A.gate = matrix(layer->gate);
    A.up = matrix(layer->up);
    A.down = matrix(layer->down);
    A.ids = ids;
    A.weights = weights;
    A.h = static_cast<uint16_t*>(workspace);
    A.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + round_up(tokens * top * 6 * layer->inner, 256));
    A.counters = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(A.part) + round_up(tokens * top * 4 * layer->features, 256));
    A.y = static_cast<uint16_t*>(y);
    A.ld_y = (int64_t)ld_y;
    A.tokens = (int)tokens;
    A.top = (int)top;
    A.pairs = (int)(tokens * top);
    A.features = (int)layer->features;
    A.inner = (int)layer->inner;
    A.experts = (int)layer->experts;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    if (mx) return type == ECF8A_BF16 ? moe<kMx4, kBf16>(A, st) : moe<kMx4, kFp16>(A, st);
    return type == ECF8A_BF16 ? moe<kE4m3, kBf16>(A, st) : moe<kE4m3, kFp16>(A, st);
}
