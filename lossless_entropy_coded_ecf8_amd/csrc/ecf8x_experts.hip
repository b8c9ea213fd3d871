// ecf8x_experts.hip -- a mixture-of-experts layer for a few tokens: the choice
// of experts, and the gated products of those that were chosen.
//
// What bounds the products is reading the chosen experts' weights, once.  Two
// kernels: gate and up with the activation (h of every pair of a token and an
// expert), then down and the weighted sum over a token's experts.  Weights go
// from memory to registers, 64 contiguous bytes a lane, and are widened there
// (exact); rows of the weight are operand A, the tokens of one expert operand B
// of the matrix instruction.  No sum crosses a workgroup.
#include "ecf8x_common.h"

namespace {

using namespace ecf8x;

constexpr int kFp32 = ECF8A_FP32, kThreads = 512, kWaves = 8;
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

// Larger keys first: the value in order, then the lower expert.  NaN is the
// largest, 0 no expert at all.
__device__ __forceinline__ uint64_t key_of(float v, int e)
{
    uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);      // -0 is 0
    if (v != v) b = 0x7FFFFFFFu;
    if (b == 0xFF800000u) return 0;
    b = b & 0x80000000u ? ~b : b | 0x80000000u;
    return (uint64_t)b << 32 | (uint32_t)~e;
}

__device__ __forceinline__ float value_of(uint64_t key)
{
    const uint32_t b = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

__device__ __forceinline__ uint64_t wave_max(uint64_t v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, d);
        v = o > v ? o : v;
    }
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// One wave a token; PER experts a lane.
template <int TYPE, int PER>
__global__ __launch_bounds__(256) void route_kernel(RouteArgs A)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= A.tokens) return;
    uint64_t key[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = 64 * i + lane;
        key[i] = 0;
        if (e >= A.experts) continue;
        float v;
        if constexpr (TYPE == kFp32) v = static_cast<const float*>(A.logits)[t * A.ld + e];
        else v = load1<TYPE>(static_cast<const uint16_t*>(A.logits) + t * A.ld + e);
        key[i] = key_of(v, e);
    }
    float all = 0.0f, most = 0.0f;
    uint64_t mine = 0;                                        // the choice that this lane holds: lane j the j-th
    for (int j = 0; j < A.top; ++j) {
        uint64_t best = key[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) best = key[i] > best ? key[i] : best;
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
        if (lane == j) mine = best;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (key[i] == best) key[i] = 0;
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
        A.ids[t * A.top + lane] = mine ? (int32_t)~(uint32_t)mine : -1;
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
    uint16_t* h;                // [pair][2][inner]: upper and lower bfloat16
    uint16_t* y;
    int64_t ld_y;
    int tokens, top, pairs, features, inner, experts;
    int slots;                  // sums that the second kernel has room for
    bool vector;                // y's rows take 8-byte stores
};

// The pairs sorted by expert, in LDS.  Order within an expert is free: a pair's
// results do not depend on its column.
struct Groups {
    uint32_t count[kExperts];                                 // of each expert, then where its pairs begin
    uint32_t total[kWaves];
    uint16_t expert[kPairs], first[kPairs + 1];               // of the chosen experts, in order
    uint16_t pair[kPairs];
};

// Returns the number of chosen experts.
__device__ __forceinline__ int group(const MoeArgs& A, Groups& G)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < A.experts; e += kThreads) G.count[e] = 0;
    int id = -1;
    if (tid < A.pairs) id = A.ids[tid];
    const bool is = id >= 0 && id < A.experts;
    __syncthreads();
    uint32_t rank = 0;
    if (is) rank = atomicAdd(&G.count[id], 1u);
    __syncthreads();
    // Two experts a thread: pairs in the low half, chosen experts in the high half of one running sum.
    const int e0 = 2 * tid, e1 = e0 + 1;
    const uint32_t c0 = e0 < A.experts ? G.count[e0] : 0, c1 = e1 < A.experts ? G.count[e1] : 0;
    const uint32_t own = (c0 + c1) | ((uint32_t)((c0 != 0) + (c1 != 0)) << 16);
    uint32_t sum = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 63) G.total[wave] = sum;
    __syncthreads();
    uint32_t before = sum - own;
    for (int i = 0; i < wave; ++i) before += G.total[i];
    const uint32_t pos = before & 0xFFFF, at = before >> 16;
    if (c0) G.expert[at] = (uint16_t)e0, G.first[at] = (uint16_t)pos;
    if (c1) G.expert[at + (c0 != 0)] = (uint16_t)e1, G.first[at + (c0 != 0)] = (uint16_t)(pos + c0);
    if (e0 < A.experts) G.count[e0] = pos;
    if (e1 < A.experts) G.count[e1] = pos + c0;
    uint32_t all = 0;
    for (int i = 0; i < kWaves; ++i) all += G.total[i];
    const int chosen = (int)(all >> 16);
    if (tid == 0) G.first[chosen] = (uint16_t)(all & 0xFFFF);
    __syncthreads();
    if (is) G.pair[G.count[id] + rank] = (uint16_t)tid;
    __syncthreads();
    return chosen;
}

// What 64 contiguous bytes of a weight row, a lane's share of a step, need: chunks
// of 16 bytes, each VALUES values and OPS operands.
template <int W>
struct Format {
    static constexpr int VALUES = W == kMx4 ? 32 : 16, OPS = VALUES / 8;
    static constexpr int UNIT = 4 * VALUES;                   // values of a lane's 64 bytes

    // Bytes and scale bytes of a stored row.
    static __device__ __forceinline__ int64_t row_bytes(int cols) { return W == kMx4 ? (cols + 127) / 128 * 64 : cols; }
    static __device__ __forceinline__ int64_t row_scales(int cols) { return (cols + 127) / 128 * 4; }
};

// The 64 bytes of a row's unit, nothing past the last column; their scales.
template <int W>
struct Weights {
    u32x4 chunk[4];
    uint32_t scales;

    __device__ __forceinline__ void load(const uint8_t* row, const uint8_t* row_scales, int unit, bool in, int cols)
    {
        scales = 0;
#pragma unroll
        for (int s = 0; s < 4; ++s) chunk[s] = u32x4{0, 0, 0, 0};
        if (!in) return;
        if constexpr (W == kMx4) {                            // stored rows are whole units
            scales = *reinterpret_cast<const uint32_t*>(row_scales + 4 * unit);
#pragma unroll
            for (int s = 0; s < 4; ++s) chunk[s] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + 64 * unit + 16 * s));
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (64 * unit + 16 * s < cols) chunk[s] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(row + 64 * unit + 16 * s));
        }
    }

    // Operand j of chunk s, in TYPE (4-bit weights: bfloat16).
    template <int TYPE>
    __device__ __forceinline__ u32x4 operand(int s, int j) const
    {
        if constexpr (W == kMx4) return widen4(chunk[s][j], scale_of(scales >> (8 * s) & 255));
        return widen8<TYPE>(chunk[s][2 * j], chunk[s][2 * j + 1]);
    }
};

// h of every pair: a workgroup takes 16 rows of gate and of up of one expert, its
// eight waves a share of the reduction each.
template <int W, int TYPE, int MF>
__global__ __launch_bounds__(kThreads) void gate_up_kernel(MoeArgs A)
{
    typedef Format<W> F;
    __shared__ Groups G;
    __shared__ f32x4 sums[kWaves][2][MF][64];
    const int chosen = group(A, G);
    if ((int)blockIdx.y >= chosen) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int e = G.expert[blockIdx.y], first = G.first[blockIdx.y], count = G.first[blockIdx.y + 1] - first;
    const int i0 = blockIdx.x * 16;
    const int64_t row = (int64_t)e * A.inner + min(i0 + c, A.inner - 1);       // rows past the last reach no result that is stored
    const uint8_t *wg = A.gate.codes + row * F::row_bytes(A.features), *wu = A.up.codes + row * F::row_bytes(A.features);
    const uint8_t *sg = A.gate.scales + row * F::row_scales(A.features), *su = A.up.scales + row * F::row_scales(A.features);
    const int units = (A.features + F::UNIT - 1) / F::UNIT, u0 = units * wave / kWaves, u1 = units * (wave + 1) / kWaves;
    for (int p0 = 0; p0 < count; p0 += 16 * MF) {
        const uint16_t* x[MF];
        bool there[MF];
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            there[m] = p0 + 16 * m + c < count;
            x[m] = A.x + (int64_t)(G.pair[first + min(p0 + 16 * m + c, count - 1)] / A.top) * A.ld_x;
        }
        f32x4 acc[2][MF] = {};
        for (int u = u0; u < u1; u += 4) {
            const int unit = u + g;
            const bool in = unit < u1;
            Weights<W> a, b;
            a.load(wg, sg, unit, in, A.features);
            b.load(wu, su, unit, in, A.features);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = unit * F::UNIT + s * F::VALUES;
                u32x4 v[MF][F::OPS];
#pragma unroll
                for (int m = 0; m < MF; ++m) {
#pragma unroll
                    for (int j = 0; j < F::OPS; ++j) v[m][j] = u32x4{0, 0, 0, 0};
                    if (in && there[m] && k < A.features) {
#pragma unroll
                        for (int j = 0; j < F::OPS; ++j) v[m][j] = *reinterpret_cast<const u32x4*>(x[m] + k + 8 * j);
                    }
                }
#pragma unroll
                for (int j = 0; j < F::OPS; ++j) {
                    const u32x4 wa = a.template operand<TYPE>(s, j), wb = b.template operand<TYPE>(s, j);
#pragma unroll
                    for (int m = 0; m < MF; ++m) {
                        if constexpr (W == kMx4 && TYPE == kFp16) {
                            u32x4 hi, lo;
                            split8_f16(v[m][j], hi, lo);
                            acc[0][m] = mfma_bf16(wa, hi, acc[0][m]);
                            acc[1][m] = mfma_bf16(wb, hi, acc[1][m]);
                            acc[0][m] = mfma_bf16(wa, lo, acc[0][m]);
                            acc[1][m] = mfma_bf16(wb, lo, acc[1][m]);
                        } else {
                            acc[0][m] = mfma<TYPE>(wa, v[m][j], acc[0][m]);
                            acc[1][m] = mfma<TYPE>(wb, v[m][j], acc[1][m]);
                        }
                    }
                }
            }
        }
        if (p0) __syncthreads();                              // the sums of the pairs before are read
#pragma unroll
        for (int m = 0; m < MF; ++m) sums[wave][0][m][lane] = acc[0][m], sums[wave][1][m][lane] = acc[1][m];
        __syncthreads();
        const int m = wave, at = p0 + 16 * m + c, i = i0 + 4 * g;
        if (m < MF && at < count && i < A.inner) {
            f32x4 a{0, 0, 0, 0}, b{0, 0, 0, 0}, h;
#pragma unroll
            for (int q = 0; q < kWaves; ++q) a += sums[q][0][m][lane], b += sums[q][1][m][lane];
            const float fa = A.gate.factors ? A.gate.factors[e] : 1.0f, fb = A.up.factors ? A.up.factors[e] : 1.0f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float v = a[q] * fa;
                h[q] = v / (1.0f + expf(-v)) * (b[q] * fb);
            }
            uint32_t hi[2], lo[2];
            split2(h[0], h[1], hi[0], lo[0]);
            split2(h[2], h[3], hi[1], lo[1]);
            uint16_t* out = A.h + (int64_t)G.pair[first + at] * 2 * A.inner + i;   // inner is a multiple of 16
            *reinterpret_cast<uint2*>(out) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(out + A.inner) = make_uint2(lo[0], lo[1]);
        }
    }
}

// y: a workgroup takes 16 RF features of every chosen expert, a wave an expert (or
// a share of its reduction, where few are chosen) at a time.  Each pair's sums go to
// a place of their own in LDS, and a token's are added in the order of its choices.
template <int W, int TYPE, int RF, int MF>
__global__ __launch_bounds__(kThreads) void down_kernel(MoeArgs A)
{
    typedef Format<W> F;
    __shared__ Groups G;
    extern __shared__ f32x4 sums[];                           // [share][pair][4 RF]
    const int chosen = group(A, G);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int k0 = blockIdx.x * 16 * RF;
    int shares = 1;
    while (shares < kWaves && chosen * shares < kWaves && 2 * shares * A.pairs <= A.slots) shares *= 2;
    const int units = (A.inner + F::UNIT - 1) / F::UNIT;
    for (int job = wave; job < chosen * shares; job += kWaves) {
        const int r = job / shares, share = job % shares, u0 = units * share / shares, u1 = units * (share + 1) / shares;
        const int e = G.expert[r], first = G.first[r], count = G.first[r + 1] - first;
        const uint8_t *w[RF], *ws[RF];
#pragma unroll
        for (int f = 0; f < RF; ++f) {
            const int64_t row = (int64_t)e * A.features + min(k0 + 16 * f + c, A.features - 1);
            w[f] = A.down.codes + row * F::row_bytes(A.inner);
            ws[f] = A.down.scales + row * F::row_scales(A.inner);
        }
        const float factor = A.down.factors ? A.down.factors[e] : 1.0f;
        for (int p0 = 0; p0 < count; p0 += 16 * MF) {
            const uint16_t* h[MF];
            bool there[MF];
            int pair[MF];
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                there[m] = p0 + 16 * m + c < count;
                pair[m] = G.pair[first + min(p0 + 16 * m + c, count - 1)];
                h[m] = A.h + (int64_t)pair[m] * 2 * A.inner;
            }
            f32x4 acc[RF][MF] = {};
            for (int u = u0; u < u1; u += 4) {
                const int unit = u + g;
                const bool in = unit < u1;
                Weights<W> a[RF];
#pragma unroll
                for (int f = 0; f < RF; ++f) a[f].load(w[f], ws[f], unit, in, A.inner);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int k = unit * F::UNIT + s * F::VALUES;
                    u32x4 v[2][MF][F::OPS];
#pragma unroll
                    for (int m = 0; m < MF; ++m) {
#pragma unroll
                        for (int j = 0; j < F::OPS; ++j) v[0][m][j] = v[1][m][j] = u32x4{0, 0, 0, 0};
                        if (in && there[m] && k < A.inner) {
#pragma unroll
                            for (int j = 0; j < F::OPS; ++j) {
                                v[0][m][j] = *reinterpret_cast<const u32x4*>(h[m] + k + 8 * j);
                                v[1][m][j] = *reinterpret_cast<const u32x4*>(h[m] + A.inner + k + 8 * j);
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < F::OPS; ++j)
#pragma unroll
                        for (int f = 0; f < RF; ++f) {
                            const u32x4 wide = a[f].template operand<kBf16>(s, j);
#pragma unroll
                            for (int m = 0; m < MF; ++m) {
                                acc[f][m] = mfma_bf16(wide, v[0][m][j], acc[f][m]);
                                acc[f][m] = mfma_bf16(wide, v[1][m][j], acc[f][m]);
                            }
                        }
                }
            }
#pragma unroll
            for (int m = 0; m < MF; ++m)
                if (there[m]) {
#pragma unroll
                    for (int f = 0; f < RF; ++f) sums[(share * A.pairs + pair[m]) * 4 * RF + 4 * f + g] = acc[f][m] * factor;
                }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < A.tokens * 4 * RF; i += kThreads) {
        const int t = i / (4 * RF), q = i % (4 * RF), k = k0 + 4 * q;
        f32x4 y{0, 0, 0, 0};
        for (int j = 0; j < A.top; ++j) {
            const int pair = t * A.top + j, id = A.ids[pair];
            if (id < 0 || id >= A.experts) continue;
            f32x4 v = sums[pair * 4 * RF + q];
            for (int s = 1; s < shares; ++s) v += sums[(s * A.pairs + pair) * 4 * RF + q];
            y += v * A.weights[pair];
        }
        if (k < A.features) store4<TYPE>(A.y + t * A.ld_y + k, y, 4, A.vector);     // features: a multiple of 16
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

// A second kernel's rows of 16 features, and the room for its sums.
constexpr int kRows = 1;

template <int W, int TYPE, int MF>
int moe(const MoeArgs& A, hipStream_t st)
{
    const int most = A.pairs < A.experts ? A.pairs : A.experts;
    gate_up_kernel<W, TYPE, MF><<<dim3((A.inner + 15) / 16, most), kThreads, 0, st>>>(A);
    const int rc = launch_status();
    if (rc != ECF8_OK) return rc;
    down_kernel<W, TYPE, kRows, MF><<<(A.features + 16 * kRows - 1) / (16 * kRows), kThreads, A.slots * kRows * 64, st>>>(A);
    return launch_status();
}

template <int W, int TYPE>
int moe(const MoeArgs& A, hipStream_t st)
{
    // Columns of the matrix instructions: 16 where an expert meets few tokens.
    if (A.tokens <= 16 || A.pairs <= 8 * A.experts) return moe<W, TYPE, 1>(A, st);
    return moe<W, TYPE, 2>(A, st);
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
    return round_up(tokens * top * 4 * layer->inner, 256);
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
    if (ld_x < layer->features || ld_y < layer->features || ld_x > (1ull << 40) || ld_y > (1ull << 40)) return ECF8_ERR_SIZE;
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
    A.y = static_cast<uint16_t*>(y);
    A.ld_y = (int64_t)ld_y;
    A.tokens = (int)tokens;
    A.top = (int)top;
    A.pairs = (int)(tokens * top);
    A.features = (int)layer->features;
    A.inner = (int)layer->inner;
    A.experts = (int)layer->experts;
    A.slots = A.pairs * kWaves < kPairs ? A.pairs * kWaves : kPairs;
    A.vector = ld_y % 4 == 0 && aligned(y, 8);
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    if (mx) return type == ECF8A_BF16 ? moe<kMx4, kBf16>(A, st) : moe<kMx4, kFp16>(A, st);
    return type == ECF8A_BF16 ? moe<kE4m3, kBf16>(A, st) : moe<kE4m3, kFp16>(A, st);
}
