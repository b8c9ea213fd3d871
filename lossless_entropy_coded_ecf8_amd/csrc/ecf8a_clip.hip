// ecf8a_clip.hip -- the global norm of many gradients, and the gradients scaled
// to a largest norm.
//
// norm = sqrt(sum g^2) has to be known before the first scaled value is written,
// so there are two launches: one reads every gradient and leaves a partial sum
// per workgroup, the other adds those up (every workgroup the same few, in the
// same order) and scales.  Both are bound by memory.  The squares are summed in
// float64: one conversion and one fused multiply-add for each value, which the
// card does in a quarter of the time the value takes to arrive, and neither
// large gradients overflow nor the order of the sum is felt.
//
// The tensors are cut into pieces of one size on the host, so that hundreds of
// small ones and a few large ones load the card alike; the second launch takes
// the pieces in the opposite order and finds the last ones still in the cache.
#include "ecf8a_common.h"

#include <algorithm>
#include <new>

namespace {

using namespace ecf8a;

constexpr int kThreads = 256;
constexpr int kStep = 16 * kThreads;          // bytes a workgroup loads at once
constexpr int kFlight = 4;                    // 16-byte loads of a lane in flight
constexpr uint32_t kMaxGrid = 2048;

struct Piece {
    const void* grad;
    void* out;
    uint64_t n;
    uint64_t pad;
};

template <int TYPE>
struct Elem {
    typedef uint16_t type;
};
template <>
struct Elem<ECF8A_FP32> {
    typedef float type;
};

template <int TYPE>
__device__ __forceinline__ float value_of(typename Elem<TYPE>::type v)
{
    if constexpr (TYPE == ECF8A_FP32) return v;
    else return load1<TYPE>(&v);
}

template <int TYPE>
__device__ __forceinline__ typename Elem<TYPE>::type scaled(typename Elem<TYPE>::type v, float by)
{
    if constexpr (TYPE == ECF8A_FP32) return v * by;
    else return round1<TYPE>(value_of<TYPE>(v) * by);
}

template <int TYPE>
__device__ __forceinline__ double squares(u32x4 v)
{
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (TYPE == ECF8A_FP32) {
            const double d = __builtin_bit_cast(float, (uint32_t)v[i]);
            s = __builtin_fma(d, d, s);
        } else {
            const f32x2 p = unpack2<TYPE>(v[i]);
            const double a = p[0], b = p[1];
            s = __builtin_fma(a, a, s);
            s = __builtin_fma(b, b, s);
        }
    }
    return s;
}

// The values of a piece before its first 16-byte border.
template <int TYPE>
__device__ __forceinline__ uint64_t head_of(const Piece& p)
{
    constexpr uint64_t size = sizeof(typename Elem<TYPE>::type);
    const uint64_t h = ((16 - (reinterpret_cast<uintptr_t>(p.grad) & 15)) & 15) / size;
    return h < p.n ? h : p.n;
}

__device__ __forceinline__ double block_sum(double v, double* lds)
{
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return lds[0] + lds[1] + lds[2] + lds[3];
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void norm_kernel(const Piece* __restrict__ pieces, uint64_t count, double* partial)
{
    typedef typename Elem<TYPE>::type T;
    constexpr int per = 16 / sizeof(T);
    __shared__ double lds[4];
    double s = 0.0;
    for (uint64_t at = blockIdx.x; at < count; at += gridDim.x) {
        const Piece p = pieces[at];
        const T* g = static_cast<const T*>(p.grad);
        const uint64_t head = head_of<TYPE>(p), units = (p.n - head) / per, tail = head + units * per;
        const u32x4* body = reinterpret_cast<const u32x4*>(g + head);
        uint64_t u = threadIdx.x;
        for (; u + (kFlight - 1) * kThreads < units; u += kFlight * kThreads) {
            u32x4 v[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) v[i] = body[u + i * kThreads];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) s += squares<TYPE>(v[i]);
        }
        for (; u < units; u += kThreads) s += squares<TYPE>(body[u]);
        if (threadIdx.x < head) {
            const double d = value_of<TYPE>(g[threadIdx.x]);
            s += d * d;
        }
        if (tail + threadIdx.x < p.n) {
            const double d = value_of<TYPE>(g[tail + threadIdx.x]);
            s += d * d;
        }
    }
    s = block_sum(s, lds);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <int TYPE>
__global__ __launch_bounds__(kThreads) void scale_kernel(const Piece* __restrict__ pieces, uint64_t count,
                                                         const double* __restrict__ partial, int parts, float max_norm,
                                                         bool in_place, float* __restrict__ norm_out)
{
    typedef typename Elem<TYPE>::type T;
    constexpr int per = 16 / sizeof(T);
    __shared__ double lds[4];
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += partial[i];
    const double norm = __builtin_sqrt(block_sum(s, lds));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
    double c = (double)max_norm / (norm + 1e-6);
    c = c > 1.0 ? 1.0 : c;                                    // a NaN stays one
    const float by = (float)c;
    if (in_place && by == 1.0f) return;
    for (uint64_t i = blockIdx.x; i < count; i += gridDim.x) {
        const Piece p = pieces[count - 1 - i];
        const T* g = static_cast<const T*>(p.grad);
        T* o = static_cast<T*>(p.out);
        const uint64_t head = head_of<TYPE>(p), units = (p.n - head) / per, tail = head + units * per;
        const bool wide = (reinterpret_cast<uintptr_t>(o + head) & 15) == 0;
        const auto put = [&](uint64_t u, u32x4 v) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (TYPE == ECF8A_FP32) v[k] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, (uint32_t)v[k]) * by);
                else {
                    const f32x2 f = unpack2<TYPE>(v[k]);
                    v[k] = pack2<TYPE>(f[0] * by, f[1] * by);
                }
            }
            T* q = o + head + u * per;
            if (wide) store16<true>(q, v);
            else store16<false>(q, v);
        };
        const u32x4* body = reinterpret_cast<const u32x4*>(g + head);
        uint64_t u = threadIdx.x;
        for (; u + (kFlight - 1) * kThreads < units; u += kFlight * kThreads) {
            u32x4 v[kFlight];
#pragma unroll
            for (int i = 0; i < kFlight; ++i) v[i] = __builtin_nontemporal_load(body + u + i * kThreads);
#pragma unroll
            for (int i = 0; i < kFlight; ++i) put(u + i * kThreads, v[i]);
        }
        for (; u < units; u += kThreads) put(u, body[u]);
        if (threadIdx.x < head) o[threadIdx.x] = scaled<TYPE>(g[threadIdx.x], by);
        if (tail + threadIdx.x < p.n) o[tail + threadIdx.x] = scaled<TYPE>(g[tail + threadIdx.x], by);
    }
}

uint64_t elem_size(uint32_t type) { return type == ECF8A_FP32 ? 4 : 2; }

// Bytes of one piece: whole loads of a workgroup, about 2048 pieces in all.
uint64_t piece_bytes(uint64_t total)
{
    const uint64_t b = round_up(total / 2048, kStep);
    return b < kStep ? kStep : b > 16 * kStep ? 16 * kStep : b;
}

// Pieces of n values from `grad` on: the borders between them lie on 16 bytes
// if `grad` does to its element (the first piece is longer by what is before).
uint64_t pieces_of(uint64_t n, uint64_t per) { return (n + per - 1) / per; }

bool total_of(const ecf8a_grad* grads, uint32_t count, uint64_t* total)
{
    uint64_t t = 0;
    for (uint32_t i = 0; i < count; ++i) {
        if (grads[i].n > (1ull << 40) - t) return false;
        t += grads[i].n;
    }
    *total = t;
    return true;
}

}  // namespace

// The piece count does not depend on the type's size being known here: pieces
// are counted in values for the larger element, which gives the most pieces.
extern "C" uint64_t ecf8a_clip_bytes(const ecf8a_grad* grads, uint32_t count)
{
    uint64_t total = 0, most = 0;
    if (count && !grads) return 0;
    if (!total_of(grads, count, &total)) return 0;
    for (uint64_t size = 2; size <= 4; size += 2) {
        uint64_t pieces = 0;
        for (uint32_t i = 0; i < count; ++i) pieces += pieces_of(grads[i].n, piece_bytes(total * size) / size);
        if (pieces > most) most = pieces;
    }
    return round_up(8ull * kMaxGrid + sizeof(Piece) * most, 256);
}

extern "C" int ecf8a_clip_prepare(const ecf8a_grad* grads, uint32_t count, uint32_t type, void* workspace,
                                  uint64_t workspace_bytes, void* hip_stream, ecf8a_clip_plan* plan)
{
    if (!plan || (count && !grads)) return ECF8_ERR_ARG;
    if (type != ECF8A_BF16 && type != ECF8A_FP16 && type != ECF8A_FP32) return ECF8_ERR_UNSUPPORTED;
    const uint64_t size = elem_size(type);
    uint64_t total = 0;
    if (!total_of(grads, count, &total)) return ECF8_ERR_SIZE;
    const uint64_t need = ecf8a_clip_bytes(grads, count);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < need) return ECF8_ERR_WORKSPACE;
    const uint64_t per = piece_bytes(total * size) / size;
    uint64_t pieces = 0;
    bool in_place = true;
    for (uint32_t i = 0; i < count; ++i) {
        const ecf8a_grad& t = grads[i];
        if (t.n && (!t.grad || !t.out || !aligned(t.grad, size) || !aligned(t.out, size))) return ECF8_ERR_ARG;
        if (t.n && t.out != t.grad) in_place = false;
        pieces += pieces_of(t.n, per);
    }
    // Every range that is read or written, in order of address: none may reach
    // into the next, but for the two of a gradient in place.
    struct Range {
        uintptr_t at, end;
    };
    Range* ranges = new (std::nothrow) Range[2ull * count + 1];
    Piece* list = new (std::nothrow) Piece[pieces + 1];
    int rc = ranges && list ? ECF8_OK : ECF8_ERR_HIP;
    if (rc == ECF8_OK) {
        uint64_t m = 0, at = 0;
        for (uint32_t i = 0; i < count; ++i) {
            const ecf8a_grad& t = grads[i];
            if (!t.n) continue;
            const uintptr_t g = reinterpret_cast<uintptr_t>(t.grad), o = reinterpret_cast<uintptr_t>(t.out);
            ranges[m++] = Range{g, g + t.n * size};
            if (o != g) ranges[m++] = Range{o, o + t.n * size};
            // Borders between pieces on 16 bytes: the first piece takes the values before the first border as well.
            const uint64_t head = ((16 - (g & 15)) & 15) / size;
            for (uint64_t from = 0; from < t.n;) {
                uint64_t to = from == 0 ? per + (head < per ? head : 0) : from + per;
                if (to > t.n) to = t.n;
                list[at++] = Piece{static_cast<const char*>(t.grad) + from * size, static_cast<char*>(t.out) + from * size,
                                   to - from, 0};
                from = to;
            }
        }
        pieces = at;
        std::sort(ranges, ranges + m, [](const Range& a, const Range& b) { return a.at < b.at; });
        for (uint64_t i = 1; i < m; ++i)
            if (ranges[i].at < ranges[i - 1].end) rc = ECF8_ERR_ARG;
    }
    // A capture would record the copy with the address of this list, and every replay would read what lies there then.
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    if (rc == ECF8_OK && hipStreamIsCapturing(static_cast<hipStream_t>(hip_stream), &capture) != hipSuccess) {
        (void)hipGetLastError();
        rc = ECF8_ERR_HIP;
    }
    if (rc == ECF8_OK && capture != hipStreamCaptureStatusNone) rc = ECF8_ERR_ARG;
    if (rc == ECF8_OK && pieces &&
        hipMemcpyAsync(static_cast<char*>(workspace) + 8ull * kMaxGrid, list, sizeof(Piece) * pieces, hipMemcpyHostToDevice,
                       static_cast<hipStream_t>(hip_stream)) != hipSuccess)
        rc = ECF8_ERR_HIP;
    delete[] ranges;
    delete[] list;
    if (rc != ECF8_OK) return rc;
    const uint32_t grid = (uint32_t)std::min<uint64_t>(std::max<uint64_t>(pieces, 1), kMaxGrid);
    *plan = ecf8a_clip_plan{workspace, workspace_bytes, pieces, count, type, grid, in_place ? 1u : 0u};
    return ECF8_OK;
}

extern "C" int ecf8a_clip_run(const ecf8a_clip_plan* plan, float max_norm, float* norm, void* hip_stream)
{
    if (!plan || !plan->workspace || !norm || !aligned(norm, 4) || !(max_norm >= 0.0f) || plan->grid < 1 ||
        plan->grid > kMaxGrid)
        return ECF8_ERR_ARG;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    double* partial = static_cast<double*>(plan->workspace);
    const Piece* pieces = reinterpret_cast<const Piece*>(static_cast<char*>(plan->workspace) + 8ull * kMaxGrid);
#define ECF8A_CLIP(TYPE)                                                                                              \
    norm_kernel<TYPE><<<plan->grid, kThreads, 0, st>>>(pieces, plan->pieces, partial);                                \
    scale_kernel<TYPE><<<plan->grid, kThreads, 0, st>>>(pieces, plan->pieces, partial, (int)plan->grid, max_norm,     \
                                                        plan->in_place != 0, norm)
    if (plan->type == ECF8A_BF16) {
        ECF8A_CLIP(ECF8A_BF16);
    } else if (plan->type == ECF8A_FP16) {
        ECF8A_CLIP(ECF8A_FP16);
    } else if (plan->type == ECF8A_FP32) {
        ECF8A_CLIP(ECF8A_FP32);
    } else {
        return ECF8_ERR_ARG;
    }
#undef ECF8A_CLIP
    return launch_status();
}
