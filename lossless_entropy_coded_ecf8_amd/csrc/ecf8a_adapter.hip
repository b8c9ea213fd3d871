// ecf8a_adapter.hip -- low-rank adapters of many requests beside a shared
// projection, forward and backward.
//
// The mathematics needs three kernels besides the grouping, because both
// factors are stored by rank row:
//   low     Z[t][r] = c * sum_k V[t][k] F[a][r][k]   h from x and down; z from dy and up
//   wide    O[t][n] = B[t][n] + sum_r Z[t][r] F[a][r][n]   out from h and up; dx from z and down
//   factor  G[a][r][n] = sum_t Z[t][r] V[t][n]       d_down from z and x; d_up from h and dy
// With R far below K and N all three are bound by reading and writing the
// tokens' rows once (and, for single tokens, by reading the factors), so the
// matrix instructions only have to keep out of the way.
//
// Z stays in float32 between the kernels.  Where it is an operand of a matrix
// instruction it goes in as two bfloat16 (split8), which costs a second
// instruction on a unit that waits for memory anyway and keeps 16 bits of it;
// the float16 factors and rows go in as two bfloat16 as well (exact), since a
// float16 cannot hold Z's range.
//
// Tokens are taken in the plan's order: sorted by adapter, each group padded
// to 16 slots, cut into chunks of at most 64 slots that share one adapter.
#include "ecf8a_common.h"

namespace {

using namespace ecf8a;

constexpr int kTile = 16;                 // slots a group is padded to: one matrix instruction's rows
constexpr int kChunk = 64;                // slots of one chunk at most
constexpr int kPlanThreads = 1024;
constexpr int kPlanLds = 15 * 1024;       // ints of LDS for the grouping
constexpr int kThreads = 256;
constexpr int kStrip = 128;               // columns of one wave: 16 lanes of 8

// The plan's workspace: a header, then what each kernel reads of the grouping.
struct PlanView {
    int* head;           // [0] chunks, [1] slots, [2] units
    i32x4* chunks;       // adapter (adapters: none), first slot, tokens, 0
    i32x4* units;        // adapter, first slot, slots, 1 if the adapter's only unit
    int* unit_start;     // per adapter, and the end
    int* slot_token;     // token of each slot, -1: padding
};

__host__ __device__ inline uint64_t plan_offset_units(uint32_t max_chunks) { return 256 + 16ull * max_chunks; }
__host__ __device__ inline uint64_t plan_offset_start(uint32_t max_chunks, uint32_t max_units)
{
    return plan_offset_units(max_chunks) + 16ull * max_units;
}
__host__ __device__ inline uint64_t plan_offset_slots(uint32_t max_chunks, uint32_t max_units, uint32_t adapters)
{
    return (plan_offset_start(max_chunks, max_units) + 4ull * (adapters + 1) + 15) / 16 * 16;
}

PlanView view_of(const ecf8a_plan& p)
{
    char* w = static_cast<char*>(p.workspace);
    return PlanView{reinterpret_cast<int*>(w), reinterpret_cast<i32x4*>(w + 256),
                    reinterpret_cast<i32x4*>(w + plan_offset_units(p.max_chunks)),
                    reinterpret_cast<int*>(w + plan_offset_start(p.max_chunks, p.max_units)),
                    reinterpret_cast<int*>(w + plan_offset_slots(p.max_chunks, p.max_units, p.adapters))};
}

// ------------------------------------------------------------- grouping

__device__ __forceinline__ int read_index(const void* index, int bytes, int64_t t, int adapters)
{
    const int64_t a = bytes == 4 ? (int64_t)static_cast<const int32_t*>(index)[t] : static_cast<const int64_t*>(index)[t];
    return a >= 0 && a < adapters ? (int)a : adapters;
}

// Exclusive prefix over the workgroup of three values at once.
__device__ __forceinline__ void block_scan3(int v[3], int total[3], int (*lds)[3])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc[3] = {v[0], v[1], v[2]};
    for (int d = 1; d < 64; d <<= 1)
        for (int i = 0; i < 3; ++i) {
            const int o = __shfl_up(inc[i], d);
            if (lane >= d) inc[i] += o;
        }
    if (lane == 63)
        for (int i = 0; i < 3; ++i) lds[wave][i] = inc[i];
    __syncthreads();
    for (int i = 0; i < 3; ++i) {
        int before = 0, all = 0;
        for (int w = 0; w < kPlanThreads / 64; ++w) {
            if (w < wave) before += lds[w][i];
            all += lds[w][i];
        }
        v[i] = before + inc[i] - v[i];
        total[i] = all;
    }
}

// Stable counting sort of the tokens by adapter, in one workgroup.  Each of
// `waves` waves owns a run of consecutive tokens and counts its own adapters
// (LDS atomics, whose order does not change a count); the prefix over adapters
// and waves gives each wave its first slot in every group, and it then places
// its tokens 64 at a time, each behind those before it.  So slots depend on the
// index alone, and every sum over a group has a fixed order.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const void* __restrict__ index, int index_bytes, int tokens,
                                                            int adapters, int waves, int unit_slots, int max_chunks,
                                                            PlanView p)
{
    __shared__ int lds[kPlanLds];
    __shared__ int scan[kPlanThreads / 64][3];
    const int groups = adapters + 1;                        // the last: no adapter
    int* const hist = lds;                                  // [waves][groups]: next slot of each wave in each group
    int* const count = lds + waves * groups;                // [groups]
    int* const chunk0 = count + groups;                     // [groups]
    int* const slot0 = chunk0 + groups;                     // [groups]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < waves * groups; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
    const int run = ((tokens + waves - 1) / waves + 63) / 64 * 64;
    const int t0 = min(tokens, wave * run), t1 = wave < waves ? min(tokens, t0 + run) : t0;
    for (int t = t0 + lane; t < t1; t += 64) atomicAdd(&hist[wave * groups + read_index(index, index_bytes, t, adapters)], 1);
    __syncthreads();
    // Per thread a run of groups, so that one scan over threads covers all.
    const int per = (groups + kPlanThreads - 1) / kPlanThreads;
    const int a0 = min(groups, tid * per), a1 = min(groups, a0 + per);
    int v[3] = {0, 0, 0}, total[3];
    for (int a = a0; a < a1; ++a) {
        int c = 0;
        for (int w = 0; w < waves; ++w) {
            const int h = hist[w * groups + a];
            hist[w * groups + a] = c;
            c += h;
        }
        count[a] = c;
        const int s = (c + kTile - 1) / kTile * kTile;
        v[0] += s;
        v[1] += (c + kChunk - 1) / kChunk;
        v[2] += a < adapters ? (s + unit_slots - 1) / unit_slots : 0;
    }
    block_scan3(v, total, scan);
    for (int a = a0; a < a1; ++a) {
        const int c = count[a], s = (c + kTile - 1) / kTile * kTile;
        slot0[a] = v[0];
        chunk0[a] = v[1];
        for (int w = 0; w < waves; ++w) hist[w * groups + a] += v[0];
        for (int i = c; i < s; ++i) p.slot_token[v[0] + i] = -1;
        if (a < adapters) {
            const int units = (s + unit_slots - 1) / unit_slots;
            p.unit_start[a] = v[2];
            for (int u = 0; u < units; ++u)
                p.units[v[2] + u] = i32x4{a, v[0] + u * unit_slots, min(unit_slots, s - u * unit_slots), units == 1};
            v[2] += units;
        }
        v[0] += s;
        v[1] += (c + kChunk - 1) / kChunk;
    }
    if (tid == 0) {
        p.head[0] = total[1];
        p.head[1] = total[0];
        p.head[2] = total[2];
        p.unit_start[adapters] = total[2];
    }
    __syncthreads();
    for (int c = tid; c < total[1]; c += kPlanThreads) {     // the last group whose first chunk is at or before c
        int lo = 0, hi = groups - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (chunk0[mid] <= c) lo = mid;
            else hi = mid - 1;
        }
        const int at = (c - chunk0[lo]) * kChunk;
        p.chunks[c] = i32x4{lo, slot0[lo] + at, min(kChunk, count[lo] - at), 0};
    }
    for (int tb = t0; tb < t1; tb += 64) {
        const int t = tb + lane;
        const int a = t < t1 ? read_index(index, index_bytes, t, adapters) : -1;
        const int first = __builtin_amdgcn_readfirstlane(a);
        int rank = 0, same = 0;
        if (__ballot(a == first || a < 0) == ~0ull) {        // one request's tokens: the usual case of a prompt
            rank = lane;
            same = (int)__popcll(__ballot(a >= 0));
        } else {
#pragma unroll
            for (int j = 0; j < 64; ++j) {
                const int o = __builtin_amdgcn_readlane(a, j);
                same += o == a;
                rank += o == a && j < lane;
            }
        }
        if (a >= 0) {
            volatile int* next = &hist[wave * groups + a];
            const int at = *next;
            p.slot_token[at + rank] = t;
            if (rank == same - 1) *next = at + same;          // one lane of each adapter, after every lane's read
        }
    }
}

// ------------------------------------------------------------- low: Z = c V F^T

// Sixteen consecutive values of a row from k on, as the operands of two matrix
// instructions.  VEC: 16-byte loads; values at or past `limit` are 0.
template <int TYPE, int VT, bool VEC, bool TAIL>
__device__ __forceinline__ void load_row16(const void* row, int k, int limit, u32x4 v[2])
{
    if constexpr (VT == kE4m3) {
        const uint8_t* p = static_cast<const uint8_t*>(row) + k;
        u32x4 b{0, 0, 0, 0};
        if constexpr (VEC) {
            if (!TAIL || k < limit) b = *reinterpret_cast<const u32x4*>(p);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (k + i < limit) b[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == kBf16) {
                v[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b[i], 1.0f, false));
                v[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b[i], 1.0f, true));
            } else {
                v[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b[i], 1.0f, false));
                v[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b[i], 1.0f, true));
            }
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(row) + k;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (VEC) {
                if (!TAIL || k + 8 * h < limit) v[h] = *reinterpret_cast<const u32x4*>(p + 8 * h);
                else v[h] = u32x4{0, 0, 0, 0};
            } else {
                v[h] = u32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + 8 * h + i < limit) v[h][i >> 1] |= (uint32_t)p[8 * h + i] << (16 * (i & 1));
            }
        }
    }
}

struct LowArgs {
    PlanView plan;
    const void* v;           // tokens' rows
    int64_t ldv;
    const uint16_t* f;       // factor (adapters, rank, width)
    const float* scaling;
    const int32_t* ranks;
    const float* v_scale;
    float* z;                // [plane][max_slots][zr]
    int64_t plane;           // floats of one plane
    int width, rank, zr, adapters;
};

// One workgroup: one chunk, 16 RT rank rows, one of gridDim.y shares of the
// width.  Its four waves take 64-column blocks in turn, so that a wave's two
// loads of a row cover whole 128-byte lines, and meet in LDS.
template <int TYPE, int VT, int RT, int NT, bool VEC>
__device__ __forceinline__ void low_body(const LowArgs& A, const i32x4 chunk, f32x4* red)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int a = chunk[0], r0 = blockIdx.z * 64;
    const int rank = A.ranks ? min(max(A.ranks[a], 0), A.rank) : A.rank;
    const void* vrow[NT];
    bool real[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {                          // padding reads row 0; its result is set to 0 below
        const int t = n * kTile < chunk[2] ? A.plan.slot_token[chunk[1] + n * kTile + c] : -1;
        real[n] = t >= 0;
        vrow[n] = static_cast<const char*>(A.v) + (VT == kE4m3 ? 1 : 2) * (int64_t)max(t, 0) * A.ldv;
    }
    const uint16_t* frow[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
        frow[r] = A.f + ((int64_t)a * A.rank + max(0, min(r0 + r * 16 + c, rank - 1))) * A.width;
    f32x4 acc[RT][NT] = {};
    const int blocks = (A.width + 63) / 64, whole = A.width / 64;
    for (int b = blockIdx.y * 4 + wave; b < blocks; b += gridDim.y * 4) {
        const int k = b * 64 + 16 * g;
        u32x4 fv[RT][2], vv[NT][2];
        if (b < whole) {
#pragma unroll
            for (int n = 0; n < NT; ++n) load_row16<TYPE, VT, VEC, false>(vrow[n], k, A.width, vv[n]);
#pragma unroll
            for (int r = 0; r < RT; ++r) load_row16<TYPE, TYPE, VEC, false>(frow[r], k, A.width, fv[r]);
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) load_row16<TYPE, VT, VEC, true>(vrow[n], k, A.width, vv[n]);
#pragma unroll
            for (int r = 0; r < RT; ++r) load_row16<TYPE, TYPE, VEC, true>(frow[r], k, A.width, fv[r]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[r][n] = mfma<TYPE>(fv[r][h], vv[n][h], acc[r][n]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) red[(wave * RT * NT + r * NT + n) * 64 + lane] = acc[r][n];
    __syncthreads();
    float scale = A.scaling[a];
    if (A.v_scale) scale *= *A.v_scale;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if ((r * NT + n) % 4 != wave || n * kTile >= chunk[2]) continue;   // tiles past the chunk are another's
            f32x4 s = red[(r * NT + n) * 64 + lane];
            for (int w = 1; w < 4; ++w) s += red[(w * RT * NT + r * NT + n) * 64 + lane];
            const int row = r0 + r * 16 + 4 * g;
            if (row >= A.zr) continue;
            f32x4 o;
            for (int i = 0; i < 4; ++i) o[i] = real[n] && row + i < rank ? s[i] * scale : 0.0f;
            float* z = A.z + blockIdx.y * A.plane + (int64_t)(chunk[1] + n * kTile + c) * A.zr + row;
            *reinterpret_cast<f32x4*>(z) = o;
        }
}

template <int TYPE, int VT, int RT, bool VEC>
__global__ __launch_bounds__(kThreads) void low_kernel(LowArgs A)
{
    __shared__ f32x4 red[4 * RT * 4 * 64];
    if ((int)blockIdx.x >= A.plan.head[0]) return;
    const i32x4 chunk = A.plan.chunks[blockIdx.x];
    if (chunk[0] >= A.adapters) return;
    if (chunk[2] <= 16) low_body<TYPE, VT, RT, 1, VEC>(A, chunk, red);
    else if (chunk[2] <= 32) low_body<TYPE, VT, RT, 2, VEC>(A, chunk, red);
    else low_body<TYPE, VT, RT, 4, VEC>(A, chunk, red);
}

// Sums the planes of a split width, in plane order.
__global__ __launch_bounds__(kThreads) void join_kernel(const float* __restrict__ planes, int64_t plane, int count,
                                                        const int* __restrict__ head, int zr, float* __restrict__ z)
{
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (i >= (int64_t)head[1] * zr) return;
    f32x4 s = *reinterpret_cast<const f32x4*>(planes + i);
    for (int p = 1; p < count; ++p) s += *reinterpret_cast<const f32x4*>(planes + p * plane + i);
    *reinterpret_cast<f32x4*>(z + i) = s;
}

// ------------------------------------------------------------- wide: O = B + Z F

struct WideArgs {
    PlanView plan;
    const float* z;
    const uint16_t* f;
    const int32_t* ranks;
    const uint16_t* base;
    int64_t ld_base;
    uint16_t* out;
    int64_t ld_out;
    int width, rank, zr, adapters;
    int groups;              // workgroups across the width
};

// Rows r .. r + 7 of the factor at this lane's eight columns, turned into one
// operand per column.  Rows that take no part are 0, whatever is stored there.
template <int TYPE, bool VEC>
__device__ __forceinline__ void load_factor(const uint16_t* f, int width, int r, int rank, int col, u32x4 hi[8], u32x4 lo[8])
{
    u32x4 w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        w[q] = u32x4{0, 0, 0, 0};
        if (r + q < rank) {
            const uint16_t* p = f + (int64_t)(r + q) * width + col;
            if constexpr (VEC) {
                if (col < width) w[q] = *reinterpret_cast<const u32x4*>(p);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < width) w[q][j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
            }
        }
    }
    transpose8(w, hi);
    if constexpr (TYPE == kFp16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) split8_f16(hi[j], hi[j], lo[j]);
    }
}

// One wave: 128 columns of one chunk.  A lane's eight columns are consecutive
// (column 8c + j goes to the j-th instruction), so that the factor's rows are
// read, and the result's rows read and written, 16 bytes at a time, and no LDS
// is used.  RB: blocks of 32 rank rows kept in registers for the whole chunk
// (0: up to 16 rows, the upper half of the slots taking lo; -1: any number,
// read again for each 16 tokens).
template <int TYPE, int RB, bool VEC>
__global__ __launch_bounds__(kThreads) void wide_kernel(WideArgs A)
{
    const int id = blockIdx.x / A.groups;                   // neighbouring workgroups: the same rows, next columns
    if (id >= A.plan.head[0]) return;
    const i32x4 chunk = A.plan.chunks[id];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int a = chunk[0], col = ((blockIdx.x - id * A.groups) * 4 + wave) * kStrip + 8 * c;
    if (col - 8 * c >= A.width) return;
    const bool bare = a >= A.adapters;
    if (bare && A.base == A.out) return;
    const int rank = bare ? 0 : A.ranks ? min(max(A.ranks[a], 0), A.rank) : A.rank;
    const uint16_t* f = A.f + (int64_t)(bare ? 0 : a) * A.rank * A.width;
    constexpr int KEEP = RB <= 0 ? 1 : RB;
    u32x4 hi[KEEP][8], lo[KEEP][8];
    if constexpr (RB == 0) load_factor<TYPE, VEC>(f, A.width, 8 * (g & 1), rank, col, hi[0], lo[0]);
    if constexpr (RB > 0) {
#pragma unroll
        for (int b = 0; b < KEEP; ++b) load_factor<TYPE, VEC>(f, A.width, 32 * b + 8 * g, rank, col, hi[b], lo[b]);
    }
    const int tiles = (chunk[2] + kTile - 1) / kTile;
    for (int tile = 0; tile < tiles; ++tile) {
        const int slot = chunk[1] + tile * kTile;
        const i32x4 tok = *reinterpret_cast<const i32x4*>(A.plan.slot_token + slot + 4 * g);
        u32x4 base[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            base[i] = u32x4{0, 0, 0, 0};
            if (!A.base || tok[i] < 0) continue;
            const uint16_t* p = A.base + tok[i] * A.ld_base + col;
            if constexpr (VEC) {
                if (col < A.width) base[i] = *reinterpret_cast<const u32x4*>(p);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < A.width) base[i][j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
            }
        }
        f32x4 acc[8] = {};
        if (!bare) {
            const float* z = A.z + (int64_t)(slot + c) * A.zr;
            if constexpr (RB == 0) {
                u32x4 zh, zl;
                const float* p = z + 8 * (g & 1);
                split8(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4), zh, zl);
                const u32x4 both = g < 2 ? zh : zl;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    acc[j] = mfma_bf16(both, hi[0][j], acc[j]);
                    if constexpr (TYPE == kFp16) acc[j] = mfma_bf16(both, lo[0][j], acc[j]);
                }
            } else {
                const int blocks = RB > 0 ? RB : (A.zr + 31) / 32;
                for (int b = 0; b < blocks; ++b) {
                    const int at = RB > 0 ? b : 0;
                    if constexpr (RB < 0) load_factor<TYPE, VEC>(f, A.width, 32 * b + 8 * g, rank, col, hi[0], lo[0]);
                    u32x4 zh, zl;
                    const float* p = z + 32 * b + 8 * g;
                    split8(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4), zh, zl);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        acc[j] = mfma_bf16(zh, hi[at][j], acc[j]);
                        acc[j] = mfma_bf16(zl, hi[at][j], acc[j]);
                        if constexpr (TYPE == kFp16) acc[j] = mfma_bf16(zh, lo[at][j], acc[j]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (tok[i] < 0) continue;
            u32x4 o;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const f32x2 b = unpack2<TYPE>(base[i][j]);
                o[j] = bare ? base[i][j] : pack2<TYPE>(b[0] + acc[2 * j][i], b[1] + acc[2 * j + 1][i]);
            }
            uint16_t* p = A.out + tok[i] * A.ld_out + col;
            if constexpr (VEC) {
                if (col < A.width) *reinterpret_cast<u32x4*>(p) = o;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j < A.width) p[j] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
            }
        }
    }
}

// ------------------------------------------------------------- factor: G = Z^T V

struct FactorArgs {
    PlanView plan;
    const float* z;
    const uint16_t* v;
    int64_t ldv;
    const int32_t* ranks;
    uint16_t* grad;          // (adapters, rank, width)
    float* part;             // [unit][zr][stride]
    int width, stride, rank, zr, adapters;
};

// One workgroup: one unit of one adapter's slots, 128 columns, 16 RT rank rows.
// Its four waves take 32 slots in turn; a lane reads eight tokens' 16 bytes and
// turns them, as load_factor does, so that the sum over tokens runs in the
// matrix instructions' reduction slots.  An adapter of one unit is written at
// once, others leave float32 partial sums that sum_kernel joins in order.
template <int TYPE, int RT, bool VEC>
__global__ __launch_bounds__(kThreads) void factor_kernel(FactorArgs A)
{
    __shared__ f32x4 red[2 * RT * 8 * 64];
    if ((int)blockIdx.y >= A.plan.head[2]) return;
    const i32x4 unit = A.plan.units[blockIdx.y];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int col = blockIdx.x * kStrip + 8 * c, r0 = blockIdx.z * 64;
    const bool inside = col < A.width;
    const int safe = inside ? col : 0;
    f32x4 acc[RT][8] = {};
    for (int s = wave * 32; s < unit[2]; s += 128) {
        const int slot = unit[1] + s + 8 * g;
        const bool have = s + 8 * g < unit[2];                // units are whole tiles of 16: eight slots are in or out
        i32x4 tok[2] = {{-1, -1, -1, -1}, {-1, -1, -1, -1}};
        if (have) {
            tok[0] = *reinterpret_cast<const i32x4*>(A.plan.slot_token + slot);
            tok[1] = *reinterpret_cast<const i32x4*>(A.plan.slot_token + slot + 4);
        }
        u32x4 w[8], t[8], tl[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int tq = tok[q >> 2][q & 3];
            w[q] = u32x4{0, 0, 0, 0};
            if (tq >= 0) {
                const uint16_t* p = A.v + tq * A.ldv + safe;
                if constexpr (VEC) w[q] = *reinterpret_cast<const u32x4*>(p);
                else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col + j < A.width) w[q][j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
                }
            }
        }
        u32x4 zh[RT], zl[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int row = r0 + r * 16 + c;
            f32x4 lo4{0, 0, 0, 0}, hi4{0, 0, 0, 0};
            if (have && row < A.zr) {
                const float* z = A.z + (int64_t)slot * A.zr + row;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    lo4[q] = z[q * A.zr];
                    hi4[q] = z[(q + 4) * A.zr];
                }
            }
            split8(lo4, hi4, zh[r], zl[r]);
        }
        transpose8(w, t);
        if constexpr (TYPE == kFp16) {
#pragma unroll
            for (int j = 0; j < 8; ++j) split8_f16(t[j], t[j], tl[j]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc[r][j] = mfma_bf16(zh[r], t[j], acc[r][j]);
                acc[r][j] = mfma_bf16(zl[r], t[j], acc[r][j]);
                if constexpr (TYPE == kFp16) acc[r][j] = mfma_bf16(zh[r], tl[j], acc[r][j]);
            }
    }
    // Waves 2 and 3 hand over to 0 and 1, and 1 to 0.
    for (int half = 2; half >= 1; half >>= 1) {
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j) red[(((wave - half) * RT + r) * 8 + j) * 64 + lane] = acc[r][j];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[r][j] += red[((wave * RT + r) * 8 + j) * 64 + lane];
        __syncthreads();
    }
    if (wave != 0 || !inside) return;
    const int a = unit[0];
    const int rank = A.ranks ? min(max(A.ranks[a], 0), A.rank) : A.rank;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = r0 + r * 16 + 4 * g + i;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = row < rank ? acc[r][j][i] : 0.0f;
            if (unit[3]) {
                if (row >= A.rank) continue;
                uint16_t* p = A.grad + ((int64_t)a * A.rank + row) * A.width + col;
                if constexpr (VEC)
                    *reinterpret_cast<u32x4*>(p) = u32x4{pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3]),
                                                         pack2<TYPE>(v[4], v[5]), pack2<TYPE>(v[6], v[7])};
                else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (col + j < A.width) p[j] = round1<TYPE>(v[j]);
                }
            } else if (row < A.zr) {
                float* p = A.part + ((int64_t)blockIdx.y * A.zr + row) * A.stride + col;
                *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
}

// The gradients of adapters with no unit (0) or several (their partial sums).
template <int TYPE>
__global__ __launch_bounds__(kThreads) void sum_kernel(FactorArgs A)
{
    const int a = blockIdx.z, row = blockIdx.y;
    const int u0 = A.plan.unit_start[a], u1 = A.plan.unit_start[a + 1];
    if (u1 - u0 == 1) return;
    for (int col = blockIdx.x * kThreads + threadIdx.x; col < A.width; col += gridDim.x * kThreads) {
        float s = 0.0f;
        for (int u = u0; u < u1; ++u) s += A.part[((int64_t)u * A.zr + row) * A.stride + col];
        A.grad[((int64_t)a * A.rank + row) * A.width + col] = round1<TYPE>(s);
    }
}

// ------------------------------------------------------------- host side

uint32_t z_rows(uint32_t rank) { return rank <= 16 ? 16 : (uint32_t)round_up(rank, 32); }

// Shares of the width that a `low` call is cut into: enough workgroups for the
// card from few chunks, each wave keeping at least one block of 64 columns.
uint32_t shares_of(const ecf8a_plan& p, uint64_t width)
{
    const uint64_t chunks = p.tokens / kChunk + (p.adapters < p.tokens ? p.adapters : p.tokens);
    uint64_t s = chunks ? 1024 / chunks : 1;
    const uint64_t most = (width + 255) / 256;
    if (s > most) s = most;
    return (uint32_t)(s < 1 ? 1 : s > 16 ? 16 : s);
}

uint64_t z_bytes(const ecf8a_plan& p, uint32_t rank) { return round_up(4ull * p.max_slots * z_rows(rank), 256); }

uint64_t low_bytes(const ecf8a_plan& p, uint32_t rank, uint64_t width)
{
    const uint64_t s = shares_of(p, width);
    return s > 1 ? s * z_bytes(p, rank) : 0;
}

uint64_t part_bytes(const ecf8a_plan& p, uint32_t rank, uint64_t width)
{
    return round_up(4ull * p.max_units * z_rows(rank) * round_up(width, kStrip), 256);
}

bool plan_ok(const ecf8a_plan* p)
{
    return p && p->tokens <= ECF8A_MAX_TOKENS && p->adapters >= 1 && p->adapters <= ECF8A_MAX_ADAPTERS;
}

int check_bank(const ecf8a_plan* plan, const ecf8a_bank* b)
{
    if (!plan_ok(plan) || !b) return ECF8_ERR_ARG;
    if (b->type != ECF8A_BF16 && b->type != ECF8A_FP16) return ECF8_ERR_UNSUPPORTED;
    if (b->adapters != plan->adapters) return ECF8_ERR_ARG;
    if (b->rank < 1 || b->rank > ECF8A_MAX_RANK || b->in_features < 1 || b->in_features > ECF8A_MAX_FEATURES ||
        b->out_features < 1 || b->out_features > ECF8A_MAX_FEATURES)
        return ECF8_ERR_SIZE;
    if (!b->down || !b->up || !b->scaling || !aligned(b->down, 2) || !aligned(b->up, 2) || !aligned(b->scaling, 4) ||
        !aligned(b->ranks, 4))
        return ECF8_ERR_ARG;
    return ECF8_OK;
}

bool vec16(const void* p, uint64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

template <int TYPE, int VT, bool VEC>
void launch_low(const LowArgs& A, dim3 grid, hipStream_t st)
{
    if (A.zr <= 16) low_kernel<TYPE, VT, 1, VEC><<<grid, kThreads, 0, st>>>(A);
    else if (A.zr <= 32) low_kernel<TYPE, VT, 2, VEC><<<grid, kThreads, 0, st>>>(A);
    else low_kernel<TYPE, VT, 4, VEC><<<grid, kThreads, 0, st>>>(A);
}

// Z of one side into `z`; `planes` holds the shares of a split width.
int run_low(const ecf8a_plan& p, const ecf8a_bank& b, const void* v, uint64_t ldv, uint32_t vt, const float* v_scale,
            const void* f, uint64_t width, float* z, float* planes, hipStream_t st)
{
    const uint32_t shares = shares_of(p, width);
    LowArgs A{view_of(p), v, (int64_t)ldv, static_cast<const uint16_t*>(f), b.scaling, b.ranks, v_scale,
              shares > 1 ? planes : z, (int64_t)(z_bytes(p, b.rank) / 4), (int)width, (int)b.rank, (int)z_rows(b.rank),
              (int)b.adapters};
    const dim3 grid(p.max_chunks, shares, (A.zr + 63) / 64);
    const bool e4m3 = vt == ECF8A_E4M3;
    const bool vec = e4m3 ? aligned(v, 16) && ldv % 16 == 0 && width % 16 == 0 && aligned(f, 16)
                          : vec16(v, ldv) && vec16(f, width);
    if (b.type == ECF8A_BF16) {
        if (e4m3) vec ? launch_low<kBf16, kE4m3, true>(A, grid, st) : launch_low<kBf16, kE4m3, false>(A, grid, st);
        else vec ? launch_low<kBf16, kBf16, true>(A, grid, st) : launch_low<kBf16, kBf16, false>(A, grid, st);
    } else {
        if (e4m3) vec ? launch_low<kFp16, kE4m3, true>(A, grid, st) : launch_low<kFp16, kE4m3, false>(A, grid, st);
        else vec ? launch_low<kFp16, kFp16, true>(A, grid, st) : launch_low<kFp16, kFp16, false>(A, grid, st);
    }
    if (shares > 1) {
        const uint64_t quads = (uint64_t)p.max_slots * A.zr / 4;
        join_kernel<<<dim3((uint32_t)((quads + kThreads - 1) / kThreads)), kThreads, 0, st>>>(
            planes, A.plane, (int)shares, A.plan.head, A.zr, z);
    }
    return launch_status();
}

template <int TYPE, bool VEC>
void launch_wide(const WideArgs& A, dim3 grid, hipStream_t st)
{
    if (A.zr <= 16) wide_kernel<TYPE, 0, VEC><<<grid, kThreads, 0, st>>>(A);
    else if (A.zr <= 32) wide_kernel<TYPE, 1, VEC><<<grid, kThreads, 0, st>>>(A);
    else if (A.zr <= 64) wide_kernel<TYPE, 2, VEC><<<grid, kThreads, 0, st>>>(A);
    else wide_kernel<TYPE, -1, VEC><<<grid, kThreads, 0, st>>>(A);
}

int run_wide(const ecf8a_plan& p, const ecf8a_bank& b, const float* z, const void* f, uint64_t width, const void* base,
             uint64_t ld_base, void* out, uint64_t ld_out, hipStream_t st)
{
    WideArgs A{view_of(p), z, static_cast<const uint16_t*>(f), b.ranks, static_cast<const uint16_t*>(base),
               (int64_t)ld_base, static_cast<uint16_t*>(out), (int64_t)ld_out, (int)width, (int)b.rank,
               (int)z_rows(b.rank), (int)b.adapters, (int)((width + 4 * kStrip - 1) / (4 * kStrip))};
    const dim3 grid((uint32_t)A.groups * p.max_chunks);
    const bool vec = vec16(f, width) && vec16(out, ld_out) && (!base || vec16(base, ld_base));
    if (b.type == ECF8A_BF16) vec ? launch_wide<kBf16, true>(A, grid, st) : launch_wide<kBf16, false>(A, grid, st);
    else vec ? launch_wide<kFp16, true>(A, grid, st) : launch_wide<kFp16, false>(A, grid, st);
    return launch_status();
}

template <int TYPE, bool VEC>
void launch_factor(const FactorArgs& A, dim3 grid, hipStream_t st)
{
    if (A.zr <= 16) factor_kernel<TYPE, 1, VEC><<<grid, kThreads, 0, st>>>(A);
    else if (A.zr <= 32) factor_kernel<TYPE, 2, VEC><<<grid, kThreads, 0, st>>>(A);
    else factor_kernel<TYPE, 4, VEC><<<grid, kThreads, 0, st>>>(A);
}

int run_factor(const ecf8a_plan& p, const ecf8a_bank& b, const float* z, const void* v, uint64_t ldv, uint64_t width,
               void* grad, float* part, hipStream_t st)
{
    const uint64_t stride = round_up(width, kStrip);
    FactorArgs A{view_of(p), z, static_cast<const uint16_t*>(v), (int64_t)ldv, b.ranks, static_cast<uint16_t*>(grad),
                 part, (int)width, (int)stride, (int)b.rank, (int)z_rows(b.rank), (int)b.adapters};
    const bool vec = vec16(v, ldv) && vec16(grad, width);
    if (p.tokens) {
        const dim3 grid((uint32_t)(stride / kStrip), p.max_units, (A.zr + 63) / 64);
        if (b.type == ECF8A_BF16) vec ? launch_factor<kBf16, true>(A, grid, st) : launch_factor<kBf16, false>(A, grid, st);
        else vec ? launch_factor<kFp16, true>(A, grid, st) : launch_factor<kFp16, false>(A, grid, st);
    }
    const dim3 grid((uint32_t)((width + kThreads - 1) / kThreads), b.rank, b.adapters);
    if (b.type == ECF8A_BF16) sum_kernel<kBf16><<<grid, kThreads, 0, st>>>(A);
    else sum_kernel<kFp16><<<grid, kThreads, 0, st>>>(A);
    return launch_status();
}

bool sizes_ok(uint64_t tokens, uint32_t adapters)
{
    return tokens <= ECF8A_MAX_TOKENS && adapters >= 1 && adapters <= ECF8A_MAX_ADAPTERS;
}

// Bounds that hold for any index: a group is padded by at most 15 slots, and
// ends in at most one chunk and one unit that is not full.
void plan_sizes(uint64_t tokens, uint32_t adapters, ecf8a_plan* p)
{
    const uint64_t bare = adapters + 1ull < tokens ? adapters + 1ull : tokens;    // groups that can hold a token
    const uint64_t used = adapters < tokens ? adapters : tokens;
    const uint64_t unit = round_up((tokens + 15) / 16, 64);
    p->tokens = tokens;
    p->adapters = adapters;
    p->unit_slots = (uint32_t)(unit < 256 ? 256 : unit);
    p->max_slots = (uint32_t)((tokens + 15 * bare) / kTile * kTile);
    p->max_chunks = (uint32_t)(tokens / kChunk + bare);
    p->max_units = (uint32_t)(tokens / p->unit_slots + used);
}

}  // namespace

extern "C" uint64_t ecf8a_plan_bytes(uint64_t tokens, uint32_t adapters)
{
    if (!sizes_ok(tokens, adapters)) return 0;
    ecf8a_plan p{};
    plan_sizes(tokens, adapters, &p);
    return round_up(plan_offset_slots(p.max_chunks, p.max_units, adapters) + 4ull * p.max_slots, 256);
}

extern "C" int ecf8a_plan_prepare(const void* index, uint32_t index_bytes, uint64_t tokens, uint32_t adapters,
                                  void* workspace, uint64_t workspace_bytes, void* hip_stream, ecf8a_plan* plan)
{
    if (!plan || (index_bytes != 4 && index_bytes != 8) || (tokens && !index) || !aligned(index, index_bytes))
        return ECF8_ERR_ARG;
    if (!sizes_ok(tokens, adapters)) return ECF8_ERR_SIZE;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < ecf8a_plan_bytes(tokens, adapters))
        return ECF8_ERR_WORKSPACE;
    ecf8a_plan p{};
    plan_sizes(tokens, adapters, &p);
    p.workspace = workspace;
    p.workspace_bytes = workspace_bytes;
    const int groups = (int)adapters + 1;
    int waves = kPlanLds / groups - 3;
    if (waves > kPlanThreads / 64) waves = kPlanThreads / 64;
    if (waves < 1) return ECF8_ERR_SIZE;
    plan_kernel<<<1, kPlanThreads, 0, static_cast<hipStream_t>(hip_stream)>>>(
        index, (int)index_bytes, (int)tokens, (int)adapters, waves, (int)p.unit_slots, (int)p.max_chunks, view_of(p));
    const int rc = launch_status();
    if (rc == ECF8_OK) *plan = p;
    return rc;
}

extern "C" uint64_t ecf8a_hidden_bytes(const ecf8a_plan* plan, uint32_t rank)
{
    if (!plan_ok(plan) || rank < 1 || rank > ECF8A_MAX_RANK) return 0;
    return z_bytes(*plan, rank);
}

extern "C" uint64_t ecf8a_add_bytes(const ecf8a_plan* plan, const ecf8a_bank* b)
{
    if (!plan_ok(plan) || !b || b->rank < 1 || b->rank > ECF8A_MAX_RANK) return 0;
    return z_bytes(*plan, b->rank) + low_bytes(*plan, b->rank, b->in_features) + 256;
}

extern "C" uint64_t ecf8a_grads_bytes(const ecf8a_plan* plan, const ecf8a_bank* b)
{
    if (!plan_ok(plan) || !b || b->rank < 1 || b->rank > ECF8A_MAX_RANK) return 0;
    const uint64_t lk = low_bytes(*plan, b->rank, b->in_features), ln = low_bytes(*plan, b->rank, b->out_features);
    const uint64_t pk = part_bytes(*plan, b->rank, b->in_features), pn = part_bytes(*plan, b->rank, b->out_features);
    uint64_t most = lk > ln ? lk : ln;
    if (pk > most) most = pk;
    if (pn > most) most = pn;
    return 2 * z_bytes(*plan, b->rank) + most + 256;
}

extern "C" int ecf8a_add(const ecf8a_plan* plan, const ecf8a_bank* bank, const void* x, uint64_t ldx, uint32_t x_type,
                         const float* x_scale, const void* base, uint64_t ld_base, void* out, uint64_t ld_out,
                         void* hidden, void* workspace, uint64_t workspace_bytes, void* hip_stream)
{
    const int rc = check_bank(plan, bank);
    if (rc != ECF8_OK) return rc;
    if (x_type != bank->type && x_type != ECF8A_E4M3) return ECF8_ERR_UNSUPPORTED;
    if (plan->tokens == 0) return ECF8_OK;
    if (!x || !out || !aligned(x, x_type == ECF8A_E4M3 ? 1 : 2) || !aligned(out, 2) || !aligned(base, 2) ||
        !aligned(x_scale, 4) || !aligned(hidden, 16) || (base == out && ld_base != ld_out))
        return ECF8_ERR_ARG;
    if (ldx < bank->in_features || ld_out < bank->out_features || (base && ld_base < bank->out_features))
        return ECF8_ERR_SIZE;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < ecf8a_add_bytes(plan, bank))
        return ECF8_ERR_WORKSPACE;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    char* w = static_cast<char*>(workspace);
    float* z = hidden ? static_cast<float*>(hidden) : reinterpret_cast<float*>(w);
    const int e = run_low(*plan, *bank, x, ldx, x_type, x_scale, bank->down, bank->in_features, z,
                          reinterpret_cast<float*>(w + z_bytes(*plan, bank->rank)), st);
    if (e != ECF8_OK) return e;
    return run_wide(*plan, *bank, z, bank->up, bank->out_features, base, ld_base, out, ld_out, st);
}

extern "C" int ecf8a_grads(const ecf8a_plan* plan, const ecf8a_bank* bank, const void* dy, uint64_t ld_dy, const void* x,
                           uint64_t ldx, const void* hidden, const void* dx_base, uint64_t ld_dx_base, void* dx,
                           uint64_t ld_dx, void* d_down, void* d_up, void* workspace, uint64_t workspace_bytes,
                           void* hip_stream)
{
    int rc = check_bank(plan, bank);
    if (rc != ECF8_OK) return rc;
    if (!d_down != !d_up || !aligned(d_down, 2) || !aligned(d_up, 2)) return ECF8_ERR_ARG;
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < ecf8a_grads_bytes(plan, bank))
        return ECF8_ERR_WORKSPACE;
    const uint64_t K = bank->in_features, N = bank->out_features;
    if (plan->tokens) {
        if (!dy || (d_down && !x) || !aligned(dy, 2) || !aligned(x, 2) || !aligned(hidden, 16) || !aligned(dx, 2) ||
            !aligned(dx_base, 2) || (dx && dx_base == dx && ld_dx_base != ld_dx))
            return ECF8_ERR_ARG;
        if (ld_dy < N || (d_down && ldx < K) || (dx && ld_dx < K) || (dx && dx_base && ld_dx_base < K))
            return ECF8_ERR_SIZE;
    }
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    char* w = static_cast<char*>(workspace);
    const uint64_t zb = z_bytes(*plan, bank->rank);
    float* z = reinterpret_cast<float*>(w);
    float* h = reinterpret_cast<float*>(w + zb);
    float* scratch = reinterpret_cast<float*>(w + 2 * zb);
    if (plan->tokens) {
        rc = run_low(*plan, *bank, dy, ld_dy, bank->type, nullptr, bank->up, N, z, scratch, st);
        if (rc == ECF8_OK && dx) rc = run_wide(*plan, *bank, z, bank->down, K, dx_base, ld_dx_base, dx, ld_dx, st);
        if (rc == ECF8_OK && d_down && !hidden)
            rc = run_low(*plan, *bank, x, ldx, bank->type, nullptr, bank->down, K, h, scratch, st);
    }
    if (rc != ECF8_OK || !d_down) return rc;
    rc = run_factor(*plan, *bank, z, x, ldx, K, d_down, scratch, st);
    if (rc != ECF8_OK) return rc;
    return run_factor(*plan, *bank, hidden ? static_cast<const float*>(hidden) : h, dy, ld_dy, N, d_up, scratch, st);
}
