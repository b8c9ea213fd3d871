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
// Z is summed in float32 and handed on as two bfloat16 (split2), the form in which
// the matrix instructions take it: 16 bits of it are kept for a second
// instruction on a unit that waits for memory anyway.  A term of the second sum is
// then off by 2^-16 of itself (float16: 2^-15), where the result's own rounding is
// 2^-8 or 2^-11; a third part would be a half more instructions and bytes of Z.  Z is
// written once in the layout of each reader: by slot for `wide` (a lane takes eight
// rank rows of a token), by rank row for `factor` (eight tokens of a rank row), so
// that both load their operands 16 bytes at a time and compute nothing.  The float16
// factors and rows go in as two bfloat16 as well (exact), since a float16 cannot hold
// Z's range.
//
// Tokens are taken in the plan's order: sorted by adapter, each group padded
// to 16 slots, cut into chunks of at most 64 slots that share one adapter.  Few
// tokens need no plan (find_group); with small factors they take one kernel that
// does `low` and `wide` for 16 of them (few_kernel).
#include "ecf8a_common.h"

#include <type_traits>

namespace {

using namespace ecf8a;

constexpr int kTile = 16;                 // slots a group is padded to: one matrix instruction's rows
constexpr int kChunk = 64;                // slots of one chunk at most
constexpr int kPlanThreads = 1024;
constexpr int kPlanLds = 30000;           // ints of LDS for the grouping: 16 waves up to 1577 adapters, 11 for 2048
constexpr int kPlanKept = 20480;          // tokens whose adapters fit beside them
constexpr int kBatch = 4;
constexpr int kThreads = 256;
constexpr int kStrip = 128;               // columns of one wave: 16 lanes of 8

// The plan's workspace: a header, then what each kernel reads of the grouping.
struct PlanView {
    int* head;           // [0] chunks, [1] slots, [2] units
    i32x4* chunks;       // adapter (adapters: none), first slot, tokens, 0
    i32x4* units;        // adapter, first slot, slots, its partial sums' number (-1: the adapter's only unit, which has none)
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

// Exclusive prefix over the workgroup of four values at once.
__device__ __forceinline__ void block_scan4(int v[4], int total[4], i32x4* lds)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int o = __shfl_up(inc[i], d);
            if (lane >= d) inc[i] += o;
        }
    if (lane == 63) lds[wave] = i32x4{inc[0], inc[1], inc[2], inc[3]};
    __syncthreads();
    i32x4 part[kPlanThreads / 64];
#pragma unroll
    for (int w = 0; w < kPlanThreads / 64; ++w) part[w] = lds[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 64; ++w) {
            if (w < wave) before += part[w][i];
            all += part[w][i];
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
                                                            int adapters, int waves, int unit_slots,
                                                            PlanView p)
{
    __shared__ int lds[kPlanLds];
    __shared__ uint16_t kept[kPlanKept];
    __shared__ i32x4 scan[kPlanThreads / 64];
    const int groups = adapters + 1;                        // the last: no adapter
    int* const hist = lds;                                  // [waves][groups]: counts, then where in each group each wave goes on
    int* const count = lds + waves * groups;                // [groups]
    int* const chunk0 = count + groups;                     // [groups]
    int* const slot0 = chunk0 + groups;                     // [groups]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < waves * groups; i += kPlanThreads) hist[i] = 0;
    __syncthreads();
    const int run = ((tokens + waves - 1) / waves + 63) / 64 * 64;
    const int t0 = min(tokens, wave * run), t1 = wave < waves ? min(tokens, t0 + run) : t0;
    const bool keep = tokens <= kPlanKept;                  // the adapters stay in LDS for the second look
    for (int t = t0; t < t1; t += 64 * kBatch) {
        int mine[kBatch];                                   // loads in flight; -1 past the end
#pragma unroll
        for (int i = 0; i < kBatch; ++i) mine[i] = t + i * 64 + lane < t1 ? read_index(index, index_bytes, t + i * 64 + lane, adapters) : -1;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int first = __builtin_amdgcn_readfirstlane(mine[i]);
            const uint64_t real = __ballot(mine[i] >= 0);
            if (__ballot(mine[i] == first || mine[i] < 0) == ~0ull) {     // one request's tokens: one addition
                if (lane == 0 && first >= 0) atomicAdd(&hist[wave * groups + first], (int)__popcll(real));
            } else if (mine[i] >= 0) {
                atomicAdd(&hist[wave * groups + mine[i]], 1);
            }
            if (keep && mine[i] >= 0) kept[t + i * 64 + lane] = (uint16_t)mine[i];
        }
    }
    __syncthreads();
    // Per thread a run of groups, so that one scan over threads covers all.
    const int per = (groups + kPlanThreads - 1) / kPlanThreads;
    const int a0 = min(groups, tid * per), a1 = min(groups, a0 + per);
    int v[4] = {0, 0, 0, 0}, total[4];                      // slots, chunks, units, units with partial sums
    for (int a = a0; a < a1; ++a) {
        int h[kPlanThreads / 64], c = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 64; ++w) h[w] = w < waves ? hist[w * groups + a] : 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 64; ++w)
            if (w < waves) {
                hist[w * groups + a] = c;
                c += h[w];
            }
        count[a] = c;
        const int s = (c + kTile - 1) / kTile * kTile;
        v[0] += s;
        v[1] += (c + kChunk - 1) / kChunk;
        const int units = a < adapters ? (s + unit_slots - 1) / unit_slots : 0;
        v[2] += units;
        v[3] += units > 1 ? units : 0;
    }
    block_scan4(v, total, scan);
    for (int a = a0; a < a1; ++a) {
        const int c = count[a], s = (c + kTile - 1) / kTile * kTile;
        slot0[a] = v[0];
        chunk0[a] = v[1];
        for (int i = c; i < s; ++i) p.slot_token[v[0] + i] = -1;
        if (a < adapters) {
            const int units = (s + unit_slots - 1) / unit_slots;
            p.unit_start[a] = v[2];
            for (int u = 0; u < units; ++u)
                p.units[v[2] + u] = i32x4{a, v[0] + u * unit_slots, min(unit_slots, s - u * unit_slots), units > 1 ? v[3] + u : -1};
            v[2] += units;
            v[3] += units > 1 ? units : 0;
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
    const auto adapter_at = [&](int t) { return t >= t1 ? -1 : keep ? (int)kept[t] : read_index(index, index_bytes, t, adapters); };
    int ahead = adapter_at(t0 + lane);
#pragma unroll 1
    for (int tb = t0; tb < t1; tb += 64) {
        const int t = tb + lane, a = ahead;
        ahead = adapter_at(t + 64);
        int rank = 0, same = 0;
        uint64_t left = __ballot(a >= 0);
        for (int tries = 0; left && tries < 8; ++tries) {     // one adapter of these 64 tokens after the other
            const int first = __builtin_amdgcn_readlane(a, __builtin_ctzll(left));
            const uint64_t mine = __ballot(a == first);
            if (a == first) {
                rank = (int)__popcll(mine & ((1ull << lane) - 1));
                same = (int)__popcll(mine);
            }
            left &= ~mine;
        }
        if (left) {                                           // many adapters: each token with every one before it
            int before = 0, all = 0;
#pragma unroll 16
            for (int j = 0; j < 64; ++j) {
                const bool equal = a == __builtin_amdgcn_readlane(a, j);
                all += equal;
                before += equal && j < lane;
            }
            if (left >> lane & 1) {
                rank = before;
                same = all;
            }
        }
        if (a >= 0) {
            volatile int* next = &hist[wave * groups + a];
            const int at = *next;
            p.slot_token[slot0[a] + at + rank] = t;
            if (rank == same - 1) *next = at + same;          // one lane of each adapter, after every lane's read
        }
    }
}

// ------------------------------------------------------------- low: Z = c V F^T

// A lane's values of a 64-column block, as the operands of two matrix instructions:
// eight from k on and eight from k + GAP on.  Values at or past `limit` are 0 (looked
// at only with TAIL).  VEC: rows of whole, aligned 16-byte units; else the same loads
// at any address, and value by value where a row ends.  16-bit rows have GAP 32, so
// that the four lanes of a row read 64 consecutive bytes; an E4M3 row's 16 bytes
// are one load (GAP 8), and the factor that goes with it follows.
template <int TYPE, int VT, int GAP, bool VEC, bool TAIL>
__device__ __forceinline__ void load_row16(const void* row, int k, int limit, u32x4 v[2])
{
    if constexpr (VT == kE4m3) {
        const uint8_t* p = static_cast<const uint8_t*>(row) + k;
        u32x4 b{0, 0, 0, 0};
        if (!TAIL || k + 16 <= limit) b = load16<VEC>(p);
        else if constexpr (!VEC) {
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
            v[h] = u32x4{0, 0, 0, 0};
            if (!TAIL || k + GAP * h + 8 <= limit) v[h] = load16<VEC>(p + GAP * h);
            else if constexpr (!VEC) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + GAP * h + i < limit) v[h][i >> 1] |= (uint32_t)p[GAP * h + i] << (16 * (i & 1));
            }
        }
    }
}

// Where a Z goes: by slot and by rank row, each as the upper and then the lower
// bfloat16; either may be absent.
struct Forms {
    uint16_t* slot;          // [2][max_slots][zr]
    uint16_t* row;           // [2][max_slots / 16][zr][16]: rows of a tile lie together (a pitch of max_slots put the
                             // rows of one load on one memory channel and took 273 us for 16384 x 18944 at rank 64)
    int64_t plane;           // max_slots * zr
    int zr;
};

// Four consecutive rank rows of one slot.
__device__ __forceinline__ void write_forms(const Forms& f, int slot, int row, f32x4 v)
{
    uint32_t h0, l0, h1, l1;
    split2(v[0], v[1], h0, l0);
    split2(v[2], v[3], h1, l1);
    if (f.slot) {
        uint16_t* p = f.slot + (int64_t)slot * f.zr + row;
        *reinterpret_cast<uint2*>(p) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(p + f.plane) = make_uint2(l0, l1);
    }
    if (f.row) {
        const uint32_t h[2] = {h0, h1}, l[2] = {l0, l1};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint16_t* p = f.row + ((int64_t)(slot / kTile) * f.zr + row + i) * kTile + slot % kTile;
            p[0] = (uint16_t)(h[i >> 1] >> (16 * (i & 1)));
            p[f.plane] = (uint16_t)(l[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// Few tokens without a plan: workgroup b looks token b's adapter up among all tokens
// (one a thread) and goes on if b is its first token, its 17th, ...  Returns the
// adapter, `adapters` for none, -1 if another workgroup has this token; list: the up
// to 16 tokens, -1 behind them.
template <int WAVES>
__device__ __forceinline__ int find_group(const void* index, int bytes, int tokens, int adapters, uint64_t* found, int* list)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x;
    const int a = read_index(index, bytes, b, adapters), own = tid < tokens ? read_index(index, bytes, tid, adapters) : -1;
    if (tid < 16) list[tid] = a >= adapters && tid == 0 ? b : -1;
    if (a >= adapters) {
        __syncthreads();
        return a;
    }
    const bool same = own == a;
    const uint64_t ballot = __ballot(same);
    if (lane == 0) found[wave] = ballot;
    __syncthreads();
    int before = 0, mine = 0;                               // of the adapter's tokens, those before b, and before this one
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        const uint64_t m = found[w];
        before += (int)__popcll(w < (b >> 6) ? m : w == (b >> 6) ? m & ((1ull << (b & 63)) - 1) : 0);
        mine += w < wave ? (int)__popcll(m) : 0;
    }
    if (before % 16) return -1;
    mine += (int)__popcll(ballot & ((1ull << lane) - 1)) - before;
    if (same && mine >= 0 && mine < 16) list[mine] = tid;
    __syncthreads();
    return a;
}

struct LowArgs {
    PlanView plan;
    const void* v;           // tokens' rows
    int64_t ldv;
    const uint16_t* f;       // factor (adapters, rank, width)
    const float* scaling;
    const int32_t* ranks;
    const float* v_scale;
    float* planes;           // [share][max_slots][zr] where the width is split, else nullptr
    Forms forms;
    int width, rank, adapters;
    int per;                 // workgroups per chunk
    const void* index;       // few tokens: the index itself, nullptr with a plan
    int index_bytes, tokens;
};

__device__ __forceinline__ int rank_of(const int32_t* ranks, int a, int rank)
{
    return ranks ? min(max(ranks[a], 0), rank) : rank;
}

// The products of RT times 16 rank rows from r0 on with NT times 16 tokens over
// the 64-column blocks first, first + step, ...  A wave's two loads of a row cover
// whole 128-byte lines.
template <int TYPE, int VT, int RT, int NT, int AHEAD, bool VEC>
__device__ __forceinline__ void low_products(const void* const* vrow, const uint16_t* f, int64_t f_row, int r0, int rank,
                                             int width, int first, int step, f32x4 (*acc)[NT])
{
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const uint16_t* frow[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) frow[r] = f + (f_row + max(0, min(r0 + r * 16 + c, rank - 1))) * width;
    constexpr int GAP = VT == kE4m3 ? 8 : 32;
    const int blocks = (width + 63) / 64, whole = width / 64, k0 = (VT == kE4m3 ? 16 : 8) * g;
    const auto products = [&](const u32x4 (*fv)[2], const u32x4 (*vv)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int n = 0; n < NT; ++n) acc[r][n] = mfma<TYPE>(fv[r][h], vv[n][h], acc[r][n]);
    };
    const auto fetch = [&](int b, u32x4 (*fv)[2], u32x4 (*vv)[2]) {
        const int k = b * 64 + k0;
#pragma unroll
        for (int n = 0; n < NT; ++n) load_row16<TYPE, VT, GAP, VEC, false>(vrow[n], k, width, vv[n]);
#pragma unroll
        for (int r = 0; r < RT; ++r) load_row16<TYPE, TYPE, GAP, VEC, false>(frow[r], k, width, fv[r]);
    };
    // The loads of AHEAD blocks are in flight together, or (1) those of the next one.
    int b = first;
    if constexpr (AHEAD > 1) {
        for (; b + (AHEAD - 1) * step < whole; b += AHEAD * step) {
            u32x4 fv[AHEAD][RT][2], vv[AHEAD][NT][2];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) fetch(b + i * step, fv[i], vv[i]);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) products(fv[i], vv[i]);
        }
        for (; b < whole; b += step) {
            u32x4 fv[RT][2], vv[NT][2];
            fetch(b, fv, vv);
            products(fv, vv);
        }
    } else if (b < whole) {
        u32x4 fv[2][RT][2], vv[2][NT][2];
        fetch(b, fv[0], vv[0]);
        while (true) {
            if (b + step < whole) fetch(b + step, fv[1], vv[1]);
            products(fv[0], vv[0]);
            b += step;
            if (b >= whole) break;
            if (b + step < whole) fetch(b + step, fv[0], vv[0]);
            products(fv[1], vv[1]);
            b += step;
            if (b >= whole) break;
        }
    }
    if (b < blocks) {                                       // the last block, not whole: zeros past the width
        const int k = b * 64 + k0;
        u32x4 fv[RT][2], vv[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) load_row16<TYPE, VT, GAP, VEC, true>(vrow[n], k, width, vv[n]);
#pragma unroll
        for (int r = 0; r < RT; ++r) load_row16<TYPE, TYPE, GAP, VEC, true>(frow[r], k, width, fv[r]);
        products(fv, vv);
    }
}

// Sums TILES results over the WAVES waves of a workgroup, in a fixed order; wave w
// gives tiles w, w + WAVES, ... to done(tile, sum).  red: WAVES / 2 * TILES * 64.
template <int WAVES, int TILES, typename F>
__device__ __forceinline__ void sum_waves(const f32x4* acc, f32x4* red, F done)
{
    constexpr int HALF = WAVES / 2;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (wave >= HALF)
#pragma unroll
        for (int i = 0; i < TILES; ++i) red[((wave - HALF) * TILES + i) * 64 + lane] = acc[i];
    __syncthreads();
    if (wave < HALF)
#pragma unroll
        for (int i = 0; i < TILES; ++i) red[(wave * TILES + i) * 64 + lane] += acc[i];
    __syncthreads();
    for (int i = wave; i < TILES; i += WAVES) {
        f32x4 s = red[i * 64 + lane];
#pragma unroll
        for (int w = 1; w < HALF; ++w) s += red[(w * TILES + i) * 64 + lane];
        done(i, s);
    }
}

// One workgroup: up to NT tiles of one chunk, 16 RT rank rows, one of gridDim.y
// shares of the width.  Its waves take 64-column blocks in turn and meet in LDS.
// token_of(n): this lane's token of tile n.
template <int TYPE, int VT, int RT, int NT, int WAVES, bool VEC, typename F>
__device__ __forceinline__ void low_body(const LowArgs& A, int a, int slot0, int tokens, f32x4* red, F token_of)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4, r0 = blockIdx.z * 64;
    const int rank = rank_of(A.ranks, a, A.rank);
    const void* vrow[NT];
    bool real[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {                          // padding reads row 0; its result is set to 0 below
        const int t = n * kTile < tokens ? token_of(n * kTile + c) : -1;
        real[n] = t >= 0;
        vrow[n] = static_cast<const char*>(A.v) + (VT == kE4m3 ? 1 : 2) * (int64_t)max(t, 0) * A.ldv;
    }
    float scale = A.scaling[a];
    if (A.v_scale) scale *= *A.v_scale;
    f32x4 acc[RT][NT] = {};
    low_products<TYPE, VT, RT, NT, RT + NT <= 2 ? 4 : RT + NT <= 4 ? 2 : 1, VEC>(vrow, A.f, (int64_t)a * A.rank, r0, rank, A.width, blockIdx.y * WAVES + wave, gridDim.y * WAVES, acc);
    sum_waves<WAVES, RT * NT>(&acc[0][0], red, [&](int tile, f32x4 s) {
        const int n = tile % NT, row = r0 + tile / NT * 16 + 4 * g;
        if (n * kTile >= tokens || row >= A.forms.zr) return;   // tiles past the chunk are another's
        bool have = false;
#pragma unroll
        for (int i = 0; i < NT; ++i) have = i == n ? real[i] : have;
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = have && row + i < rank ? s[i] * scale : 0.0f;
        const int slot = slot0 + n * kTile + c;
        if (A.planes) *reinterpret_cast<f32x4*>(A.planes + blockIdx.y * A.forms.plane + (int64_t)slot * A.forms.zr + row) = o;
        else write_forms(A.forms, slot, row, o);
    });
}

// 16 waves where 128 registers hold their loads in flight.
constexpr int low_waves(int rt, int nt) { return rt <= 2 && nt <= 2 ? 16 : 8; }

// With a plan: NT and the shares are chosen so that 256 workgroups or more read the
// rows.  INDEX: few tokens without a plan; the groups found are written down as
// chunks of one tile, slots 16 b on, for wide_kernel to read as it reads a plan.
template <int TYPE, int VT, int RT, int NT, bool VEC, bool INDEX>
__global__ __launch_bounds__(64 * low_waves(RT, NT)) void low_kernel(LowArgs A)
{
    constexpr int WAVES = low_waves(RT, NT);
    __shared__ f32x4 red[WAVES / 2 * RT * NT * 64];
    if constexpr (INDEX) {
        __shared__ uint64_t found[WAVES];
        __shared__ int list[16];
        const int b = blockIdx.x, a = find_group<WAVES>(A.index, A.index_bytes, A.tokens, A.adapters, found, list);
        if (blockIdx.y == 0 && threadIdx.x < 16) {
            if (threadIdx.x == 0) {
                int n = 0;
                for (int i = 0; i < 16; ++i) n += a >= 0 && list[i] >= 0;
                A.plan.chunks[b] = i32x4{a < 0 ? A.adapters : a, b * kTile, n, 0};
                if (b == 0) A.plan.head[0] = A.tokens;
            }
            A.plan.slot_token[b * kTile + threadIdx.x] = a < 0 ? -1 : list[threadIdx.x];
        }
        if (a < 0 || a >= A.adapters) return;
        low_body<TYPE, VT, RT, 1, WAVES, VEC>(A, a, b * kTile, kTile, red, [&](int i) { return list[i]; });
    } else {
        const int id = blockIdx.x / A.per, at = (blockIdx.x - id * A.per) * NT * kTile;
        const i32x4 chunk = A.plan.chunks[id];
        if (id >= A.plan.head[0] || chunk[0] >= A.adapters || at >= chunk[2]) return;
        const int tokens = min(chunk[2] - at, NT * kTile), slot = chunk[1] + at;
        const auto token_of = [&](int i) { return A.plan.slot_token[slot + i]; };
        if (NT >= 2 && tokens <= kTile) low_body<TYPE, VT, RT, 1, WAVES, VEC>(A, chunk[0], slot, tokens, red, token_of);
        else low_body<TYPE, VT, RT, NT, WAVES, VEC>(A, chunk[0], slot, tokens, red, token_of);
    }
}

// Sums the planes of a split width, in plane order.
__global__ __launch_bounds__(kThreads) void join_kernel(const float* __restrict__ planes, int count,
                                                        const int* __restrict__ head, Forms f)
{
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (i >= (int64_t)head[1] * f.zr) return;
    f32x4 s{0, 0, 0, 0};
    for (int p = 0; p < count; p += 8) {                    // eight loads in flight
        f32x4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = *reinterpret_cast<const f32x4*>(planes + min(p + j, count - 1) * f.plane + i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (p + j < count) s += v[j];
    }
    const int slot = (int)(i / f.zr);
    write_forms(f, slot, (int)(i - (int64_t)slot * f.zr), s);
}

// ------------------------------------------------------------- wide: O = B + Z F

struct WideArgs {
    PlanView plan;
    const uint16_t* z;       // by slot
    const float* planes;     // PLANES: the shares' sums instead, [shares][slot][zr]
    int64_t plane;
    int shares;
    const uint16_t* f;
    const int32_t* ranks;
    const uint16_t* base;
    int64_t ld_base;
    uint16_t* out;
    int64_t ld_out;
    int width, rank, zr, adapters;
    int groups;              // workgroups across the width
};

// Eight columns of a row, 0 past the width.
template <bool VEC>
__device__ __forceinline__ u32x4 load_cols(const uint16_t* row, int col, int width)
{
    u32x4 v{0, 0, 0, 0};
    if (VEC ? col < width : col + 8 <= width) v = load16<VEC>(row + col);
    else if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < width) v[j >> 1] |= (uint32_t)row[col + j] << (16 * (j & 1));
    }
    return v;
}

template <bool VEC>
__device__ __forceinline__ void store_cols(uint16_t* row, int col, int width, u32x4 v)
{
    if (VEC ? col < width : col + 8 <= width) store16<VEC>(row + col, v);
    else if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (col + j < width) row[col + j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
    }
}

// Rows r .. r + 7 of the factor at this lane's eight columns.  Rows that take no
// part are 0, whatever is stored there.
template <bool VEC>
__device__ __forceinline__ void load_factor(const uint16_t* f, int width, int r, int rank, int col, u32x4 w[8])
{
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        w[q] = u32x4{0, 0, 0, 0};
        if (r + q < rank) w[q] = load_cols<VEC>(f + (int64_t)(r + q) * width, col, width);
    }
}

// ... turned into one operand per column (lo: of a float16, the rest of it).
template <int TYPE>
__device__ __forceinline__ void turn_factor(const u32x4 w[8], u32x4 hi[8], u32x4 lo[8])
{
    transpose8(w, hi);
    if constexpr (TYPE == kFp16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) split8_f16(hi[j], hi[j], lo[j]);
    }
}

// One row's eight columns: base plus the results of its token, rounded once.
template <int TYPE>
__device__ __forceinline__ u32x4 add_row(u32x4 base, const f32x4* acc, int i)
{
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const f32x2 b = unpack2<TYPE>(base[j]);
        o[j] = pack2<TYPE>(b[0] + acc[2 * j][i], b[1] + acc[2 * j + 1][i]);
    }
    return o;
}

// The products of 16 tokens with 32 rank rows at this lane's eight columns.  HALF: up
// to 16 rank rows, whose lower bfloat16 take the upper half of the reduction slots,
// so that one instruction does both.  CAREFUL: see any_not_finite.
template <int TYPE, bool HALF, bool CAREFUL>
__device__ __forceinline__ void wide_products(u32x4 zh, u32x4 zl, const u32x4* hi, const u32x4* lo, f32x4* acc)
{
    const auto kept_finite = [](u32x4 v) {
        asm volatile("" : "+v"(v));                         // not to be found once and kept in registers
        return finite(v);
    };
    const bool lower = HALF && (threadIdx.x & 32);          // lanes that hold the lower halves' slots
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        acc[j] = mfma_bf16(zh, CAREFUL && lower ? kept_finite(hi[j]) : hi[j], acc[j]);
        if constexpr (!HALF) acc[j] = mfma_bf16(zl, CAREFUL ? kept_finite(hi[j]) : hi[j], acc[j]);
        if constexpr (TYPE == kFp16) acc[j] = mfma_bf16(CAREFUL ? kept_finite(zh) : zh, lo[j], acc[j]);
    }
}

// Eight rank rows of one slot from the shares' sums, added in order.
__device__ __forceinline__ void sum_planes(const float* z, int64_t plane, int shares, u32x4& zh, u32x4& zl)
{
    f32x4 s0{0, 0, 0, 0}, s1{0, 0, 0, 0};
    for (int p = 0; p < shares; p += 4) {                   // eight loads in flight
        f32x4 v0[4], v1[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float* q = z + min(p + j, shares - 1) * plane;
            v0[j] = *reinterpret_cast<const f32x4*>(q);
            v1[j] = *reinterpret_cast<const f32x4*>(q + 4);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (p + j < shares) {
                s0 += v0[j];
                s1 += v1[j];
            }
    }
    split8(s0, s1, zh, zl);
}

// One wave: 128 columns of one chunk.  A lane's eight columns are consecutive
// (column 8c + j goes to the j-th instruction), so that the factor's rows are
// read, and the result's rows read and written, 16 bytes at a time, and no LDS
// is used.  RB: blocks of 32 rank rows kept in registers for the whole chunk
// (0: up to 16 rows; -1: any number, read again for each 16 tokens).
//
// Bound by the rows' way in and out.  What keeps that busy is many waves rather
// than many loads of each: with the rows of all four tiles sent for at once a wave
// holds 158 to 255 registers, and 8192 tokens x 14336 columns at rank 32 take 108
// us, 16384 x 13824 at rank 64 take 338; tile by tile 88 and 188 (5.3 and 4.8
// TB/s).  The result is stored past the caches, which are left to the base rows
// (2048 x 8192 at rank 16: 17 -> 13 us).
// Workgroups run along the rows, whatever die each falls on: columns kept to a die,
// so that its cache holds their part of the factor, take 94 us at 8192 x 14336 and
// 204 at 16384 x 13824; chunks of rows kept to a die 92 and 197.
template <int TYPE, int RB, bool VEC, bool PLANES>
__device__ __forceinline__ void wide_rows(const WideArgs& A, int group)
{
    const int id = group / A.groups;                        // neighbouring workgroups: the same rows, next columns
    const i32x4 chunk = A.plan.chunks[id];                  // there for every id, and sent for with the count
    if (id >= A.plan.head[0]) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int a = chunk[0], col = ((group - id * A.groups) * 4 + wave) * kStrip + 8 * c;
    if (col - 8 * c >= A.width) return;
    const bool bare = a >= A.adapters;
    if (bare && A.base == A.out) return;
    const int tiles = (chunk[2] + kTile - 1) / kTile;
    const int rank = bare ? 0 : rank_of(A.ranks, a, A.rank);
    const uint16_t* f = A.f + (int64_t)(bare ? 0 : a) * A.rank * A.width;
    constexpr int KEEP = RB <= 0 ? 1 : RB;
    u32x4 hi[KEEP][8], lo[KEEP][8];
    if constexpr (RB >= 0) {
#pragma unroll
        for (int b = 0; b < KEEP; ++b) {
            u32x4 w[8];
            load_factor<VEC>(f, A.width, RB == 0 ? 8 * (g & 1) : 32 * b + 8 * g, rank, col, w);
            turn_factor<TYPE>(w, hi[b], lo[b]);
        }
    }
    for (int tile = 0; tile < tiles; ++tile) {
        const int slot = chunk[1] + tile * kTile;
        const i32x4 tok = *reinterpret_cast<const i32x4*>(A.plan.slot_token + slot + 4 * g);
        u32x4 base[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            base[i] = u32x4{0, 0, 0, 0};
            if (A.base && tok[i] >= 0) base[i] = load_cols<VEC>(A.base + tok[i] * A.ld_base, col, A.width);
        }
        if (bare) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (tok[i] >= 0) store_cols<VEC>(A.out + tok[i] * A.ld_out, col, A.width, base[i]);
            continue;
        }
        const int64_t at = (int64_t)(slot + c) * A.zr;
        f32x4 acc[8] = {};
        const auto tile_products = [&](auto careful) {
            if constexpr (RB == 0) {
                u32x4 both, rest;
                if constexpr (PLANES) {
                    sum_planes(A.planes + at + 8 * (g & 1), A.plane, A.shares, both, rest);
                    both = g < 2 ? both : rest;
                } else {
                    both = *reinterpret_cast<const u32x4*>(A.z + at + 8 * (g & 1) + (g < 2 ? 0 : A.plane));
                }
                wide_products<TYPE, true, careful>(both, both, hi[0], lo[0], acc);
            } else {
                const auto block = [&](int b, int keep) {
                    u32x4 zh, zl;
                    if constexpr (PLANES) sum_planes(A.planes + at + 32 * b + 8 * g, A.plane, A.shares, zh, zl);
                    else {
                        zh = *reinterpret_cast<const u32x4*>(A.z + at + 32 * b + 8 * g);
                        zl = *reinterpret_cast<const u32x4*>(A.z + at + 32 * b + 8 * g + A.plane);
                    }
                    wide_products<TYPE, false, careful>(zh, zl, hi[keep], lo[keep], acc);
                };
                if constexpr (RB > 0) {
#pragma unroll
                    for (int b = 0; b < RB; ++b) block(b, b);
                } else {
                    for (int b = 0; b < (A.zr + 31) / 32; ++b) {
                        u32x4 w[8];
                        load_factor<VEC>(f, A.width, 32 * b + 8 * g, rank, col, w);
                        turn_factor<TYPE>(w, hi[0], lo[0]);
                        block(b, 0);
                    }
                }
            }
        };
        tile_products(std::false_type{});
        if (any_not_finite<8>(acc)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = f32x4{0, 0, 0, 0};
            tile_products(std::true_type{});
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (tok[i] >= 0) store_cols<VEC>(A.out + tok[i] * A.ld_out, col, A.width, add_row<TYPE>(base[i], acc, i));
    }
}

template <int TYPE, int RB, bool VEC, bool PLANES>
__global__ __launch_bounds__(kThreads, TYPE == kBf16 ? (RB == 0 || (RB == 1 && !PLANES) ? 4 : 3) : 2) void wide_kernel(WideArgs A)
{
    wide_rows<TYPE, RB, VEC, PLANES>(A, blockIdx.x);
}

// ------------------------------------------------------------- few tokens: both at once

struct FewArgs {
    PlanView plan;           // used where index is nullptr
    const void* index;
    int index_bytes, tokens;
    const void* v;
    int64_t ldv;
    const uint16_t* f;       // (adapters, rank, in)
    const uint16_t* f2;      // (adapters, rank, out)
    const float* scaling;
    const int32_t* ranks;
    const float* v_scale;
    const uint16_t* base;
    int64_t ld_base;
    uint16_t* out;           // nullptr: only the forms are wanted
    int64_t ld_out;
    Forms forms;             // by rank row, for the gradients; row nullptr: not wanted
    int in, width, rank, adapters;
};

// One workgroup: 16 tokens of one adapter, from their rows to the result.  Its
// waves split the input width for `low`, leave h in LDS, and split the output width
// for `wide`.  One launch, no workspace and no grouping beforehand.  What bounds it
// is how fast one compute unit reads both factors of its adapter, about 30 GB/s
// however many loads are in flight (256 KB: 4 us for each half): it is taken for
// small factors only.
constexpr int kFewWaves = 8;              // few enough to have 256 registers each, for loads in flight

template <int TYPE, int VT, int RT, bool VEC>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(FewArgs A)
{
    constexpr int ZR = 16 * RT, WAVES = kFewWaves;
    __shared__ f32x4 red[WAVES / 2 * RT * 64];
    __shared__ __attribute__((aligned(16))) uint16_t zs[2][16][ZR + 8];   // 8 more: rows meet different banks
    __shared__ uint64_t found[WAVES];
    __shared__ __attribute__((aligned(16))) int list[16];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, g = lane >> 4;
    int a, slot0 = 0;
    if (A.index) {
        a = find_group<WAVES>(A.index, A.index_bytes, A.tokens, A.adapters, found, list);
        if (a < 0) return;
    } else {
        const int id = blockIdx.x / 4, at = (blockIdx.x & 3) * kTile;
        const i32x4 chunk = A.plan.chunks[id];
        if (id >= A.plan.head[0] || at >= chunk[2]) return;
        a = chunk[0];
        slot0 = chunk[1] + at;
        if (tid < 16) list[tid] = A.plan.slot_token[slot0 + tid];
        __syncthreads();
    }
    if (a >= A.adapters) {                                  // no adapter: the rows themselves
        if (!A.out || A.base == A.out) return;
        for (int i = wave; i < 16; i += WAVES) {
            const int t = list[i];
            if (t < 0) continue;
            for (int col = 8 * lane; col < A.width; col += 8 * 64) {
                u32x4 v{0, 0, 0, 0};
                if (A.base) v = load_cols<VEC>(A.base + t * A.ld_base, col, A.width);
                store_cols<VEC>(A.out + t * A.ld_out, col, A.width, v);
            }
        }
        return;
    }
    const int rank = rank_of(A.ranks, a, A.rank);
    const bool real = list[c] >= 0;
    const void* vrow = static_cast<const char*>(A.v) + (VT == kE4m3 ? 1 : 2) * (int64_t)max(list[c], 0) * A.ldv;
    // The first strip's rows and the first block of its factor do not wait for h.
    const i32x4 tok = *reinterpret_cast<const i32x4*>(&list[4 * g]);
    const uint16_t* f = A.f2 + (int64_t)a * A.rank * A.width;
    u32x4 base[4], w[8];
    const auto fetch = [&](int col) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            base[i] = u32x4{0, 0, 0, 0};
            if (A.base && tok[i] >= 0) base[i] = load_cols<VEC>(A.base + tok[i] * A.ld_base, col, A.width);
        }
        load_factor<VEC>(f, A.width, RT == 1 ? 8 * (g & 1) : 8 * g, rank, col, w);
    };
    if (A.out && wave * kStrip < A.width) fetch(wave * kStrip + 8 * c);
    f32x4 acc[RT][1] = {};
    low_products<TYPE, VT, RT, 1, RT == 1 && TYPE == kBf16 ? 8 : RT <= 2 ? 4 : 2, VEC>(&vrow, A.f, (int64_t)a * A.rank, 0, rank, A.in, wave, WAVES, acc);
    float scale = A.scaling[a];
    if (A.v_scale) scale *= *A.v_scale;
    sum_waves<WAVES, RT>(&acc[0][0], red, [&](int tile, f32x4 s) {
        const int row = tile * 16 + 4 * g;
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = real && row + i < rank ? s[i] * scale : 0.0f;
        uint32_t h0, l0, h1, l1;
        split2(o[0], o[1], h0, l0);
        split2(o[2], o[3], h1, l1);
        *reinterpret_cast<uint2*>(&zs[0][c][row]) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(&zs[1][c][row]) = make_uint2(l0, l1);
        if (A.forms.row && row < A.forms.zr) write_forms(A.forms, slot0 + c, row, o);
    });
    __syncthreads();
    if (!A.out) return;
    for (int strip = wave * kStrip; strip < A.width; strip += WAVES * kStrip) {
        const int col = strip + 8 * c;
        f32x4 sum[8] = {};
        u32x4 hi[8], lo[8], row[4] = {base[0], base[1], base[2], base[3]};
        turn_factor<TYPE>(w, hi, lo);
        if (strip + WAVES * kStrip < A.width) fetch(col + WAVES * kStrip);
        const auto strip_products = [&](auto careful) {
            if constexpr (RT == 1) {
                const u32x4 both = *reinterpret_cast<const u32x4*>(&zs[g >> 1][c][8 * (g & 1)]);
                wide_products<TYPE, true, careful>(both, both, hi, lo, sum);
            } else {
#pragma unroll
                for (int b = 0; b < RT / 2; ++b) {
                    if (b || (careful && RT > 2)) {
                        u32x4 more[8];
                        load_factor<VEC>(f, A.width, 32 * b + 8 * g, rank, col, more);
                        turn_factor<TYPE>(more, hi, lo);
                    }
                    wide_products<TYPE, false, careful>(*reinterpret_cast<const u32x4*>(&zs[0][c][32 * b + 8 * g]),
                                                        *reinterpret_cast<const u32x4*>(&zs[1][c][32 * b + 8 * g]), hi, lo, sum);
                }
            }
        };
        strip_products(std::false_type{});
        if (any_not_finite<8>(sum)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = f32x4{0, 0, 0, 0};
            strip_products(std::true_type{});
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (tok[i] >= 0) store_cols<VEC>(A.out + tok[i] * A.ld_out, col, A.width, add_row<TYPE>(row[i], sum, i));
    }
}

// ------------------------------------------------------------- factor: G = Z^T V

struct FactorSide {
    const uint16_t* z;       // by rank row
    const uint16_t* v;
    int64_t ldv;
    uint16_t* grad;          // (adapters, rank, width)
    float* part;             // [units with partial sums][zr][stride]
    int width, stride;
};

struct FactorArgs {
    PlanView plan;
    FactorSide side[2];      // d_down from z and x, d_up from h and dy
    const int32_t* ranks;
    int64_t plane;
    int rank, zr, adapters;
    int groups;              // workgroups across side 0
};

// One wave: one unit of one adapter's slots, 128 columns of one side, 16 RT rank
// rows.  The four waves of a workgroup take neighbouring columns of the same slots
// (HALVES 2: two strips of columns, and for each two halves of 64 rank rows), so
// that a wave's Z or V comes from the first-level cache for another.  64 rank rows
// in one wave hold 276 registers, one wave per SIMD: 267 us for 16384 x 18944.  A lane reads
// eight tokens' 16 bytes and turns them, as the factor is turned in `wide`, so that
// the sum over tokens runs in the matrix instructions' reduction slots.  An
// adapter of one unit is written at once, others leave float32 partial sums that
// sum_kernel joins in order.
template <int TYPE, int RT, int HALVES, bool VEC>
__device__ __forceinline__ void factor_unit(const FactorArgs& A, int group, int at_unit, int rank0)
{
    const i32x4 unit = A.plan.units[at_unit];
    if (at_unit >= A.plan.head[2]) return;
    const bool second = group >= A.groups;
    const FactorSide& S = A.side[second];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int strip = (group - (second ? A.groups : 0)) * (4 / HALVES) + wave / HALVES;
    const int col = strip * kStrip + 8 * c, r0 = rank0 + wave % HALVES * 32;
    if (strip * kStrip >= S.width || r0 >= A.zr) return;
    f32x4 acc[RT][8] = {};
    i32x4 tok[2];
    u32x4 w[8];
    const auto tokens_of = [&](int s) {
        tok[0] = tok[1] = i32x4{-1, -1, -1, -1};
        if (s + 8 * g < unit[2]) {                            // units are whole tiles of 16: eight slots are in or out
            tok[0] = *reinterpret_cast<const i32x4*>(A.plan.slot_token + unit[1] + s + 8 * g);
            tok[1] = *reinterpret_cast<const i32x4*>(A.plan.slot_token + unit[1] + s + 8 * g + 4);
        }
    };
    const auto rows_of = [&]() {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int tq = tok[q >> 2][q & 3];
            w[q] = u32x4{0, 0, 0, 0};
            if (tq >= 0) w[q] = load_cols<VEC>(S.v + tq * S.ldv, col, S.width);
        }
    };
    // The rows are not sent for ahead of their turn: that takes 32 registers, and a
    // third wave per SIMD hides more (8192 x 18432 at rank 32: 92 -> 62 us).
    const auto unit_sum = [&](auto careful) {
        tokens_of(0);
        for (int s = 0; s < unit[2]; s += 32) {
            rows_of();
            tokens_of(s + 32);
            const bool have = s + 8 * g < unit[2];
            u32x4 zh[RT], zl[RT], t[8], tl[8];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int row = r0 + r * 16 + c;
                zh[r] = zl[r] = u32x4{0, 0, 0, 0};
                if (have && row < A.zr) {
                    const int slot = unit[1] + s + 8 * g;
                    const uint16_t* z = S.z + ((int64_t)(slot / kTile) * A.zr + row) * kTile + slot % kTile;
                    zh[r] = *reinterpret_cast<const u32x4*>(z);
                    zl[r] = *reinterpret_cast<const u32x4*>(z + A.plane);
                }
            }
            transpose8(w, t);
            if constexpr (TYPE == kFp16) {
#pragma unroll
                for (int j = 0; j < 8; ++j) split8_f16(t[j], t[j], tl[j]);
            }
            if constexpr (!careful) {
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        acc[r][j] = mfma_bf16(zh[r], t[j], acc[r][j]);
                        acc[r][j] = mfma_bf16(zl[r], t[j], acc[r][j]);
                        if constexpr (TYPE == kFp16) acc[r][j] = mfma_bf16(zh[r], tl[j], acc[r][j]);
                    }
            } else {                                          // in place, in an order that needs no copies
                const auto products = [&](const u32x4* z, const u32x4* v) {
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[r][j] = mfma_bf16(z[r], v[j], acc[r][j]);
                };
                products(zh, t);
                if constexpr (TYPE == kFp16) {
#pragma unroll
                    for (int r = 0; r < RT; ++r) zh[r] = finite(zh[r]);
                    products(zh, tl);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) t[j] = finite(t[j]);
                products(zl, t);
            }
        }
    };
    unit_sum(std::false_type{});
    if (any_not_finite<8 * RT>(&acc[0][0])) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[r][j] = f32x4{0, 0, 0, 0};
        unit_sum(std::true_type{});
    }
    if (col >= S.width) return;
    const int a = unit[0], rank = rank_of(A.ranks, a, A.rank);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = r0 + r * 16 + 4 * g + i;
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = row < rank ? acc[r][j][i] : 0.0f;
            if (unit[3] < 0) {
                if (row >= A.rank) continue;
                store_cols<VEC>(S.grad + ((int64_t)a * A.rank + row) * S.width, col, S.width,
                                u32x4{pack2<TYPE>(v[0], v[1]), pack2<TYPE>(v[2], v[3]), pack2<TYPE>(v[4], v[5]),
                                      pack2<TYPE>(v[6], v[7])});
            } else if (row < A.zr) {
                float* p = S.part + ((int64_t)unit[3] * A.zr + row) * S.stride + col;
                *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
                *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
            }
        }
}

constexpr int factor_waves(int type, int rt) { return (rt == 1 ? 4 : 3) - (type == kFp16); }   // per SIMD

template <int TYPE, int RT, int HALVES, bool VEC>
__global__ __launch_bounds__(kThreads, factor_waves(TYPE, RT)) void factor_kernel(FactorArgs A)
{
    factor_unit<TYPE, RT, HALVES, VEC>(A, blockIdx.x, blockIdx.y, blockIdx.z * 64);
}

// dx and both factors' gradients need only z and h: one launch for both, the
// workgroups of one spread evenly among those of the other, so that rows on their way
// in and out and waits for rows to be multiplied overlap: 4096 tokens of 4096 and 4096
// at rank 16 take 28 us instead of 17 + 14; 16384 of 5120 and 13824 at rank 64 take
// 272 both ways, but for the launch between (whole calls: 103 -> 97, 650 -> 642).
// Over rank 64 `wide` reads its factor again for each 64 rank rows and stays apart.
template <int TYPE, int RB, int RT, int HALVES, bool VEC>
__global__ __launch_bounds__(kThreads, factor_waves(TYPE, RT)) void wide_and_factor_kernel(WideArgs W, FactorArgs F, uint32_t factor_groups,
                                                                                         uint32_t across)
{
    const uint32_t before = (uint32_t)((uint64_t)blockIdx.x * factor_groups / gridDim.x);
    const uint32_t until = (uint32_t)((uint64_t)(blockIdx.x + 1) * factor_groups / gridDim.x);
    if (until > before) factor_unit<TYPE, RT, HALVES, VEC>(F, before % across, before / across, 0);
    else wide_rows<TYPE, RB, VEC, false>(W, blockIdx.x - before);
}

// The gradients of adapters with no unit (0) or several (their partial sums).
template <int TYPE, bool VEC>
__global__ __launch_bounds__(kThreads) void sum_kernel(FactorArgs A, int first)
{
    const int a = blockIdx.z, row = blockIdx.y;
    const int u0 = A.plan.unit_start[a], u1 = A.plan.unit_start[a + 1];
    if (u1 - u0 == 1) return;
    const bool second = (int)blockIdx.x >= first;
    const FactorSide& S = A.side[second];
    const int col = ((blockIdx.x - (second ? first : 0)) * kThreads + threadIdx.x) * 4;
    if (col >= S.width) return;
    f32x4 s{0, 0, 0, 0};
    const int first_part = u1 > u0 ? A.plan.units[u0][3] : 0, parts = u1 - u0;      // an adapter's parts lie together
    for (int u = 0; u < parts; u += 4) {                    // four loads in flight, added in order
        f32x4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = *reinterpret_cast<const f32x4*>(S.part + ((int64_t)(first_part + min(u + j, parts - 1)) * A.zr + row) * S.stride + col);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (u + j < parts) s += v[j];
    }
    uint16_t* p = S.grad + ((int64_t)a * A.rank + row) * S.width + col;
    if (VEC) *reinterpret_cast<uint2*>(p) = make_uint2(pack2<TYPE>(s[0], s[1]), pack2<TYPE>(s[2], s[3]));
    else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < S.width) p[i] = round1<TYPE>(s[i]);
    }
}

// ------------------------------------------------------------- host side

uint32_t z_rows(uint32_t rank) { return rank <= 16 ? 16 : (uint32_t)round_up(rank, 32); }

// How a `low` call covers the chunks: tiles of one workgroup, and the shares of
// the width where that leaves fewer than 256 workgroups.  More tiles read the factor
// less often, fewer fill the card from fewer tokens.  Measured (bfloat16): 16384 x
// 13824, rank 64: 111 us with four tiles, 153 with two, 254 with one; 8192 x 4096,
// rank 32: 26, 35, 27, rank 64: 33, 28, 41; 4096 x 4096, rank 16: four tiles in three
// shares 11.6 and a join, one tile unsplit 11.1.
struct LowShape {
    uint32_t tiles, shares;
};

LowShape low_shape(const ecf8a_plan& p, uint32_t rank, uint64_t width)
{
    const uint64_t used = p.adapters < p.tokens ? p.adapters : p.tokens;
    LowShape s{p.tokens < 8192 ? 1u : p.tokens >= 16384 || rank <= 32 ? 4u : 2u, 1};
    const uint64_t groups = p.tokens / (kTile * s.tiles) + used;
    uint64_t shares = groups ? 256 / groups : 1;
    const uint64_t most = (width + 511) / 512;
    if (shares > most) shares = most;
    s.shares = (uint32_t)(shares < 1 ? 1 : shares > 16 ? 16 : shares);
    return s;
}

uint64_t form_bytes(const ecf8a_plan& p, uint32_t rank) { return round_up(4ull * p.max_slots * z_rows(rank), 256); }

uint64_t low_bytes(const ecf8a_plan& p, uint32_t rank, uint64_t width)
{
    const uint64_t s = low_shape(p, rank, width).shares;
    return s > 1 ? round_up(s * 4ull * p.max_slots * z_rows(rank), 256) : 0;
}

// Units that leave partial sums: those of adapters with several.  Such an adapter has c > unit_slots tokens and
// ceil(c / unit_slots) <= 2 c / unit_slots units, so their number follows the tokens and not the bank (8192 tokens, 2048
// adapters of rank 64, 8192 x 8192: 0.2 GB, where a place for every unit would take 8.7).
uint64_t max_parts(const ecf8a_plan& p)
{
    if (p.tokens <= p.unit_slots) return 0;
    const uint64_t most = 2 * p.tokens / p.unit_slots;
    return most < p.max_units ? most : p.max_units;
}

uint64_t part_bytes(const ecf8a_plan& p, uint32_t rank, uint64_t width)
{
    return round_up(4ull * max_parts(p) * z_rows(rank) * round_up(width, kStrip), 256);
}

bool plan_ok(const ecf8a_plan* p)
{
    return p && p->tokens <= ECF8A_MAX_TOKENS && p->adapters >= 1 && p->adapters <= ECF8A_MAX_ADAPTERS && p->unit_slots >= 1;
}

int check_bank(const ecf8a_bank* b)
{
    if (!b) return ECF8_ERR_ARG;
    if (b->type != ECF8A_BF16 && b->type != ECF8A_FP16) return ECF8_ERR_UNSUPPORTED;
    if (b->adapters < 1 || b->adapters > ECF8A_MAX_ADAPTERS || b->rank < 1 || b->rank > ECF8A_MAX_RANK ||
        b->in_features < 1 || b->in_features > ECF8A_MAX_FEATURES || b->out_features < 1 ||
        b->out_features > ECF8A_MAX_FEATURES)
        return ECF8_ERR_SIZE;
    if (!b->down || !b->up || !b->scaling || !aligned(b->down, 2) || !aligned(b->up, 2) || !aligned(b->scaling, 4) ||
        !aligned(b->ranks, 4))
        return ECF8_ERR_ARG;
    return ECF8_OK;
}

bool vec16(const void* p, uint64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

// One direction of the pair: rows v of width `in` through factor f, and through
// factor f2 onto base rows of width `out_width`.
struct Pass {
    const void* v;
    uint64_t ldv;
    uint32_t vt;
    const float* v_scale;
    const void* f;
    uint64_t in;
    const void* f2;
    uint64_t width;
    const void* base;
    uint64_t ld_base;
    void* out;               // nullptr: only the forms
    uint64_t ld_out;
};

bool vec_low(const Pass& s)
{
    return s.vt == ECF8A_E4M3 ? aligned(s.v, 16) && s.ldv % 16 == 0 && s.in % 16 == 0 && aligned(s.f, 16)
                              : vec16(s.v, s.ldv) && vec16(s.f, s.in);
}

bool vec_wide(const Pass& s)
{
    return vec16(s.f2, s.width) && vec16(s.out, s.ld_out) && (!s.base || vec16(s.base, s.ld_base));
}

// Few tokens: from the index itself, without a plan.
bool few(uint64_t tokens, const ecf8a_bank& b) { return tokens <= ECF8A_FEW_TOKENS && b.rank <= ECF8A_FEW_RANK; }

// Whether few_kernel does both halves at once: factors of up to 256 KB, which one
// compute unit reads in about as long as a second launch takes.  One token, 4096 x
// 4096 at rank 16 (256 KB): 11.2 us in one kernel, 5.7 + 5.6 in two; 64 tokens, 8192
// x 8192 at rank 16 (512 KB): 22.5 us in one, 7.9 + 7.7 in two.
bool one_kernel(uint64_t tokens, const ecf8a_bank& b)
{
    return few(tokens, b) && 2ull * b.rank * (b.in_features + b.out_features) <= 256u << 10;
}

// Shares of the width for few tokens: every token may have an adapter of its own, or
// all of them one.
uint32_t few_shares(uint64_t tokens, uint64_t width)
{
    uint64_t s = 512 / (tokens ? tokens : 1);
    const uint64_t most = (width + 511) / 512;
    if (s < 4) s = 4;
    if (s > most) s = most;
    return (uint32_t)(s < 1 ? 1 : s > 8 ? 8 : s);
}

// The workspace of ecf8a_add_few: the groups as wide_kernel reads a plan's, then the
// shares' sums.
PlanView few_view(void* workspace, uint64_t tokens)
{
    char* w = static_cast<char*>(workspace);
    return PlanView{reinterpret_cast<int*>(w), reinterpret_cast<i32x4*>(w + 256), nullptr, nullptr,
                    reinterpret_cast<int*>(w + 256 + 16 * tokens)};
}
uint64_t few_planes_at(uint64_t tokens) { return round_up(256 + 16 * tokens + 4 * kTile * tokens, 256); }

template <int TYPE, int VT, bool VEC>
void launch_few(const FewArgs& A, uint32_t grid, hipStream_t st)
{
    if (A.rank <= 16) few_kernel<TYPE, VT, 1, VEC><<<grid, 64 * kFewWaves, 0, st>>>(A);
    else if (A.rank <= 32) few_kernel<TYPE, VT, 2, VEC><<<grid, 64 * kFewWaves, 0, st>>>(A);
    else few_kernel<TYPE, VT, 4, VEC><<<grid, 64 * kFewWaves, 0, st>>>(A);
}

int run_few(const PlanView& view, uint32_t grid, const void* index, uint32_t index_bytes, uint64_t tokens,
            const ecf8a_bank& b, const Pass& s, const Forms& forms, hipStream_t st)
{
    const FewArgs A{view, index, (int)index_bytes, (int)tokens, s.v, (int64_t)s.ldv, static_cast<const uint16_t*>(s.f),
                    static_cast<const uint16_t*>(s.f2), b.scaling, b.ranks, s.v_scale,
                    static_cast<const uint16_t*>(s.base), (int64_t)s.ld_base, static_cast<uint16_t*>(s.out),
                    (int64_t)s.ld_out, forms, (int)s.in, (int)s.width, (int)b.rank, (int)b.adapters};
    const bool vec = vec_low(s) && (!s.out || vec_wide(s)), e4m3 = s.vt == ECF8A_E4M3;
    if (b.type == ECF8A_BF16) {
        if (e4m3) vec ? launch_few<kBf16, kE4m3, true>(A, grid, st) : launch_few<kBf16, kE4m3, false>(A, grid, st);
        else vec ? launch_few<kBf16, kBf16, true>(A, grid, st) : launch_few<kBf16, kBf16, false>(A, grid, st);
    } else {
        if (e4m3) vec ? launch_few<kFp16, kE4m3, true>(A, grid, st) : launch_few<kFp16, kE4m3, false>(A, grid, st);
        else vec ? launch_few<kFp16, kFp16, true>(A, grid, st) : launch_few<kFp16, kFp16, false>(A, grid, st);
    }
    return launch_status();
}

template <int TYPE, int VT, int RT, bool VEC>
void launch_low_tiles(const LowArgs& A, dim3 grid, uint32_t tiles, hipStream_t st)
{
    if (A.index) low_kernel<TYPE, VT, RT, 1, VEC, true><<<grid, 64 * low_waves(RT, 1), 0, st>>>(A);
    else if (tiles == 1) low_kernel<TYPE, VT, RT, 1, VEC, false><<<grid, 64 * low_waves(RT, 1), 0, st>>>(A);
    else if (tiles == 2) low_kernel<TYPE, VT, RT, 2, VEC, false><<<grid, 64 * low_waves(RT, 2), 0, st>>>(A);
    else low_kernel<TYPE, VT, RT, 4, VEC, false><<<grid, 64 * low_waves(RT, 4), 0, st>>>(A);
}

template <int TYPE, int VT, bool VEC>
void launch_low(const LowArgs& A, dim3 grid, uint32_t tiles, hipStream_t st)
{
    if (A.forms.zr <= 16) launch_low_tiles<TYPE, VT, 1, VEC>(A, grid, tiles, st);
    else if (A.forms.zr <= 32) launch_low_tiles<TYPE, VT, 2, VEC>(A, grid, tiles, st);
    else launch_low_tiles<TYPE, VT, 4, VEC>(A, grid, tiles, st);
}

void launch_low_pass(const LowArgs& A, const ecf8a_bank& b, const Pass& s, dim3 grid, uint32_t n, hipStream_t st)
{
    const bool e4m3 = s.vt == ECF8A_E4M3, vec = vec_low(s);
    if (b.type == ECF8A_BF16) {
        if (e4m3) vec ? launch_low<kBf16, kE4m3, true>(A, grid, n, st) : launch_low<kBf16, kE4m3, false>(A, grid, n, st);
        else vec ? launch_low<kBf16, kBf16, true>(A, grid, n, st) : launch_low<kBf16, kBf16, false>(A, grid, n, st);
    } else {
        if (e4m3) vec ? launch_low<kFp16, kE4m3, true>(A, grid, n, st) : launch_low<kFp16, kE4m3, false>(A, grid, n, st);
        else vec ? launch_low<kFp16, kFp16, true>(A, grid, n, st) : launch_low<kFp16, kFp16, false>(A, grid, n, st);
    }
}

LowArgs low_args(const PlanView& view, const ecf8a_bank& b, const Pass& s, const Forms& forms, float* planes, int per)
{
    return LowArgs{view, s.v, (int64_t)s.ldv, static_cast<const uint16_t*>(s.f), b.scaling, b.ranks, s.v_scale, planes, forms,
                   (int)s.in, (int)b.rank, (int)b.adapters, per, nullptr, 0, 0};
}

// Z of one side in the forms wanted; shares of a split width go to `planes` and are
// joined, or left there for wide_kernel to add up where no form by rank row is wanted.
void run_low(const ecf8a_plan& p, const ecf8a_bank& b, const Pass& s, const Forms& forms, float* planes, hipStream_t st)
{
    const LowShape shape = low_shape(p, b.rank, s.in);
    const LowArgs A = low_args(view_of(p), b, s, forms, shape.shares > 1 ? planes : nullptr, (int)(4 / shape.tiles));
    launch_low_pass(A, b, s, dim3(p.max_chunks * (4 / shape.tiles), shape.shares, (forms.zr + 63) / 64), shape.tiles, st);
    if (shape.shares > 1 && forms.row) {
        const uint64_t quads = (uint64_t)p.max_slots * forms.zr / 4;
        join_kernel<<<dim3((uint32_t)((quads + kThreads - 1) / kThreads)), kThreads, 0, st>>>(planes, (int)shape.shares,
                                                                                            A.plan.head, forms);
    }
}

template <int TYPE, bool VEC, bool PLANES>
void launch_wide_z(const WideArgs& A, dim3 grid, hipStream_t st)
{
    if (A.zr <= 16) wide_kernel<TYPE, 0, VEC, PLANES><<<grid, kThreads, 0, st>>>(A);
    else if (A.zr <= 32) wide_kernel<TYPE, 1, VEC, PLANES><<<grid, kThreads, 0, st>>>(A);
    else if (A.zr <= 64) wide_kernel<TYPE, 2, VEC, PLANES><<<grid, kThreads, 0, st>>>(A);
    else wide_kernel<TYPE, -1, VEC, PLANES><<<grid, kThreads, 0, st>>>(A);
}

template <int TYPE, bool VEC>
void launch_wide(const WideArgs& A, dim3 grid, hipStream_t st)
{
    if (A.planes) launch_wide_z<TYPE, VEC, true>(A, grid, st);
    else launch_wide_z<TYPE, VEC, false>(A, grid, st);
}

WideArgs wide_args(const PlanView& view, const ecf8a_bank& b, const Pass& s, const Forms& forms, const float* planes, uint32_t shares)
{
    return WideArgs{view, forms.slot, planes, forms.plane, (int)shares, static_cast<const uint16_t*>(s.f2), b.ranks,
                    static_cast<const uint16_t*>(s.base), (int64_t)s.ld_base, static_cast<uint16_t*>(s.out),
                    (int64_t)s.ld_out, (int)s.width, (int)b.rank, forms.zr, (int)b.adapters,
                    (int)((s.width + 4 * kStrip - 1) / (4 * kStrip))};
}

void launch_wide_pass(const PlanView& view, const ecf8a_bank& b, const Pass& s, const Forms& forms, const float* planes,
                      uint32_t shares, uint32_t chunks, hipStream_t st)
{
    const WideArgs A = wide_args(view, b, s, forms, planes, shares);
    const dim3 grid((uint32_t)A.groups * chunks);
    const bool vec = vec_wide(s);
    if (b.type == ECF8A_BF16) vec ? launch_wide<kBf16, true>(A, grid, st) : launch_wide<kBf16, false>(A, grid, st);
    else vec ? launch_wide<kFp16, true>(A, grid, st) : launch_wide<kFp16, false>(A, grid, st);
}

// One direction, whichever way.  `forms.row` is written if it is given.
int run_pass(const ecf8a_plan& p, const ecf8a_bank& b, const Pass& s, Forms forms, float* planes, hipStream_t st)
{
    if (one_kernel(p.tokens, b)) {
        forms.slot = nullptr;
        return run_few(view_of(p), 4 * p.max_chunks, nullptr, 0, p.tokens, b, s, forms, st);
    }
    if (!s.out) forms.slot = nullptr;
    run_low(p, b, s, forms, planes, st);
    if (s.out) {
        const uint32_t shares = low_shape(p, b.rank, s.in).shares;
        launch_wide_pass(view_of(p), b, s, forms, shares > 1 && !forms.row ? planes : nullptr, shares, p.max_chunks, st);
    }
    return launch_status();
}

template <int TYPE, bool VEC>
void launch_factor(const FactorArgs& A, dim3 grid, hipStream_t st)
{
    if (A.zr <= 16) factor_kernel<TYPE, 1, 1, VEC><<<grid, kThreads, 0, st>>>(A);
    else if (A.zr <= 32) factor_kernel<TYPE, 2, 1, VEC><<<grid, kThreads, 0, st>>>(A);
    else factor_kernel<TYPE, 2, 2, VEC><<<grid, kThreads, 0, st>>>(A);
}

// Columns of a factor_kernel workgroup.
uint32_t factor_columns(int zr) { return zr <= 32 ? 4 * kStrip : 2 * kStrip; }

template <int TYPE, bool VEC>
void launch_both(const WideArgs& W, const FactorArgs& F, uint32_t wide_groups, uint32_t factor_groups, uint32_t across, hipStream_t st)
{
    const uint32_t grid = wide_groups + factor_groups;
    if (F.zr <= 16) wide_and_factor_kernel<TYPE, 0, 1, 1, VEC><<<grid, kThreads, 0, st>>>(W, F, factor_groups, across);
    else if (F.zr <= 32) wide_and_factor_kernel<TYPE, 1, 2, 1, VEC><<<grid, kThreads, 0, st>>>(W, F, factor_groups, across);
    else wide_and_factor_kernel<TYPE, 2, 2, 2, VEC><<<grid, kThreads, 0, st>>>(W, F, factor_groups, across);
}

// The factors' gradients; dx: its `wide` pass, if it is still to be done.
int run_factor(const ecf8a_plan& p, const ecf8a_bank& b, const FactorArgs& A, const WideArgs* dx, bool dx_vec, hipStream_t st)
{
    bool vec = true;
    for (const FactorSide& s : A.side) vec = vec && vec16(s.v, s.ldv) && vec16(s.grad, s.width);
    const uint32_t columns = factor_columns(A.zr), groups = A.groups + (A.side[1].stride + columns - 1) / columns;
    if (dx) {
        const bool both = vec && dx_vec;
        const uint32_t wide_groups = (uint32_t)dx->groups * p.max_chunks, factor_groups = groups * p.max_units;
        if (b.type == ECF8A_BF16)
            both ? launch_both<kBf16, true>(*dx, A, wide_groups, factor_groups, groups, st)
                 : launch_both<kBf16, false>(*dx, A, wide_groups, factor_groups, groups, st);
        else
            both ? launch_both<kFp16, true>(*dx, A, wide_groups, factor_groups, groups, st)
                 : launch_both<kFp16, false>(*dx, A, wide_groups, factor_groups, groups, st);
    } else if (p.tokens) {
        const dim3 grid(groups, p.max_units, (A.zr + 63) / 64);
        if (b.type == ECF8A_BF16) vec ? launch_factor<kBf16, true>(A, grid, st) : launch_factor<kBf16, false>(A, grid, st);
        else vec ? launch_factor<kFp16, true>(A, grid, st) : launch_factor<kFp16, false>(A, grid, st);
    }
    const uint32_t four = 4 * kThreads, first = (A.side[0].width + four - 1) / four, rest = (A.side[1].width + four - 1) / four;
    const dim3 grid(first + rest, b.rank, b.adapters);
    if (b.type == ECF8A_BF16)
        vec ? sum_kernel<kBf16, true><<<grid, kThreads, 0, st>>>(A, (int)first) : sum_kernel<kBf16, false><<<grid, kThreads, 0, st>>>(A, (int)first);
    else
        vec ? sum_kernel<kFp16, true><<<grid, kThreads, 0, st>>>(A, (int)first) : sum_kernel<kFp16, false><<<grid, kThreads, 0, st>>>(A, (int)first);
    return launch_status();
}

Forms forms_of(const ecf8a_plan& p, uint32_t rank, void* slot, void* row)
{
    const int zr = (int)z_rows(rank);
    return Forms{static_cast<uint16_t*>(slot), static_cast<uint16_t*>(row), (int64_t)p.max_slots * zr, zr};
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
        index, (int)index_bytes, (int)tokens, (int)adapters, waves, (int)p.unit_slots, view_of(p));
    const int rc = launch_status();
    if (rc == ECF8_OK) *plan = p;
    return rc;
}

extern "C" uint64_t ecf8a_hidden_bytes(const ecf8a_plan* plan, uint32_t rank)
{
    if (!plan_ok(plan) || rank < 1 || rank > ECF8A_MAX_RANK) return 0;
    return form_bytes(*plan, rank);
}

extern "C" uint64_t ecf8a_add_bytes(const ecf8a_plan* plan, const ecf8a_bank* b)
{
    if (!plan_ok(plan) || !b || b->rank < 1 || b->rank > ECF8A_MAX_RANK) return 0;
    if (one_kernel(plan->tokens, *b)) return 0;
    return form_bytes(*plan, b->rank) + low_bytes(*plan, b->rank, b->in_features) + 256;
}

extern "C" uint64_t ecf8a_grads_bytes(const ecf8a_plan* plan, const ecf8a_bank* b)
{
    if (!plan_ok(plan) || !b || b->rank < 1 || b->rank > ECF8A_MAX_RANK) return 0;
    const uint64_t lk = low_bytes(*plan, b->rank, b->in_features), ln = low_bytes(*plan, b->rank, b->out_features);
    const uint64_t parts = part_bytes(*plan, b->rank, b->in_features) + part_bytes(*plan, b->rank, b->out_features);
    const uint64_t low = lk > ln ? lk : ln;
    return 3 * form_bytes(*plan, b->rank) + (low > parts ? low : parts) + 256;
}

extern "C" int ecf8a_few(uint64_t tokens, const ecf8a_bank* bank)
{
    return bank && few(tokens, *bank) ? 1 : 0;
}

// The checks of x, base and out that both ways of adding share.
static int check_add(const ecf8a_bank* bank, const void* x, uint64_t ldx, uint32_t x_type, const float* x_scale,
                     const void* base, uint64_t ld_base, const void* out, uint64_t ld_out)
{
    if (!x || !out || !aligned(x, x_type == ECF8A_E4M3 ? 1 : 2) || !aligned(out, 2) || !aligned(base, 2) ||
        !aligned(x_scale, 4) || (base == out && ld_base != ld_out))
        return ECF8_ERR_ARG;
    if (ldx < bank->in_features || ld_out < bank->out_features || (base && ld_base < bank->out_features))
        return ECF8_ERR_SIZE;
    return ECF8_OK;
}

extern "C" uint64_t ecf8a_add_few_bytes(uint64_t tokens, const ecf8a_bank* b)
{
    if (!b || !few(tokens, *b) || one_kernel(tokens, *b)) return 0;
    return round_up(few_planes_at(tokens) + 4ull * few_shares(tokens, b->in_features) * kTile * tokens * z_rows(b->rank), 256);
}

extern "C" int ecf8a_add_few(const void* index, uint32_t index_bytes, uint64_t tokens, const ecf8a_bank* bank, const void* x,
                             uint64_t ldx, uint32_t x_type, const float* x_scale, const void* base, uint64_t ld_base,
                             void* out, uint64_t ld_out, void* workspace, uint64_t workspace_bytes, void* hip_stream)
{
    int rc = check_bank(bank);
    if (rc != ECF8_OK) return rc;
    if (x_type != bank->type && x_type != ECF8A_E4M3) return ECF8_ERR_UNSUPPORTED;
    if ((index_bytes != 4 && index_bytes != 8) || (tokens && !index) || !aligned(index, index_bytes)) return ECF8_ERR_ARG;
    if (!few(tokens, *bank)) return ECF8_ERR_SIZE;
    if (tokens == 0) return ECF8_OK;
    rc = check_add(bank, x, ldx, x_type, x_scale, base, ld_base, out, ld_out);
    if (rc != ECF8_OK) return rc;
    hipStream_t st = static_cast<hipStream_t>(hip_stream);
    const Pass s{x, ldx, x_type, x_scale, bank->down, bank->in_features, bank->up, bank->out_features, base, ld_base, out, ld_out};
    if (one_kernel(tokens, *bank))
        return run_few(PlanView{}, (uint32_t)tokens, index, index_bytes, tokens, *bank, s, Forms{}, st);
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < ecf8a_add_few_bytes(tokens, bank))
        return ECF8_ERR_WORKSPACE;
    const int zr = (int)z_rows(bank->rank);
    const Forms forms{nullptr, nullptr, (int64_t)kTile * (int64_t)tokens * zr, zr};
    const PlanView view = few_view(workspace, tokens);
    float* planes = reinterpret_cast<float*>(static_cast<char*>(workspace) + few_planes_at(tokens));
    const uint32_t shares = few_shares(tokens, s.in);
    LowArgs A = low_args(view, *bank, s, forms, planes, 1);
    A.index = index;
    A.index_bytes = (int)index_bytes;
    A.tokens = (int)tokens;
    launch_low_pass(A, *bank, s, dim3((uint32_t)tokens, shares), 1, st);
    launch_wide_pass(view, *bank, s, forms, planes, shares, (uint32_t)tokens, st);
    return launch_status();
}

extern "C" int ecf8a_add(const ecf8a_plan* plan, const ecf8a_bank* bank, const void* x, uint64_t ldx, uint32_t x_type,
                         const float* x_scale, const void* base, uint64_t ld_base, void* out, uint64_t ld_out,
                         void* hidden, void* workspace, uint64_t workspace_bytes, void* hip_stream)
{
    if (!plan_ok(plan)) return ECF8_ERR_ARG;
    int rc = check_bank(bank);
    if (rc != ECF8_OK) return rc;
    if (x_type != bank->type && x_type != ECF8A_E4M3) return ECF8_ERR_UNSUPPORTED;
    if (bank->adapters != plan->adapters || !aligned(hidden, 16)) return ECF8_ERR_ARG;
    if (plan->tokens == 0) return ECF8_OK;
    rc = check_add(bank, x, ldx, x_type, x_scale, base, ld_base, out, ld_out);
    if (rc != ECF8_OK) return rc;
    const uint64_t need = ecf8a_add_bytes(plan, bank);
    if (need && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return ECF8_ERR_WORKSPACE;
    char* w = static_cast<char*>(workspace);
    const Pass s{x, ldx, x_type, x_scale, bank->down, bank->in_features, bank->up, bank->out_features, base, ld_base, out, ld_out};
    return run_pass(*plan, *bank, s, forms_of(*plan, bank->rank, w, hidden),
                    need ? reinterpret_cast<float*>(w + form_bytes(*plan, bank->rank)) : nullptr,
                    static_cast<hipStream_t>(hip_stream));
}

extern "C" int ecf8a_grads(const ecf8a_plan* plan, const ecf8a_bank* bank, const void* dy, uint64_t ld_dy, const void* x,
                           uint64_t ldx, const void* hidden, const void* dx_base, uint64_t ld_dx_base, void* dx,
                           uint64_t ld_dx, void* d_down, void* d_up, void* workspace, uint64_t workspace_bytes,
                           void* hip_stream)
{
    if (!plan_ok(plan)) return ECF8_ERR_ARG;
    int rc = check_bank(bank);
    if (rc != ECF8_OK) return rc;
    if (bank->adapters != plan->adapters || !d_down != !d_up || !aligned(d_down, 2) || !aligned(d_up, 2))
        return ECF8_ERR_ARG;
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
    const uint64_t fb = form_bytes(*plan, bank->rank);
    void* const z_row = d_down ? w + fb : nullptr;
    float* const scratch = reinterpret_cast<float*>(w + 3 * fb);
    const Pass s{dy, ld_dy, bank->type, nullptr, bank->up, N, bank->down, K, dx_base, ld_dx_base, dx, ld_dx};
    const Forms zf = forms_of(*plan, bank->rank, w, z_row);
    // dx waits for the factors' launch where both are wanted and `wide` keeps the factor in registers.
    const bool later = plan->tokens && dx && d_down && bank->rank <= 64 && !one_kernel(plan->tokens, *bank);
    if (plan->tokens && (dx || d_down)) {
        if (later) run_low(*plan, *bank, s, zf, scratch, st);
        else rc = run_pass(*plan, *bank, s, zf, scratch, st);
        if (rc == ECF8_OK && d_down && !hidden) {
            const Pass h{x, ldx, bank->type, nullptr, bank->down, K, bank->up, N, nullptr, 0, nullptr, 0};
            rc = run_pass(*plan, *bank, h, forms_of(*plan, bank->rank, nullptr, w + 2 * fb), scratch, st);
        }
    }
    if (rc != ECF8_OK || !d_down) return rc;
    const Forms z = forms_of(*plan, bank->rank, nullptr, z_row);
    const uint64_t sk = round_up(K, kStrip), sn = round_up(N, kStrip);
    const uint16_t* h = static_cast<const uint16_t*>(hidden ? hidden : w + 2 * fb);
    float* const part_up = scratch + part_bytes(*plan, bank->rank, K) / 4;
    const uint64_t columns = factor_columns(z.zr);
    const FactorArgs A{view_of(*plan),
                       {{z.row, static_cast<const uint16_t*>(x), (int64_t)ldx, static_cast<uint16_t*>(d_down), scratch, (int)K, (int)sk},
                        {h, static_cast<const uint16_t*>(dy), (int64_t)ld_dy, static_cast<uint16_t*>(d_up), part_up, (int)N, (int)sn}},
                       bank->ranks, z.plane, (int)bank->rank, z.zr, (int)bank->adapters, (int)((sk + columns - 1) / columns)};
    const WideArgs W = wide_args(view_of(*plan), *bank, s, zf, nullptr, 1);
    return run_factor(*plan, *bank, A, later ? &W : nullptr, vec_wide(s), st);
}
