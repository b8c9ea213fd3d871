// ecf8x_stream.h -- the product of a few tokens with a weight that streams past them.
//
// What bounds it is the stream of weights from memory.  A workgroup takes
// R rows of the weight; both operands go from memory to LDS without
// passing registers, 64 KG bytes of each row a step, into STAGES buffers, so that
// all but one of them are on their way while one is multiplied.  (Loads to
// registers in the matrix instruction's own layout, 16 rows in a run of lanes, came
// at 2.2 to 2.9 TB/s; a run of lanes here reads whole rows.)  The waves stand in RG
// row groups of 16 RF rows and KG shares of the step: a wave reads one 16-byte unit
// of each of its rows a step, 16 values of E4M3 or a block of 32 in 4 bits, and
// widens it for two or four operands, which meet the tokens of all its row fragments.
// A step is 128 bytes of a row at least, a whole line: steps of 64 bytes with four waves
// and twice the stages took 52 us where these take 32 (32 tokens x 28672 x 8192).
//
// Weight rows are operand A and tokens operand B: lane (c, g) of a result holds
// token 16 m + c, rows 4 g .. 4 g + 3 of fragment f.
#ifndef ECF8X_STREAM_H
#define ECF8X_STREAM_H

#include "ecf8x_common.h"

namespace ecf8x {

constexpr int kThree = 6;                 // x as three bfloat16 rows, which add up to its float32 values

typedef __amdgpu_buffer_rsrc_t Rsrc;
typedef __attribute__((address_space(3))) void LdsMem;

// Every offset is inside the operand: the range is left open.
__device__ __forceinline__ Rsrc buffer_of(const void* p) { return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, ~0, 0x00020000); }

// The wave's number, known to be the same in all of its lanes.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// The value of the lane N on, of every 16 (0 past the last).
template <int N>
__device__ __forceinline__ float lane_on(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x100 + N, 0xF, 0xF, true));
}

// All but the newest LOADS loads have arrived, and every LDS access is done, in
// every wave of the workgroup.
template <int LOADS>
__device__ __forceinline__ void wait_and_meet()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(LOADS) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// TR: rows of tokens that a stage holds, 16 MF, or 4 or 8 where there are no more (lanes then share them).
// ROOM: KB of LDS for the stages; 0: half of a compute unit's, for two workgroups, where three stages fit in it (of tokens in three
// parts two: 128 experts of 4096 x 1024, 64 tokens, 313 us, and in all of it 348), else all.
template <int W, int X, int MF, int RG, int TR = 16 * MF, int ROOM = 0>
struct Stream {
    static constexpr int RF = 2, NW = 8, KG = NW / RG, kThreads = 64 * NW;
    static constexpr int R = 16 * RF * RG;                     // rows
    static constexpr int VALUES = W == kMx4 ? 32 : 16;         // of a 16-byte unit of weights
    static constexpr int STEP = 4 * KG * VALUES;               // values of a step
    static constexpr int WU = 4 * KG;                          // units of a weight row's step
    static constexpr int XU = X == kMx4 ? 4 * KG : (X == kThree ? 3 : 1) * STEP / 8;   // of a token's
    static constexpr int PLANE = X == kThree ? XU / 3 : XU;    // of one of its rows
    // Four token rows of three parts: columns 4 p .. 4 p + 3 of operand B hold part p of the rows, so that one instruction takes
    // all of a row's parts (the last four columns repeat the last part and are not used).
    static constexpr bool PACKED = X == kThree && TR == 4;
    static constexpr int kW = R * WU, kX = TR * XU;       // units of a stage
    static constexpr int kS = W == kMx4 ? R * KG : 0, kXS = X == kMx4 ? TR * KG : 0;   // dwords of scales
    static constexpr int kStage = 16 * (kW + kX) + 4 * (kS + kXS);
    // 8 KB of a workgroup's share are left to the callers.
    static constexpr int kFit = 72 * 1024 / kStage, kMost = 152 * 1024 / kStage,
                         kRoom = ROOM ? ROOM * 1024 / kStage : kFit >= (X == kThree ? 2 : 3) ? kFit : kMost,
                         STAGES = kRoom < 8 ? kRoom : 8;
    static constexpr int kSums = 16 * 64 * NW * RF * MF, kLds = STAGES * kStage > kSums ? STAGES * kStage : kSums;
    // Loads of a wave and a stage: the same in every wave, some with part of its lanes.
    static constexpr int kWaveX = kX / NW, kEachX = (kWaveX + 63) / 64;
    static constexpr int kLoads = kW / kThreads + (kS > 0) + kEachX + (kXS > 0);
    static constexpr int kAhead = (STAGES - 2) * kLoads;
    static_assert(RG * KG == NW && kW == 128 * NW && STAGES >= 2 && (TR == 16 * MF || (TR < 16 && MF == 1)) && kLds <= 152 * 1024 && kAhead < 64, "LDS and the load counter");
    static_assert(kX % NW == 0 && kXS / NW <= 64 && kS / NW <= 64 && kStage % 16 == 0, "waves stage alike");

    // Lanes of a wave that send for its token unit i.
    static __device__ __forceinline__ int lanes_of(int i) { return kWaveX - 64 * i < 64 ? kWaveX - 64 * i : 64; }

    // Where unit u of a row of `units` lies, so that 16 rows' units of one number fall in different banks.
    template <int UNITS>
    static __device__ __forceinline__ int turn(int row)
    {
        static_assert(UNITS == 8 || UNITS % 16 == 0, "whole turns");
        return UNITS == 8 ? row >> 1 & 7 : row & 15;
    }

    // The same for a token row, which place p of it says to which part it belongs.
    static __device__ __forceinline__ int turn_x(int row, int p) { return PACKED ? row | p / PLANE << 2 : turn<XU>(row); }

    // The unit of a token row that lies at place p: where a lane group has four neighbouring units, places are numbered
    // so that the groups' places of one read are neighbours, which the lanes of one cycle spread over all banks.
    static constexpr bool FOURS = W == kMx4 && (X == kBf16 || X == kThree);
    static __device__ __forceinline__ int token_unit(int p) { return FOURS ? (p & ~15) | (p & 3) << 2 | (p >> 2 & 3) : p; }

    // The rows that this wave sends for, 16 RF / KG of them: its fragment's first row, and the last that exists
    // from there on.
    struct Rows {
        const uint8_t *codes, *scales;
        int last;
    };

    // Fragment of the rows that wave w stages, in the order [row group][fragment].
    static __device__ __forceinline__ int fragment(int w) { return w * (R / NW) / 16; }

    struct Places {
        Rsrc w, s, x, xs;
        uint32_t at_w[2], at_s, at_x[kEachX], at_xs;
    };

    // token(i): byte offset of token row i (0 .. TR - 1) from x, for kMx4 its number.  plane: bytes from one of its three rows
    // to the next.
    template <class Token>
    static __device__ __forceinline__ Places places(const Rows& rows, uint32_t row_bytes, uint32_t row_scales, const void* x, const void* x_scales,
                                                    uint32_t plane, Token token)
    {
        const int lane = threadIdx.x & 63, wave = wave_id();
        Places p;
        p.w = buffer_of(rows.codes);
        p.s = buffer_of(rows.scales);
        p.x = buffer_of(x);
        p.xs = buffer_of(x_scales);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = wave * 128 + i * 64 + lane, row = u / WU, local = row % 16;
            p.at_w[i] = (uint32_t)min(local, rows.last) * row_bytes + 16 * ((u % WU) ^ turn<WU>(row));
        }
        p.at_s = p.at_xs = 0;
        if constexpr (W == kMx4) {
            const int d = wave * 32 + (lane & 31), row = d / KG;
            p.at_s = (uint32_t)min(row % 16, rows.last) * row_scales + 4 * (d % KG);
        }
#pragma unroll
        for (int i = 0; i < kEachX; ++i) {
            const int u = wave * kWaveX + i * 64 + lane % lanes_of(i), row = u / XU;
            const int unit = token_unit((u % XU) ^ turn_x(row, u % XU));
            if constexpr (X == kMx4) p.at_x[i] = (uint32_t)token(row) * row_bytes + 16 * unit;
            else p.at_x[i] = (uint32_t)token(row) + unit / PLANE * plane + 16 * (unit % PLANE);
        }
        if constexpr (X == kMx4) {
            const int d = wave * (kXS / NW) + lane % (kXS / NW);
            p.at_xs = (uint32_t)token(d / KG) * row_scales + 4 * (d % KG);
        }
        return p;
    }

    static __device__ __forceinline__ void stage(const Places& p, int step, char* buf)
    {
        const int lane = threadIdx.x & 63, wave = wave_id();
        u32x4 *lw = reinterpret_cast<u32x4*>(buf), *lx = lw + kW;
        uint32_t *ls = reinterpret_cast<uint32_t*>(lx + kX), *lxs = ls + kS;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(p.w, (LdsMem*)(lw + wave * 128 + i * 64), 16, p.at_w[i], step * 16 * WU, 0, 2);
        if constexpr (W == kMx4) {
            if (lane < 32) __builtin_amdgcn_raw_ptr_buffer_load_lds(p.s, (LdsMem*)(ls + wave * 32), 4, p.at_s, step * 4 * KG, 0, 0);
        }
        const int bytes = X == kMx4 ? 16 * WU : 2 * STEP;      // of a token's plane
#pragma unroll
        for (int i = 0; i < kEachX; ++i)
            if (lanes_of(i) == 64 || lane < lanes_of(i))
                __builtin_amdgcn_raw_ptr_buffer_load_lds(p.x, (LdsMem*)(lx + wave * kWaveX + i * 64), 16, p.at_x[i], step * bytes, 0, 0);
        if constexpr (X == kMx4) {
            if (lane < kXS / NW) __builtin_amdgcn_raw_ptr_buffer_load_lds(p.xs, (LdsMem*)(lxs + wave * (kXS / NW)), 4, p.at_xs, step * 4 * KG, 0, 0);
        }
    }

    // The step where the reduction of `cols` values ends: zeros past it.  The places are byte offsets already; the value
    // that a unit begins with tells whether it is in.
    static __device__ __forceinline__ void stage_tail(const Places& p, const Rows& rows, const void* x, const void* x_scales, int step, int cols,
                                                      char* buf)
    {
        const int lane = threadIdx.x & 63, wave = wave_id(), left = cols - step * STEP;
        u32x4 *lw = reinterpret_cast<u32x4*>(buf), *lx = lw + kW;
        uint32_t *ls = reinterpret_cast<uint32_t*>(lx + kX), *lxs = ls + kS;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int u = wave * 128 + i * 64 + lane, unit = (u % WU) ^ turn<WU>(u / WU);
            u32x4 v{0, 0, 0, 0};
            if (unit * VALUES < left) v = *reinterpret_cast<const u32x4*>(rows.codes + p.at_w[i] + step * 16 * WU);
            lw[u] = v;
        }
        if constexpr (W == kMx4) {
            const int d = wave * 32 + lane;
            if (lane < 32) ls[d] = 128 * (d % KG) < left ? *reinterpret_cast<const uint32_t*>(rows.scales + p.at_s + step * 4 * KG) : 0;
        }
        const int bytes = X == kMx4 ? 16 * WU : 2 * STEP;
#pragma unroll
        for (int i = 0; i < kEachX; ++i) {
            const int u = wave * kWaveX + i * 64 + lane, unit = token_unit((u % XU) ^ turn_x(u / XU, u % XU)) % PLANE;
            if (lane >= lanes_of(i)) break;
            u32x4 v{0, 0, 0, 0};
            if (unit * (X == kMx4 ? 32 : 8) < left) v = *reinterpret_cast<const u32x4*>(static_cast<const char*>(x) + p.at_x[i] + step * bytes);
            lx[u] = v;
        }
        if constexpr (X == kMx4) {
            const int d = wave * (kXS / NW) + lane;
            if (lane < kXS / NW)
                lxs[d] = 128 * (d % KG) < left ? *reinterpret_cast<const uint32_t*>(static_cast<const char*>(x_scales) + p.at_xs + step * 4 * KG) : 0;
        }
    }

    // What a wave reads of a stage.
    struct Operands {
        static constexpr int OPS = X == kMx4 ? 1 : VALUES / 8;
        // float16 tokens and 4-bit weights: a block's power of two need not fit float16, so each instruction takes one
        // block of 32 (lane group g its values 8 g ..), unscaled, and its result is scaled, exactly, as it is added.
        static constexpr bool BLOCKS = X == kFp16 && W == kMx4;
        static constexpr int PLANES = PACKED ? 1 : XU / PLANE;     // of an operand's column
        u32x4 w[RF], x[MF][OPS][PLANES];
        uint32_t sw[RF], sx[MF];                       // BLOCKS: sw[0], of row 4 g + c % 4 of fragment c / 4 % 2

        __device__ __forceinline__ void read(const char* buf)
        {
            const int lane = threadIdx.x & 63, wave = wave_id(), c = lane & 15, g = lane >> 4, rg = wave % RG, q = wave / RG;
            const u32x4 *lw = reinterpret_cast<const u32x4*>(buf), *lx = lw + kW;
            const uint32_t *ls = reinterpret_cast<const uint32_t*>(lx + kX), *lxs = ls + kS;
#pragma unroll
            for (int f = 0; f < RF; ++f) {
                const int row = (rg * RF + f) * 16 + c;
                if constexpr (BLOCKS) {
                    if (f == 0) sw[0] = ls[((rg * RF + (c >> 2 & 1)) * 16 + 4 * g + (c & 3)) * KG + q];
                } else {
                    w[f] = lw[row * WU + ((4 * q + g) ^ turn<WU>(row))];
                    if constexpr (W == kMx4) sw[f] = ls[row * KG + q];
                }
            }
            // In the order in which the products take them, which begin with the first.
#pragma unroll
            for (int j = 0; j < OPS; ++j) {
                if constexpr (BLOCKS) {
#pragma unroll
                    for (int f = 0; f < RF; ++f) {
                        const int row = (rg * RF + f) * 16 + c;
                        w[f][j] = reinterpret_cast<const uint32_t*>(lw + row * WU + ((4 * q + j) ^ turn<WU>(row)))[g];
                    }
                }
#pragma unroll
                for (int m = 0; m < MF; ++m) {
                    const int row = (16 * m + c) % TR, unit = BLOCKS || FOURS ? (4 * q + j) * 4 + g : (4 * q + g) * OPS + j;
#pragma unroll
                    for (int p = 0; p < PLANES; ++p) {
                        const int place = (PACKED ? min(c >> 2, 2) : p) * PLANE + unit;
                        x[m][j][p] = lx[row * XU + (place ^ turn_x(row, place))];
                    }
                    if constexpr (X == kMx4) sx[m] = lxs[row * KG + q];
                }
            }
        }

        // 16-bit operands are of x's type, or bfloat16 where x is split.
        __device__ __forceinline__ void multiply(f32x4 (*acc)[MF])
        {
            const int g = threadIdx.x >> 4 & 3;
            if constexpr (X == kMx4) {
#pragma unroll
                for (int m = 0; m < MF; ++m)
#pragma unroll
                    for (int f = 0; f < RF; ++f) acc[f][m] = mfma_mx4<0>(w[f], x[m][0][0], acc[f][m], sw[f] >> (8 * g), sx[m] >> (8 * g));
            } else if constexpr (BLOCKS) {
                // A block's sums are added while the next block's are made.
                f32x4 sums[2][RF][MF];
                float scale[2];
                static_assert(RF == 2, "eight rows of a group");
#pragma unroll
                for (int j = 0; j < 5; ++j) {
                    if (j < 4) {
#pragma unroll
                        for (int f = 0; f < RF; ++f) {
                            const u32x4 wide = widen4_f16(w[f][j]);
#pragma unroll
                            for (int m = 0; m < MF; ++m) sums[j & 1][f][m] = mfma_f16(wide, x[m][j][0], f32x4{0, 0, 0, 0});
                        }
                        scale[j & 1] = value_of(scale_at(sw[0], j));
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (j > 0) {
#pragma unroll
                        for (int m = 0; m < MF; ++m) {
                            acc[0][m] = add_scaled<0>(acc[0][m], sums[~j & 1][0][m], scale[~j & 1]);
                            acc[1][m] = add_scaled<1>(acc[1][m], sums[~j & 1][1][m], scale[~j & 1]);
                        }
                    }
                }
            } else {
                constexpr int TYPE = X == kFp16 ? kFp16 : kBf16;
                float scale[RF];
#pragma unroll
                for (int f = 0; f < RF; ++f) scale[f] = W == kMx4 ? scale_of(sw[f] >> (8 * g)) : 1.0f;
#pragma unroll
                for (int j = 0; j < OPS; ++j) {
                    u32x4 wide[RF];
#pragma unroll
                    for (int f = 0; f < RF; ++f) {
                        if constexpr (W == kMx4) wide[f] = widen4(w[f][j], scale[f]);
                        else wide[f] = widen8<TYPE>(w[f][2 * j], w[f][2 * j + 1]);
                    }
#pragma unroll
                    for (int m = 0; m < MF; ++m)
#pragma unroll
                        for (int p = 0; p < PLANES; ++p)
#pragma unroll
                            for (int f = 0; f < RF; ++f) acc[f][m] = mfma<TYPE>(wide[f], x[m][j][p], acc[f][m]);
                }
            }
        }
    };

    // The buffers are told apart by __restrict__: else every LDS read waits for the loads to LDS in flight.
    static __device__ __forceinline__ void stage_and_multiply(const Places& p, int later, char* __restrict__ to, const char* __restrict__ from,
                                                              f32x4 (*acc)[MF])
    {
        stage(p, later, to);
        __builtin_amdgcn_sched_barrier(0);                     // loads leave before the products that hide them
        Operands now;
        now.read(from);
        now.multiply(acc);
    }

    // The reduction of `cols` values from step 0 of the places; every wave of the workgroup.  Afterwards the waves with q = wave / RG = 0 hold
    // the sums of row group wave % RG, and LDS may be used again after a barrier.
    static __device__ __forceinline__ void run(const Rows& rows, const Places& p, const void* x, const void* x_scales, int cols, char* lds,
                                               f32x4 (*acc)[MF])
    {
        const int steps = cols / STEP, wave = wave_id(), lane = threadIdx.x & 63;
        // At the end of step s the stage of step s + 1 has to be there, and only those behind it may be under way.  Steps
        // past the last are replaced by the last, so that this count holds in every step.
        if (steps > 0) {
#pragma unroll
            for (int s = 0; s < STAGES - 1; ++s) stage(p, min(s, steps - 1), lds + s * kStage);
            wait_and_meet<kAhead>();
        }
        int use = 0, fill = STAGES - 1;
        for (int s = 0; s < steps; ++s) {
            stage_and_multiply(p, min(s + STAGES - 1, steps - 1), lds + fill * kStage, lds + use * kStage, acc);
            wait_and_meet<kAhead>();
            use = use == STAGES - 1 ? 0 : use + 1;
            fill = fill == STAGES - 1 ? 0 : fill + 1;
        }
        wait_and_meet<0>();                                    // no load to LDS is under way from here on
        if (steps * STEP < cols) {
            stage_tail(p, rows, x, x_scales, steps, cols, lds);
            wait_and_meet<0>();
            Operands now;
            now.read(lds);
            now.multiply(acc);
            wait_and_meet<0>();
        }
        f32x4* sums = reinterpret_cast<f32x4*>(lds);           // [wave][RF][MF][lane]
        if (wave >= RG) {
#pragma unroll
            for (int f = 0; f < RF; ++f)
#pragma unroll
                for (int m = 0; m < MF; ++m) sums[((wave * RF + f) * MF + m) * 64 + lane] = acc[f][m];
        }
        __syncthreads();
        if (wave < RG) {
#pragma unroll
            for (int f = 0; f < RF; ++f)
#pragma unroll
                for (int m = 0; m < MF; ++m)
#pragma unroll
                    for (int q = 1; q < KG; ++q) acc[f][m] += sums[(((q * RG + wave) * RF + f) * MF + m) * 64 + lane];
            if constexpr (PACKED) {
#pragma unroll
                for (int f = 0; f < RF; ++f) {
                    const f32x4 v = acc[f][0];
                    acc[f][0] = f32x4{v[0] + (lane_on<4>(v[0]) + lane_on<8>(v[0])), v[1] + (lane_on<4>(v[1]) + lane_on<8>(v[1])),
                                      v[2] + (lane_on<4>(v[2]) + lane_on<8>(v[2])), v[3] + (lane_on<4>(v[3]) + lane_on<8>(v[3]))};
                }
            }
        }
    }
};

}  // namespace ecf8x

#endif
