// Device building blocks of the bf16 products' tiles: matrix-instruction
// fragments from stages that hold rows or summed steps, the multiplication of a
// stage, and results that trade places for whole cache lines.
//
// v_mfma_f32_16x16x32_bf16 on 16 channels (first operand) x 16 rows: lane l holds
// of each operand summed channels 8 (l / 16) .. + 7 of row (channel) l % 16, and
// of the result row l % 16, channels 4 (l / 16) + j in register j.
// (v_mfma_f32_32x32x16_bf16, with half the operand reads, was 8 to 13% slower at
// many rows: the chip lowers its clock to stay within its power.)
#pragma once

#include "moe_tiles.h"

namespace moe {
namespace tile {
namespace train {

// A block's tile: BM rows x BN channels on WR x WC waves of MT x NF fragments, STEP
// summed channels a stage, STAGES stages in LDS.
template <int BM_, int BN_, int WR_, int WC_, int STEP_, int STAGES_>
struct TileShape {
    static constexpr int BM = BM_, BN = BN_, WR = WR_, WC = WC_, kStep = STEP_, kStages = STAGES_;
    static constexpr int kWaves = WR * WC, kThreads = kWaves * kWave;
    static constexpr int MT = BM / 16 / WR, NF = BN / 16 / WC;
    static constexpr int kHalves = kStep / 32;                    // matrix instructions deep
    static constexpr int kRow = kStep * 2;                        // bytes of a row
    static constexpr int kW = BM * kRow, kBytes = kW + BN * kRow;  // a stage: rows, then channels
    static constexpr int kA = kW / 1024 / kWaves, kB = BN * kRow / 1024 / kWaves;  // a wave's loads of a stage
    static constexpr int kLoads = kA + kB;
};

// The stages of a block: separate variables, so that the compiler knows which
// reads follow which loads.
struct Stages {
    uint8_t *s0, *s1, *s2, *s3;
};

// ---- an operand whose rows hold what is summed over, 128 or 64 bytes of it ------------
//
// 16-byte piece c of a row sits at position c ^ (row / (16 / pieces) % pieces) in
// LDS: 16 rows, which are read at once, then cover all banks (256 bytes).  A load has
// 1 KB: lane l holds position l % pieces of row l / pieces; the waves load adjacent
// rows.

template <typename S>
struct RowPlaces {
    static constexpr int kPieces = S::kRow / 16;
    static constexpr int kPass = kWave / kPieces * S::kWaves;  // rows that the waves load at once
    static __device__ __forceinline__ int swizzle(int row) { return row / (16 / kPieces) & (kPieces - 1); }
    // This lane's row in a pass, and its first summed channel.
    static __device__ __forceinline__ int row(int wave, int lane) { return kWave / kPieces * wave + lane / kPieces; }
    static __device__ __forceinline__ int channel(int wave, int lane)
    {
        return ((lane & (kPieces - 1)) ^ swizzle(row(wave, lane))) * 8;
    }
    // This lane's place in a fragment's rows; the step's second half: ^ 64.
    static __device__ __forceinline__ int read(int lane)
    {
        const int r = lane & 15;
        return r * S::kRow + (((lane >> 4) ^ swizzle(r)) * 16);
    }
};

// ---- an operand whose rows are the summed steps, 256 or 128 channels of them -----------
//
// 32 bytes (16 channels) c of step s sit at position c ^ (s % 4 + s / 8 % 2 * 4):
// what 32 lanes read at once then covers all banks.  A load has 1 KB, two or four steps.
// ds_read_b64_tr_b16 hands each of 16 lanes 4 steps of one of 16 channels.

template <int COLS>
struct StepPlaces {
    static constexpr int kLanes = COLS / 8, kSteps = kWave / kLanes;  // lanes of a step, steps of a load
    static __device__ __forceinline__ int swizzle(int s) { return (s & 3) | ((s >> 1) & 4); }
    // This lane's step and channel in load n.
    static __device__ __forceinline__ int step(int n, int lane) { return kSteps * n + lane / kLanes; }
    static __device__ __forceinline__ int channel(int n, int lane)
    {
        return ((((lane & (kLanes - 1)) >> 1) ^ swizzle(step(n, lane))) * 2 + (lane & 1)) * 8;
    }
    // This lane's place in a fragment's first step; fragment f: ^ 32 f.
    static __device__ __forceinline__ int read(int lane)
    {
        const int s = 8 * (lane >> 4) + ((lane >> 2) & 3);
        return s * 2 * COLS + swizzle(s) * 32 + (lane & 3) * 8;
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// 16 channels of 32 steps from `at`, this lane's place in the first.
template <int COLS>
__device__ __forceinline__ dev::bf16x8 read_steps(const uint8_t *at)
{
    const auto four = [](const uint8_t *p) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
    };
    const s16x4 lo = four(at), hi = four(at + 8 * COLS);
    return __builtin_bit_cast(dev::bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ---- multiplication ------------------------------------------------------------------------

// The fragments of half a step (32 summed channels).
template <typename S, int MT>
struct Fragments {
    dev::bf16x8 x[MT], w[S::NF];
};

// Fragment number N of half h of a stage, in the order that multiply() needs them.
template <int N, typename S, int MT, typename Reads>
__device__ __forceinline__ void read_fragment(Fragments<S, MT> &to, const uint8_t *st, int h, const Reads &reads)
{
    if constexpr (N < S::NF)
        to.w[N] = reads.w(st, N, h);
    else
        to.x[N - S::NF] = reads.x(st, N - S::NF, h);
}

// acc += w x where the sum is.  In assembly because the compiler, left to choose the
// result's registers, moves sums about once they fill the accumulators (500 moves in a
// loop of 256 matrix instructions).  It does not know of the waits that these need:
// before a sum is read or moved, which end_turn() has, and two cycles after a vector
// instruction wrote an operand.  Operands come from LDS, whose loads the compiler
// waits for; a test of the compiled code looks for anything else that writes them (the
// wait beside each of these instead cost 4 to 7%).
__device__ __forceinline__ void mfma_in_place(dev::f32x4 &acc, const dev::bf16x8 &w, const dev::bf16x8 &x)
{
    asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0"
        : "+a"(acc)
        : "v"(__builtin_bit_cast(dev::u32x4, w)), "v"(__builtin_bit_cast(dev::u32x4, x)));
}

// The same for a sum outside the accumulators, and w from anywhere.
__device__ __forceinline__ void mfma_beside(dev::f32x4 &sum, const dev::bf16x8 &w, const dev::bf16x8 &x)
{
    asm("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0"
        : "+v"(sum)
        : "v"(__builtin_bit_cast(dev::u32x4, w)), "v"(__builtin_bit_cast(dev::u32x4, x)));
}

// The end of a loop of them: when it is the last turn (at >= end, uniform), the wait
// before a sum is read or moved (at most 19 cycles).  It has to stand here, in one
// piece with the loop: the compiler may move sums as soon as the loop is left.
__device__ __forceinline__ void end_turn(int at, int end)
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_cmp_lt_i32 %0, %1\n\ts_cbranch_scc1 .Lturn%=\n\ts_nop 15\n\ts_nop 7\n.Lturn%=:" ::"s"(at), "s"(end)
                 : "scc", "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// acc += half a step that is in registers, while half h of the stage `st` is read
// into `next` and, with LOAD, step `kb_load` loads into the stage `free`.  One wave
// has the SIMD: what is issued between two matrix instructions has to fit beside
// one, so reads and loads stand one by one among them, the reads first (loads all
// at once in the first half: 12% slower).  extra(i): more to do after row fragment i.
template <bool LOAD, typename S, int MT, typename Reads, typename Loads, typename Extra>
__device__ __forceinline__ void multiply(dev::f32x4 (&acc)[S::NF][MT], const Fragments<S, MT> &now, Fragments<S, MT> &next,
                                         const uint8_t *st, int h, const Reads &reads, const Loads &loads, uint8_t *free,
                                         int kb_load, const Extra &extra)
{
    constexpr int kAll = MT * S::NF, kReads = MT + S::NF, kGap = kAll / kReads > 3 ? 3 : kAll / kReads;
    for_each<kAll>([&](auto Q) {
        constexpr int q = decltype(Q)::value, i = q / S::NF, f = q % S::NF;
        if constexpr (q % kGap == 0 && q / kGap < kReads)
            read_fragment<q / kGap, S, MT>(next, st, h, reads);
        if constexpr (LOAD)
            loads.template issue<q * S::kLoads / kAll, (q + 1) * S::kLoads / kAll>(free, kb_load);
        mfma_in_place(acc[f][i], now.w[f], now.x[i]);
        if constexpr (f == S::NF - 1)
            extra(std::integral_constant<int, i>());
        __builtin_amdgcn_sched_barrier(0);
    });
}

// acc += the stage `st`, two waves per SIMD: fragments are read as they are needed,
// while step `kb_load` loads into the stage `free`.  extra(i, x): more to do after row
// fragment i, whose halves are x.
template <typename S, int MT, typename Reads, typename Loads, typename Extra>
__device__ __forceinline__ void multiply_stage(dev::f32x4 (&acc)[S::NF][MT], const uint8_t *st, const Reads &reads,
                                               const Loads &loads, uint8_t *free, int kb_load, const Extra &extra)
{
    constexpr int H = S::kHalves;
    dev::bf16x8 w[S::NF][H], x[2][H];
    for_each<S::NF>([&](auto F) {
        constexpr int f = decltype(F)::value;
        for_each<H>([&](auto N) { w[f][decltype(N)::value] = reads.w(st, f, decltype(N)::value); });
        if constexpr (f == 0)
            for_each<H>([&](auto N) { x[0][decltype(N)::value] = reads.x(st, 0, decltype(N)::value); });
    });
    for_each<MT>([&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (i + 1 < MT)
            for_each<H>([&](auto N) { x[(i + 1) & 1][decltype(N)::value] = reads.x(st, i + 1, decltype(N)::value); });
        for_each<H * S::NF>([&](auto Q) {
            constexpr int h = decltype(Q)::value / S::NF, f = decltype(Q)::value % S::NF;
            acc[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[f][h], x[i & 1][h], acc[f][i], 0, 0, 0);
        });
        extra(I, x[i & 1]);
        loads.template issue<i * S::kLoads / MT, (i + 1) * S::kLoads / MT>(free, kb_load);
        __builtin_amdgcn_sched_barrier(0);
    });
}

template <int NF, int MT>
__device__ __forceinline__ void clear(dev::f32x4 (&acc)[NF][MT])
{
    for_each<NF * MT>([&](auto N) {
        constexpr int n = decltype(N)::value;
        acc[n / MT][n % MT] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    });
}

// ---- results --------------------------------------------------------------------------------

constexpr int kStreamed = 2;  // stores marked non-temporal: L2 stays with the operands

// Two fragments' 16 rows x 32 channels as bf16, 8 adjacent channels per lane: row
// lane % 16, channels (g & 1) * 16 + (g >> 1) * 8 .. + 7, g = lane / 16.
__device__ __forceinline__ dev::u32x4 to_lanes(const dev::f32x4 &a, const dev::f32x4 &b)
{
    const auto lo = __builtin_amdgcn_permlane16_swap(dev::pack_bf16(a[0], a[1]), dev::pack_bf16(b[0], b[1]), false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(dev::pack_bf16(a[2], a[3]), dev::pack_bf16(b[2], b[3]), false, false);
    return dev::u32x4{lo[0], hi[0], lo[1], hi[1]};
}

// a and b += what to_lanes made of two fragments.
__device__ __forceinline__ void add_lanes(dev::f32x4 &a, dev::f32x4 &b, const dev::u32x4 &s)
{
    const auto lo = __builtin_amdgcn_permlane16_swap(s[0], s[2], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(s[1], s[3], false, false);
    a += dev::f32x4{dev::bf16_lo(lo[0]), dev::bf16_hi(lo[0]), dev::bf16_lo(hi[0]), dev::bf16_hi(hi[0])};
    b += dev::f32x4{dev::bf16_lo(lo[1]), dev::bf16_hi(lo[1]), dev::bf16_lo(hi[1]), dev::bf16_hi(hi[1])};
}

// Two vectors of one row, 64 channels with those of four lanes: after, the first
// is of row r % 8 and the second of row r % 8 + 8 (r = lane % 16), the lower lanes'
// (r < 8) the first 32 channels, the upper ones' the others: a store covers whole
// cache lines, 128 bytes of each of 8 rows.  Its own inverse.
__device__ __forceinline__ void trade_rows(dev::u32x4 &a, dev::u32x4 &b, bool low)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t other = __builtin_amdgcn_update_dpp(0, low ? b[j] : a[j], 0x128, 0xF, 0xF, true);
        a[j] = low ? a[j] : other;
        b[j] = low ? other : b[j];
    }
}

// Rows of `channels` bf16 in memory of which a tile's rows and a wave's channels are
// written or read: channels below `inside`, at c + shift.
struct Lines {
    __amdgpu_buffer_rsrc_t at;
    int32_t valid, inside, shift, channels;
    __device__ __forceinline__ uint32_t offset(int32_t row, int32_t c) const
    {
        return row < valid && c < inside ? ((uint32_t)row * (uint32_t)channels + c + shift) * 2 : 0x80000000u;
    }
};

// 16 rows x 64 channels (four fragments) from row0, c0 as bf16.
__device__ __forceinline__ void store_lines(const Lines &to, const dev::f32x4 &v0, const dev::f32x4 &v1,
                                            const dev::f32x4 &v2, const dev::f32x4 &v3, int row0, int32_t c0, int lane)
{
    const int r = lane & 15, g = lane >> 4;
    const bool low = r < 8;
    dev::u32x4 a = to_lanes(v0, v1), b = to_lanes(v2, v3);
    trade_rows(a, b, low);
    const int32_t c = c0 + (low ? 0 : 32) + (g & 1) * 16 + (g >> 1) * 8;
    __builtin_amdgcn_raw_buffer_store_b128(a, to.at, to.offset(row0 + (r & 7), c), 0, kStreamed);
    __builtin_amdgcn_raw_buffer_store_b128(b, to.at, to.offset(row0 + (r & 7) + 8, c), 0, kStreamed);
}

// 16 rows x 32 channels (two fragments) from row0, c0 of fp32 rows of `channels`;
// with ADD, added to what is there.
template <bool ADD>
__device__ __forceinline__ void store_wide(__amdgpu_buffer_rsrc_t to, const dev::f32x4 &v0, const dev::f32x4 &v1, int row0,
                                           int valid, int32_t c0, int32_t channels, int lane)
{
    const int r = lane & 15, g = lane >> 4;
    const bool low = r < 8;
    dev::u32x4 s[2] = {__builtin_bit_cast(dev::u32x4, v0), __builtin_bit_cast(dev::u32x4, v1)};
    trade_rows(s[0], s[1], low);
    const int32_t c = c0 + (low ? 0 : 16) + 4 * g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = row0 + (r & 7) + 8 * h;
        const uint32_t off = row < valid && c < channels ? ((uint32_t)row * (uint32_t)channels + c) * 4 : 0x80000000u;
        if constexpr (ADD)
            s[h] = __builtin_bit_cast(dev::u32x4, __builtin_bit_cast(dev::f32x4, s[h]) +
                                                      __builtin_bit_cast(dev::f32x4, __builtin_amdgcn_raw_buffer_load_b128(to, off, 0, 0)));
        __builtin_amdgcn_raw_buffer_store_b128(s[h], to, off, 0, kStreamed);
    }
}

// 16 rows x 32 channels (two fragments) as bf16: 64 bytes of a row.
__device__ __forceinline__ void store_pair(const Lines &to, const dev::f32x4 &v0, const dev::f32x4 &v1, int row0, int32_t c0,
                                           int lane)
{
    const int r = lane & 15, g = lane >> 4;
    const int32_t c = c0 + (g & 1) * 16 + (g >> 1) * 8;
    __builtin_amdgcn_raw_buffer_store_b128(to_lanes(v0, v1), to.at, to.offset(row0 + r, c), 0, kStreamed);
}

// Adds the bf16 that store_lines would overwrite to four fragments.
__device__ __forceinline__ void add_lines(const Lines &from, dev::f32x4 *v, int row0, int32_t c0, int lane)
{
    const int r = lane & 15, g = lane >> 4;
    const bool low = r < 8;
    const int32_t c = c0 + (low ? 0 : 32) + (g & 1) * 16 + (g >> 1) * 8;
    dev::u32x4 a = __builtin_amdgcn_raw_buffer_load_b128(from.at, from.offset(row0 + (r & 7), c), 0, 0);
    dev::u32x4 b = __builtin_amdgcn_raw_buffer_load_b128(from.at, from.offset(row0 + (r & 7) + 8, c), 0, 0);
    trade_rows(a, b, low);
    add_lanes(v[0], v[1], a);
    add_lanes(v[2], v[3], b);
}

}  // namespace train
}  // namespace tile
}  // namespace moe
