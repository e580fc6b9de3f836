// The gradient of the experts' products to their weights and biases on gfx950:
//
//   dw[e, j, c] = sum over rows of e of dy[row, j] a[row, c],  dbias[e, j] = sum of dy[row, j]
//
// A block holds 256 x 256 (or 128 x 256) of one expert's weights and walks its rows, 32 a step.
// Both operands are summed over their slow axis: the stages hold them as they lie
// in memory and ds_read_b64_tr_b16 hands each lane four rows of one channel.
// dbias comes from the same fragments, times ones.
//
// Bound by the matrix cores where a tile has many rows: 8192^3 740 us (1485 TFLOP/s), 32,768
// dense rows, 4096 x 7168 1391.  32 experts x 1024 rows, 4096 x 7168: 1820 us in bf16, 1940
// from 8-bit rows, 2150 with fp32 results: a tile is 32 steps long and its 128 or 256 kB of
// results, 1.9 or 3.8 GB in all, go out while nothing multiplies.  8191 rows, 768 x 2048: 35
// us for five parts and 8 to join them.
#include "moe_train_internal.h"
#include "moe_train_tiles.h"

namespace moe {

namespace {

using namespace tile;
using namespace tile::train;

// A tile's rows are channels of dy, its channels a's.
// Four waves, one per SIMD, each with 128 x 128; four stages.
using Weights256 = TileShape<256, 256, 2, 2, 32, 4>;
// Four waves with 64 x 128, two blocks per compute unit; three stages.
using Weights128 = TileShape<128, 256, 2, 2, 32, 3>;

// Tiles along dy's channels that walk a's together.  256 x 256, bf16 results, 4 / 5 / 6 / 8 of
// them: 32 experts x 1024 rows, 4096 x 7168 1889 / 1884 / 1885 / 1917 us, 2048 x 7168 967 / 954 /
// 963 / 982, 7168 x 2048 968 / 945 / 947 / 970; 8 experts x 4096 rows, 4096 x 4096 875 / 878 / 869 /
// 862; 32,768 dense rows, 4096 x 7168 1459 / 1482 / 1466 / 1458; 8192^3, fp32 813 / 815 / 812 / 809.
// 128 x 256, 32 experts, 4096 x 7168: 4 / 8 / 16 / 32 of them 2032 / 2007 / 1988 / 2052.
template <typename S>
constexpr int group_tiles() { return S::BM == 256 ? 5 : 16; }

struct WeightTile {
    int32_t e, split, mt, nt, rows;
    int64_t row0;
};

// 8 channels of four rows of a in 8 bits with their scales, on their way to a
// stage as bf16.
template <int QUANT>
struct Rows8 {
    dev::u32x2 v[4];
    uint32_t s[4];  // as they are stored

    __device__ __forceinline__ dev::u32x4 bf16(int i) const
    {
        dev::u32x4 out;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                const float f = __uint_as_float(s[i]);
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(v[i][j], false);
                const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(v[i][j], true);
                out[2 * j] = dev::pack_bf16(lo[0] * f, lo[1] * f);
                out[2 * j + 1] = dev::pack_bf16(hi[0] * f, hi[1] * f);
            } else {
                // the conversion takes the exponent field alone: 0 is 2^-127, 255 NaN
                const float f = __uint_as_float(s[i] << 23);
                out[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i][j], f, false));
                out[2 * j + 1] =
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i][j], f, true));
            }
        }
        return out;
    }
};
template <>
struct Rows8<MOE_QUANT_NONE> {};

// The loads of one tile.  Rows past the split's end lie past the buffers' ends and
// are read as zeros, and so are channels past the last.
template <typename S, int QUANT>
struct WeightLoads {
    static constexpr int kStep = S::kStep, kHalf = S::kW;
    using Dy = StepPlaces<S::BM>;
    using A = StepPlaces<S::BN>;
    static constexpr int kRowsPerPass = A::kSteps * S::kWaves;
    const uint16_t *dy;
    const uint8_t *a, *scale;
    uint32_t so, sstep, to;  // 8 bits: this lane's first scale, and its place in a stage
    uint32_t yo[2], ao[2];  // this lane's place in its first rows
    uint32_t ystep, astep;  // two passes of all waves further (a in 8 bits: one)
    int32_t rows, n, k, wave;

    __device__ __forceinline__ void set(const GradWeightArgs &p, const WeightTile &at, int wave_, int lane)
    {
        wave = wave_;
        lane = here(lane);
        rows = at.rows;
        n = p.n;
        k = p.k;
        dy = p.dy + at.row0 * n;
        a = static_cast<const uint8_t *>(p.a) + at.row0 * k * (QUANT == MOE_QUANT_NONE ? 2 : 1);
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {  // passes by turns
            const int u = wave + odd * S::kWaves;
            const int32_t j = at.mt * S::BM + Dy::channel(u, lane), i = at.nt * S::BN + A::channel(u, lane);
            yo[odd] = j < n ? (uint32_t)Dy::step(u, lane) * (uint32_t)n * 2 + (uint32_t)j * 2 : 0x80000000u;
            ao[odd] = i < k ? (uint32_t)A::step(u, lane) * (uint32_t)k * 2 + (uint32_t)i * 2 : 0x80000000u;
        }
        ystep = 4u * Dy::kSteps * S::kWaves * (uint32_t)n;
        astep = 4u * kRowsPerPass * (uint32_t)k;
        if constexpr (QUANT != MOE_QUANT_NONE) {
            const int s = A::step(wave, lane);
            const int32_t piece = lane & 31, at_c = at.nt * S::BN + piece * 8;
            ao[0] = at_c < k ? (uint32_t)s * (uint32_t)k + (uint32_t)at_c : 0x80000000u;
            astep = kRowsPerPass * (uint32_t)k;
            so = at_c < k ? (uint32_t)s * scale_bytes() + (uint32_t)(at_c / (QUANT == MOE_QUANT_MXFP8 ? 32 : 128)) *
                                                              (QUANT == MOE_QUANT_FP8_F32 ? 4 : 1)
                          : 0x80000000u;
            sstep = kRowsPerPass * scale_bytes();
            to = (uint32_t)s * 512 + (((piece >> 1) ^ A::swizzle(s)) * 2 + (piece & 1)) * 16;
            scale = static_cast<const uint8_t *>(p.a_scale) + at.row0 * scale_bytes();
        }
    }
    // Bytes of a row's scales.
    __device__ __forceinline__ uint32_t scale_bytes() const
    {
        const uint32_t b = (uint32_t)k / kQuantGroup;
        return QUANT == MOE_QUANT_FP8_UE8M0 ? (b + 3) / 4 * 4 : b * 4;
    }
    // a in 8 bits: pass i of step kb's rows into registers, and from there into a stage.
    __device__ __forceinline__ void fetch(Rows8<QUANT> &rows8, int i, int kb) const
    {
        const int32_t r0 = kb * kStep;
        const uint32_t left = (uint32_t)max(0, min(kStep, rows - r0));
        const __amdgpu_buffer_rsrc_t av = buffer(a + (int64_t)r0 * k, left * (uint32_t)k);
        const __amdgpu_buffer_rsrc_t sv = buffer(scale + (int64_t)r0 * scale_bytes(), left * scale_bytes());
        rows8.v[i] = __builtin_amdgcn_raw_buffer_load_b64(av, ao[0] + i * astep, 0, 0);
        if constexpr (QUANT == MOE_QUANT_FP8_F32)
            rows8.s[i] = __builtin_amdgcn_raw_buffer_load_b32(sv, so + i * sstep, 0, 0);
        else
            rows8.s[i] = __builtin_amdgcn_raw_buffer_load_b8(sv, so + i * sstep, 0, 0);
    }
    __device__ __forceinline__ void put(const Rows8<QUANT> &rows8, int i, uint8_t *st) const
    {
        // 8 rows further the swizzle's third bit turns
        static_assert(kRowsPerPass == 8, "rows of a pass");
        *reinterpret_cast<dev::u32x4 *>(st + kHalf + (to ^ (i & 1) * 128) + i * kRowsPerPass * 512) = rows8.bf16(i);
    }
    // Loads FROM .. TO - 1 of step kb (8 bits: dy's).
    template <int FROM, int TO>
    __device__ __forceinline__ void issue(uint8_t *st, int kb) const
    {
        const int32_t r0 = kb * kStep;
        const uint32_t left = (uint32_t)max(0, min(kStep, rows - r0));
        for_each<TO - FROM>([&](auto N) {
            constexpr int j = FROM + decltype(N)::value, i = j < S::kA ? j : j - S::kA;
            if constexpr (j < S::kA)
                load_lds<16>(buffer(dy + (int64_t)r0 * n, left * (uint32_t)n * 2), st + (wave + S::kWaves * i) * 1024,
                             yo[i & 1] + (i >> 1) * ystep, 0);
            else if constexpr (QUANT == MOE_QUANT_NONE)
                load_lds<16>(buffer(a + (int64_t)r0 * k * 2, left * (uint32_t)k * 2),
                             st + kHalf + (wave + S::kWaves * i) * 1024, ao[i & 1] + (i >> 1) * astep, 0);
        });
    }
};

template <typename S>
struct WeightReads {
    int row, column, m0, n0;
    __device__ __forceinline__ WeightReads(int wave, int lane)
    {
        row = StepPlaces<S::BM>::read(lane);
        column = StepPlaces<S::BN>::read(lane);
        m0 = wave / S::WC * S::MT;
        n0 = wave % S::WC * S::NF;
    }
    __device__ __forceinline__ dev::bf16x8 x(const uint8_t *st, int i, int) const
    {
        return read_steps<S::BM>(st + (row ^ (m0 + i) * 32));
    }
    __device__ __forceinline__ dev::bf16x8 w(const uint8_t *st, int f, int) const
    {
        return read_steps<S::BN>(st + S::kW + (column ^ (n0 + f) * 32));
    }
};

// The waves that share a row of fragments share its sums for the bias.
template <typename S>
constexpr int bias_sums() { return S::MT / S::WC; }

// Results: channels 16 (MT wr + i) .. of dy, 16 (NF wc + f) .. of a.  Parts of a
// split go to the workspace.
template <typename S>
__device__ __forceinline__ void write_weights(const GradWeightArgs &p, const dev::f32x4 (&acc)[S::NF][S::MT],
                                              const dev::f32x4 (&sums)[bias_sums<S>()], const WeightTile &at, int wr,
                                              int wc, int lane)
{
    constexpr int MT = S::MT, NF = S::NF;
    lane = here(lane);
    const int32_t j0 = at.mt * S::BM, c0 = at.nt * S::BN + wc * NF * 16;
    const int32_t valid = min(S::BM, p.n - j0);
    const bool parts = p.splits > 1;
    const int64_t group = parts ? (int64_t)at.e * p.splits + at.split : at.e;
    const int64_t first = (group * p.n + j0) * p.k;
    const int r = lane & 15, g = lane >> 4;
    if (!parts && p.dw_bf16) {
        const Lines out = {buffer(static_cast<uint16_t *>(p.dw) + first, (uint32_t)valid * (uint32_t)p.k * 2), valid, p.k, 0,
                           p.k};
        for_each<MT>([&](auto I) {
            constexpr int i = decltype(I)::value;
            for_each<NF / 4>([&](auto F) {
                constexpr int f = 4 * decltype(F)::value;
                store_lines(out, acc[f][i], acc[f + 1][i], acc[f + 2][i], acc[f + 3][i], (wr * MT + i) * 16, c0 + f * 16,
                            lane);
            });
            __builtin_amdgcn_sched_barrier(0);
        });
    } else {
        const __amdgpu_buffer_rsrc_t out =
            buffer((parts ? p.partial : static_cast<float *>(p.dw)) + first, (uint32_t)valid * (uint32_t)p.k * 4);
        const auto store = [&](auto add) {
            for_each<MT>([&](auto I) {
                constexpr int i = decltype(I)::value;
                for_each<NF / 2>([&](auto F) {
                    constexpr int f = 2 * decltype(F)::value;
                    store_wide<decltype(add)::value>(out, acc[f][i], acc[f + 1][i], (wr * MT + i) * 16, valid, c0 + f * 16, p.k,
                                                     lane);
                });
                __builtin_amdgcn_sched_barrier(0);
            });
        };
        if (!parts && p.accumulate)
            store(std::true_type());
        else
            store(std::false_type());
    }
    if (p.dbias != nullptr && at.nt == 0 && g == 0) {
        float *out = parts ? p.partial + (int64_t)p.E * p.splits * p.n * p.k : p.dbias;
#pragma unroll
        for (int b = 0; b < bias_sums<S>(); ++b) {
            const int row = (wr * MT + wc * bias_sums<S>() + b) * 16 + r;
            if (row < valid) {
                float *to = out + group * p.n + j0 + row;
                *to = !parts && p.accumulate ? *to + sums[b][0] : sums[b][0];
            }
        }
    }
}

// Sets of rows in 8 bits on their way.
template <typename S>
constexpr int rows8_sets() { return S::kStages == 4 ? 2 : 1; }

// The loads that a tile begins with: four stages, or two of three; of a in 8 bits the
// first one or two through registers.
template <typename S, int QUANT>
__device__ __forceinline__ void start_weights(const GradWeightArgs &p, const WeightTile &at, const Stages &st,
                                              Rows8<QUANT> (&rows8)[rows8_sets<S>()], int wave, int lane)
{
    WeightLoads<S, QUANT> loads;
    loads.set(p, at, wave, lane);
    if constexpr (QUANT != MOE_QUANT_NONE) {
#pragma unroll
        for (int u = 0; u < rows8_sets<S>(); ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                loads.fetch(rows8[u], i, u);
        __builtin_amdgcn_sched_barrier(0);
    }
    loads.template issue<0, S::kLoads>(st.s0, 0);
    __builtin_amdgcn_sched_barrier(0);  // in this order: the waits count
    loads.template issue<0, S::kLoads>(st.s1, 1);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (S::kStages == 4) {
        loads.template issue<0, S::kLoads>(st.s2, 2);
        __builtin_amdgcn_sched_barrier(0);
        loads.template issue<0, S::kLoads>(st.s3, 3);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// Multiplies a tile whose first loads are in flight, then starts the next tile's
// (`more`) and writes the results.
//
// a in 8 bits goes through registers.  Four stages: rows fetched in step u are put into
// their stage in step u + 2 and read in step u + 3; three: put in step u + 1, read in
// step u + 2.  Loads come back in order, so waiting for them sooner would wait for dy's
// too.
template <typename S, int QUANT, bool BIAS>
__device__ __forceinline__ void run_weights(const GradWeightArgs &p, const WeightTile &at, const WeightTile &next, bool more,
                                            const Stages &st, Rows8<QUANT> (&rows8)[rows8_sets<S>()], int wave, int lane)
{
    constexpr int MT = S::MT, NF = S::NF, kBias = bias_sums<S>();
    constexpr bool k8 = QUANT != MOE_QUANT_NONE;
    // a stage's loads that go to LDS, and the loads of a step
    constexpr int kDma = k8 ? S::kA : S::kLoads, kStepLoads = k8 ? kDma + 8 : kDma;
    WeightLoads<S, QUANT> loads;
    loads.set(p, at, wave, lane);
    const WeightReads<S> reads(wave, here(lane));
    const int wr = wave / S::WC, wc = wave % S::WC;
    const int KB = scalar((at.rows + S::kStep - 1) / S::kStep);
    dev::f32x4 acc[NF][MT], sums[kBias];
    clear(acc);
#pragma unroll
    for (int b = 0; b < kBias; ++b)
        sums[b] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (k8) {
#pragma unroll
        for (int u = 0; u < rows8_sets<S>(); ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                loads.put(rows8[u], i, u == 0 ? st.s0 : st.s1);
                loads.fetch(rows8[u], i, rows8_sets<S>() + u);
            }
        __builtin_amdgcn_sched_barrier(0);
    }
    const __bf16 one = (__bf16)1.0f;
    const dev::bf16x8 ones = {one, one, one, one, one, one, one, one};
    const auto add_bias = [&](const uint8_t *cur) {
        if constexpr (BIAS) {  // the waves of a row of fragments share its sums, read again
#pragma unroll
            for (int b = 0; b < kBias; ++b) {
                const dev::bf16x8 x = reads.x(cur, wc * kBias + b, 0);
                if constexpr (S::kStages == 4)
                    mfma_beside(sums[b], ones, x);  // the compiler would take accumulators for them
                else
                    sums[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, x, sums[b], 0, 0, 0);
            }
        }
    };
    // Whole rounds: steps past the last multiply zeros.  Ways out between the steps would
    // have the sums change registers where they meet.
    if constexpr (S::kStages == 4) {
        static_assert(MT == 8 && S::kHalves == 1, "four passes of a step's rows: put, then fetched");
        Fragments<S, MT> even, odd;
        wait_and_meet<3 * kDma>();
        for_each<MT + NF>([&](auto N) { read_fragment<decltype(N)::value, S, MT>(even, st.s0, 0, reads); });
        // cur: the stage of step kb, after: kb + 1, put: kb + 2
        const auto step = [&](Fragments<S, MT> &now, Fragments<S, MT> &then, Rows8<QUANT> &r8, uint8_t *cur, uint8_t *after,
                              uint8_t *put, int kb) {
            if constexpr (BIAS)
                add_bias(cur);
            wait_and_meet<2 * kStepLoads>();
            multiply<true, S, MT>(acc, now, then, after, 0, reads, loads, cur, kb + 4, [&](auto I) {
                constexpr int i = decltype(I)::value;
                if constexpr (k8 && i < 4)
                    loads.put(r8, i, put);
                if constexpr (k8 && i >= 4)
                    loads.fetch(r8, i - 4, kb + 4);
            });
        };
        for (int kb = 0; kb < KB; kb += 4) {
            step(even, odd, rows8[0], st.s0, st.s1, st.s2, kb);
            step(odd, even, rows8[1], st.s1, st.s2, st.s3, kb + 1);
            step(even, odd, rows8[0], st.s2, st.s3, st.s0, kb + 2);
            step(odd, even, rows8[1], st.s3, st.s0, st.s1, kb + 3);
            end_turn(kb + 4, KB);
        }
    } else {
        static_assert(MT == 4 && S::kHalves == 1, "a pass of a step's rows beside each row fragment");
        // cur: the stage of step kb, after: kb + 1, free: kb + 2
        // Bias sums: bf16 rows read their fragments again before the products; with the
        // registers that 8-bit rows take, the places they are read from would be spilled
        // in the loop, whose counted loads each reload waits for, so those use a fragment
        // where it is multiplied, in the wave that sums it.  Read again / in place: 8191
        // rows, 768 x 2048, UE8M0 90 / 59 us, fp32 scales 91 / 66, bf16 41 / 47; 8 experts
        // x 512 rows, 512 x 1024 26.4 / 22.3, 30.0 / 25.3, 16.0 / 18.2.
        const auto step = [&](uint8_t *cur, uint8_t *after, uint8_t *free, int kb) {
            wait_and_meet<kStepLoads>();
            if constexpr (!k8)
                add_bias(cur);
            multiply_stage<S, MT>(acc, cur, reads, loads, free, kb + 2, [&](auto I, const dev::bf16x8 (&x)[1]) {
                constexpr int i = decltype(I)::value;
                if constexpr (BIAS && k8)
                    if (i / kBias == wc)
                        sums[i % kBias] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, x[0], sums[i % kBias], 0, 0, 0);
                if constexpr (k8) {
                    loads.put(rows8[0], i, after);
                    loads.fetch(rows8[0], i, kb + 2);
                }
            });
        };
        for (int kb = 0; kb < KB; kb += 3) {
            step(st.s0, st.s1, st.s2, kb);
            step(st.s1, st.s2, st.s0, kb + 1);
            step(st.s2, st.s0, st.s1, kb + 2);
        }
    }
    wait_and_meet<0>();
    if (more)
        start_weights<S, QUANT>(p, next, st, rows8, wave, lane);
    write_weights<S>(p, acc, sums, at, wr, wc, lane);
}

template <typename S, int QUANT>
__global__ __launch_bounds__(S::kThreads, S::kStages == 4 ? 1 : 2) void grad_weight_tiles(GradWeightArgs p, int32_t m_tiles,
                                                                                        int32_t n_tiles)
{
    constexpr int kStep = S::kStep, kGroupM = group_tiles<S>();
    __shared__ alignas(1024) uint8_t st0[S::kBytes], st1[S::kBytes], st2[S::kBytes];
    __shared__ alignas(1024) uint8_t st3[S::kStages == 4 ? S::kBytes : 16];
    const Stages st = {st0, st1, st2, st3};
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = scalar(threadIdx.x / kWave);
    const int32_t tiles = m_tiles * n_tiles;
    const int64_t n_work = (int64_t)tiles * p.E * p.splits;
    const auto locate = [&](int64_t work) {
        WeightTile at;
        const int32_t part = scalar((int32_t)(work / tiles));
        const int32_t t = scalar((int32_t)(work - (int64_t)part * tiles));
        at.e = scalar(part / p.splits);
        at.split = scalar(part - at.e * p.splits);
        const int32_t grp = scalar(t / (kGroupM * n_tiles)), in_grp = scalar(t - grp * kGroupM * n_tiles);
        const int32_t wide = min(kGroupM, m_tiles - grp * kGroupM);
        at.nt = scalar(in_grp / wide);
        at.mt = scalar(grp * kGroupM + in_grp - at.nt * wide);
        const int32_t rows = p.recv_count != nullptr ? word_of(p.recv_count, at.e) : p.dense_rows;
        const int32_t steps = (rows + kStep - 1) / kStep;
        const int32_t s0 = scalar((int32_t)((int64_t)steps * at.split / p.splits));
        const int32_t s1 = scalar((int32_t)((int64_t)steps * (at.split + 1) / p.splits));
        at.rows = scalar(min(rows, s1 * kStep) - min(rows, s0 * kStep));
        at.row0 = (int64_t)(p.expert_offset != nullptr ? word_of(p.expert_offset, at.e) : 0) + (int64_t)s0 * kStep;
        return at;
    };
    // workgroups go to the 8 XCDs in turn: each XCD takes a contiguous run of
    // the work, so that the tiles of one expert share its L2
    const int64_t run = (n_work + 7) / 8;
    const int64_t base = (int64_t)(blockIdx.x & 7) * run;
    const int64_t end = min(run, n_work - base);
    int64_t idx = blockIdx.x >> 3;
    if (idx >= end)
        return;
    Rows8<QUANT> rows8[rows8_sets<S>()];
    WeightTile next = locate(base + idx);
    start_weights<S, QUANT>(p, next, st, rows8, wave, lane);
    for (;;) {
        const WeightTile at = next;
        idx += gridDim.x >> 3;
        const bool more = idx < end;
        if (more)
            next = locate(base + idx);
        if (p.dbias != nullptr && at.nt == 0)
            run_weights<S, QUANT, true>(p, at, next, more, st, rows8, wave, lane);
        else
            run_weights<S, QUANT, false>(p, at, next, more, st, rows8, wave, lane);
        if (!more)
            break;
    }
}

// dw and dbias from the parts of a split, added in order: 4 values per thread.
__global__ __launch_bounds__(kBlockThreads) void grad_weight_join(GradWeightArgs p, int64_t quads, int64_t all)
{
    const int64_t size = (int64_t)p.n * p.k, q = (int64_t)blockIdx.x * kBlockThreads + threadIdx.x;
    const bool bias = q >= quads;
    if (q >= all)
        return;
    const int64_t of = bias ? p.n : size;                    // values of a part
    const int64_t i = (bias ? q - quads : q) * 4;
    const int64_t e = i / of, at = i - e * of;
    const float *from = p.partial + (bias ? (int64_t)p.E * p.splits * size : 0) + e * p.splits * of + at;
    dev::f32x4 v = *reinterpret_cast<const dev::f32x4 *>(from);
    for (int s = 1; s < p.splits; ++s)
        v += *reinterpret_cast<const dev::f32x4 *>(from + s * of);
    if (!bias && p.dw_bf16) {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.dw) + i) =
            make_uint2(dev::pack_bf16(v[0], v[1]), dev::pack_bf16(v[2], v[3]));
        return;
    }
    using Quad = float __attribute__((ext_vector_type(4), aligned(4)));  // dbias has a float's alignment
    Quad *to = reinterpret_cast<Quad *>((bias ? p.dbias : static_cast<float *>(p.dw)) + i);
    *to = p.accumulate ? *to + v : v;
}

int64_t weight_tiles(int32_t E, int32_t n, int32_t k, int32_t rows)
{
    return (int64_t)E * ((n + rows - 1) / rows) * ((k + 255) / 256);
}

// 256 x 256 on one block per compute unit, or 128 x 256 on two, which hide each other's waits
// and results but read a half more: whichever takes less, by rounds over the compute units.
// In eighths of a step of a wide round a wide round takes 8 steps and 96, two narrow blocks
// 9 and 76, one alone 5 and 64.  128 / 256 (bf16 rows, fp32 results, us): 8192 dense rows,
// 64 wide tiles 82 / 157, 128 125 / 160, 144 182 / 154, 256 230 / 204, 272 304 / 349, 384 350 /
// 378, 448 440 / 376; 2048 dense rows, 128 tiles 38 / 48, 448 128 / 120; 32 experts, 4096 x
// 7168, 64 rows each 795 / 797 (bf16 results 444 / 580), 256 1231 / 1243 (831 / 937), 512 1696 /
// 1544 (1210 / 1222), 1024 2487 / 2184 (2038 / 1900); 256 rows each, 768 x 768 (288 tiles) 27.5 /
// 44.2; 8 experts x 512 rows, 2048 x 4096 104 / 110 (82 / 91).  Of 170 such pairs the rule takes the
// slower side by more than 3% in four (at most 10%: 512 rows in many rounds).
bool wide_weights(int64_t max_rows, int32_t E, int32_t n, int32_t k)
{
    const int64_t cus = device_cu_count(), steps = max_rows / E / Weights256::kStep;
    const int64_t wide = weight_tiles(E, n, k, 256), narrow = weight_tiles(E, n, k, 128), left = narrow % (2 * cus);
    const int64_t rounds = (wide + cus - 1) / cus, pairs = narrow / (2 * cus) + (left > cus), alone = left > 0 && left <= cus;
    return rounds * (8 * steps + 96) <= pairs * (9 * steps + 76) + alone * (5 * steps + 64);
}

template <typename S>
hipError_t launch_weights(const GradWeightArgs &p, hipStream_t stream)
{
    const int32_t m_tiles = (p.n + S::BM - 1) / S::BM, n_tiles = (p.k + S::BN - 1) / S::BN;
    const int64_t work = (int64_t)m_tiles * n_tiles * p.E * p.splits;
    // the blocks that compute units hold (LDS), a multiple of the 8 XCDs
    const int64_t most = ((S::kStages == 4 ? 1 : 2) * device_cu_count() + 7) / 8 * 8;
    const dim3 grid((uint32_t)(work < most ? (work + 7) / 8 * 8 : most)), block(S::kThreads);
    switch (p.a_quant) {
    case MOE_QUANT_FP8_F32:
        hipLaunchKernelGGL((grad_weight_tiles<S, MOE_QUANT_FP8_F32>), grid, block, 0, stream, p, m_tiles, n_tiles);
        break;
    case MOE_QUANT_FP8_UE8M0:
        hipLaunchKernelGGL((grad_weight_tiles<S, MOE_QUANT_FP8_UE8M0>), grid, block, 0, stream, p, m_tiles, n_tiles);
        break;
    case MOE_QUANT_MXFP8:
        hipLaunchKernelGGL((grad_weight_tiles<S, MOE_QUANT_MXFP8>), grid, block, 0, stream, p, m_tiles, n_tiles);
        break;
    default:
        hipLaunchKernelGGL((grad_weight_tiles<S, MOE_QUANT_NONE>), grid, block, 0, stream, p, m_tiles, n_tiles);
    }
    return hipGetLastError();
}

}  // namespace

int32_t grad_weight_splits(int64_t max_rows, int32_t E, int32_t n, int32_t k)
{
    if (wide_weights(max_rows, E, n, k))  // never where narrow tiles alone leave compute units free
        return 1;
    // One block per compute unit, of at least 512 rows: more of them write and read more
    // parts (8191 rows, 768 x 2048, 48 tiles: 256 / 384 / 512 blocks 42 / 45 / 48 us; 2048 x 2048,
    // 128 tiles: 81 / 93 / 88)
    const int64_t most = max_rows / E / 512, splits = device_cu_count() / weight_tiles(E, n, k, 128);
    return (int32_t)(splits < 1 || most < 1 ? 1 : splits < most ? splits : most);
}

hipError_t launch_grad_weight(const GradWeightArgs &p, hipStream_t stream)
{
    const hipError_t e = wide_weights(p.max_rows, p.E, p.n, p.k) ? launch_weights<Weights256>(p, stream)
                                                                 : launch_weights<Weights128>(p, stream);
    if (e != hipSuccess || p.splits == 1)
        return e;
    const int64_t quads = (int64_t)p.E * p.n * p.k / 4, all = quads + (p.dbias != nullptr ? (int64_t)p.E * p.n / 4 : 0);
    hipLaunchKernelGGL(grad_weight_join, dim3((uint32_t)((all + kBlockThreads - 1) / kBlockThreads)), dim3(kBlockThreads),
                       0, stream, p, quads, all);
    return hipGetLastError();
}

}  // namespace moe
