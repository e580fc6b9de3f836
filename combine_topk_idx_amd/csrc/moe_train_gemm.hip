// The experts' products in bf16 on gfx950: forward (with bias, activation and
// residual, or as a gated block) and the gradient to the rows.
//
//   forward    p[row, j]  = sum over c of a[row, c] w[e, j, c]
//   gradient   da[row, c] = sum over j of dy[row, j] w[e, j, c]
//
// The weights are the matrix instruction's first operand: a lane's results belong
// to one row and four output channels, and lanes that trade results make
// whole cache lines of a row.  The gradient sums over the slow axis of the same
// weights: its stages hold them as they lie in memory, and transposing reads
// (ds_read_b64_tr_b16) hand each lane steps of one channel.
//
// Bound by the matrix cores at the clock that the chip's power allows: 32,768 dense rows,
// 7168 -> 2 x 2048 gated 1396 us (1380 TFLOP/s), gradient 1389; 8192^3 719 us gated, 741
// linear, 735 gradient (1484 to 1530 TFLOP/s).  32 experts with 900 to 1150 rows each take
// 1680 us (with 8-bit saved rows 1770 to 1830): a ninth row of tiles on some compute units
// where the mean is 8.3, weights that 32 experts do not share, results that nothing overlaps.
// Few rows are bound by the weights' bytes: 128 tokens x 8 over 64 experts, 2048 -> 7168 337
// us (5.6 TB/s).  No LDS bank conflicts in any of them.
#include "moe_act.h"
#include "moe_train_tiles.h"

namespace moe {

namespace {

using namespace tile;
using namespace tile::train;

// What is summed over, and the rows' channels.
template <TrainProduct P>
__device__ __forceinline__ int32_t depth(const TrainGemmArgs &p) { return P == kGradInput ? p.n : p.k; }

// The loads of one tile: descriptors (uniform) and this lane's offsets.  Rows
// past the tile's end are zeros, which spare their loads and the matrix units' power
// (4096 unequal rows over 32 experts: 0.7% against copies of the last row); channels past
// the last are read as that one (the gradient's: as zeros).  Neither is stored.  Summed
// channels past the last are zeros in both operands: bit 31 of an offset takes it
// past its buffer's end, which the range check turns into zeros.
template <TrainProduct P, typename S>
struct TileLoads {
    using Rows = RowPlaces<S>;
    __amdgpu_buffer_rsrc_t a, w[2];
    uint32_t ao[S::kA], wo[P == kGradInput ? 2 : S::kB];
    const uint16_t *we;  // the gradient's weights
    uint32_t piece;      // first summed channel of this lane's pieces within a step
    int32_t K, wave, stride;

    __device__ __forceinline__ void set(const TrainGemmArgs &p, const TileAt &at, int wave_, int lane)
    {
        wave = wave_;
        lane = here(lane);
        K = depth<P>(p);
        const uint32_t row_bytes = (uint32_t)K * 2;
        const int row = Rows::row(wave, lane);
        piece = Rows::channel(wave, lane);
        a = buffer(p.rows + at.row0 * K, (uint32_t)at.valid * row_bytes);
#pragma unroll
        for (int i = 0; i < S::kA; ++i)
            ao[i] = row + Rows::kPass * i < at.valid ? (uint32_t)(row + Rows::kPass * i) * row_bytes + piece * 2 : 0x80000000u;
        if constexpr (P == kGradInput) {
            stride = p.k;
#pragma unroll
            for (int odd = 0; odd < 2; ++odd) {  // passes by turns
                const int n = wave + odd * S::kWaves;
                const int32_t c = at.nt * S::BN + StepPlaces<S::BN>::channel(n, lane);
                wo[odd] = c < p.k ? (uint32_t)StepPlaces<S::BN>::step(n, lane) * (uint32_t)stride * 2 + (uint32_t)c * 2 : 0x80000000u;
            }
            we = p.w + (int64_t)at.e * p.n * p.k;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // gated: half a tile of gate channels, then the up channels of the same h
                constexpr int kHalf = S::BN / 2;
                const int32_t of = P == kGated ? p.n / 2 : p.n;
                const int32_t c = min(P == kGated ? at.nt * kHalf : at.nt * S::BN + h * kHalf, of - 1);
                const int32_t left = min(kHalf, of - c);
                w[h] = buffer(p.w + ((int64_t)at.e * p.n + (P == kGated ? h * of : 0) + c) * K,
                              (uint32_t)left * row_bytes);
#pragma unroll
                for (int i = 0; i < S::kB / 2; ++i)
                    wo[S::kB / 2 * h + i] = (uint32_t)min(row + Rows::kPass * i, left - 1) * row_bytes + piece * 2;
            }
        }
    }
    // Loads FROM .. TO - 1 of step kb; steps after the last cost no memory access.
    template <int FROM, int TO>
    __device__ __forceinline__ void issue(uint8_t *st, int kb) const
    {
        const int32_t k0 = kb * S::kStep;
        const uint32_t past = (int32_t)piece + k0 < K ? 0u : 0x80000000u;
        const uint32_t at_k = k0 < K ? (uint32_t)k0 * 2 : 0u;
        for_each<TO - FROM>([&](auto N) {
            constexpr int j = FROM + decltype(N)::value;
            if constexpr (j < S::kA) {
                load_lds<16>(a, st + (wave + S::kWaves * j) * 1024, ao[j] | past, at_k);
            } else {
                constexpr int i = j - S::kA;
                uint8_t *to = st + S::kW + (wave + S::kWaves * i) * 1024;
                if constexpr (P == kGradInput) {
                    const __amdgpu_buffer_rsrc_t ws =
                        buffer(we + (int64_t)k0 * stride, (uint32_t)max(0, min(S::kStep, K - k0)) * (uint32_t)stride * 2);
                    load_lds<16>(ws, to, wo[i & 1] + (uint32_t)(i >> 1) * 2 * StepPlaces<S::BN>::kSteps * S::kWaves * (uint32_t)stride * 2, 0);
                } else {
                    load_lds<16>(w[i / (S::kB / 2)], to, wo[i] | past, at_k);
                }
            }
        });
    }
};

// Where a lane finds its fragments in a stage.
template <TrainProduct P, typename S, int MT>
struct TileReads {
    int row, column, rows, channels;

    __device__ __forceinline__ TileReads(int wave, int lane)
    {
        row = RowPlaces<S>::read(lane);
        rows = wave / S::WC * MT * 16 * S::kRow;
        channels = wave % S::WC;
        column = StepPlaces<S::BN>::read(lane);
    }
    // 16 rows, or 16 channels, of half h of a step.
    __device__ __forceinline__ dev::bf16x8 x(const uint8_t *st, int i, int h) const
    {
        return *reinterpret_cast<const dev::bf16x8 *>(st + rows + i * 16 * S::kRow + (row ^ h * 64));
    }
    __device__ __forceinline__ dev::bf16x8 w(const uint8_t *st, int f, int h) const
    {
        if constexpr (P == kGradInput)
            return read_steps<S::BN>(st + S::kW + (column ^ (channels * S::NF + f) * 32) + h * 64 * S::BN);
        // gated: the first half of a wave's fragments are gate channels
        constexpr int kHalf = S::NF / 2;
        const int c = P == kGated ? (channels * kHalf + f % kHalf) * 16 + f / kHalf * (S::BN / 2) : (channels * S::NF + f) * 16;
        return *reinterpret_cast<const dev::bf16x8 *>(st + S::kW + c * S::kRow + (row ^ h * 64));
    }
};

// ---- results ----------------------------------------------------------------------

// How the waves of a tile share the 128-channel blocks of saved rows in 8 bits: a
// block is that of one to four waves; an MXFP8 block is a pair of fragments.
template <TrainProduct P, typename S>
struct SavedBlocks {
    static constexpr int kHalves = P == kGated ? 2 : 1;       // gate and up, or all channels
    static constexpr int kOwn = S::NF / kHalves;              // fragments of a half, per wave
    static constexpr int kShare = kQuantGroup / (kOwn * 16);  // waves of a block
    static constexpr bool kWhole = kShare <= S::WC;           // a tile has whole blocks
};

// Largest magnitude of a row's channels in COUNT fragments of a wave.
template <int COUNT>
__device__ __forceinline__ float largest(const dev::f32x4 *v)
{
    float m = 0.0f;
#pragma unroll
    for (int f = 0; f < COUNT; ++f)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            m = fmaxf(m, fabsf(v[f][j]));
    m = fmaxf(m, __shfl_xor(m, 16));
    return fmaxf(m, __shfl_xor(m, 32));
}

// One row fragment's saved rows in 8 bits.
template <TrainProduct P, int QUANT, typename S>
__device__ __forceinline__ void save_quantized(const TrainGemmArgs &p, const dev::f32x4 (&v)[S::NF], const TileAt &at,
                                               int row0, int wc, int lane, const float (*wave_max)[S::WC][S::BM])
{
    using B = SavedBlocks<P, S>;
    const int32_t half = P == kGated ? p.n / 2 : p.n;
    constexpr int kScale = QUANT == MOE_QUANT_FP8_UE8M0 ? 1 : 4;  // bytes of 128 channels' scales
    const int32_t NB = p.n / kQuantGroup, row_scale = (NB * kScale + 3) / 4 * 4;
    const __amdgpu_buffer_rsrc_t out =
        buffer(static_cast<uint8_t *>(p.saved) + at.row0 * p.n, (uint32_t)at.valid * (uint32_t)p.n);
    const __amdgpu_buffer_rsrc_t scales =
        buffer(static_cast<uint8_t *>(p.saved_scale) + at.row0 * row_scale, (uint32_t)at.valid * (uint32_t)row_scale);
    const int g = lane >> 4, row = row0 + (lane & 15);
#pragma unroll
    for (int h = 0; h < B::kHalves; ++h) {
        float m = 0.0f;
        if constexpr (QUANT != MOE_QUANT_MXFP8 && B::kShare == 1)
            m = largest<B::kOwn>(&v[h * B::kOwn]);
        if constexpr (QUANT != MOE_QUANT_MXFP8 && B::kShare > 1) {
#pragma unroll
            for (int u = 0; u < B::kShare; ++u)
                m = fmaxf(m, wave_max[h][wc / B::kShare * B::kShare + u][row]);
        }
#pragma unroll
        for (int f = 0; f < B::kOwn; f += 2) {
            const int32_t c = at.nt * (S::BN / B::kHalves) + (wc * B::kOwn + f) * 16;
            const bool inside = row < at.valid && c < half;
            const int32_t channel = c + h * half;
            const dev::f32x4 *of = &v[h * B::kOwn + f];
            if constexpr (QUANT == MOE_QUANT_MXFP8)
                m = largest<2>(of);
            const dev::BlockScale<QUANT> bs(m);
            uint32_t e4m3[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
                e4m3[u] = dev::pack_e4m3(bs.apply(of[u][0]), bs.apply(of[u][1]), bs.apply(of[u][2]), bs.apply(of[u][3]));
            const auto pair = __builtin_amdgcn_permlane16_swap(e4m3[0], e4m3[1], false, false);
            const uint32_t off = (uint32_t)row * (uint32_t)p.n + channel + (g & 1) * 16 + (g >> 1) * 8;
            __builtin_amdgcn_raw_buffer_store_b64(dev::u32x2{pair[0], pair[1]}, out, inside ? off : 0x80000000u, 0, 0);
            if constexpr (QUANT == MOE_QUANT_MXFP8) {
                const uint32_t soff = (uint32_t)row * row_scale + channel / 32;
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)bs.byte, scales, inside && g == 0 ? soff : 0x80000000u, 0, 0);
            } else if (f == 0) {
                const int32_t b = channel / kQuantGroup;
                const bool one = inside && g == 0 && wc % B::kShare == 0;
                const uint32_t soff = one ? (uint32_t)row * row_scale + b * kScale : 0x80000000u;
                if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(bs.s), scales, soff, 0, 0);
                } else {
                    __builtin_amdgcn_raw_buffer_store_b8((uint8_t)bs.byte, scales, soff, 0, 0);
                    if (b == NB - 1)  // the last word's unused high bytes are 0
                        for (int u = 1; u <= row_scale - NB; ++u)
                            __builtin_amdgcn_raw_buffer_store_b8((uint8_t)0, scales, soff, u, 0);
                }
            }
        }
    }
}

// COUNT adjacent fragments of one row fragment.
template <int COUNT>
__device__ __forceinline__ void store_fragments(const Lines &to, const dev::f32x4 *v, int row0, int32_t c0, int lane)
{
    if constexpr (COUNT == 2) {
        store_pair(to, v[0], v[1], row0, c0, lane);
    } else {
#pragma unroll
        for (int f = 0; f < COUNT; f += 4)
            store_lines(to, v[f], v[f + 1], v[f + 2], v[f + 3], row0, c0 + f * 16, lane);
    }
}

// Writes a wave's results, one row fragment at a time, from the sums into other
// registers: sums that an epilogue changes would leave the accumulators.  Beside 1680 us
// without saved rows (32 experts, 32,768 rows, 2 x 2048 channels) they take 70 us in bf16
// (537 MB) and 110 in 8 bits, which the waves quantize before the next tile; the row maxima
// by lane swaps instead of shuffles, 16-byte stores and non-temporal ones change nothing.
template <TrainProduct P, typename S, int MT>
__device__ __forceinline__ void write_tile(const TrainGemmArgs &p, const dev::f32x4 (&acc)[S::NF][MT], const TileAt &at,
                                           int wr, int wc, int lane, float (*wave_max)[S::WC][S::BM])
{
    constexpr int NF = S::NF;
    using B = SavedBlocks<P, S>;
    lane = here(lane);
    const int g = lane >> 4;
    const int32_t channels = P == kGated ? p.n / 2 : P == kGradInput ? p.k : p.n;
    // this wave's channels (gated: of a half)
    const int32_t c0 = P == kGated ? at.nt * (S::BN / 2) + wc * (NF / 2) * 16 : at.nt * S::BN + wc * NF * 16;
    const uint32_t bytes = (uint32_t)at.valid * (uint32_t)channels * 2;
    const Lines out = {buffer(p.y + at.row0 * channels, bytes), at.valid, channels, 0, channels};
    Lines saved, residual;
    dev::f32x4 add[NF];
    if constexpr (P != kGradInput)
        saved = Lines{buffer(p.saved != nullptr ? static_cast<uint16_t *>(p.saved) + at.row0 * p.n : p.y,
                             (uint32_t)at.valid * (uint32_t)p.n * 2),
                      at.valid, channels, 0, p.n};
    if constexpr (P == kLinear) {
        residual = Lines{buffer(p.residual != nullptr ? p.residual + at.row0 * channels : p.y, bytes), at.valid, channels, 0,
                         channels};
        const __amdgpu_buffer_rsrc_t bias =
            buffer(p.bias != nullptr ? p.bias + (int64_t)at.e * p.n : p.y, p.bias != nullptr ? (uint32_t)p.n * 2 : 0);
#pragma unroll
        for (int f = 0; f < NF; ++f) {  // zeros past the buffer's end
            const dev::u32x2 b = __builtin_amdgcn_raw_buffer_load_b64(bias, (uint32_t)(c0 + f * 16 + 4 * g) * 2, 0, 0);
            add[f] = dev::f32x4{dev::bf16_lo(b[0]), dev::bf16_hi(b[0]), dev::bf16_lo(b[1]), dev::bf16_hi(b[1])};
        }
    }
    const auto row_sums = [&](auto I, dev::f32x4 (&v)[NF]) {
        constexpr int i = decltype(I)::value;
        for_each<NF>([&](auto F) {
            constexpr int f = decltype(F)::value;
            v[f] = acc[f][i];
            if constexpr (P == kLinear)
                v[f] += add[f];
        });
    };
    const bool quantized = P != kGradInput && B::kWhole && p.saved != nullptr && p.saved_quant != MOE_QUANT_NONE;
    if constexpr (P != kGradInput && B::kWhole && B::kShare > 1) {
        if (quantized && p.saved_quant != MOE_QUANT_MXFP8) {
            for_each<MT>([&](auto I) {
                dev::f32x4 v[NF];
                row_sums(I, v);
#pragma unroll
                for (int h = 0; h < B::kHalves; ++h) {
                    const float m = largest<B::kOwn>(&v[h * B::kOwn]);
                    if (g == 0)
                        wave_max[h][wc][(wr * MT + decltype(I)::value) * 16 + lane] = m;
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            meet();
        }
    }
    for_each<MT>([&](auto I) {
        const int row0 = (wr * MT + decltype(I)::value) * 16;
        dev::f32x4 v[NF];
        row_sums(I, v);
        if constexpr (P != kGradInput) {
            if constexpr (B::kWhole) {
                if (quantized && p.saved_quant == MOE_QUANT_FP8_F32)
                    save_quantized<P, MOE_QUANT_FP8_F32, S>(p, v, at, row0, wc, lane, wave_max);
                else if (quantized && p.saved_quant == MOE_QUANT_FP8_UE8M0)
                    save_quantized<P, MOE_QUANT_FP8_UE8M0, S>(p, v, at, row0, wc, lane, wave_max);
                else if (quantized)
                    save_quantized<P, MOE_QUANT_MXFP8, S>(p, v, at, row0, wc, lane, wave_max);
            }
            if (!quantized && p.saved != nullptr) {
                store_fragments<B::kOwn>(saved, v, row0, c0, lane);
                if constexpr (P == kGated) {
                    Lines up = saved;
                    up.shift = channels;
                    store_fragments<B::kOwn>(up, v + B::kOwn, row0, c0, lane);
                }
            }
        }
        if constexpr (P == kGated)
            dev::for_act(p.act, [&](auto act) {
#pragma unroll
                for (int f = 0; f < NF / 2; ++f)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[f][j] = dev::act_value<decltype(act)::value>(v[f][j]) * v[f + NF / 2][j];
            });
        if constexpr (P == kLinear) {
            if (p.act != MOE_ACT_NONE)
                dev::for_act(p.act, [&](auto act) {
#pragma unroll
                    for (int f = 0; f < NF; ++f)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[f][j] = dev::act_value<decltype(act)::value>(v[f][j]);
                });
            if (p.residual != nullptr) {
#pragma unroll
                for (int f = 0; f < NF; f += 4)
                    add_lines(residual, &v[f], row0, c0 + f * 16, lane);
            }
        }
        store_fragments<P == kGated ? NF / 2 : NF>(out, v, row0, c0, lane);
        __builtin_amdgcn_sched_barrier(0);  // one row fragment's registers at a time
    });
}

// 128 rows: eight waves, two per SIMD, three stages of which two are in flight.
using Rows128 = TileShape<128, 256, 2, 4, 64, 3>;
// 256 rows: four waves, one per SIMD, each with 128 x 128: the LDS reads of a
// matrix instruction fall to two thirds of what eight waves of 128 x 64 need, which
// together with the loads' writes would keep LDS as busy as the matrix cores.
using Rows256 = TileShape<256, 256, 2, 2, 64, 2>;
// 64 rows and 128 channels: four waves, three stages, two blocks per compute unit.  Four
// times the blocks of 128 x 256, for calls too small to fill the chip with those: a step
// takes 0.35 us instead of 0.75, mostly latency.
using Rows64 = TileShape<64, 128, 2, 2, 64, 3>;
// The same for gated products saved in 8 bits, which need the 128 channels of a block of
// both halves.
using Wide64 = TileShape<64, 256, 2, 2, 64, 3>;
template <typename S>
constexpr int blocks_per_cu() { return S::BM == 64 && S::BN == 128 ? 2 : 1; }  // what LDS holds of their stages

// Starts the loads of a tile's first two stages.
template <TrainProduct P, typename S>
__device__ __forceinline__ void start_tile(const TrainGemmArgs &p, const TileAt &at, const Stages &st, int wave, int lane)
{
    TileLoads<P, S> loads;
    loads.set(p, at, wave, lane);
    loads.template issue<0, S::kLoads>(st.s0, 0);
    __builtin_amdgcn_sched_barrier(0);  // in this order: the waits count
    loads.template issue<0, S::kLoads>(st.s1, 1);
    __builtin_amdgcn_sched_barrier(0);
}

// Multiplies a tile whose first two stages are in flight, then starts the next
// tile's (`more`) and writes the results.
template <TrainProduct P, typename S, int MT>
__device__ __forceinline__ void run_tile(const TrainGemmArgs &p, const TileAt &at, const TileAt &next, bool more,
                                         const Stages &st, float (*wave_max)[S::WC][S::BM], int wave, int lane)
{
    TileLoads<P, S> loads;
    loads.set(p, at, wave, lane);
    const TileReads<P, S, MT> reads(wave, here(lane));
    const int KB = scalar((loads.K + S::kStep - 1) / S::kStep);
    dev::f32x4 acc[S::NF][MT];
    clear(acc);
    if constexpr (S::kStages == 3) {
        const auto step = [&](uint8_t *cur, uint8_t *free, int kb) {
            wait_and_meet<S::kLoads>();
            multiply_stage<S, MT>(acc, cur, reads, loads, free, kb + 2, [](auto, const auto &) {});
        };
        // The first steps stand before the loop: there the compiler's own waits allow
        // for the stores of the tile before, in the loop they would hold up each turn.
        step(st.s0, st.s2, 0);
        if (KB > 1) {
            step(st.s1, st.s0, 1);
            int kb = 2;
            for (; kb + 3 <= KB; kb += 3) {
                step(st.s2, st.s1, kb);
                step(st.s0, st.s2, kb + 1);
                step(st.s1, st.s0, kb + 2);
            }
            if (kb < KB)
                step(st.s2, st.s1, kb);
            if (kb + 1 < KB)
                step(st.s0, st.s2, kb + 1);
        }
    } else {
        // Half a step is read while the half before is multiplied.  Between a step's
        // halves the waves meet: the next stage is there and this one has been read, so
        // the step after next loads into it.
        Fragments<S, MT> first, second;
        const auto none = [](auto) {};
        const auto step = [&](uint8_t *cur, uint8_t *other, int kb) {
            multiply<false, S, MT>(acc, first, second, cur, 1, reads, loads, cur, 0, none);
            wait_and_meet<0>();
            multiply<true, S, MT>(acc, second, first, other, 0, reads, loads, cur, kb + 2, none);
        };
        wait_and_meet<S::kLoads>();
        for_each<MT + S::NF>([&](auto N) { read_fragment<decltype(N)::value, S, MT>(first, st.s0, 0, reads); });
        // Whole pairs: a step past the last multiplies zeros.  With a remainder of its own
        // the sums would change registers where the ways meet.
        for (int kb = 0; kb < KB; kb += 2) {
            step(st.s0, st.s1, kb);
            step(st.s1, st.s0, kb + 1);
            end_turn(kb + 2, KB);
        }
    }
    wait_and_meet<0>();
    if (more)
        start_tile<P, S>(p, next.scalars(), st, wave, lane);
    write_tile<P, S, MT>(p, acc, at, wave / S::WC, wave % S::WC, lane, wave_max);
}

template <TrainProduct P, typename S>
__global__ __launch_bounds__(S::kThreads, blocks_per_cu<S>()) void train_gemm_tiles(TrainGemmArgs p, int32_t n_tiles)
{
    constexpr int BM = S::BM;
    __shared__ int32_t tile_start[kMaxExperts / kGroup + 1];
    __shared__ int32_t red[S::kWaves];
    __shared__ alignas(1024) uint8_t st0[S::kBytes], st1[S::kBytes];
    __shared__ alignas(1024) uint8_t st2[S::kStages == 3 ? S::kBytes : 16];
    const Stages st = {st0, st1, st2, nullptr};
    __shared__ float wave_max[P == kGated ? 2 : 1][S::WC][BM];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = scalar(threadIdx.x / kWave);
    scan_tiles<BM, S::kThreads>(p, tile_start, red);
    const int64_t n_work = (int64_t)scalar(tile_start[(p.E + kGroup - 1) / kGroup]) * n_tiles;
    // workgroups go to the 8 XCDs in turn: each XCD takes a contiguous run of
    // the work, so that the tiles of one expert share its L2
    const int64_t run = (n_work + 7) / 8;
    const int64_t base = (int64_t)(blockIdx.x & 7) * run;
    const int64_t end = min(run, n_work - base);

    // tiles of an expert: groups of 3 to 5 row tiles, alike in size; inside a group
    // the row tiles of one channel tile are adjacent (they share its weights)
    const auto locate = [&](int32_t m, int32_t rem) {  // number m * n_tiles + rem
        TileAt at;
        const ExpertAt ex = find_expert<BM>(p, tile_start, m);
        const int32_t e_tiles = (ex.rows + BM - 1) / BM;
        const int32_t groups = max(1, (e_tiles + 2) / 4), size = (e_tiles + groups - 1) / groups;
        const int32_t grp = (m - ex.start) / size;
        const int32_t in_grp = (m - ex.start) % size * n_tiles + rem;
        const int32_t grp_rows = min(size, e_tiles - grp * size);
        at.e = scalar(ex.e);
        at.nt = scalar(in_grp / grp_rows);
        const int32_t first = scalar((grp * size + in_grp % grp_rows) * BM);
        at.valid = scalar(min(BM, ex.rows - first));
        at.row0 = (int64_t)(p.expert_offset != nullptr ? word_of(p.expert_offset, at.e) : 0) + first;
        return at;
    };
    int64_t idx = blockIdx.x >> 3;
    if (idx >= end)
        return;
    int32_t m = scalar((int32_t)((base + idx) / n_tiles));
    int32_t rem = scalar((int32_t)((base + idx) - (int64_t)m * n_tiles));
    const int32_t m_step = scalar((gridDim.x >> 3) / n_tiles), rem_step = (gridDim.x >> 3) - m_step * n_tiles;
    TileAt next = locate(m, rem);
    start_tile<P, S>(p, next, st, wave, lane);
    for (;;) {
        const TileAt at = next.scalars();
        idx += gridDim.x >> 3;
        const bool more = idx < end;
        m += m_step;
        rem += rem_step;
        if (rem >= n_tiles) {
            rem -= n_tiles;
            ++m;
        }
        if (more)
            next = locate(m, rem);
        // a tile that is not full takes the code for its size
        constexpr int MT = S::MT, kWide = 16 * S::WR;
        if (at.valid > MT / 2 * kWide)
            run_tile<P, S, MT>(p, at, next, more, st, wave_max, wave, lane);
        else if (MT == 2 || at.valid > MT / 4 * kWide)
            run_tile<P, S, MT / 2>(p, at, next, more, st, wave_max, wave, lane);
        else if constexpr (MT > 2)
            run_tile<P, S, MT / 4>(p, at, next, more, st, wave_max, wave, lane);
        if (!more)
            break;
    }
}

// ---------------------------------------------------------------------------
// Few rows and too few tiles for the chip: 16 R rows x 16 weight rows (16 channels,
// or 8 gate and 8 up channels) per block, whose waves share the summed channels, 64
// at a time, and add up in LDS, in order.
//
// Bound by latency and the weights' bytes: the tiles above would leave most compute
// units idle, with one step's round trip to memory after the other.  One row, 7168 -> 2 x
// 2048: 12.8 us, 4.6 TB/s.
// ---------------------------------------------------------------------------

constexpr int kStripWaves = 8;

template <TrainProduct P, int R>
__global__ __launch_bounds__(kStripWaves *kWave) void train_gemm_strips(TrainGemmArgs p, int32_t strips)
{
    __shared__ int32_t tile_start[kMaxExperts / kGroup + 1];
    __shared__ int32_t red[kStripWaves];
    __shared__ dev::f32x4 part[kStripWaves][R][kWave];
    constexpr int kStripRows = 16 * R, kChannels = P == kGated ? 8 : 16;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = scalar(threadIdx.x / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int32_t K = p.k, half = p.n / 2;
    const int32_t channels = P == kGated ? half : p.n;
    const int KB = (K + 63) / 64, whole = K / 64;
    scan_tiles<kStripRows, kStripWaves * kWave>(p, tile_start, red);
    const int64_t n_work = (int64_t)scalar(tile_start[(p.E + kGroup - 1) / kGroup]) * strips;

    for (int64_t work = blockIdx.x; work < n_work; work += gridDim.x) {
        const int32_t m = scalar((int32_t)(work / strips));
        const int32_t c0 = scalar((int32_t)(work - (int64_t)m * strips)) * kChannels;
        const ExpertAt ex = find_expert<kStripRows>(p, tile_start, m);
        const int32_t first = (m - ex.start) * kStripRows, valid = min(kStripRows, ex.rows - first);
        const int64_t row0 = (int64_t)(p.expert_offset != nullptr ? word_of(p.expert_offset, ex.e) : 0) + first;
        // rows past the end: the last one, channels past the end: the last one
        const int32_t c = P == kGated ? c0 + (r & 7) + (r >> 3) * half : min(c0 + r, p.n - 1);
        const uint16_t *w = p.w + ((int64_t)ex.e * p.n + c) * K + 8 * g;
        const uint16_t *x[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
            x[i] = p.rows + (row0 + min(16 * i + r, valid - 1)) * K + 8 * g;
        struct Block {
            dev::bf16x8 w[2], x[R][2];
        };
        const auto fill = [&](Block &b, int kb) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t at = kb * 64 + h * 32;
                b.w[h] = *reinterpret_cast<const dev::bf16x8 *>(w + at);
#pragma unroll
                for (int i = 0; i < R; ++i)
                    b.x[i][h] = *reinterpret_cast<const dev::bf16x8 *>(x[i] + at);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        dev::f32x4 acc[R];
#pragma unroll
        for (int i = 0; i < R; ++i)
            acc[i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const auto use = [&](const Block &b) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < R; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.w[h], b.x[i][h], acc[i], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        };
        if (wave < whole) {
            // four blocks in flight; past the last one, the last one again
            constexpr int S = kStripWaves;
            const int count = (whole - wave + S - 1) / S, last = wave + (count - 1) * S;
            Block b0, b1, b2, b3;
            fill(b0, wave);
            fill(b1, min(wave + S, last));
            fill(b2, min(wave + 2 * S, last));
            for (int i = 0; i < count; i += 4) {
                const int kb = wave + i * S;
                fill(b3, min(kb + 3 * S, last));
                use(b0);
                if (i + 1 >= count)
                    break;
                fill(b0, min(kb + 4 * S, last));
                use(b1);
                if (i + 2 >= count)
                    break;
                fill(b1, min(kb + 5 * S, last));
                use(b2);
                if (i + 3 >= count)
                    break;
                fill(b2, min(kb + 6 * S, last));
                use(b3);
            }
        }
        if (whole < KB && wave == whole % kStripWaves) {  // the rest: pieces of 8, zeros past the last
            const dev::bf16x8 zero = {};
            Block b;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t at = whole * 64 + h * 32;
                const bool inside = at + 8 * g < K;
                b.w[h] = inside ? *reinterpret_cast<const dev::bf16x8 *>(w + at) : zero;
#pragma unroll
                for (int i = 0; i < R; ++i)
                    b.x[i][h] = inside ? *reinterpret_cast<const dev::bf16x8 *>(x[i] + at) : zero;
            }
            use(b);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
            part[wave][i][lane] = acc[i];
        __syncthreads();
        if (wave < R) {  // a wave per 16 rows
            dev::f32x4 v = part[0][wave][lane];
#pragma unroll
            for (int u = 1; u < kStripWaves; ++u)
                v += part[u][wave][lane];
            const int32_t row = 16 * wave + r;
            const bool live = row < valid;
            // channels 4 g .. of 16; gated: the upper lanes' are the up channels of the lower's
            const int32_t at = P == kGated ? c0 + 4 * (g & 1) : c0 + 4 * g;
            const bool inside = live && at < channels;
            const auto pack = [](const dev::f32x4 &f) { return make_uint2(dev::pack_bf16(f[0], f[1]), dev::pack_bf16(f[2], f[3])); };
            const auto unpack = [](const uint2 &u) {
                return dev::f32x4{dev::bf16_lo(u.x), dev::bf16_hi(u.x), dev::bf16_lo(u.y), dev::bf16_hi(u.y)};
            };
            if (P == kLinear && p.bias != nullptr && inside)
                v += unpack(*reinterpret_cast<const uint2 *>(p.bias + (int64_t)ex.e * p.n + at));
            if (p.saved != nullptr && inside)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.saved) + (row0 + row) * p.n + at +
                                           (P == kGated ? (g >> 1) * half : 0)) = pack(v);
            dev::f32x4 up;
            if constexpr (P == kGated) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    up[j] = __shfl_xor(v[j], 32);
            }
            dev::for_act(p.act, [&](auto act) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = dev::act_value<decltype(act)::value>(v[j]);
            });
            uint16_t *y = p.y + (row0 + row) * channels + at;
            if constexpr (P == kGated) {
                v *= up;
                if (inside && g < 2)
                    *reinterpret_cast<uint2 *>(y) = pack(v);
            } else if (inside) {
                if (p.residual != nullptr)
                    v += unpack(*reinterpret_cast<const uint2 *>(p.residual + (row0 + row) * p.n + at));
                *reinterpret_cast<uint2 *>(y) = pack(v);
            }
        }
        __syncthreads();  // part is rewritten by the next strip
    }
}

// Row tiles of `rows` rows that a call can have: a segment's last one is partial.
int64_t max_tiles(const TrainGemmArgs &p, int32_t rows)
{
    if (p.recv_count == nullptr)
        return (p.max_rows + rows - 1) / rows;
    return p.max_rows / rows + (p.max_rows < p.E ? p.max_rows : p.E);
}

template <TrainProduct P, typename S>
hipError_t launch_tiles(const TrainGemmArgs &p, hipStream_t stream)
{
    const int32_t channels = P == kGated ? p.n / 2 : P == kGradInput ? p.k : p.n;
    const int32_t width = P == kGated ? S::BN / 2 : S::BN;
    const int32_t n_tiles = (channels + width - 1) / width;
    const int64_t tiles = max_tiles(p, S::BM) * n_tiles;
    // one block per compute unit (its stages fill LDS), a multiple of the 8 XCDs
    const int64_t cus = (blocks_per_cu<S>() * device_cu_count() + 7) / 8 * 8;
    const int64_t grid = tiles < cus ? (tiles + 7) / 8 * 8 : cus;
    hipLaunchKernelGGL((train_gemm_tiles<P, S>), dim3((uint32_t)grid), dim3(S::kThreads), 0, stream, p, n_tiles);
    return hipGetLastError();
}

template <TrainProduct P, int R>
hipError_t launch_strips(const TrainGemmArgs &p, hipStream_t stream)
{
    const int32_t strips = P == kGated ? p.n / 16 : (p.n + 15) / 16;
    const int64_t work = max_tiles(p, 16 * R) * strips, most = 8 * (int64_t)device_cu_count();
    hipLaunchKernelGGL((train_gemm_strips<P, R>), dim3((uint32_t)(work < most ? work : most)), dim3(kStripWaves * kWave), 0,
                       stream, p, strips);
    return hipGetLastError();
}

// Row tiles that evenly routed experts have, about: half of them end in one more.
int64_t likely_tiles(const TrainGemmArgs &p, int32_t rows)
{
    if (p.recv_count == nullptr)
        return (p.max_rows + rows - 1) / rows;
    const int64_t used = p.max_rows < p.E ? p.max_rows : p.E;
    const int64_t tiles = p.max_rows / rows + p.E / 2;
    return tiles < used ? used : tiles;
}

template <TrainProduct P>
hipError_t launch_product(const TrainGemmArgs &p, hipStream_t stream)
{
    const int64_t cus = device_cu_count();
    const bool quantized = p.saved != nullptr && p.saved_quant != MOE_QUANT_NONE;
    if constexpr (P != kGradInput) {
        // Strips for up to 32 rows per expert, while three blocks per compute unit hold them
        // all (in a graph, the same weights again, 64-row tiles / strips): one row, 7168 -> 4096
        // (256 strips) 38 / 13.6 us, 2048 -> 7168 (448) 14.7 / 11.0; 16 rows, 512 -> 512 (32) 7.0 /
        // 6.1; 32 rows, 7168 -> 4096 (512) 38 / 26, 2048 -> 2048 (256) 14.7 / 12.0; 8 experts, 2048 ->
        // 1024, 2 rows each (576) 15.4 / 12.7, 16 rows (1024) 15.5 / 23.8.  More rows take 64-row
        // tiles whatever their number: strips of 32 rows lose as soon as there are more of them
        // than compute units (64 rows, 2048 -> 4096 12.5 / 22.8, 7168 -> 4096 39 / 49; 96 rows, 2048 ->
        // 2048 14.6 / 22.3), and gain below that only with many summed channels (64 rows, 512 -> 512
        // 7.1 / 7.9, 2048 -> 2048 12.5 / 12.0, 7168 -> 2048 38 / 26).  8-bit saved rows need the 128
        // channels of a block together, which strips do not have.
        const int32_t strips = P == kGated ? p.n / 16 : (p.n + 15) / 16;
        const int64_t rows = (p.max_rows + p.E - 1) / p.E;
        if (!quantized && rows <= 32 && max_tiles(p, 16) * strips <= 3 * cus)
            return rows <= 16 ? launch_strips<P, 1>(p, stream) : launch_strips<P, 2>(p, stream);
    }
    const int32_t channels = P == kGated ? p.n / 2 : P == kGradInput ? p.k : p.n;
    const auto rounds = [&](int32_t rows, int32_t width) {  // over the compute units
        return (likely_tiles(p, rows) * ((channels + width - 1) / width) + cus - 1) / cus;
    };
    const int64_t rounds128 = rounds(128, P == kGated ? 128 : 256);
    // 64-row tiles, one per compute unit, take half the time of 128-row tiles with twice the
    // channels, two as long: 128 / 64 rows per tile: 128 dense rows, 2048 -> 2048 (32 tiles of
    // 64 rows) 25.7 / 12.6 us; 2048 rows, 1024 -> 1024 (256) 17.4 / 9.9, 2048 -> 2048 (512) 27.9 /
    // 25.6; 8 experts x 256 rows, 2048 -> 2048 (576) 29.3 / 34.0; 32 experts x 128 rows, 512 ->
    // 1536 (960, against two rounds) 28.9 / 19.7; 4096 dense rows, 2048 -> 2048 (1024) 37 / 50.
    if (!(P == kGated && quantized) && rounds(64, P == kGated ? 64 : 128) <= 2 * rounds128)
        return launch_tiles<P, Rows64>(p, stream);
    // As wide as the others, one per compute unit: not where a call has no more of them (8-bit
    // rows of fp32 scales, 128 / 64 rows per tile: 64 rows, 7168 -> 4096 58 / 63 us; 512 rows 79 /
    // 64; 512 rows, 2048 -> 2048 31.0 / 24.3, 4096 rows (512 tiles) 42 / 54; 32 experts x 128
    // rows, 512 -> 1536 43 / 27).
    if constexpr (P == kGated)
        if (quantized && likely_tiles(p, 64) > likely_tiles(p, 128) && rounds(64, 128) <= rounds128)
            return launch_tiles<P, Wide64>(p, stream);
    // 256-row tiles need half as many rounds over the compute units, each of 1.6 times
    // the time.  128 / 256 rows per tile: 4096 dense rows, 2048 -> 2048 (1 / 1 rounds) 34 /
    // 55 us; 1111, 2056 -> 7184 (2 / 1) 69 / 63; 16 experts x 512 rows, 2048 -> 2048 (3 / 2)
    // 82 / 109; 32 experts, 7168 -> 4096, 704 rows (12 / 7) 1396 / 1199, 512 (9 / 5) 1001 /
    // 979; 256 rows, 2048 -> 7168 (9 / 6) 319 / 371.
    if (8 * rounds(256, P == kGated ? 128 : 256) <= 5 * rounds128)
        return launch_tiles<P, Rows256>(p, stream);
    return launch_tiles<P, Rows128>(p, stream);
}

}  // namespace

hipError_t launch_train_gemm(const TrainGemmArgs &a, TrainProduct product, hipStream_t stream)
{
    switch (product) {
    case kLinear:
        return launch_product<kLinear>(a, stream);
    case kGated:
        return launch_product<kGated>(a, stream);
    default:
        return launch_product<kGradInput>(a, stream);
    }
}

}  // namespace moe
