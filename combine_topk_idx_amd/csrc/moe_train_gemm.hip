// The experts' products in bf16 on gfx950: forward (with bias, activation and
// residual, or as a gated block) and the gradient to the rows.
//
//   forward    p[row, j]  = sum over c of a[row, c] w[e, j, c]
//   gradient   da[row, c] = sum over j of dy[row, j] w[e, j, c]
//
// v_mfma_f32_16x16x32_bf16 with the weights as its first operand: a lane's four
// results belong to one row and four adjacent output channels, and lanes that
// trade results make whole cache lines of a row.  The gradient sums over the slow
// axis of the same weights: its stages hold them as they lie in memory, and
// ds_read_b64_tr_b16 hands each lane four steps of one channel.
#include "moe_act.h"
#include "moe_train_tiles.h"

namespace moe {

namespace {

using namespace tile;
using namespace tile::train;

constexpr int kMGroup = 8;                    // row tiles that walk the channel tiles together

// What is summed over, and the rows' channels.
template <TrainProduct P>
__device__ __forceinline__ int32_t depth(const TrainGemmArgs &p) { return P == kGradInput ? p.n : p.k; }

template <int BM>
struct Stage {
    static constexpr int kW = BM * kStep * 2;
    static constexpr int kBytes = kW + kTileN * kStep * 2;
    static constexpr int kLoads = BM / 64 + 4;  // loads of a wave per step
};

// The loads of one tile: descriptors (uniform) and this lane's offsets.  Rows
// past the tile's end are read as its last row and channels past the last as that
// one (the gradient's: as zeros); what comes of the copies is not stored.  Summed
// channels past the last are zeros in both operands: bit 31 of an offset takes it
// past its buffer's end, which the range check turns into zeros.
template <TrainProduct P, int BM>
struct TileLoads {
    __amdgpu_buffer_rsrc_t a, w[2];
    uint32_t ao[BM / 64], wo[4];
    const uint16_t *we;  // the gradient's weights
    uint32_t piece;      // first summed channel of this lane's pieces within a step
    int32_t K, wave, stride;

    __device__ __forceinline__ void set(const TrainGemmArgs &p, const TileAt &at, int wave_, int lane)
    {
        wave = wave_;
        K = depth<P>(p);
        const uint32_t row_bytes = (uint32_t)K * 2;
        // 16-byte piece c of a row sits at position c ^ ((row >> 1) & 7) in LDS:
        // the 16 rows of a fragment then cover all banks.  A wave loads rows 8 j
        // .. 8 j + 7, j = wave (mod 8): lane l holds position l % 8 of row l / 8.
        piece = ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)) * 8;
        const int row = 8 * wave + (lane >> 3);
        a = buffer(p.rows + at.row0 * K, (uint32_t)at.valid * row_bytes);
#pragma unroll
        for (int i = 0; i < BM / 64; ++i)
            ao[i] = (uint32_t)min(row + 64 * i, at.valid - 1) * row_bytes + piece * 2;
        if constexpr (P == kGradInput) {
            // 32 bytes (16 channels) of step s sit at position c ^ (s & 3 | s >> 1 & 4)
            // of its 512: what 32 lanes read at once then covers all banks.  A wave
            // loads steps 2 j and 2 j + 1, j = wave (mod 8).
            stride = p.k;
            const int s = 2 * wave + (lane >> 5);
            const int f = (s & 3) | ((s >> 1) & 4);
            const int32_t c = at.nt * kTileN + ((((lane & 31) >> 1) ^ f) * 2 + (lane & 1)) * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wo[i] = c < p.k ? (uint32_t)(s + 16 * i) * (uint32_t)stride * 2 + (uint32_t)c * 2 : 0x80000000u;
            we = p.w + (int64_t)at.e * p.n * p.k;
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // gated: 128 gate channels, then the up channels of the same h
                const int32_t of = P == kGated ? p.n / 2 : p.n;
                const int32_t c = min(P == kGated ? at.nt * 128 : at.nt * kTileN + h * 128, of - 1);
                const int32_t left = min(128, of - c);
                w[h] = buffer(p.w + ((int64_t)at.e * p.n + (P == kGated ? h * of : 0) + c) * K,
                              (uint32_t)left * row_bytes);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    wo[2 * h + i] = (uint32_t)min(row + 64 * i, left - 1) * row_bytes + piece * 2;
            }
        }
    }
    // Loads FROM .. TO - 1 of step kb; steps after the last cost no memory access.
    template <int FROM, int TO>
    __device__ __forceinline__ void issue(uint8_t *st, int kb) const
    {
        constexpr int kA = BM / 64;
        const int32_t k0 = kb * kStep;
        const uint32_t past = (int32_t)piece + k0 < K ? 0u : 0x80000000u;
        const uint32_t at_k = k0 < K ? (uint32_t)k0 * 2 : 0u;
        __amdgpu_buffer_rsrc_t ws;
        if constexpr (P == kGradInput && TO > kA)
            ws = buffer(we + (int64_t)k0 * stride, (uint32_t)max(0, min(kStep, K - k0)) * (uint32_t)stride * 2);
#pragma unroll
        for (int j = FROM; j < TO; ++j) {
            if (j < kA) {
                load_lds<16>(a, st + (wave + 8 * j) * 1024, ao[j] | past, at_k);
            } else {
                const int i = j - kA;
                uint8_t *to = st + Stage<BM>::kW + (wave + 8 * i) * 1024;
                if constexpr (P == kGradInput)
                    load_lds<16>(ws, to, wo[i], 0);
                else
                    load_lds<16>(w[i >> 1], to, wo[i] | past, at_k);
            }
        }
    }
};

// acc += the stage's step for this wave's MT row fragments and kNF channel
// fragments, while step `kb_load` loads into the stage `free`: its loads are
// spread over the matrix instructions.
template <TrainProduct P, int BM, int MT>
__device__ __forceinline__ void multiply_stage(dev::f32x4 (&acc)[kNF][MT], const uint8_t *st, int wr, int wc, int lane,
                                               const TileLoads<P, BM> &loads, uint8_t *free, int kb_load)
{
    constexpr int kLoads = Stage<BM>::kLoads;
    const int r = lane & 15, g = lane >> 4;
    const int rswz = (r >> 1) & 7;
    const int rlo = r * 128 + ((g ^ rswz) * 16), rhi = r * 128 + (((4 + g) ^ rswz) * 16);
    const uint8_t *rows = st + wr * MT * 16 * 128;
    const uint8_t *ws = st + Stage<BM>::kW;
    const int column = (8 * g + (r >> 2)) * 2 * kTileN + ((r >> 2) | (g & 1) << 2) * 32 + (r & 3) * 8;
    Fragment w[kNF], x[2];
#pragma unroll
    for (int f = 0; f < kNF; ++f) {
        if constexpr (P == kGradInput) {
            w[f] = read_columns<kTileN>(ws + (column ^ (wc * 4 + f) * 32));
        } else {
            const int c = P == kGated ? wc * 32 + (f & 1) * 16 + (f >> 1) * 128 : wc * 64 + f * 16;
            w[f] = read_rows(ws + c * 128, rlo, rhi);
        }
        if (f == 0)
            x[0] = read_rows(rows, rlo, rhi);
    }
    const auto part = [&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (i + 1 < MT)
            x[(i + 1) & 1] = read_rows(rows + (i + 1) * 16 * 128, rlo, rhi);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < kNF; ++f)
                acc[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[f].h[h], x[i & 1].h[h], acc[f][i], 0, 0, 0);
        loads.template issue<i * kLoads / MT, (i + 1) * kLoads / MT>(free, kb_load);
        __builtin_amdgcn_sched_barrier(0);
    };
    for_each<MT>(part);
}

// ---- results ----------------------------------------------------------------------

// The rows' bf16 that store_lines would overwrite, as fragments of fp32.
__device__ __forceinline__ void load_lines(__amdgpu_buffer_rsrc_t in, dev::f32x4 (&v)[kNF], int row0, int valid,
                                           int32_t c0, int32_t channels, int lane)
{
    const int r = lane & 15, g = lane >> 4;
    const bool low = r < 8;
    const int32_t c = c0 + (low ? 0 : 32) + (g & 1) * 16 + (g >> 1) * 8;
    dev::u32x4 s[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = row0 + h * 8 + (r & 7);
        const uint32_t off = row < valid && c < channels ? ((uint32_t)row * (uint32_t)channels + c) * 2 : 0x80000000u;
        s[h] = __builtin_amdgcn_raw_buffer_load_b128(in, off, 0, 0);
    }
    trade_rows(s, low);
    trade_fragments(s[0]);
    trade_fragments(s[1]);
#pragma unroll
    for (int f = 0; f < kNF; ++f) {
        const uint32_t lo = s[f >> 1][(f & 1) * 2], hi = s[f >> 1][(f & 1) * 2 + 1];
        v[f] = dev::f32x4{dev::bf16_lo(lo), dev::bf16_hi(lo), dev::bf16_lo(hi), dev::bf16_hi(hi)};
    }
}

// One pair of fragments -- 32 adjacent channels from c0 of 16 rows -- as bf16.
__device__ __forceinline__ void store_pair(__amdgpu_buffer_rsrc_t out, const dev::f32x4 &a, const dev::f32x4 &b, int row,
                                           int valid, int32_t c0, bool inside, int32_t channels, int g)
{
    dev::u32x4 s = pack_fragments(a, b);
    trade_fragments(s);
    const int32_t c = c0 + (g & 1) * 16 + (g >> 1) * 8;
    const uint32_t off = row < valid && inside ? ((uint32_t)row * (uint32_t)channels + c) * 2 : 0x80000000u;
    __builtin_amdgcn_raw_buffer_store_b128(s, out, off, 0, kStreamed);
}

// Saved rows in 8 bits.  A 128-channel block is that of two waves (of four in
// each of the gated block's halves); an MXFP8 block is a pair of fragments.
template <TrainProduct P, int QUANT, int MT, int BM>
__device__ __forceinline__ void save_quantized(const TrainGemmArgs &p, const dev::f32x4 (&acc)[kNF][MT], const TileAt &at,
                                               int wr, int wc, int lane, float (*wave_max)[kWaveCols][BM])
{
    const int r = lane & 15, g = lane >> 4;
    const int32_t half = P == kGated ? p.n / 2 : p.n;
    constexpr int kScale = QUANT == MOE_QUANT_FP8_UE8M0 ? 1 : 4;  // bytes of 128 channels' scales
    const int32_t NB = p.n / kQuantGroup, row_scale = (NB * kScale + 3) / 4 * 4;
    const __amdgpu_buffer_rsrc_t out =
        buffer(static_cast<uint8_t *>(p.saved) + at.row0 * p.n, (uint32_t)at.valid * (uint32_t)p.n);
    const __amdgpu_buffer_rsrc_t scales =
        buffer(static_cast<uint8_t *>(p.saved_scale) + at.row0 * row_scale, (uint32_t)at.valid * (uint32_t)row_scale);
    const auto largest = [&](int i, int h) {  // of this wave's 32 channels of its row
        float m = 0.0f;
#pragma unroll
        for (int f = 2 * h; f < 2 * h + 2; ++f)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                m = fmaxf(m, fabsf(acc[f][i][j]));
        m = fmaxf(m, __shfl_xor(m, 16));
        return fmaxf(m, __shfl_xor(m, 32));
    };
    if constexpr (QUANT != MOE_QUANT_MXFP8) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float m = largest(i, h);
                if (g == 0)
                    wave_max[h][wc][(wr * MT + i) * 16 + r] = m;
            }
        meet();
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = (wr * MT + i) * 16 + r;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // gated: pair h is the gate's or the up product's; else 32 of 64 channels
            const int32_t c = P == kGated ? at.nt * 128 + wc * 32 : at.nt * kTileN + wc * 64 + h * 32;
            const bool inside = row < at.valid && c < half;
            const int32_t channel = c + (P == kGated ? h * half : 0);
            float m;
            if constexpr (QUANT == MOE_QUANT_MXFP8) {
                m = largest(i, h);
            } else if constexpr (P == kGated) {
                m = fmaxf(fmaxf(wave_max[h][0][row], wave_max[h][1][row]),
                          fmaxf(wave_max[h][2][row], wave_max[h][3][row]));
            } else {
                m = fmaxf(fmaxf(wave_max[0][wc][row], wave_max[1][wc][row]),
                          fmaxf(wave_max[0][wc ^ 1][row], wave_max[1][wc ^ 1][row]));
            }
            const dev::BlockScale<QUANT> bs(m);
            uint32_t q[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const dev::f32x4 &v = acc[2 * h + f][i];
                q[f] = dev::pack_e4m3(bs.apply(v[0]), bs.apply(v[1]), bs.apply(v[2]), bs.apply(v[3]));
            }
            const auto pair = __builtin_amdgcn_permlane16_swap(q[0], q[1], false, false);
            const uint32_t off = (uint32_t)row * (uint32_t)p.n + channel + (g & 1) * 16 + (g >> 1) * 8;
            __builtin_amdgcn_raw_buffer_store_b64(dev::u32x2{pair[0], pair[1]}, out, inside ? off : 0x80000000u, 0, 0);
            if constexpr (QUANT == MOE_QUANT_MXFP8) {
                const uint32_t soff = (uint32_t)row * row_scale + channel / 32;
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)bs.byte, scales, inside && g == 0 ? soff : 0x80000000u, 0, 0);
            } else {
                const int32_t b = channel / kQuantGroup;
                const bool first = P == kGated ? wc == 0 : h == 0 && (wc & 1) == 0;
                const uint32_t soff = inside && g == 0 && first ? (uint32_t)row * row_scale + b * kScale : 0x80000000u;
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

// Writes a wave's results: rows 16 (MT wr + i) + (lane % 16), channels 4 (lane /
// 16) + j of fragment f.
template <TrainProduct P, int MT, int BM>
__device__ __forceinline__ void write_tile(const TrainGemmArgs &p, dev::f32x4 (&acc)[kNF][MT], const TileAt &at, int wr,
                                           int wc, int lane, float (*wave_max)[kWaveCols][BM])
{
    const int r = lane & 15, g = lane >> 4;
    if constexpr (P == kGradInput) {
        const __amdgpu_buffer_rsrc_t out = buffer(p.y + at.row0 * p.k, (uint32_t)at.valid * (uint32_t)p.k * 2);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const dev::f32x4 v[kNF] = {acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
            store_lines(out, v, (wr * MT + i) * 16, at.valid, at.nt * kTileN + wc * 64, p.k, lane);
        }
        return;
    }
    const int32_t c0 = at.nt * kTileN + wc * 64;
    if (P == kLinear && p.bias != nullptr) {
        const __amdgpu_buffer_rsrc_t bias = buffer(p.bias + (int64_t)at.e * p.n, (uint32_t)p.n * 2);
#pragma unroll
        for (int f = 0; f < kNF; ++f) {
            const dev::u32x2 b = __builtin_amdgcn_raw_buffer_load_b64(bias, (uint32_t)(c0 + f * 16 + 4 * g) * 2, 0, 0);
            const dev::f32x4 add = {dev::bf16_lo(b[0]), dev::bf16_hi(b[0]), dev::bf16_lo(b[1]), dev::bf16_hi(b[1])};
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[f][i] += add;
        }
    }
    if (p.saved != nullptr) {
        if (p.saved_quant == MOE_QUANT_FP8_F32) {
            save_quantized<P, MOE_QUANT_FP8_F32, MT, BM>(p, acc, at, wr, wc, lane, wave_max);
        } else if (p.saved_quant == MOE_QUANT_FP8_UE8M0) {
            save_quantized<P, MOE_QUANT_FP8_UE8M0, MT, BM>(p, acc, at, wr, wc, lane, wave_max);
        } else if (p.saved_quant == MOE_QUANT_MXFP8) {
            save_quantized<P, MOE_QUANT_MXFP8, MT, BM>(p, acc, at, wr, wc, lane, wave_max);
        } else {
            const __amdgpu_buffer_rsrc_t out = buffer(static_cast<uint16_t *>(p.saved) + at.row0 * p.n,
                                                      (uint32_t)at.valid * (uint32_t)p.n * 2);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int row = (wr * MT + i) * 16;
                if constexpr (P == kGated) {
                    const int32_t c = at.nt * 128 + wc * 32, half = p.n / 2;
                    const bool inside = c + (g & 1) * 16 + (g >> 1) * 8 < half;
                    store_pair(out, acc[0][i], acc[1][i], row + r, at.valid, c, inside, p.n, g);
                    store_pair(out, acc[2][i], acc[3][i], row + r, at.valid, c + half, inside, p.n, g);
                } else {
                    const dev::f32x4 v[kNF] = {acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
                    store_lines(out, v, row, at.valid, c0, p.n, lane);
                }
            }
        }
    }
    if constexpr (P == kGated) {
        const int32_t inter = p.n / 2;
        const __amdgpu_buffer_rsrc_t out = buffer(p.y + at.row0 * inter, (uint32_t)at.valid * (uint32_t)inter * 2);
        const int32_t c = at.nt * 128 + wc * 32;
        const bool inside = c + (g & 1) * 16 + (g >> 1) * 8 < inter;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[f][i][j] = dev::act_value(p.act, acc[f][i][j]) * acc[f + 2][i][j];
            store_pair(out, acc[0][i], acc[1][i], (wr * MT + i) * 16 + r, at.valid, c, inside, inter, g);
        }
    } else if constexpr (P == kLinear) {
        const uint32_t bytes = (uint32_t)at.valid * (uint32_t)p.n * 2;
        const __amdgpu_buffer_rsrc_t out = buffer(p.y + at.row0 * p.n, bytes);
        const bool add = p.residual != nullptr;
        const __amdgpu_buffer_rsrc_t residual = buffer(add ? p.residual + at.row0 * p.n : p.y, add ? bytes : 0);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = (wr * MT + i) * 16;
            dev::f32x4 v[kNF];
#pragma unroll
            for (int f = 0; f < kNF; ++f)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[f][j] = dev::act_value(p.act, acc[f][i][j]);
            if (add) {
                dev::f32x4 res[kNF];
                load_lines(residual, res, row, at.valid, c0, p.n, lane);
#pragma unroll
                for (int f = 0; f < kNF; ++f)
                    v[f] += res[f];
            }
            store_lines(out, v, row, at.valid, c0, p.n, lane);
        }
    }
}

// Starts the loads of a tile's first NS - 1 stages.
template <TrainProduct P, int BM, int NS>
__device__ __forceinline__ void start_tile(const TrainGemmArgs &p, const TileAt &at, uint8_t *st0, uint8_t *st1, int wave,
                                           int lane)
{
    TileLoads<P, BM> loads;
    loads.set(p, at, wave, lane);
    loads.template issue<0, Stage<BM>::kLoads>(st0, 0);
    __builtin_amdgcn_sched_barrier(0);  // in this order: the waits count
    if constexpr (NS == 3)
        loads.template issue<0, Stage<BM>::kLoads>(st1, 1);
    __builtin_amdgcn_sched_barrier(0);
}

// Multiplies a tile whose first NS - 1 stages are in flight, then starts the
// next tile's (`more`) and writes the results.
template <TrainProduct P, int BM, int NS, int MT>
__device__ __forceinline__ void run_tile(const TrainGemmArgs &p, const TileAt &at, const TileAt &next, bool more,
                                         uint8_t *st0, uint8_t *st1, uint8_t *st2, float (*wave_max)[kWaveCols][BM],
                                         int wave, int lane)
{
    TileLoads<P, BM> loads;
    loads.set(p, at, wave, lane);
    constexpr int kAhead = Stage<BM>::kLoads * (NS - 2);
    const int wr = wave / kWaveCols, wc = wave % kWaveCols;
    const int KB = (loads.K + kStep - 1) / kStep;
    dev::f32x4 acc[kNF][MT];
#pragma unroll
    for (int f = 0; f < kNF; ++f)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[f][i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const auto step = [&](uint8_t *cur, uint8_t *free, int kb) {
        wait_and_meet<kAhead>();
        multiply_stage<P, BM, MT>(acc, cur, wr, wc, lane, loads, free, kb + NS - 1);
    };
    // The first steps stand before the loop: there the compiler's own waits allow
    // for the stores of the tile before, in the loop they would hold up each turn.
    step(st0, NS == 3 ? st2 : st1, 0);
    if constexpr (NS == 3) {
        if (KB > 1) {
            step(st1, st0, 1);
            int kb = 2;
            for (; kb + 3 <= KB; kb += 3) {
                step(st2, st1, kb);
                step(st0, st2, kb + 1);
                step(st1, st0, kb + 2);
            }
            if (kb < KB)
                step(st2, st1, kb);
            if (kb + 1 < KB)
                step(st0, st2, kb + 1);
        }
    } else {
        int kb = 1;
        for (; kb + 2 <= KB; kb += 2) {
            step(st1, st0, kb);
            step(st0, st1, kb + 1);
        }
        if (kb < KB)
            step(st1, st0, kb);
    }
    wait_and_meet<0>();
    if (more)
        start_tile<P, BM, NS>(p, next.scalars(), st0, st1, wave, lane);
    write_tile<P, MT, BM>(p, acc, at, wr, wc, lane, wave_max);
}

template <TrainProduct P, int BM, int NS>
__global__ __launch_bounds__(kTileThreads) void train_gemm_tiles(TrainGemmArgs p, int32_t n_tiles)
{
    __shared__ int32_t tile_start[kMaxExperts / kGroup + 1];
    __shared__ int32_t red[kTileWaves];
    // separate variables: the compiler then knows which reads follow which loads
    __shared__ alignas(1024) uint8_t st0[Stage<BM>::kBytes];
    __shared__ alignas(1024) uint8_t st1[Stage<BM>::kBytes];
    __shared__ alignas(1024) uint8_t st2[NS == 3 ? Stage<BM>::kBytes : 16];
    __shared__ float wave_max[P == kGradInput ? 1 : 2][kWaveCols][BM];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = scalar(threadIdx.x / kWave);
    scan_tiles<BM>(p, tile_start, red);
    const int64_t n_work = (int64_t)scalar(tile_start[(p.E + kGroup - 1) / kGroup]) * n_tiles;
    // workgroups go to the 8 XCDs in turn: each XCD takes a contiguous run of
    // the work, so that the tiles of one expert share its L2
    const int64_t run = (n_work + 7) / 8;
    const int64_t base = (int64_t)(blockIdx.x & 7) * run;
    const int64_t end = min(run, n_work - base);

    // tiles of an expert: groups of kMGroup row tiles; inside a group the row
    // tiles of one channel tile are adjacent (they share its weights)
    const auto locate = [&](int32_t m, int32_t rem) {  // number m * n_tiles + rem
        TileAt at;
        const ExpertAt ex = find_expert<BM>(p, tile_start, m);
        const int32_t e_tiles = (ex.rows + BM - 1) / BM;
        const int32_t grp = (m - ex.start) / kMGroup;
        const int32_t in_grp = (m - ex.start) % kMGroup * n_tiles + rem;
        const int32_t grp_rows = min(kMGroup, e_tiles - grp * kMGroup);
        at.e = scalar(ex.e);
        at.nt = scalar(in_grp / grp_rows);
        const int32_t first = scalar((grp * kMGroup + in_grp % grp_rows) * BM);
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
    start_tile<P, BM, NS>(p, next, st0, st1, wave, lane);
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
        constexpr int MT = BM / 16 / kWaveRows, M2 = (MT + 1) / 2, M1 = (MT + 3) / 4;
        if (at.valid > M2 * 32)
            run_tile<P, BM, NS, MT>(p, at, next, more, st0, st1, st2, wave_max, wave, lane);
        else if (at.valid > M1 * 32)
            run_tile<P, BM, NS, M2>(p, at, next, more, st0, st1, st2, wave_max, wave, lane);
        else
            run_tile<P, BM, NS, M1>(p, at, next, more, st0, st1, st2, wave_max, wave, lane);
        if (!more)
            break;
    }
}

// Row tiles of `rows` rows that a call can have: a segment's last one is partial.
int64_t max_tiles(const TrainGemmArgs &p, int32_t rows)
{
    if (p.recv_count == nullptr)
        return (p.max_rows + rows - 1) / rows;
    return p.max_rows / rows + (p.max_rows < p.E ? p.max_rows : p.E);
}

template <TrainProduct P, int BM, int NS>
hipError_t launch_tiles(const TrainGemmArgs &p, hipStream_t stream)
{
    const int32_t channels = P == kGated ? p.n / 2 : P == kGradInput ? p.k : p.n;
    const int32_t width = P == kGated ? kTileN / 2 : kTileN;
    const int32_t n_tiles = (channels + width - 1) / width;
    const int64_t tiles = max_tiles(p, BM) * n_tiles;
    // one block per compute unit (its stages fill LDS), a multiple of the 8 XCDs
    const int64_t cus = (device_cu_count() + 7) / 8 * 8;
    const int64_t grid = tiles < cus ? (tiles + 7) / 8 * 8 : cus;
    hipLaunchKernelGGL((train_gemm_tiles<P, BM, NS>), dim3((uint32_t)grid), dim3(kTileThreads), 0, stream, p, n_tiles);
    return hipGetLastError();
}

template <TrainProduct P>
hipError_t launch_product(const TrainGemmArgs &p, hipStream_t stream)
{
    if (p.max_rows / p.E >= 512)
        return launch_tiles<P, 256, 2>(p, stream);
    return launch_tiles<P, 128, 3>(p, stream);
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
