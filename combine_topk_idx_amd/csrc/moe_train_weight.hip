// The gradient of the experts' products to their weights and biases on gfx950:
//
//   dw[e, j, c] = sum over rows of e of dy[row, j] a[row, c],  dbias[e, j] = sum of dy[row, j]
//
// A block holds 256 x 256 of one expert's weights and walks its rows, 64 a step.
// Both operands are summed over their slow axis: the stages hold them as they lie
// in memory and ds_read_b64_tr_b16 hands each lane four rows of one channel.
// dbias comes from the same fragments, times ones.
#include "moe_train_internal.h"
#include "moe_train_tiles.h"

namespace moe {

namespace {

using namespace tile;
using namespace tile::train;

constexpr int kTileM = 256;  // channels of dy per block
constexpr int kStageBytes = (kTileM + kTileN) * kStep * 2;
constexpr int kHalf = kTileM * kStep * 2;  // a's channels follow dy's
constexpr int MT = kTileM / 16 / kWaveRows;

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
template <int QUANT>
struct WeightLoads {
    const uint16_t *dy;
    const uint8_t *a, *scale;
    uint32_t so, sstep, to;  // 8 bits: this lane's first scale, and its place in a stage
    uint32_t yo, ao;     // this lane's place in its first row
    uint32_t ystep, astep;  // 16 rows further
    int32_t rows, n, k, wave;

    __device__ __forceinline__ void set(const GradWeightArgs &p, const WeightTile &at, int wave_, int lane)
    {
        wave = wave_;
        rows = at.rows;
        n = p.n;
        k = p.k;
        dy = p.dy + at.row0 * n;
        a = static_cast<const uint8_t *>(p.a) + at.row0 * k * (QUANT == MOE_QUANT_NONE ? 2 : 1);
        // 32 bytes (16 channels) of row s sit at position c ^ (s & 3 | s >> 1 & 4) of
        // its 512: what 32 lanes read at once then covers all banks.  A wave loads
        // rows 2 j and 2 j + 1, j = wave (mod 8).
        const int s = 2 * wave + (lane >> 5);
        const int f = (s & 3) | ((s >> 1) & 4);
        const int32_t c = ((((lane & 31) >> 1) ^ f) * 2 + (lane & 1)) * 8;
        const int32_t j = at.mt * kTileM + c, i = at.nt * kTileN + c;
        yo = j < n ? (uint32_t)s * (uint32_t)n * 2 + (uint32_t)j * 2 : 0x80000000u;
        ao = i < k ? (uint32_t)s * (uint32_t)k * 2 + (uint32_t)i * 2 : 0x80000000u;
        ystep = 32u * (uint32_t)n;
        astep = 32u * (uint32_t)k;
        if constexpr (QUANT != MOE_QUANT_NONE) {
            const int32_t piece = lane & 31, at_c = at.nt * kTileN + piece * 8;
            ao = at_c < k ? (uint32_t)s * (uint32_t)k + (uint32_t)at_c : 0x80000000u;
            astep = 16u * (uint32_t)k;
            so = at_c < k ? (uint32_t)s * scale_bytes() + (uint32_t)(at_c / (QUANT == MOE_QUANT_MXFP8 ? 32 : 128)) *
                                                              (QUANT == MOE_QUANT_FP8_F32 ? 4 : 1)
                          : 0x80000000u;
            sstep = 16u * scale_bytes();
            to = (uint32_t)s * 512 + (((piece >> 1) ^ f) * 2 + (piece & 1)) * 16;
            scale = static_cast<const uint8_t *>(p.a_scale) + at.row0 * scale_bytes();
        }
    }
    // Bytes of a row's scales.
    __device__ __forceinline__ uint32_t scale_bytes() const
    {
        const uint32_t b = (uint32_t)k / kQuantGroup;
        return QUANT == MOE_QUANT_FP8_UE8M0 ? (b + 3) / 4 * 4 : b * 4;
    }
    // a in 8 bits: the rows of step kb into registers, and from there into a stage.
    __device__ __forceinline__ void fetch(Rows8<QUANT> &rows8, int kb) const
    {
        const int32_t r0 = kb * kStep;
        const uint32_t left = (uint32_t)max(0, min(kStep, rows - r0));
        const __amdgpu_buffer_rsrc_t av = buffer(a + (int64_t)r0 * k, left * (uint32_t)k);
        const __amdgpu_buffer_rsrc_t sv = buffer(scale + (int64_t)r0 * scale_bytes(), left * scale_bytes());
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rows8.v[i] = __builtin_amdgcn_raw_buffer_load_b64(av, ao + i * astep, 0, 0);
            if constexpr (QUANT == MOE_QUANT_FP8_F32)
                rows8.s[i] = __builtin_amdgcn_raw_buffer_load_b32(sv, so + i * sstep, 0, 0);
            else
                rows8.s[i] = __builtin_amdgcn_raw_buffer_load_b8(sv, so + i * sstep, 0, 0);
        }
    }
    __device__ __forceinline__ void put(const Rows8<QUANT> &rows8, uint8_t *st) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<dev::u32x4 *>(st + kHalf + to + i * 16 * 512) = rows8.bf16(i);
    }
    // Loads FROM .. TO - 1 of the 8 of step kb.
    template <int FROM, int TO>
    __device__ __forceinline__ void issue(uint8_t *st, int kb) const
    {
        const int32_t r0 = kb * kStep;
        const uint32_t left = (uint32_t)max(0, min(kStep, rows - r0));
#pragma unroll
        for (int j = FROM; j < TO; ++j) {
            const int i = j & 3;
            if (j < 4)
                load_lds<16>(buffer(dy + (int64_t)r0 * n, left * (uint32_t)n * 2), st + (wave + 8 * i) * 1024,
                             yo + i * ystep, 0);
            else if constexpr (QUANT == MOE_QUANT_NONE)
                load_lds<16>(buffer(a + (int64_t)r0 * k * 2, left * (uint32_t)k * 2),
                             st + kHalf + (wave + 8 * i) * 1024, ao + i * astep, 0);
        }
    }
};

struct WeightSums {
    dev::f32x4 w[kNF][MT];
    dev::f32x4 bias[MT / kWaveCols];  // the waves of a row share its fragments
};

template <int QUANT>
__device__ __forceinline__ void multiply_rows(WeightSums &acc, const uint8_t *st, int wr, int wc, int lane, bool bias,
                                              const WeightLoads<QUANT> &loads, uint8_t *free, int kb_load)
{
    const int r = lane & 15, g = lane >> 4;
    const int column = (8 * g + (r >> 2)) * 2 * kTileN + ((r >> 2) | (g & 1) << 2) * 32 + (r & 3) * 8;
    const uint8_t *rows = st, *ws = st + kHalf;
    Fragment w[kNF], x[2];
    x[0] = read_columns<kTileM>(rows + (column ^ (wr * MT) * 32));
#pragma unroll
    for (int f = 0; f < kNF; ++f)
        w[f] = read_columns<kTileN>(ws + (column ^ (wc * 4 + f) * 32));
    const auto part = [&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (i + 1 < MT)
            x[(i + 1) & 1] = read_columns<kTileM>(rows + (column ^ (wr * MT + i + 1) * 32));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int f = 0; f < kNF; ++f)
                acc.w[f][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[f].h[h], x[i & 1].h[h], acc.w[f][i], 0, 0, 0);
        if (bias && wc == (i & (kWaveCols - 1))) {
            const __bf16 one = (__bf16)1.0f;
            const dev::bf16x8 ones = {one, one, one, one, one, one, one, one};
#pragma unroll
            for (int h = 0; h < 2; ++h)
                acc.bias[i / kWaveCols] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, x[i & 1].h[h],
                                                                                  acc.bias[i / kWaveCols], 0, 0, 0);
        }
        loads.template issue<i, i + 1>(free, kb_load);
        __builtin_amdgcn_sched_barrier(0);
    };
    static_assert(MT == 8, "a load per fragment of rows");
    for_each<MT>(part);
}

// Results: channels 16 (MT wr + i) + (lane % 16) of dy, 4 (lane / 16) + j of
// fragment f.  Parts of a split go to the workspace.
__device__ __forceinline__ void write_weights(const GradWeightArgs &p, const WeightSums &acc, const WeightTile &at, int wr,
                                              int wc, int lane)
{
    const int r = lane & 15, g = lane >> 4;
    const int32_t j0 = at.mt * kTileM, c0 = at.nt * kTileN + wc * 64;
    const int32_t valid = min(kTileM, p.n - j0);
    const bool parts = p.splits > 1;
    const int64_t group = parts ? (int64_t)at.e * p.splits + at.split : at.e;
    const int64_t first = (group * p.n + j0) * p.k;
    if (!parts && p.dw_bf16) {
        const __amdgpu_buffer_rsrc_t out =
            buffer(static_cast<uint16_t *>(p.dw) + first, (uint32_t)valid * (uint32_t)p.k * 2);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const dev::f32x4 v[kNF] = {acc.w[0][i], acc.w[1][i], acc.w[2][i], acc.w[3][i]};
            store_lines(out, v, (wr * MT + i) * 16, valid, c0, p.k, lane);
        }
    } else {
        const bool add = !parts && p.accumulate;
        const __amdgpu_buffer_rsrc_t out =
            buffer((parts ? p.partial : static_cast<float *>(p.dw)) + first, (uint32_t)valid * (uint32_t)p.k * 4);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int f = 0; f < kNF; ++f) {
                const int row = (wr * MT + i) * 16 + r;
                const int32_t c = c0 + f * 16 + 4 * g;
                const uint32_t off = row < valid && c < p.k ? ((uint32_t)row * (uint32_t)p.k + c) * 4 : 0x80000000u;
                dev::f32x4 v = acc.w[f][i];
                if (add)
                    v += __builtin_bit_cast(dev::f32x4, __builtin_amdgcn_raw_buffer_load_b128(out, off, 0, 0));
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(dev::u32x4, v), out, off, 0, kStreamed);
            }
    }
    if (p.dbias != nullptr && at.nt == 0 && g == 0) {
        float *out = parts ? p.partial + (int64_t)p.E * p.splits * p.n * p.k : p.dbias;
#pragma unroll
        for (int b = 0; b < MT / kWaveCols; ++b) {
            const int row = (wr * MT + b * kWaveCols + wc) * 16 + r;
            if (row < valid) {
                float *to = out + group * p.n + j0 + row;
                *to = !parts && p.accumulate ? *to + acc.bias[b][0] : acc.bias[b][0];
            }
        }
    }
}

template <int QUANT>
__global__ __launch_bounds__(kTileThreads) void grad_weight_tiles(GradWeightArgs p, int32_t m_tiles, int32_t n_tiles)
{
    __shared__ alignas(1024) uint8_t st0[kStageBytes];
    __shared__ alignas(1024) uint8_t st1[kStageBytes];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = scalar(threadIdx.x / kWave);
    const int wr = wave / kWaveCols, wc = wave % kWaveCols;
    const int64_t tiles = (int64_t)m_tiles * n_tiles;
    const int64_t n_work = tiles * p.E * p.splits;
    for (int64_t work = blockIdx.x; work < n_work; work += gridDim.x) {
        WeightTile at;
        const int32_t part = scalar((int32_t)(work / tiles));
        const int32_t t = scalar((int32_t)(work - part * tiles));
        at.e = scalar(part / p.splits);
        at.split = part - at.e * p.splits;
        at.nt = scalar(t / m_tiles);
        at.mt = t - at.nt * m_tiles;
        const int32_t rows = p.recv_count != nullptr ? word_of(p.recv_count, at.e) : p.dense_rows;
        const int32_t steps = (rows + kStep - 1) / kStep;
        const int32_t s0 = scalar((int32_t)((int64_t)steps * at.split / p.splits));
        const int32_t s1 = scalar((int32_t)((int64_t)steps * (at.split + 1) / p.splits));
        at.rows = scalar(min(rows, s1 * kStep) - min(rows, s0 * kStep));
        at.row0 = (int64_t)(p.expert_offset != nullptr ? word_of(p.expert_offset, at.e) : 0) + s0 * kStep;
        const bool bias = p.dbias != nullptr && at.nt == 0;

        WeightLoads<QUANT> loads;
        loads.set(p, at, wave, lane);
        WeightSums acc;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int f = 0; f < kNF; ++f)
                acc.w[f][i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < MT / kWaveCols; ++b)
            acc.bias[b] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        loads.template issue<0, 8>(st0, 0);
        Rows8<QUANT> rows8;
        if constexpr (QUANT != MOE_QUANT_NONE) {
            loads.fetch(rows8, 0);
            loads.put(rows8, st0);
        }
        const int KB = s1 - s0;
        const auto step = [&](uint8_t *cur, uint8_t *free, int kb) {
            wait_and_meet<0>();
            if constexpr (QUANT != MOE_QUANT_NONE)
                loads.fetch(rows8, kb + 1);
            multiply_rows<QUANT>(acc, cur, wr, wc, lane, bias, loads, free, kb + 1);
            if constexpr (QUANT != MOE_QUANT_NONE)
                loads.put(rows8, free);
        };
        int kb = 0;
        for (; kb + 2 <= KB; kb += 2) {
            step(st0, st1, kb);
            step(st1, st0, kb + 1);
        }
        if (kb < KB)
            step(st0, st1, kb);
        write_weights(p, acc, at, wr, wc, lane);
        wait_and_meet<0>();  // the next tile loads into both stages
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
    dev::f32x4 *to = reinterpret_cast<dev::f32x4 *>((bias ? p.dbias : static_cast<float *>(p.dw)) + i);
    *to = p.accumulate ? *to + v : v;
}

}  // namespace

int32_t grad_weight_splits(int64_t max_rows, int32_t E, int32_t n, int32_t k)
{
    const int64_t tiles = (int64_t)E * ((n + kTileM - 1) / kTileM) * ((k + kTileN - 1) / kTileN);
    const int64_t steps = max_rows / E / kStep;  // of an expert, evenly routed
    const int64_t splits = tiles >= 128 ? 1 : 256 / tiles;
    return (int32_t)(splits < steps / 8 ? splits : steps / 8 < 1 ? 1 : steps / 8);
}

hipError_t launch_grad_weight(const GradWeightArgs &p, hipStream_t stream)
{
    const int32_t m_tiles = (p.n + kTileM - 1) / kTileM, n_tiles = (p.k + kTileN - 1) / kTileN;
    const int64_t work = (int64_t)m_tiles * n_tiles * p.E * p.splits;
    const int64_t cus = device_cu_count();
    const dim3 grid((uint32_t)(work < cus ? work : cus)), block(kTileThreads);
    switch (p.a_quant) {
    case MOE_QUANT_FP8_F32:
        hipLaunchKernelGGL((grad_weight_tiles<MOE_QUANT_FP8_F32>), grid, block, 0, stream, p, m_tiles, n_tiles);
        break;
    case MOE_QUANT_FP8_UE8M0:
        hipLaunchKernelGGL((grad_weight_tiles<MOE_QUANT_FP8_UE8M0>), grid, block, 0, stream, p, m_tiles, n_tiles);
        break;
    case MOE_QUANT_MXFP8:
        hipLaunchKernelGGL((grad_weight_tiles<MOE_QUANT_MXFP8>), grid, block, 0, stream, p, m_tiles, n_tiles);
        break;
    default:
        hipLaunchKernelGGL((grad_weight_tiles<MOE_QUANT_NONE>), grid, block, 0, stream, p, m_tiles, n_tiles);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1)
        return e;
    const int64_t quads = (int64_t)p.E * p.n * p.k / 4, all = quads + (p.dbias != nullptr ? (int64_t)p.E * p.n / 4 : 0);
    hipLaunchKernelGGL(grad_weight_join, dim3((uint32_t)((all + kBlockThreads - 1) / kBlockThreads)), dim3(kBlockThreads),
                       0, stream, p, quads, all);
    return hipGetLastError();
}

}  // namespace moe
