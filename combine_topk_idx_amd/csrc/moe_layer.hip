// A whole expert layer for at most 64 tokens on gfx950: two kernels, no
// dispatch.
//
//   gate_up:  h[t,k]  = bf16( silu(W13g[e] x[t]) * (W13u[e] x[t]) )
//   down:     out[t]  = bf16( sum_k topk_w[t,k] * W2[e] h[t,k] )
//
// Both are bound by the weights of the experts that the batch reaches, each
// byte of which is read once: a wave streams 16 weight rows straight from
// memory into matrix-instruction operands, converting 8-bit values to bf16 on
// the way (exact), and the activations stay bf16.  Tokens are the columns of
// the product.  gate_up has a block per (expert, 16 channels of h); down has a
// block per 16 output channels that walks every expert, with a zero column
// where a token does not use the expert, so that the weighted sum over a
// token's experts is the accumulation itself, in a fixed order and without
// atomics.
#include "moe_mma.h"

namespace moe {

namespace {

constexpr int kLayerWaves = 4;                       // gate_up: channel slices of one product
constexpr int kDownWaves = 8;                        // down: waves that share the experts
constexpr int kLayerMaxPairs = MOE_LAYER_MAX_TOKENS * kMaxTopk;
constexpr int kChunk = 64;                           // channels per weight load: 16 per lane

// 16 E4M3 values (16 bytes) times a power of two -> two bf16 operands of 8.
__device__ __forceinline__ void to_bf16(const dev::u32x4 &v, float scale, dev::bf16x8 &lo, dev::bf16x8 &hi)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const dev::bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[j], scale, false);
        const dev::bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[j], scale, true);
        lo[4 * j] = a[0], lo[4 * j + 1] = a[1], lo[4 * j + 2] = b[0], lo[4 * j + 3] = b[1];
        const dev::bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 + j], scale, false);
        const dev::bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[2 + j], scale, true);
        hi[4 * j] = c[0], hi[4 * j + 1] = c[1], hi[4 * j + 2] = d[0], hi[4 * j + 3] = d[1];
    }
}

// One lane's part of a 16-row weight strip (row `row` of [rows, k], or a clamped
// one): the 128 channels of block kb as four bf16 operands of 8 channels each
// (channels 16 g .. of each 64: the columns use the same order), multiplied by
// the block's scale where that is a power of two.
template <int QUANT>
struct Weights {
    dev::u32x4 v[QUANT == MOE_QUANT_NONE ? 4 : 2];
    float s[2];   // power-of-two scales of the two 64-channel halves; FP8_F32: s[0] = the block's scale

    __device__ __forceinline__ void load(const uint8_t *w, const void *scale, int64_t row, int64_t nb, int k, int kb,
                                         int g)
    {
        const int KB = k / kQuantGroup;
        if constexpr (QUANT == MOE_QUANT_NONE) {
            const uint8_t *p = w + (row * k + (int64_t)kb * kQuantGroup + 16 * g) * 2;
            v[0] = *reinterpret_cast<const dev::u32x4 *>(p);
            v[1] = *reinterpret_cast<const dev::u32x4 *>(p + 16);
            v[2] = *reinterpret_cast<const dev::u32x4 *>(p + 128);
            v[3] = *reinterpret_cast<const dev::u32x4 *>(p + 144);
        } else {
            const uint8_t *p = w + row * k + (int64_t)kb * kQuantGroup + 16 * g;
            v[0] = *reinterpret_cast<const dev::u32x4 *>(p);
            v[1] = *reinterpret_cast<const dev::u32x4 *>(p + 64);
            if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                s[0] = static_cast<const float *>(scale)[nb * KB + kb];
            } else if constexpr (QUANT == MOE_QUANT_FP8_UE8M0) {
                const uint8_t b = static_cast<const uint8_t *>(scale)[nb * ((KB + 3) / 4 * 4) + kb];
                s[0] = s[1] = __uint_as_float((uint32_t)b << 23);
            } else {
                const uint8_t *q = static_cast<const uint8_t *>(scale) + (row * KB + kb) * 4 + (g >> 1);
                s[0] = __uint_as_float((uint32_t)q[0] << 23);
                s[1] = __uint_as_float((uint32_t)q[2] << 23);
            }
        }
    }
    // acc += W * x over the block; x: four operands of the column
    __device__ __forceinline__ void fma(const dev::bf16x8 x[4], dev::f32x4 &acc, const dev::bf16x8 wv[4]) const
    {
        if constexpr (QUANT == MOE_QUANT_FP8_F32) {
            dev::f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], x[j], d, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] = __builtin_fmaf(d[j], s[0], acc[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], x[j], acc, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void convert(dev::bf16x8 wv[4]) const
    {
        if constexpr (QUANT == MOE_QUANT_NONE) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                wv[j] = __builtin_bit_cast(dev::bf16x8, v[j]);
        } else if constexpr (QUANT == MOE_QUANT_FP8_F32) {
            to_bf16(v[0], 1.0f, wv[0], wv[1]);
            to_bf16(v[1], 1.0f, wv[2], wv[3]);
        } else {
            to_bf16(v[0], s[0], wv[0], wv[1]);
            to_bf16(v[1], s[1], wv[2], wv[3]);
        }
    }
};

// The matching operands of a column: 128 channels of a bf16 row, zeros where
// there is no row.
__device__ __forceinline__ void load_column(const uint16_t *row, bool on, int kb, int g, dev::bf16x8 x[4])
{
    const uint16_t *p = row + kb * kQuantGroup + 16 * g;
    dev::u32x4 v[4] = {};
    if (on) {
        v[0] = *reinterpret_cast<const dev::u32x4 *>(p);
        v[1] = *reinterpret_cast<const dev::u32x4 *>(p + 8);
        v[2] = *reinterpret_cast<const dev::u32x4 *>(p + 64);
        v[3] = *reinterpret_cast<const dev::u32x4 *>(p + 72);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        x[j] = __builtin_bit_cast(dev::bf16x8, v[j]);
}

// Block (pair p, 16 channels of h): runs for the first pair of each expert and
// computes h for every pair of that expert, 16 at a time.
template <int QUANT>
__global__ __launch_bounds__(kLayerWaves *kWave) void layer_gate_up(LayerArgs a)
{
    __shared__ int32_t ids[kLayerMaxPairs];
    __shared__ int16_t list[kLayerMaxPairs];
    __shared__ int32_t n_list;
    __shared__ float part[kLayerWaves][2][kWave][4];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int P = a.T * a.K;
    const int pair = blockIdx.y;
    const int tile = blockIdx.x;
    const int32_t e = __builtin_amdgcn_readfirstlane(a.topk_idx[pair]);
    if (e < 0 || e >= a.E)
        return;
    for (int i = tid; i < P; i += kLayerWaves * kWave)
        ids[i] = a.topk_idx[i];
    __syncthreads();
    bool earlier = false;
    for (int i = lane; i < pair; i += kWave)
        earlier |= ids[i] == e;
    if (__ballot(earlier) != 0)  // every wave finds the same
        return;
    if (wave == 0) {
        int n = 0;
        for (int i0 = 0; i0 < P; i0 += kWave) {
            const int i = i0 + lane;
            const bool mine = i >= pair && i < P && ids[i] == e;
            const uint64_t m = __ballot(mine);
            if (mine)
                list[n + dev::lanes_below(m)] = (int16_t)i;
            n += __popcll(m);
        }
        if (lane == 0)
            n_list = n;
    }
    __syncthreads();
    const int n = n_list;
    const int KB = a.H / kQuantGroup;
    const int c0 = tile * 16;
    const int64_t grow = (int64_t)e * 2 * a.I + c0 + r, urow = grow + a.I;
    const int NBn = 2 * a.I / kQuantGroup;
    const int64_t gnb = (int64_t)e * NBn + c0 / kQuantGroup, unb = gnb + a.I / kQuantGroup;

    for (int j0 = 0; j0 < n; j0 += 16) {
        const bool on = j0 + r < n;
        const int my = on ? list[j0 + r] : 0;
        const uint16_t *x = a.x + (int64_t)(my / a.K) * a.H;
        dev::f32x4 accg = {0.0f, 0.0f, 0.0f, 0.0f}, accu = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int kb = wave; kb < KB; kb += kLayerWaves) {
            Weights<QUANT> wg, wu;
            wg.load(a.w13, a.w13_scale, grow, gnb, a.H, kb, g);
            wu.load(a.w13, a.w13_scale, urow, unb, a.H, kb, g);
            dev::bf16x8 xv[4], wv[4];
            load_column(x, on, kb, g, xv);
            wg.convert(wv);
            wg.fma(xv, accg, wv);
            wu.convert(wv);
            wu.fma(xv, accu, wv);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            part[wave][0][lane][j] = accg[j];
            part[wave][1][lane][j] = accu[j];
        }
        __syncthreads();
        if (wave == 0) {
            float gv[4] = {}, uv[4] = {};
#pragma unroll
            for (int w = 0; w < kLayerWaves; ++w)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    gv[j] += part[w][0][lane][j];
                    uv[j] += part[w][1][lane][j];
                }
            if (on)
                *reinterpret_cast<uint2 *>(a.h + (int64_t)my * a.I + c0 + g * 4) =
                    make_uint2(dev::pack_bf16(dev::swiglu(gv[0], uv[0]), dev::swiglu(gv[1], uv[1])),
                               dev::pack_bf16(dev::swiglu(gv[2], uv[2]), dev::swiglu(gv[3], uv[3])));
        }
        __syncthreads();
    }
}

// Block of 16 output channels: walks the experts (wave w takes every
// kDownWaves-th one), tokens in groups of 16 columns.
template <int QUANT, int G>
__global__ __launch_bounds__(kDownWaves *kWave) void layer_down(LayerArgs a)
{
    __shared__ int32_t ids[kLayerMaxPairs];
    __shared__ int16_t leaders[kLayerMaxPairs];
    __shared__ int32_t n_leaders;
    __shared__ float part[kDownWaves][G][kWave][4];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int P = a.T * a.K;
    for (int i = tid; i < P; i += kDownWaves * kWave)
        ids[i] = a.topk_idx[i];
    if (tid == 0)
        n_leaders = 0;
    __syncthreads();
    if (wave == 0) {  // the first pair of every expert, in pair order
        int n = 0;
        for (int i0 = 0; i0 < P; i0 += kWave) {
            const int i = i0 + lane;
            bool lead = i < P && ids[i] >= 0 && ids[i] < a.E;
            for (int j = 0; lead && j < i; ++j)
                lead = ids[j] != ids[i];
            const uint64_t m = __ballot(lead);
            if (lead)
                leaders[n + dev::lanes_below(m)] = (int16_t)i;
            n += __popcll(m);
        }
        if (lane == 0)
            n_leaders = n;
    }
    __syncthreads();
    const int n = n_leaders;
    const int KB = a.I / kQuantGroup;
    const int c0 = blockIdx.x * 16;
    const int NBn = a.H / kQuantGroup;

    dev::f32x4 acc[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
        acc[i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = wave; j < n; j += kDownWaves) {
        const int32_t e = __builtin_amdgcn_readfirstlane(ids[leaders[j]]);
        const int64_t row = (int64_t)e * a.H + c0 + r;
        const int64_t nb = (int64_t)e * NBn + c0 / kQuantGroup;
        // this lane's tokens: their pair of the expert and its weight (summed where it is there twice)
        int pair[G];
        float gate[G];
        uint64_t any[G];
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int t = i * 16 + r;
            pair[i] = -1;
            gate[i] = 0.0f;
            if (t < a.T)
                for (int k = 0; k < a.K; ++k)
                    if (ids[t * a.K + k] == e) {
                        gate[i] += a.topk_w[t * a.K + k];
                        if (pair[i] < 0)
                            pair[i] = t * a.K + k;
                    }
            any[i] = __ballot(pair[i] >= 0);
        }
        dev::f32x4 sum[G];
#pragma unroll
        for (int i = 0; i < G; ++i)
            sum[i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int kb = 0; kb < KB; ++kb) {
            Weights<QUANT> w;
            w.load(a.w2, a.w2_scale, row, nb, a.I, kb, g);
            dev::bf16x8 wv[4], xv[4];
            w.convert(wv);
#pragma unroll
            for (int i = 0; i < G; ++i)
                if (any[i] != 0) {
                    load_column(a.h + (int64_t)max(pair[i], 0) * a.I, pair[i] >= 0, kb, g, xv);
                    w.fma(xv, sum[i], wv);
                }
        }
#pragma unroll
        for (int i = 0; i < G; ++i)
            if (pair[i] >= 0)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[i][q] = __builtin_fmaf(sum[i][q], gate[i], acc[i][q]);
    }
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
            part[wave][i][lane][q] = acc[i][q];
    __syncthreads();
    if (wave < G) {
        float v[4] = {};
#pragma unroll
        for (int w = 0; w < kDownWaves; ++w)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] += part[w][wave][lane][q];
        const int t = wave * 16 + r;
        if (t < a.T)
            *reinterpret_cast<uint2 *>(a.out + (int64_t)t * a.H + c0 + g * 4) =
                make_uint2(dev::pack_bf16(v[0], v[1]), dev::pack_bf16(v[2], v[3]));
    }
}

template <int QUANT>
hipError_t launch_quant(const LayerArgs &a, hipStream_t stream)
{
    hipLaunchKernelGGL((layer_gate_up<QUANT>), dim3(a.I / 16, a.T * a.K), dim3(kLayerWaves * kWave), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const dim3 grid(a.H / 16), block(kDownWaves * kWave);
    if (a.T <= 16)
        hipLaunchKernelGGL((layer_down<QUANT, 1>), grid, block, 0, stream, a);
    else if (a.T <= 32)
        hipLaunchKernelGGL((layer_down<QUANT, 2>), grid, block, 0, stream, a);
    else
        hipLaunchKernelGGL((layer_down<QUANT, 4>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer(const LayerArgs &a, int32_t quant, hipStream_t stream)
{
    switch (quant) {
    case MOE_QUANT_NONE:
        return launch_quant<MOE_QUANT_NONE>(a, stream);
    case MOE_QUANT_FP8_F32:
        return launch_quant<MOE_QUANT_FP8_F32>(a, stream);
    case MOE_QUANT_FP8_UE8M0:
        return launch_quant<MOE_QUANT_FP8_UE8M0>(a, stream);
    default:
        return launch_quant<MOE_QUANT_MXFP8>(a, stream);
    }
}

}  // namespace moe
