// Row kernels of the expert layer's gradients on gfx950: the activations' (from
// saved rows in bf16 or 8 bits) and combine's.  Both read each input once and
// write each output once; HBM bounds them.
//
// 65,536 rows of 2048 channels, gated, MXFP8: 1.35 GB in 261 us, 5.2 TB/s.  Combine's, 8192
// tokens x 8, 7168 channels: 2.0 GB in 400 us, 5.0 TB/s (a copy reaches 4.9).  Small calls
// take 4 us of a launch and two dependent round trips.
#include "moe_act.h"

namespace moe {

namespace {

// The value of a stored power-of-two scale byte.
__device__ __forceinline__ float byte_scale(uint32_t b)
{
    return __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
}

// Scale of the block that holds channel c of row `row`, m channels wide.
template <int QUANT>
__device__ __forceinline__ float row_scale(const void *scale, int64_t row, int32_t m, int32_t c)
{
    if constexpr (QUANT == MOE_QUANT_FP8_F32)
        return static_cast<const float *>(scale)[row * (m / kQuantGroup) + c / kQuantGroup];
    else if constexpr (QUANT == MOE_QUANT_FP8_UE8M0)
        return byte_scale(static_cast<const uint8_t *>(scale)[row * ((m / kQuantGroup + 3) / 4 * 4) + c / kQuantGroup]);
    else if constexpr (QUANT == MOE_QUANT_MXFP8)
        return byte_scale(static_cast<const uint8_t *>(scale)[row * (m / 32) + c / 32]);
    return 1.0f;
}

__device__ __forceinline__ void unpack_bf16(const uint4 &u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = dev::bf16_lo(w[j]);
        v[2 * j + 1] = dev::bf16_hi(w[j]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(dev::pack_bf16(v[0], v[1]), dev::pack_bf16(v[2], v[3]), dev::pack_bf16(v[4], v[5]),
                      dev::pack_bf16(v[6], v[7]));
}

// 8 channels of a saved row, as they are stored.
template <int QUANT>
struct Saved {
    uint4 v;  // 8-bit formats: two words
    float s;
    __device__ __forceinline__ void load(const ActBackwardArgs &a, int64_t row, int32_t m, int32_t c)
    {
        if constexpr (QUANT == MOE_QUANT_NONE) {
            v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.saved) + row * m + c);
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.saved) + row * m + c);
            v = make_uint4(w.x, w.y, 0, 0);
            s = row_scale<QUANT>(a.saved_scale, row, m, c);
        }
    }
    __device__ __forceinline__ void values(float (&f)[8]) const
    {
        if constexpr (QUANT == MOE_QUANT_NONE) {
            unpack_bf16(v, f);
        } else {
            const uint32_t w[2] = {v.x, v.y};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[j], false);
                const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[j], true);
                f[4 * j] = lo[0] * s;
                f[4 * j + 1] = lo[1] * s;
                f[4 * j + 2] = hi[0] * s;
                f[4 * j + 3] = hi[1] * s;
            }
        }
    }
};

// `per` threads per row (a power of two), 8 channels each at a time.
template <bool GATED, int QUANT>
__global__ __launch_bounds__(kBlockThreads) void activation_backward_kernel(ActBackwardArgs a, int32_t per)
{
    const int32_t m = GATED ? 2 * a.n : a.n;
    const int32_t rows_per_block = kBlockThreads / per, sub = threadIdx.x / per;
    for (int64_t row = (int64_t)blockIdx.x * rows_per_block + sub; row < a.rows;
         row += (int64_t)gridDim.x * rows_per_block) {
        if (a.row_to_pair != nullptr && a.row_to_pair[row] < 0)
            continue;
        for (int32_t c = (threadIdx.x - sub * per) * 8; c < a.n; c += per * 8) {
            const uint4 dyv = *reinterpret_cast<const uint4 *>(a.dy + row * a.n + c);
            Saved<QUANT> g, u;
            g.load(a, row, m, c);
            if constexpr (GATED)
                u.load(a, row, m, a.n + c);
            float dy[8], gv[8], uv[8], dg[8], du[8], y[8];
            unpack_bf16(dyv, dy);
            g.values(gv);
            if constexpr (GATED)
                u.values(uv);
            dev::for_act(a.act, [&](auto act) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float f, slope;
                    dev::act_both<decltype(act)::value>(gv[j], f, slope);
                    if constexpr (GATED) {
                        dg[j] = dy[j] * uv[j] * slope;
                        du[j] = dy[j] * f;
                        y[j] = f * uv[j];
                    } else {
                        dg[j] = dy[j] * slope;
                        y[j] = f;
                    }
                }
            });
            *reinterpret_cast<uint4 *>(a.dsaved + row * m + c) = pack8(dg);
            if constexpr (GATED)
                *reinterpret_cast<uint4 *>(a.dsaved + row * m + a.n + c) = pack8(du);
            if (a.y != nullptr)
                *reinterpret_cast<uint4 *>(a.y + row * a.n + c) = pack8(y);
        }
    }
}

// A wave per pair: its row of y and of dy, and its token's of dout, which the
// waves of one token share in the caches.
__global__ __launch_bounds__(kBlockThreads) void combine_backward_kernel(CombineBackwardArgs a, int64_t pairs)
{
    constexpr int kVecs = 4;  // 16-byte vectors per lane and array in flight
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t step = (int64_t)gridDim.x * kWavesPerBlock;
    for (int64_t p = (int64_t)blockIdx.x * kWavesPerBlock + threadIdx.x / kWave; p < pairs; p += step) {
        const int32_t row = a.pair_to_row[p];
        if (row < 0) {
            if (a.dtopk_w != nullptr && lane == 0)
                a.dtopk_w[p] = 0.0f;
            continue;
        }
        const float w = a.topk_w[p];
        const uint16_t *dout = a.dout + p / a.K * a.H;
        const uint16_t *y = a.y + (int64_t)row * a.H;
        uint16_t *dy = a.dy + (int64_t)row * a.H;
        const bool dot = a.dtopk_w != nullptr;
        float sum[kVecs] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int32_t c0 = lane * 8; c0 < a.H; c0 += kVecs * kWave * 8) {
            uint4 d[kVecs], v[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int32_t c = c0 + i * kWave * 8;
                if (c < a.H) {
                    d[i] = *reinterpret_cast<const uint4 *>(dout + c);
                    if (dot)
                        v[i] = *reinterpret_cast<const uint4 *>(y + c);
                }
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int32_t c = c0 + i * kWave * 8;
                if (c >= a.H)
                    break;
                float df[8], vf[8], out[8];
                unpack_bf16(d[i], df);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    out[j] = w * df[j];
                *reinterpret_cast<uint4 *>(dy + c) = pack8(out);
                if (dot) {
                    unpack_bf16(v[i], vf);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sum[i] = __builtin_fmaf(df[j], vf[j], sum[i]);
                }
            }
        }
        if (dot) {
            float s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
            for (int m = 1; m < kWave; m <<= 1)
                s += __shfl_xor(s, m);
            if (lane == 0)
                a.dtopk_w[p] = s;
        }
    }
}

template <bool GATED>
hipError_t launch_act(const ActBackwardArgs &a, hipStream_t stream)
{
    int32_t per = 1;
    while (per < kBlockThreads && per * 8 < a.n)
        per *= 2;
    const int64_t blocks = ((int64_t)a.rows * per + kBlockThreads - 1) / kBlockThreads;
    const int64_t most = (int64_t)device_cu_count() * 32;
    const dim3 grid((uint32_t)(blocks < most ? blocks : most)), block(kBlockThreads);
    switch (a.quant) {
    case MOE_QUANT_FP8_F32:
        hipLaunchKernelGGL((activation_backward_kernel<GATED, MOE_QUANT_FP8_F32>), grid, block, 0, stream, a, per);
        break;
    case MOE_QUANT_FP8_UE8M0:
        hipLaunchKernelGGL((activation_backward_kernel<GATED, MOE_QUANT_FP8_UE8M0>), grid, block, 0, stream, a, per);
        break;
    case MOE_QUANT_MXFP8:
        hipLaunchKernelGGL((activation_backward_kernel<GATED, MOE_QUANT_MXFP8>), grid, block, 0, stream, a, per);
        break;
    default:
        hipLaunchKernelGGL((activation_backward_kernel<GATED, MOE_QUANT_NONE>), grid, block, 0, stream, a, per);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_activation_backward(const ActBackwardArgs &a, bool gated, hipStream_t stream)
{
    return gated ? launch_act<true>(a, stream) : launch_act<false>(a, stream);
}

hipError_t launch_combine_backward(const CombineBackwardArgs &a, hipStream_t stream)
{
    const int64_t pairs = (int64_t)a.T * a.K;
    const int64_t blocks = (pairs + kWavesPerBlock - 1) / kWavesPerBlock;
    const int64_t most = (int64_t)device_cu_count() * 64;
    hipLaunchKernelGGL(combine_backward_kernel, dim3((uint32_t)(blocks < most ? blocks : most)), dim3(kBlockThreads), 0,
                       stream, a, pairs);
    return hipGetLastError();
}

}  // namespace moe
