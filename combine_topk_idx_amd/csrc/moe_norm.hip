// Residual add + root-mean-square norm on gfx950, with the normed rows in 8
// bits beside or instead of bf16.
//
//   r = bf16(x + residual), y = r / sqrt(mean(r^2) + eps) * weight
//
// One pass: a row stays in its threads' registers between the sum of squares
// and the outputs, so every input is read once and every output written once.
// Lanes hold 8 channels (one 16-byte load), so a 128-channel quantization block
// is 16 adjacent lanes -- one DPP row -- and an MX block of 32 is one quad.
#include "moe_mma.h"

namespace moe {

namespace {

// max over a row of 16 lanes
__device__ __forceinline__ float max16(float v)
{
    v = dev::max8(v);
    return fmaxf(v, dev::dpp<0x140>(v));  // row_mirror: the other half of the row
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1)
        v += __shfl_xor(v, m);
    return v;
}

// A row is handled by THREADS threads with up to NV vectors of 8 channels each
// (H <= 8 * THREADS * NV); the block holds ROWS rows, the grid those from `first`.
template <int QUANT, int THREADS, int ROWS, int NV>
__global__ __launch_bounds__(THREADS *ROWS) void rmsnorm_kernel(NormArgs a, int64_t first)
{
    constexpr int kWaves = THREADS / kWave;
    __shared__ float red[ROWS][kWaves];
    const int sub = ROWS == 1 ? 0 : threadIdx.x / THREADS;
    const int tid = threadIdx.x - sub * THREADS;
    const int lane = tid & (kWave - 1);
    const int64_t t = first + (int64_t)blockIdx.x * ROWS + sub;
    const bool live = ROWS == 1 || t < a.T;
    const int nvec = a.H / 8;
    const int64_t base = t * a.H;

    uint4 v[NV], wv[NV], rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * THREADS + tid) * 8;
        if (live && c < a.H) {
            v[i] = *reinterpret_cast<const uint4 *>(a.x + base + c);
            if (a.residual != nullptr)
                rv[i] = *reinterpret_cast<const uint4 *>(a.residual + base + c);
            wv[i] = *reinterpret_cast<const uint4 *>(a.weight + c);
        } else {
            v[i] = rv[i] = wv[i] = make_uint4(0, 0, 0, 0);
        }
    }
    // a sum per vector and half of its words: chains of 4 terms, not one of 8 NV
    float part[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        uint32_t *p = reinterpret_cast<uint32_t *>(&v[i]);
        const uint32_t *q = reinterpret_cast<const uint32_t *>(&rv[i]);
        if (a.residual != nullptr) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                p[j] = dev::pack_bf16(dev::bf16_lo(p[j]) + dev::bf16_lo(q[j]),
                                      dev::bf16_hi(p[j]) + dev::bf16_hi(q[j]));
            const int c = (i * THREADS + tid) * 8;
            if (live && c < a.H)
                *reinterpret_cast<uint4 *>(a.residual_out + base + c) = v[i];
        }
        float even = 0.0f, odd = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = dev::bf16_lo(p[j]), hi = dev::bf16_hi(p[j]);
            even = __builtin_fmaf(lo, lo, even);
            odd = __builtin_fmaf(hi, hi, odd);
        }
        part[i] = even + odd;
    }
    static_assert(NV == 4, "pairs of pairs");
    float sum = wave_sum((part[0] + part[1]) + (part[2] + part[3]));
    if constexpr (kWaves > 1) {
        if (lane == 0)
            red[sub][tid / kWave] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            sum += red[sub][w];
    }
    const float inv = 1.0f / sqrtf(sum / (float)a.H + a.eps);

    const int NB = a.H / kQuantGroup;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vec = i * THREADS + tid;
        const int c = vec * 8;
        const bool on = live && vec < nvec;
        const uint32_t *p = reinterpret_cast<const uint32_t *>(&v[i]);
        const uint32_t *w = reinterpret_cast<const uint32_t *>(&wv[i]);
        float y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[2 * j] = dev::bf16_lo(p[j]) * inv * dev::bf16_lo(w[j]);
            y[2 * j + 1] = dev::bf16_hi(p[j]) * inv * dev::bf16_hi(w[j]);
        }
        if (on && a.out != nullptr)
            *reinterpret_cast<uint4 *>(a.out + base + c) =
                make_uint4(dev::pack_bf16(y[0], y[1]), dev::pack_bf16(y[2], y[3]), dev::pack_bf16(y[4], y[5]),
                           dev::pack_bf16(y[6], y[7]));
        if constexpr (QUANT != MOE_QUANT_NONE) {
            float amax = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                amax = fmaxf(amax, fabsf(y[j]));
            if constexpr (QUANT == MOE_QUANT_MXFP8) {
                amax = fmaxf(amax, dev::dpp<0xB1>(amax));
                amax = fmaxf(amax, dev::dpp<0x4E>(amax));
            } else {
                amax = max16(amax);
            }
            const dev::BlockScale<QUANT> bs(amax);
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                d[j] = bs.apply(y[j]);
            if (on) {
                *reinterpret_cast<uint2 *>(a.out_q + base + c) =
                    make_uint2(dev::pack_e4m3(d[0], d[1], d[2], d[3]), dev::pack_e4m3(d[4], d[5], d[6], d[7]));
                if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                    if ((vec & 15) == 0)
                        static_cast<float *>(a.out_scale)[t * NB + (vec >> 4)] = bs.s;
                } else if constexpr (QUANT == MOE_QUANT_MXFP8) {
                    if ((vec & 3) == 0)
                        static_cast<uint8_t *>(a.out_scale)[t * (a.H / 32) + (vec >> 2)] = (uint8_t)bs.byte;
                } else {
                    const int blk = vec >> 4;
                    uint8_t *row = static_cast<uint8_t *>(a.out_scale) + t * ((NB + 3) / 4 * 4);
                    if ((vec & 15) == 0)
                        row[blk] = (uint8_t)bs.byte;
                    // the last word's unused high bytes are 0
                    if (blk == NB - 1 && (vec & 15) > 0 && blk + (vec & 15) < (NB + 3) / 4 * 4)
                        row[blk + (vec & 15)] = 0;
                }
            }
        }
    }
}

template <int QUANT, int THREADS, int ROWS, int NV>
hipError_t launch(const NormArgs &a, hipStream_t stream)
{
    // A grid's threads are counted in 32 bits (past that it wraps, without an error).
    constexpr int64_t kRows = ((int64_t)1 << 31) / THREADS;
    for (int64_t first = 0; first < a.T; first += kRows) {
        const int64_t rows = a.T - first < kRows ? a.T - first : kRows;
        hipLaunchKernelGGL((rmsnorm_kernel<QUANT, THREADS, ROWS, NV>), dim3((uint32_t)((rows + ROWS - 1) / ROWS)),
                           dim3(THREADS * ROWS), 0, stream, a, first);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

template <int QUANT>
hipError_t launch_quant(const NormArgs &a, hipStream_t stream)
{
    // A wave per row without a barrier, four rows per block, or four waves per row:
    // 8192 rows of 1024 channels 14.6 / 26.0 us, of 2048 32.6 / 32.5.  More threads
    // than the row needs leave lanes idle: 16 waves for 7168 channels 262 us at 16,384
    // rows, four 187 (5.7 TB/s; one row: 3.7 us, launch and two dependent round trips).
    // Past 8192 channels a row needs the registers of more than four waves: 4096 rows of
    // 32,768 channels 230 us (5.3 TB/s), of 16,384 126 (4.8), of 12,288 101 (4.5), of
    // 8320, which fill half the lanes, 80 (3.8).
    if (a.H <= 2048)
        return launch<QUANT, 64, 4, 4>(a, stream);
    if (a.H <= 8192)
        return launch<QUANT, 256, 1, 4>(a, stream);
    return launch<QUANT, 1024, 1, 4>(a, stream);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs &a, int32_t quant, hipStream_t stream)
{
    if (a.out_q == nullptr)
        return launch_quant<MOE_QUANT_NONE>(a, stream);
    switch (quant) {
    case MOE_QUANT_FP8_F32:
        return launch_quant<MOE_QUANT_FP8_F32>(a, stream);
    case MOE_QUANT_FP8_UE8M0:
        return launch_quant<MOE_QUANT_FP8_UE8M0>(a, stream);
    default:
        return launch_quant<MOE_QUANT_MXFP8>(a, stream);
    }
}

}  // namespace moe
