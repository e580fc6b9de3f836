// The experts' products on dispatched FP8 rows on gfx950, plain and with a
// fused SwiGLU + requantization.
//
//   y[row, j] = sum over blocks b of sa[row, b] sw[j, b] * sum_{c in b} a[row, c] w[j, c]
//
// One v_mfma_f32_16x16x128_f8f6f4 covers 16 output channels x 16 rows x one
// 128-channel block.  The weights are its first operand, so a lane's four
// results belong to one row and four adjacent output channels: the fp32 scale
// of a block is one product per lane and the outputs leave in 8-byte pieces.
// fp32 scales are applied to each block's result as it is added to the running
// sum; power-of-two scales go into the matrix instruction (one byte per 32
// channels of a lane's row) and the sum stays in its accumulator.
#include "moe_mma.h"

namespace moe {

namespace {

constexpr int kGemmThreads = 256;
constexpr int kGemmWaves = kGemmThreads / kWave;
constexpr int kNF = 4;                        // 16-channel fragments per wave
constexpr int kTileN = kGemmWaves * kNF * 16;  // output channels per block

// tile_start[e] = row tiles of BM rows before expert e; [E] = all.  Block-wide,
// ends with a barrier.
template <int BM>
__device__ inline void scan_tiles(const int32_t *recv_count, int32_t E, int32_t dense_rows, int32_t *tile_start,
                                  int32_t *red)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int per = (E + kGemmThreads - 1) / kGemmThreads;
    const int e0 = min(E, tid * per), e1 = min(E, e0 + per);
    int32_t local = 0;
    for (int e = e0; e < e1; ++e)
        local += ((recv_count != nullptr ? recv_count[e] : dense_rows) + BM - 1) / BM;
    const int32_t incl = dev::wave_inclusive_sum(local);
    if (lane == kWave - 1)
        red[wave] = incl;
    __syncthreads();
    int32_t run = dev::sum_before<kGemmWaves>(red, wave) + incl - local;
    for (int e = e0; e < e1; ++e) {
        tile_start[e] = run;
        run += ((recv_count != nullptr ? recv_count[e] : dense_rows) + BM - 1) / BM;
    }
    if (tid == kGemmThreads - 1)
        tile_start[E] = run;
    __syncthreads();
}

// Expert of row tile m: the last e with tile_start[e] <= m.
__device__ __forceinline__ int find_expert(const int32_t *tile_start, int32_t E, int32_t m)
{
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tile_start[mid] <= m)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <int QUANT, int MT, bool SWIGLU>
__global__ __launch_bounds__(kGemmThreads) void expert_gemm_kernel(ExpertGemmArgs p, int32_t n_tiles)
{
    constexpr int BM = MT * 16;
    __shared__ int32_t tile_start[kMaxExperts + 1];
    __shared__ int32_t red[kGemmWaves];
    __shared__ float wave_max[kGemmWaves][BM];
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int KB = p.k / kQuantGroup;
    const int KW = (KB + 3) / 4;
    scan_tiles<BM>(p.recv_count, p.E, p.dense_rows, tile_start, red);
    const int64_t n_work = (int64_t)tile_start[p.E] * n_tiles;

    for (int64_t work = blockIdx.x; work < n_work; work += gridDim.x) {
        const int32_t m = (int32_t)(work / n_tiles);
        const int32_t nt = (int32_t)(work - (int64_t)m * n_tiles);
        const int e = __builtin_amdgcn_readfirstlane(find_expert(tile_start, p.E, m));
        const int32_t first = (m - tile_start[e]) * BM;
        const int64_t seg = p.recv_count != nullptr ? p.expert_offset[e] : 0;
        const int32_t count = p.recv_count != nullptr ? p.recv_count[e] : p.dense_rows;
        const int32_t valid = min(BM, count - first);
        const int64_t row0 = seg + first;

        // this lane's row of each row group, and this wave's channel fragments
        int64_t arow[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
            arow[i] = row0 + min(i * 16 + r, valid - 1);
        int32_t n0[kNF];
        int64_t wrow[kNF];
#pragma unroll
        for (int f = 0; f < kNF; ++f) {
            if constexpr (SWIGLU)
                n0[f] = nt * 128 + wave * 32 + (f & 1) * 16 + (f >= 2 ? p.n / 2 : 0);
            else
                n0[f] = nt * kTileN + wave * 64 + f * 16;
            wrow[f] = (int64_t)e * p.n + min(n0[f] + r, p.n - 1);
        }
        dev::f32x4 acc[kNF][MT];
#pragma unroll
        for (int f = 0; f < kNF; ++f)
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[f][i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        const int NBn = (p.n + kQuantGroup - 1) / kQuantGroup;
        for (int kb = 0; kb < KB; ++kb) {
            dev::i32x8 wf[kNF];
            float swf[kNF];
            int swb[kNF];
#pragma unroll
            for (int f = 0; f < kNF; ++f) {
                wf[f] = dev::load_frag(p.w + wrow[f] * p.k + (int64_t)kb * kQuantGroup, g);
                const int64_t nb = (int64_t)e * NBn + min(n0[f], p.n - 1) / kQuantGroup;
                if constexpr (QUANT == MOE_QUANT_FP8_F32)
                    swf[f] = static_cast<const float *>(p.w_scale)[nb * KB + kb];
                else if constexpr (QUANT == MOE_QUANT_FP8_UE8M0)
                    swb[f] = static_cast<const uint8_t *>(p.w_scale)[nb * KW * 4 + kb];
                else
                    swb[f] = static_cast<const uint8_t *>(p.w_scale)[wrow[f] * KB * 4 + kb * 4 + g];
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const dev::i32x8 af = dev::load_frag(p.a + arow[i] * p.k + (int64_t)kb * kQuantGroup, g);
                float saf = 0.0f;
                int sab = 0;
                if constexpr (QUANT == MOE_QUANT_FP8_F32)
                    saf = static_cast<const float *>(p.a_scale)[arow[i] * KB + kb];
                else if constexpr (QUANT == MOE_QUANT_FP8_UE8M0)
                    sab = static_cast<const uint8_t *>(p.a_scale)[arow[i] * KW * 4 + kb];
                else
                    sab = static_cast<const uint8_t *>(p.a_scale)[arow[i] * KB * 4 + kb * 4 + g];
#pragma unroll
                for (int f = 0; f < kNF; ++f) {
                    if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                        const dev::f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
                        const dev::f32x4 d =
                            __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[f], af, z, 0, 0, 0, 0, 0, 0);
                        const float s = saf * swf[f];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[f][i][j] = __builtin_fmaf(d[j], s, acc[f][i][j]);
                    } else {
                        acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[f], af, acc[f][i], 0, 0, 0,
                                                                                      swb[f], 0, sab);
                    }
                }
            }
        }

        if constexpr (!SWIGLU) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int32_t row = i * 16 + r;
#pragma unroll
                for (int f = 0; f < kNF; ++f) {
                    const int32_t n = n0[f] + g * 4;
                    if (row < valid && n < p.n)
                        *reinterpret_cast<uint2 *>(p.y + (row0 + row) * p.n + n) =
                            make_uint2(dev::pack_bf16(acc[f][i][0], acc[f][i][1]),
                                       dev::pack_bf16(acc[f][i][2], acc[f][i][3]));
                }
            }
        } else {
            const int32_t inter = p.n / 2;
            // h in the place of the gate accumulators; largest magnitude per row and wave
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float amax = 0.0f;
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[f][i][j] = dev::swiglu(acc[f][i][j], acc[f + 2][i][j]);
                        amax = fmaxf(amax, fabsf(acc[f][i][j]));
                    }
                amax = fmaxf(amax, __shfl_xor(amax, 16));
                amax = fmaxf(amax, __shfl_xor(amax, 32));
                if (g == 0)
                    wave_max[wave][i * 16 + r] = amax;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int32_t row = i * 16 + r;
                float amax = wave_max[wave][row];
                if constexpr (QUANT != MOE_QUANT_MXFP8) {
#pragma unroll
                    for (int w = 0; w < kGemmWaves; ++w)
                        amax = fmaxf(amax, wave_max[w][row]);
                }
                const dev::BlockScale<QUANT> bs(amax);
                if (row < valid) {
                    const int64_t grow = row0 + row;
#pragma unroll
                    for (int f = 0; f < 2; ++f)
                        *reinterpret_cast<uint32_t *>(p.h + grow * inter + n0[f] + g * 4) =
                            dev::pack_e4m3(bs.apply(acc[f][i][0]), bs.apply(acc[f][i][1]), bs.apply(acc[f][i][2]),
                                           bs.apply(acc[f][i][3]));
                    const int HB = inter / kQuantGroup;
                    if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                        if (wave == 0 && g == 0)
                            static_cast<float *>(p.h_scale)[grow * HB + nt] = bs.s;
                    } else if constexpr (QUANT == MOE_QUANT_FP8_UE8M0) {
                        const int HW = (HB + 3) / 4 * 4;
                        uint8_t *sc = static_cast<uint8_t *>(p.h_scale) + grow * HW;
                        if (wave == 0 && g == 0) {
                            sc[nt] = (uint8_t)bs.byte;
                            if (nt == HB - 1)  // the last word's unused high bytes are 0
                                for (int b = HB; b < HW; ++b)
                                    sc[b] = 0;
                        }
                    } else {
                        if (g == 0)
                            static_cast<uint8_t *>(p.h_scale)[grow * HB * 4 + nt * 4 + wave] = (uint8_t)bs.byte;
                    }
                }
            }
            __syncthreads();  // wave_max is rewritten by the next tile
        }
    }
}

template <int QUANT, int MT, bool SWIGLU>
hipError_t launch(const ExpertGemmArgs &p, hipStream_t stream)
{
    constexpr int BM = MT * 16;
    const int32_t n_tiles = SWIGLU ? p.n / 256 : (p.n + kTileN - 1) / kTileN;
    // a segment's last tile is partial: at most one more tile per expert that has rows
    const int64_t parts = p.max_rows < p.E ? p.max_rows : p.E;
    int64_t grid = (p.max_rows / BM + parts) * n_tiles;
    const int64_t cap = (int64_t)1 << 30;
    grid = grid < 1 ? 1 : grid > cap ? cap : grid;
    hipLaunchKernelGGL((expert_gemm_kernel<QUANT, MT, SWIGLU>), dim3((uint32_t)grid), dim3(kGemmThreads), 0, stream,
                       p, n_tiles);
    return hipGetLastError();
}

template <int QUANT, bool SWIGLU>
hipError_t launch_rows(const ExpertGemmArgs &p, hipStream_t stream)
{
    const int64_t per_expert = p.max_rows / p.E;
    if (per_expert <= 16)
        return launch<QUANT, 1, SWIGLU>(p, stream);
    return launch<QUANT, 4, SWIGLU>(p, stream);
}

template <bool SWIGLU>
hipError_t launch_quant(const ExpertGemmArgs &p, int32_t quant, hipStream_t stream)
{
    switch (quant) {
    case MOE_QUANT_FP8_F32:
        return launch_rows<MOE_QUANT_FP8_F32, SWIGLU>(p, stream);
    case MOE_QUANT_FP8_UE8M0:
        return launch_rows<MOE_QUANT_FP8_UE8M0, SWIGLU>(p, stream);
    default:
        return launch_rows<MOE_QUANT_MXFP8, SWIGLU>(p, stream);
    }
}

}  // namespace

hipError_t launch_expert_gemm(const ExpertGemmArgs &a, int32_t quant, bool swiglu, hipStream_t stream)
{
    return swiglu ? launch_quant<true>(a, quant, stream) : launch_quant<false>(a, quant, stream);
}

}  // namespace moe
