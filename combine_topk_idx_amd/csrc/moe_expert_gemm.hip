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

// Writes a tile's results: bf16 outputs, or SwiGLU + quantization of the gate
// (f < 2) and up fragments.  Block-wide with SWIGLU.
template <int QUANT, int MT, bool SWIGLU, int BM>
__device__ __forceinline__ void write_tile(const ExpertGemmArgs &p, dev::f32x4 (&acc)[kNF][MT],
                                           const int32_t (&n0)[kNF], int64_t row0, int32_t valid, int32_t nt, int wave,
                                           int lane, float (*wave_max)[BM])
{
    const int r = lane & 15, g = lane >> 4;
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
                        }
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

        write_tile<QUANT, MT, SWIGLU>(p, acc, n0, row0, valid, nt, wave, lane, wave_max);
    }
}

// ---------------------------------------------------------------------------
// Large row groups: MT * 16 rows x 256 channels per block.
//
// Each of the four waves owns 64 channels and all the tile's rows, so a weight
// byte goes from memory to the registers of the one wave that multiplies it,
// one block of 128 channels ahead of its use, and only the rows -- which all
// four waves read -- pass through LDS (double buffered, one barrier per block).
// ---------------------------------------------------------------------------

constexpr int kMGroup = 8;   // row tiles that walk the channel tiles together

// (a condition inside the block loop would split it, and the compiler then moves
// the matrix instructions past the barrier)
template <int QUANT, int BM>
struct TileLds {
    alignas(16) uint8_t rows[2][BM * kQuantGroup];
    uint32_t sa[2][kGemmThreads];   // scale word of each row (a slot per thread: stores need no condition)
    uint32_t sw[2][kGemmThreads];   // and of the weights' channels (MXFP8) or blocks (the first two)
};

// A tile of work: rows [row0, row0 + valid) of expert e, channel tile nt.
struct TileAt {
    int32_t e, nt, valid;
    int64_t row0;
};

// Buffer descriptor over `bytes` bytes (loads past them return 0), the same in
// every lane.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, uint32_t bytes)
{
    const uint64_t a = (uint64_t)p;
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)(hi << 32 | lo), 0, __builtin_amdgcn_readfirstlane(bytes),
                                             0x00020000);
}
__device__ __forceinline__ dev::u32x4 load16(__amdgpu_buffer_rsrc_t b, uint32_t voff, uint32_t soff)
{
    return __builtin_bit_cast(dev::u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, voff, soff, 0));
}
__device__ __forceinline__ dev::i32x8 join(const dev::u32x4 &l, const dev::u32x4 &h)
{
    return dev::i32x8{(int)l[0], (int)l[1], (int)l[2], (int)l[3], (int)h[0], (int)h[1], (int)h[2], (int)h[3]};
}

template <int QUANT, int BM, bool SWIGLU, int MT>
__device__ __forceinline__ void run_tile(const ExpertGemmArgs &p, const TileAt &at, TileLds<QUANT, BM> &lds,
                                         float (*wave_max)[BM])
{
    constexpr int kRows = MT * 16;
    constexpr int kStage = kRows * 8 / kGemmThreads;  // 16-byte pieces per thread and block
    constexpr int GR = 1;                             // row fragments read together
    static_assert(MT >= 2 && MT % GR == 0 && kRows <= kGemmThreads, "staging covers whole row groups");
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const uint32_t k = (uint32_t)p.k;
    const int KB = p.k / kQuantGroup;
    const int SW = QUANT == MOE_QUANT_FP8_UE8M0 ? (KB + 3) / 4 : KB;  // scale words of a row
    const int NBn = (p.n + kQuantGroup - 1) / kQuantGroup;

    // rows: piece tid % 8 of row tid / 8 + 32 j; rows past the segment read as 0
    const __amdgpu_buffer_rsrc_t abuf = buffer(p.a + at.row0 * p.k, (uint32_t)at.valid * k);
    const uint32_t avo = (uint32_t)(tid >> 3) * k + (tid & 7) * 16;
    // their scale words: row tid
    const __amdgpu_buffer_rsrc_t sabuf =
        buffer(static_cast<const uint32_t *>(p.a_scale) + at.row0 * SW, (uint32_t)at.valid * SW * 4);
    const uint32_t savo = (uint32_t)tid * SW * 4;
    // weights: 64 channels of this wave (SwiGLU: 32 of the gate, 32 of the up half)
    int32_t n0[kNF];
    __amdgpu_buffer_rsrc_t wbuf[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int32_t c = SWIGLU ? at.nt * 128 + wave * 32 + h * (p.n / 2) : at.nt * kTileN + wave * 64 + h * 32;
        n0[2 * h] = c;
        n0[2 * h + 1] = c + 16;
        const int32_t left = max(0, min(32, p.n - c));
        wbuf[h] = buffer(p.w + ((int64_t)at.e * p.n + min(c, p.n - 1)) * p.k, (uint32_t)left * k);
    }
    const uint32_t wvo = (uint32_t)r * k + 16 * g;
    // their scale words: MXFP8 one per channel (channel tid of the tile), else
    // one per 128-channel block (threads 0 and 1)
    uint32_t sw_row;
    if constexpr (QUANT == MOE_QUANT_MXFP8)
        sw_row = SWIGLU ? at.nt * 128 + (tid & 127) + (tid >> 7) * (p.n / 2) : min(at.nt * kTileN + tid, p.n - 1);
    else
        sw_row = SWIGLU ? at.nt + (tid & 1) * (NBn / 2) : min(at.nt * 2 + (tid & 1), NBn - 1);
    const uint32_t sw_rows = QUANT == MOE_QUANT_MXFP8 ? p.n : NBn;
    const __amdgpu_buffer_rsrc_t swbuf =
        buffer(static_cast<const uint32_t *>(p.w_scale) + (int64_t)at.e * sw_rows * SW, sw_rows * SW * 4);
    const uint32_t swvo = sw_row * SW * 4;
    // 16-byte piece c of a row sits at position c ^ ((row >> 1) & 7) in LDS: the
    // 16 rows of a fragment then cover all banks
    const int spos = (tid >> 3) * kQuantGroup + (((tid & 7) ^ ((tid >> 4) & 7)) * 16);
    const int rswz = (r >> 1) & 7;
    const int rlo = r * kQuantGroup + ((g ^ rswz) * 16), rhi = r * kQuantGroup + (((4 + g) ^ rswz) * 16);

    dev::f32x4 acc[kNF][MT];
#pragma unroll
    for (int f = 0; f < kNF; ++f)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[f][i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    dev::u32x4 xr[kStage];
    uint32_t sav, swv;
    dev::u32x4 wf[2][2 * kNF];
    // All loads of block kb.  The block after the last one is asked for as an
    // address past every buffer's end, which costs no memory access.
    const auto load = [&](dev::u32x4(&w)[2 * kNF], int kb) {
        const uint32_t past = kb < KB ? 0u : 0x80000000u;
        const uint32_t at_k = (uint32_t)kb * kQuantGroup | past;
        const int word = QUANT == MOE_QUANT_FP8_UE8M0 ? min(kb, KB - 1) >> 2 : min(kb, KB - 1);
#pragma unroll
        for (int j = 0; j < kStage; ++j)
            xr[j] = load16(abuf, avo, (uint32_t)(32 * j) * k + at_k);
        sav = __builtin_amdgcn_raw_buffer_load_b32(sabuf, savo, word * 4, 0);
        swv = __builtin_amdgcn_raw_buffer_load_b32(swbuf, swvo, word * 4, 0);
#pragma unroll
        for (int f = 0; f < kNF; ++f) {
            const uint32_t so = (uint32_t)(16 * (f & 1)) * k + at_k;
            w[2 * f] = load16(wbuf[f >> 1], wvo, so);
            w[2 * f + 1] = load16(wbuf[f >> 1], wvo + 64, so);
        }
    };
    // Rows and scales of the loaded block, into LDS buffer `buf`.
    const auto store = [&](int buf) {
#pragma unroll
        for (int j = 0; j < kStage; ++j)
            *reinterpret_cast<dev::u32x4 *>(&lds.rows[buf][spos + 32 * j * kQuantGroup]) = xr[j];
        lds.sa[buf][tid] = sav;
        lds.sw[buf][tid] = swv;
    };
    // One block of 128 channels: GR row fragments at a time, the next ones read
    // from LDS while these are multiplied.
    const auto multiply = [&](const dev::u32x4(&w)[2 * kNF], int buf, int u) {
        float swf[2] = {};
        int swb[kNF] = {};
        if constexpr (QUANT == MOE_QUANT_FP8_F32) {
            swf[0] = __uint_as_float(lds.sw[buf][SWIGLU ? 0 : wave >> 1]);
            swf[1] = SWIGLU ? __uint_as_float(lds.sw[buf][1]) : swf[0];
        } else if constexpr (QUANT == MOE_QUANT_FP8_UE8M0) {
            swb[0] = swb[1] = (int)(lds.sw[buf][SWIGLU ? 0 : wave >> 1] >> (8 * u));
            swb[2] = swb[3] = SWIGLU ? (int)(lds.sw[buf][1] >> (8 * u)) : swb[0];
        } else {
#pragma unroll
            for (int f = 0; f < kNF; ++f) {
                const int n = SWIGLU ? wave * 32 + (f & 1) * 16 + (f >> 1) * 128 + r : wave * 64 + f * 16 + r;
                swb[f] = (int)(lds.sw[buf][n] >> (8 * g));
            }
        }
        const uint8_t *rows = lds.rows[buf];
        dev::u32x4 lo[2][GR], hi[2][GR];
        uint32_t sv[2][GR];
        const auto read = [&](int b, int i0) {
#pragma unroll
            for (int i = 0; i < GR; ++i) {
                lo[b][i] = *reinterpret_cast<const dev::u32x4 *>(rows + rlo + (i0 + i) * 16 * kQuantGroup);
                hi[b][i] = *reinterpret_cast<const dev::u32x4 *>(rows + rhi + (i0 + i) * 16 * kQuantGroup);
                sv[b][i] = lds.sa[buf][(i0 + i) * 16 + r];
            }
        };
        read(0, 0);
#pragma unroll
        for (int c = 0; c < MT / GR; ++c) {
            if (c + 1 < MT / GR)
                read((c + 1) & 1, (c + 1) * GR);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < GR; ++i) {
                const dev::i32x8 x = join(lo[c & 1][i], hi[c & 1][i]);
                const uint32_t s = sv[c & 1][i];
                if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                    const float s0 = __uint_as_float(s) * swf[0];
                    const float s1 = SWIGLU ? __uint_as_float(s) * swf[1] : s0;
#pragma unroll
                    for (int f = 0; f < kNF; ++f) {
                        const dev::f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
                        const dev::f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            join(w[2 * f], w[2 * f + 1]), x, z, 0, 0, 0, 0, 0, 0);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[f][c * GR + i][j] = __builtin_fmaf(d[j], f < 2 ? s0 : s1, acc[f][c * GR + i][j]);
                    }
                } else {
                    const int sb = (int)(s >> (8 * (QUANT == MOE_QUANT_FP8_UE8M0 ? u : g)));
#pragma unroll
                    for (int f = 0; f < kNF; ++f)
                        acc[f][c * GR + i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            join(w[2 * f], w[2 * f + 1]), x, acc[f][c * GR + i], 0, 0, 0, swb[f], 0, sb);
                }
            }
        }
    };

    load(wf[0], 0);
    store(0);
    __syncthreads();
    for (int kb = 0; kb < KB; kb += 2) {
        load(wf[1], kb + 1);
        __builtin_amdgcn_sched_barrier(0);
        multiply(wf[0], 0, kb & 3);
        store(1);
        __syncthreads();
        load(wf[0], kb + 2);
        __builtin_amdgcn_sched_barrier(0);
        // an odd block count ends with a block of zeros
        multiply(wf[1], 1, (kb + 1) & 3);
        store(0);
        __syncthreads();
    }
    write_tile<QUANT, MT, SWIGLU>(p, acc, n0, at.row0, at.valid, at.nt, wave, lane, wave_max);
}

template <int QUANT, bool SWIGLU, int MT, int OCC>
__global__ __launch_bounds__(kGemmThreads, OCC) void expert_gemm_tiles(ExpertGemmArgs p, int32_t n_tiles)
{
    constexpr int BM = MT * 16;
    __shared__ int32_t tile_start[kMaxExperts + 1];
    __shared__ int32_t red[kGemmWaves];
    __shared__ float wave_max[kGemmWaves][BM];
    __shared__ TileLds<QUANT, BM> lds;
    scan_tiles<BM>(p.recv_count, p.E, p.dense_rows, tile_start, red);
    const int64_t n_work = (int64_t)__builtin_amdgcn_readfirstlane(tile_start[p.E]) * n_tiles;
    // workgroups go to the 8 XCDs in turn: each XCD takes a contiguous run of
    // the work, so that the tiles of one expert share its L2
    const int64_t run = (n_work + 7) / 8;

    for (int64_t idx = blockIdx.x >> 3; idx < run; idx += gridDim.x >> 3) {
        const int64_t work = (int64_t)(blockIdx.x & 7) * run + idx;
        if (work >= n_work)
            break;
        // tiles of an expert: groups of kMGroup row tiles; inside a group the
        // row tiles of one channel tile are adjacent (they share its weights)
        TileAt at;
        at.e = __builtin_amdgcn_readfirstlane(find_expert(tile_start, p.E, (int32_t)(work / n_tiles)));
        const int32_t e_first = __builtin_amdgcn_readfirstlane(tile_start[at.e]);
        const int32_t e_tiles = __builtin_amdgcn_readfirstlane(tile_start[at.e + 1]) - e_first;
        const int64_t local = work - (int64_t)e_first * n_tiles;
        const int32_t grp = (int32_t)(local / ((int64_t)kMGroup * n_tiles));
        const int32_t in_grp = (int32_t)(local - (int64_t)grp * kMGroup * n_tiles);
        const int32_t grp_rows = min(kMGroup, e_tiles - grp * kMGroup);
        at.nt = __builtin_amdgcn_readfirstlane(in_grp / grp_rows);
        const int32_t first = __builtin_amdgcn_readfirstlane((grp * kMGroup + in_grp % grp_rows) * BM);
        const int32_t count =
            __builtin_amdgcn_readfirstlane(p.recv_count != nullptr ? p.recv_count[at.e] : p.dense_rows);
        const int32_t seg = __builtin_amdgcn_readfirstlane(p.recv_count != nullptr ? p.expert_offset[at.e] : 0);
        at.valid = min(BM, count - first);
        at.row0 = (int64_t)seg + first;
        // a segment's last tile takes the code for its size
        if (MT <= 2 || at.valid > BM / 2)
            run_tile<QUANT, BM, SWIGLU, MT>(p, at, lds, wave_max);
        else if (MT <= 4 || at.valid > BM / 4)
            run_tile<QUANT, BM, SWIGLU, (MT > 2 ? MT / 2 : MT)>(p, at, lds, wave_max);
        else
            run_tile<QUANT, BM, SWIGLU, (MT > 4 ? MT / 4 : MT)>(p, at, lds, wave_max);
        __syncthreads();  // LDS is reused by the next tile
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

template <int QUANT, bool SWIGLU, int MT, int OCC>
hipError_t launch_tiles(const ExpertGemmArgs &p, hipStream_t stream)
{
    constexpr int BM = MT * 16;
    const int32_t n_tiles = SWIGLU ? p.n / 256 : (p.n + kTileN - 1) / kTileN;
    const int64_t parts = p.max_rows < p.E ? p.max_rows : p.E;
    int64_t grid = ((p.max_rows / BM + parts) * n_tiles + 7) / 8 * 8;
    const int64_t cap = (int64_t)1 << 30;
    grid = grid < 8 ? 8 : grid > cap ? cap : grid;
    hipLaunchKernelGGL((expert_gemm_tiles<QUANT, SWIGLU, MT, OCC>), dim3((uint32_t)grid), dim3(kGemmThreads), 0,
                       stream, p, n_tiles);
    return hipGetLastError();
}

template <int QUANT, bool SWIGLU>
hipError_t launch_rows(const ExpertGemmArgs &p, hipStream_t stream)
{
    const int64_t per_expert = p.max_rows / p.E;
    if (per_expert <= 16)
        return launch<QUANT, 1, SWIGLU>(p, stream);
    if (per_expert <= 128)
        return launch_tiles<QUANT, SWIGLU, 4, 2>(p, stream);
    return launch_tiles<QUANT, SWIGLU, 8, 2>(p, stream);
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
