// The experts' products on dispatched FP8 rows on gfx950, plain and with a
// fused SwiGLU + requantization.
//
//   y[row, j] = sum over blocks b of sa[row, b] sw[j, b] * sum_{c in b} a[row, c] w[j, c]
//
// One v_mfma_f32_16x16x128_f8f6f4 covers 16 output channels x 16 rows x one
// 128-channel block.  The weights are its first operand, so a lane's four
// results belong to one row and four adjacent output channels: the fp32 scale
// of a block is one product per lane, and lanes that trade results make whole
// cache lines of a row.  fp32 scales are applied to each block's result as it is
// added to the running sum; power-of-two scales go into the matrix instruction
// (one byte per 32 channels of a lane's row) and the sum stays in its accumulator.
//
// Bounds and measurements (one MI355X; times of calls in a row):
//   a few rows in all: latency (expert_gemm_strips).  One row, 7168 -> 7168: 15 us;
//   few rows per expert: the weights' bytes.  128 experts x 8 rows, 768 -> 2048:
//   45 us; 256 experts x 8 rows, 7168 -> 2 x 2048, SwiGLU: 1.27 ms, 5.9 TB/s;
//   many rows: the matrix cores and LDS.  8192 dense rows, 7168 -> 8192, UE8M0:
//   383 us, 2510 TFLOP/s (a library's product of 8192^3 with one scale: 2718);
//   in between: the start and end of a tile (a block's results leave while nothing
//   multiplies), 65,536 rows of 256 experts, 2048 -> 7168: 1.35 ms, 1430 TFLOP/s.
// Weights loaded to registers instead of LDS took twice as long (each of the two
// wave rows reads them), blocks of 320 rows and K walks that start apart the same.
#include <type_traits>

#include "moe_mma.h"

namespace moe {

namespace {

constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / kWave;
constexpr int kWaveRows = 2, kWaveCols = 4;   // waves over the tile's rows and channels
constexpr int kNF = 4;                        // 16-channel fragments per wave
constexpr int kTileN = kWaveCols * kNF * 16;  // output channels per block
// Row tiles that walk the channel tiles together: 4 / 8 / 16 / 32 of them, 65,536
// rows, 64 experts, 2048 -> 7168: 1108 / 1053 / 1054 / 1058 us; 8192 dense rows, 7168 ->
// 8192: 377 / 376 / 384 / 417.
constexpr int kMGroup = 8;
constexpr int kGroup = 4;                     // experts per entry of a block's table of tiles

// A value that is the same in every lane, in a scalar register.  Where the
// compiler can tell that it is, it drops a plain readfirstlane, may keep the
// value in a vector register all the same (a quotient, threadIdx.x / 64) and
// then turns each load through a descriptor that depends on it into a loop:
// the empty asm hides what it can tell.
__device__ __forceinline__ int32_t scalar(int32_t v)
{
    asm("" : "+v"(v));
    return __builtin_amdgcn_readfirstlane(v);
}

// Word i (uniform) of an array that the kernel does not write, by a scalar load:
// a vector load would wait for every load before it, whole stages of a tile.
__device__ __forceinline__ int32_t word_of(const int32_t *a, int32_t i)
{
    return reinterpret_cast<const __attribute__((address_space(4))) int32_t *>((uint64_t)a)[i];
}

// tile_start[i] = row tiles of BM rows before expert kGroup i, [ceil(E / kGroup)]
// = all: a table of every expert would not fit beside the stages.  Block-wide,
// ends with a barrier.
template <int BM>
__device__ inline void scan_tiles(const ExpertGemmArgs &p, int32_t *tile_start, int32_t *red)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int groups = (p.E + kGroup - 1) / kGroup;
    const int per = (groups + kTileThreads - 1) / kTileThreads;
    const int e0 = min(groups, tid * per) * kGroup, e1 = min(groups, (tid + 1) * per) * kGroup;
    const auto tiles = [&](int e) {
        return ((e >= p.E ? 0 : p.recv_count != nullptr ? p.recv_count[e] : p.dense_rows) + BM - 1) / BM;
    };
    int32_t local = 0;
    for (int e = e0; e < e1; ++e)
        local += tiles(e);
    const int32_t incl = dev::wave_inclusive_sum(local);
    if (lane == kWave - 1)
        red[wave] = incl;
    __syncthreads();
    int32_t run = dev::sum_before<kTileWaves>(red, wave) + incl - local;
    for (int e = e0; e < e1; ++e) {
        if (e % kGroup == 0)
            tile_start[e / kGroup] = run;
        run += tiles(e);
    }
    if (tid == kTileThreads - 1)
        tile_start[groups] = run;
    __syncthreads();
}

// An expert, the number of its first row tile and of its rows.
struct ExpertAt {
    int32_t e, start, rows;
};

// The expert that row tile m (uniform, below the number of all) belongs to.
template <int BM>
__device__ __forceinline__ ExpertAt find_expert(const ExpertGemmArgs &p, const int32_t *tile_start, int32_t m)
{
    int lo = 0, hi = (p.E + kGroup - 1) / kGroup;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (scalar(tile_start[mid]) <= m)
            lo = mid;
        else
            hi = mid;
    }
    if (p.recv_count == nullptr)
        return ExpertAt{0, 0, p.dense_rows};
    int32_t rows[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
        rows[i] = word_of(p.recv_count, min(lo * kGroup + i, p.E - 1));
    ExpertAt at = {lo * kGroup, scalar(tile_start[lo]), rows[0]};
#pragma unroll
    for (int i = 1; i < kGroup; ++i) {
        const int32_t after = at.start + (at.rows + BM - 1) / BM;
        if (m >= after)
            at = ExpertAt{lo * kGroup + i, after, rows[i]};
    }
    return at;
}

// A tile of work: rows [row0, row0 + valid) of expert e, channel tile nt.
struct TileAt {
    int32_t e, nt, valid;
    int64_t row0;
    __device__ __forceinline__ TileAt scalars() const
    {
        const uint64_t lo = (uint32_t)scalar((int32_t)row0), hi = (uint32_t)scalar((int32_t)(row0 >> 32));
        return TileAt{scalar(e), scalar(nt), scalar(valid), (int64_t)(hi << 32 | lo)};
    }
};

// Two 16-byte pieces as one operand.
__device__ __forceinline__ dev::i32x8 join(const dev::u32x4 &l, const dev::u32x4 &h)
{
    return dev::i32x8{(int)l[0], (int)l[1], (int)l[2], (int)l[3], (int)h[0], (int)h[1], (int)h[2], (int)h[3]};
}

// Buffer descriptor over `bytes` bytes (loads past them return 0), the same in
// every lane.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void *p, uint32_t bytes)
{
    const uint64_t a = (uint64_t)p;
    const uint64_t lo = (uint32_t)scalar((int32_t)a);
    const uint64_t hi = (uint32_t)scalar((int32_t)(a >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void *)(hi << 32 | lo), 0, scalar((int32_t)bytes),
                                             0x00020000);
}

// Waits for this wave's LDS accesses, then for the block's other waves, and
// leaves memory accesses on their way.
__device__ __forceinline__ void meet()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Writes a wave's results: rows 16 MT wr + 16 i + (lane % 16), channels n0[f] + 4
// (lane / 16) + j.  bf16 outputs, or (SWIGLU; fragments f < 2 hold the gate,
// f >= 2 the up products) SwiGLU and quantization, block-wide: the WC waves of
// a row share its 128-channel block (each has one MX block of 32).
template <int QUANT, int MT, bool SWIGLU, int BM>
__device__ __forceinline__ void write_tile(const ExpertGemmArgs &p, dev::f32x4 (&acc)[kNF][MT], const TileAt &at,
                                           int wr, int wc, int lane, float (*wave_max)[BM])
{
    const int r = lane & 15, g = lane >> 4;
    if constexpr (!SWIGLU) {
        // Two fragments' results change places between odd and even rows of 16
        // lanes: a lane then has 8 adjacent channels of its row, and 4 lanes half of
        // the row's 64.  The other half comes from the lane 8 further, for the
        // half that one needs: a store then covers whole cache lines, 128 bytes of
        // each of 8 rows.  Rows and channels past the end go past the buffer's,
        // which drops them.  The stores are marked as streamed (non-temporal), which
        // leaves L2 to the weights (8192 dense rows, 7168 -> 8192, UE8M0: 424 -> 382 us).
        constexpr int kStreamed = 2;
        const __amdgpu_buffer_rsrc_t out = buffer(p.y + at.row0 * p.n, (uint32_t)at.valid * (uint32_t)p.n * 2);
        const bool low = r < 8;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            dev::u32x4 v[2];
#pragma unroll
            for (int f = 0; f < kNF; f += 2) {
                const auto lo = __builtin_amdgcn_permlane16_swap(dev::pack_bf16(acc[f][i][0], acc[f][i][1]),
                                                                 dev::pack_bf16(acc[f + 1][i][0], acc[f + 1][i][1]),
                                                                 false, false);
                const auto hi = __builtin_amdgcn_permlane16_swap(dev::pack_bf16(acc[f][i][2], acc[f][i][3]),
                                                                 dev::pack_bf16(acc[f + 1][i][2], acc[f + 1][i][3]),
                                                                 false, false);
                v[f / 2] = dev::u32x4{lo[0], hi[0], lo[1], hi[1]};
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t other = __builtin_amdgcn_update_dpp(0, low ? v[1][j] : v[0][j], 0x128, 0xF, 0xF, true);
                v[0][j] = low ? v[0][j] : other;
                v[1][j] = low ? other : v[1][j];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int32_t row = (wr * MT + i) * 16 + h * 8 + (r & 7);
                const int32_t n = at.nt * kTileN + wc * 64 + (low ? 0 : 32) + (g & 1) * 16 + (g >> 1) * 8;
                const uint32_t off = row < at.valid && n < p.n ? ((uint32_t)row * (uint32_t)p.n + n) * 2 : 0x80000000u;
                __builtin_amdgcn_raw_buffer_store_b128(v[h], out, off, 0, kStreamed);
            }
        }
    } else {
        const int32_t inter = p.n / 2;
        const __amdgpu_buffer_rsrc_t out = buffer(p.h + at.row0 * inter, (uint32_t)at.valid * (uint32_t)inter);
        constexpr int kScale = QUANT == MOE_QUANT_FP8_UE8M0 ? 1 : 4;  // bytes of 128 channels' scales
        const int HB = inter / kQuantGroup, HW = (HB * kScale + 3) / 4 * 4;
        const __amdgpu_buffer_rsrc_t scales =
            buffer(static_cast<uint8_t *>(p.h_scale) + at.row0 * HW, (uint32_t)at.valid * (uint32_t)HW);
        // h in the place of the gate accumulators; largest magnitude per row of
        // this wave's 32 channels, an MXFP8 block: the other formats' 128 are those
        // of the waves of a row
        float amax[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            amax[i] = 0.0f;
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[f][i][j] = dev::swiglu(acc[f][i][j], acc[f + 2][i][j]);
                    amax[i] = fmaxf(amax[i], fabsf(acc[f][i][j]));
                }
            amax[i] = fmaxf(amax[i], __shfl_xor(amax[i], 16));
            amax[i] = fmaxf(amax[i], __shfl_xor(amax[i], 32));
            if (QUANT != MOE_QUANT_MXFP8 && g == 0)
                wave_max[wc][(wr * MT + i) * 16 + r] = amax[i];
        }
        if constexpr (QUANT != MOE_QUANT_MXFP8)
            meet();
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int32_t row = (wr * MT + i) * 16 + r;
            if constexpr (QUANT != MOE_QUANT_MXFP8) {
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    amax[i] = fmaxf(amax[i], wave_max[w][row]);
            }
            const dev::BlockScale<QUANT> bs(amax[i]);
            uint32_t q[2];
#pragma unroll
            for (int f = 0; f < 2; ++f)
                q[f] = dev::pack_e4m3(bs.apply(acc[f][i][0]), bs.apply(acc[f][i][1]), bs.apply(acc[f][i][2]),
                                      bs.apply(acc[f][i][3]));
            // 8 adjacent channels per lane, as above
            const auto pair = __builtin_amdgcn_permlane16_swap(q[0], q[1], false, false);
            const uint32_t off = (uint32_t)row * (uint32_t)inter + at.nt * 128 + wc * 32 + (g & 1) * 16 + (g >> 1) * 8;
            __builtin_amdgcn_raw_buffer_store_b64(dev::u32x2{pair[0], pair[1]}, out,
                                                  row < at.valid ? off : 0x80000000u, 0, 0);
            const bool one = row < at.valid && g == 0 && (QUANT == MOE_QUANT_MXFP8 || wc == 0);
            const uint32_t soff = one ? (uint32_t)row * HW + at.nt * kScale + (QUANT == MOE_QUANT_MXFP8 ? wc : 0)
                                      : 0x80000000u;
            if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(bs.s), scales, soff, 0, 0);
            } else {
                __builtin_amdgcn_raw_buffer_store_b8((uint8_t)bs.byte, scales, soff, 0, 0);
                if constexpr (QUANT == MOE_QUANT_FP8_UE8M0)
                    if (at.nt == HB - 1)  // the last word's unused high bytes are 0
                        for (int b = 1; b <= HW - HB; ++b)
                            __builtin_amdgcn_raw_buffer_store_b8((uint8_t)0, scales, soff, b, 0);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// BM rows x 256 channels per block of 8 waves.
//
// Rows and weights of one 128-channel block form a stage, which loads straight
// from memory into LDS (no registers in between); NS stages are in turn, so
// NS - 1 blocks are in flight while one is multiplied.  A wave waits for its
// own loads of a stage, a barrier makes the others' visible, and the stage that
// was multiplied before the barrier takes the next block.  Blocks are
// persistent, one per compute unit: the first stages of a block's next tile
// load while it writes its last one's results.
// ---------------------------------------------------------------------------

// Four of an operand's eight registers.
__device__ __forceinline__ dev::u32x4 half(const dev::i32x8 &v, int at)
{
    return dev::u32x4{(uint32_t)v[at], (uint32_t)v[at + 1], (uint32_t)v[at + 2], (uint32_t)v[at + 3]};
}

// Memory -> LDS: BYTES per lane, lane l to dst + l * BYTES.
template <int BYTES>
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t b, uint8_t *dst, uint32_t voff, uint32_t soff)
{
    auto *to = (__attribute__((address_space(3))) void *)dst;
    if constexpr (BYTES == 16)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b, to, 16, voff, soff, 0, 0);
    else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(b, to, 4, voff, soff, 0, 0);
}

// Waits until at most VM of this wave's memory accesses are outstanding and all
// of its LDS reads are done, then for the block's other waves.  VM counts the
// loads that were issued after those waited for, and loads only: stores issued
// after loads into LDS may complete before them (a count that took the stores of
// the tile before to be behind this tile's loads gave stages that were not there).
template <int VM>
__device__ __forceinline__ void wait_and_meet()
{
    static_assert(VM < 64, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(VM) : "memory");
}

// f(0), f(1), .. f(N - 1) with the number as a type.
template <int N, typename F>
__device__ __forceinline__ void for_each(const F &f)
{
    if constexpr (N > 0) {
        for_each<N - 1>(f);
        f(std::integral_constant<int, N - 1>());
    }
}

// One stage in LDS: rows, then weights.
template <int BM>
struct Stage {
    static constexpr int kW = BM * kQuantGroup;
    static constexpr int kBytes = kW + kTileN * kQuantGroup;
    static constexpr int kLoads = 1 + BM / 64 + 4;  // loads of a wave per step, scales first
};

// The scales of four blocks in LDS: per row, then per channel (MXFP8) or
// 128-channel block (the first two), the four blocks' words or their one word
// of bytes.  A row's scales of one block are a few bytes of a line of their
// own: read once per four blocks they cost L2 a quarter (MXFP8, gate and up
// products of 32,768 rows, 64 experts, 7168 -> 2 x 2048: 1465 -> 1141 us).
// Two chunks take turns; the third place takes what the loads that keep the
// count (TileLoads::issue) bring.
template <int QUANT, int BM>
struct Chunk {
    static constexpr int kWord = QUANT == MOE_QUANT_FP8_UE8M0 ? 4 : 16;
    static constexpr int kEntries = BM + (QUANT == MOE_QUANT_MXFP8 ? kTileN : kWave);
    static constexpr int kBytes = kEntries * kWord;
    static constexpr int kAll = 2 * kBytes + kWave * kWord;
    static_assert(kEntries <= kTileThreads, "one load");
};

// The loads of one tile: descriptors (uniform) and this lane's offsets.
// Rows past the tile's end are read as its last row and channels past the last
// as that one: every address is inside its array, and what comes of the
// copies is not stored.  The descriptors' range check serves one purpose, the
// blocks after the last one (bit 31 of a lane's offset, see issue); it compares
// the lane's offset with num_records minus the scalar offset, so the scalar
// offset always stays below num_records.
template <int QUANT, bool SWIGLU, int BM>
struct TileLoads {
    __amdgpu_buffer_rsrc_t a, w[2], s;
    uint32_t ao[BM / 64], wo[SWIGLU ? 2 : 4], so;  // rows, weights (both halves alike with SWIGLU), scales
    int KB, wave;
    using C = Chunk<QUANT, BM>;

    __device__ __forceinline__ void set(const ExpertGemmArgs &p, const TileAt &at, int wave_, int lane)
    {
        wave = wave_;
        const uint32_t k = (uint32_t)p.k;
        KB = p.k / kQuantGroup;
        const int SW = QUANT == MOE_QUANT_FP8_UE8M0 ? (KB + 3) / 4 : KB;  // scale words of a row
        const int NBn = (p.n + kQuantGroup - 1) / kQuantGroup;
        // 16-byte piece c of a row sits at position c ^ ((row >> 1) & 7) in LDS:
        // the 16 rows of a fragment then cover all banks.  A wave loads rows 8 j
        // .. 8 j + 7, j = wave (mod 8): lane l holds position l % 8 of row l / 8.
        const uint32_t piece = ((lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7)) * 16;
        const int row = 8 * wave + (lane >> 3);
        a = buffer(p.a + at.row0 * p.k, (uint32_t)at.valid * k);
#pragma unroll
        for (int i = 0; i < BM / 64; ++i)
            ao[i] = (uint32_t)min(row + 64 * i, at.valid - 1) * k + piece;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int32_t c = min(SWIGLU ? at.nt * 128 + h * (p.n / 2) : at.nt * kTileN + h * 128, p.n - 1);
            const int32_t left = min(128, p.n - c);
            w[h] = buffer(p.w + ((int64_t)at.e * p.n + c) * p.k, (uint32_t)left * k);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                wo[SWIGLU ? i : 2 * h + i] = (uint32_t)min(row + 64 * i, left - 1) * k + piece;
        }
        // scales: the first BM / 64 waves load the rows', the others the weights'
        const bool of_rows = wave < BM / kWave;
        const int t = (of_rows ? wave : wave - BM / kWave) * kWave + lane;
        const int32_t w_rows = QUANT == MOE_QUANT_MXFP8 ? p.n : NBn;
        const int32_t w_row = QUANT == MOE_QUANT_MXFP8
                                  ? (SWIGLU ? at.nt * 128 + (t & 127) + (t >> 7) * (p.n / 2) : at.nt * kTileN + t)
                                  : (SWIGLU ? at.nt + (t & 1) * (NBn / 2) : at.nt * 2 + (t & 1));
        const void *src = of_rows ? p.a_scale : p.w_scale;
        const int64_t first = of_rows ? at.row0 : (int64_t)at.e * w_rows;
        const int32_t rows = of_rows ? at.valid : w_rows;
        s = buffer(static_cast<const uint32_t *>(src) + first * SW, (uint32_t)rows * SW * 4);
        so = (uint32_t)min(of_rows ? t : w_row, rows - 1) * SW * 4;
    }
    // Loads FROM .. TO - 1 of step `at` (NS - 1 blocks before `kb`): block kb into a
    // stage and, every fourth step, the scales of the next four blocks into
    // the chunk that is not in use.  The blocks after the last are asked for
    // past the buffers' ends, which costs no memory access, and so are scales in
    // the other steps: every step has the same number of loads.
    template <int FROM, int TO>
    __device__ __forceinline__ void issue(uint8_t *st, int kb, uint8_t *chunks, int at) const
    {
        constexpr int kA = BM / 64;
        const uint32_t past = kb < KB ? 0u : 0x80000000u;
        const uint32_t at_k = kb < KB ? (uint32_t)kb * kQuantGroup : 0u;
#pragma unroll
        for (int j = FROM; j < TO; ++j) {
            if (j == 0) {
                const int c = (at >> 2) + 1;
                const bool turn = (at & 3) == 0 && wave < C::kEntries / kWave, some = turn && 4 * c < KB;
                const uint32_t to = turn ? (uint32_t)((c & 1) * C::kBytes + wave * kWave * C::kWord) : 2 * C::kBytes;
                load_lds<C::kWord>(s, chunks + to, so | (some ? 0u : 0x80000000u),
                                   some ? (uint32_t)c * C::kWord : 0u);
            } else if (j < 1 + kA) {
                const int i = j - 1;
                load_lds<16>(a, st + (wave + 8 * i) * 1024, ao[i] | past, at_k);
            } else {
                const int i = j - 1 - kA;
                load_lds<16>(w[i >> 1], st + Stage<BM>::kW + (wave + 8 * i) * 1024, wo[SWIGLU ? i & 1 : i] | past,
                             at_k);
            }
        }
    }
};

// acc += the stage's block for this wave's MT row fragments and kNF channel
// fragments, while block `kb_load` loads into the stage `free`: its loads are
// spread over the matrix instructions (all at once they would hold up the
// wave's LDS reads until the address unit has taken them).
//
// The 8-bit instruction adds its products eight at a time, aligned to the
// largest of the eight, and drops what lies 13 binary places below that one:
// 1.4e-5 (rms) of a block's result, where the bf16 instruction stays near 1e-8
// at half the rate.  A bf16 result, or values in 8 bits beside a power of two,
// hide that under their own rounding (2^-8, 2^-4); the fp32 scales of SwiGLU's
// rows show it, so in that format every block goes through bf16 operands,
// which hold E4M3 values exactly.  8-bit / bf16 there: 32,768 skewed rows, 64
// experts, 7168 -> 2 x 2048, 1.40 / 2.21 ms, scales 1.15e-5 / 2e-7 off (rms); 2048
// rows, 256 experts 1.21 / 1.31 ms.  With power-of-two scales, 64 experts x 512 rows:
// UE8M0 1.12 / 1.88 ms, MXFP8 1.18 / 1.98, a thousandth of the E4M3 values one step off
// (1.3e-3 of the whole, where the format's rounding is 2.6e-2) / none.
template <int QUANT, bool SWIGLU>
constexpr bool through_bf16() { return QUANT == MOE_QUANT_FP8_F32 && SWIGLU; }

template <int QUANT, bool SWIGLU, int BM, int MT>
__device__ __forceinline__ void multiply_stage(dev::f32x4 (&acc)[kNF][MT], const uint8_t *st, int wr, int wc, int lane,
                                               const TileLoads<QUANT, SWIGLU, BM> &loads, uint8_t *free, int kb_load,
                                               uint8_t *chunks, int kb)
{
    using C = Chunk<QUANT, BM>;
    constexpr int kLoads = Stage<BM>::kLoads;
    constexpr bool kBf16 = through_bf16<QUANT, SWIGLU>();
    const int r = lane & 15, g = lane >> 4;
    const int rswz = (r >> 1) & 7;
    const int rlo = r * kQuantGroup + ((g ^ rswz) * 16), rhi = r * kQuantGroup + (((4 + g) ^ rswz) * 16);
    const uint8_t *rows = st + wr * MT * 16 * kQuantGroup;
    const int u = kb & 3;
    const uint8_t *sc = chunks + ((kb >> 2) & 1) * C::kBytes + (QUANT == MOE_QUANT_FP8_UE8M0 ? 0 : 4 * u);
    const auto scale = [&](int entry) { return *reinterpret_cast<const uint32_t *>(sc + entry * C::kWord); };
    dev::i32x8 w[kNF], x[2];
    dev::bf16x8 wv[kBf16 ? kNF : 1][4];
    uint32_t sx[MT];
    int swb[kNF];
    float swf[2];
    const auto read_row = [&](int i) {
        x[i & 1] = join(*reinterpret_cast<const dev::u32x4 *>(rows + rlo + i * 16 * kQuantGroup),
                        *reinterpret_cast<const dev::u32x4 *>(rows + rhi + i * 16 * kQuantGroup));
    };
#pragma unroll
    for (int f = 0; f < kNF; ++f) {
        const int c = SWIGLU ? wc * 32 + (f & 1) * 16 + (f >> 1) * 128 : wc * 64 + f * 16;
        const uint8_t *src = st + Stage<BM>::kW + c * kQuantGroup;
        w[f] = join(*reinterpret_cast<const dev::u32x4 *>(src + rlo), *reinterpret_cast<const dev::u32x4 *>(src + rhi));
        if constexpr (QUANT == MOE_QUANT_MXFP8)
            swb[f] = (int)(scale(BM + c + r) >> (8 * g));
        if (f == 0) {
            read_row(0);
            // all scales before this step's load of scales: the compiler has reads
            // of the chunks wait for the last load into them
#pragma unroll
            for (int i = 0; i < MT; ++i)
                sx[i] = scale((wr * MT + i) * 16 + r);
        }
    }
    if constexpr (QUANT == MOE_QUANT_FP8_F32) {
        swf[0] = __uint_as_float(scale(BM + (SWIGLU ? 0 : wc >> 1)));
        swf[1] = SWIGLU ? __uint_as_float(scale(BM + 1)) : swf[0];
    } else if constexpr (QUANT == MOE_QUANT_FP8_UE8M0) {
        swb[0] = swb[1] = (int)(scale(BM + (SWIGLU ? 0 : wc >> 1)) >> (8 * u));
        swb[2] = swb[3] = SWIGLU ? (int)(scale(BM + 1) >> (8 * u)) : swb[0];
    }
    const auto part = [&](auto I) {
        constexpr int i = decltype(I)::value;
        if constexpr (i + 1 < MT)
            read_row(i + 1);
        if constexpr (QUANT == MOE_QUANT_FP8_F32) {
            const float s0 = __uint_as_float(sx[i]) * swf[0];
            const float s1 = SWIGLU ? __uint_as_float(sx[i]) * swf[1] : s0;
            dev::f32x4 d[kNF];
            dev::bf16x8 xv[4];
            if constexpr (kBf16)
                dev::block_to_bf16<QUANT>(half(x[i & 1], 0), half(x[i & 1], 4), 0, g, xv);
#pragma unroll
            for (int f = 0; f < kNF; ++f) {
                const dev::f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (kBf16) {
                    if constexpr (i == 0)
                        dev::block_to_bf16<QUANT>(half(w[f], 0), half(w[f], 4), 0, g, wv[f]);
                    d[f] = z;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        d[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[f][j], xv[j], d[f], 0, 0, 0);
                } else {
                    d[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[f], x[i & 1], z, 0, 0, 0, 0, 0, 0);
                }
            }
            loads.template issue<i * kLoads / MT, (i + 1) * kLoads / MT>(free, kb_load, chunks, kb);
#pragma unroll
            for (int f = 0; f < kNF; ++f)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[f][i][j] = __builtin_fmaf(d[f][j], f < 2 ? s0 : s1, acc[f][i][j]);
        } else {
            const int sb = (int)(sx[i] >> (8 * (QUANT == MOE_QUANT_FP8_UE8M0 ? u : g)));
#pragma unroll
            for (int f = 0; f < kNF; ++f)
                acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w[f], x[i & 1], acc[f][i], 0, 0, 0,
                                                                              swb[f], 0, sb);
            loads.template issue<i * kLoads / MT, (i + 1) * kLoads / MT>(free, kb_load, chunks, kb);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    for_each<MT>(part);
}

// Starts the loads of a tile's first NS - 1 stages.
template <int QUANT, bool SWIGLU, int BM, int NS>
__device__ __forceinline__ void start_tile(const ExpertGemmArgs &p, const TileAt &at, uint8_t *st0, uint8_t *st1,
                                           uint8_t *chunks, int wave, int lane)
{
    TileLoads<QUANT, SWIGLU, BM> loads;
    loads.set(p, at, wave, lane);
    loads.template issue<0, Stage<BM>::kLoads>(st0, 0, chunks, -4);
    __builtin_amdgcn_sched_barrier(0);  // in this order: the waits count
    if constexpr (NS == 3)
        loads.template issue<0, Stage<BM>::kLoads>(st1, 1, chunks, -3);
    __builtin_amdgcn_sched_barrier(0);
}

// Multiplies a tile whose first NS - 1 stages are in flight, then starts the
// next tile's (`more`) and writes the results.
template <int QUANT, bool SWIGLU, int BM, int NS, int MT>
__device__ __forceinline__ void run_tile(const ExpertGemmArgs &p, const TileAt &at, const TileAt &next, bool more,
                                         uint8_t *st0, uint8_t *st1, uint8_t *st2, uint8_t *chunks,
                                         float (*wave_max)[BM], int wave, int lane)
{
    TileLoads<QUANT, SWIGLU, BM> loads;
    loads.set(p, at, wave, lane);
    // the load of scales, first of its step and mostly without effect, is not counted
    constexpr int kAhead = (Stage<BM>::kLoads - 1) * (NS - 2);
    const int wr = wave / kWaveCols, wc = wave % kWaveCols;
    const int KB = loads.KB;
    dev::f32x4 acc[kNF][MT];
#pragma unroll
    for (int f = 0; f < kNF; ++f)
#pragma unroll
        for (int i = 0; i < MT; ++i)
            acc[f][i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const auto step = [&](uint8_t *cur, uint8_t *free, int kb) {
        wait_and_meet<kAhead>();
        multiply_stage<QUANT, SWIGLU, BM, MT>(acc, cur, wr, wc, lane, loads, free, kb + NS - 1, chunks, kb);
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
        start_tile<QUANT, SWIGLU, BM, NS>(p, next.scalars(), st0, st1, chunks, wave, lane);
    write_tile<QUANT, MT, SWIGLU, BM>(p, acc, at, wr, wc, lane, wave_max);
}

template <int QUANT, bool SWIGLU, int BM, int NS>
__global__ __launch_bounds__(kTileThreads) void expert_gemm_tiles(ExpertGemmArgs p, int32_t n_tiles)
{
    __shared__ int32_t tile_start[kMaxExperts / kGroup + 1];
    __shared__ int32_t red[kTileWaves];
    // separate variables: the compiler then knows which reads follow which loads
    __shared__ alignas(1024) uint8_t st0[Stage<BM>::kBytes];
    __shared__ alignas(1024) uint8_t st1[Stage<BM>::kBytes];
    __shared__ alignas(1024) uint8_t st2[NS == 3 ? Stage<BM>::kBytes : 16];
    __shared__ alignas(16) uint8_t chunks[Chunk<QUANT, BM>::kAll];
    __shared__ float wave_max[SWIGLU && QUANT != MOE_QUANT_MXFP8 ? kWaveCols : 1][BM];
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
    start_tile<QUANT, SWIGLU, BM, NS>(p, next, st0, st1, chunks, wave, lane);
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
            run_tile<QUANT, SWIGLU, BM, NS, MT>(p, at, next, more, st0, st1, st2, chunks, wave_max, wave, lane);
        else if (at.valid > M1 * 32)
            run_tile<QUANT, SWIGLU, BM, NS, M2>(p, at, next, more, st0, st1, st2, chunks, wave_max, wave, lane);
        else
            run_tile<QUANT, SWIGLU, BM, NS, M1>(p, at, next, more, st0, st1, st2, chunks, wave_max, wave, lane);
        if (!more)
            break;
    }
}

// ---------------------------------------------------------------------------
// Few rows and too few tiles for the chip: 16 rows x 16 channels per block, whose
// waves share the blocks of 128 input channels and add up in LDS, in order.
//
// Bound by latency: the tiles above would leave most compute units idle, with
// one step's round trip to memory after the other.
// ---------------------------------------------------------------------------

template <int QUANT>
__global__ __launch_bounds__(kTileThreads) void expert_gemm_strips(ExpertGemmArgs p, int32_t strips)
{
    __shared__ int32_t tile_start[kMaxExperts / kGroup + 1];
    __shared__ int32_t red[kTileWaves];
    __shared__ dev::f32x4 part[kTileWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = scalar(threadIdx.x / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int KB = p.k / kQuantGroup;
    const int KW = (KB + 3) / 4;
    const int NBn = (p.n + kQuantGroup - 1) / kQuantGroup;
    scan_tiles<16>(p, tile_start, red);
    const int64_t n_work = (int64_t)scalar(tile_start[(p.E + kGroup - 1) / kGroup]) * strips;

    for (int64_t work = blockIdx.x; work < n_work; work += gridDim.x) {
        const int32_t m = scalar((int32_t)(work / strips));
        const int32_t c0 = scalar((int32_t)(work - (int64_t)m * strips)) * 16;
        const ExpertAt ex = find_expert<16>(p, tile_start, m);
        const int32_t first = (m - ex.start) * 16, valid = min(16, ex.rows - first);
        const int64_t row0 = (int64_t)(p.expert_offset != nullptr ? word_of(p.expert_offset, ex.e) : 0) + first;
        // rows past the end: the last one, channels past the end: the last one
        const int64_t arow = row0 + min(r, valid - 1);
        const int32_t c = min(c0 + r, p.n - 1);
        const int64_t wrow = (int64_t)ex.e * p.n + c;
        const int64_t srow = QUANT == MOE_QUANT_MXFP8 ? wrow : (int64_t)ex.e * NBn + c0 / kQuantGroup;
        struct Block {
            dev::u32x4 w[2], x[2];
            uint32_t sw, sx;  // scales as they are stored
        };
        const auto fill = [&](Block &b, int kb) {
            const uint8_t *w = p.w + wrow * p.k + (int64_t)kb * kQuantGroup + 16 * g;
            const uint8_t *x = p.a + arow * p.k + (int64_t)kb * kQuantGroup + 16 * g;
            b.w[0] = *reinterpret_cast<const dev::u32x4 *>(w);
            b.w[1] = *reinterpret_cast<const dev::u32x4 *>(w + 64);
            b.x[0] = *reinterpret_cast<const dev::u32x4 *>(x);
            b.x[1] = *reinterpret_cast<const dev::u32x4 *>(x + 64);
            if constexpr (QUANT == MOE_QUANT_FP8_UE8M0) {
                b.sw = static_cast<const uint8_t *>(p.w_scale)[srow * KW * 4 + kb];
                b.sx = static_cast<const uint8_t *>(p.a_scale)[arow * KW * 4 + kb];
            } else {
                b.sw = static_cast<const uint32_t *>(p.w_scale)[srow * KB + kb];
                b.sx = static_cast<const uint32_t *>(p.a_scale)[arow * KB + kb];
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        dev::f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        const auto use = [&](const Block &b) {
            const dev::f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (QUANT == MOE_QUANT_FP8_F32) {
                const dev::f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    join(b.w[0], b.w[1]), join(b.x[0], b.x[1]), z, 0, 0, 0, 0, 0, 0);
                const float s = __uint_as_float(b.sx) * __uint_as_float(b.sw);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[j] = __builtin_fmaf(d[j], s, acc[j]);
            } else {
                const int shift = QUANT == MOE_QUANT_MXFP8 ? 8 * g : 0;
                acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    join(b.w[0], b.w[1]), join(b.x[0], b.x[1]), acc, 0, 0, 0, (int)(b.sw >> shift), 0,
                    (int)(b.sx >> shift));
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        constexpr int S = kTileWaves;
        if (wave < KB) {
            // four blocks in flight; past the last one, the last one again
            const int count = (KB - wave + S - 1) / S, last = wave + (count - 1) * S;
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
        part[wave][lane] = acc;
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int w = 1; w < kTileWaves; ++w)
                acc += part[w][lane];
            if (r < valid && c0 + 4 * g < p.n)
                *reinterpret_cast<uint2 *>(p.y + (row0 + r) * p.n + c0 + 4 * g) =
                    make_uint2(dev::pack_bf16(acc[0], acc[1]), dev::pack_bf16(acc[2], acc[3]));
        }
        __syncthreads();  // part is rewritten by the next strip
    }
}

// Row tiles of `rows` rows that a call can have: a segment's last one is partial.
int64_t max_tiles(const ExpertGemmArgs &p, int32_t rows)
{
    if (p.recv_count == nullptr)
        return (p.max_rows + rows - 1) / rows;
    return p.max_rows / rows + (p.max_rows < p.E ? p.max_rows : p.E);
}

template <int QUANT, bool SWIGLU, int BM, int NS>
hipError_t launch_tiles(const ExpertGemmArgs &p, hipStream_t stream)
{
    const int32_t n_tiles = SWIGLU ? p.n / 256 : (p.n + kTileN - 1) / kTileN;
    const int64_t tiles = max_tiles(p, BM) * n_tiles;
    // one block per compute unit (its stages fill LDS), a multiple of the 8 XCDs
    const int64_t cus = (device_cu_count() + 7) / 8 * 8;
    const int64_t grid = tiles < cus ? (tiles + 7) / 8 * 8 : cus;
    hipLaunchKernelGGL((expert_gemm_tiles<QUANT, SWIGLU, BM, NS>), dim3((uint32_t)grid), dim3(kTileThreads), 0,
                       stream, p, n_tiles);
    return hipGetLastError();
}

template <int QUANT, bool SWIGLU>
hipError_t launch_rows(const ExpertGemmArgs &p, hipStream_t stream)
{
    if constexpr (!SWIGLU) {
        const int64_t cus = device_cu_count();
        // Strips while there are few: a block's round trips take 5 us and more, and two
        // blocks fit a compute unit.  fp32 scales, in a graph, tiles / strips: one row,
        // 512 -> 512 6.8 / 3.8 us, 2048 -> 2048 13.1 / 5.6, 7168 -> 7168 (448 strips) 35.6 /
        // 15.3; 32 rows, 7168 -> 7168 (896) 36 / 47; 64 rows, 2048 -> 2048 (512) 15.2 / 13.7,
        // MXFP8 13.4 / 15.9; 4 rows each of 16 experts, 7168 ->
        // 512 (640) 36.5 / 19.4, of 8 experts, 2048 -> 2048 (1280) 14.6 / 20.8.
        const int32_t strips = (p.n + 15) / 16;
        const int64_t work = max_tiles(p, 16) * strips;
        if (2 * work <= 5 * cus) {
            hipLaunchKernelGGL((expert_gemm_strips<QUANT>), dim3((uint32_t)work), dim3(kTileThreads), 0, stream, p,
                               strips);
            return hipGetLastError();
        }
        // 256-row tiles read the weights half as often, with one stage less in flight
        // and larger remainders.  2048 -> 7168, 64 experts, 128 / 256 rows: 256 rows per
        // expert fp32 scales 421 / 446 us, UE8M0 376 / 387, MXFP8 390 / 427; 512: 683 /
        // 668, 631 / 613, 642 / 644; 1024: 1243 / 1199, 1168 / 1059, 1214 / 1114 (the 256-row
        // kernels of fp32 scales and MXFP8 spill 8 and 15 registers).
        // For SwiGLU (7168 -> 2 x 2048) 512: 1099 / 1201, 768: 1536 / 1654, 1024: 1996 /
        // 1977, and the registers spill.  Fewer tiles than compute units: 128 rows.
        if (p.max_rows / p.E >= 512 && max_tiles(p, 256) * ((p.n + kTileN - 1) / kTileN) >= cus)
            return launch_tiles<QUANT, SWIGLU, 256, 2>(p, stream);
    }
    return launch_tiles<QUANT, SWIGLU, 128, 3>(p, stream);
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
