// Device building blocks of the bf16 products' tiles: matrix-instruction
// fragments from stages that hold rows or summed steps, and results that trade
// places for whole cache lines.
#pragma once

#include "moe_tiles.h"

namespace moe {
namespace tile {
namespace train {

constexpr int kWaveRows = 2, kWaveCols = 4;   // waves over the tile's rows and channels
constexpr int kNF = 4;                        // 16-channel fragments per wave
constexpr int kTileN = kWaveCols * kNF * 16;  // output channels per block
constexpr int kStep = 64;                     // summed channels of a stage: 128 bytes of a row

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Four steps of this lane's channel: the lanes of 16 read 4 steps x 16 channels.
__device__ __forceinline__ s16x4 read_steps(const uint8_t *p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)p);
}

__device__ __forceinline__ dev::bf16x8 join_steps(const s16x4 &lo, const s16x4 &hi)
{
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(dev::bf16x8, (s16x8)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Both halves of a step for 16 rows or channels.
struct Fragment {
    dev::bf16x8 h[2];
};

// From rows of 128 bytes, `base` the fragment's first; lo, hi: this lane's pieces.
__device__ __forceinline__ Fragment read_rows(const uint8_t *base, int lo, int hi)
{
    return Fragment{{*reinterpret_cast<const dev::bf16x8 *>(base + lo), *reinterpret_cast<const dev::bf16x8 *>(base + hi)}};
}

// From 64 steps of 2 * COLS bytes; `at`: this lane's place in the first.
template <int COLS>
__device__ __forceinline__ Fragment read_columns(const uint8_t *at)
{
    Fragment f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        f.h[h] = join_steps(read_steps(at + h * 64 * COLS), read_steps(at + h * 64 * COLS + 8 * COLS));
    return f;
}

constexpr int kStreamed = 2;  // stores marked non-temporal: L2 stays with the operands

// A lane has 4 adjacent channels of one row in each of two fragments (packed
// bf16, words lo and hi of each); after: 8 adjacent channels of that row, at
// (g & 1) * 16 + (g >> 1) * 8 of the two fragments' 32.  Its own inverse.
__device__ __forceinline__ void trade_fragments(dev::u32x4 &v)
{
    const auto lo = __builtin_amdgcn_permlane16_swap(v[0], v[2], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(v[1], v[3], false, false);
    v = dev::u32x4{lo[0], hi[0], lo[1], hi[1]};
}

// Two such vectors of one row, 64 channels with those of four lanes: after, v[0]
// is of row r % 8 and v[1] of row r % 8 + 8, the lower lanes' (r < 8) the first 32
// channels, the upper ones' the others: a store covers whole cache lines, 128
// bytes of each of 8 rows.  Its own inverse.
__device__ __forceinline__ void trade_rows(dev::u32x4 (&v)[2], bool low)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t other = __builtin_amdgcn_update_dpp(0, low ? v[1][j] : v[0][j], 0x128, 0xF, 0xF, true);
        v[0][j] = low ? v[0][j] : other;
        v[1][j] = low ? other : v[1][j];
    }
}

__device__ __forceinline__ dev::u32x4 pack_fragments(const dev::f32x4 &a, const dev::f32x4 &b)
{
    return dev::u32x4{dev::pack_bf16(a[0], a[1]), dev::pack_bf16(a[2], a[3]), dev::pack_bf16(b[0], b[1]),
                      dev::pack_bf16(b[2], b[3])};
}

// The wave's 64 adjacent channels from c0 of 16 rows as bf16, whole lines.
__device__ __forceinline__ void store_lines(__amdgpu_buffer_rsrc_t out, const dev::f32x4 (&v)[kNF], int row0, int valid,
                                            int32_t c0, int32_t channels, int lane)
{
    const int r = lane & 15, g = lane >> 4;
    const bool low = r < 8;
    dev::u32x4 s[2] = {pack_fragments(v[0], v[1]), pack_fragments(v[2], v[3])};
    trade_fragments(s[0]);
    trade_fragments(s[1]);
    trade_rows(s, low);
    const int32_t c = c0 + (low ? 0 : 32) + (g & 1) * 16 + (g >> 1) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = row0 + h * 8 + (r & 7);
        const uint32_t off = row < valid && c < channels ? ((uint32_t)row * (uint32_t)channels + c) * 2 : 0x80000000u;
        __builtin_amdgcn_raw_buffer_store_b128(s[h], out, off, 0, kStreamed);
    }
}

}  // namespace train
}  // namespace tile
}  // namespace moe
