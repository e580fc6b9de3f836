// Device building blocks of the grouped products' tile kernels: the table of
// the experts' row tiles, uniform values, buffer descriptors, loads from memory
// into LDS and the waits for them.  `Args` has recv_count, expert_offset (NULL:
// one group of dense_rows rows), E and dense_rows.
#pragma once

#include <type_traits>

#include "moe_mma.h"

namespace moe {
namespace tile {

constexpr int kTileThreads = 512;
constexpr int kTileWaves = kTileThreads / kWave;
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

// This lane's number, anew: what is computed from it stays with the code that uses
// it.  Kept over a loop of tiles instead, it fills registers that the tiles need, is
// spilled, and each reload waits for every store before it.
__device__ __forceinline__ int here(int lane)
{
    asm volatile("" : "+v"(lane));
    return lane;
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
template <int BM, int THREADS = kTileThreads, typename Args>
__device__ inline void scan_tiles(const Args &p, int32_t *tile_start, int32_t *red)
{
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int groups = (p.E + kGroup - 1) / kGroup;
    const int per = (groups + THREADS - 1) / THREADS;
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
    int32_t run = dev::sum_before<THREADS / kWave>(red, wave) + incl - local;
    for (int e = e0; e < e1; ++e) {
        if (e % kGroup == 0)
            tile_start[e / kGroup] = run;
        run += tiles(e);
    }
    if (tid == THREADS - 1)
        tile_start[groups] = run;
    __syncthreads();
}

// An expert, the number of its first row tile and of its rows.
struct ExpertAt {
    int32_t e, start, rows;
};

// The expert that row tile m (uniform, below the number of all) belongs to.
template <int BM, typename Args>
__device__ __forceinline__ ExpertAt find_expert(const Args &p, const int32_t *tile_start, int32_t m)
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

}  // namespace tile
}  // namespace moe
