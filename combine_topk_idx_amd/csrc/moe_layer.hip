// A whole expert layer for at most 64 tokens on gfx950: two kernels, no
// dispatch.
//
//   gate_up:  h[t,k]  = bf16( silu(W13g[e] x[t]) * (W13u[e] x[t]) )
//   down:     out[t]  = bf16( sum_k topk_w[t,k] * W2[e] h[t,k] )
//
// Both are bound by the weights of the experts that the batch reaches, each
// byte of which is read once: a wave streams 16 weight rows straight from
// memory into matrix-instruction operands, converting 8-bit values to bf16 on
// the way (exact), and the activations stay bf16.  Between the kernels h is
// bf16 too, as the definition says: the operand of the second product, and the
// one rounding between x and out (half a step, 2^-8, of each value: the output
// is 2.3e-3 off, rms, instead of the 1.7e-3 of its own rounding).
//
// Tokens are the columns of the products: an expert's tokens are packed into
// groups of 16.  gate_up has a block per (expert, 16 or 32 channels of h); down has
// a block per 16 or 32 output channels that walks every expert used and adds each
// one's columns, times the router's weight, to its tokens' sums in LDS, per wave
// and at last over the waves in a fixed order, without atomics.
#include "moe_mma.h"

namespace moe {

namespace {

constexpr int kLayerWaves = 4;                       // gate_up: channel slices of one product
constexpr int kDownWaves = 8;                         // down: waves that share the experts
constexpr int kRing1 = 3, kRing2 = 2;
constexpr int kLayerMaxPairs = MOE_LAYER_MAX_TOKENS * kMaxTopk;

// One lane's part of a 16-row weight strip (row `row` of [rows, k], or a clamped
// one): the 128 channels of block kb as four bf16 operands of 8 channels each
// (channels 16 g .. of each 64: the columns use the same order), multiplied by
// the block's scale where that is a power of two.
template <int QUANT>
struct Weights {
    dev::u32x4 v[QUANT == MOE_QUANT_NONE ? 4 : 2];
    // The block's scale as it is stored (computing with it here would wait for
    // the load): fp32 bits, the exponent byte, or the four MX blocks' bytes.
    uint32_t s;

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
                s = static_cast<const uint32_t *>(scale)[nb * KB + kb];
            } else if constexpr (QUANT == MOE_QUANT_FP8_UE8M0) {
                s = static_cast<const uint8_t *>(scale)[nb * ((KB + 3) / 4 * 4) + kb];
            } else {
                s = static_cast<const uint32_t *>(scale)[row * KB + kb];
            }
        }
    }
    // acc += W * x over the block; x: four operands of the column
    __device__ __forceinline__ void fma(const dev::u32x4 x[4], dev::f32x4 &acc, const dev::bf16x8 wv[4]) const
    {
        if constexpr (QUANT == MOE_QUANT_FP8_F32) {
            dev::f32x4 d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], __builtin_bit_cast(dev::bf16x8, x[j]), d, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[j] = __builtin_fmaf(d[j], __uint_as_float(s), acc[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv[j], __builtin_bit_cast(dev::bf16x8, x[j]), acc, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void convert(dev::bf16x8 wv[4], int g) const
    {
        if constexpr (QUANT == MOE_QUANT_NONE) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                wv[j] = __builtin_bit_cast(dev::bf16x8, v[j]);
        } else {
            dev::block_to_bf16<QUANT>(v[0], v[1], s, g, wv);
        }
    }
};

// The matching operands of a column: 128 channels of a bf16 row.  Columns
// without a token read some other token's row: no column's result depends on
// another column, and theirs are not used.
__device__ __forceinline__ void load_column(const uint16_t *row, int kb, int g, dev::u32x4 v[4])
{
    const uint16_t *p = row + kb * kQuantGroup + 16 * g;
    v[0] = *reinterpret_cast<const dev::u32x4 *>(p);
    v[1] = *reinterpret_cast<const dev::u32x4 *>(p + 8);
    v[2] = *reinterpret_cast<const dev::u32x4 *>(p + 64);
    v[3] = *reinterpret_cast<const dev::u32x4 *>(p + 72);
}

// The experts that a batch reaches, one slot per candidate: where the batch has
// no more pairs than there are experts, slot i stands for the expert of pair i
// and counts if no earlier pair has it; otherwise slot e stands for expert e.
// gate_up leaves the mask of the slot's tokens (0: the slot does not count) for
// down.
__host__ __device__ __forceinline__ int32_t layer_slots(int32_t pairs, int32_t E) { return pairs <= E ? pairs : E; }

// Columns of one expert: the tokens of `mask`, in order.  token_pair[c] = token *
// K + its first pair's k, per wave in LDS (n <= 64 entries).
__device__ __forceinline__ int list_tokens(const int32_t *ids, int32_t T, int32_t K, int32_t e, int lane,
                                           uint64_t &mask, int32_t *token_pair)
{
    int first = -1;
    if (lane < T)
        for (int k = K - 1; k >= 0; --k)
            first = ids[lane * K + k] == e ? k : first;
    mask = __ballot(first >= 0);
    if (first >= 0)
        token_pair[dev::lanes_below(mask)] = lane * K + first;
    return __popcll(mask);
}

// Block (slot, 16 F channels of h): each wave takes every kLayerWaves-th block
// of 128 input channels, the next one's loads in flight, and all the expert's
// tokens.
template <int QUANT, int G, int F>
__global__ __launch_bounds__(kLayerWaves *kWave, 2) void layer_gate_up(LayerArgs a)
{
    __shared__ int32_t ids[kLayerMaxPairs];
    __shared__ int32_t pairs[kLayerWaves][kWave];
    __shared__ float part[kLayerWaves][2 * F][G][kWave][4];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int P = a.T * a.K;
    const int slot = blockIdx.y, tile = blockIdx.x;
    const bool by_pair = P <= a.E;
    for (int i = tid; i < P; i += kLayerWaves * kWave)
        ids[i] = a.topk_idx[i];
    __syncthreads();
    const int32_t e = by_pair ? __builtin_amdgcn_readfirstlane(ids[slot]) : slot;
    bool counts = e >= 0 && e < a.E;
    if (by_pair) {
        bool earlier = false;
        for (int i = lane; i < slot; i += kWave)
            earlier |= ids[i] == e;
        counts = counts && __ballot(earlier) == 0;  // the same in every wave
    }
    uint64_t mask = 0;
    int n = 0;
    if (counts)
        n = list_tokens(ids, a.T, a.K, e, lane, mask, pairs[wave]);
    if (tile == 0 && tid == 0)
        a.masks[slot] = mask;
    if (n == 0)
        return;
    const int KB = a.H / kQuantGroup;
    const int c0 = tile * 16 * F;
    const int NBn = 2 * a.I / kQuantGroup;
    // fragments 0 .. F - 1: gate channels, F .. 2 F - 1: up channels
    int64_t row[2 * F], nb[2 * F];
#pragma unroll
    for (int f = 0; f < 2 * F; ++f) {
        const int c = c0 + (f % F) * 16 + (f / F) * a.I;
        row[f] = (int64_t)e * 2 * a.I + c + r;
        nb[f] = (int64_t)e * NBn + c / kQuantGroup;
    }
    const uint16_t *x[G];
#pragma unroll
    for (int i = 0; i < G; ++i)
        x[i] = a.x + (int64_t)(pairs[wave][i * 16 + r < n ? i * 16 + r : 0] / a.K) * a.H;
    dev::f32x4 acc[2 * F][G];
#pragma unroll
    for (int f = 0; f < 2 * F; ++f)
#pragma unroll
        for (int i = 0; i < G; ++i)
            acc[f][i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    struct Stage {
        Weights<QUANT> w[2 * F];
        dev::u32x4 x[4];
    };
    // No load is conditional inside the loop: where paths with and without
    // loads in flight meet, the compiler waits for all of them.
    const auto fill = [&](Stage &st, int kb) {
#pragma unroll
        for (int f = 0; f < 2 * F; ++f)
            st.w[f].load(a.w13, a.w13_scale, row[f], nb[f], a.H, kb, g);
        load_column(x[0], kb, g, st.x);
        __builtin_amdgcn_sched_barrier(0);
    };
    const auto use = [&](const Stage &st, int kb) {
#pragma unroll
        for (int f = 0; f < 2 * F; ++f) {
            dev::bf16x8 wv[4];
            st.w[f].convert(wv, g);
            st.w[f].fma(st.x, acc[f][0], wv);
#pragma unroll
            for (int i = 1; i < G; ++i)
                if (i * 16 < n) {
                    dev::u32x4 xi[4];
                    load_column(x[i], kb, g, xi);
                    st.w[f].fma(xi, acc[f][i], wv);
                }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    if (wave < KB) {
        constexpr int S = kLayerWaves;
        Stage s0, s1;
        int kb = wave;
        fill(s0, kb);
        for (; kb + 2 * S < KB; kb += 2 * S) {
            fill(s1, kb + S);
            use(s0, kb);
            fill(s0, kb + 2 * S);
            use(s1, kb + S);
        }
        if (kb + S < KB) {
            fill(s1, kb + S);
            use(s0, kb);
            use(s1, kb + S);
        } else {
            use(s0, kb);
        }
    }
#pragma unroll
    for (int f = 0; f < 2 * F; ++f)
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                part[wave][f][i][lane][j] = acc[f][i][j];
    __syncthreads();
    for (int u = wave; u < F * G; u += kLayerWaves) {  // one fragment and column group per wave
        const int f = u % F, i = u / F;
        float gv[4] = {}, uv[4] = {};
#pragma unroll
        for (int w = 0; w < kLayerWaves; ++w)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                gv[j] += part[w][f][i][lane][j];
                uv[j] += part[w][F + f][i][lane][j];
            }
        if (i * 16 + r < n)
            *reinterpret_cast<uint2 *>(a.h + (int64_t)pairs[wave][i * 16 + r] * a.I + c0 + f * 16 + g * 4) =
                make_uint2(dev::pack_bf16(dev::swiglu(gv[0], uv[0]), dev::swiglu(gv[1], uv[1])),
                           dev::pack_bf16(dev::swiglu(gv[2], uv[2]), dev::swiglu(gv[3], uv[3])));
    }
}

// Block of 16 F output channels: its waves share the experts (and, with few of
// them, the input channels: `slices` waves per expert).  A wave adds its
// experts' weighted results to its own sums per token in LDS, in a fixed
// order; the waves' sums are added at the end.
template <int QUANT, int G, int F, int R>
__global__ __launch_bounds__(kDownWaves *kWave) void layer_down(LayerArgs a, int32_t slices)
{
    constexpr int kT = G * 16, NW = kDownWaves;
    __shared__ int32_t ids[kLayerMaxPairs];
    __shared__ float weights[kLayerMaxPairs];
    __shared__ int16_t used[kLayerMaxPairs];
    __shared__ int32_t n_used;
    __shared__ int32_t pairs[NW][kWave];
    __shared__ float sums[NW][kT][16 * F];
    const int tid = threadIdx.x, lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int r = lane & 15, g = lane >> 4;
    const int P = a.T * a.K;
    const int slots = layer_slots(P, a.E);
    for (int i = tid; i < P; i += NW * kWave) {
        ids[i] = a.topk_idx[i];
        weights[i] = a.topk_w[i];
    }
    if (wave == 0) {  // the slots that count, in order
        int n = 0;
        for (int i0 = 0; i0 < slots; i0 += kWave) {
            const bool mine = i0 + lane < slots && a.masks[i0 + lane] != 0;
            const uint64_t m = __ballot(mine);
            if (mine)
                used[n + dev::lanes_below(m)] = (int16_t)(i0 + lane);
            n += __popcll(m);
        }
        if (lane == 0)
            n_used = n;
    }
    for (int i = lane; i < kT * 16 * F; i += kWave)
        (&sums[wave][0][0])[i] = 0.0f;
    __syncthreads();
    const int KB = a.I / kQuantGroup;
    const int c0 = blockIdx.x * 16 * F;
    const int NBn = a.H / kQuantGroup;
    const int units = __builtin_amdgcn_readfirstlane(n_used) * slices;

    // A wave's work: the 128-channel blocks of the units wave, wave + NW, ...,
    // R - 1 of them in flight while one is used.
    struct Stage {
        Weights<QUANT> w[F];
        dev::u32x4 x[4];
        int pair[G];      // this lane's columns: token * K + its first pair's k, or -1
        int e, n, kb;
        bool last;        // the unit's last block
    };
    int unit = wave, e = 0, kb = 0, end = 0, n = 0, pair[G];  // the block that loads next
    const auto start_unit = [&]() {
        const int slot = __builtin_amdgcn_readfirstlane(used[unit / slices]);
        const int slice = unit % slices;
        e = P <= a.E ? __builtin_amdgcn_readfirstlane(ids[slot]) : slot;
        kb = slice * KB / slices;
        end = (slice + 1) * KB / slices;
        uint64_t mask;
        n = list_tokens(ids, a.T, a.K, e, lane, mask, pairs[wave]);
#pragma unroll
        for (int i = 0; i < G; ++i)
            pair[i] = i * 16 + r < n ? pairs[wave][i * 16 + r] : -1;
    };
    // Loads are never conditional, see gate_up: past the last block, that one again.
    const auto fill = [&](Stage &st) {
#pragma unroll
        for (int f = 0; f < F; ++f)
            st.w[f].load(a.w2, a.w2_scale, (int64_t)e * a.H + c0 + f * 16 + r,
                         (int64_t)e * NBn + (c0 + f * 16) / kQuantGroup, a.I, kb, g);
        // lane 0 has a token (the lane read comes before the choice: in a branch
        // of its own only the lanes without one would take part)
        const int first = __builtin_amdgcn_readfirstlane(pair[0]);
        const int row = max(pair[0] >= 0 ? pair[0] : first, 0);
        load_column(a.h + (int64_t)row * a.I, kb, g, st.x);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < G; ++i)
            st.pair[i] = pair[i];
        st.e = e, st.n = n, st.kb = kb, st.last = kb + 1 == end;
        if (kb + 1 < end) {
            ++kb;
        } else if (unit + NW < units) {
            unit += NW;
            start_unit();
        }
    };
    dev::f32x4 acc[F][G];
#pragma unroll
    for (int f = 0; f < F; ++f)
#pragma unroll
        for (int i = 0; i < G; ++i)
            acc[f][i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const auto use = [&](const Stage &st) {
#pragma unroll
        for (int f = 0; f < F; ++f) {
            dev::bf16x8 wv[4];
            st.w[f].convert(wv, g);
            st.w[f].fma(st.x, acc[f][0], wv);
#pragma unroll
            for (int i = 1; i < G; ++i)
                if (i * 16 < st.n) {
                    dev::u32x4 xi[4];
                    load_column(a.h + (int64_t)max(st.pair[i], 0) * a.I, st.kb, g, xi);
                    st.w[f].fma(xi, acc[f][i], wv);
                }
        }
        if (st.last) {  // the unit's weighted results
#pragma unroll
            for (int i = 0; i < G; ++i) {
                if (st.pair[i] >= 0) {
                    const int token = st.pair[i] / a.K;
                    float gate = 0.0f;
                    for (int k = 0; k < a.K; ++k)
                        if (ids[token * a.K + k] == st.e)
                            gate += weights[token * a.K + k];
#pragma unroll
                    for (int f = 0; f < F; ++f) {
                        float *s = &sums[wave][token][16 * f + 4 * g];
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            s[q] = __builtin_fmaf(acc[f][i][q], gate, s[q]);
                    }
                }
#pragma unroll
                for (int f = 0; f < F; ++f)
                    acc[f][i] = dev::f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    if (unit < units) {
        int left = 0;
        for (int u = wave; u < units; u += NW)
            left += (u % slices + 1) * KB / slices - u % slices * KB / slices;
        Stage st[R];
        start_unit();
#pragma unroll
        for (int j = 0; j < R - 1; ++j)
            fill(st[j]);
        for (bool more = true; more;) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                fill(st[(j + R - 1) % R]);
                use(st[j]);
                if (--left == 0) {
                    more = false;
                    break;
                }
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * 4 * F; i += NW * kWave) {  // 4 channels of a token
        const int token = i / (4 * F), q = (i % (4 * F)) * 4;
        float v[4] = {};
#pragma unroll
        for (int u = 0; u < NW; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] += sums[u][token][q + j];
        *reinterpret_cast<uint2 *>(a.out + (int64_t)token * a.H + c0 + q) =
            make_uint2(dev::pack_bf16(v[0], v[1]), dev::pack_bf16(v[2], v[3]));
    }
}

template <int QUANT, int G>
hipError_t launch_groups(const LayerArgs &a, hipStream_t stream)
{
    const int32_t slots = layer_slots(a.T * a.K, a.E);
    const int32_t cus = device_cu_count();
    // 32 channels of h per block read x half as often, where enough blocks are left.
    // Whole layer, 7168 -> 2048, 64 experts, top 8, 16 / 32 channels: 48 tokens fp32
    // scales 543 / 520 us, UE8M0 528 / 497, MXFP8 666 / 666; 64 tokens 587 / 547, 567 /
    // 521, 704 / 694; 24 tokens 451 / 450, 456 / 450, 574 / 564.  With fewer blocks 16
    // tokens, 32 experts, 4096 -> 1536: 127 / 130, 128 / 131, 149 / 145.  MXFP8 spills 6
    // registers there.  bf16 weights would spill 66: 48 tokens 969 / 1052 us, 64 tokens
    // 990 / 1065, 8 tokens 631 / 636.
    constexpr int kWide = QUANT == MOE_QUANT_NONE ? 1 : 2;
    if (kWide > 1 && (int64_t)slots * (a.I / (16 * kWide)) >= 8 * cus)
        hipLaunchKernelGGL((layer_gate_up<QUANT, G, kWide>), dim3(a.I / (16 * kWide), slots),
                           dim3(kLayerWaves * kWave), 0, stream, a);
    else
        hipLaunchKernelGGL((layer_gate_up<QUANT, G, 1>), dim3(a.I / 16, slots), dim3(kLayerWaves * kWave), 0, stream,
                           a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int32_t KB = a.I / kQuantGroup;
    int32_t slices = slots < kDownWaves ? (kDownWaves + slots - 1) / slots : 1;
    slices = slices < KB ? slices : KB;
    // 16 output channels per block where that is one block per compute unit at most,
    // with a ring of three, else 32 with a ring of two.  Whole layer, 16 / 32: 5
    // tokens, MXFP8, H = 2048: 55 / 66 us; H = 7168: 1 token 73 / 67, 48 tokens 573 / 516.
    if (a.H / 16 <= cus)
        hipLaunchKernelGGL((layer_down<QUANT, G, 1, kRing1>), dim3(a.H / 16), dim3(kDownWaves * kWave), 0, stream, a,
                           slices);
    else
        hipLaunchKernelGGL((layer_down<QUANT, G, 2, kRing2>), dim3(a.H / 32), dim3(kDownWaves * kWave), 0, stream, a,
                           slices);
    return hipGetLastError();
}

template <int QUANT>
hipError_t launch_quant(const LayerArgs &a, hipStream_t stream)
{
    if (a.T <= 16)
        return launch_groups<QUANT, 1>(a, stream);
    if (a.T <= 32)
        return launch_groups<QUANT, 2>(a, stream);
    return launch_groups<QUANT, 4>(a, stream);
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
