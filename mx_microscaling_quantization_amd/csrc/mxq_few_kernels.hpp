// mxq_few_kernels.hpp -- gfx950 kernels of a whole mixture-of-experts layer for a
// few tokens (a decode step).
//
//     out[t] = sum over j of weights[t][j] * y[t][j]
//     y[t][j] = act(x[t] @ W1_e) @ W2_e,   e = ids[t][j]
//     act(z) = silu(z), or silu(z[.. F - 1]) * z[F ..] (swiglu)
//
// W1 [K, F or 2 F] and W2 [F, N] of each expert in MX, quantized along the
// contraction (32 values of one column share an E8M0). With few tokens the time is that
// of reading the chosen experts' weights once, so nothing else is worth a launch:
// two kernels, the first up to the activation, the second the down projection and
// the weighted sum over the slots. There is no sort: each workgroup finds the a-th
// expert that is in use, and the pairs that chose it, from the ids themselves (about 2
// us, all workgroups at the same time).
//
// Weights' bytes bound both kernels from some tens of experts on (16 x 4 pairs, 32 experts of
// e4m3fn, 4096 -> 2 x 2048 -> 4096: 69 and 48 us, 7.0 and 5.0 TB/s); one token's are launches and
// latency (8 of 128 experts of e2m1, 2048 -> 2 x 768 -> 2048: 9 to 10 and 9 us); with e2m1 and
// several tokens an expert, widening the weights (61 x 6 pairs of f16, 64 experts, 2016 -> 1440
// -> 2012: 20 and 30 us).
//
// The activations stay as they come: weights are widened to bf16 in registers, which is
// exact for every code (3 fraction bits at most) and scale byte but the rarest (values below
// 2^-133, see few_sums_low, and 255, see few_exact), and the products run on the bf16 matrix
// cores with fp32 sums. An f16 x is the sum of two bf16 numbers exactly; what is
// between the two products (fp32) is kept as two bf16 numbers, 16 bits of it (fewer below
// 2^-117, where the second one's last bit is 2^-133).
//
// v_mfma_f32_16x16x32_bf16: lane l = i + 16 g supplies values k = 8 g .. 8 g + 7 of row
// (column) i; result register r of lane l is D[4 g + r][i]. One instruction is one MX
// block of 16 columns, and a lane's 8 values are two containers of its column.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_grouped_kernels.hpp"

namespace mxq {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));

enum { kActSilu = 0, kActSwiglu = 1 };

constexpr uint32_t kFewPairs = 1024;     // pairs a workgroup finds its expert among
constexpr uint32_t kFewWaves = 8;        // waves that share the contraction, at most
constexpr uint32_t kFewThreads = 64 * kFewWaves;

constexpr int kFewLaneCols = 4;                     // columns of a lane
constexpr uint32_t kFewCols = 16u * kFewLaneCols;   // and of a workgroup

// ----------------------------------------------------------------------------
// Which expert, which pairs
// ----------------------------------------------------------------------------

struct FewRoute {
    uint8_t used[kFewWaves][1024];       // experts in use, a byte each; every wave has its own copy
    uint32_t count;                      // pairs of this workgroup's expert, in order
    uint16_t pairs[kFewPairs];
};

// This workgroup's place: one of the experts in use (in order of their numbers; `active`
// of them are), its pairs, which are then in route.pairs in order, and a column tile. Each
// XCD gets consecutive places, so that a line of weights that two column tiles share is
// read into one L2. False where there is no place for this workgroup. Every thread of the
// workgroup takes part. Each wave finds the expert by itself, so that one barrier is all
// (the list of pairs, by wave 0).
struct FewPlace {
    uint32_t expert, count, tile, active;
};

template <typename ID>
__device__ __forceinline__ bool few_route(FewRoute &route, const void *ids_, uint32_t n, uint32_t experts,
                                          uint32_t tiles, FewPlace &place)
{
    const ID *ids = reinterpret_cast<const ID *>(ids_);
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr uint32_t per = kFewPairs / 64u;
    volatile uint8_t *used = route.used[wave];
    ID id[per];
#pragma unroll
    for (uint32_t q = 0; q < per; q++)
        if (64u * q < n)
            id[q] = ids[min(64u * q + lane, n - 1u)];
    // (bytes, not bits: lanes that name one expert write the same byte, where atomic ors of
    // one word go one after the other, 5 us for 366 pairs of 64 experts)
    volatile uint32_t *words = reinterpret_cast<volatile uint32_t *>(used);
#pragma unroll
    for (uint32_t k = 0; k < 4; k++)
        words[64u * k + lane] = 0;
#pragma unroll
    for (uint32_t q = 0; q < per; q++)
        if (64u * q < n && id[q] >= 0 && (uint64_t)id[q] < experts)
            used[id[q]] = 1;
    // lane l has experts 16 l .. 16 l + 15
    uint32_t flags = 0;
#pragma unroll
    for (uint32_t k = 0; k < 4; k++)     // four bytes of 0 or 1 to four bits
        flags |= ((words[4u * lane + k] * 0x01020408u) >> 24) << (4u * k);
    uint32_t before = __popc(flags);
    const uint32_t own = before;
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)before, d);
        before += lane >= d ? o : 0u;
    }
    place.active = (uint32_t)__builtin_amdgcn_readlane((int)before, 63);
    before -= own;
    const uint32_t t = xcd_tile(blockIdx.x, place.active * tiles);
    const uint32_t a = t / tiles;
    place.tile = t - a * tiles;
    if (a >= place.active)
        return false;
    // the lane that has the a-th of them
    uint32_t bit = 0;
    const bool here = a >= before && a < before + own;
    if (here) {
        for (uint32_t k = a - before; k > 0; k--)
            flags &= flags - 1u;
        bit = 16u * lane + (uint32_t)__builtin_ctz(flags);
    }
    const uint32_t at = (uint32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(here));
    place.expert = (uint32_t)__builtin_amdgcn_readlane((int)bit, (int)at);
    if (wave == 0) {
        uint32_t count = 0;
#pragma unroll
        for (uint32_t q = 0; q < per; q++)
            if (64u * q < n) {
                const bool mine = 64u * q + lane < n && id[q] == (ID)place.expert;
                const uint64_t match = __builtin_amdgcn_ballot_w64(mine);
                if (mine)
                    route.pairs[count + (uint32_t)__popcll(match & ((1ull << lane) - 1ull))] =
                        (uint16_t)(64u * q + lane);
                count += (uint32_t)__popcll(match);
            }
        if (lane == 0)
            route.count = count;
    }
    __syncthreads();
    place.count = (uint32_t)__builtin_amdgcn_readfirstlane((int)route.count);
    return true;
}

// ----------------------------------------------------------------------------
// Weights and activations of one MX block
// ----------------------------------------------------------------------------

// An expert's matrix [K, C] in MX: K / 4 rows of C containers, K / 32 rows of C scale bytes.
struct FewMatrix {
    const uint8_t *data, *scale;
    uint32_t C;
};

template <int FMT> struct FewBlock {
    static constexpr int dwords = kFewLaneCols * (FMT == kOutE2M1 ? 2 : 4) / 4;
    uint32_t v[2][dwords];     // containers of view rows 2 g and 2 g + 1
    uint32_t scale;            // E8M0 of the columns
};

// Block b, the lane's columns from its offsets on (past every buffer where it has none).
template <int FMT>
__device__ __forceinline__ void few_load(FewBlock<FMT> &r, const __amdgpu_buffer_rsrc_t &data,
                                         const __amdgpu_buffer_rsrc_t &scale, uint32_t C, uint32_t b, uint32_t at_data,
                                         uint32_t at_scale)
{
    constexpr uint32_t CB = FMT == kOutE2M1 ? 2 : 4;
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const uint32_t row = (8u * b + q) * CB * C;
        if constexpr (FewBlock<FMT>::dwords == 2) {
            const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(data, at_data, row, kBufferNT);
            r.v[q][0] = w.x;
            r.v[q][1] = w.y;
        } else {
            const u32x4_t w = __builtin_amdgcn_raw_buffer_load_b128(data, at_data, row, kBufferNT);
#pragma unroll
            for (int k = 0; k < 4; k++)
                r.v[q][k] = w[k];
        }
    }
    r.scale = __builtin_amdgcn_raw_buffer_load_b32(scale, at_scale, b * C, 0);
}

// The scale byte of column u, in an fp32 number's exponent.
template <int FMT> __device__ __forceinline__ uint32_t few_exponent(const FewBlock<FMT> &r, int u)
{
    return (u < 3 ? r.scale << (23 - 8 * u) : r.scale >> 1) & 0x7F800000u;
}

// Below this byte a code times its scale may be below 2^-133, bf16's last bit (e5m2: below 10,
// e4m3fn: below 3; e2m1's smallest value times 2^-127 is above it).
constexpr uint32_t kFewLow = 16;

// Whether this lane has a column with such a byte and a code that is not zero (a quantized block
// of zeros has byte 1).
template <int FMT> __device__ __forceinline__ bool few_low(const FewBlock<FMT> &r)
{
    if constexpr (FMT == kOutE2M1) {
        return false;
    } else {
        bool low = false;
        const uint32_t v = r.scale & 0xF0F0F0F0u;    // (a byte of zeros borrows)
        if (wave_any(((v - 0x01010101u) & ~v & 0x80808080u) != 0))
#pragma unroll
            for (int u = 0; u < kFewLaneCols; u++)
                low |= few_exponent(r, u) < kFewLow << 23 && ((r.v[0][u] | r.v[1][u]) & 0x7F7F7F7Fu) != 0;
        return low;
    }
}

// Column u's 8 values times s, as bf16.
template <int FMT> __device__ __forceinline__ bf16x8_t few_widen(const FewBlock<FMT> &r, int u, float s)
{
    bf16x2_t p[4];
    if constexpr (FMT == kOutE2M1) {
        // byte 1 of a container holds elements 0 and 1, byte 0 elements 2 and 3
#define MXQ_FEW_FP4(q, sel) __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.v[q][u >> 1], s, sel)
        if (u & 1) {
            p[0] = MXQ_FEW_FP4(0, 3);
            p[1] = MXQ_FEW_FP4(0, 2);
            p[2] = MXQ_FEW_FP4(1, 3);
            p[3] = MXQ_FEW_FP4(1, 2);
        } else {
            p[0] = MXQ_FEW_FP4(0, 1);
            p[1] = MXQ_FEW_FP4(0, 0);
            p[2] = MXQ_FEW_FP4(1, 1);
            p[3] = MXQ_FEW_FP4(1, 0);
        }
#undef MXQ_FEW_FP4
    } else {
#pragma unroll
        for (int q = 0; q < 2; q++) {
            if constexpr (FMT == kOutE4M3FN) {
                p[2 * q] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.v[q][u], s, false);
                p[2 * q + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r.v[q][u], s, true);
            } else {
                p[2 * q] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(r.v[q][u], s, false);
                p[2 * q + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(r.v[q][u], s, true);
            }
        }
    }
    return bf16x8_t{p[0].x, p[0].y, p[1].x, p[1].y, p[2].x, p[2].y, p[3].x, p[3].y};
}

// The left operand: rows of bf16 (IN kInBF16), of f16, or of fp32 kept as two planes of
// bf16 (kInSplit), `plane` values apart.
enum { kInSplit = 2 };

template <int IN> struct FewRows {
    static constexpr int terms = IN == kInBF16 ? 1 : 2;
    static constexpr int loads = IN == kInSplit ? 2 : 1;
};

template <int IN> struct FewLeft {
    u32x4_t v[FewRows<IN>::loads];
};

template <int IN>
__device__ __forceinline__ void few_left(FewLeft<IN> &r, const uint16_t *row, uint64_t plane, uint32_t k)
{
    r.v[0] = *reinterpret_cast<const u32x4_t *>(row + k);
    if constexpr (IN == kInSplit)
        r.v[1] = *reinterpret_cast<const u32x4_t *>(row + plane + k);
}

// Two fp32 values as the bf16 pairs whose sums are nearest to them. (What an infinity
// leaves is a NaN, and the results that it reaches are computed again, see few_exact.)
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &high, uint32_t &low)
{
    high = bf16_pair(a, b);
    low = bf16_pair(a - __uint_as_float(high << 16), b - __uint_as_float(high & 0xFFFF0000u));
}

template <int IN> __device__ __forceinline__ void few_terms(const FewLeft<IN> &r, bf16x8_t (&t)[FewRows<IN>::terms])
{
    if constexpr (IN == kInF16) {
        u32x4_t high, low;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const uint32_t word = r.v[0][k];   // (a bit cast of the element itself takes element 0)
            const f16x2_t p = __builtin_bit_cast(f16x2_t, word);
            uint32_t h, l;
            split_pair((float)p.x, (float)p.y, h, l);
            high[k] = h;
            low[k] = l;
        }
        t[0] = __builtin_bit_cast(bf16x8_t, high);
        t[1] = __builtin_bit_cast(bf16x8_t, low);
    } else {
#pragma unroll
        for (int q = 0; q < FewRows<IN>::loads; q++)
            t[q] = __builtin_bit_cast(bf16x8_t, r.v[q]);
    }
}

// One result with every scale byte at its value (255 is 2^128, which the widening reads as
// NaN): the plain sum in order, in 64 bits, for results that came out not finite.
template <int FMT, int IN>
__device__ __attribute__((noinline)) float few_exact(const uint8_t *data, const uint8_t *scale, uint32_t C,
                                                     uint32_t col, uint32_t K, const uint16_t *row, uint64_t plane)
{
    double sum = 0.0;
    for (uint32_t p = 0; p < K / 4u; p++) {
        const int e = (int)scale[(uint64_t)(p / 8u) * C + col] - 127;
        f32x2_t v[2];
        if constexpr (FMT == kOutE2M1) {
            const uint32_t w = *reinterpret_cast<const uint16_t *>(data + ((uint64_t)p * C + col) * 2u);
            v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
            v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(data + ((uint64_t)p * C + col) * 4u);
            if constexpr (FMT == kOutE4M3FN) {
                v[0] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
                v[1] = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
            } else {
                v[0] = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
                v[1] = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; k++) {
            float x;
            if constexpr (IN == kInF16)
                x = (float)__builtin_bit_cast(_Float16, row[4u * p + k]);
            else
                x = __uint_as_float((uint32_t)row[4u * p + k] << 16);
            if constexpr (IN == kInSplit)
                x += __builtin_isfinite(x) ? __uint_as_float((uint32_t)row[plane + 4u * p + k] << 16) : 0.0f;
            sum += __builtin_ldexp((double)v[k >> 1][k & 1] * x, e);
        }
    }
    return (float)sum;
}

// ----------------------------------------------------------------------------
// The products of one expert's pairs with the columns of a workgroup of NM matrices
// ----------------------------------------------------------------------------

// Blocks in flight, activations and weights alike: loads return in order, so waiting for
// a later block's activations would be waiting for the weights before them.
constexpr int few_depth(int MT) { return MT == 1 ? 4 : MT == 2 ? 3 : 2; }

// MT tiles of 16 pairs from pair `first` on. Wave w takes the MX blocks w, w + waves, .. of the
// contraction and leaves its sums in registers. True where a weight may be too small for
// that (few_low): then few_sums_low has to take them.
template <int FMT, int IN, int NM, int MT>
__device__ __forceinline__ bool few_sums(f32x4_t (&acc)[MT][NM][kFewLaneCols], const __amdgpu_buffer_rsrc_t &data,
                                         const __amdgpu_buffer_rsrc_t &scale, uint32_t C, uint32_t blocks,
                                         const uint32_t (&at_data)[NM], const uint32_t (&at_scale)[NM],
                                         const uint16_t *const (&rows)[MT], uint64_t plane, uint32_t wave, uint32_t waves, uint32_t g)
{
    constexpr int D = few_depth(MT);
    constexpr int terms = FewRows<IN>::terms;
    FewBlock<FMT> w[D][NM];
    FewLeft<IN> x[D][MT];
    const uint32_t n = blocks > wave ? (blocks - wave + waves - 1u) / waves : 0u;
    if (n == 0)
        return false;
    bool low = false;
    const auto fetch = [&](int q, uint32_t s) {
        const uint32_t b = wave + waves * min(s, n - 1u);   // (past the end: the last one again, not used)
#pragma unroll
        for (int t = 0; t < MT; t++)
            few_left<IN>(x[q][t], rows[t], plane, 32u * b + 8u * g);
#pragma unroll
        for (int k = 0; k < NM; k++)
            few_load<FMT>(w[q][k], data, scale, C, b, at_data[k], at_scale[k]);
    };
#pragma unroll
    for (int q = 0; q < D - 1; q++)
        fetch(q, q);
    for (uint32_t s = 0; s < n; s += D)
#pragma unroll
        for (int q = 0; q < D; q++) {
            fetch((q + D - 1) % D, s + q + D - 1);
            __builtin_amdgcn_sched_barrier(0);
            if (s + q < n) {
                bf16x8_t a[MT][terms];
#pragma unroll
                for (int t = 0; t < MT; t++)
                    few_terms<IN>(x[q][t], a[t]);
#pragma unroll
                for (int k = 0; k < NM; k++) {
                    low |= few_low(w[q][k]);
#pragma unroll
                    for (int u = 0; u < kFewLaneCols; u++) {
                        const bf16x8_t b = few_widen<FMT>(w[q][k], u, __uint_as_float(few_exponent(w[q][k], u)));
#pragma unroll
                        for (int t = 0; t < MT; t++)
#pragma unroll
                            for (int e = terms - 1; e >= 0; e--)
                                acc[t][k][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][e], b, acc[t][k][u], 0, 0, 0);
                    }
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    return wave_any(low);
}

// The same sums where weights are below what bf16 holds: a column's weights under a low byte times
// 2^64, and its sum over the block (a result register's column is its lane's) times 2^-64.
template <int FMT, int IN, int NM, int MT>
__device__ __forceinline__ void few_sums_low(f32x4_t (&acc)[MT][NM][kFewLaneCols],
                                             const __amdgpu_buffer_rsrc_t &data, const __amdgpu_buffer_rsrc_t &scale,
                                             uint32_t C, uint32_t blocks, const uint32_t (&at_data)[NM],
                                             const uint32_t (&at_scale)[NM], const uint16_t *const (&rows)[MT],
                                             uint64_t plane, uint32_t wave, uint32_t waves, uint32_t g)
{
    constexpr int terms = FewRows<IN>::terms;
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
        for (int k = 0; k < NM; k++)
#pragma unroll
            for (int u = 0; u < kFewLaneCols; u++)
                acc[t][k][u] = f32x4_t{};
#pragma unroll 1
    for (uint32_t s = wave; s < blocks; s += waves) {
        bf16x8_t a[MT][terms];
#pragma unroll
        for (int t = 0; t < MT; t++) {
            FewLeft<IN> x;
            few_left<IN>(x, rows[t], plane, 32u * s + 8u * g);
            few_terms<IN>(x, a[t]);
        }
#pragma unroll
        for (int k = 0; k < NM; k++) {
            FewBlock<FMT> w;
            few_load<FMT>(w, data, scale, C, s, at_data[k], at_scale[k]);
#pragma unroll
            for (int u = 0; u < kFewLaneCols; u++) {
                const uint32_t e = few_exponent(w, u);
                const bool low = e < kFewLow << 23;
                const bf16x8_t b = few_widen<FMT>(w, u, __uint_as_float(low ? e + (64u << 23) : e));
                const float back = low ? 0x1p-64f : 1.0f;
#pragma unroll
                for (int t = 0; t < MT; t++) {
                    f32x4_t sum = {};
#pragma unroll
                    for (int q = terms - 1; q >= 0; q--)
                        sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][q], b, sum, 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        acc[t][k][u][r] = __builtin_fmaf(sum[r], back, acc[t][k][u][r]);
                }
            }
        }
    }
}

// Two values that a workgroup on another XCD will read in the same launch, and such a read.
// Each XCD has its own L2; accesses at agent scope go past it.
__device__ __forceinline__ void store_shared(float *p, float a, float b)
{
    const uint64_t v = (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
    __hip_atomic_store(reinterpret_cast<uint64_t *>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x2_t load_shared(const float *p)
{
    const uint64_t v =
        __hip_atomic_load(reinterpret_cast<const uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return f32x2_t{__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))};
}

// What a workgroup does with each finished result: stage 1 the activation, stage 2 the
// pair's row of y.
struct FewOut {
    uint16_t *h;         // stage 1: two planes [pairs, F] of bf16
    float *y;            // stage 2: [pairs, N]
    uint64_t plane;      // pairs * F
    uint32_t cols;       // F or N
};

__device__ __forceinline__ float silu(float z) { return z / (1.0f + __expf(-z)); }

template <int FMT, int IN, int NM, int MT>
__device__ __forceinline__ void few_tiles(float (*sums)[NM * 16][64], uint32_t waves, const FewRoute &route, uint32_t first,
                                          uint32_t count, const FewMatrix &m, uint32_t K, const uint16_t *left,
                                          uint32_t slots, uint64_t plane, uint32_t n0, const FewOut &out)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63u, i = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr uint32_t CB = FMT == kOutE2M1 ? 2 : 4;
    constexpr int U = kFewLaneCols;
    const __amdgpu_buffer_rsrc_t data =
        __builtin_amdgcn_make_buffer_rsrc((void *)m.data, (short)0, (int)(K / 4u * CB * m.C), kMmBufferFlags);
    const __amdgpu_buffer_rsrc_t scale =
        __builtin_amdgcn_make_buffer_rsrc((void *)m.scale, (short)0, (int)(K / 32u * m.C), kMmBufferFlags);
    uint32_t at_data[NM], at_scale[NM];
#pragma unroll
    for (int k = 0; k < NM; k++) {
        const uint32_t col = n0 + U * i, c = col + k * out.cols;
        at_data[k] = col < out.cols ? 2u * g * CB * m.C + CB * c : kDropOffset;
        // (where the lane has no column the last ones' scales: a zero would look like a low byte)
        at_scale[k] = min(col, out.cols - U) + k * out.cols;
    }
    // (a tile's rows past the last pair repeat it; their results are not used)
    const uint16_t *rows[MT];
#pragma unroll
    for (int t = 0; t < MT; t++) {
        const uint32_t pair = route.pairs[min(first + 16u * t + i, count - 1u)];
        rows[t] = left + (uint64_t)(IN == kInSplit ? pair : pair / slots) * K;
    }
    f32x4_t acc[MT][NM][U];
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
        for (int k = 0; k < NM; k++)
#pragma unroll
            for (int u = 0; u < U; u++)
                acc[t][k][u] = f32x4_t{};
    if (few_sums<FMT, IN, NM, MT>(acc, data, scale, m.C, K / 32u, at_data, at_scale, rows, plane, wave, waves, g))
        few_sums_low<FMT, IN, NM, MT>(acc, data, scale, m.C, K / 32u, at_data, at_scale, rows, plane, wave, waves, g);

    // 16 pairs at a time, through LDS
#pragma unroll
    for (int t = 0; t < MT; t++) {
        if (first + 16u * t >= count)
            break;
        __syncthreads();     // the last ones' sums have been read
#pragma unroll
        for (int k = 0; k < NM; k++)
#pragma unroll
            for (int u = 0; u < U; u++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    sums[wave][(k * U + u) * 4 + r][lane] = acc[t][k][u][r];
        __syncthreads();
        // two columns at a time
        for (uint32_t at = tid; at < 512u; at += 64u * waves) {
            const uint32_t row = at >> 5, c = 2u * (at & 31u), col = n0 + c;
            if (first + 16u * t + row >= count || col >= out.cols)
                continue;
            const uint32_t pair = route.pairs[first + 16u * t + row];
            float z[NM][2];
#pragma unroll
            for (int k = 0; k < NM; k++)
#pragma unroll
                for (uint32_t q = 0; q < 2; q++) {
                    const uint32_t reg = (k * 4 + (c + q) % 4u) * 4u + (row & 3u);
                    const uint32_t l = 16u * (row >> 2) + (c + q) / 4u;
                    float v = 0.0f;
#pragma unroll
                    for (uint32_t w = 0; w < kFewWaves; w++)
                        v += w < waves ? sums[min(w, waves - 1u)][reg][l] : 0.0f;
                    if (!__builtin_isfinite(v))
                        v = few_exact<FMT, IN>(m.data, m.scale, m.C, col + q + k * out.cols, K,
                                               left + (uint64_t)(IN == kInSplit ? pair : pair / slots) * K, plane);
                    z[k][q] = v;
                }
            const uint64_t o = (uint64_t)pair * out.cols + col;
            if constexpr (IN == kInSplit) {
                store_shared(out.y + o, z[0][0], z[0][1]);
            } else {
                float h[2];
#pragma unroll
                for (int q = 0; q < 2; q++)
                    h[q] = NM == 2 ? silu(z[0][q]) * z[NM - 1][q] : silu(z[0][q]);
                uint32_t high, low;
                split_pair(h[0], h[1], high, low);
                *reinterpret_cast<uint32_t *>(out.h + o) = high;
                *reinterpret_cast<uint32_t *>(out.h + out.plane + o) = low;
            }
        }
    }
}

// All of the expert's pairs, up to 16 MX at a time.
template <int FMT, int IN, int NM, int MX>
__device__ __forceinline__ void few_expert(float (*sums)[NM * 16][64], uint32_t waves, const FewRoute &route, uint32_t count,
                                           const FewMatrix &m, uint32_t K, const uint16_t *left, uint32_t slots,
                                           uint64_t plane, uint32_t n0, const FewOut &out)
{
    for (uint32_t first = 0; first < count; first += 16u * MX) {
        if (MX == 4 && count - first > 32u)
            few_tiles<FMT, IN, NM, MX>(sums, waves, route, first, count, m, K, left, slots, plane, n0, out);
        else if (count - first > 16u)
            few_tiles<FMT, IN, NM, 2>(sums, waves, route, first, count, m, K, left, slots, plane, n0, out);
        else
            few_tiles<FMT, IN, NM, 1>(sums, waves, route, first, count, m, K, left, slots, plane, n0, out);
    }
}

// ----------------------------------------------------------------------------
// The two kernels: a workgroup (of any number of waves up to 8) has an expert in use and 64 columns
// ----------------------------------------------------------------------------

extern __shared__ float few_lds[];   // a wave's sums of 16 pairs, for each wave

// Waves per SIMD that the registers are to leave room for.
constexpr int few_room(int fmt, int NM, int MX) { return MX == 4 || NM == 2 ? 2 : fmt == kOutE2M1 ? 3 : 4; }

template <int FMT, int IN, int ACT, int MX, typename ID>
__global__ __launch_bounds__(kFewThreads, few_room(FMT, ACT == kActSwiglu ? 2 : 1, MX)) void few_up_kernel(
    const uint16_t *__restrict__ x, uint32_t K, const void *__restrict__ ids, uint32_t pairs, uint32_t slots,
    uint32_t experts, const uint8_t *__restrict__ w, const uint8_t *__restrict__ w_scale, uint32_t F, uint32_t tiles,
    uint16_t *__restrict__ h, uint32_t *__restrict__ arrived, uint32_t down_tiles, uint16_t *__restrict__ out_rows,
    uint32_t N)
{
    constexpr int NM = ACT == kActSwiglu ? 2 : 1;
    constexpr uint32_t CB = FMT == kOutE2M1 ? 2 : 4;
    __shared__ FewRoute route;
    // (e2m1's gated sums of 64 pairs do not fit the registers)
    constexpr int MT = NM == 2 && FMT == kOutE2M1 ? 2 : MX;
    const auto sums = reinterpret_cast<float(*)[NM * 16][64]>(few_lds);
    FewPlace at;
    if (few_route<ID>(route, ids, pairs, experts, tiles, at)) {
        const uint32_t C = NM * F;
        const FewMatrix m = {w + (uint64_t)at.expert * (K / 4u) * CB * C,
                             w_scale + (uint64_t)at.expert * (K / 32u) * C, C};
        const FewOut out = {h, nullptr, (uint64_t)pairs * F, F};
        few_expert<FMT, IN, NM, MT>(sums, blockDim.x / 64u, route, at.count, m, K, x, slots, 0, at.tile * kFewCols,
                                    out);
    }
    // for the second kernel: each token's count of pairs that have an expert, up to zero in
    // every column tile; a token without any gets its zeros
    const uint32_t lane = threadIdx.x & 63u, tokens = pairs / slots;
    for (uint32_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        const ID e = reinterpret_cast<const ID *>(ids)[t * slots + min(lane, slots - 1u)];
        const uint32_t has =
            (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(lane < slots && e >= 0 && (uint64_t)e < experts));
        for (uint32_t k = threadIdx.x; k < down_tiles; k += blockDim.x)
            arrived[k * tokens + t] = 0u - has;
        if (has == 0)
            for (uint32_t c = 4u * threadIdx.x; c < N; c += 4u * blockDim.x)
                *reinterpret_cast<u32x2_t *>(out_rows + (uint64_t)t * N + c) = u32x2_t{0u, 0u};
    }
}

// A workgroup that has written its columns of its pairs' rows of y says so for each pair's
// token, and adds up the slots of the tokens that are complete with that, in slot order:
// the sums do not depend on the order of arrival. No workgroup waits for another.
//
// What orders a row of y before its reader, which may be on another XCD: rows are written and
// read by agent-scope atomics (store_shared), which go past the XCD's L2 to memory that all
// share, so neither an L2 that still holds a row back nor one that holds an old one is in
// between. A wave counts a store in vmcnt until memory has acknowledged it; each waits for
// that count to be zero, then for the barrier, and only then one of them adds to the counter,
// itself an agent-scope atomic. The reader's loads are issued behind a barrier that follows
// the counter's answer. That is the target's rule for such accesses, and not HIP's memory
// model, which would have a release before the counter and an acquire behind it: these also write
// back, and drop, everything else in an L2, each time (16 x 4 pairs, 32 experts of e4m3fn, 4096 ->
// 2048 -> 4096, the whole layer: 115 us; with the release 333, with both 340; with ordinary
// stores and fences this kernel alone 440).
template <int FMT, int IN, int MX, typename ID>
__global__ __launch_bounds__(kFewThreads, few_room(FMT, 1, MX)) void few_down_kernel(
    const uint16_t *__restrict__ h, uint32_t F, const void *__restrict__ ids, uint32_t pairs, uint32_t slots,
    uint32_t experts, const uint8_t *__restrict__ w, const uint8_t *__restrict__ w_scale, uint32_t N, uint32_t tiles,
    float *y, uint32_t *arrived, const float *__restrict__ weights, uint16_t *__restrict__ out)
{
    constexpr uint32_t CB = FMT == kOutE2M1 ? 2 : 4;
    __shared__ FewRoute route;
    __shared__ uint32_t complete;
    const auto sums = reinterpret_cast<float(*)[16][64]>(few_lds);
    FewPlace at;
    if (!few_route<ID>(route, ids, pairs, experts, tiles, at))
        return;
    const uint32_t n0 = at.tile * kFewCols;
    const FewMatrix m = {w + (uint64_t)at.expert * (F / 4u) * CB * N, w_scale + (uint64_t)at.expert * (F / 32u) * N, N};
    const FewOut o = {nullptr, y, 0, N};
    few_expert<FMT, kInSplit, 1, MX>(sums, blockDim.x / 64u, route, at.count, m, F, h, slots, (uint64_t)pairs * F, n0,
                                     o);
    const ID *id = reinterpret_cast<const ID *>(ids);
    if (threadIdx.x == 0)
        complete = 0;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    for (uint32_t k = threadIdx.x; k < at.count; k += blockDim.x) {
        const uint32_t t = route.pairs[k] / slots;
        const uint32_t before = __hip_atomic_fetch_add(&arrived[at.tile * (pairs / slots) + t], 1u, __ATOMIC_RELAXED,
                                                       __HIP_MEMORY_SCOPE_AGENT);
        if (before + 1u == 0u)       // (the sums have been read: their memory holds the list)
            reinterpret_cast<uint16_t *>(few_lds)[atomicAdd(&complete, 1u)] = (uint16_t)t;
    }
    __syncthreads();
    const uint32_t tokens = complete;
    // two columns of two of them at a time, and eight slots' reads of each (one by one, each
    // read waits for the one before)
    constexpr uint32_t half = kFewCols / 2u;
    const uint32_t items = tokens * half;
    for (uint32_t q0 = threadIdx.x; q0 < items; q0 += 2u * blockDim.x) {
        uint32_t t[2], col[2];
        float sum[2][2] = {};
#pragma unroll
        for (uint32_t k = 0; k < 2; k++) {
            const uint32_t q = min(q0 + k * blockDim.x, items - 1u);
            t[k] = reinterpret_cast<const uint16_t *>(few_lds)[q / half];
            col[k] = min(n0 + 2u * (q % half), N - 2u);
        }
        for (uint32_t j0 = 0; j0 < slots; j0 += 8u) {
            f32x2_t v[2][8];
            float wt[2][8];
            bool in[2][8];
#pragma unroll
            for (uint32_t k = 0; k < 2; k++)
#pragma unroll
                for (uint32_t j = 0; j < 8; j++) {
                    const uint32_t p = t[k] * slots + min(j0 + j, slots - 1u);
                    const ID e = id[p];
                    in[k][j] = j0 + j < slots && e >= 0 && (uint64_t)e < experts;
                    wt[k][j] = weights[p];
                    v[k][j] = load_shared(y + (uint64_t)p * N + col[k]);
                }
#pragma unroll
            for (uint32_t k = 0; k < 2; k++)
#pragma unroll
                for (uint32_t j = 0; j < 8; j++)
                    if (in[k][j]) {
                        sum[k][0] = __builtin_fmaf(wt[k][j], v[k][j].x, sum[k][0]);
                        sum[k][1] = __builtin_fmaf(wt[k][j], v[k][j].y, sum[k][1]);
                    }
        }
#pragma unroll
        for (uint32_t k = 0; k < 2; k++) {
            // (an item past the last repeats it, a column past the last the last two)
            uint32_t bits;
            if constexpr (IN == kInBF16)
                bits = bf16_pair(sum[k][0], sum[k][1]);
            else
                bits = __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)sum[k][0], (_Float16)sum[k][1]});
            *reinterpret_cast<uint32_t *>(out + (uint64_t)t[k] * N + col[k]) = bits;
        }
    }
}

} // namespace mxq
