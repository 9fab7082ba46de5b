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
// expert that is in use, and the pairs that chose it, from the ids themselves (up to 1024,
// in a few hundred cycles, and all workgroups at the same time).
//
// The activations stay as they come: weights are widened to bf16 in registers, which is
// exact for every code (3 fraction bits at most) and scale byte but the rarest
// (values below 2^-133 round, and 255 is below), and the products run on the bf16 matrix
// cores with fp32 sums. An f16 x is the sum of two bf16 numbers exactly; what is
// between the two products (fp32) is kept as two bf16 numbers, 16 bits of it.
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
constexpr uint32_t kFewWaves = 8;        // waves that share the contraction
constexpr uint32_t kFewThreads = 64 * kFewWaves;
constexpr uint32_t kFewCols = 64;        // columns of a workgroup: 16 lanes x 4
constexpr int kFewU = 4;

// ----------------------------------------------------------------------------
// Which expert, which pairs
// ----------------------------------------------------------------------------

struct FewRoute {
    uint32_t mask[32];                   // experts in use
    uint32_t counts[kFewPairs / 64];     // pairs of this workgroup's expert per 64 ids
    uint16_t pairs[kFewPairs];
};

// The `a`-th expert in use (in order of its number): its number and its count of
// pairs, which are then in route.pairs in order; `active` experts are in use. False where
// there is no a-th one. Every thread of the workgroup takes part.
template <typename ID>
__device__ __forceinline__ bool few_route(FewRoute &route, const void *ids_, uint32_t n, uint32_t experts, uint32_t a,
                                          uint32_t &expert, uint32_t &count, uint32_t &active)
{
    const ID *ids = reinterpret_cast<const ID *>(ids_);
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    constexpr uint32_t per = kFewPairs / kFewThreads;
    if (tid < 32u)
        route.mask[tid] = 0;
    __syncthreads();
    uint32_t mine[per];
#pragma unroll
    for (uint32_t q = 0; q < per; q++) {
        const uint32_t p = q * kFewThreads + tid;
        mine[q] = 0xFFFFFFFFu;
        if (p < n) {
            const ID id = ids[p];
            if (id >= 0 && (uint64_t)id < experts) {
                mine[q] = (uint32_t)id;
                atomicOr(&route.mask[mine[q] >> 5], 1u << (mine[q] & 31u));
            }
        }
    }
    __syncthreads();
    // lane l < 32 scans the bits of word l
    const uint32_t word = lane < 32u ? route.mask[lane] : 0u;
    uint32_t before = __popc(word);
    const uint32_t own = before;
#pragma unroll
    for (uint32_t d = 1; d < 32; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)before, d);
        before += lane >= d ? o : 0u;
    }
    active = (uint32_t)__builtin_amdgcn_readlane((int)before, 31);
    before -= own;
    if (a >= active)
        return false;
    // the lane whose word holds the a-th bit
    uint32_t bit = 0;
    const bool here = lane < 32u && a >= before && a < before + own;
    if (here) {
        uint32_t w = word;
        for (uint32_t k = a - before; k > 0; k--)
            w &= w - 1u;
        bit = 32u * lane + (uint32_t)__builtin_ctz(w);
    }
    const uint32_t at = (uint32_t)__builtin_ctzll(__builtin_amdgcn_ballot_w64(here));
    expert = (uint32_t)__builtin_amdgcn_readlane((int)bit, (int)at);
    uint64_t match[per];
#pragma unroll
    for (uint32_t q = 0; q < per; q++) {
        match[q] = __builtin_amdgcn_ballot_w64(mine[q] == expert);
        if (lane == 0)
            route.counts[q * kFewWaves + wave] = (uint32_t)__popcll(match[q]);
    }
    __syncthreads();
    count = 0;
    uint32_t first[per];
#pragma unroll
    for (uint32_t c = 0; c < kFewPairs / 64u; c++) {
#pragma unroll
        for (uint32_t q = 0; q < per; q++)
            if (c == q * kFewWaves + wave)
                first[q] = count;
        count += route.counts[c];
    }
#pragma unroll
    for (uint32_t q = 0; q < per; q++)
        if (mine[q] == expert)
            route.pairs[first[q] + (uint32_t)__popcll(match[q] & ((1ull << lane) - 1ull))] =
                (uint16_t)(q * kFewThreads + tid);
    __syncthreads();
    count = (uint32_t)__builtin_amdgcn_readfirstlane((int)count);
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
    static constexpr int dwords = FMT == kOutE2M1 ? 2 : 4;
    uint32_t v[2][dwords];   // containers of view rows 2 g and 2 g + 1, four columns
    uint32_t scale;          // E8M0 of the four columns
};

// Block b, columns col .. col + 3 (an offset past every buffer where the lane has none).
template <int FMT>
__device__ __forceinline__ void few_load(FewBlock<FMT> &r, const __amdgpu_buffer_rsrc_t &data,
                                         const __amdgpu_buffer_rsrc_t &scale, uint32_t C, uint32_t b, uint32_t at_data,
                                         uint32_t at_scale)
{
    constexpr uint32_t CB = FMT == kOutE2M1 ? 2 : 4;
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const uint32_t row = (8u * b + q) * CB * C;
        if constexpr (FMT == kOutE2M1) {
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

// Column u's 8 values times their scale, as bf16.
template <int FMT> __device__ __forceinline__ bf16x8_t few_widen(const FewBlock<FMT> &r, int u)
{
    const float s = __uint_as_float((u < 3 ? r.scale << (23 - 8 * u) : r.scale >> 1) & 0x7F800000u);
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

// Two fp32 values as the bf16 pairs whose sums are nearest to them.
__device__ __forceinline__ void split_pair(float a, float b, uint32_t &high, uint32_t &low)
{
    high = bf16_pair(a, b);
    const float ha = __uint_as_float(high << 16), hb = __uint_as_float(high & 0xFFFF0000u);
    // (an infinity has no second part)
    low = bf16_pair(__builtin_isfinite(ha) ? a - ha : 0.0f, __builtin_isfinite(hb) ? b - hb : 0.0f);
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
                x += __uint_as_float((uint32_t)row[plane + 4u * p + k] << 16);
            sum += __builtin_ldexp((double)v[k >> 1][k & 1] * x, e);
        }
    }
    return (float)sum;
}

// ----------------------------------------------------------------------------
// The products of one expert's pairs with 64 columns of NM matrices
// ----------------------------------------------------------------------------

// MT tiles of 16 pairs from pair `first` on. Wave w takes the MX blocks w, w + 8, .. of the
// contraction, `DEPTH` of them in flight, and leaves its sums in registers.
template <int FMT, int IN, int NM, int MT>
__device__ __forceinline__ void few_sums(f32x4_t (&acc)[MT][NM][kFewU], const __amdgpu_buffer_rsrc_t &data,
                                         const __amdgpu_buffer_rsrc_t &scale, uint32_t C, uint32_t blocks,
                                         const uint32_t (&at_data)[NM], const uint32_t (&at_scale)[NM],
                                         const uint16_t *const (&rows)[MT], uint64_t plane, uint32_t wave, uint32_t g)
{
    constexpr int DEPTH = MT == 4 ? 2 : 4;
    constexpr int terms = FewRows<IN>::terms;
    FewBlock<FMT> w[DEPTH][NM];
    FewLeft<IN> x[DEPTH][MT];
    const uint32_t n = blocks > wave ? (blocks - wave + kFewWaves - 1) / kFewWaves : 0u;
    if (n == 0)
        return;
    const auto fetch = [&](int q, uint32_t s) {
        const uint32_t b = wave + kFewWaves * min(s, n - 1u);   // (past the end: the last one again, not used)
#pragma unroll
        for (int k = 0; k < NM; k++)
            few_load<FMT>(w[q][k], data, scale, C, b, at_data[k], at_scale[k]);
#pragma unroll
        for (int t = 0; t < MT; t++)
            few_left<IN>(x[q][t], rows[t], plane, 32u * b + 8u * g);
    };
#pragma unroll
    for (int q = 0; q < DEPTH - 1; q++)
        fetch(q, q);
    for (uint32_t s = 0; s < n; s += DEPTH)
#pragma unroll
        for (int q = 0; q < DEPTH; q++) {
            fetch((q + DEPTH - 1) % DEPTH, s + q + DEPTH - 1);
            __builtin_amdgcn_sched_barrier(0);
            if (s + q < n) {
                bf16x8_t a[MT][terms];
#pragma unroll
                for (int t = 0; t < MT; t++)
                    few_terms<IN>(x[q][t], a[t]);
#pragma unroll
                for (int k = 0; k < NM; k++)
#pragma unroll
                    for (int u = 0; u < kFewU; u++) {
                        const bf16x8_t b = few_widen<FMT>(w[q][k], u);
#pragma unroll
                        for (int t = 0; t < MT; t++)
#pragma unroll
                            for (int e = terms - 1; e >= 0; e--)
                                acc[t][k][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[t][e], b, acc[t][k][u], 0, 0, 0);
                    }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
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
__device__ __forceinline__ void few_tiles(float (*sums)[NM * kFewU * 4][64], const FewRoute &route, uint32_t first,
                                          uint32_t count, const FewMatrix &m, uint32_t K, const uint16_t *left,
                                          uint32_t slots, uint64_t plane, uint32_t n0, const FewOut &out)
{
    const uint32_t tid = threadIdx.x, lane = tid & 63u, i = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr uint32_t CB = FMT == kOutE2M1 ? 2 : 4;
    const __amdgpu_buffer_rsrc_t data =
        __builtin_amdgcn_make_buffer_rsrc((void *)m.data, (short)0, (int)(K / 4u * CB * m.C), kMmBufferFlags);
    const __amdgpu_buffer_rsrc_t scale =
        __builtin_amdgcn_make_buffer_rsrc((void *)m.scale, (short)0, (int)(K / 32u * m.C), kMmBufferFlags);
    uint32_t at_data[NM], at_scale[NM];
#pragma unroll
    for (int k = 0; k < NM; k++) {
        const uint32_t col = n0 + 4u * i, c = col + k * out.cols;
        at_data[k] = col < out.cols ? 2u * g * CB * m.C + CB * c : kDropOffset;
        at_scale[k] = col < out.cols ? c : kDropOffset;
    }
    // (a tile's rows past the last pair repeat it; their results are not used)
    const uint16_t *rows[MT];
#pragma unroll
    for (int t = 0; t < MT; t++) {
        const uint32_t pair = route.pairs[min(first + 16u * t + i, count - 1u)];
        rows[t] = left + (uint64_t)(IN == kInSplit ? pair : pair / slots) * K;
    }
    f32x4_t acc[MT][NM][kFewU];
#pragma unroll
    for (int t = 0; t < MT; t++)
#pragma unroll
        for (int k = 0; k < NM; k++)
#pragma unroll
            for (int u = 0; u < kFewU; u++)
                acc[t][k][u] = f32x4_t{};
    few_sums<FMT, IN, NM, MT>(acc, data, scale, m.C, K / 32u, at_data, at_scale, rows, plane, wave, g);

#pragma unroll
    for (int t = 0; t < MT; t++) {
        if (first + 16u * t >= count)
            break;
        __syncthreads();     // the last tile's sums have been read
#pragma unroll
        for (int k = 0; k < NM; k++)
#pragma unroll
            for (int u = 0; u < kFewU; u++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    sums[wave][(k * kFewU + u) * 4 + r][lane] = acc[t][k][u][r];
        __syncthreads();
        // 16 rows x 64 columns, two columns a thread
        const uint32_t row = tid >> 5, c = 2u * (tid & 31u), col = n0 + c;
        if (first + 16u * t + row >= count || col >= out.cols)
            continue;
        const uint32_t pair = route.pairs[first + 16u * t + row];
        float z[NM][2];
#pragma unroll
        for (int k = 0; k < NM; k++)
#pragma unroll
            for (uint32_t q = 0; q < 2; q++) {
                const uint32_t reg = (k * kFewU + (c + q) % 4u) * 4u + (row & 3u), l = 16u * (row >> 2) + (c + q) / 4u;
                float v = sums[0][reg][l];
#pragma unroll
                for (uint32_t w = 1; w < kFewWaves; w++)
                    v += sums[w][reg][l];
                if (!__builtin_isfinite(v))
                    v = few_exact<FMT, IN>(m.data, m.scale, m.C, col + q + k * out.cols, K,
                                           left + (uint64_t)(IN == kInSplit ? pair : pair / slots) * K, plane);
                z[k][q] = v;
            }
        const uint64_t o = (uint64_t)pair * out.cols + col;
        if constexpr (IN == kInSplit) {
            *reinterpret_cast<float2 *>(out.y + o) = float2{z[0][0], z[0][1]};
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

template <int FMT, int IN, int NM>
__device__ __forceinline__ void few_expert(float (*sums)[NM * kFewU * 4][64], const FewRoute &route, uint32_t count,
                                           const FewMatrix &m, uint32_t K, const uint16_t *left, uint32_t slots,
                                           uint64_t plane, uint32_t n0, const FewOut &out)
{
    uint32_t first = 0;
    for (; count - first > 32u; first += 64u) {
        few_tiles<FMT, IN, NM, 4>(sums, route, first, count, m, K, left, slots, plane, n0, out);
        if (count - first <= 64u)
            return;
    }
    if (count - first > 16u)
        few_tiles<FMT, IN, NM, 2>(sums, route, first, count, m, K, left, slots, plane, n0, out);
    else
        few_tiles<FMT, IN, NM, 1>(sums, route, first, count, m, K, left, slots, plane, n0, out);
}

// ----------------------------------------------------------------------------
// The two kernels: workgroup (a, tile) has the a-th expert in use and 64 columns
// ----------------------------------------------------------------------------

template <int FMT, int IN, int ACT, typename ID>
__global__ __launch_bounds__(kFewThreads) void few_up_kernel(
    const uint16_t *__restrict__ x, uint32_t K, const void *__restrict__ ids, uint32_t pairs, uint32_t slots,
    uint32_t experts, const uint8_t *__restrict__ w, const uint8_t *__restrict__ w_scale, uint32_t F, uint32_t tiles,
    uint16_t *__restrict__ h, uint32_t *__restrict__ arrived, uint32_t arrivals)
{
    constexpr int NM = ACT == kActSwiglu ? 2 : 1;
    constexpr uint32_t CB = FMT == kOutE2M1 ? 2 : 4;
    __shared__ FewRoute route;
    __shared__ float sums[kFewWaves][NM * kFewU * 4][64];
    const uint32_t a = blockIdx.x / tiles, tile = blockIdx.x - a * tiles;
    // the second kernel's counters
    if (blockIdx.x == 0)
        for (uint32_t k = threadIdx.x; k < arrivals; k += kFewThreads)
            arrived[k] = 0;
    uint32_t expert, count, active;
    if (!few_route<ID>(route, ids, pairs, experts, a, expert, count, active))
        return;
    const uint32_t C = NM * F;
    const FewMatrix m = {w + (uint64_t)expert * (K / 4u) * CB * C, w_scale + (uint64_t)expert * (K / 32u) * C, C};
    const FewOut out = {h, nullptr, (uint64_t)pairs * F, F};
    few_expert<FMT, IN, NM>(sums, route, count, m, K, x, slots, 0, tile * kFewCols, out);
}

// The workgroup that is the last of its columns' adds up the pairs' rows in slot
// order. Arrivals only say that the others' rows are written; the sums do not depend on
// their order.
template <int FMT, int IN, typename ID>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(
    const uint16_t *__restrict__ h, uint32_t F, const void *__restrict__ ids, uint32_t pairs, uint32_t slots,
    uint32_t experts, const uint8_t *__restrict__ w, const uint8_t *__restrict__ w_scale, uint32_t N, uint32_t tiles,
    float *y, uint32_t *arrived, const float *__restrict__ weights, uint16_t *__restrict__ out)
{
    constexpr uint32_t CB = FMT == kOutE2M1 ? 2 : 4;
    __shared__ FewRoute route;
    __shared__ float sums[kFewWaves][kFewU * 4][64];
    __shared__ uint32_t last;
    const uint32_t a = blockIdx.x / tiles, tile = blockIdx.x - a * tiles;
    const uint32_t n0 = tile * kFewCols;
    uint32_t expert, count, active = 0;
    if (few_route<ID>(route, ids, pairs, experts, a, expert, count, active)) {
        const FewMatrix m = {w + (uint64_t)expert * (F / 4u) * CB * N, w_scale + (uint64_t)expert * (F / 32u) * N, N};
        const FewOut o = {nullptr, y, 0, N};
        few_expert<FMT, kInSplit, 1>(sums, route, count, m, F, h, slots, (uint64_t)pairs * F, n0, o);
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0)
            last = atomicAdd(&arrived[tile], 1u) == active - 1u ? 1u : 0u;
        __syncthreads();
        if (!last)
            return;
        __threadfence();
    } else if (a > 0 || active > 0) {
        return;
    }
    // (no expert in use: the first workgroup of the columns writes zeros)
    const ID *id = reinterpret_cast<const ID *>(ids);
    const uint32_t tokens = pairs / slots;
    for (uint32_t q = threadIdx.x; q < tokens * (kFewCols / 2u); q += kFewThreads) {
        const uint32_t t = q / (kFewCols / 2u), col = n0 + 2u * (q % (kFewCols / 2u));
        if (col >= N)
            continue;
        float sum[2] = {0.0f, 0.0f};
        for (uint32_t j = 0; j < slots; j++) {
            const uint32_t p = t * slots + j;
            if (id[p] >= 0 && (uint64_t)id[p] < experts) {
                const float2 v = *reinterpret_cast<const float2 *>(y + (uint64_t)p * N + col);
                sum[0] = __builtin_fmaf(weights[p], v.x, sum[0]);
                sum[1] = __builtin_fmaf(weights[p], v.y, sum[1]);
            }
        }
        uint32_t bits;
        if constexpr (IN == kInBF16)
            bits = bf16_pair(sum[0], sum[1]);
        else
            bits = __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)sum[0], (_Float16)sum[1]});
        *reinterpret_cast<uint32_t *>(out + (uint64_t)t * N + col) = bits;
    }
}

} // namespace mxq
