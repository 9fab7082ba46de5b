// mxq_fp4_kernels.hpp -- gfx950 products with e2m1 weights.
//
//     out[r][n] = sum over k < 4P of L[k][r] * R_g[k][n] for r in group g
// (one group of all rows, or the groups of a plan's offsets as in
// mxq_grouped_kernels.hpp), X[k][c] = decode(q) * 2^(E8M0 - 127), fp32 sums of
// the matrix cores. R is e2m1; L is e2m1, e4m3fn or e5m2.
//
// Operand layout is the quantize's: row p of an operand holds, for each of its
// C columns, the container of elements 4p .. 4p + 3: four bytes of FP8, or 16 bits
// of e2m1 whose nibbles are, from the lowest on, elements 2, 3, 0, 1.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 (lane layout measured on gfx950): lane
// l = i + 32 h supplies 32 of the 64 values of row (column) i.
//   e2m1: nibble n (0 .. 31, four registers) is k = 32 h + n, so half h holds MX
//         block h of the step: containers 8 h .. 8 h + 7.
//   FP8:  byte b (0 .. 31, eight registers) is k = 16 h + b below 16 and
//         32 + 16 h + (b - 16) from there on: containers 4 h .. 4 h + 3 of block 0,
//         then of block 1.
// Half h's scale byte is block h's in both. The lane order inside an e2m1
// container is another permutation of its four k than FP8's: two e2m1 operands
// agree as they are; beside FP8 the container's bytes are swapped.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_grouped_kernels.hpp"

namespace mxq {

template <> struct MfmaFmt<kOutE2M1> { static constexpr int value = 4; };

template <int FMT> struct Container { static constexpr uint32_t bytes = FMT == kOutE2M1 ? 2 : 4; };

template <uint32_t CB>
__device__ __forceinline__ MmSource fp4_source(const uint8_t *data, const uint8_t *scale, uint32_t C, uint32_t c0)
{
    MmSource s;
    s.pitch = CB * C;
    s.data = data + (uint64_t)CB * c0;
    s.scale = scale + c0;
    s.C = C;
    s.scale_cols = C - c0;
    s.col_bytes = CB * c0;
    return s;
}

// First scale row of the aligned MX blocks from `block` on (a multiple of 2 or 4):
// the image keeps four block rows together, so they are adjacent in both layouts.
__device__ __forceinline__ uint64_t scale_row(uint32_t block, uint32_t dense)
{
    return dense ? block : (block & 3u) + 32ull * (block >> 2);
}

// This workgroup's tile; without offsets all rows are one group.
template <uint32_t TILE, uint32_t COLS, uint32_t WALK, uint32_t ES>
__device__ __forceinline__ bool fp4_job(GroupedJob &job, const int32_t *offsets, uint32_t groups, uint32_t M,
                                        uint32_t N, uint32_t tiles_n, uint32_t lane)
{
    if (offsets)
        return rows_job<TILE, COLS, WALK, ES, 2u>(job, offsets, groups, M, N, tiles_n, lane);
    const uint32_t t = xcd_tile(blockIdx.x, gridDim.x);
    const uint32_t tiles_m = (M + TILE - 1) / TILE;
    const uint32_t walk = t / (WALK * tiles_n);
    const uint32_t rows = min(WALK, tiles_m - walk * WALK);
    const uint32_t in_walk = t - walk * WALK * tiles_n;
    const uint32_t col = in_walk / rows;
    job.m0 = (walk * WALK + in_walk - col * rows) * TILE;
    job.n0 = col * COLS;
    job.row_end = M;
    job.one_tile = M <= TILE;
    return true;
}

// ----------------------------------------------------------------------------
// Operands straight from memory to registers
// ----------------------------------------------------------------------------

// 32 rows x 32 U columns of a step: A container m0 + i, B containers n0 + U i + u.
template <int LF, int U> struct Fp4Raw {
    uint32_t a[8];
    uint32_t b[8][U / 2];   // two containers per register
    uint32_t as, bs;        // byte u of bs: B sub-tile u
};

// K step `step`, or zeros without any access to memory where step >= end. NT: the
// weights with the non-temporal hint.
template <int LF, int U, int NT>
__device__ __forceinline__ void fp4_load(Fp4Raw<LF, U> &r, const MmSource &sa, const MmSource &sb, uint32_t P,
                                         uint32_t step, uint32_t end, uint32_t dense, uint32_t i, uint32_t h)
{
    static_assert(U == 2 || U == 4, "4 or 8 bytes per lane and row");
    const bool in = step < end;
    step = in ? step : 0u;
    const uint32_t nrows = in ? min(P - step * kMmStepRows, kMmStepRows) : 0u;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sa.data + (uint64_t)step * kMmStepRows * sa.pitch), (short)0,
        in ? (int)(nrows * sa.pitch - sa.col_bytes) : 0, kMmBufferFlags);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sb.data + (uint64_t)step * kMmStepRows * sb.pitch), (short)0,
        in ? (int)(nrows * sb.pitch - sb.col_bytes) : 0, kMmBufferFlags);
    const uint32_t vb = 8u * h * sb.pitch + 2u * U * i;
#pragma unroll
    for (uint32_t v = 0; v < 8; v++) {
        if constexpr (U == 4) {
            const u32x2_t w = __builtin_amdgcn_raw_buffer_load_b64(rb, vb, v * sb.pitch, NT ? kBufferNT : 0);
            r.b[v][0] = w.x;
            r.b[v][1] = w.y;
        } else {
            r.b[v][0] = __builtin_amdgcn_raw_buffer_load_b32(rb, vb, v * sb.pitch, NT ? kBufferNT : 0);
        }
    }
    if constexpr (LF == kOutE2M1) {
        const uint32_t va = 8u * h * sa.pitch + 2u * i;
#pragma unroll
        for (uint32_t v = 0; v < 8; v++)
            r.a[v] = __builtin_amdgcn_raw_buffer_load_b16(ra, va, v * sa.pitch, 0);
    } else {
        const uint32_t va = 4u * h * sa.pitch + 4u * i;
#pragma unroll
        for (uint32_t v = 0; v < 8; v++)
            r.a[v] = __builtin_amdgcn_raw_buffer_load_b32(ra, va, ((v < 4 ? 0u : 8u) + (v & 3u)) * sa.pitch, 0);
    }
    // the step's blocks 2 step and 2 step + 1: lane half h's is the second row
    const uint64_t srow = scale_row(2u * step, dense);
    const __amdgpu_buffer_rsrc_t qa = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sa.scale + srow * sa.C), (short)0, in ? (int)(nrows / 8u * sa.C - (sa.C - sa.scale_cols)) : 0,
        kMmBufferFlags);
    const __amdgpu_buffer_rsrc_t qb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sb.scale + srow * sb.C), (short)0, in ? (int)(nrows / 8u * sb.C - (sb.C - sb.scale_cols)) : 0,
        kMmBufferFlags);
    r.as = __builtin_amdgcn_raw_buffer_load_b8(qa, h * sa.C + i, 0, 0);
    if constexpr (U == 4)
        r.bs = __builtin_amdgcn_raw_buffer_load_b32(qb, h * sb.C + 4u * i, 0, 0);
    else
        r.bs = __builtin_amdgcn_raw_buffer_load_b16(qb, h * sb.C + 2u * i, 0, 0);
}

template <int LF, int U> __device__ __forceinline__ i32x8_t fp4_a(const Fp4Raw<LF, U> &r)
{
    if constexpr (LF == kOutE2M1)
        return i32x8_t{(int)__builtin_amdgcn_perm(r.a[1], r.a[0], 0x05040100u),
                       (int)__builtin_amdgcn_perm(r.a[3], r.a[2], 0x05040100u),
                       (int)__builtin_amdgcn_perm(r.a[5], r.a[4], 0x05040100u),
                       (int)__builtin_amdgcn_perm(r.a[7], r.a[6], 0x05040100u), 0, 0, 0, 0};
    else
        return i32x8_t{(int)r.a[0], (int)r.a[1], (int)r.a[2], (int)r.a[3],
                       (int)r.a[4], (int)r.a[5], (int)r.a[6], (int)r.a[7]};
}

// B sub-tile u: the containers of rows 2j and 2j + 1 side by side in register j,
// their bytes swapped beside FP8.
template <int LF, int U> __device__ __forceinline__ i32x8_t fp4_b(const Fp4Raw<LF, U> &r, int u)
{
    constexpr uint32_t low = LF == kOutE2M1 ? 0x05040100u : 0x04050001u;
    constexpr uint32_t high = LF == kOutE2M1 ? 0x07060302u : 0x06070203u;
    i32x8_t o = {};
#pragma unroll
    for (int j = 0; j < 4; j++)
        o[j] = (int)__builtin_amdgcn_perm(r.b[2 * j + 1][u >> 1], r.b[2 * j][u >> 1], u & 1 ? high : low);
    return o;
}

template <int F, int SEL>
__device__ __forceinline__ f32x16_t fp4_mfma(const i32x8_t &a, const i32x8_t &b, const f32x16_t &acc, uint32_t as,
                                             uint32_t bs)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, F, 4, 0, (int)as, SEL, (int)bs);
}

template <int LF, int U>
__device__ __forceinline__ void fp4_products(f32x16_t (&acc)[U], const Fp4Raw<LF, U> &r)
{
    constexpr int F = MfmaFmt<LF>::value;
    const i32x8_t a = fp4_a(r);
    acc[0] = fp4_mfma<F, 0>(a, fp4_b(r, 0), acc[0], r.as, r.bs);
    acc[1] = fp4_mfma<F, 1>(a, fp4_b(r, 1), acc[1], r.as, r.bs);
    if constexpr (U == 4) {
        acc[2] = fp4_mfma<F, 2>(a, fp4_b(r, 2), acc[2], r.as, r.bs);
        acc[3] = fp4_mfma<F, 3>(a, fp4_b(r, 3), acc[3], r.as, r.bs);
    }
}

// ----------------------------------------------------------------------------
// Scale bytes of 255
// ----------------------------------------------------------------------------

// The values of the blocks whose scale byte is 255 (`own`: of this lane's scale, the
// block of its half), the others zeroed. FP8 halves hold parts of both blocks.
template <int FMT> __device__ __forceinline__ i32x8_t fp4_keep_255(const i32x8_t &v, bool own, uint32_t h)
{
    if constexpr (FMT == kOutE2M1) {
        i32x8_t o = {};
#pragma unroll
        for (int k = 0; k < 4; k++)
            o[k] = own ? v[k] : 0;
        return o;
    } else {
        const bool other = __shfl_xor((int)own, 32) != 0;
        return mm_keep_blocks(v, h ? other : own, h ? own : other);
    }
}

// The rare path: the results of rows m0 .. and columns n0 .. (up to `rows` and `cols`
// of them, bounded by row_end and N) computed again, 32 x 32 at a time, with every
// E8M0 byte at its value. The matrix cores read 255 as NaN; here it is fed as 254
// (2^127) and each flagged block counted twice per flagged side: (A, B) + (A', B) +
// (A', B') + (A, B') with A' and B' the flagged blocks alone. An infinity of A has its
// products in (A, B); the other three, which would multiply it by zeros too, leave it out.
template <int LF, int EPI>
__device__ __attribute__((noinline)) void fp4_rare_part(const uint8_t *lhs, const uint8_t *lhs_scale,
                                                        const uint8_t *rhs, const uint8_t *rhs_scale, uint32_t P,
                                                        uint32_t M, uint32_t N, uint32_t m0, uint32_t n0,
                                                        uint32_t rows, uint32_t cols, uint32_t row_end, uint32_t dense,
                                                        void *out)
{
    constexpr int F = MfmaFmt<LF>::value;
    const uint32_t lane = __lane_id();
    const uint32_t i = lane & 31u, h = lane >> 5;
    const uint32_t nsteps = (P + kMmStepRows - 1) / kMmStepRows;
    for (uint32_t m = m0; m < min(m0 + rows, row_end); m += 32u)
        for (uint32_t n = n0; n < min(n0 + cols, N); n += 64u) {
            const MmSource sa = fp4_source<Container<LF>::bytes>(lhs, lhs_scale, M, m);
            const MmSource sb = fp4_source<2u>(rhs, rhs_scale, N, n);
            f32x16_t acc[2] = {{}, {}};
            for (uint32_t s = 0; s < nsteps; s++) {
                Fp4Raw<LF, 2> r;
                fp4_load<LF, 2, 0>(r, sa, sb, P, s, nsteps, dense, i, h);
                const i32x8_t a = fp4_a(r), fa = mm_finite_codes<F>(a);
                const i32x8_t ta = fp4_keep_255<LF>(fa, r.as == 255u, h);
                const uint32_t as = min(r.as, 254u);
#pragma unroll
                for (int u = 0; u < 2; u++) {
                    const uint32_t byte = (r.bs >> (8 * u)) & 0xFFu, bs = min(byte, 254u);
                    const i32x8_t b = fp4_b(r, u), tb = fp4_keep_255<kOutE2M1>(b, byte == 255u, h);
                    acc[u] = fp4_mfma<F, 0>(a, b, acc[u], as, bs);
                    acc[u] = fp4_mfma<F, 0>(ta, b, acc[u], as, bs);
                    acc[u] = fp4_mfma<F, 0>(ta, tb, acc[u], as, bs);
                    acc[u] = fp4_mfma<F, 0>(fa, tb, acc[u], as, bs);
                }
            }
#pragma unroll
            for (int q = 0; q < 16; q++) {
                const uint32_t row = m + 8u * (q >> 2) + 4u * h + (q & 3), col = n + 2u * i;
                if (row >= row_end || col >= N)
                    continue;
                const uint64_t o = (uint64_t)row * N + col;
                if constexpr (EPI == kEpiF32)
                    *reinterpret_cast<float2 *>(reinterpret_cast<float *>(out) + o) = float2{acc[0][q], acc[1][q]};
                else
                    *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(out) + o) =
                        bf16_pair(acc[0][q], acc[1][q]);
            }
        }
}

// ----------------------------------------------------------------------------
// Few rows per group, or few tiles: the weights stream through registers
// ----------------------------------------------------------------------------
//
// As in grouped_stream_kernel: a workgroup of CW * KW waves computes 32 rows x 32 U CW
// columns; KW waves share the K steps of a set of columns and add their sums
// through LDS in wave order. A row of 32 lanes reads 64 U contiguous bytes; 16-bit
// containers of two rows are put side by side by one byte permute per register.
//
// Bound by the weights' bytes with many groups (64 groups of 32 rows, 4096 x 2048, e4m3fn:
// 51 us, 5.9 TB/s), and by the latency of a launch and of the first loads for one small
// product (16 x 4096 x 4096: 9.5 us with 32 x 64 tiles of eight waves, 21 with 32 x 256).

// K steps s0 .. s1 - 1, kFp4Ahead of them in flight.
constexpr int kFp4Ahead = 3;
template <int LF, int U, int NT>
__device__ __forceinline__ void fp4_steps(f32x16_t (&acc)[U], const MmSource &sa, const MmSource &sb, uint32_t P,
                                          uint32_t s0, uint32_t s1, uint32_t dense, uint32_t i, uint32_t h)
{
    Fp4Raw<LF, U> r[kFp4Ahead + 1];
#pragma unroll
    for (int q = 0; q < kFp4Ahead; q++)
        fp4_load<LF, U, NT>(r[q], sa, sb, P, s0 + q, s1, dense, i, h);
    for (uint32_t s = s0; s < s1; s += kFp4Ahead + 1)
#pragma unroll
        for (int q = 0; q <= kFp4Ahead; q++) {
            fp4_load<LF, U, NT>(r[(q + kFp4Ahead) % (kFp4Ahead + 1)], sa, sb, P, s + q + kFp4Ahead, s1, dense, i, h);
            __builtin_amdgcn_sched_barrier(0);
            fp4_products<LF, U>(acc, r[q]);
            __builtin_amdgcn_sched_barrier(0);
        }
}

template <int LF, int EPI, int U, int CW, int KW>
__global__ __launch_bounds__(64 * CW * KW, 2) void fp4_stream_kernel(
    const uint8_t *__restrict__ lhs, const uint8_t *__restrict__ lhs_scale, const uint8_t *__restrict__ rhs,
    const uint8_t *__restrict__ rhs_scale, const int32_t *__restrict__ offsets, uint32_t groups, uint32_t P,
    uint32_t M, uint32_t N, uint32_t tiles_n, uint32_t dense, void *__restrict__ out)
{
    constexpr uint32_t RW = 16 / KW;   // result registers each wave adds up
    constexpr uint32_t COLS = 32u * U;
    __shared__ __attribute__((aligned(16))) float sums[CW][KW][16][64][U];
    __shared__ uint32_t rare[CW];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t cw = wave % CW, kw = wave / CW;
    const uint32_t i = lane & 31u, h = lane >> 5;

    GroupedJob job = {lhs, lhs_scale, rhs, rhs_scale, (uint8_t *)out, P, 0, 0, 0, false};
    if (!fp4_job<kStreamRows, CW * COLS, 1, EPI == kEpiF32 ? 4 : 2>(job, offsets, groups, M, N, tiles_n, lane))
        return;
    const uint32_t n0 = job.n0 + cw * COLS;
    const MmSource sa = fp4_source<Container<LF>::bytes>(job.lhs, job.lhs_scale, M, job.m0);
    const MmSource sb = fp4_source<2u>(job.rhs, job.rhs_scale, N, n0);
    if (threadIdx.x < CW)
        rare[threadIdx.x] = 0;

    f32x16_t acc[U];
#pragma unroll
    for (int u = 0; u < U; u++)
        acc[u] = f32x16_t{};
    // (a wave past the last column takes no step)
    const uint32_t nsteps = n0 < N ? (P + kMmStepRows - 1) / kMmStepRows : 0u;
    const uint32_t per = (nsteps + KW - 1) / KW;
    const uint32_t s0 = min(kw * per, nsteps), s1 = min(s0 + per, nsteps);
    // weights that are read once go past the caches
    if (job.one_tile)
        fp4_steps<LF, U, 1>(acc, sa, sb, P, s0, s1, dense, i, h);
    else
        fp4_steps<LF, U, 0>(acc, sa, sb, P, s0, s1, dense, i, h);

#pragma unroll
    for (int r = 0; r < 16; r++)
#pragma unroll
        for (int u = 0; u < U; u++)
            sums[cw][kw][r][lane][u] = acc[u][r];
    __syncthreads();
    float v[RW][U];
    bool finite = true;
#pragma unroll
    for (uint32_t k = 0; k < RW; k++) {
        const uint32_t r = kw * RW + k;
        const bool in = job.m0 + 8u * (r >> 2) + 4u * h + (r & 3u) < job.row_end;
#pragma unroll
        for (int u = 0; u < U; u++) {
            float x = sums[cw][0][r][lane][u];
#pragma unroll
            for (int w = 1; w < KW; w++)
                x += sums[cw][w][r][lane][u];
            v[k][u] = x;
            finite = finite && (__builtin_isfinite(x) || !in || n0 + U * i >= N);
        }
    }
    if (wave_any(!finite) && lane == 0)
        atomicOr(&rare[cw], 1u);
    __syncthreads();
    if (__builtin_amdgcn_readfirstlane(rare[cw]) != 0) {
        if (kw == 0)
            fp4_rare_part<LF, EPI>(job.lhs, job.lhs_scale, job.rhs, job.rhs_scale, P, M, N, job.m0, n0, kStreamRows,
                                   COLS, job.row_end, dense, job.out);
        return;
    }
    constexpr uint32_t ES = EPI == kEpiF32 ? 4 : 2;
    const bool lines = whole_lines<EPI>(N);
#pragma unroll
    for (uint32_t k = 0; k < RW; k++) {
        const uint32_t r = kw * RW + k, m = job.m0 + 8u * (r >> 2) + (r & 3u);
        if constexpr (U == 4) {
            if (lines)
                grouped_store<EPI, 4, 1>(v[k], m, h, job.row_end, n0 + 4u * i, N, job.out);
            else
                grouped_store<EPI, 4, 0>(v[k], m, h, job.row_end, n0 + 4u * i, N, job.out);
        } else {
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                job.out + (uint64_t)m * N * ES, (short)0, (int)(kDropOffset - 1u), kMmBufferFlags);
            const uint32_t col = n0 + 2u * i;
            const uint32_t at = m + 4u * h < job.row_end && col < N ? (4u * h * N + col) * ES : kDropOffset;
            if constexpr (EPI == kEpiF32)
                __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{__float_as_uint(v[k][0]), __float_as_uint(v[k][1])}, rs,
                                                      (int)at, 0, 0);
            else
                __builtin_amdgcn_raw_buffer_store_b32(bf16_pair(v[k][0], v[k][1]), rs, (int)at, 0, 0);
        }
    }
}

// ----------------------------------------------------------------------------
// Many rows: square tiles through LDS
// ----------------------------------------------------------------------------
//
// Four waves, one per SIMD of a CU, each a square of (32 FR)^2 results of a tile of
// T = 64 FR: 256 x 256 (FR = 4) or 128 x 128 (FR = 2). Per K step of 64 a wave reads 2 FR
// operands for FR^2 MFMAs, half as many per MFMA as the FP8 product's 64 x 128 waves, and
// an e2m1 operand is half the bytes.
//
// An e2m1 operand comes out of LDS transposed by the read itself:
// ds_read_b64_tr_b16 takes, per 16 lanes, four rows of 16 containers and gives each lane
// four containers of one column, so two reads are a lane's 32 values, in the
// registers that the MFMA wants. FP8 containers are 32 bits: a lane reads its column's
// dword of each row. E8M0 bytes of one operand come by ds_read_b64_tr_b8, which gives
// each lane its column's bytes of the step pair's blocks: byte t is K step t's, picked by
// op_sel.
//
// LDS holds a stage (two K steps, 32 operand rows) row by row as the copies
// (buffer_load_dwordx4 ... lds) land it: 1 KiB each, 16 bytes a lane. Which 16-byte chunk
// a lane fetches is free, and is chosen so that the four rows (and two adjacent
// 16-column groups) of a transposing read, or the two halves of an FP8 read, lie in
// different banks: see fp4_chunk and fp8_chunk.
//
// The weights are the A operand, so that a lane holds four adjacent columns of
// one result row; the results go through LDS once to leave in whole lines.
//
// Operands of a step are read while the products before it run, each wave's reads spread
// over its products, and copies are two or more stages ahead, so that one barrier a stage is
// all that waits. 8192 x 8192 x 8192 takes 279 us in e2m1 by e2m1 (3.94 PFLOP/s; 297 with the
// reads bunched) and 421 us in e4m3fn by e2m1 (2.61 PFLOP/s): with FP8 the matrix
// instructions take twice as long, and an operand 8 LDS reads in place of 4.

constexpr int kTileThreads = 256;
constexpr uint32_t kTileRows = 32;   // operand rows per stage

// Where chunk c of row p of an e2m1 operand lies in its row, and back. Rows 0..3 differ in
// bits 1 and 2 (the lowest bank bits of 32-byte pieces), columns 16 apart in bit 3.
__device__ __forceinline__ uint32_t fp4_chunk(uint32_t c, uint32_t p)
{
    return c ^ (2u * (p & 3u)) ^ (8u * ((c >> 1) & 1u));
}
__device__ __forceinline__ uint32_t fp4_chunk_at(uint32_t at, uint32_t p)
{
    const uint32_t c = at ^ (2u * (p & 3u));
    return c ^ (8u * ((c >> 1) & 1u));
}
// FP8: the two lane halves read rows whose quads are odd and even.
__device__ __forceinline__ uint32_t fp8_chunk(uint32_t c, uint32_t p) { return c ^ (8u * ((p >> 2) & 1u)); }

template <int LF, int FR> struct TileLayout {
    static constexpr uint32_t T = 64u * FR;
    static constexpr uint32_t rowL = T * Container<LF>::bytes, rowR = T * 2u;
    static constexpr uint32_t offR = kTileRows * rowL, offSL = offR + kTileRows * rowR, offSR = offSL + 4u * T;
    static constexpr uint32_t stage = offSR + 4u * T;
    static constexpr int stages = FR == 4 && LF == kOutE2M1 ? 4 : 3;
    // copies per wave and stage: operand rows, then scale rows
    static constexpr int copies = (int)(kTileRows * (rowL + rowR) / 4096u + 8u * T / 1024u);
    static constexpr uint32_t bytes = stages * stage;
    static constexpr uint32_t pitch = 32u * FR * 4u + 16u;    // a wave's result row in LDS
    static_assert(4u * 32u * pitch <= bytes, "the results' rows fit the stages");
};

// A wave's 8 operand rows 8 w .. 8 w + 7 of a stage. P is a multiple of 8: all of them are
// in the operand, or none.
template <int FMT, uint32_t ROW>
__device__ __forceinline__ void tile_copy_rows(const MmSource &s, uint8_t *dst, uint32_t P, uint32_t row0, uint32_t w,
                                               uint32_t lane)
{
    constexpr uint32_t per = 1024u / ROW, lanes = ROW / 16u;   // rows per copy, lanes per row
    // (past the operand the range is empty, whatever the address)
    const uint32_t p0 = row0 + 8u * w;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(s.data + (uint64_t)p0 * s.pitch), (short)0, p0 < P ? (int)(8u * s.pitch - s.col_bytes) : 0,
        kMmBufferFlags);
    const uint32_t row = lane / lanes, at = lane % lanes;
#pragma unroll
    for (uint32_t j = 0; j < 8u / per; j++) {
        const uint32_t p = per * j + row;
        const uint32_t c = FMT == kOutE2M1 ? fp4_chunk_at(at, p) : fp8_chunk(at, p);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)(dst + (8u * w + per * j) * ROW), 16,
                                                 row * s.pitch + 16u * c, per * j * s.pitch, 0, 0);
    }
}

// T / 64 scale rows each 4 bytes a lane: unit u of 4 (T = 256) or 2 (T = 128).
template <uint32_t T>
__device__ __forceinline__ void tile_copy_scale(const MmSource &s, uint8_t *dst, uint32_t P, uint32_t block,
                                                uint32_t dense, uint32_t u, uint32_t lane)
{
    constexpr uint32_t per = 256u / T, lanes = T / 4u;
    // (all uniform; said so, or the address is built in vector registers)
    const uint32_t blocks = P / 8u, left = block < blocks ? blocks - block : 0u;
    const uint32_t bytes = left > 0u ? min(left, 4u) * s.C - (s.C - s.scale_cols) : 0u;
    const uint64_t at = scale_row(block, dense) * s.C;
    const uint64_t p = (uint64_t)(uintptr_t)s.scale + at;
    const uint32_t low = __builtin_amdgcn_readfirstlane((uint32_t)p);
    const uint32_t high = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(uintptr_t)((uint64_t)high << 32 | low), (short)0, (int)__builtin_amdgcn_readfirstlane(bytes),
        kMmBufferFlags);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)(dst + 256u * u), 4,
                                             (lane / lanes) * s.C + 4u * (lane % lanes), per * u * s.C, 0, 0);
}

template <int LF, int FR>
__device__ __forceinline__ void tile_copy(const MmSource &sl, const MmSource &sr, uint8_t *__restrict__ st, uint32_t P,
                                          uint32_t stage, uint32_t dense, uint32_t w, uint32_t lane)
{
    typedef TileLayout<LF, FR> L;
    tile_copy_rows<LF, L::rowL>(sl, st, P, stage * kTileRows, w, lane);
    tile_copy_rows<kOutE2M1, L::rowR>(sr, st + L::offR, P, stage * kTileRows, w, lane);
    if constexpr (FR == 4) {
        tile_copy_scale<L::T>(sl, st + L::offSL, P, 4u * stage, dense, w, lane);
        tile_copy_scale<L::T>(sr, st + L::offSR, P, 4u * stage, dense, w, lane);
    } else {
        const bool left = w < 2u;
        tile_copy_scale<L::T>(left ? sl : sr, st + (left ? L::offSL : L::offSR), P, 4u * stage, dense, w & 1u, lane);
    }
}

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x2_t read_tr16(const uint8_t *p)
{
    return __builtin_bit_cast(
        i32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_t *)(p)));
}
__device__ __forceinline__ i32x2_t read_tr8(const uint8_t *p)
{
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2_t *)(p));
}

// One K step's operands of a wave.
template <int FR> struct TileOps {
    i32x8_t l[FR], r[FR];
};

// Lane-constant LDS offsets of the reads.
template <int FR> struct TileLane {
    uint32_t l[FR], r[FR];   // operand sub-tile, K step 0
    uint32_t sl, sr;         // scales of sub-tile 0
};

template <int FMT, int FR> __device__ __forceinline__ void tile_offsets(uint32_t (&o)[FR], uint32_t part, uint32_t lane)
{
    constexpr uint32_t row = 64u * FR * Container<FMT>::bytes;
    const uint32_t i = lane & 31u, h = lane >> 5;
#pragma unroll
    for (uint32_t f = 0; f < FR; f++) {
        const uint32_t c0 = 32u * (FR * part + f);    // the sub-tile's first column
        if constexpr (FMT == kOutE2M1) {
            const uint32_t L = i & 15u;
            const uint32_t chunk = c0 / 8u + 2u * (i >> 4) + ((L & 3u) >> 1);
            o[f] = (8u * h + (L >> 2)) * row + 16u * fp4_chunk(chunk, L >> 2) + 8u * (L & 1u);
        } else {
            o[f] = 4u * h * row + 16u * fp8_chunk(c0 / 4u + (i >> 2), 4u * h) + 4u * (i & 3u);
        }
    }
}

// Sub-tile operand of K step t (compile-time): e2m1 containers 8 h .. 8 h + 7 of the step.
template <int FMT, uint32_t ROW>
__device__ __forceinline__ i32x8_t tile_read(const uint8_t *p, uint32_t t)
{
    if constexpr (FMT == kOutE2M1) {
        const i32x2_t a = read_tr16(p + 16u * t * ROW), b = read_tr16(p + (16u * t + 4u) * ROW);
        return i32x8_t{a.x, a.y, b.x, b.y, 0, 0, 0, 0};
    } else {
        i32x8_t o;
#pragma unroll
        for (int v = 0; v < 8; v++)
            o[v] = *reinterpret_cast<const int *>(p + (16u * t + (v < 4 ? 0u : 8u) + (v & 3)) * ROW);
        return o;
    }
}

// A K step's operands, and a stage's scales. (The stage pointers here and in tile_copy are
// restrict: without that the compiler takes a read for one of what a copy in flight
// writes, and waits for all copies in front of it.)
template <int LF, int FR>
__device__ __forceinline__ void tile_read_step(const uint8_t *__restrict__ st, const TileLane<FR> &at, uint32_t t,
                                               TileOps<FR> &x)
{
    typedef TileLayout<LF, FR> L;
#pragma unroll
    for (int f = 0; f < FR; f++) {
        x.r[f] = tile_read<kOutE2M1, L::rowR>(st + L::offR + at.r[f], t);
        x.l[f] = tile_read<LF, L::rowL>(st + at.l[f], t);
    }
}

template <int FR>
__device__ __forceinline__ void tile_read_scales(const uint8_t *__restrict__ st, const TileLane<FR> &at,
                                                 uint32_t (&cl)[FR], uint32_t (&cr)[FR])
{
#pragma unroll
    for (int f = 0; f < FR; f++) {
        cl[f] = (uint32_t)read_tr8(st + at.sl + 32u * f).x;
        cr[f] = (uint32_t)read_tr8(st + at.sr + 32u * f).x;
    }
}

// The order of what stands before it, to the last scheduling barrier: a few reads behind
// each product, so that the matrix cores never wait for their issue.
template <int PRODUCTS, int READS> __device__ __forceinline__ void tile_interleave()
{
#pragma unroll
    for (int k = 0; k < PRODUCTS; k++) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, (READS + PRODUCTS - 1) / PRODUCTS, 0);
    }
}

// The sums so far are issued before anything below.
template <int FR> __device__ __forceinline__ void tile_pin(f32x16_t (&acc)[FR][FR])
{
#pragma unroll
    for (int b = 0; b < FR; b++)
#pragma unroll
        for (int a = 0; a < FR; a++)
            if constexpr (FR == 4)      // (in the registers that the sums of a 256-row tile fill)
                asm volatile("" : "+a"(acc[b][a]));
            else
                asm volatile("" : "+v"(acc[b][a]));
}

template <int LF, int FR, int T>
__device__ __forceinline__ void tile_products(f32x16_t (&acc)[FR][FR], const TileOps<FR> &x, const uint32_t (&sl)[FR],
                                              const uint32_t (&sr)[FR])
{
    constexpr int F = MfmaFmt<LF>::value;
#pragma unroll
    for (int b = 0; b < FR; b++) {
        i32x8_t r = x.r[b];
        if constexpr (LF != kOutE2M1)
#pragma unroll
            for (int k = 0; k < 4; k++)     // the bytes of each container swapped
                r[k] = (int)__builtin_amdgcn_perm((uint32_t)r[k], (uint32_t)r[k], 0x02030001u);
#pragma unroll
        for (int a = 0; a < FR; a++)
            acc[b][a] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(r, x.l[a], acc[b][a], 4, F, T, (int)sr[b], T,
                                                                        (int)sl[a]);
    }
}

template <int LF, int EPI, int FR>
__global__ __launch_bounds__(kTileThreads, FR == 4 ? 1 : 2) void fp4_tile_kernel(
    const uint8_t *__restrict__ lhs, const uint8_t *__restrict__ lhs_scale, const uint8_t *__restrict__ rhs,
    const uint8_t *__restrict__ rhs_scale, const int32_t *__restrict__ offsets, uint32_t groups, uint32_t P,
    uint32_t M, uint32_t N, uint32_t tiles_n, uint32_t dense, void *__restrict__ out)
{
    typedef TileLayout<LF, FR> L;
    constexpr uint32_t ES = EPI == kEpiF32 ? 4 : 2;
    __shared__ __attribute__((aligned(16))) uint8_t lds[L::bytes];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t i = lane & 31u, h = lane >> 5;
    const uint32_t wl = wave & 1u, wr = wave >> 1;

    GroupedJob job = {lhs, lhs_scale, rhs, rhs_scale, (uint8_t *)out, P, 0, 0, 0, false};
    if (!fp4_job<L::T, L::T, FR == 4 ? 4 : 8, ES>(job, offsets, groups, M, N, tiles_n, lane))
        return;
    const MmSource sl = fp4_source<Container<LF>::bytes>(job.lhs, job.lhs_scale, M, job.m0);
    const MmSource sr = fp4_source<2u>(job.rhs, job.rhs_scale, N, job.n0);

    TileLane<FR> at;
    tile_offsets<LF, FR>(at.l, wl, lane);
    tile_offsets<kOutE2M1, FR>(at.r, wr, lane);
    // a lane pair's scale row: blocks h and 2 + h of the stage, 8 columns per lane
    const uint32_t srow = (h + (i & 2u)) * L::T + 16u * (i >> 4) + 8u * (i & 1u);
    at.sl = L::offSL + srow + 32u * FR * wl;
    at.sr = L::offSR + srow + 32u * FR * wr;

    f32x16_t acc[FR][FR];
#pragma unroll
    for (int b = 0; b < FR; b++)
#pragma unroll
        for (int a = 0; a < FR; a++)
            acc[b][a] = f32x16_t{};

    const uint32_t n = (P + kTileRows - 1) / kTileRows;
#pragma unroll
    for (uint32_t s = 0; s < L::stages - 1; s++)
        tile_copy<LF, FR>(sl, sr, lds + s * L::stage, P, s, dense, wave, lane);
    __builtin_amdgcn_s_waitcnt(mm_wait_vm((L::stages - 2) * L::copies));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);

    constexpr int reads = FR * (LF == kOutE2M1 ? 4 : 6);    // instructions of a step's operands
    TileOps<FR> x, y;
    uint32_t cl[FR], cr[FR], dl[FR], dr[FR];
    tile_read_step<LF, FR>(lds, at, 0, x);
    tile_read_scales<FR>(lds, at, cl, cr);
    uint32_t cur = 0;
    for (uint32_t s = 0; s < n; s++) {
        // step 1's reads, the copies of a later stage into the stage before this one, which
        // every wave has read, and step 0's products
        const uint32_t fre = cur == 0 ? L::stages - 1 : cur - 1u;
        const uint32_t nxt = cur == L::stages - 1 ? 0u : cur + 1u;
        __builtin_amdgcn_sched_barrier(0);
        tile_read_step<LF, FR>(lds + cur * L::stage, at, 1, y);
        tile_copy<LF, FR>(sl, sr, lds + fre * L::stage, P, s + L::stages - 1, dense, wave, lane);
        tile_products<LF, FR, 0>(acc, x, cl, cr);
        tile_pin(acc);
        __builtin_amdgcn_sched_barrier(0);
        // my reads of this stage and my copies of the next one are through; after the
        // barrier everyone's are
        __builtin_amdgcn_s_waitcnt(mm_wait_vm_lgkm((L::stages - 2) * L::copies));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        // step 1's products; behind them the next stage's first reads
        tile_read_step<LF, FR>(lds + nxt * L::stage, at, 0, x);
        tile_read_scales<FR>(lds + nxt * L::stage, at, dl, dr);
        tile_products<LF, FR, 1>(acc, y, cl, cr);
        tile_interleave<FR * FR, reads + 2 * FR>();
        tile_pin(acc);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < FR; f++) {
            cl[f] = dl[f];
            cr[f] = dr[f];
        }
        cur = nxt;
    }
    // no copy may land in the LDS that the results take, nor any wave still read there
    __builtin_amdgcn_s_waitcnt(mm_wait_vm_lgkm(0));
    __builtin_amdgcn_s_barrier();

    const uint32_t m0 = job.m0 + 32u * FR * wl, n0 = job.n0 + 32u * FR * wr;
    if (m0 >= job.row_end || n0 >= N)
        return;
    float zero[FR] = {};
#pragma unroll
    for (int b = 0; b < FR; b++)
#pragma unroll
        for (int a = 0; a < FR; a++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                zero[a] = __builtin_fmaf(acc[b][a][r], 0.0f, zero[a]);
    float all = zero[0];
#pragma unroll
    for (int a = 1; a < FR; a++)
        all += zero[a];
    if (wave_any(!(all == 0.0f))) {
        fp4_rare_part<LF, EPI>(job.lhs, job.lhs_scale, job.rhs, job.rhs_scale, P, M, N, m0, n0, 32u * FR, 32u * FR,
                               job.row_end, dense, job.out);
        return;
    }
    // 32 result rows at a time through this wave's own part of LDS
    uint8_t *mine = lds + wave * 32u * L::pitch;
    typedef uint32_t u32x4_8_t __attribute__((ext_vector_type(4), aligned(8)));
    constexpr uint32_t vec = 16u / ES, lanes = 32u * FR / vec, step = 64u / lanes;   // lanes per row, rows per store
#pragma unroll
    for (int a = 0; a < FR; a++) {
#pragma unroll
        for (int b = 0; b < FR; b++)
#pragma unroll
            for (int q = 0; q < 4; q++) {
                uint8_t *p = mine + i * L::pitch + (32u * b + 8u * q + 4u * h) * ES;
                const f32x16_t &v = acc[b][a];
                if constexpr (EPI == kEpiF32)
                    *reinterpret_cast<float4 *>(p) = float4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                else
                    *reinterpret_cast<uint2 *>(p) = uint2{bf16_pair(v[4 * q], v[4 * q + 1]),
                                                          bf16_pair(v[4 * q + 2], v[4 * q + 3])};
            }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const uint32_t col = n0 + vec * (lane % lanes);
#pragma unroll
        for (uint32_t k = 0; k < 32u / step; k++) {
            const uint32_t row = step * k + lane / lanes, m = m0 + 32u * a + row;
            const u32x4_t v = *reinterpret_cast<const u32x4_t *>(mine + row * L::pitch + 16u * (lane % lanes));
            if (m < job.row_end) {
                uint8_t *p = job.out + ((uint64_t)m * N + col) * ES;
                if (col + vec <= N)
                    *reinterpret_cast<u32x4_8_t *>(p) = u32x4_8_t{v[0], v[1], v[2], v[3]};
                else if (EPI != kEpiF32 && col + 4u <= N)
                    *reinterpret_cast<u32x2_t *>(p) = u32x2_t{v[0], v[1]};
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

} // namespace mxq
