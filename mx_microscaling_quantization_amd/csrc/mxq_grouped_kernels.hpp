// mxq_grouped_kernels.hpp -- gfx950 products of the experts of a
// mixture-of-experts layer: MX operands whose columns (the sorted rows of the
// tokens) fall into groups, one per expert.
//
// Operand layout and arithmetic are the scaled matmul's
// (mxq_matmul_kernels.hpp): X[k][c] = decode(q) * 2^(E8M0 - 127), fp32 sums of
// the matrix cores, which add the products of one 32-value block in fixed
// point with about 13 fraction bits below the largest of them. With group g
// the columns offsets[g] .. offsets[g + 1] - 1:
//   rows:   out[r][n]    = sum over k of L[k][r] * R_g[k][n] for r in group g,
//           zero for the rows of no group (before the first one, past the last)
//   wgrad:  out[g][m][n] = sum over k in group g of L[k][m] * R[k][n]
//           (the sorted rows are the contraction: groups of whole MX blocks)
//
// Group sizes are known only on the device, so a launch has as many
// workgroups as any grouping of R rows needs, and each finds its tile from
// the offsets. Nothing read or written depends on offsets being sensible:
// they are clamped to 0 .. R, and no group ends before it starts.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_matmul_kernels.hpp"

namespace mxq {

// ----------------------------------------------------------------------------
// From a tile's number to its group
// ----------------------------------------------------------------------------

struct GroupTile {
    uint32_t group;     // `groups`: the rows past the last group
    uint32_t m0, end;   // the tile's first row, the group's end
    uint32_t first;     // the group's first row
};

__device__ __forceinline__ void group_bounds(const int32_t *offsets, uint32_t groups, uint32_t R, uint32_t g,
                                             uint32_t &first, uint32_t &end)
{
    const int32_t a = offsets[g], b = g < groups ? offsets[g + 1] : (int32_t)R;
    first = min((uint32_t)max(a, 0), R);
    end = max(min((uint32_t)max(b, 0), R), first);
}

// Every wave looks its tile up by itself: lane l adds up the row tiles of
// `per` consecutive groups (the rows past the last one count as a group), a
// scan over the lanes gives each lane's first tile and the number of tiles.
struct GroupScan {
    uint32_t per, first;    // groups per lane; this lane's first row tile
    uint32_t real;          // row tiles of the groups
    uint32_t total;         // the same with those past the last group
};

template <uint32_t TILE>
__device__ __forceinline__ GroupScan group_scan(const int32_t *offsets, uint32_t groups, uint32_t R, uint32_t lane)
{
    GroupScan s;
    s.per = groups / 64u + 1u;
    uint32_t n = 0;
    for (uint32_t q = 0; q < s.per; q++) {
        const uint32_t g = lane * s.per + q;
        if (g <= groups) {
            uint32_t a, b;
            group_bounds(offsets, groups, R, g, a, b);
            n += (b - a + TILE - 1) / TILE;
        }
    }
    uint32_t v = n;
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)v, d);
        v += lane >= d ? o : 0u;
    }
    s.first = v - n;
    s.total = (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
    uint32_t a, b;
    group_bounds(offsets, groups, R, groups, a, b);
    s.real = s.total - (uint32_t)__builtin_amdgcn_readfirstlane((int)((b - a + TILE - 1) / TILE));
    return s;
}

// Row tile `tile` (< total).
template <uint32_t TILE>
__device__ __forceinline__ GroupTile group_find(const int32_t *offsets, uint32_t groups, uint32_t R,
                                                const GroupScan &s, uint32_t tile)
{
    const uint32_t l = (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(s.first <= tile)) - 1u;
    uint32_t left = tile - (uint32_t)__builtin_amdgcn_readlane((int)s.first, (int)l);
    GroupTile t = {groups, R, R, R};
    for (uint32_t q = 0; q < s.per; q++) {
        const uint32_t g = l * s.per + q;
        if (g > groups)
            break;
        uint32_t a, b;
        group_bounds(offsets, groups, R, g, a, b);
        const uint32_t n = (b - a + TILE - 1) / TILE;
        if (left < n) {
            t = {g, a + left * TILE, b, a};
            break;
        }
        left -= n;
    }
    t.group = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.group);
    t.m0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.m0);
    t.end = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.end);
    t.first = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.first);
    return t;
}

// Number of workgroup w among `n` tiles such that XCD w % 8 gets consecutive
// ones; >= n for a workgroup without a tile. The launch may have more
// workgroups than tiles: what is spread evenly are the tiles there are.
__device__ __forceinline__ uint32_t xcd_tile(uint32_t w, uint32_t n)
{
    const uint32_t q = n / kMmXcds;
    if (w / kMmXcds < q)
        return (w % kMmXcds) * q + w / kMmXcds;
    return w;   // the tail: w >= 8 q, in place
}

// The 8-byte aligned `bytes` at p (a multiple of 8), share `index` of `count`
// of them by this workgroup's threads, as zeros.
__device__ __forceinline__ void zero_share(uint8_t *p, uint64_t bytes, uint32_t index, uint32_t count)
{
    typedef uint32_t u32x4_8_t __attribute__((ext_vector_type(4), aligned(8)));
    const uint64_t units = bytes / 16u;
    const uint64_t end = units * (index + 1ull) / count;
    for (uint64_t u = units * index / count + threadIdx.x; u < end; u += blockDim.x)
        __builtin_nontemporal_store(u32x4_8_t{0u, 0u, 0u, 0u}, reinterpret_cast<u32x4_8_t *>(p) + u);
    if (index + 1 == count && threadIdx.x == 0 && bytes % 16u != 0)
        *reinterpret_cast<u32x2_t *>(p + bytes - 8u) = u32x2_t{0u, 0u};
}

// A workgroup's tile: operands from their first row on, first output row and
// column, the end of the output's rows.
struct GroupedJob {
    const uint8_t *lhs, *lhs_scale, *rhs, *rhs_scale;
    uint8_t *out;
    uint32_t P, m0, n0, row_end;
    bool one_tile;    // (rows) the group has no other row tile
};

// Rows: the groups' tiles (TILE rows x COLS columns) are walked in sets of WALK
// tile rows column by column, so that the workgroups an XCD runs at a time share
// operand panels. The rows of no group, past the last one or before the first (the
// offsets of some experts of a plan), are cleared by further workgroups,
// which are not part of the XCDs' even shares (64 experts, 62 of them used, x 32
// rows, 4096 x 2048: with them some XCDs got 70 products for their 64 places, 101
// us instead of 81). The launch has at least one tile row of them. False: this
// workgroup has no product. RC: bytes of a container of the weights.
template <uint32_t TILE, uint32_t COLS, uint32_t WALK, uint32_t ES, uint32_t RC = 4>
__device__ __forceinline__ bool rows_job(GroupedJob &job, const int32_t *offsets, uint32_t groups, uint32_t M,
                                         uint32_t N, uint32_t tiles_n, uint32_t lane)
{
    const GroupScan s = group_scan<TILE>(offsets, groups, M, lane);
    const uint32_t real = s.real * tiles_n;
    const uint32_t t = xcd_tile(blockIdx.x, real);
    if (t >= real) {
        uint32_t a, b;
        group_bounds(offsets, groups, M, groups, a, b);
        const uint32_t before = min((uint32_t)max(offsets[0], 0), M);
        const uint32_t tiles = s.total - s.real + (before + TILE - 1) / TILE;
        const uint32_t n = min(tiles * tiles_n, gridDim.x - real);
        if (t - real < n) {
            zero_share(job.out + (uint64_t)a * N * ES, (uint64_t)(b - a) * N * ES, t - real, n);
            zero_share(job.out, (uint64_t)before * N * ES, t - real, n);
        }
        return false;
    }
    const uint32_t walk = t / (WALK * tiles_n);
    const uint32_t rows = min(WALK, s.real - walk * WALK);
    const uint32_t in_walk = t - walk * WALK * tiles_n;
    const uint32_t col = in_walk / rows;
    const GroupTile g = group_find<TILE>(offsets, groups, M, s, walk * WALK + in_walk - col * rows);
    job.m0 = g.m0;
    job.n0 = col * COLS;
    job.row_end = g.end;
    job.one_tile = g.end - g.first <= TILE;
    job.rhs += (uint64_t)g.group * job.P * N * RC;
    job.rhs_scale += (uint64_t)g.group * (job.P / 8u) * N;
    return true;
}

// Wgrad: P operand rows in all, group g's are offsets[g] / 4 .. The tiles of one
// group are spread over the XCDs (each gets consecutive ones), so that a large
// group's work is. An empty group's result is cleared as one run of memory
// instead of tile by tile (20 groups of 3264 x 3932, 18 of them empty: 240 us in
// tiles).
template <uint32_t TILE, uint32_t COLS, uint32_t WALK, uint32_t ES>
__device__ __forceinline__ bool wgrad_job(GroupedJob &job, const int32_t *offsets, uint32_t groups, uint32_t M,
                                          uint32_t N, uint32_t tiles_n)
{
    const uint32_t tiles_m = (M + TILE - 1) / TILE, per = tiles_m * tiles_n;
    const uint32_t g = blockIdx.x / per;
    const uint32_t t = xcd_tile(blockIdx.x - g * per, per);
    uint32_t a, b;
    group_bounds(offsets, groups, 4u * job.P, g, a, b);
    a = __builtin_amdgcn_readfirstlane(a / 32u);   // whole blocks
    b = __builtin_amdgcn_readfirstlane(b / 32u);
    job.out += (uint64_t)g * M * N * ES;
    if (a == b) {
        zero_share(job.out, (uint64_t)M * N * ES, t, per);
        return false;
    }
    const uint32_t walk = t / (WALK * tiles_n);
    const uint32_t rows = min(WALK, tiles_m - walk * WALK);
    const uint32_t in_walk = t - walk * WALK * tiles_n;
    const uint32_t col = in_walk / rows;
    job.m0 = (walk * WALK + in_walk - col * rows) * TILE;
    job.n0 = col * COLS;
    job.row_end = M;
    job.one_tile = false;
    job.lhs += (uint64_t)a * 8u * 4u * M;
    job.lhs_scale += (uint64_t)a * M;
    job.rhs += (uint64_t)a * 8u * 4u * N;
    job.rhs_scale += (uint64_t)a * N;
    job.P = (b - a) * 8u;
    return true;
}

enum { kGroupRows = 0, kGroupWgrad = 1 };

template <int MODE, uint32_t TILE, uint32_t COLS, uint32_t WALK, uint32_t ES>
__device__ __forceinline__ bool grouped_job(GroupedJob &job, const int32_t *offsets, uint32_t groups, uint32_t M,
                                            uint32_t N, uint32_t tiles_n, uint32_t lane)
{
    if constexpr (MODE == kGroupRows)
        return rows_job<TILE, COLS, WALK, ES>(job, offsets, groups, M, N, tiles_n, lane);
    else
        return wgrad_job<TILE, COLS, WALK, ES>(job, offsets, groups, M, N, tiles_n);
}

// ----------------------------------------------------------------------------
// Results
// ----------------------------------------------------------------------------

// Two fp32 values as bf16 bits, rounded to nearest even by the conversion
// instruction (the scaled matmul's own six-instruction rounding, one value at a
// time, took 2 us of a 256 x 256 tile).
__device__ __forceinline__ uint32_t bf16_pair(float a, float b)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t){a, b}, bf16x2_t));
}

// 4 adjacent results per lane: row m + HROWS h (m the same for the wave) from column
// col on; N % 4 == 0. A lane past the group's rows or the columns gives an
// offset that the buffer's range check drops: no branch, so that the stores stay
// in one block (see wave_any).
template <int EPI, uint32_t HROWS, int NT>
__device__ __forceinline__ void grouped_store(const float *v, uint32_t m, uint32_t h, uint32_t row_end, uint32_t col,
                                              uint32_t N, void *__restrict__ out)
{
    constexpr uint32_t ES = EPI == kEpiF32 ? 4 : 2;
    // 8 rows of up to 2^27 bytes stay under the dropped offset
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (uint8_t *)out + (uint64_t)m * N * ES, (short)0, (int)(kDropOffset - 1u), kMmBufferFlags);
    const bool in = m + HROWS * h < row_end && col < N;
    const uint32_t at = in ? (HROWS * h * N + col) * ES : kDropOffset;
    if constexpr (EPI == kEpiF32)
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                                       __float_as_uint(v[2]), __float_as_uint(v[3])},
                                               rs, (int)at, 0, NT ? kBufferNT : 0);
    else
        __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}, rs, (int)at, 0,
                                              NT ? kBufferNT : 0);
}

// Whether rows of N results start on 128-byte lines. Their stores then have the
// non-temporal hint (weight gradients of 2048 x 4096: 277 -> 262 us); otherwise two
// tiles write parts of one line, which the hint keeps the L2 from putting
// together (38 groups of 3296 x 2132: 155 us, 236 with it). The lines' ends still cost
// half as many requests again: 52 groups of 32 rows, 3680 x 1388, 156 us; x 1408, 102.
template <int EPI> __device__ __forceinline__ bool whole_lines(uint32_t N)
{
    return N % (EPI == kEpiF32 ? 32u : 64u) == 0;
}

// Whether a lane's condition holds anywhere in the wave, as a scalar that the
// compiler knows to be one. (A ballot compared with zero it takes for a
// condition per lane, and also a scalar branch with branches per lane inside is
// turned into one side after the other: what one side needs is then kept in
// memory around a call in the other, and the results' stores wait for the
// reloads, that is for each other: 1.5 us of a 256 x 256 tile.)
__device__ __forceinline__ bool wave_any(bool lane_has)
{
    const uint64_t m = __builtin_amdgcn_ballot_w64(lane_has);
    return __builtin_amdgcn_readfirstlane((uint32_t)m | (uint32_t)(m >> 32)) != 0;
}

template <int EPI, int NT>
__device__ __forceinline__ void grouped_store_tile(const f32x16_t (&acc)[2][4], const GroupedJob &job, uint32_t N,
                                                   uint32_t wm0, uint32_t col, uint32_t h)
{
#pragma unroll
    for (int r = 0; r < 16; r++)
#pragma unroll
        for (int a = 0; a < 2; a++) {
            const float v[4] = {acc[a][0][r], acc[a][1][r], acc[a][2][r], acc[a][3][r]};
            grouped_store<EPI, 8, NT>(v, wm0 + 16u * (r >> 2) + 2u * (r & 3) + a, h, job.row_end, col, N, job.out);
        }
}

// A wave's 64 x 128 sums from row wm0 and column wn0. Where one is not finite (a
// scale byte of 255, or a sum that is not by itself) the wave computes its
// part again on the scaled matmul's rare path.
template <int F, int EPI>
__device__ __forceinline__ void grouped_results(const f32x16_t (&acc)[2][4], const GroupedJob &job, uint32_t M,
                                                uint32_t N, uint32_t wm0, uint32_t wn0, uint32_t i, uint32_t h)
{
    // a part past the group's rows or the columns has nothing to store, and its
    // sums times a NaN are no reason for the rare path
    if (wm0 >= job.row_end || wn0 >= N)
        return;
    // 0 times a finite sum is a zero, of anything else a NaN that stays: one
    // instruction per sum, in eight chains (a class test per sum and the scalar
    // logic to collect them took 0.7 us more per tile)
    float zero[8] = {};
#pragma unroll
    for (int a = 0; a < 2; a++)
#pragma unroll
        for (int u = 0; u < 4; u++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                zero[4 * a + u] = __builtin_fmaf(acc[a][u][r], 0.0f, zero[4 * a + u]);
    const float all = ((zero[0] + zero[1]) + (zero[2] + zero[3])) + ((zero[4] + zero[5]) + (zero[6] + zero[7]));
    if (wave_any(!(all == 0.0f))) {
        mm_rare_part<F, EPI>(job.lhs, job.lhs_scale, job.rhs, job.rhs_scale, job.P, M, N, wm0, wn0, 1u, job.out,
                             nullptr, 0, job.row_end);
        return;
    }
    if (whole_lines<EPI>(N))
        grouped_store_tile<EPI, 1>(acc, job, N, wm0, wn0 + 4u * i, h);
    else
        grouped_store_tile<EPI, 0>(acc, job, N, wm0, wn0 + 4u * i, h);
}

// ----------------------------------------------------------------------------
// Long contractions of many rows: the scaled matmul's 256 x 256 tile
// ----------------------------------------------------------------------------

template <int FMT, int EPI, int MODE>
__global__ __launch_bounds__(kMmThreads) void grouped_matmul_kernel(
    const uint8_t *__restrict__ lhs, const uint8_t *__restrict__ lhs_scale, const uint8_t *__restrict__ rhs,
    const uint8_t *__restrict__ rhs_scale, const int32_t *__restrict__ offsets, uint32_t groups, uint32_t P,
    uint32_t M, uint32_t N, uint32_t tiles_n, void *__restrict__ out)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[kMmStages * kMmStageBytes + kMmSpareBytes];
    constexpr int F = MfmaFmt<FMT>::value;
    constexpr uint32_t ES = EPI == kEpiF32 ? 4 : 2;
    const uint32_t tid = threadIdx.x;
    const uint32_t lane = tid & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t grp = wave >> 2, wq = wave & 3u;

    GroupedJob job = {lhs, lhs_scale, rhs, rhs_scale, (uint8_t *)out, P, 0, 0, 0, false};
    if (!grouped_job<MODE, kMmTile, kMmTile, kMmGroupRows, ES>(job, offsets, groups, M, N, tiles_n, lane))
        return;
    MmSource src;
    mm_source(src, grp ? job.rhs : job.lhs, grp ? job.rhs_scale : job.lhs_scale, grp ? N : M, grp ? job.n0 : job.m0);
    f32x16_t acc[2][4];
    mm_tile_product<F>(acc, lds, src, job.P, 1u, grp, wq, lane);
    grouped_results<F, EPI>(acc, job, M, N, job.m0 + 64u * wq, job.n0 + 128u * grp, lane & 31u, lane >> 5);
}

// ----------------------------------------------------------------------------
// Middling groups and short contractions: a 128 x 256 tile
// ----------------------------------------------------------------------------
//
// Four waves of 64 x 128, one per SIMD; two workgroups share a CU (registers
// and LDS of half a CU each) and fill each other's waits, prologues and
// epilogues. Operands pass through LDS as in the 256 x 256 tile: three stages,
// one barrier per K step, the copies of step s + 2 issued when step s is read.
// Per K step the workgroup copies 16 operand rows of 256 containers (rhs) and of
// 128 (lhs, two rows per load), and 2 scale rows of each: 7 loads per wave.
// LDS bounds it: per step a CU's 8 waves read 96 KiB and 48 KiB are copied in, some
// 1150 cycles at 128 bytes each, for 1024 of the matrix cores; the 256 x 256 tile
// copies 32 KiB (16 groups of 2048 rows, 4096 x 4096: 545 us, that one 495).
constexpr int kMidThreads = 256;
constexpr uint32_t kMidRows = 128;
constexpr uint32_t kMidQuadA = kMidRows * 16 + 128;   // an lhs row quad, padded
constexpr uint32_t kMidB = 4 * kMidQuadA;             // rhs row quads (kMmQuadPitch each) after them
constexpr uint32_t kMidScaleA = kMidB + 4 * kMmQuadPitch, kMidScaleB = kMidScaleA + 2 * kMidRows;
constexpr uint32_t kMidStageBytes = kMidScaleB + 2 * kMmTile;
constexpr int kMidCopies = 7;

// Copies of K step `step` by wave w: rhs row quad w; lhs row pairs 2 w and
// 2 w + 1; one scale load (waves 0 and 1: rhs row w; wave 2: both lhs rows;
// wave 3: an empty one, so that every wave has the same count).
template <int NT>
__device__ __forceinline__ void mid_copy(const MmSource &sa, const MmSource &sb, uint8_t *stage, uint8_t *spare,
                                         uint32_t P, uint32_t step, uint32_t w, uint32_t lane)
{
    const bool in = step * kMmStepRows < P;
    const uint32_t nrows = in ? min(P - step * kMmStepRows, kMmStepRows) : 0u;
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sb.data + (in ? (uint64_t)step * kMmStepRows * sb.pitch : 0ull)), (short)0,
        in ? (int)(nrows * sb.pitch - sb.col_bytes) : 0, kMmBufferFlags);
#pragma unroll
    for (uint32_t v = 0; v < 4; v++)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void_t *)(stage + kMidB + kMmQuadPitch * w + 1024u * v), 16,
                                                 16u * lane, (4u * w + v) * sb.pitch, 0, NT ? kBufferNT : 0);
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sa.data + (in ? (uint64_t)step * kMmStepRows * sa.pitch : 0ull)), (short)0,
        in ? (int)(nrows * sa.pitch - sa.col_bytes) : 0, kMmBufferFlags);
    const uint32_t va = (lane >> 5) * sa.pitch + 16u * (lane & 31u);
#pragma unroll
    for (uint32_t j = 0; j < 2; j++)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t *)(stage + kMidQuadA * w + 1024u * j), 16, va,
                                                 (4u * w + 2u * j) * sa.pitch, 0, 0);
    const MmSource &s = w == 2u ? sa : sb;
    const uint32_t kb = 2u * step + (w < 2u ? w : 0u);
    const bool ok = w < 3u && kb < P / 8u;
    const uint32_t blocks = w == 2u ? min(P / 8u - (ok ? kb : 0u), 2u) : 1u;
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(s.scale + (uint64_t)__builtin_amdgcn_readfirstlane(ok ? kb : 0u) * s.C), (short)0,
        ok ? (int)(blocks * s.C - s.col_bytes / 4u) : 0, kMmBufferFlags);
    const uint32_t vs = w == 2u ? (lane >> 5) * s.C + 4u * (lane & 31u) : 4u * lane;
    uint8_t *dst = w < 2u ? stage + kMidScaleB + kMmTile * w : w == 2u ? stage + kMidScaleA : spare;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void_t *)dst, 4, vs, 0, 0, 0);
}

// The product of one tile: this wave's 64 x 128 sums from row wm, column wn of it.
template <int F, int NT>
__device__ __forceinline__ void mid_steps(f32x16_t (&acc)[2][4], uint8_t *lds, const MmSource &sa, const MmSource &sb,
                                          uint32_t P, uint32_t wm, uint32_t wn, uint32_t wave, uint32_t lane)
{
    const uint32_t i = lane & 31u, h = lane >> 5;
    uint8_t *spare = lds + kMmStages * kMidStageBytes;
#pragma unroll
    for (int a = 0; a < 2; a++)
#pragma unroll
        for (int u = 0; u < 4; u++)
            acc[a][u] = f32x16_t{};
    const uint32_t a_off = kMidQuadA * h + 4u * (wm + 2u * i), b_off = kMidB + kMmQuadPitch * h + 4u * (wn + 4u * i);
    const uint32_t a_sc = kMidScaleA + kMidRows * h + wm + 2u * i, b_sc = kMidScaleB + kMmTile * h + wn + 4u * i;
    const uint32_t nsteps = (P + kMmStepRows - 1) / kMmStepRows;
#pragma unroll
    for (uint32_t st = 0; st < 2; st++)
        mid_copy<NT>(sa, sb, lds + st * kMidStageBytes, spare, P, st, wave, lane);
    uint32_t cur_i = 0;
    for (uint32_t s = 0; s < nsteps; s++) {
        const uint32_t fre_i = cur_i == 0 ? kMmStages - 1 : cur_i - 1u;   // step s - 1's stage
        const uint8_t *st = lds + cur_i * kMidStageBytes;
        // my copies of step s are through; after the barrier everyone's are,
        // and everyone has read step s - 1
        __builtin_amdgcn_s_waitcnt(mm_wait_vm(kMidCopies));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        MmRaw r;
#pragma unroll
        for (int v = 0; v < 8; v++) {
            const uint32_t *pa = reinterpret_cast<const uint32_t *>(
                st + a_off + (v < 4 ? 0u : 2u * kMidQuadA) + 4u * kMidRows * (v & 3));
            const uint32_t *pb = reinterpret_cast<const uint32_t *>(
                st + b_off + (v < 4 ? 0u : 2u * kMmQuadPitch) + 1024u * (v & 3));
            r.a[v][0] = pa[0];
            r.a[v][1] = pa[1];
#pragma unroll
            for (int u = 0; u < 4; u++)
                r.b[v][u] = pb[u];
        }
        r.as[0] = st[a_sc];
        r.as[1] = st[a_sc + 1];
        r.bs = *reinterpret_cast<const uint32_t *>(st + b_sc);
        mid_copy<NT>(sa, sb, lds + fre_i * kMidStageBytes, spare, P, s + 2, wave, lane);
        __builtin_amdgcn_s_waitcnt(mm_wait_vm_lgkm(63));   // my reads
        __builtin_amdgcn_sched_barrier(0);
        i32x8_t aop[2], bop[4];
#pragma unroll
        for (int a = 0; a < 2; a++)
            aop[a] = i32x8_t{(int)r.a[0][a], (int)r.a[1][a], (int)r.a[2][a], (int)r.a[3][a],
                             (int)r.a[4][a], (int)r.a[5][a], (int)r.a[6][a], (int)r.a[7][a]};
#pragma unroll
        for (int u = 0; u < 4; u++)
            bop[u] = i32x8_t{(int)r.b[0][u], (int)r.b[1][u], (int)r.b[2][u], (int)r.b[3][u],
                             (int)r.b[4][u], (int)r.b[5][u], (int)r.b[6][u], (int)r.b[7][u]};
#pragma unroll
        for (int a = 0; a < 2; a++) {
            acc[a][0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aop[a], bop[0], acc[a][0], F, F, 0,
                                                                        (int)r.as[a], 0, (int)r.bs);
            acc[a][1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aop[a], bop[1], acc[a][1], F, F, 0,
                                                                        (int)r.as[a], 1, (int)r.bs);
            acc[a][2] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aop[a], bop[2], acc[a][2], F, F, 0,
                                                                        (int)r.as[a], 2, (int)r.bs);
            acc[a][3] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(aop[a], bop[3], acc[a][3], F, F, 0,
                                                                        (int)r.as[a], 3, (int)r.bs);
        }
        __builtin_amdgcn_sched_barrier(0);
        cur_i = cur_i == kMmStages - 1 ? 0u : cur_i + 1u;
    }
    // no copy may land in the LDS of the workgroup that comes after this one
    __builtin_amdgcn_s_waitcnt(kWaitAllCopies);
}

template <int FMT, int EPI, int MODE>
__global__ __launch_bounds__(kMidThreads, 2) void grouped_mid_kernel(
    const uint8_t *__restrict__ lhs, const uint8_t *__restrict__ lhs_scale, const uint8_t *__restrict__ rhs,
    const uint8_t *__restrict__ rhs_scale, const int32_t *__restrict__ offsets, uint32_t groups, uint32_t P,
    uint32_t M, uint32_t N, uint32_t tiles_n, void *__restrict__ out)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[kMmStages * kMidStageBytes + kMmSpareBytes];
    constexpr int F = MfmaFmt<FMT>::value;
    constexpr uint32_t ES = EPI == kEpiF32 ? 4 : 2;
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t wm = 64u * (wave & 1u), wn = 128u * (wave >> 1);

    GroupedJob job = {lhs, lhs_scale, rhs, rhs_scale, (uint8_t *)out, P, 0, 0, 0, false};
    if (!grouped_job<MODE, kMidRows, kMmTile, 2 * kMmGroupRows, ES>(job, offsets, groups, M, N, tiles_n, lane))
        return;
    MmSource sa, sb;
    mm_source(sa, job.lhs, job.lhs_scale, M, job.m0);
    mm_source(sb, job.rhs, job.rhs_scale, N, job.n0);
    f32x16_t acc[2][4];
    // a group of one row tile reads its weights once, past the caches (128 experts x
    // 128 rows, 4096 x 1536: 182 -> 172 us; with two row tiles, 64 experts x 256 rows of
    // 2048 x 2048: 97 us, 117 with the hint)
    if (MODE == kGroupRows && job.one_tile)
        mid_steps<F, 1>(acc, lds, sa, sb, job.P, wm, wn, wave, lane);
    else
        mid_steps<F, 0>(acc, lds, sa, sb, job.P, wm, wn, wave, lane);
    grouped_results<F, EPI>(acc, job, M, N, job.m0 + wm, job.n0 + wn, lane & 31u, lane >> 5);
}

// ----------------------------------------------------------------------------
// Few rows per group, or few tiles: the weights stream through registers
// ----------------------------------------------------------------------------
//
// With few rows a product is bound by reading its expert's weights once. A
// workgroup of CW * KW waves computes 32 rows x 128 CW columns: CW waves side by
// side, each set of columns by KW waves that share the K steps. A wave loads the
// weights straight into the MFMA's lane mapping (16 bytes per lane and operand
// row: 512 contiguous bytes of each row), the next step's loads in flight, and
// keeps its own sums; at the end the KW waves' sums are added through LDS, in
// wave order. More rows per group take more row tiles, which find the weights in
// the caches.
//
// Lane mapping as in mxq_matmul_kernels.hpp: lane (i, h) supplies operand rows
// 4 h .. 4 h + 3 and 8 + 4 h .. 11 + 4 h of a step; A takes container m0 + i, B
// sub-tile u container n0 + 4 i + u, so result register r of sub-tile u is
// out[m0 + 8 (r >> 2) + 4 h + (r & 3)][n0 + 4 i + u].
constexpr uint32_t kStreamRows = 32;
constexpr uint32_t kStreamCols = 128;

struct StreamRaw {
    u32x4_t b[8];
    uint32_t a[8];
    uint32_t as, bs;     // the scale of A; byte u: of B sub-tile u
};

// The operand bytes and scales of K step `step`, or zeros without any access to
// memory where step >= end (end <= the number of steps). NT: the weights with
// the non-temporal hint.
template <int NT>
__device__ __forceinline__ void stream_load(StreamRaw &r, const MmSource &sa, const MmSource &sb, uint32_t P,
                                            uint32_t step, uint32_t end, uint32_t i, uint32_t h)
{
    const bool in = step < end;
    step = in ? step : 0u;
    const uint32_t nrows = in ? min(P - step * kMmStepRows, kMmStepRows) : 0u;
    const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sa.data + (uint64_t)step * kMmStepRows * sa.pitch), (short)0,
        in ? (int)(nrows * sa.pitch - sa.col_bytes) : 0, kMmBufferFlags);
    const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sb.data + (uint64_t)step * kMmStepRows * sb.pitch), (short)0,
        in ? (int)(nrows * sb.pitch - sb.col_bytes) : 0, kMmBufferFlags);
    const uint32_t va = 4u * h * sa.pitch + 4u * i, vb = 4u * h * sb.pitch + 16u * i;
#pragma unroll
    for (int v = 0; v < 8; v++)
        r.b[v] = __builtin_amdgcn_raw_buffer_load_b128(rb, vb, ((v < 4 ? 0u : 8u) + (v & 3)) * sb.pitch,
                                                       NT ? kBufferNT : 0);
#pragma unroll
    for (int v = 0; v < 8; v++)
        r.a[v] = __builtin_amdgcn_raw_buffer_load_b32(ra, va, ((v < 4 ? 0u : 8u) + (v & 3)) * sa.pitch, 0);
    // the step's scale rows 2 step + h, from the tile's first column on
    const __amdgpu_buffer_rsrc_t qa = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sa.scale + 2ull * step * sa.C), (short)0, in ? (int)(nrows / 8u * sa.C - sa.col_bytes / 4u) : 0,
        kMmBufferFlags);
    const __amdgpu_buffer_rsrc_t qb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sb.scale + 2ull * step * sb.C), (short)0, in ? (int)(nrows / 8u * sb.C - sb.col_bytes / 4u) : 0,
        kMmBufferFlags);
    r.as = __builtin_amdgcn_raw_buffer_load_b8(qa, h * sa.C + i, 0, 0);
    r.bs = __builtin_amdgcn_raw_buffer_load_b32(qb, h * sb.C + 4u * i, 0, 0);
}

__device__ __forceinline__ i32x8_t stream_a(const StreamRaw &r)
{
    return i32x8_t{(int)r.a[0], (int)r.a[1], (int)r.a[2], (int)r.a[3], (int)r.a[4], (int)r.a[5], (int)r.a[6],
                   (int)r.a[7]};
}

__device__ __forceinline__ i32x8_t stream_b(const StreamRaw &r, int u)
{
    return i32x8_t{(int)r.b[0][u], (int)r.b[1][u], (int)r.b[2][u], (int)r.b[3][u],
                   (int)r.b[4][u], (int)r.b[5][u], (int)r.b[6][u], (int)r.b[7][u]};
}

template <int F> __device__ __forceinline__ void stream_products(f32x16_t (&acc)[4], const StreamRaw &r)
{
    const i32x8_t a = stream_a(r);
    acc[0] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, stream_b(r, 0), acc[0], F, F, 0, (int)r.as, 0,
                                                             (int)r.bs);
    acc[1] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, stream_b(r, 1), acc[1], F, F, 0, (int)r.as, 1,
                                                             (int)r.bs);
    acc[2] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, stream_b(r, 2), acc[2], F, F, 0, (int)r.as, 2,
                                                             (int)r.bs);
    acc[3] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, stream_b(r, 3), acc[3], F, F, 0, (int)r.as, 3,
                                                             (int)r.bs);
}

// K steps s0 .. s1 - 1. Two register sets: one step's loads are in flight while
// the other's products are taken. (Without the scheduling fences the compiler
// moves the loads behind the products, and nothing overlaps; a third set
// changed nothing.)
template <int F, int NT>
__device__ __forceinline__ void stream_steps(f32x16_t (&acc)[4], const MmSource &sa, const MmSource &sb, uint32_t P,
                                             uint32_t s0, uint32_t s1, uint32_t i, uint32_t h)
{
    StreamRaw r0, r1;
    stream_load<NT>(r0, sa, sb, P, s0, s1, i, h);
    for (uint32_t s = s0; s < s1; s += 2) {
        stream_load<NT>(r1, sa, sb, P, s + 1u, s1, i, h);
        __builtin_amdgcn_sched_barrier(0);
        stream_products<F>(acc, r0);
        __builtin_amdgcn_sched_barrier(0);
        stream_load<NT>(r0, sa, sb, P, s + 2u, s1, i, h);
        __builtin_amdgcn_sched_barrier(0);
        stream_products<F>(acc, r1);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The rare path (scale bytes of 255, see mm_step_255): one wave computes its 32
// x 128 part over all K steps and stores it.
template <int F, int EPI>
__device__ __attribute__((noinline)) void stream_rare_part(const uint8_t *lhs, const uint8_t *lhs_scale,
                                                           const uint8_t *rhs, const uint8_t *rhs_scale, uint32_t P,
                                                           uint32_t M, uint32_t N, uint32_t m0, uint32_t n0,
                                                           uint32_t row_end, void *out)
{
    const uint32_t lane = __lane_id();
    const uint32_t i = lane & 31u, h = lane >> 5;
    MmSource sa, sb;
    mm_source(sa, lhs, lhs_scale, M, m0);
    mm_source(sb, rhs, rhs_scale, N, n0);
    f32x16_t acc[4];
#pragma unroll
    for (int u = 0; u < 4; u++)
        acc[u] = f32x16_t{};
    const uint32_t nsteps = (P + kMmStepRows - 1) / kMmStepRows;
    for (uint32_t s = 0; s < nsteps; s++) {
        StreamRaw r;
        stream_load<0>(r, sa, sb, P, s, nsteps, i, h);
        const i32x8_t bv[4] = {stream_b(r, 0), stream_b(r, 1), stream_b(r, 2), stream_b(r, 3)};
        // a block past the operand has zero data: any scale but 255 will do
        const bool in = 2u * s + h < P / 8u;
        mm_step_255<F>(acc, stream_a(r), bv, in ? r.as : 0x7Fu, in ? r.bs : 0x7F7F7F7Fu, h);
    }
#pragma unroll
    for (int r = 0; r < 16; r++) {
        const float v[4] = {acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
        grouped_store<EPI, 4, 0>(v, m0 + 8u * (r >> 2) + (r & 3), h, row_end, n0 + 4u * i, N, out);
    }
}

template <int FMT, int EPI, int CW, int KW>
__global__ __launch_bounds__(64 * CW * KW, 2) void grouped_stream_kernel(
    const uint8_t *__restrict__ lhs, const uint8_t *__restrict__ lhs_scale, const uint8_t *__restrict__ rhs,
    const uint8_t *__restrict__ rhs_scale, const int32_t *__restrict__ offsets, uint32_t groups, uint32_t P,
    uint32_t M, uint32_t N, uint32_t tiles_n, void *__restrict__ out)
{
    constexpr int F = MfmaFmt<FMT>::value;
    constexpr uint32_t RW = 16 / KW;   // result registers each wave adds up
    __shared__ __attribute__((aligned(16))) float sums[CW][KW][16][64][4];
    __shared__ uint32_t rare[CW];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t cw = wave % CW, kw = wave / CW;
    const uint32_t i = lane & 31u, h = lane >> 5;

    GroupedJob job = {lhs, lhs_scale, rhs, rhs_scale, (uint8_t *)out, P, 0, 0, 0, false};
    if (!rows_job<kStreamRows, CW * kStreamCols, 1, EPI == kEpiF32 ? 4 : 2>(job, offsets, groups, M, N, tiles_n, lane))
        return;
    const uint32_t n0 = job.n0 + cw * kStreamCols;
    MmSource sa, sb;
    mm_source(sa, job.lhs, job.lhs_scale, M, job.m0);
    mm_source(sb, job.rhs, job.rhs_scale, N, n0);
    if (threadIdx.x < CW)
        rare[threadIdx.x] = 0;

    f32x16_t acc[4];
#pragma unroll
    for (int u = 0; u < 4; u++)
        acc[u] = f32x16_t{};
    // (a wave past the last column takes no step)
    const uint32_t nsteps = n0 < N ? (P + kMmStepRows - 1) / kMmStepRows : 0u;
    const uint32_t per = (nsteps + KW - 1) / KW;
    const uint32_t s0 = min(kw * per, nsteps), s1 = min(s0 + per, nsteps);
    // A group of one row tile reads its weights once: past the caches, which
    // streams faster (64 experts x 32 rows, 4096 x 2048: 93 -> 87 us; with two row
    // tiles, 64 rows of 2048 x 2048, where the second finds them in the cache: 57 us, 69
    // with the hint).
    if (job.one_tile)
        stream_steps<F, 1>(acc, sa, sb, P, s0, s1, i, h);
    else
        stream_steps<F, 0>(acc, sa, sb, P, s0, s1, i, h);

#pragma unroll
    for (int r = 0; r < 16; r++)
        *reinterpret_cast<float4 *>(sums[cw][kw][r][lane]) = float4{acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
    __syncthreads();
    float v[RW][4];
    bool finite = true;
#pragma unroll
    for (uint32_t k = 0; k < RW; k++) {
        const uint32_t r = kw * RW + k;
        float4 x = *reinterpret_cast<const float4 *>(sums[cw][0][r][lane]);
#pragma unroll
        for (int w = 1; w < KW; w++) {
            const float4 y = *reinterpret_cast<const float4 *>(sums[cw][w][r][lane]);
            x.x += y.x;
            x.y += y.y;
            x.z += y.z;
            x.w += y.w;
        }
        v[k][0] = x.x;
        v[k][1] = x.y;
        v[k][2] = x.z;
        v[k][3] = x.w;
        finite = finite && __builtin_isfinite(x.x) && __builtin_isfinite(x.y) && __builtin_isfinite(x.z) &&
                 __builtin_isfinite(x.w);
    }
    if (wave_any(!finite) && lane == 0)
        atomicOr(&rare[cw], 1u);
    __syncthreads();
    if (__builtin_amdgcn_readfirstlane(rare[cw]) != 0) {
        if (kw == 0)
            stream_rare_part<F, EPI>(job.lhs, job.lhs_scale, job.rhs, job.rhs_scale, P, M, N, job.m0, n0, job.row_end,
                                     job.out);
    } else {
        const bool lines = whole_lines<EPI>(N);
#pragma unroll
        for (uint32_t k = 0; k < RW; k++) {
            const uint32_t r = kw * RW + k, m = job.m0 + 8u * (r >> 2) + (r & 3u);
            if (lines)
                grouped_store<EPI, 4, 1>(v[k], m, h, job.row_end, n0 + 4u * i, N, job.out);
            else
                grouped_store<EPI, 4, 0>(v[k], m, h, job.row_end, n0 + 4u * i, N, job.out);
        }
    }
}

} // namespace mxq
