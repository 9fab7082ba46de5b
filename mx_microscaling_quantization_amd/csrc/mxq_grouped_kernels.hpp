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
//           zero for the rows past the last group
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
    uint32_t per, first, total;   // groups per lane; this lane's first row tile; all row tiles
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
    return s;
}

// Row tile `tile` (< total).
template <uint32_t TILE>
__device__ __forceinline__ GroupTile group_find(const int32_t *offsets, uint32_t groups, uint32_t R,
                                                const GroupScan &s, uint32_t tile)
{
    const uint32_t l = (uint32_t)__popcll(__builtin_amdgcn_ballot_w64(s.first <= tile)) - 1u;
    uint32_t left = tile - (uint32_t)__builtin_amdgcn_readlane((int)s.first, (int)l);
    GroupTile t = {groups, R, R};
    for (uint32_t q = 0; q < s.per; q++) {
        const uint32_t g = l * s.per + q;
        if (g > groups)
            break;
        uint32_t a, b;
        group_bounds(offsets, groups, R, g, a, b);
        const uint32_t n = (b - a + TILE - 1) / TILE;
        if (left < n) {
            t = {g, a + left * TILE, b};
            break;
        }
        left -= n;
    }
    t.group = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.group);
    t.m0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.m0);
    t.end = (uint32_t)__builtin_amdgcn_readfirstlane((int)t.end);
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

// 4 adjacent results of row m from column col on; N % 4 == 0.
template <int EPI>
__device__ __forceinline__ void grouped_store(const float *v, uint32_t m, uint32_t row_end, uint32_t col, uint32_t N,
                                              void *__restrict__ out)
{
    if (m >= row_end || col >= N)
        return;
    const uint64_t o = (uint64_t)m * N + col;
    if constexpr (EPI == kEpiF32)
        *reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + o) = float4{v[0], v[1], v[2], v[3]};
    else
        *reinterpret_cast<uint2 *>(reinterpret_cast<uint16_t *>(out) + o) =
            uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
}

// ----------------------------------------------------------------------------
// Many rows per group: the scaled matmul's 256 x 256 tile
// ----------------------------------------------------------------------------

enum { kGroupRows = 0, kGroupWgrad = 1 };

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

    uint32_t m0, n0, row_end;
    if constexpr (MODE == kGroupRows) {
        // M sorted rows, P operand rows. Tile rows of all groups in order,
        // walked in fours column by column as the scaled matmul does.
        const GroupScan s = group_scan<kMmTile>(offsets, groups, M, lane);
        const uint32_t t = xcd_tile(blockIdx.x, s.total * tiles_n);
        if (t >= s.total * tiles_n)
            return;
        const uint32_t walk = t / (kMmGroupRows * tiles_n);
        const uint32_t first_row = walk * kMmGroupRows;
        const uint32_t rows = min((uint32_t)kMmGroupRows, s.total - first_row);
        const uint32_t in_walk = t - walk * kMmGroupRows * tiles_n;
        const GroupTile g = group_find<kMmTile>(offsets, groups, M, s, first_row + in_walk % rows);
        m0 = g.m0;
        n0 = in_walk / rows * kMmTile;
        row_end = g.end;
        if (g.group >= groups) {
            P = 0;   // no operand rows: the product is zero
        } else {
            rhs += (uint64_t)g.group * P * N * 4u;
            rhs_scale += (uint64_t)g.group * (P / 8u) * N;
        }
    } else {
        // P operand rows in all; group g's are offsets[g] / 4 .. The tiles of
        // one group are spread over the XCDs (each gets consecutive ones), so
        // that a large group's work is.
        const uint32_t tiles_m = (M + kMmTile - 1) / kMmTile, per = tiles_m * tiles_n;
        const uint32_t g = blockIdx.x / per;
        const uint32_t t = xcd_tile(blockIdx.x - g * per, per);
        const uint32_t walk = t / (kMmGroupRows * tiles_n);
        const uint32_t first_row = walk * kMmGroupRows;
        const uint32_t rows = min((uint32_t)kMmGroupRows, tiles_m - first_row);
        const uint32_t in_walk = t - walk * kMmGroupRows * tiles_n;
        m0 = (first_row + in_walk % rows) * kMmTile;
        n0 = in_walk / rows * kMmTile;
        row_end = M;
        uint32_t a, b;
        group_bounds(offsets, groups, 4u * P, g, a, b);
        a = __builtin_amdgcn_readfirstlane(a / 32u);   // whole blocks
        b = __builtin_amdgcn_readfirstlane(b / 32u);
        lhs += (uint64_t)a * 8u * 4u * M;
        lhs_scale += (uint64_t)a * M;
        rhs += (uint64_t)a * 8u * 4u * N;
        rhs_scale += (uint64_t)a * N;
        P = (b - a) * 8u;
        out = (uint8_t *)out + (uint64_t)g * M * N * ES;
    }

    MmSource src;
    mm_source(src, grp ? rhs : lhs, grp ? rhs_scale : lhs_scale, grp ? N : M, grp ? n0 : m0);
    f32x16_t acc[2][4];
    mm_tile_product<F>(acc, lds, src, P, 1u, grp, wq, lane);

    const uint32_t wm0 = m0 + 64u * wq, wn0 = n0 + 128u * grp;
    bool finite = true;
#pragma unroll
    for (int a = 0; a < 2; a++)
#pragma unroll
        for (int u = 0; u < 4; u++)
#pragma unroll
            for (int r = 0; r < 16; r++)
                finite = finite && __builtin_isfinite(acc[a][u][r]);
    // a scale byte of 255, or a sum that is not finite by itself: the rare
    // path, as in the scaled matmul
    if (__builtin_amdgcn_ballot_w64(!finite) != 0) {
        mm_rare_part<F, EPI>(lhs, lhs_scale, rhs, rhs_scale, P, M, N, wm0, wn0, 1u, out, nullptr, 0, row_end);
        __builtin_amdgcn_endpgm();
    }
    const uint32_t i = lane & 31u, h = lane >> 5;
#pragma unroll
    for (int r = 0; r < 16; r++)
#pragma unroll
        for (int a = 0; a < 2; a++) {
            const float v[4] = {acc[a][0][r], acc[a][1][r], acc[a][2][r], acc[a][3][r]};
            grouped_store<EPI>(v, wm0 + 16u * (r >> 2) + 8u * h + 2u * (r & 3) + a, row_end, wn0 + 4u * i, N, out);
        }
}

// ----------------------------------------------------------------------------
// Few rows per group: the weights stream through registers
// ----------------------------------------------------------------------------
//
// With few rows a product is bound by reading its expert's weights once. A
// workgroup of WAVES waves computes 32 * MS rows x 128 columns; each wave takes
// its share of the K steps, loads the weights straight into the MFMA's lane
// mapping (16 bytes per lane and operand row: 512 contiguous bytes of each
// row) with the next steps' loads in flight, and keeps its own sums. At the
// end the waves' sums are added through LDS, in wave order, one 32-row
// sub-tile at a time.
//
// Lane mapping as in mxq_matmul_kernels.hpp: lane (i, h) supplies operand rows
// 4 h .. 4 h + 3 and 8 + 4 h .. 11 + 4 h of a step; A sub-tile a takes container
// m0 + MS i + a, B sub-tile u container n0 + 4 i + u, so result register r of
// sub-tile (a, u) is out[m0 + MS (8 (r >> 2) + 4 h + (r & 3)) + a][n0 + 4 i + u].
constexpr uint32_t kStreamCols = 128;

template <int MS> struct StreamRaw {
    u32x4_t b[8];
    uint32_t a[8][MS];
    uint32_t as, bs;     // byte a (u): the scale of A sub-tile a (B sub-tile u)
};

// The operand bytes and scales of K step `step`, or zeros without any access to
// memory where step >= end (end <= the number of steps).
template <int MS>
__device__ __forceinline__ void stream_load(StreamRaw<MS> &r, const MmSource &sa, const MmSource &sb, uint32_t P,
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
    const uint32_t va = 4u * h * sa.pitch + 4u * MS * i, vb = 4u * h * sb.pitch + 16u * i;
#pragma unroll
    for (int v = 0; v < 8; v++) {
        const uint32_t row = (v < 4 ? 0u : 8u) + (v & 3);
        r.b[v] = __builtin_amdgcn_raw_buffer_load_b128(rb, vb, row * sb.pitch, 0);
    }
#pragma unroll
    for (int v = 0; v < 8; v++) {
        const uint32_t row = (v < 4 ? 0u : 8u) + (v & 3);
        if constexpr (MS == 1) {
            r.a[v][0] = __builtin_amdgcn_raw_buffer_load_b32(ra, va, row * sa.pitch, 0);
        } else if constexpr (MS == 2) {
            const u32x2_t d = __builtin_amdgcn_raw_buffer_load_b64(ra, va, row * sa.pitch, 0);
            r.a[v][0] = d.x;
            r.a[v][1] = d.y;
        } else {
            const u32x4_t d = __builtin_amdgcn_raw_buffer_load_b128(ra, va, row * sa.pitch, 0);
#pragma unroll
            for (int a = 0; a < 4; a++)
                r.a[v][a] = d[a];
        }
    }
    // the step's scale rows 2 step + h, from the tile's first column on
    const uint32_t blocks = nrows / 8u;
    const __amdgpu_buffer_rsrc_t qa = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sa.scale + 2ull * step * sa.C), (short)0, in ? (int)(blocks * sa.C - sa.col_bytes / 4u) : 0,
        kMmBufferFlags);
    const __amdgpu_buffer_rsrc_t qb = __builtin_amdgcn_make_buffer_rsrc(
        (void *)(sb.scale + 2ull * step * sb.C), (short)0, in ? (int)(blocks * sb.C - sb.col_bytes / 4u) : 0,
        kMmBufferFlags);
    if constexpr (MS == 1)
        r.as = __builtin_amdgcn_raw_buffer_load_b8(qa, h * sa.C + i, 0, 0);
    else if constexpr (MS == 2)
        r.as = __builtin_amdgcn_raw_buffer_load_b16(qa, h * sa.C + 2u * i, 0, 0);
    else
        r.as = __builtin_amdgcn_raw_buffer_load_b32(qa, h * sa.C + 4u * i, 0, 0);
    r.bs = __builtin_amdgcn_raw_buffer_load_b32(qb, h * sb.C + 4u * i, 0, 0);
}

template <int F, int MS>
__device__ __forceinline__ void stream_products(f32x16_t (&acc)[MS][4], const StreamRaw<MS> &r)
{
#pragma unroll
    for (int u = 0; u < 4; u++) {
        const i32x8_t b = {(int)r.b[0][u], (int)r.b[1][u], (int)r.b[2][u], (int)r.b[3][u],
                           (int)r.b[4][u], (int)r.b[5][u], (int)r.b[6][u], (int)r.b[7][u]};
        // the byte of a scale register is an immediate of the instruction:
        // shifted into byte 0 here
        const int bs = (int)(r.bs >> (8 * u));
#pragma unroll
        for (int a = 0; a < MS; a++) {
            const i32x8_t av = {(int)r.a[0][a], (int)r.a[1][a], (int)r.a[2][a], (int)r.a[3][a],
                                (int)r.a[4][a], (int)r.a[5][a], (int)r.a[6][a], (int)r.a[7][a]};
            acc[a][u] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, b, acc[a][u], F, F, 0,
                                                                        (int)(r.as >> (8 * a)), 0, bs);
        }
    }
}

// The rare path (scale bytes of 255, see mm_step_255): one wave computes
// sub-tile `a` over all K steps and stores it.
template <int F, int EPI, int MS>
__device__ __attribute__((noinline)) void stream_rare_part(const uint8_t *lhs, const uint8_t *lhs_scale,
                                                           const uint8_t *rhs, const uint8_t *rhs_scale, uint32_t P,
                                                           uint32_t M, uint32_t N, uint32_t m0, uint32_t n0,
                                                           uint32_t row_end, uint32_t a, void *out)
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
        StreamRaw<MS> r;
        stream_load<MS>(r, sa, sb, P, s, nsteps, i, h);
        i32x8_t av, bv[4];
#pragma unroll
        for (int v = 0; v < 8; v++) {
            uint32_t x = r.a[v][0];
#pragma unroll
            for (int k = 1; k < MS; k++)
                x = a == (uint32_t)k ? r.a[v][k] : x;
            av[v] = (int)x;
#pragma unroll
            for (int u = 0; u < 4; u++)
                bv[u][v] = (int)r.b[v][u];
        }
        // a block past the operand has zero data: any scale but 255 will do
        const bool in = 2u * s + h < P / 8u;
        mm_step_255<F>(acc, av, bv, in ? (r.as >> (8u * a)) & 0xFFu : 0x7Fu, in ? r.bs : 0x7F7F7F7Fu, h);
    }
#pragma unroll
    for (int r = 0; r < 16; r++) {
        const float v[4] = {acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
        grouped_store<EPI>(v, m0 + MS * (8u * (r >> 2) + 4u * h + (r & 3)) + a, row_end, n0 + 4u * i, N, out);
    }
}

template <int FMT, int EPI, int MS, int CW, int KW, int DEPTH>
__global__ __launch_bounds__(64 * CW * KW, 2) void grouped_stream_kernel(
    const uint8_t *__restrict__ lhs, const uint8_t *__restrict__ lhs_scale, const uint8_t *__restrict__ rhs,
    const uint8_t *__restrict__ rhs_scale, const int32_t *__restrict__ offsets, uint32_t groups, uint32_t P,
    uint32_t M, uint32_t N, uint32_t tiles_n, void *__restrict__ out)
{
    constexpr int F = MfmaFmt<FMT>::value;
    constexpr uint32_t TILE = 32 * MS, RW = 16 / KW;   // result registers each wave adds up
    __shared__ __attribute__((aligned(16))) float sums[CW][KW][16][64][4];
    __shared__ uint32_t rare[MS][CW];
    const uint32_t lane = threadIdx.x & 63u;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t cw = wave % CW, kw = wave / CW;
    const uint32_t i = lane & 31u, h = lane >> 5;

    const GroupScan sc = group_scan<TILE>(offsets, groups, M, lane);
    const uint32_t t = xcd_tile(blockIdx.x, sc.total * tiles_n);
    if (t >= sc.total * tiles_n)
        return;
    const uint32_t tr = t / tiles_n;
    const GroupTile g = group_find<TILE>(offsets, groups, M, sc, tr);
    const uint32_t n0 = ((t - tr * tiles_n) * CW + cw) * kStreamCols;
    if (g.group >= groups) {
        P = 0;
    } else {
        rhs += (uint64_t)g.group * P * N * 4u;
        rhs_scale += (uint64_t)g.group * (P / 8u) * N;
    }
    MmSource sa, sb;
    mm_source(sa, lhs, lhs_scale, M, g.m0);
    mm_source(sb, rhs, rhs_scale, N, n0);
    if (threadIdx.x < MS * CW)
        (&rare[0][0])[threadIdx.x] = 0;

    f32x16_t acc[MS][4];
#pragma unroll
    for (int a = 0; a < MS; a++)
#pragma unroll
        for (int u = 0; u < 4; u++)
            acc[a][u] = f32x16_t{};
    const uint32_t nsteps = n0 < N ? (P + kMmStepRows - 1) / kMmStepRows : 0u;
    const uint32_t per = (nsteps + KW - 1) / KW;
    const uint32_t s0 = min(kw * per, nsteps), s1 = min(s0 + per, nsteps);
    // DEPTH register sets: the loads of DEPTH - 1 steps are in flight while one
    // step's products are taken. (Without the scheduling fences the compiler
    // moves the loads behind the products, and nothing overlaps.)
    StreamRaw<MS> raw[DEPTH];
#pragma unroll
    for (uint32_t d = 0; d < DEPTH - 1; d++)
        stream_load<MS>(raw[d], sa, sb, P, s0 + d, s1, i, h);
    for (uint32_t s = s0; s < s1; s += DEPTH) {
#pragma unroll
        for (uint32_t d = 0; d < DEPTH; d++) {
            stream_load<MS>(raw[(d + DEPTH - 1) % DEPTH], sa, sb, P, s + d + DEPTH - 1, s1, i, h);
            __builtin_amdgcn_sched_barrier(0);
            stream_products<F, MS>(acc, raw[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

#pragma unroll
    for (int a = 0; a < MS; a++) {
#pragma unroll
        for (int r = 0; r < 16; r++)
            *reinterpret_cast<float4 *>(sums[cw][kw][r][lane]) =
                float4{acc[a][0][r], acc[a][1][r], acc[a][2][r], acc[a][3][r]};
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
        if (__builtin_amdgcn_ballot_w64(!finite) != 0 && lane == 0)
            atomicOr(&rare[a][cw], 1u);
        __syncthreads();   // and every wave has read this sub-tile's sums
        if (rare[a][cw]) {
            if (kw == 0)
                stream_rare_part<F, EPI, MS>(lhs, lhs_scale, rhs, rhs_scale, P, M, N, g.m0, n0, g.end, (uint32_t)a,
                                             out);
            continue;
        }
#pragma unroll
        for (uint32_t k = 0; k < RW; k++) {
            const uint32_t r = kw * RW + k;
            grouped_store<EPI>(v[k], g.m0 + MS * (8u * (r >> 2) + 4u * h + (r & 3u)) + a, g.end, n0 + 4u * i, N, out);
        }
    }
}

} // namespace mxq
