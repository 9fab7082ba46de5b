// mxq_act_kernels.hpp -- gfx950 kernels of a gated activation between two products
// on MX operands: its result quantized for the next product, its input kept in 8
// bits for the backward pass, and that pass.
//
//   forward   z [R, W] (W = F, or 2 F: the gate's columns, then the other's)
//             h = silu(z_g) or silu(z_g) * z_u, rounded to z's type
//             -> h quantized along its rows (dim -1), z quantized in 8 x 4 blocks
//   backward  z~ = the kept z decoded, da [R, F]
//             dz_g = da * (z~_u) * s (1 + z~_g (1 - s)),  dz_u = da * z~_g s,
//             s = 1 / (1 + e^-z~_g), h = act(z~), each rounded to da's type
//             -> dz quantized along its rows (for the input's gradient) and down its
//                columns (for the first weights'), h down its columns (for the
//                second weights')
//
// One pass over memory: a byte for each kept value and each code. A thread has 8 rows
// x 8 columns of every matrix, two 8 x 4 blocks; a wave 32 rows x 128 columns, four
// blocks of 32 along the rows and one down. A block along a row is four
// neighbouring lanes' (two quad permutes), one down a column four lanes' 16 apart
// (two lane swaps). The rounded values go through the quantize's own helpers
// (mxq_quantize_kernels.hpp), so the bytes are those of quantizing them by themselves.
//
// Memory bounds both passes (bf16, e4m3fn, swiglu of 16384 x 4096, results in memory not
// written just before: forward 90 us, 5.3 TB/s; backward 114 us, 5.4 TB/s; a copy of 4 GiB
// runs at 4.7 TB/s). What costs is the layout of the codes along the rows: 128
// bytes of each view row for a tile. In the backward pass the arithmetic (some 45
// instructions for each of the tile's values) takes as long as the memory at its peak, under
// which it hides: with the five instructions that mend four overflow codes left to a
// mode of the conversions it took no less.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_axis_kernels.hpp"
#include "mxq_few_kernels.hpp"

namespace mxq {

constexpr uint32_t kActRows = 32, kActCols = 128;

// Two fp32 values in a 16-bit type, rounded to nearest even.
template <int IN> __device__ __forceinline__ uint32_t pack16(float a, float b)
{
    if constexpr (IN == kInBF16)
        return bf16_pair(a, b);
    else
        return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b});
}

template <int IN> __device__ __forceinline__ f32x2_t unpack16(uint32_t w)
{
    if constexpr (IN == kInBF16) {
        return f32x2_t{__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
    } else {
        const f16x2_t p = __builtin_bit_cast(f16x2_t, w);
        return f32x2_t{(float)p.x, (float)p.y};
    }
}

// 1 / (1 + e^-z): the hardware's 2^x and reciprocal (one step of fp32 each). The
// reciprocal gives zero for results below 2^-126, which gates from -87.4 down to where e^-z leaves
// fp32 (-88.7) have while silu of them is a normal number, so it is taken of a quarter.
__device__ __forceinline__ float sigmoid(float z)
{
    const float t = __builtin_amdgcn_exp2f(z * -1.44269504088896340736f);
    return 0.25f * __builtin_amdgcn_rcpf(__builtin_fmaf(t, 0.25f, 0.25f));
}

// A thread's 8 rows x 8 columns as pairs of columns.
typedef uint32_t ActBlock[8][4];

// Two halves of 16 bytes each of what a lane has to write: swapped between the wave's
// halves so that lanes l and l + 32 have the two of lane l (x), then of lane l + 32 (y).
// Stored like that an instruction writes whole runs of memory; a lane's own halves one
// after the other left every other 16 bytes of them to the next one (backward, silu, 16384
// x 4096: 74 us, 70 so; swiglu in f16, 16384 x 1408: 47.5 and 44.4).
__device__ __forceinline__ void act_swap(u32x4_t &x, u32x4_t &y)
{
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const uint32_t a = x[k], b = y[k];
        const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
        x[k] = r[0];
        y[k] = r[1];
    }
}

// ---- along the rows ----------------------------------------------------------------

// Codes and scales of the rows' blocks of 32: containers of view rows p0 and p0 + 1 (the
// thread's columns), rows row0 .. row0 + 7, of a [., R] view. whole: all 32 rows of the wave
// are there.
template <int IN, int OUT>
__device__ __forceinline__ void act_along(const ActBlock &w, int emax, uint64_t R, uint32_t row0, uint32_t p0,
                                          uint32_t lane, bool whole, uint8_t *__restrict__ data,
                                          uint8_t *__restrict__ scale)
{
    uint32_t e[8], code[2][8];
    bool special = false;
#pragma unroll
    for (int r = 0; r < 8; r += 2) {
        uint32_t m[2];
#pragma unroll
        for (int q = 0; q < 2; q++)
            m[q] = pk_max_u16(pk_max_u16(w[r + q][0] & 0x7FFF7FFFu, w[r + q][1] & 0x7FFF7FFFu),
                              pk_max_u16(w[r + q][2] & 0x7FFF7FFFu, w[r + q][3] & 0x7FFF7FFFu));
        // both rows' maxima in one register, then over the four lanes of the block
        uint32_t v = pk_max_u16(__builtin_amdgcn_perm(m[1], m[0], 0x05040100u),
                                __builtin_amdgcn_perm(m[1], m[0], 0x07060302u));
        v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));
        v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const uint32_t mag = half16(v, q);
            special |= mag > InfBits<IN>::value;
            e[r + q] = block_e8m0<IN>(mag, emax);
            const float s = e8m0_to_scale(e[r + q]);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const uint32_t *x = &w[r + q][2 * j];
                if constexpr (OUT == kOutE2M1)
                    code[j][r + q] = fp4_container<IN, 0>(0u, x[0], x[1], s);
                else
                    code[j][r + q] = fp8x4<IN, OUT>(x[0], x[1], s);
            }
        }
    }
    if (special)    // (one branch for all: sixteen kept the compiler from ordering anything)
#pragma unroll
        for (int r = 0; r < 8; r++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                fix_special_codes<IN, OUT, 1>(&w[r][2 * j], &e[r], &code[j][r]);
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const uint64_t at = (uint64_t)(p0 + j) * R + row0;
        if constexpr (OUT == kOutE2M1) {
            u32x4_t v;
#pragma unroll
            for (int k = 0; k < 4; k++)
                v[k] = (code[j][2 * k] & 0xFFFFu) | code[j][2 * k + 1] << 16;
            *reinterpret_cast<u32x4_t *>(data + 2u * at) = v;
        } else {
            u32x4_t x = {code[j][0], code[j][1], code[j][2], code[j][3]};
            u32x4_t y = {code[j][4], code[j][5], code[j][6], code[j][7]};
            uint8_t *p = data + 4u * at;
            if (whole) {
                // An even lane takes the first halves of its own and of the next lane's
                // (whose view row is two on), that one the second: a store's eight lanes of
                // four rows apart fill the 128 bytes of a line. Past the caches, as whole
                // lines go best (forward with the kept values' so too, swiglu, 16384 x
                // 4096: 110 -> 98 us; with the lines in halves 133 in place of 113, backward).
                const bool odd = (lane & 1u) != 0;
                u32x4_t a, b;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint32_t give = odd ? x[k] : y[k];
                    const uint32_t got = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)give, 0xB1, 0xF, 0xF, true);
                    a[k] = odd ? got : x[k];
                    b[k] = odd ? y[k] : got;
                }
                const uint64_t two = 8u * R;    // view rows
                __builtin_nontemporal_store(a, reinterpret_cast<u32x4_t *>(odd ? p + 16u - two : p));
                __builtin_nontemporal_store(b, reinterpret_cast<u32x4_t *>(odd ? p + 16u : p + two));
            } else {
                *reinterpret_cast<u32x4_t *>(p) = x;
                *reinterpret_cast<u32x4_t *>(p + 16u) = y;
            }
        }
    }
    if ((lane & 3u) == 0)
        *reinterpret_cast<u32x2_t *>(scale + (uint64_t)(p0 / 8u) * R + row0) =
            u32x2_t{e[0] | e[1] << 8 | e[2] << 16 | e[3] << 24, e[4] | e[5] << 8 | e[6] << 16 | e[7] << 24};
}

// ---- down the columns ---------------------------------------------------------------

// Codes and scales of the columns' blocks of 32: rows row0 .. row0 + 7 of columns col ..
// col + 7 of a [R / 4, C] view (R a multiple of 32).
template <int IN, int OUT>
__device__ __forceinline__ void act_down(const ActBlock &w, int emax, uint64_t C, uint32_t row0, uint32_t col,
                                         uint32_t lane, uint8_t *__restrict__ data, uint8_t *__restrict__ scale)
{
    uint32_t e[8], code[2][8];
    bool special = false;
    // rows 4 j .. 4 j + 3 of column 2 k + q
    const auto column = [&](int j, int k, int q, uint32_t (&x)[2]) {
        const uint32_t pick = q ? 0x07060302u : 0x05040100u;
        x[0] = __builtin_amdgcn_perm(w[4 * j + 1][k], w[4 * j][k], pick);
        x[1] = __builtin_amdgcn_perm(w[4 * j + 3][k], w[4 * j + 2][k], pick);
    };
#pragma unroll
    for (int k = 0; k < 4; k++) {
        uint32_t v = 0;
#pragma unroll
        for (int r = 0; r < 8; r++)
            v = pk_max_u16(v, w[r][k] & 0x7FFF7FFFu);
        // lanes 16 and 32 apart hold the block's other rows
        const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = pk_max_u16(a[0], a[1]);
        const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = pk_max_u16(b[0], b[1]);
#pragma unroll
        for (int q = 0; q < 2; q++) {
            const uint32_t mag = half16(v, q);
            special |= mag > InfBits<IN>::value;
            e[2 * k + q] = block_e8m0<IN>(mag, emax);
            const float s = e8m0_to_scale(e[2 * k + q]);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                uint32_t x[2];
                column(j, k, q, x);
                if constexpr (OUT == kOutE2M1)
                    code[j][2 * k + q] = fp4_container<IN, 0>(0u, x[0], x[1], s);
                else
                    code[j][2 * k + q] = fp8x4<IN, OUT>(x[0], x[1], s);
            }
        }
    }
    if (special)
#pragma unroll
        for (int c = 0; c < 8; c++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                uint32_t x[2];
                column(j, c >> 1, c & 1, x);
                fix_special_codes<IN, OUT, 1>(x, &e[c], &code[j][c]);
            }
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const uint64_t at = (uint64_t)(row0 / 4u + j) * C + col;
        if constexpr (OUT == kOutE2M1) {
            u32x4_t v;
#pragma unroll
            for (int k = 0; k < 4; k++)
                v[k] = (code[j][2 * k] & 0xFFFFu) | code[j][2 * k + 1] << 16;
            *reinterpret_cast<u32x4_t *>(data + 2u * at) = v;
        } else {
            u32x4_t x = {code[j][0], code[j][1], code[j][2], code[j][3]};
            u32x4_t y = {code[j][4], code[j][5], code[j][6], code[j][7]};
            act_swap(x, y);
            // rows of lanes 0 .. 31, then of lanes 32 .. 63 (16 rows of the tensor on)
            uint8_t *p = data + 4u * at + (lane >> 5) * 16u - (lane >> 5) * 16u * C;
            // past the caches, whole lines as they are
            __builtin_nontemporal_store(x, reinterpret_cast<u32x4_t *>(p));
            __builtin_nontemporal_store(y, reinterpret_cast<u32x4_t *>(p + 16u * C));
        }
    }
    if (lane < 16u)
        *reinterpret_cast<u32x2_t *>(scale + (uint64_t)(row0 / 32u) * C + col) =
            u32x2_t{e[0] | e[1] << 8 | e[2] << 16 | e[3] << 24, e[4] | e[5] << 8 | e[6] << 16 | e[7] << 24};
}

// ---- kept values ------------------------------------------------------------------------

// The thread's two 8 x 4 blocks as codes and scales of a [R, W] tensor.
template <int IN, int OUT>
__device__ __forceinline__ void act_keep(const ActBlock &w, int emax, uint64_t W, uint32_t row0, uint32_t col,
                                         uint8_t *__restrict__ data, uint8_t *__restrict__ scale)
{
    uint32_t e[2];
    uint32_t code[8][2];
    bool special = false;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        uint32_t v = 0;
#pragma unroll
        for (int r = 0; r < 8; r++)
            v = pk_max_u16(v, pk_max_u16(w[r][2 * j] & 0x7FFF7FFFu, w[r][2 * j + 1] & 0x7FFF7FFFu));
        const uint32_t mag = max(v & 0xFFFFu, v >> 16);
        special |= mag > InfBits<IN>::value;
        e[j] = block_e8m0<IN>(mag, emax);
        const float s = e8m0_to_scale(e[j]);
#pragma unroll
        for (int r = 0; r < 8; r++)
            code[r][j] = fp8x4<IN, OUT>(w[r][2 * j], w[r][2 * j + 1], s);
    }
    if (special)
#pragma unroll
        for (int r = 0; r < 8; r++)
            fix_special_codes<IN, OUT, 2>(w[r], e, code[r]);
#pragma unroll
    for (int r = 0; r < 8; r++)
        __builtin_nontemporal_store(u32x2_t{code[r][0], code[r][1]},
                                    reinterpret_cast<u32x2_t *>(data + (row0 + r) * W + col));
    *reinterpret_cast<uint16_t *>(scale + (row0 / 8u) * (W / 4u) + col / 4u) = (uint16_t)(e[0] | e[1] << 8);
}

// The kept values of row row0 + r, columns col .. col + 7, decoded.
template <int SV>
__device__ __forceinline__ void act_decode(u32x2_t c, const float (&s)[2], float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int word = (int)(j ? c.y : c.x);
        f32x2_t a, b;
        if constexpr (SV == kOutE4M3FN) {
            a = __builtin_amdgcn_cvt_pk_f32_fp8(word, false);
            b = __builtin_amdgcn_cvt_pk_f32_fp8(word, true);
        } else {
            a = __builtin_amdgcn_cvt_pk_f32_bf8(word, false);
            b = __builtin_amdgcn_cvt_pk_f32_bf8(word, true);
        }
        v[4 * j] = a.x * s[j];
        v[4 * j + 1] = a.y * s[j];
        v[4 * j + 2] = b.x * s[j];
        v[4 * j + 3] = b.y * s[j];
    }
}

// 2^(e - 127) of the two blocks' bytes; 255 (2^128) as infinity's neighbour is not an fp32
// number, so it is left to `twice`.
__device__ __forceinline__ bool act_scales(uint32_t bytes, float (&s)[2])
{
    bool any = false;
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const uint32_t e = (bytes >> (8 * j)) & 0xFFu;
        any |= e == 255u;
        s[j] = __uint_as_float(max(min(e, 254u) << 23, 0x00400000u));   // (byte 0: 2^-127)
    }
    return any;
}

// ---- the kernels ----------------------------------------------------------------------------

// Workgroup (a wave) -> tile of 32 rows x 128 columns.
struct ActTile {
    uint32_t row0, col;
    bool whole;     // 32 rows
};
__device__ __forceinline__ ActTile act_tile(uint32_t R, uint32_t tiles_c)
{
    const uint32_t t = tile_index<kMmXcds>();
    const uint32_t band = t / tiles_c, lane = threadIdx.x;
    return ActTile{band * kActRows + 8u * (lane >> 4), (t - band * tiles_c) * kActCols + 8u * (lane & 15u),
                   band * kActRows + kActRows <= R};
}

// R a multiple of 8, F of 32: whole lanes of a quad are in or out.
template <int IN, int OUT, int SV, int ACT>
__global__ __launch_bounds__(64) void act_quantize_kernel(const uint16_t *__restrict__ z, uint32_t R, uint32_t F,
                                                          uint32_t tiles_c, int emax, int emax_saved,
                                                          uint8_t *__restrict__ data, uint8_t *__restrict__ scale,
                                                          uint8_t *__restrict__ saved,
                                                          uint8_t *__restrict__ saved_scale)
{
    constexpr int NM = ACT == kActSwiglu ? 2 : 1;
    const ActTile t = act_tile(R, tiles_c);
    if (t.row0 >= R || t.col >= F)
        return;
    const uint64_t W = (uint64_t)NM * F;
    ActBlock w[NM];
#pragma unroll
    for (int r = 0; r < 8; r++)
#pragma unroll
        for (int k = 0; k < NM; k++) {
            const u32x4_t v = __builtin_nontemporal_load(
                reinterpret_cast<const u32x4_t *>(z + (t.row0 + r) * W + (uint64_t)k * F + t.col));
#pragma unroll
            for (int c = 0; c < 4; c++)
                w[k][r][c] = v[c];
        }
#pragma unroll
    for (int k = 0; k < NM; k++)
        act_keep<IN, SV>(w[k], emax_saved, W, t.row0, k * F + t.col, saved, saved_scale);
    ActBlock h;
#pragma unroll
    for (int r = 0; r < 8; r++)
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const f32x2_t g = unpack16<IN>(w[0][r][c]);
            float a = g.x * sigmoid(g.x), b = g.y * sigmoid(g.y);
            if constexpr (NM == 2) {
                const f32x2_t u = unpack16<IN>(w[1][r][c]);
                a *= u.x;
                b *= u.y;
            }
            h[r][c] = pack16<IN>(a, b);
        }
    act_along<IN, OUT>(h, emax, R, t.row0, t.col / 4u, threadIdx.x, t.whole, data, scale);
}

// R and F multiples of 32.
template <int IN, int OUT, int SV, int ACT>
__global__ __launch_bounds__(64, 2) void act_backward_kernel(
    const uint16_t *__restrict__ grad, const uint8_t *__restrict__ saved, const uint8_t *__restrict__ saved_scale,
    uint32_t R, uint32_t F, uint32_t tiles_c, int emax, uint8_t *__restrict__ rows_data,
    uint8_t *__restrict__ rows_scale, uint8_t *__restrict__ cols_data, uint8_t *__restrict__ cols_scale,
    uint8_t *__restrict__ h_data, uint8_t *__restrict__ h_scale)
{
    constexpr int NM = ACT == kActSwiglu ? 2 : 1;
    const ActTile t = act_tile(R, tiles_c);
    if (t.col >= F)
        return;
    const uint64_t W = (uint64_t)NM * F;
    u32x4_t da[8];
    u32x2_t code[NM][8];
    uint32_t sb[NM];
#pragma unroll
    for (int r = 0; r < 8; r++) {
        da[r] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4_t *>(grad + (uint64_t)(t.row0 + r) * F + t.col));
#pragma unroll
        for (int k = 0; k < NM; k++)
            code[k][r] = __builtin_nontemporal_load(
                reinterpret_cast<const u32x2_t *>(saved + (t.row0 + r) * W + (uint64_t)k * F + t.col));
    }
#pragma unroll
    for (int k = 0; k < NM; k++)
        sb[k] = *reinterpret_cast<const uint16_t *>(saved_scale + (t.row0 / 8u) * (W / 4u) + (k * F + t.col) / 4u);
    float s[NM][2];
    bool twice = false;
#pragma unroll
    for (int k = 0; k < NM; k++)
        twice |= act_scales(sb[k], s[k]);

    ActBlock dz[NM], h;
#pragma unroll
    for (int r = 0; r < 8; r++) {
        __builtin_amdgcn_sched_barrier(0);
        float v[NM][8];
#pragma unroll
        for (int k = 0; k < NM; k++) {
            act_decode<SV>(code[k][r], s[k], v[k]);
            if (twice)
#pragma unroll
                for (int c = 0; c < 8; c++)
                    v[k][c] *= ((sb[k] >> (8 * (c >> 2))) & 0xFFu) == 255u ? 2.0f : 1.0f;
        }
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const uint32_t word = da[r][c];
            const f32x2_t d = unpack16<IN>(word);
            float out[NM + 1][2];
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const float g = v[0][2 * c + q], x = q ? d.y : d.x;
                const float sg = sigmoid(g), a = g * sg;
                const float slope = __builtin_fmaf(a, 1.0f - sg, sg);
                if constexpr (NM == 2) {
                    const float u = v[NM - 1][2 * c + q];
                    out[0][q] = x * u * slope;
                    out[1][q] = x * a;
                    out[NM][q] = a * u;
                } else {
                    out[0][q] = x * slope;
                    out[NM][q] = a;
                }
            }
#pragma unroll
            for (int k = 0; k < NM; k++)
                dz[k][r][c] = pack16<IN>(out[k][0], out[k][1]);
            h[r][c] = pack16<IN>(out[NM][0], out[NM][1]);
            // (rounded here, not where it is first used: a word instead of its operands)
#pragma unroll
            for (int k = 0; k < NM; k++)
                asm volatile("" : "+v"(dz[k][r][c]));
            asm volatile("" : "+v"(h[r][c]));
        }
    }
    // one after the other: mixed, their temporaries fill the registers, as do the masked
    // values that two of them would share
    __builtin_amdgcn_sched_barrier(0);
    act_down<IN, OUT>(h, emax, F, t.row0, t.col, threadIdx.x, h_data, h_scale);
#pragma unroll
    for (int k = 0; k < NM; k++) {
        __builtin_amdgcn_sched_barrier(0);
        act_along<IN, OUT>(dz[k], emax, R, t.row0, (k * F + t.col) / 4u, threadIdx.x, true, rows_data,
                           rows_scale);
#pragma unroll
        for (int r = 0; r < 8; r++)
#pragma unroll
            for (int c = 0; c < 4; c++)
                asm volatile("" : "+v"(dz[k][r][c]));
        __builtin_amdgcn_sched_barrier(0);
        act_down<IN, OUT>(dz[k], emax, W, t.row0, k * F + t.col, threadIdx.x, cols_data, cols_scale);
    }
}

} // namespace mxq
