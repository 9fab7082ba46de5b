// mxq_fp4_api.hip -- mxq_scaled_matmul_fp4 and mxq_grouped_matmul_fp4: validation,
// the choice of tile and the launch of the kernels in mxq_fp4_kernels.hpp on the
// caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"
#include "mxq_host.hpp"
#include "mxq_fp4_kernels.hpp"

namespace {

using mxq_host::grid_fits;

typedef void (*fp4_fn)(const uint8_t *, const uint8_t *, const uint8_t *, const uint8_t *, const int32_t *, uint32_t,
                       uint32_t, uint32_t, uint32_t, uint32_t, uint32_t, void *);

enum { kTile256 = 0, kTile128 = 1, kStreamWide = 2, kStream = 3, kStreamNarrow = 4 };

// Rows, columns and threads of each form's tile.
struct Form {
    int64_t rows, cols;
    uint32_t threads;
};
constexpr Form kForms[] = {{256, 256, 256}, {128, 128, 256}, {32, 256, 256}, {32, 128, 256}, {32, 64, 512}};

template <int LF, int EPI> fp4_fn pick_form(int form)
{
    switch (form) {
    case kTile256: return mxq::fp4_tile_kernel<LF, EPI, 4>;
    case kTile128: return mxq::fp4_tile_kernel<LF, EPI, 2>;
    case kStreamWide: return mxq::fp4_stream_kernel<LF, EPI, 4, 2, 2>;
    case kStream: return mxq::fp4_stream_kernel<LF, EPI, 4, 1, 4>;
    default: return mxq::fp4_stream_kernel<LF, EPI, 2, 1, 8>;
    }
}

template <int LF> fp4_fn pick_res(int res_dtype, int form)
{
    return res_dtype == MXQ_RES_F32 ? pick_form<LF, mxq::kEpiF32>(form) : pick_form<LF, mxq::kEpiBF16>(form);
}

fp4_fn pick(int lhs_fmt, int res_dtype, int form)
{
    switch (lhs_fmt) {
    case MXQ_OUT_E4M3FN: return pick_res<mxq::kOutE4M3FN>(res_dtype, form);
    case MXQ_OUT_E5M2: return pick_res<mxq::kOutE5M2>(res_dtype, form);
    default: return pick_res<mxq::kOutE2M1>(res_dtype, form);
    }
}

int run(const void *lhs, const void *lhs_scale, const void *rhs, const void *rhs_scale, const int32_t *offsets,
        int64_t groups, int64_t P, int64_t M, int64_t N, int lhs_fmt, int res_dtype, unsigned dense, void *out,
        void *stream)
{
    if (lhs_fmt != MXQ_OUT_E4M3FN && lhs_fmt != MXQ_OUT_E5M2 && lhs_fmt != MXQ_OUT_E2M1)
        return MXQ_E_OUT_DTYPE;
    if (res_dtype != MXQ_RES_F32 && res_dtype != MXQ_RES_BF16)
        return MXQ_E_RES_DTYPE;
    if (P < 0 || P % 8 != 0)
        return MXQ_E_SHAPE_P8;
    if (M < 0 || N < 0 || N % 4 != 0)
        return MXQ_E_SHAPE_F4;
    if (P > ((int64_t)1 << 29) - 1 || M > MXQ_MATMUL_MAX_COLS || N > MXQ_MATMUL_MAX_COLS)
        return MXQ_E_OVERFLOW;
    if (M == 0 || N == 0)
        return MXQ_OK;
    if (!out || (P > 0 && (!lhs || !lhs_scale || !rhs || !rhs_scale)))
        return MXQ_E_NULL;
    if (((uintptr_t)lhs | (uintptr_t)lhs_scale | (uintptr_t)rhs | (uintptr_t)rhs_scale | (uintptr_t)out |
         (uintptr_t)offsets) & 15u)
        return MXQ_E_ALIGN;

    // The form follows from the number of tiles: the streams' smallest tiles of which there is
    // at most one for each of the 256 CUs share a contraction among the most waves and CUs.
    // From 128-row tiles on two fit a CU, and 256-row tiles, with half the copies per product,
    // win where there are enough of them (us, one group, e4m3fn by e2m1; in brackets e2m1 by
    // e2m1; narrow: 32 x 64, stream: 32 x 128, wide: 32 x 256):
    //   M x K x N             narrow  stream  wide      128 x 128    256 x 256
    //   16 x 4096 x 4096         9.5    12.8  21.1
    //   128 x 4096 x 4096        9.9    11.5  18.1 (17) 20.3 (13.1)  53.7 (33.6)
    //   256 x 4096 x 4096       18.7    15.0  18.5
    //   512 x 4096 x 4096       35.2    22.9  18.7 (18) 20.7 (13.6)  55.2 (34.3)
    //   2048 x 4096 x 4096                    55 (53)   32.9 (23.4)  57.6 (36.5)
    //   16 x 8192 x 8192        15.8    20.7  35.1
    //   256 x 8192 x 8192                     44 (44)   37.5 (23.3)  102 (60.5)
    //   256 x 4096 x 14336                    41 (40)   21.3 (15.0)  55.6 (35.2)
    //   1024 x 4096 x 14336                  140 (140)  57.3 (41.5)  58.0 (38.8)
    //   2048 x 8192 x 8192                   314 (312)  113 (81.9)   109 (70.7)
    // Groups of up to 64 rows stream their weights whatever their number (64 x 64 rows, 4096 x
    // 2048: wide 74 (72), 128 x 128 84 (68)).
    // Between the square tiles the rounds decide: a round of two 128-row tiles on each CU
    // takes half of one of 256-row tiles' time, 3 % more than that, or 15 % for e2m1 by e2m1
    // (whose products wait for copies more), but its last round is half as long, and a group's
    // last tile, filled by half on average, half as large. Uneven groups, 256 x 256 and 128 x
    // 128: 16 x 2048 rows, 4096 x 4096, 565 (358) and 536 (398); 16 x 512, 171 (112) and 134
    // (97); 64 x 512, 4096 x 2048, 334 (212) and 309 (223); 8 x 2048, 8192 x 2048, 336 (198) and
    // 252 (176). A short contraction is mostly the stores of its results, which two tiles on
    // a CU overlap.
    const int64_t mean = M / groups, kCus = 256;
    const auto tiles = [&](int form) {
        const Form &f = kForms[form];
        return ((M + f.rows - 1) / f.rows) * ((N + f.cols - 1) / f.cols);
    };
    const auto rounds = [&](int form, int64_t on_cu) {
        const Form &f = kForms[form];
        const int64_t down = offsets ? M / f.rows + (groups + 1) / 2 : (M + f.rows - 1) / f.rows;
        return (down * ((N + f.cols - 1) / f.cols) + on_cu * kCus - 1) / (on_cu * kCus);
    };
    int form;
    if (tiles(kStreamNarrow) <= kCus)
        form = kStreamNarrow;
    else if (tiles(kStream) <= kCus)
        form = kStream;
    else if (mean <= 64)
        form = kStreamWide;
    else if (P <= 256 || rounds(kTile128, 2) * (lhs_fmt == MXQ_OUT_E2M1 ? 115 : 103) < rounds(kTile256, 1) * 200)
        form = kTile128;
    else
        form = kTile256;
    // the square tiles copy 16 bytes of containers and 4 scale bytes at a time, which a pitch of other
    // row counts does not allow (2047 and 2048 x 8192 x 8192: 319 (317) and 109 (70) us)
    if (M % 4 != 0 && form <= kTile128)
        form = kStreamWide;

    const Form &f = kForms[form];
    const int64_t tiles_n = (N + f.cols - 1) / f.cols;
    // every group, and the rows past the last one, may end with a part of a tile
    const int64_t tiles_m = offsets ? M / f.rows + groups + 1 : (M + f.rows - 1) / f.rows;
    if (!grid_fits(tiles_m, tiles_n, f.threads))
        return MXQ_E_OVERFLOW;
    fp4_fn k = pick(lhs_fmt, res_dtype, form);
    const uint8_t *a0 = (const uint8_t *)lhs, *a1 = (const uint8_t *)lhs_scale, *a2 = (const uint8_t *)rhs,
                  *a3 = (const uint8_t *)rhs_scale;
    uint32_t g = (uint32_t)groups, p = (uint32_t)P, m = (uint32_t)M, n = (uint32_t)N, tn = (uint32_t)tiles_n;
    uint32_t d = dense ? 1u : 0u;
    void *args[] = {&a0, &a1, &a2, &a3, &offsets, &g, &p, &m, &n, &tn, &d, &out};
    const hipError_t err = hipLaunchKernel((const void *)k, dim3((uint32_t)(tiles_m * tiles_n)), dim3(f.threads), args,
                                           0, (hipStream_t)stream);
    return err == hipSuccess ? MXQ_OK : MXQ_E_HIP;
}

} // namespace

extern "C" {

int mxq_scaled_matmul_fp4(const void *lhs, const void *lhs_scale, const void *rhs, const void *rhs_scale, int64_t P,
                          int64_t M, int64_t N, int lhs_fmt, int res_dtype, unsigned flags, void *out, void *stream)
{
    if (flags & ~(unsigned)MXQ_FLAG_DENSE_SCALE)
        return MXQ_E_FLAGS;
    return run(lhs, lhs_scale, rhs, rhs_scale, nullptr, 1, P, M, N, lhs_fmt, res_dtype, flags & MXQ_FLAG_DENSE_SCALE,
               out, stream);
}

int mxq_grouped_matmul_fp4(const void *lhs, const void *lhs_scale, const void *rhs, const void *rhs_scale,
                           const int32_t *offsets, int64_t groups, int64_t P, int64_t rows, int64_t N, int lhs_fmt,
                           int res_dtype, void *out, void *stream)
{
    if (groups < 1 || groups > MXQ_MOE_MAX_EXPERTS)
        return MXQ_E_MOE;
    if (rows < 0 || rows % 4 != 0)
        return MXQ_E_ROWS;
    if (!offsets && rows > 0 && N > 0)
        return MXQ_E_NULL;
    return run(lhs, lhs_scale, rhs, rhs_scale, offsets, groups, P, rows, N, lhs_fmt, res_dtype, 1u, out, stream);
}

} // extern "C"
