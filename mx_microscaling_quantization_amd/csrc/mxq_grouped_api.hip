// mxq_grouped_api.hip -- mxq_grouped_matmul and mxq_grouped_matmul_wgrad:
// validation, the choice of tile and the launch of the kernels in
// mxq_grouped_kernels.hpp on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"
#include "mxq_host.hpp"
#include "mxq_grouped_kernels.hpp"

namespace {

using mxq_host::grid_fits;

typedef void (*grouped_fn)(const uint8_t *, const uint8_t *, const uint8_t *, const uint8_t *, const int32_t *,
                           uint32_t, uint32_t, uint32_t, uint32_t, uint32_t, void *);

template <int FMT, int EPI> grouped_fn pick_kernel(int kind)
{
    switch (kind) {
    case 0: return mxq::grouped_matmul_kernel<FMT, EPI, mxq::kGroupRows>;
    case 1: return mxq::grouped_matmul_kernel<FMT, EPI, mxq::kGroupWgrad>;
    case 2: return mxq::grouped_mid_kernel<FMT, EPI, mxq::kGroupRows>;
    case 5: return mxq::grouped_mid_kernel<FMT, EPI, mxq::kGroupWgrad>;
    case 3: return mxq::grouped_stream_kernel<FMT, EPI, 2, 2>;
    default: return mxq::grouped_stream_kernel<FMT, EPI, 1, 4>;
    }
}

grouped_fn pick(int fmt, int res_dtype, int kind)
{
    if (fmt == MXQ_OUT_E4M3FN)
        return res_dtype == MXQ_RES_F32 ? pick_kernel<mxq::kOutE4M3FN, mxq::kEpiF32>(kind)
                                        : pick_kernel<mxq::kOutE4M3FN, mxq::kEpiBF16>(kind);
    return res_dtype == MXQ_RES_F32 ? pick_kernel<mxq::kOutE5M2, mxq::kEpiF32>(kind)
                                    : pick_kernel<mxq::kOutE5M2, mxq::kEpiBF16>(kind);
}

// P % 8, column counts, types and pointers of both products; `empty`: no
// operand byte is read.
int check(const void *lhs, const void *lhs_scale, const void *rhs, const void *rhs_scale, const int32_t *offsets,
          int64_t groups, int64_t P, int64_t M, int64_t N, int fmt, int res_dtype, const void *out, bool empty)
{
    if (fmt != MXQ_OUT_E4M3FN && fmt != MXQ_OUT_E5M2)
        return MXQ_E_OUT_DTYPE;
    if (res_dtype != MXQ_RES_F32 && res_dtype != MXQ_RES_BF16)
        return MXQ_E_RES_DTYPE;
    if (groups < 1 || groups > MXQ_MOE_MAX_EXPERTS)
        return MXQ_E_MOE;
    if (P < 0 || P % 8 != 0)
        return MXQ_E_SHAPE_P8;
    if (M < 0 || N < 0 || M % 4 != 0 || N % 4 != 0)
        return MXQ_E_SHAPE_F4;
    if (P > ((int64_t)1 << 29) - 1 || M > MXQ_MATMUL_MAX_COLS || N > MXQ_MATMUL_MAX_COLS)
        return MXQ_E_OVERFLOW;
    if (M == 0 || N == 0)
        return MXQ_OK;
    if (!offsets || !out || (!empty && (!lhs || !lhs_scale || !rhs || !rhs_scale)))
        return MXQ_E_NULL;
    if (((uintptr_t)lhs | (uintptr_t)lhs_scale | (uintptr_t)rhs | (uintptr_t)rhs_scale | (uintptr_t)out |
         (uintptr_t)offsets) & 15u)
        return MXQ_E_ALIGN;
    return MXQ_OK;
}

int launch(grouped_fn k, int64_t blocks, uint32_t threads, const void *lhs, const void *lhs_scale, const void *rhs,
           const void *rhs_scale, const int32_t *offsets, int64_t groups, int64_t P, int64_t M, int64_t N,
           int64_t tiles_n, void *out, void *stream)
{
    const uint8_t *a0 = (const uint8_t *)lhs, *a1 = (const uint8_t *)lhs_scale, *a2 = (const uint8_t *)rhs,
                  *a3 = (const uint8_t *)rhs_scale;
    uint32_t g = (uint32_t)groups, p = (uint32_t)P, m = (uint32_t)M, n = (uint32_t)N, tn = (uint32_t)tiles_n;
    void *args[] = {&a0, &a1, &a2, &a3, &offsets, &g, &p, &m, &n, &tn, &out};
    const hipError_t err = hipLaunchKernel((const void *)k, dim3((uint32_t)blocks), dim3(threads), args, 0,
                                           (hipStream_t)stream);
    return err == hipSuccess ? MXQ_OK : MXQ_E_HIP;
}

} // namespace

extern "C" {

int mxq_grouped_matmul(const void *lhs, const void *lhs_scale, const void *rhs, const void *rhs_scale,
                       const int32_t *offsets, int64_t groups, int64_t P, int64_t rows, int64_t N, int fmt,
                       int res_dtype, void *out, void *stream)
{
    const int rc = check(lhs, lhs_scale, rhs, rhs_scale, offsets, groups, P, rows, N, fmt, res_dtype, out, P == 0);
    if (rc != MXQ_OK || rows == 0 || N == 0)
        return rc;
    // The tile follows from the mean rows per group, the length of the
    // contraction and the number of tiles (268 MB of e4m3fn weights, 2048 x 2048 and
    // 4096 x 4096 up to 128 rows, 4096 x 4096 and 4096 x 2048 from there on; groups of
    // one size; us, all forms in turn):
    //   rows per group  32-row tiles  128-row tiles  256-row tiles
    //   32                 46-48          59-66          72-82
    //   64                 58-59          59-67          74-84
    //   80                   79             68             -
    //   96                 80-92          59-70          75-86
    //   128                  94           59-71          78-85
    //   256                   -             87             71
    //   352                   -          130-132        125-126
    //   512                   -          148-149        131-132
    //   2048 (4096 x 4096)    -            545            495
    // With sizes of 0.6 to 1.4 times the mean, more of the tiles are parts of one: 352
    // rows 135-137 and 121, 2048 rows 573 and 538. (The border of 384 is from groups of
    // about 350 rows at which the two forms took 124 and 127; in this table the 256-row
    // tiles lead from 256 rows on.)
    // A short contraction is mostly the stores of its results, which several
    // smaller workgroups on a CU overlap with other tiles' products (16 experts,
    // 32768 rows, 4096 columns: 64 values 65 us, 256-row tiles 72; 512 values
    // 113 and 116; 1024 values 166 and 168; 2048 values 301 and 275).
    // Where 128-row tiles do not fill half of the CUs, the time is one tile's
    // whole contraction, which the small ones share out among their waves
    // (512 x 4096 by 4096 x 4096: 25 us and 46; with 168 such tiles, 1536 rows
    // over 2048 values by 3584 columns: 30 and 27).
    const int64_t mean = rows / groups, kCus = 256;
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    int64_t tiles_n = up(N, mxq::kMmTile);
    int kind = 0;
    if (mean <= 64 || 2 * up(rows, mxq::kMidRows) * tiles_n <= kCus)
        kind = 3;
    else if (mean <= 384 || P <= 256)
        kind = 2;
    // with fewer small tiles than that, narrower ones whose four waves all share
    // the contraction (32 rows per expert, 4096 x 4096: 8 experts, 128 tiles, 25 us,
    // wide ones 33; 10 experts, 160 tiles, 40 and 34)
    if (kind == 3 && 2 * up(rows, mxq::kStreamRows) * tiles_n <= kCus) {
        kind = 4;
        tiles_n = up(N, mxq::kStreamCols);
    }
    // every group, and the rows past the last one, may end with a part of a tile
    const int64_t tile = kind >= 3 ? mxq::kStreamRows : kind == 2 ? mxq::kMidRows : mxq::kMmTile;
    const int64_t tiles_m = rows / tile + groups + 1;
    const uint32_t threads = kind ? 256 : mxq::kMmThreads;
    if (!grid_fits(tiles_m, tiles_n, threads))
        return MXQ_E_OVERFLOW;
    return launch(pick(fmt, res_dtype, kind), tiles_m * tiles_n, threads, lhs, lhs_scale, rhs, rhs_scale, offsets,
                  groups, P, rows, N, tiles_n, out, stream);
}

int mxq_grouped_matmul_wgrad(const void *lhs, const void *lhs_scale, const void *rhs, const void *rhs_scale,
                             const int32_t *offsets, int64_t groups, int64_t P, int64_t M, int64_t N, int fmt,
                             int res_dtype, void *out, void *stream)
{
    const int rc = check(lhs, lhs_scale, rhs, rhs_scale, offsets, groups, P, M, N, fmt, res_dtype, out, P == 0);
    if (rc != MXQ_OK || M == 0 || N == 0)
        return rc;
    // With little to multiply per group the time is that of writing the result,
    // which several smaller workgroups on a CU overlap with the products of
    // others (32 weight gradients of 2048 x 2048, 288 rows of the contraction per
    // group: 79 us, 256-row tiles 91; 39 of 1920 x 768, 512 rows: 54 and 64;
    // 35 of 672 x 3328, 1056 rows: 117 and 123, of sizes of 0.6 to 1.4 times that 117
    // and 114; 16 of 2048 x 4096, 768 rows: 130 and 136, uneven 134 and 132, 2048 rows:
    // 276 and 258).
    const bool mid = 4 * P / groups < 768;
    const int64_t tile = mid ? mxq::kMidRows : mxq::kMmTile;
    const uint32_t threads = mid ? mxq::kMidThreads : mxq::kMmThreads;
    const int64_t tiles_m = (M + tile - 1) / tile, tiles_n = (N + mxq::kMmTile - 1) / mxq::kMmTile;
    if (!grid_fits(tiles_m, tiles_n, threads) || !grid_fits(tiles_m * tiles_n, groups, threads))
        return MXQ_E_OVERFLOW;
    return launch(pick(fmt, res_dtype, mid ? 5 : 1), tiles_m * tiles_n * groups, threads, lhs, lhs_scale, rhs,
                  rhs_scale, offsets, groups, P, M, N, tiles_n, out, stream);
}

} // extern "C"
