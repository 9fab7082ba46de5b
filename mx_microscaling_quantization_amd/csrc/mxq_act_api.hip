// mxq_act_api.hip -- mxq_act_quantize and mxq_act_quantize_backward: validation and
// the launch of the kernels in mxq_act_kernels.hpp (one wave per 32 rows x 128 columns)
// on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"
#include "mxq_host.hpp"
#include "mxq_act_kernels.hpp"

namespace {

using mxq_host::emax_of;
using mxq_host::grid_fits;

typedef void (*fwd_fn)(const uint16_t *, uint32_t, uint32_t, uint32_t, int, int, uint8_t *, uint8_t *, uint8_t *,
                       uint8_t *);
typedef void (*bwd_fn)(const uint16_t *, const uint8_t *, const uint8_t *, uint32_t, uint32_t, uint32_t, int,
                       uint8_t *, uint8_t *, uint8_t *, uint8_t *, uint8_t *, uint8_t *);

template <int IN, int OUT, int SV> void pick_act(int act, fwd_fn &fwd, bwd_fn &bwd)
{
    if (act == MXQ_ACT_SWIGLU) {
        fwd = mxq::act_quantize_kernel<IN, OUT, SV, mxq::kActSwiglu>;
        bwd = mxq::act_backward_kernel<IN, OUT, SV, mxq::kActSwiglu>;
    } else {
        fwd = mxq::act_quantize_kernel<IN, OUT, SV, mxq::kActSilu>;
        bwd = mxq::act_backward_kernel<IN, OUT, SV, mxq::kActSilu>;
    }
}

template <int IN, int OUT> void pick_saved(int saved, int act, fwd_fn &fwd, bwd_fn &bwd)
{
    if (saved == MXQ_OUT_E4M3FN)
        pick_act<IN, OUT, mxq::kOutE4M3FN>(act, fwd, bwd);
    else
        pick_act<IN, OUT, mxq::kOutE5M2>(act, fwd, bwd);
}

template <int IN> void pick_out(int out, int saved, int act, fwd_fn &fwd, bwd_fn &bwd)
{
    switch (out) {
    case MXQ_OUT_E4M3FN: return pick_saved<IN, mxq::kOutE4M3FN>(saved, act, fwd, bwd);
    case MXQ_OUT_E5M2: return pick_saved<IN, mxq::kOutE5M2>(saved, act, fwd, bwd);
    default: return pick_saved<IN, mxq::kOutE2M1>(saved, act, fwd, bwd);
    }
}

void pick(int in, int out, int saved, int act, fwd_fn &fwd, bwd_fn &bwd)
{
    if (in == MXQ_IN_BF16)
        pick_out<mxq::kInBF16>(out, saved, act, fwd, bwd);
    else
        pick_out<mxq::kInF16>(out, saved, act, fwd, bwd);
}

// Types and sizes of both directions; rows a multiple of `align`.
int check(int64_t R, int64_t F, int in_dtype, int out_dtype, int saved_dtype, int act, int64_t align)
{
    if (in_dtype != MXQ_IN_BF16 && in_dtype != MXQ_IN_F16)
        return MXQ_E_IN_DTYPE;
    if (out_dtype != MXQ_OUT_E4M3FN && out_dtype != MXQ_OUT_E5M2 && out_dtype != MXQ_OUT_E2M1)
        return MXQ_E_OUT_DTYPE;
    if (saved_dtype != MXQ_OUT_E4M3FN && saved_dtype != MXQ_OUT_E5M2)
        return MXQ_E_OUT_DTYPE;
    if (act != MXQ_ACT_SILU && act != MXQ_ACT_SWIGLU)
        return MXQ_E_ACT;
    if (R < 0 || R % align != 0 || F < 0 || F % 32 != 0)
        return MXQ_E_SHAPE_P8;
    // columns and rows are 32-bit in the kernels, with room for a part of a tile
    if (R > ((int64_t)1 << 31) - 64 || F > ((int64_t)1 << 30) - 256)
        return MXQ_E_OVERFLOW;
    return MXQ_OK;
}

int64_t tiles_of(int64_t n, int64_t tile) { return (n + tile - 1) / tile; }

} // namespace

extern "C" {

int mxq_act_quantize(const void *z, int64_t R, int64_t F, int in_dtype, int out_dtype, int saved_dtype, int act,
                     void *data_out, void *scale_out, void *saved, void *saved_scale, void *stream)
{
    const int rc = check(R, F, in_dtype, out_dtype, saved_dtype, act, 8);
    if (rc != MXQ_OK || R == 0 || F == 0)
        return rc;
    if (!z || !data_out || !scale_out || !saved || !saved_scale)
        return MXQ_E_NULL;
    if (((uintptr_t)z | (uintptr_t)data_out | (uintptr_t)scale_out | (uintptr_t)saved | (uintptr_t)saved_scale) & 15u)
        return MXQ_E_ALIGN;
    const int64_t tiles_r = tiles_of(R, mxq::kActRows), tiles_c = tiles_of(F, mxq::kActCols);
    if (!grid_fits(tiles_r, tiles_c, 64))
        return MXQ_E_OVERFLOW;
    fwd_fn fwd;
    bwd_fn bwd;
    pick(in_dtype, out_dtype, saved_dtype, act, fwd, bwd);
    uint32_t r = (uint32_t)R, f = (uint32_t)F, tc = (uint32_t)tiles_c;
    int e = emax_of(out_dtype), es = emax_of(saved_dtype);
    void *args[] = {&z, &r, &f, &tc, &e, &es, &data_out, &scale_out, &saved, &saved_scale};
    const hipError_t err = hipLaunchKernel((const void *)fwd, dim3((uint32_t)(tiles_r * tiles_c)), dim3(64), args, 0,
                                           (hipStream_t)stream);
    return err == hipSuccess ? MXQ_OK : MXQ_E_HIP;
}

int mxq_act_quantize_backward(const void *grad, const void *saved, const void *saved_scale, int64_t R, int64_t F,
                              int in_dtype, int out_dtype, int saved_dtype, int act, void *rows_data, void *rows_scale,
                              void *cols_data, void *cols_scale, void *h_data, void *h_scale, void *stream)
{
    const int rc = check(R, F, in_dtype, out_dtype, saved_dtype, act, 32);
    if (rc != MXQ_OK || R == 0 || F == 0)
        return rc;
    if (!grad || !saved || !saved_scale || !rows_data || !rows_scale || !cols_data || !cols_scale || !h_data ||
        !h_scale)
        return MXQ_E_NULL;
    if (((uintptr_t)grad | (uintptr_t)saved | (uintptr_t)saved_scale | (uintptr_t)rows_data | (uintptr_t)rows_scale |
         (uintptr_t)cols_data | (uintptr_t)cols_scale | (uintptr_t)h_data | (uintptr_t)h_scale) & 15u)
        return MXQ_E_ALIGN;
    const int64_t tiles_r = tiles_of(R, mxq::kActRows), tiles_c = tiles_of(F, mxq::kActCols);
    if (!grid_fits(tiles_r, tiles_c, 64))
        return MXQ_E_OVERFLOW;
    fwd_fn fwd;
    bwd_fn bwd;
    pick(in_dtype, out_dtype, saved_dtype, act, fwd, bwd);
    uint32_t r = (uint32_t)R, f = (uint32_t)F, tc = (uint32_t)tiles_c;
    int e = emax_of(out_dtype);
    void *args[] = {&grad, &saved, &saved_scale, &r, &f, &tc, &e, &rows_data, &rows_scale, &cols_data, &cols_scale,
                    &h_data, &h_scale};
    const hipError_t err = hipLaunchKernel((const void *)bwd, dim3((uint32_t)(tiles_r * tiles_c)), dim3(64), args, 0,
                                           (hipStream_t)stream);
    return err == hipSuccess ? MXQ_OK : MXQ_E_HIP;
}

} // extern "C"
