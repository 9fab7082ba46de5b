// mxq_few_api.hip -- mxq_moe_few_tokens: validation and the launch of the two kernels
// in mxq_few_kernels.hpp on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"
#include "mxq_host.hpp"
#include "mxq_few_kernels.hpp"

namespace {

using mxq_host::grid_fits;

typedef void (*up_fn)(const uint16_t *, uint32_t, const void *, uint32_t, uint32_t, uint32_t, const uint8_t *,
                      const uint8_t *, uint32_t, uint32_t, uint16_t *, uint32_t *, uint32_t, uint16_t *, uint32_t);
typedef void (*down_fn)(const uint16_t *, uint32_t, const void *, uint32_t, uint32_t, uint32_t, const uint8_t *,
                        const uint8_t *, uint32_t, uint32_t, float *, uint32_t *, const float *, uint16_t *);

struct Kernels {
    up_fn up;
    down_fn down;
};

template <int FMT, int IN, int MX, typename ID> Kernels pick_act(int act)
{
    return {act == MXQ_ACT_SWIGLU ? (up_fn)mxq::few_up_kernel<FMT, IN, mxq::kActSwiglu, MX, ID>
                                  : (up_fn)mxq::few_up_kernel<FMT, IN, mxq::kActSilu, MX, ID>,
            mxq::few_down_kernel<FMT, IN, MX, ID>};
}

template <int FMT, int IN, int MX> Kernels pick_id(int id_bytes, int act)
{
    return id_bytes == 8 ? pick_act<FMT, IN, MX, int64_t>(act) : pick_act<FMT, IN, MX, int32_t>(act);
}

template <int FMT, int IN> Kernels pick_rows(bool many, int id_bytes, int act)
{
    return many ? pick_id<FMT, IN, 4>(id_bytes, act) : pick_id<FMT, IN, 2>(id_bytes, act);
}

template <int FMT> Kernels pick_in(int in_dtype, bool many, int id_bytes, int act)
{
    return in_dtype == MXQ_IN_BF16 ? pick_rows<FMT, mxq::kInBF16>(many, id_bytes, act)
                                   : pick_rows<FMT, mxq::kInF16>(many, id_bytes, act);
}

Kernels pick(int fmt, int in_dtype, bool many, int id_bytes, int act)
{
    switch (fmt) {
    case MXQ_OUT_E4M3FN: return pick_in<mxq::kOutE4M3FN>(in_dtype, many, id_bytes, act);
    case MXQ_OUT_E5M2: return pick_in<mxq::kOutE5M2>(in_dtype, many, id_bytes, act);
    default: return pick_in<mxq::kOutE2M1>(in_dtype, many, id_bytes, act);
    }
}

// Tokens, slots, experts and the lengths of the contractions and of the result.
int check_sizes(int64_t tokens, int64_t K, int64_t slots, int64_t experts, int64_t F, int64_t N)
{
    if (tokens < 0 || slots < 1 || slots > MXQ_MOE_MAX_SLOTS || experts < 1 || experts > MXQ_MOE_MAX_EXPERTS ||
        tokens > MXQ_MOE_FEW_PAIRS / slots)
        return MXQ_E_MOE;
    if (K < 0 || F < 0 || K % 32 != 0 || F % 32 != 0)
        return MXQ_E_SHAPE_P8;
    if (N < 0 || N % 4 != 0)
        return MXQ_E_SHAPE_F4;
    // an expert's matrix is one buffer with 31-bit offsets
    const int64_t most = ((int64_t)1 << 31) - 1;
    if (K > most || F > most / 2 || N > most || (F > 0 && K > most / (2 * F)) || (N > 0 && F > most / N))
        return MXQ_E_OVERFLOW;
    return MXQ_OK;
}

int64_t round16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

int64_t tiles_of(int64_t cols) { return (cols + mxq::kFewCols - 1) / mxq::kFewCols; }

// Waves of a workgroup: eight share a contraction where there are few workgroups, four
// where there are enough of them to fill the CUs' places.
uint32_t waves_of(int64_t workgroups) { return workgroups > 256 ? 4u : 8u; }

} // namespace

extern "C" {

size_t mxq_moe_few_tokens_workspace_bytes(int64_t tokens, int64_t slots, int64_t F, int64_t N)
{
    if (check_sizes(tokens, 0, slots, 1, F, N) != MXQ_OK)
        return 0;
    const int64_t pairs = tokens * slots;
    return (size_t)(round16(4 * pairs * F) + round16(4 * pairs * N) + round16(4 * tiles_of(N) * tokens));
}

int mxq_moe_few_tokens(const void *x, int64_t tokens, int64_t K, int in_dtype, const void *ids, int id_bytes,
                       const float *weights, int64_t slots, int64_t experts, const void *w1, const void *w1_scale,
                       const void *w2, const void *w2_scale, int64_t F, int64_t N, int fmt, int act, void *workspace,
                       void *out, void *stream)
{
    if (in_dtype != MXQ_IN_BF16 && in_dtype != MXQ_IN_F16)
        return MXQ_E_IN_DTYPE;
    if (fmt != MXQ_OUT_E4M3FN && fmt != MXQ_OUT_E5M2 && fmt != MXQ_OUT_E2M1)
        return MXQ_E_OUT_DTYPE;
    if (act != MXQ_ACT_SILU && act != MXQ_ACT_SWIGLU)
        return MXQ_E_ACT;
    if (id_bytes != 4 && id_bytes != 8)
        return MXQ_E_ELEM_DTYPE;
    const int rc = check_sizes(tokens, K, slots, experts, F, N);
    if (rc != MXQ_OK || tokens == 0 || N == 0)
        return rc;
    if (!ids || !weights || !workspace || !out || (K > 0 && (!x || (F > 0 && (!w1 || !w1_scale)))) ||
        (F > 0 && (!w2 || !w2_scale)))
        return MXQ_E_NULL;
    if (((uintptr_t)x | (uintptr_t)ids | (uintptr_t)weights | (uintptr_t)w1 | (uintptr_t)w1_scale | (uintptr_t)w2 |
         (uintptr_t)w2_scale | (uintptr_t)workspace | (uintptr_t)out) & 15u)
        return MXQ_E_ALIGN;

    uint32_t pairs = (uint32_t)(tokens * slots), s = (uint32_t)slots, e = (uint32_t)experts;
    uint32_t k = (uint32_t)K, f = (uint32_t)F, n = (uint32_t)N;
    // as many workgroups as any assignment has experts in use; at least one column tile
    // of the first kernel, which also prepares the second one's counters
    const int64_t used = pairs < e ? pairs : e;
    const int64_t up_tiles = F > 0 ? tiles_of(F) : 1, down_tiles = tiles_of(N);
    if (!grid_fits(used, up_tiles, mxq::kFewThreads) || !grid_fits(used, down_tiles, mxq::kFewThreads))
        return MXQ_E_OVERFLOW;
    const uint32_t up_waves = waves_of(used * up_tiles), down_waves = waves_of(used * down_tiles);
    const uint32_t lds = 4u * 16u * 64u;      // a wave's sums of 16 pairs with one matrix
    uint32_t ut = (uint32_t)up_tiles, dt = (uint32_t)down_tiles;
    uint16_t *h = (uint16_t *)workspace;
    float *y = (float *)((uint8_t *)workspace + round16(4 * (int64_t)pairs * F));
    uint32_t *arrived = (uint32_t *)((uint8_t *)y + round16(4 * (int64_t)pairs * N));
    const Kernels kernels = pick(fmt, in_dtype, pairs > 24 * used, id_bytes, act);
    void *a1[] = {&x, &k, &ids, &pairs, &s, &e, &w1, &w1_scale, &f, &ut, &h, &arrived, &dt, &out, &n};
    if (hipLaunchKernel((const void *)kernels.up, dim3((uint32_t)(used * up_tiles)), dim3(64u * up_waves), a1,
                        up_waves * lds * (act == MXQ_ACT_SWIGLU ? 2u : 1u), (hipStream_t)stream) != hipSuccess)
        return MXQ_E_HIP;
    void *a2[] = {&h, &f, &ids, &pairs, &s, &e, &w2, &w2_scale, &n, &dt, &y, &arrived, &weights, &out};
    const hipError_t err = hipLaunchKernel((const void *)kernels.down, dim3((uint32_t)(used * down_tiles)),
                                           dim3(64u * down_waves), a2, down_waves * lds, (hipStream_t)stream);
    return err == hipSuccess ? MXQ_OK : MXQ_E_HIP;
}

} // extern "C"
