// mxq_clip_api.hip -- mxq_clip_grad_norm: validation, the tensors' tables and
// the launches of the kernels in mxq_clip_kernels.hpp on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"
#include "mxq_host.hpp"
#include "mxq_clip_kernels.hpp"

namespace {

// Workgroups of a norm launch: 8 per CU, fewer when there are not that many tiles.
constexpr uint32_t kClipBlocks = 2048;

// Elements of a tensor and tiles of a launch, for a dispatch's 2^32 work-items:
// one tensor has at most 2^36 * 4 bytes in tiles of 2^15.
constexpr int64_t kMaxElements = (int64_t)1 << 36;
constexpr uint64_t kMaxTiles = (uint64_t)1 << 23;

uint32_t elem_bytes(int type) { return type == MXQ_ELEM_F32 ? 4u : 2u; }

uint64_t tiles_of(int64_t elements, int type)
{
    const uint64_t per = (uint64_t)mxq::kClipTileVecs * 16 / elem_bytes(type);
    return ((uint64_t)elements + per - 1) / per;
}

int check_tensors(const int64_t *elements, const int *types, int64_t count)
{
    if (count < 0)
        return MXQ_E_ROWS;
    if (count > 0 && (!elements || !types))
        return MXQ_E_NULL;
    for (int64_t i = 0; i < count; i++) {
        if (types[i] != MXQ_ELEM_BF16 && types[i] != MXQ_ELEM_F16 && types[i] != MXQ_ELEM_F32)
            return MXQ_E_ELEM_DTYPE;
        if (elements[i] < 0)
            return MXQ_E_ROWS;
        if (elements[i] > kMaxElements)
            return MXQ_E_OVERFLOW;
    }
    return MXQ_OK;
}

// The next launch's table from tensor `*next` on: up to kClipTensors tensors
// that have elements, and at most kMaxTiles. Returns its workgroups.
uint32_t fill(mxq::ClipTable &t, const void *const *in, void *const *out, const int64_t *elements, const int *types,
              int64_t count, int64_t *next)
{
    uint64_t tiles = 0;
    t.tensors = 0;
    t.first_tile[0] = 0;
    for (; *next < count && t.tensors < mxq::kClipTensors; ++*next) {
        const int64_t i = *next;
        if (elements[i] == 0)
            continue;
        const uint64_t more = tiles_of(elements[i], types[i]);
        if (tiles + more > kMaxTiles)
            break;
        tiles += more;
        t.in[t.tensors] = in ? in[i] : nullptr;
        t.out[t.tensors] = out ? out[i] : nullptr;
        t.elements[t.tensors] = (uint64_t)elements[i];
        t.type[t.tensors] = (uint8_t)types[i];
        t.first_tile[++t.tensors] = (uint32_t)tiles;
    }
    return tiles < kClipBlocks ? (uint32_t)tiles : kClipBlocks;
}

// Partial sums of all launches.
int64_t partials(const int64_t *elements, const int *types, int64_t count)
{
    mxq::ClipTable t;
    int64_t n = 0;
    for (int64_t next = 0; next < count;)
        n += fill(t, nullptr, nullptr, elements, types, count, &next);
    return n;
}

} // namespace

extern "C" {

size_t mxq_clip_grad_norm_workspace_bytes(const int64_t *elements, const int *elem_dtypes, int64_t count)
{
    if (check_tensors(elements, elem_dtypes, count) != MXQ_OK)
        return 0;
    return (size_t)(partials(elements, elem_dtypes, count) + 1) * 8;
}

int mxq_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *elements, const int *elem_dtypes,
                       int64_t count, double max_norm, float *norm, void *workspace, void *stream)
{
    int rc = check_tensors(elements, elem_dtypes, count);
    if (rc != MXQ_OK)
        return rc;
    if (outs && !(max_norm >= 0.0))
        return MXQ_E_VALUE;
    if (!norm || !workspace || (count > 0 && !grads))
        return MXQ_E_NULL;
    if (((uintptr_t)norm & 3u) || ((uintptr_t)workspace & 15u))
        return MXQ_E_ALIGN;
    bool in_place = true;
    for (int64_t i = 0; i < count; i++) {
        if (elements[i] == 0)
            continue;
        if (!grads[i] || (outs && !outs[i]))
            return MXQ_E_NULL;
        // tensors may start at any of their elements
        if (((uintptr_t)grads[i] | (outs ? (uintptr_t)outs[i] : 0)) & (elem_bytes(elem_dtypes[i]) - 1))
            return MXQ_E_ALIGN;
        in_place = in_place && outs && outs[i] == grads[i];
    }

    mxq::ClipTable t;
    double *partial = (double *)workspace;
    uint32_t total = 0, most = 0;   // partial sums; tiles of the largest launch
    int launches = 0;
    hipError_t err = hipSuccess;
    for (int64_t next = 0; next < count && err == hipSuccess;) {
        const uint32_t blocks = fill(t, grads, outs, elements, elem_dtypes, count, &next);
        if (blocks == 0)
            continue;
        double *here = partial + total;
        void *args[] = {&t, &here};
        err = hipLaunchKernel((const void *)mxq::clip_norm_kernel, dim3(blocks), dim3(mxq::kClipThreads), args, 0,
                              (hipStream_t)stream);
        total += blocks;
        most = t.first_tile[t.tensors] > most ? t.first_tile[t.tensors] : most;
        launches++;
    }
    // One launch's partial sums are added by the scaling pass itself, every
    // workgroup reading all of them; of several, or where there are many
    // tiles (a workgroup for each then), or where nothing is scaled, by a
    // launch of its own.
    const bool own_total = !outs || launches != 1 || most > 2 * kClipBlocks;
    if (own_total && err == hipSuccess) {
        void *args[] = {&partial, &total, &norm};
        err = hipLaunchKernel((const void *)mxq::clip_total_kernel, dim3(1), dim3(mxq::kClipThreads), args, 0,
                              (hipStream_t)stream);
    }
    if (!outs || launches == 0)
        return err == hipSuccess ? MXQ_OK : MXQ_E_HIP;
    const double *sums = own_total ? partial + total : partial;
    uint32_t n = own_total ? 1u : total, place = in_place ? 1u : 0u;
    float *norm_out = own_total ? nullptr : norm;
    for (int64_t next = 0; next < count && err == hipSuccess;) {
        const uint32_t blocks = fill(t, grads, outs, elements, elem_dtypes, count, &next);
        if (blocks == 0)
            continue;
        void *args[] = {&t, &sums, &n, &max_norm, &place, &norm_out};
        const uint32_t tiles = t.first_tile[t.tensors];
        err = hipLaunchKernel((const void *)mxq::clip_scale_kernel, dim3(own_total ? tiles : blocks),
                              dim3(mxq::kClipThreads), args, 0, (hipStream_t)stream);
    }
    return err == hipSuccess ? MXQ_OK : MXQ_E_HIP;
}

} // extern "C"
