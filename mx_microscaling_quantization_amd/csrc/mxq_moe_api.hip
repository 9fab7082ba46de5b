// mxq_moe_api.hip -- mxq_moe_sort, mxq_moe_gather_quantize, mxq_moe_combine
// and mxq_moe_combine_backward: validation, launch geometry and dispatch of
// the kernels in mxq_moe_kernels.hpp on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq.h"
#include "mxq_host.hpp"
#include "mxq_moe_kernels.hpp"

namespace {

using mxq_host::check_shape;
using mxq_host::emax_of;
using mxq_host::grid_fits;
using mxq_host::kMaxF;

// Pairs, sorted rows and the numbers in between are 32-bit in the kernels.
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 65536;

int check_pairs(int64_t tokens, int64_t slots)
{
    if (tokens < 0 || slots < 1 || slots > MXQ_MOE_MAX_SLOTS)
        return MXQ_E_MOE;
    return tokens > kMaxRows / slots ? MXQ_E_OVERFLOW : MXQ_OK;
}

int check_rows(int64_t rows)
{
    if (rows < 0 || rows % 4 != 0)
        return MXQ_E_ROWS;
    return rows > kMaxRows ? MXQ_E_OVERFLOW : MXQ_OK;
}

bool misaligned(const void *a, const void *b = nullptr, const void *c = nullptr, const void *d = nullptr,
                const void *e = nullptr, const void *f = nullptr)
{
    return ((uintptr_t)a | (uintptr_t)b | (uintptr_t)c | (uintptr_t)d | (uintptr_t)e | (uintptr_t)f) & 15u;
}

int status_of(hipError_t err) { return err == hipSuccess ? MXQ_OK : MXQ_E_HIP; }

// ---- sort ------------------------------------------------------------------

// One workgroup up to this many pairs (4096 pairs: 7.9 us; 8192: 12.2 us in
// one workgroup, 8.7 in two launches).
constexpr int64_t kSortOneBlock = 4096;

// Workgroups of a longer list: 2048 pairs each, 4096 where every workgroup's
// reading all chunks' counts would be the larger part (524288 pairs and 256
// experts: 17.3 us with 2048, 14.9 with 4096; with 8 experts 10.4 and 11.0),
// and more where that makes more than kSortBlocks.
int64_t sort_blocks(int64_t pairs, int64_t experts)
{
    if (pairs <= kSortOneBlock)
        return 1;
    int64_t b = (pairs + 2047) / 2048;
    if (b * b * experts * 4 > 32 << 20)
        b = (pairs + 4095) / 4096;
    return b < mxq::kSortBlocks ? b : mxq::kSortBlocks;
}

template <typename ID>
int sort_launch(const void *ids_, int64_t pairs, int64_t experts, int64_t align, int64_t rows, int32_t *offsets,
                int32_t *src, int32_t *dest, void *workspace, hipStream_t stream)
{
    const int64_t blocks = sort_blocks(pairs, experts);
    const int64_t step = mxq::kSortThreads;   // 64 pairs per wave
    const ID *ids = (const ID *)ids_;
    uint32_t n = (uint32_t)pairs, chunk = (uint32_t)((pairs + blocks * step - 1) / (blocks * step) * step);
    uint32_t e = (uint32_t)experts, pitch = (e + 3u) & ~3u, a = (uint32_t)align, r = (uint32_t)rows, bits = 0;
    while ((1u << bits) < e)
        bits++;
    uint32_t *counts = (uint32_t *)workspace;
    if (blocks > 1) {
        void *args[] = {&ids, &n, &chunk, &e, &pitch, &counts};
        const hipError_t err = hipLaunchKernel((const void *)mxq::sort_count_kernel<ID>, dim3((uint32_t)blocks),
                                               dim3(mxq::kSortThreads), args, 4 * pitch, stream);
        if (err != hipSuccess)
            return MXQ_E_HIP;
    }
    const void *k = blocks > 1 ? (const void *)mxq::sort_place_kernel<ID, 0>
                               : (const void *)mxq::sort_place_kernel<ID, 1>;
    void *args[] = {&ids, &n, &chunk, &e, &pitch, &a, &r, &bits, &counts, &offsets, &src, &dest};
    return status_of(hipLaunchKernel(k, dim3((uint32_t)blocks), dim3(mxq::kSortThreads), args,
                                     4 * (e * mxq::kSortWaves + pitch * 3), stream));
}

// ---- gather and quantize ---------------------------------------------------

typedef void (*along_fn)(const uint16_t *, const int32_t *, uint32_t, uint32_t, uint32_t, uint32_t, uint64_t, uint32_t,
                         int, uint32_t, uint8_t *, uint8_t *);
typedef void (*down_fn)(const uint16_t *, const int32_t *, uint32_t, uint32_t, uint32_t, uint32_t, uint64_t, uint32_t,
                        uint32_t, int, uint32_t, uint8_t *, uint8_t *);

template <int IN> along_fn along_pick(int out)
{
    switch (out) {
    case MXQ_OUT_E4M3FN: return mxq::gather_quantize_along_kernel<IN, mxq::kOutE4M3FN>;
    case MXQ_OUT_E5M2: return mxq::gather_quantize_along_kernel<IN, mxq::kOutE5M2>;
    default: return mxq::gather_quantize_along_kernel<IN, mxq::kOutE2M1>;
    }
}

template <int IN, int OUT> down_fn down_pick_nb(int nb, bool runs)
{
    switch (nb) {
    case 4: return runs ? mxq::gather_quantize_down_kernel<IN, OUT, 4, 1>
                        : mxq::gather_quantize_down_kernel<IN, OUT, 4, 0>;
    case 2: return mxq::gather_quantize_down_kernel<IN, OUT, 2, 0>;
    default: return mxq::gather_quantize_down_kernel<IN, OUT, 1, 0>;
    }
}

template <int IN> down_fn down_pick(int out, int nb, bool runs)
{
    switch (out) {
    case MXQ_OUT_E4M3FN: return down_pick_nb<IN, mxq::kOutE4M3FN>(nb, runs);
    case MXQ_OUT_E5M2: return down_pick_nb<IN, mxq::kOutE5M2>(nb, runs);
    default: return down_pick_nb<IN, mxq::kOutE2M1>(nb, runs);
    }
}

// ---- combine ---------------------------------------------------------------

// Lanes per token: as many as a row has vectors, in steps of 2 from 4 to 64.
int lanes_for(int64_t vecs)
{
    return vecs <= 4 ? 4 : vecs <= 8 ? 8 : vecs <= 16 ? 16 : vecs <= 32 ? 32 : 64;
}

template <int DT, int WEIGHTED> const void *combine_pick(int lanes)
{
    switch (lanes) {
    case 4: return (const void *)mxq::combine_kernel<DT, WEIGHTED, 4>;
    case 8: return (const void *)mxq::combine_kernel<DT, WEIGHTED, 8>;
    case 16: return (const void *)mxq::combine_kernel<DT, WEIGHTED, 16>;
    case 32: return (const void *)mxq::combine_kernel<DT, WEIGHTED, 32>;
    default: return (const void *)mxq::combine_kernel<DT, WEIGHTED, 64>;
    }
}

template <int DT>
int combine_launch(const void *y_, int64_t rows, int64_t N, const int32_t *dest, const float *weights, int64_t tokens,
                   int64_t slots, void *out_, hipStream_t stream)
{
    typedef typename mxq::Elem<DT>::type T;
    const int64_t vecs = (N + mxq::Elem<DT>::vec - 1) / mxq::Elem<DT>::vec;
    const int lanes = lanes_for(vecs);
    const int64_t parts = lanes == 64 ? (vecs + 63) / 64 : 1, per = 256 / lanes;
    if (!grid_fits(tokens, parts, lanes) || !grid_fits((tokens * parts + per - 1) / per, 1, 256))
        return MXQ_E_OVERFLOW;
    T *out = (T *)out_;
    const T *y = rows > 0 ? (const T *)y_ : out;   // row 0 is read (and not used) for a pair without a row
    uint32_t r = (uint32_t)rows, n = (uint32_t)N, v = (uint32_t)vecs, p = (uint32_t)parts, t = (uint32_t)tokens,
             s = (uint32_t)slots;
    const void *k = weights ? combine_pick<DT, 1>(lanes) : combine_pick<DT, 0>(lanes);
    void *args[] = {&y, &r, &n, &v, &p, &dest, &weights, &t, &s, &out};
    return status_of(hipLaunchKernel(k, dim3((uint32_t)((tokens * parts + per - 1) / per)), dim3(256), args, 0,
                                     stream));
}

template <int DT> const void *combine_backward_pick(int lanes, int64_t vecs)
{
    switch (lanes) {
    case 4: return (const void *)mxq::combine_backward_kernel<DT, 4, 1>;
    case 8: return (const void *)mxq::combine_backward_kernel<DT, 8, 1>;
    case 16: return (const void *)mxq::combine_backward_kernel<DT, 16, 1>;
    case 32: return (const void *)mxq::combine_backward_kernel<DT, 32, 1>;
    default: break;
    }
    return vecs <= 64 ? (const void *)mxq::combine_backward_kernel<DT, 64, 1>
                      : (const void *)mxq::combine_backward_kernel<DT, 64, 2>;
}

template <int DT>
int combine_backward_launch(const void *grad_, const void *y_, int64_t rows, int64_t N, const int32_t *src,
                            const int32_t *dest, const float *weights, int64_t tokens, int64_t slots, void *grad_y_,
                            float *grad_w, hipStream_t stream)
{
    typedef typename mxq::Elem<DT>::type T;
    const int64_t vecs = (N + mxq::Elem<DT>::vec - 1) / mxq::Elem<DT>::vec;
    const int lanes = lanes_for(vecs);
    const int64_t pairs = tokens * slots, per = 256 / lanes;
    const int64_t row_blocks = (rows + per - 1) / per, pair_blocks = (pairs + 255) / 256;
    if (!grid_fits(row_blocks + pair_blocks, 1, 256))
        return MXQ_E_OVERFLOW;
    const T *grad = (const T *)grad_, *y = (const T *)y_;
    T *grad_y = (T *)grad_y_;
    uint32_t r = (uint32_t)rows, n = (uint32_t)N, v = (uint32_t)vecs, p = (uint32_t)pairs, s = (uint32_t)slots;
    uint32_t b = (uint32_t)row_blocks;
    void *args[] = {&grad, &y, &r, &n, &v, &src, &dest, &weights, &p, &s, &b, &grad_y, &grad_w};
    return status_of(hipLaunchKernel(combine_backward_pick<DT>(lanes, vecs), dim3((uint32_t)(row_blocks + pair_blocks)),
                                     dim3(256), args, 0, stream));
}

int check_elem(int elem_dtype)
{
    return elem_dtype == MXQ_ELEM_BF16 || elem_dtype == MXQ_ELEM_F16 || elem_dtype == MXQ_ELEM_F32 ? MXQ_OK
                                                                                                 : MXQ_E_ELEM_DTYPE;
}

// Checks shared by combine and its gradient.
int check_combine(int64_t rows, int64_t N, int elem_dtype, int64_t tokens, int64_t slots)
{
    int rc = check_elem(elem_dtype);
    if (rc == MXQ_OK)
        rc = check_pairs(tokens, slots);
    if (rc != MXQ_OK)
        return rc;
    if (rows < 0 || N < 0)
        return MXQ_E_ROWS;
    return rows > kMaxRows || N > kMaxF / 2 ? MXQ_E_OVERFLOW : MXQ_OK;
}

} // namespace

extern "C" {

int64_t mxq_moe_rows(int64_t tokens, int64_t slots, int64_t experts, int64_t align)
{
    if (check_pairs(tokens, slots) != MXQ_OK || experts < 1 || experts > MXQ_MOE_MAX_EXPERTS || align < 4 ||
        align > MXQ_MOE_MAX_ALIGN || align % 4 != 0)
        return -1;
    const int64_t pairs = tokens * slots, used = experts < pairs ? experts : pairs;
    const int64_t rows = (pairs + used * (align - 1)) / align * align;
    return rows > kMaxRows ? -1 : rows;
}

size_t mxq_moe_sort_workspace_bytes(int64_t tokens, int64_t slots, int64_t experts)
{
    if (check_pairs(tokens, slots) != MXQ_OK || experts < 1 || experts > MXQ_MOE_MAX_EXPERTS)
        return 0;
    const int64_t blocks = sort_blocks(tokens * slots, experts);
    return blocks > 1 ? (size_t)(blocks * ((experts + 3) / 4 * 4) * 4) : 0;
}

int mxq_moe_sort(const void *ids, int id_bytes, int64_t tokens, int64_t slots, int64_t experts, int64_t align,
                 int32_t *offsets, int32_t *src, int32_t *dest, void *workspace, void *stream)
{
    if (id_bytes != 4 && id_bytes != 8)
        return MXQ_E_ELEM_DTYPE;
    int rc = check_pairs(tokens, slots);
    if (rc != MXQ_OK)
        return rc;
    if (experts < 1 || experts > MXQ_MOE_MAX_EXPERTS || align < 4 || align > MXQ_MOE_MAX_ALIGN || align % 4 != 0)
        return MXQ_E_MOE;
    const int64_t rows = mxq_moe_rows(tokens, slots, experts, align);
    if (rows < 0)
        return MXQ_E_OVERFLOW;
    const int64_t pairs = tokens * slots;
    if (!offsets || (pairs > 0 && (!ids || !src || !dest)) ||
        (mxq_moe_sort_workspace_bytes(tokens, slots, experts) > 0 && !workspace))
        return MXQ_E_NULL;
    if (misaligned(ids, offsets, src, dest, workspace))
        return MXQ_E_ALIGN;
    // no pairs: one workgroup writes the offsets, all zero
    return id_bytes == 4
               ? sort_launch<int32_t>(ids, pairs, experts, align, rows, offsets, src, dest, workspace,
                                      (hipStream_t)stream)
               : sort_launch<int64_t>(ids, pairs, experts, align, rows, offsets, src, dest, workspace,
                                      (hipStream_t)stream);
}

int mxq_moe_gather_quantize(const void *x, int64_t tokens, int64_t slots, int64_t K, int in_dtype, int out_dtype,
                            int dim, unsigned flags, const int32_t *src, int64_t rows, void *data_out,
                            void *scale_out, void *stream)
{
    if (in_dtype != MXQ_IN_BF16 && in_dtype != MXQ_IN_F16)
        return MXQ_E_IN_DTYPE;
    if (out_dtype != MXQ_OUT_E4M3FN && out_dtype != MXQ_OUT_E5M2 && out_dtype != MXQ_OUT_E2M1)
        return MXQ_E_OUT_DTYPE;
    if (flags & ~(unsigned)(MXQ_FLAG_ALT_EMAX | MXQ_FLAG_DENSE_SCALE))
        return MXQ_E_FLAGS;
    if (dim < 0)
        dim += 2;
    if (dim != 0 && dim != 1)
        return MXQ_E_DIM;
    int rc = check_pairs(tokens, slots);
    if (rc == MXQ_OK)
        rc = check_rows(rows);
    if (rc != MXQ_OK)
        return rc;
    if (K < 0)
        return MXQ_E_SHAPE_F4;
    const bool down = dim == 0;
    const int64_t B = down ? rows : K, O = down ? K : rows;   // block axis and the other
    if (B % 32 != 0)
        return MXQ_E_SHAPE_P8;
    if (O > kMaxF / 4 || K > kMaxF)
        return MXQ_E_OVERFLOW;
    rc = check_shape(B / 4, 4 * O);
    if (rc != MXQ_OK)
        return rc;
    if (rows == 0 || K == 0)
        return MXQ_OK;
    // without tokens every row is empty and x is never read for its values,
    // but a lane without a token reads its first row: ask for one
    if (tokens == 0)
        return MXQ_E_ROWS;
    if (!x || !src || !data_out || !scale_out)
        return MXQ_E_NULL;
    if (misaligned(x, src, data_out, scale_out))
        return MXQ_E_ALIGN;

    const uint16_t *a0 = (const uint16_t *)x;
    const int32_t *a1 = src;
    uint32_t a2 = (uint32_t)rows, a3 = (uint32_t)(tokens * slots);
    uint32_t shift = 31; // slot_div's constants
    while ((1ll << (shift - 31)) < slots)
        shift++;
    uint32_t mul = (uint32_t)((((uint64_t)1 << shift) + slots - 1) / slots);
    uint64_t a5 = (uint64_t)K;
    int bias = emax_of(out_dtype) - ((flags & MXQ_FLAG_ALT_EMAX) ? 1 : 0);
    uint32_t dense = (flags & MXQ_FLAG_DENSE_SCALE) ? 1u : 0u;
    uint8_t *d = (uint8_t *)data_out, *s = (uint8_t *)scale_out;
    if (down) {
        const int nb = K % 4 == 0 ? 4 : K % 2 == 0 ? 2 : 1;   // columns per thread
        const int64_t strips = K / nb, tiles = (strips + 63) / 64;
        if (!grid_fits(rows / 32, tiles, 64))
            return MXQ_E_OVERFLOW;
        // rows are read again (more than one slot), x does not fit the XCDs'
        // L2s as it is (4 MiB each), and one run of its columns fits one (run by run
        // and band by band: 4096 x 8 rows of 4096 36 and 36 us, 8192 x 8 61 and 89;
        // beyond one L2 the gain is smaller and the order is not used: 16384 x 4 rows
        // 94 and 104, 16384 x 8 177 and 204)
        const bool runs = slots > 1 && tokens * K * 2 > 8 * (4 << 20) && tokens * 512 <= 4 << 20;
        down_fn k = in_dtype == MXQ_IN_BF16 ? down_pick<mxq::kInBF16>(out_dtype, nb, runs)
                                            : down_pick<mxq::kInF16>(out_dtype, nb, runs);
        uint32_t a6 = (uint32_t)strips, a7 = (uint32_t)tiles;
        void *args[] = {&a0, &a1, &a2, &a3, &mul, &shift, &a5, &a6, &a7, &bias, &dense, &d, &s};
        return status_of(hipLaunchKernel((const void *)k, dim3((uint32_t)(rows / 32 * tiles)), dim3(64), args, 0,
                                         (hipStream_t)stream));
    }
    const int64_t tiles = (rows + mxq::kAlongRows - 1) / mxq::kAlongRows, ktiles = (K / 32 + 1) / 2;
    if (!grid_fits(ktiles, tiles, 64 * mxq::kAlongWaves))
        return MXQ_E_OVERFLOW;
    along_fn k = in_dtype == MXQ_IN_BF16 ? along_pick<mxq::kInBF16>(out_dtype) : along_pick<mxq::kInF16>(out_dtype);
    uint32_t a6 = (uint32_t)tiles;
    void *args[] = {&a0, &a1, &a2, &a3, &mul, &shift, &a5, &a6, &bias, &dense, &d, &s};
    return status_of(hipLaunchKernel((const void *)k, dim3((uint32_t)(ktiles * tiles)), dim3(64 * mxq::kAlongWaves),
                                     args, 0, (hipStream_t)stream));
}

int mxq_moe_combine(const void *y, int64_t rows, int64_t N, int elem_dtype, const int32_t *dest,
                    const float *weights, int64_t tokens, int64_t slots, void *out, void *stream)
{
    const int rc = check_combine(rows, N, elem_dtype, tokens, slots);
    if (rc != MXQ_OK)
        return rc;
    if (tokens == 0 || N == 0)
        return MXQ_OK;
    if ((rows > 0 && !y) || !dest || !out)
        return MXQ_E_NULL;
    if (misaligned(y, dest, weights, out))
        return MXQ_E_ALIGN;
    hipStream_t st = (hipStream_t)stream;
    switch (elem_dtype) {
    case MXQ_ELEM_BF16: return combine_launch<mxq::kElemBF16>(y, rows, N, dest, weights, tokens, slots, out, st);
    case MXQ_ELEM_F16: return combine_launch<mxq::kElemF16>(y, rows, N, dest, weights, tokens, slots, out, st);
    default: return combine_launch<mxq::kElemF32>(y, rows, N, dest, weights, tokens, slots, out, st);
    }
}

int mxq_moe_combine_backward(const void *grad, const void *y, int64_t rows, int64_t N, int elem_dtype,
                             const int32_t *src, const int32_t *dest, const float *weights, int64_t tokens,
                             int64_t slots, void *grad_y, float *grad_weights, void *stream)
{
    const int rc = check_combine(rows, N, elem_dtype, tokens, slots);
    if (rc != MXQ_OK)
        return rc;
    if (tokens == 0 && (rows == 0 || N == 0))
        return MXQ_OK;
    // N == 0 still has weight gradients: zeros
    if ((tokens > 0 && (!dest || !weights || !grad_weights)) || (rows > 0 && !src) ||
        (N > 0 && ((tokens > 0 && !grad) || (rows > 0 && (!y || !grad_y)))))
        return MXQ_E_NULL;
    if (misaligned(grad, y, src, dest, weights, grad_y) || misaligned(grad_weights))
        return MXQ_E_ALIGN;
    hipStream_t st = (hipStream_t)stream;
    switch (elem_dtype) {
    case MXQ_ELEM_BF16:
        return combine_backward_launch<mxq::kElemBF16>(grad, y, rows, N, src, dest, weights, tokens, slots, grad_y,
                                                       grad_weights, st);
    case MXQ_ELEM_F16:
        return combine_backward_launch<mxq::kElemF16>(grad, y, rows, N, src, dest, weights, tokens, slots, grad_y,
                                                      grad_weights, st);
    default:
        return combine_backward_launch<mxq::kElemF32>(grad, y, rows, N, src, dest, weights, tokens, slots, grad_y,
                                                      grad_weights, st);
    }
}

} // extern "C"
