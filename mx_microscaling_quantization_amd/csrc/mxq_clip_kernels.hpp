// mxq_clip_kernels.hpp -- gfx950 kernels of the global norm over many tensors
// and of clipping them by it.
//
//   norm   = sqrt(sum over all tensors and elements of g^2)
//   factor = max_norm / norm where max_norm < norm < infinity, else 1
//   out    = round(g * factor)
//
// The squares are added in 64 bits: a square of any finite element neither
// overflows nor vanishes there, and the norm of 2^40 elements is good to the
// last bits of its 32-bit result. One pass reads every element once and
// leaves one partial sum per workgroup; the scaling pass reads the partial
// sums (every workgroup adds all of them, in the same order, so all of them
// use the same factor) and each element once more. Nothing depends on the
// order in which workgroups run.
//
// Tensors are cut into tiles of 32 KiB, 8 vectors of 16 bytes per thread. The
// tensors' addresses travel in the kernel's arguments, so a call copies nothing
// to the device and can be captured in a graph; a launch holds up to
// kClipTensors of them, and a workgroup looks its tile's tensor up there.
//
// Bound by memory: 48 bf16 tensors of 8.4 M elements, norm alone 140 us (5.7
// TB/s of reads), scaled into others 390 us (6.2 TB/s of three passes).
// Workgroups in flight work on neighbouring tiles (contiguous shares of the
// tiles per workgroup: 434 us), the scaling's last loads and its stores are
// non-temporal (both ordinary: 434 us), and a large scaling has a workgroup
// per tile, which ends without waiting for its stores (2048 workgroups that
// take tiles in turn: 424 us, also with the next tile's loads ahead).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_moe_kernels.hpp"

namespace mxq {

constexpr uint32_t kClipTensors = 112;   // 112 * 32 bytes of table: under the 4 KiB of a kernel's arguments
constexpr uint32_t kClipThreads = 256;
constexpr uint32_t kClipVecs = 8;       // vectors of 16 bytes per thread and tile
constexpr uint32_t kClipTileVecs = kClipVecs * kClipThreads;

struct ClipTable {
    const void *in[kClipTensors];
    void *out[kClipTensors];
    uint64_t elements[kClipTensors];
    uint32_t first_tile[kClipTensors + 1];
    uint8_t type[kClipTensors];
    uint32_t tensors;
};
static_assert(sizeof(ClipTable) <= 3900, "a kernel's arguments are limited to 4 KiB");

// Tensor of tile `tile`: the last one whose first tile is not past it.
__device__ __forceinline__ uint32_t clip_find(const ClipTable &t, uint32_t tile)
{
    uint32_t lo = 0, hi = t.tensors - 1;
    while (lo < hi) {
        const uint32_t mid = (lo + hi + 1) / 2;
        if (t.first_tile[mid] <= tile)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// A thread's part of a tile: kClipVecs vectors of 16 bytes, 256 vectors apart. Bytes
// past the tensor are zeros.
struct ClipPart {
    u32x4_any_t v[kClipVecs];
    uint32_t type;
    uint8_t *out;      // the part's first byte of the result
    uint64_t left;     // bytes from there to the tensor's end (0: none)
};

// Its place: tensor `n` is looked up from the one of the tile before or after.
__device__ __forceinline__ const uint8_t *clip_place(const ClipTable &t, uint32_t tile, uint32_t &n, ClipPart &part)
{
    while (tile >= t.first_tile[n + 1])
        n++;
    while (tile < t.first_tile[n])
        n--;
    part.type = t.type[n];
    const uint64_t bytes = t.elements[n] * (part.type == kElemF32 ? 4u : 2u);
    const uint64_t at = (uint64_t)(tile - t.first_tile[n]) * (kClipTileVecs * 16u) + threadIdx.x * 16u;
    part.out = (uint8_t *)t.out[n] + at;
    part.left = at < bytes ? bytes - at : 0;
    return (const uint8_t *)t.in[n] + at;
}

template <int NT> __device__ __forceinline__ void clip_load(const uint8_t *p, ClipPart &part)
{
#pragma unroll
    for (uint32_t i = 0; i < kClipVecs; i++) {
        const uint32_t skip = i * kClipThreads * 16u;
        if (part.left >= skip + 16u) {
            const u32x4_any_t *q = reinterpret_cast<const u32x4_any_t *>(p + skip);
            part.v[i] = NT ? __builtin_nontemporal_load(q) : *q;
        } else {
            u32x4_any_t v = {0u, 0u, 0u, 0u};
#pragma unroll
            for (uint32_t k = 0; k < 8; k++)
                if (part.left > skip + 2u * k)
                    v[k / 2] |= (uint32_t)*reinterpret_cast<const uint16_t *>(p + skip + 2u * k) << (16u * (k & 1u));
            part.v[i] = v;
        }
    }
}

template <int DT> __device__ __forceinline__ double clip_squares(const ClipPart &part)
{
    constexpr uint32_t V = Elem<DT>::vec;
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (uint32_t i = 0; i < kClipVecs; i++) {
        float f[V];
        elems_to_f32<DT>(__builtin_bit_cast(ElemVec<DT>, part.v[i]), f);
#pragma unroll
        for (uint32_t k = 0; k < V; k += 2) {
            const double a = f[k], b = f[k + 1];
            s0 = __builtin_fma(a, a, s0);
            s1 = __builtin_fma(b, b, s1);
        }
    }
    return s0 + s1;
}

// F: float, or double for a factor below fp32's normal numbers.
template <int DT, typename F> __device__ __forceinline__ void clip_store(const ClipPart &part, F factor)
{
    typedef typename Elem<DT>::type T;
    constexpr uint32_t V = Elem<DT>::vec, S = sizeof(T);
#pragma unroll
    for (uint32_t i = 0; i < kClipVecs; i++) {
        const uint64_t skip = i * kClipThreads * 16u;
        float f[V];
        elems_to_f32<DT>(__builtin_bit_cast(ElemVec<DT>, part.v[i]), f);
#pragma unroll
        for (uint32_t k = 0; k < V; k++)
            f[k] = (float)(f[k] * factor);
        const uint64_t n = part.left > skip ? (part.left - skip) / S : 0;
        store_elems<DT, 1>((T *)(part.out + skip), n < V ? (uint32_t)n : V, f);
    }
}

template <typename F> __device__ __forceinline__ void clip_store_as(const ClipPart &part, F factor)
{
    if (part.type == kElemBF16)
        clip_store<kElemBF16>(part, factor);
    else if (part.type == kElemF16)
        clip_store<kElemF16>(part, factor);
    else
        clip_store<kElemF32>(part, factor);
}

// The workgroup's sum of `v`, in a fixed order, in every thread.
__device__ __forceinline__ double clip_block_sum(double v, double *lds)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d);
    __syncthreads();
    if ((threadIdx.x & 63u) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// The sum of `count` partial sums, in every thread.
__device__ __forceinline__ double clip_total(const double *partial, uint32_t count, double *lds)
{
    double s = 0.0;
    for (uint32_t i = threadIdx.x; i < count; i += kClipThreads)
        s += partial[i];
    return clip_block_sum(s, lds);
}

__global__ __launch_bounds__(kClipThreads) void clip_norm_kernel(ClipTable table, double *__restrict__ partial)
{
    __shared__ double lds[4];
    const uint32_t tiles = table.first_tile[table.tensors];
    uint32_t tile = blockIdx.x;
    double sum = 0.0;
    if (tile < tiles) {
        uint32_t n = clip_find(table, tile);
        for (; tile < tiles; tile += gridDim.x) {
            ClipPart part;
            clip_load<0>(clip_place(table, tile, n, part), part);
            if (part.type == kElemBF16)
                sum += clip_squares<kElemBF16>(part);
            else if (part.type == kElemF16)
                sum += clip_squares<kElemF16>(part);
            else
                sum += clip_squares<kElemF32>(part);
        }
    }
    sum = clip_block_sum(sum, lds);
    if (threadIdx.x == 0)
        partial[blockIdx.x] = sum;
}

// The partial sums of several launches into one (partial[count]), and the norm.
__global__ __launch_bounds__(kClipThreads) void clip_total_kernel(double *__restrict__ partial, uint32_t count,
                                                                  float *__restrict__ norm)
{
    __shared__ double lds[4];
    const double total = clip_total(partial, count, lds);
    if (threadIdx.x == 0) {
        partial[count] = total;
        norm[0] = (float)__builtin_sqrt(total);
    }
}

// Tiles are taken from the last one back: what the norm pass read last is what
// the caches still hold. `in_place`: every tensor's
// result goes over its input, so a factor of 1 leaves nothing to do.
__global__ __launch_bounds__(kClipThreads) void clip_scale_kernel(ClipTable table,
                                                                  const double *__restrict__ partial, uint32_t count,
                                                                  double max_norm, uint32_t in_place,
                                                                  float *__restrict__ norm_out)
{
    __shared__ double lds[4];
    const double norm = __builtin_sqrt(clip_total(partial, count, lds));
    if (norm_out && blockIdx.x == 0 && threadIdx.x == 0)
        norm_out[0] = (float)norm;
    const bool clip = norm > max_norm && norm < __builtin_inf();
    if (in_place && !clip)
        return;
    // the factor is rounded to fp32 but where that would leave it fewer bits (a norm
    // of 1e41, which only the 64-bit sum holds, clipped to 1): products in 64 bits,
    // rounded once, then
    const double exact = clip ? max_norm / norm : 1.0;
    const float factor = (float)exact;
    const bool tiny = exact < 0x1p-126;
    const uint32_t tiles = table.first_tile[table.tensors];
    uint32_t back = blockIdx.x;   // tiles from the end
    if (back >= tiles)
        return;
    uint32_t n = clip_find(table, tiles - 1 - back);
    for (; back < tiles; back += gridDim.x) {
        ClipPart part;
        clip_load<1>(clip_place(table, tiles - 1 - back, n, part), part);
        if (tiny)
            clip_store_as(part, exact);
        else
            clip_store_as(part, factor);
    }
}

} // namespace mxq
