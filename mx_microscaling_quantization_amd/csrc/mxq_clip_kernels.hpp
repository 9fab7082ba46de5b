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
// Tensors are cut into tiles of 1024 16-byte vectors. A workgroup takes a
// contiguous range of the launch's tiles and looks up the first one's tensor
// once. The tensors' addresses travel in the kernel's arguments, so a call
// copies nothing to the device and can be captured in a graph; a launch holds
// up to kClipTensors of them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxq_moe_kernels.hpp"

namespace mxq {

constexpr uint32_t kClipTensors = 112;   // 112 * 32 bytes of table: under the 4 KiB of a kernel's arguments
constexpr uint32_t kClipThreads = 256;
constexpr uint32_t kClipTileVecs = 1024; // 16 KiB: 4 vectors per thread

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

template <int DT> __device__ __forceinline__ double clip_tile_sum(const void *in, uint64_t elements, uint64_t tile)
{
    typedef typename Elem<DT>::type T;
    constexpr uint32_t V = Elem<DT>::vec;
    const T *p = (const T *)in;
    const uint64_t first = tile * kClipTileVecs * V + (uint64_t)threadIdx.x * V;
    double s0 = 0.0, s1 = 0.0;
    float f[4][V];
#pragma unroll
    for (uint32_t i = 0; i < 4; i++) {
        const uint64_t at = first + (uint64_t)i * kClipThreads * V;
        const uint64_t left = at < elements ? elements - at : 0;
        load_elems<DT>(p + at, left < V ? (uint32_t)left : V, f[i]);
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; i++)
#pragma unroll
        for (uint32_t k = 0; k < V; k += 2) {
            const double a = f[i][k], b = f[i][k + 1];
            s0 = __builtin_fma(a, a, s0);
            s1 = __builtin_fma(b, b, s1);
        }
    return s0 + s1;
}

template <int DT>
__device__ __forceinline__ void clip_tile_scale(const void *in, void *out, uint64_t elements, uint64_t tile,
                                                float factor)
{
    typedef typename Elem<DT>::type T;
    constexpr uint32_t V = Elem<DT>::vec;
    const uint64_t first = tile * kClipTileVecs * V + (uint64_t)threadIdx.x * V;
    float f[4][V];
#pragma unroll
    for (uint32_t i = 0; i < 4; i++) {
        const uint64_t at = first + (uint64_t)i * kClipThreads * V;
        const uint64_t left = at < elements ? elements - at : 0;
        load_elems<DT>((const T *)in + at, left < V ? (uint32_t)left : V, f[i]);
    }
#pragma unroll
    for (uint32_t i = 0; i < 4; i++) {
        const uint64_t at = first + (uint64_t)i * kClipThreads * V;
        const uint64_t left = at < elements ? elements - at : 0;
#pragma unroll
        for (uint32_t k = 0; k < V; k++)
            f[i][k] *= factor;
        store_elems<DT>((T *)out + at, left < V ? (uint32_t)left : V, f[i]);
    }
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

// The tiles of workgroup b: an even share of the launch's.
__device__ __forceinline__ uint32_t clip_first_tile(uint32_t tiles, uint32_t block)
{
    return (uint32_t)((uint64_t)tiles * block / gridDim.x);
}

__global__ __launch_bounds__(kClipThreads) void clip_norm_kernel(ClipTable table, double *__restrict__ partial)
{
    __shared__ double lds[4];
    const uint32_t tiles = table.first_tile[table.tensors];
    uint32_t tile = clip_first_tile(tiles, blockIdx.x);
    const uint32_t end = clip_first_tile(tiles, blockIdx.x + 1);
    double sum = 0.0;
    if (tile < end) {
        uint32_t n = clip_find(table, tile);
        for (; tile < end; tile++) {
            while (tile >= table.first_tile[n + 1])
                n++;
            const uint64_t local = tile - table.first_tile[n];
            if (table.type[n] == kElemBF16)
                sum += clip_tile_sum<kElemBF16>(table.in[n], table.elements[n], local);
            else if (table.type[n] == kElemF16)
                sum += clip_tile_sum<kElemF16>(table.in[n], table.elements[n], local);
            else
                sum += clip_tile_sum<kElemF32>(table.in[n], table.elements[n], local);
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

// Tiles are walked from the end of each workgroup's range: what the norm
// pass read last is what the caches still hold. `in_place`: every tensor's
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
    const float factor = clip ? (float)(max_norm / norm) : 1.0f;
    const uint32_t tiles = table.first_tile[table.tensors];
    const uint32_t first = clip_first_tile(tiles, blockIdx.x);
    uint32_t tile = clip_first_tile(tiles, blockIdx.x + 1);
    if (first == tile)
        return;
    uint32_t n = clip_find(table, tile - 1);
    while (tile-- > first) {
        while (tile < table.first_tile[n])
            n--;
        const uint64_t local = tile - table.first_tile[n];
        if (table.type[n] == kElemBF16)
            clip_tile_scale<kElemBF16>(table.in[n], table.out[n], table.elements[n], local, factor);
        else if (table.type[n] == kElemF16)
            clip_tile_scale<kElemF16>(table.in[n], table.out[n], table.elements[n], local, factor);
        else
            clip_tile_scale<kElemF32>(table.in[n], table.out[n], table.elements[n], local, factor);
    }
}

} // namespace mxq
