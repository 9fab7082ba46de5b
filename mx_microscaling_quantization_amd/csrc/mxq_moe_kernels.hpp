// mxq_moe_kernels.hpp -- gfx950 kernels around the experts of a
// mixture-of-experts layer: pairs sorted by expert, token rows gathered into
// that order and MX-quantized, results brought back to token order with their
// weights, and that step's gradient.
//
// A pair is (token t, slot j), numbered t * slots + j. Sorted rows hold the
// pairs expert by expert, in pair order within an expert, each expert's group
// starting at a multiple of `align` rows:
//   offsets[0] = 0, offsets[e + 1] = offsets[e] + align * ceil(count[e] / align)
//   dest[pair] = the pair's row, -1 for a pair whose id is no expert's
//   src[row]   = the row's pair, -1 for the rows between groups' ends and past
//                the last group
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mxq_axis_kernels.hpp"

namespace mxq {

// ----------------------------------------------------------------------------
// Sort by expert
// ----------------------------------------------------------------------------
//
// A counting sort. A workgroup of 16 waves takes a contiguous chunk of pairs,
// a wave a contiguous part of the chunk. It counts its experts in LDS, one
// row of counts per wave; the counts of everything before a wave's part then
// give where its first pair of each expert goes, and each wave places its
// pairs 64 at a time: lanes with the same expert find each other with one
// ballot per bit of the expert number, their rank in that set gives the
// order, and one of them advances the wave's position of that expert. Nothing
// depends on the order in which waves or workgroups run.
//
// One workgroup sorts a short list in one launch. A longer one takes two
// launches, of up to kSortBlocks workgroups: the counts of each chunk go to
// the workspace, then every workgroup sums the chunks' counts itself (all of
// them for the group sizes, those before its own for its positions).
constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortWaves = kSortThreads / 64;
constexpr uint32_t kSortBlocks = 256;

template <typename ID>
__device__ __forceinline__ uint32_t sort_key(const ID *ids, uint32_t pair, uint32_t pairs, uint32_t experts)
{
    if (pair >= pairs)
        return experts;
    const ID id = ids[pair];
    return id >= 0 && id < (ID)experts ? (uint32_t)id : experts;
}

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, uint32_t lane)
{
#pragma unroll
    for (uint32_t d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_up((int)v, d);
        v += lane >= d ? o : 0u;
    }
    return v;
}

// A wave takes its part in batches of 4 pairs per lane, loaded together; with
// one batch (chunks of up to kSortBatch pairs) the counting's keys are kept for
// the placing.
constexpr uint32_t kSortKeys = 4;
constexpr uint32_t kSortBatch = kSortKeys * kSortThreads;

template <typename ID>
__device__ __forceinline__ void sort_load(const ID *ids, uint32_t first, uint32_t pairs, uint32_t experts,
                                          uint32_t lane, uint32_t (&key)[kSortKeys])
{
#pragma unroll
    for (uint32_t k = 0; k < kSortKeys; k++)
        key[k] = sort_key(ids, first + 64u * k + lane, pairs, experts);
}

// Counts of this wave's part, `key` its first batch, into row[0 .. experts).
template <typename ID>
__device__ __forceinline__ void sort_count(const ID *ids, uint32_t first, uint32_t part, uint32_t pairs,
                                           uint32_t experts, uint32_t lane, uint32_t (&key)[kSortKeys], uint32_t *row)
{
    for (uint32_t p = 0; p < part; p += 64 * kSortKeys) {
        if (p > 0)
            sort_load(ids, first + p, pairs, experts, lane, key);
#pragma unroll
        for (uint32_t k = 0; k < kSortKeys; k++)
            if (key[k] < experts && p + 64u * k < part)
                atomicAdd(row + key[k], 1u);
    }
}

// Launch 1 of 2: counts[block][expert] of each workgroup's chunk, in rows of
// `pitch` (experts rounded up to 4, the rest zero). The 16 waves share one row
// of LDS counts.
template <typename ID>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(const ID *__restrict__ ids, uint32_t pairs,
                                                                  uint32_t chunk, uint32_t experts, uint32_t pitch,
                                                                  uint32_t *__restrict__ counts)
{
    extern __shared__ uint32_t row[];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const uint32_t part = chunk / kSortWaves;
    const uint32_t first = blockIdx.x * chunk + wave * part;
    uint32_t key[kSortKeys];
    sort_load(ids, first, pairs, experts, lane, key);
    for (uint32_t e = tid; e < pitch; e += kSortThreads)
        row[e] = 0;
    __syncthreads();
    sort_count(ids, first, part, pairs, experts, lane, key, row);
    __syncthreads();
    for (uint32_t e = tid; e < pitch; e += kSortThreads)
        counts[(uint64_t)blockIdx.x * pitch + e] = row[e];
}

// Launch 2 of 2 (SINGLE = 0), or the whole sort in one workgroup (SINGLE = 1,
// no counts in memory). Chunks are multiples of 64 * kSortWaves pairs and
// blocks * chunk < 2^32 (checked on the host).
//   LDS: kSortWaves rows of counts, then 3 arrays of `pitch`: each group's
//   pairs, the pairs of it before this chunk, its first row
template <typename ID, int SINGLE>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(const ID *__restrict__ ids, uint32_t pairs,
                                                                  uint32_t chunk, uint32_t experts, uint32_t pitch,
                                                                  uint32_t align, uint32_t rows, uint32_t key_bits,
                                                                  const uint32_t *__restrict__ counts,
                                                                  int32_t *__restrict__ offsets,
                                                                  int32_t *__restrict__ src,
                                                                  int32_t *__restrict__ dest)
{
    extern __shared__ uint32_t lds[];
    __shared__ uint32_t wave_total[kSortWaves];
    uint32_t *total = lds + kSortWaves * experts, *before = total + pitch, *start = before + pitch;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    const uint32_t blocks = gridDim.x, block = blockIdx.x;
    const uint32_t part = chunk / kSortWaves;
    const uint32_t first = block * chunk + wave * part;
    uint32_t key[kSortKeys];
    sort_load(ids, first, pairs, experts, lane, key);

    for (uint32_t n = tid; n < kSortWaves * experts + 2 * pitch; n += kSortThreads)
        lds[n] = 0;
    __syncthreads();
    uint32_t *mine = lds + wave * experts;
    sort_count(ids, first, part, pairs, experts, lane, key, mine);
    if constexpr (!SINGLE) {
        // the workgroup's threads as rows of `width`, 4 experts each: each row
        // sums its share of the chunks
        uint32_t width = 16;
        while (4u * width < experts)
            width <<= 1;
        const uint32_t e = 4u * (tid & (width - 1)), r = tid / width, n = kSortThreads / width;
        u32x4_t all = {0u, 0u, 0u, 0u}, prior = all;
        if (e < pitch) {
#pragma unroll 8
            for (uint32_t b = r; b < blocks; b += n) {
                const u32x4_t c = *reinterpret_cast<const u32x4_t *>(counts + (uint64_t)b * pitch + e);
                all += c;
                prior += b < block ? c : u32x4_t{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (uint32_t k = 0; k < 4; k++) {
                atomicAdd(total + e + k, all[k]);
                atomicAdd(before + e + k, prior[k]);
            }
        }
    }
    __syncthreads();

    // thread e: group e's size, then the groups' first rows by a scan
    const uint32_t e = tid;
    uint32_t sum = 0, c[kSortWaves] = {};
    if (e < experts) {
#pragma unroll
        for (uint32_t w = 0; w < kSortWaves; w++)
            c[w] = lds[w * experts + e];
#pragma unroll
        for (uint32_t w = 0; w < kSortWaves; w++)
            sum += c[w];
        if constexpr (SINGLE)
            total[e] = sum;
        else
            sum = total[e];
    }
    const uint32_t padded = (sum + align - 1) / align * align;
    const uint32_t scan = wave_scan(padded, lane);
    if (lane == 63)
        wave_total[wave] = scan;
    __syncthreads();
    uint32_t base = 0;
    for (uint32_t w = 0; w < wave; w++)
        base += wave_total[w];
    if (e < experts) {
        const uint32_t at = base + scan - padded;
        start[e] = at;
        uint32_t here = at + before[e];   // the chunk's first row of group e, then each wave's
#pragma unroll
        for (uint32_t w = 0; w < kSortWaves; w++) {
            lds[w * experts + e] = here;
            here += c[w];
        }
        if (block == 0) {
            offsets[e] = (int32_t)at;
            if (e + 1 == experts)
                offsets[experts] = (int32_t)(at + padded);
        }
    }
    __syncthreads();

    for (uint32_t p = 0; p < part && first + p < pairs; p += 64 * kSortKeys) {
        if (part > 64 * kSortKeys)
            sort_load(ids, first + p, pairs, experts, lane, key);
#pragma unroll
        for (uint32_t k = 0; k < kSortKeys; k++) {
            const uint32_t pair = first + p + 64u * k + lane;
            if (p + 64u * k >= part)
                break;
            uint64_t same = __ballot(key[k] < experts);
            for (uint32_t b = 0; b < key_bits; b++) {
                const uint64_t set = __ballot((key[k] >> b) & 1u);
                same &= (key[k] >> b) & 1u ? set : ~set;
            }
            uint32_t row = 0;
            const uint32_t leader = same ? (uint32_t)__builtin_ctzll(same) : lane;
            if (key[k] < experts && lane == leader)
                row = atomicAdd(mine + key[k], (uint32_t)__popcll(same));
            row = (uint32_t)__shfl((int)row, (int)leader) +
                  (uint32_t)__popcll(same & ((1ull << lane) - 1ull));
            if (pair < pairs) {
                dest[pair] = key[k] < experts ? (int32_t)row : -1;
                if (key[k] < experts && row < rows)
                    src[row] = (int32_t)pair;
            }
        }
    }
    // rows without a pair: a wave per group, then past the last group
    for (uint32_t g = block * kSortWaves + wave; g < experts; g += blocks * kSortWaves) {
        const uint32_t end = g + 1 < experts ? start[g + 1] : start[g] + (total[g] + align - 1) / align * align;
        for (uint32_t r = start[g] + total[g] + lane; r < end && r < rows; r += 64)
            src[r] = -1;
    }
    const uint32_t last = start[experts - 1] + (total[experts - 1] + align - 1) / align * align;
    for (uint32_t r = last + block * kSortThreads + tid; r < rows; r += blocks * kSortThreads)
        src[r] = -1;
}

// ----------------------------------------------------------------------------
// Rows of a list of elements
// ----------------------------------------------------------------------------

enum { kElemBF16 = 0, kElemF16 = 1, kElemF32 = 2 };

template <int DT> struct Elem { typedef uint16_t type; static constexpr uint32_t vec = 8; };
template <> struct Elem<kElemF32> { typedef float type; static constexpr uint32_t vec = 4; };

template <int DT> __device__ __forceinline__ float elem_to_f32(typename Elem<DT>::type v)
{
    if constexpr (DT == kElemF32)
        return v;
    else if constexpr (DT == kElemBF16)
        return __uint_as_float((uint32_t)v << 16);
    else
        return (float)__builtin_bit_cast(_Float16, v);
}

// One rounding, to nearest even; a NaN stays a NaN.
template <int DT> __device__ __forceinline__ typename Elem<DT>::type elem_from_f32(float v)
{
    if constexpr (DT == kElemF32)
        return v;
    else if constexpr (DT == kElemBF16)
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    else
        return __builtin_bit_cast(uint16_t, (_Float16)v);
}

// 16 bytes of a row at element alignment: rows of any length start anywhere,
// and the memory path takes 16-byte accesses at any element boundary.
template <int DT> struct __attribute__((packed, aligned(sizeof(typename Elem<DT>::type)))) ElemVec {
    typename Elem<DT>::type v[Elem<DT>::vec];
};

typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

template <int DT> __device__ __forceinline__ void elems_to_f32(const ElemVec<DT> &t, float *f)
{
#pragma unroll
    for (uint32_t i = 0; i < Elem<DT>::vec; i++)
        f[i] = elem_to_f32<DT>(t.v[i]);
}

// `n` (1 .. vec) elements at p; elements past n are zero.
template <int DT, int NT = 0>
__device__ __forceinline__ ElemVec<DT> load_vec(const typename Elem<DT>::type *p, uint32_t n)
{
    constexpr uint32_t V = Elem<DT>::vec;
    if (n >= V) {
        const u32x4_any_t *q = reinterpret_cast<const u32x4_any_t *>(p);
        return __builtin_bit_cast(ElemVec<DT>, NT ? __builtin_nontemporal_load(q) : *q);
    }
    ElemVec<DT> t = {};
#pragma unroll
    for (uint32_t i = 0; i < V; i++)
        if (i < n)
            t.v[i] = p[i];
    return t;
}

template <int DT> __device__ __forceinline__ void load_elems(const typename Elem<DT>::type *p, uint32_t n, float *f)
{
    elems_to_f32<DT>(load_vec<DT>(p, n), f);
}

template <int DT, int NT = 0>
__device__ __forceinline__ void store_elems(typename Elem<DT>::type *p, uint32_t n, const float *f)
{
    constexpr uint32_t V = Elem<DT>::vec;
    if (n >= V) {
        ElemVec<DT> t;
#pragma unroll
        for (uint32_t i = 0; i < V; i++)
            t.v[i] = elem_from_f32<DT>(f[i]);
        u32x4_any_t *q = reinterpret_cast<u32x4_any_t *>(p);
        const u32x4_any_t x = __builtin_bit_cast(u32x4_any_t, t);
        if constexpr (NT)
            __builtin_nontemporal_store(x, q);
        else
            *q = x;
    } else {
#pragma unroll
        for (uint32_t i = 0; i < V; i++)
            if (i < n)
                p[i] = elem_from_f32<DT>(f[i]);
    }
}

// A row of N elements is read in ceil(N / vec) vectors. The last one of a row
// that is not a multiple of them starts earlier, at N - vec, so that it is a
// whole vector too (its first elements are then also the previous one's:
// results are written twice, with the same value, and sums leave them out);
// only rows shorter than a vector are taken element by element.
struct RowVec {
    uint32_t first, n;   // first element, elements (vec, or N in a short row)
    uint32_t again;      // of these, elements the previous vector has too
};

template <uint32_t V> __device__ __forceinline__ RowVec row_vec(uint32_t N, uint32_t vec)
{
    const uint32_t at = vec * V;
    if (N < V)
        return {0, N, 0};
    const uint32_t first = min(at, N - V);
    return {first, V, at - first};
}

// ----------------------------------------------------------------------------
// Combine: out[t] = sum over j of w[t][j] * y[dest[t][j]]
// ----------------------------------------------------------------------------
//
// LANES lanes take one token's row (64: a wave takes 64 vectors of it, and the
// token's rows and weights are wave-uniform), a lane one vector of the result.
// Up to kCombineSlots rows are loaded before the first is added, in slot order,
// in f32, rounded once: the result does not depend on the launch. A dest
// outside [0, rows) adds nothing, whatever its weight (its load goes to row 0
// instead, which the host sees is there); a token none of whose pairs has a
// row gets zeros.
constexpr uint32_t kCombineSlots = 8;

template <int DT, int WEIGHTED, uint32_t LANES, uint32_t S>
__device__ __forceinline__ void combine_slots(const typename Elem<DT>::type *y, uint32_t rows, uint32_t N,
                                              const RowVec &rv, const int32_t *dest, const float *weights, float *acc)
{
    constexpr uint32_t V = Elem<DT>::vec;
    uint32_t r[S];
    float w[S];
    ElemVec<DT> x[S];
#pragma unroll
    for (uint32_t j = 0; j < S; j++) {
        r[j] = (uint32_t)dest[j];
        w[j] = WEIGHTED ? weights[j] : 1.0f;
        if constexpr (LANES == 64)
            r[j] = (uint32_t)__builtin_amdgcn_readfirstlane((int)r[j]);
    }
    // y past the caches: of 512 MB 108 us, 128 without the hint; behind the product
    // that wrote y (213 MB) the two take 110 and 121 (a second reading in a row
    // would take 39 and 33)
#pragma unroll
    for (uint32_t j = 0; j < S; j++)
        x[j] = load_vec<DT, 1>(y + (uint64_t)(r[j] < rows ? r[j] : 0u) * N + rv.first, rv.n);
#pragma unroll
    for (uint32_t j = 0; j < S; j++) {
        if (r[j] < rows) {
            float f[V];
            elems_to_f32<DT>(x[j], f);
#pragma unroll
            for (uint32_t i = 0; i < V; i++)
                acc[i] = WEIGHTED ? __builtin_fmaf(w[j], f[i], acc[i]) : acc[i] + f[i];
        }
    }
}

template <int DT, int WEIGHTED, uint32_t LANES>
__global__ __launch_bounds__(256) void combine_kernel(const typename Elem<DT>::type *__restrict__ y, uint32_t rows,
                                                      uint32_t N, uint32_t vecs, uint32_t parts,
                                                      const int32_t *__restrict__ dest,
                                                      const float *__restrict__ weights, uint32_t tokens,
                                                      uint32_t slots, typename Elem<DT>::type *__restrict__ out)
{
    constexpr uint32_t V = Elem<DT>::vec;
    uint32_t item = blockIdx.x * (256u / LANES) + threadIdx.x / LANES;   // (token, part of 64 vectors)
    if constexpr (LANES == 64)
        item = (uint32_t)__builtin_amdgcn_readfirstlane((int)item);
    const uint32_t t = LANES == 64 ? item / parts : item;
    const uint32_t vec = (LANES == 64 ? item - t * parts : 0u) * 64u + threadIdx.x % LANES;
    if (t >= tokens || vec >= vecs)
        return;
    const RowVec rv = row_vec<V>(N, vec);
    const int32_t *d = dest + (uint64_t)t * slots;
    const float *w = weights + (WEIGHTED ? (uint64_t)t * slots : 0u);
    float acc[V] = {};
    uint32_t j = 0;
    for (; j + kCombineSlots <= slots; j += kCombineSlots)
        combine_slots<DT, WEIGHTED, LANES, kCombineSlots>(y, rows, N, rv, d + j, w + j, acc);
    if (slots & 4u) {
        combine_slots<DT, WEIGHTED, LANES, 4>(y, rows, N, rv, d + j, w + j, acc);
        j += 4;
    }
    if (slots & 2u) {
        combine_slots<DT, WEIGHTED, LANES, 2>(y, rows, N, rv, d + j, w + j, acc);
        j += 2;
    }
    if (slots & 1u)
        combine_slots<DT, WEIGHTED, LANES, 1>(y, rows, N, rv, d + j, w + j, acc);
    store_elems<DT>(out + (uint64_t)t * N + rv.first, rv.n, acc);
}

// ----------------------------------------------------------------------------
// The gradient of combine
// ----------------------------------------------------------------------------
//
//   grad_y[r]    = w[src[r]] * grad[src[r] / slots], zero for a row without a pair
//   grad_w[t][j] = sum over n of grad[t][n] * y[dest[t][j]][n], zero for a pair
//                  without a row
//
// LANES lanes take one sorted row: they read y's row and the token's gradient
// row, write grad_y's row and keep the products' sum in registers until one
// reduction (in a fixed order). Row by row, y and grad_y stream in order; the
// gradient rows are read once per slot, all but the first time from the caches.
// (Token by token, with the gradient row read once and `slots` rows of y and
// grad_y open at a time, 6007 x 8 rows of 2052 bf16 took 161 us.)
// Workgroups past the rows' own clear grad_w of the pairs without a row: of each
// pair exactly one of the two, the one row that dest and src both name or these,
// writes it.
// A lane has KV vectors of each row in flight: one where the row has up to 64, else
// two at a time. y and grad_y go past the caches (rows of 4096 bf16, 16384 x 4:
// 226 us, 254 without the hint). The stores keep the hint also where rows are not
// whole lines (ordinary stores: 6007 x 8 rows of 2052 97 us, 94 with it; 16384 x 4 rows
// of 4100 270 and 251).
template <int DT, uint32_t LANES, uint32_t KV>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const typename Elem<DT>::type *__restrict__ grad, const typename Elem<DT>::type *__restrict__ y, uint32_t rows,
    uint32_t N, uint32_t vecs, const int32_t *__restrict__ src, const int32_t *__restrict__ dest,
    const float *__restrict__ weights, uint32_t pairs, uint32_t slots, uint32_t row_blocks,
    typename Elem<DT>::type *__restrict__ grad_y, float *__restrict__ grad_w)
{
    constexpr uint32_t V = Elem<DT>::vec;
    if (blockIdx.x >= row_blocks) {
        const uint32_t pair = (blockIdx.x - row_blocks) * 256u + threadIdx.x;
        if (pair < pairs) {
            const uint32_t r = (uint32_t)dest[pair];
            if (r >= rows || (uint32_t)src[r] != pair)
                grad_w[pair] = 0.0f;
        }
        return;
    }
    uint32_t r = blockIdx.x * (256u / LANES) + threadIdx.x / LANES;
    if constexpr (LANES == 64)
        r = (uint32_t)__builtin_amdgcn_readfirstlane((int)r);
    const uint32_t lane = threadIdx.x % LANES;
    if (r >= rows)
        return;   // (a row's lanes leave together, and the sums stay within them)
    const uint32_t pair = (uint32_t)src[r];
    typename Elem<DT>::type *gy = grad_y + (uint64_t)r * N;
    if (pair >= pairs) {
        const float zero[V] = {};
        for (uint32_t vec = lane; vec < vecs; vec += LANES) {
            const RowVec rv = row_vec<V>(N, vec);
            store_elems<DT>(gy + rv.first, rv.n, zero);
        }
        return;
    }
    const float w = weights[pair];
    const typename Elem<DT>::type *yr = y + (uint64_t)r * N, *g = grad + (uint64_t)(pair / slots) * N;
    float acc = 0.0f;
    for (uint32_t v0 = lane; v0 < vecs; v0 += KV * LANES) {
        ElemVec<DT> gx[KV], yx[KV];
#pragma unroll
        for (uint32_t k = 0; k < KV; k++) {
            // a lane past the row takes its first vector again, and drops it
            const RowVec rv = row_vec<V>(N, v0 + k * LANES < vecs ? v0 + k * LANES : 0u);
            gx[k] = load_vec<DT>(g + rv.first, rv.n);
            yx[k] = load_vec<DT, 1>(yr + rv.first, rv.n);
        }
#pragma unroll
        for (uint32_t k = 0; k < KV; k++) {
            if (v0 + k * LANES >= vecs)
                break;
            const RowVec rv = row_vec<V>(N, v0 + k * LANES);
            float a[V], b[V];
            elems_to_f32<DT>(gx[k], a);
            elems_to_f32<DT>(yx[k], b);
            if (rv.again == 0) {
#pragma unroll
                for (uint32_t i = 0; i < V; i++)
                    acc = __builtin_fmaf(a[i], b[i], acc);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < V; i++)
                    if (i >= rv.again)
                        acc = __builtin_fmaf(a[i], b[i], acc);
            }
#pragma unroll
            for (uint32_t i = 0; i < V; i++)
                a[i] *= w;
            store_elems<DT, 1>(gy + rv.first, rv.n, a);
        }
    }
#pragma unroll
    for (int d = LANES / 2; d > 0; d >>= 1)
        acc += __shfl_xor(acc, d);
    // (src and dest may disagree: a pair that the caller took out of dest alone is a
    // pair without a row, whose zero the other workgroups write)
    if (lane == 0 && (uint32_t)dest[pair] == r)
        grad_w[pair] = acc;
}

// ----------------------------------------------------------------------------
// Gather and quantize
// ----------------------------------------------------------------------------
//
// The quantize of the [rows, K] tensor whose row r is x[src[r] / slots] (zeros
// where src[r] is no pair), with blocks along its rows (the along kernel's
// tile, lane mapping and LDS transpose, see mxq_axis_kernels.hpp) or down its
// columns (the down kernel's). The row numbers are the only difference in
// what is read; the result bytes are those of quantize_axis on that tensor.

// pair / slots for pair < 2^31: with shift = 31 + ceil(log2 slots) and mul =
// ceil(2^shift / slots) (under 2^32), mul * slots exceeds 2^shift by less than
// slots <= 2^(shift - 31), too little to reach the next quotient.
__device__ __forceinline__ uint32_t slot_div(uint32_t pair, uint32_t mul, uint32_t shift)
{
    return (uint32_t)(((uint64_t)pair * mul) >> shift);
}

// Tiles are numbered K column by K column and every XCD takes consecutive
// ones: a token's 128 bytes of a K column, wanted by the rows of all its
// slots, are then read by one XCD, once from memory and from its L2 after that
// (8192 x 8 rows of 4096 bf16: 97 us with tiles dealt out to the XCDs in turn,
// 77 us so; 71 with the lanes reading their rows' numbers themselves instead of
// through LDS; ordinary instead of non-temporal stores 108).
template <int IN, int OUT>
__global__ __launch_bounds__(64 * kAlongWaves) void gather_quantize_along_kernel(
    const uint16_t *__restrict__ x, const int32_t *__restrict__ src, uint32_t rows, uint32_t pairs, uint32_t div_mul,
    uint32_t div_shift, uint64_t K, uint32_t tiles_m, int emax_bias, uint32_t dense, uint8_t *__restrict__ data,
    uint8_t *__restrict__ scale)
{
    constexpr uint32_t RT = kAlongRows, KG = kAlongWaveRows / 32;
    constexpr uint32_t CB = OUT == kOutE2M1 ? 2 : 4;
    constexpr uint32_t PITCH = RT * CB + 16;
    __shared__ __attribute__((aligned(16))) uint8_t codes[16 * PITCH];
    __shared__ __attribute__((aligned(16))) uint8_t e8m0[2 * RT];

    const uint32_t t = threadIdx.x, w = t >> 6, l = t & 63u;
    const uint32_t c = l & 7u, i = l >> 3, q = c & 3u, bl = c >> 2;
    const uint32_t tile = tile_index<8>();
    const uint32_t tk = tile / tiles_m;
    const uint32_t m0 = (tile - tk * tiles_m) * RT;
    const uint32_t G = (uint32_t)(K / 32);
    const uint32_t g = tk * 2u + bl;

    // the lane's rows come in fours, all inside or all past the tensor
    u32x4_t sr[KG];
#pragma unroll
    for (uint32_t kg = 0; kg < KG; kg++) {
        const uint32_t r = m0 + kAlongWaveRows * w + 4u * i + 32u * kg;
        sr[kg] = *reinterpret_cast<const u32x4_t *>(src + (r < rows ? r : 0u));
        sr[kg] = r < rows ? sr[kg] : u32x4_t{~0u, ~0u, ~0u, ~0u};
    }
    u32x4_t v[4 * KG];
#pragma unroll
    for (uint32_t k = 0; k < 4 * KG; k++) {
        const uint32_t pair = sr[k >> 2][k & 3u];
        const uint32_t tok = slot_div(pair, div_mul, div_shift);
        const bool ok = g < G && pair < pairs;
        v[k] = *reinterpret_cast<const u32x4_t *>(x + (ok ? (uint64_t)tok * K + g * 32u : 0u) + 8u * q);
        v[k] = ok ? v[k] : u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (uint32_t kg = 0; kg < KG; kg++) {
        uint32_t lo[4], hi[4], eb[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const u32x4_t a = v[4 * kg + j];
            uint32_t mm = pk_max_u16(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu);
            mm = pk_max_u16(mm, a.z & 0x7FFF7FFFu);
            mm = pk_max_u16(mm, a.w & 0x7FFF7FFFu);
            const uint32_t mag = quad_max(max(mm & 0xFFFFu, mm >> 16));
            uint32_t e[1] = {block_e8m0<IN>(mag, emax_bias)};
            const float s = e8m0_to_scale(e[0]);
            uint32_t w0[2] = {a.x, a.y}, w1[2] = {a.z, a.w};
            uint32_t o0[1], o1[1];
            if constexpr (OUT == kOutE2M1) {
                o0[0] = fp4_container<IN, 0>(0u, w0[0], w0[1], s);
                o1[0] = fp4_container<IN, 0>(0u, w1[0], w1[1], s);
            } else {
                o0[0] = fp8x4<IN, OUT>(w0[0], w0[1], s);
                o1[0] = fp8x4<IN, OUT>(w1[0], w1[1], s);
            }
            if (mag > InfBits<IN>::value || e[0] == 254u) {
                fix_special_codes<IN, OUT, 1>(w0, e, o0);
                fix_special_codes<IN, OUT, 1>(w1, e, o1);
            }
            lo[j] = o0[0];
            hi[j] = o1[0];
            eb[j] = e[0];
        }
        const uint32_t r = kAlongWaveRows * w + 4u * i + 32u * kg;
        uint8_t *s0 = codes + (8u * bl + 2u * q) * PITCH + CB * r;
        if constexpr (OUT == kOutE2M1) {
            *reinterpret_cast<u32x2_t *>(s0) = u32x2_t{lo[0] | lo[1] << 16, lo[2] | lo[3] << 16};
            *reinterpret_cast<u32x2_t *>(s0 + PITCH) = u32x2_t{hi[0] | hi[1] << 16, hi[2] | hi[3] << 16};
        } else {
            *reinterpret_cast<u32x4_t *>(s0) = u32x4_t{lo[0], lo[1], lo[2], lo[3]};
            *reinterpret_cast<u32x4_t *>(s0 + PITCH) = u32x4_t{hi[0], hi[1], hi[2], hi[3]};
        }
        if (q == 0)
            *reinterpret_cast<uint32_t *>(e8m0 + bl * RT + r) = eb[0] | eb[1] << 8 | eb[2] << 16 | eb[3] << 24;
    }
    __syncthreads();

    // `rows` is a multiple of 4 (checked on the host): 4 rows per lane
    using T = typename std::conditional<OUT == kOutE2M1, u32x2_t, u32x4_t>::type;
    constexpr uint32_t VPW = 16 / kAlongWaves, SPR = RT / 256;
    T val[VPW][SPR];
#pragma unroll
    for (uint32_t j = 0; j < VPW; j++)
#pragma unroll
        for (uint32_t s = 0; s < SPR; s++)
            val[j][s] = *reinterpret_cast<const T *>(codes + (VPW * w + j) * PITCH + CB * (256u * s + 4u * l));
#pragma unroll
    for (uint32_t j = 0; j < VPW; j++) {
        const uint32_t vr = VPW * w + j;
        const uint64_t p = (uint64_t)tk * 16u + vr;
#pragma unroll
        for (uint32_t s = 0; s < SPR; s++) {
            const uint32_t r = 256u * s + 4u * l;
            if (tk * 2u + (vr >> 3) < G && m0 + r < rows)
                store<1>(reinterpret_cast<T *>(data + (p * rows + m0 + r) * CB), val[j][s]);
        }
    }
    for (uint32_t idx = t; idx < 2 * RT / 4; idx += 64 * kAlongWaves) {
        const uint32_t strip = idx / (RT / 4), r = 4u * (idx - strip * (RT / 4));
        const uint32_t gg = tk * 2u + strip;
        if (gg < G && m0 + r < rows) {
            const uint64_t slot = dense ? gg : (gg & 3u) + 32ull * (gg >> 2);
            store<1>(reinterpret_cast<uint32_t *>(scale + slot * rows + m0 + r),
                     *reinterpret_cast<const uint32_t *>(e8m0 + strip * RT + r));
        }
    }
}

// Blocks of 32 sorted rows (rows % 32 == 0, groups aligned to 32: no block
// spans two experts). Lane r < 32 looks up row r's token, and every lane gets
// all 32 of them in scalar registers before the lanes past the tensor leave.
// RUNS: tiles are numbered run of columns by run of columns and every XCD takes
// consecutive ones, so that a token's 512 bytes of a run come from that XCD's
// L2 for all slots but the first (8192 x 8 rows of 4096 bf16: 89 -> 61 us); else
// band by band, which writes in order (16384 x 1 rows of 8192: 61 us in either order).
template <int IN, int OUT, int NB, int RUNS>
__global__ __launch_bounds__(64) void gather_quantize_down_kernel(const uint16_t *__restrict__ x,
                                                                  const int32_t *__restrict__ src, uint32_t rows,
                                                                  uint32_t pairs, uint32_t div_mul,
                                                                  uint32_t div_shift, uint64_t N, uint32_t nstrips,
                                                                  uint32_t tiles_per_band, int emax_bias,
                                                                  uint32_t dense, uint8_t *__restrict__ data,
                                                                  uint8_t *__restrict__ scale)
{
    constexpr int NW = (NB + 1) / 2;
    constexpr uint32_t LANE_BYTES = OUT == kOutE2M1 ? 2 * NB : 4 * NB;
    const uint32_t tile = tile_index<RUNS ? 8 : 0>(), bands = gridDim.x / tiles_per_band;
    const uint32_t run = RUNS ? tile / bands : tile % tiles_per_band;
    const uint32_t band = RUNS ? tile - run * bands : tile / tiles_per_band;
    const uint32_t strip = run * 64u + threadIdx.x;
    const uint32_t pair = (uint32_t)src[band * 32u + (threadIdx.x & 31u)];   // rows % 32 == 0
    const int32_t mine = pair < pairs ? (int32_t)slot_div(pair, div_mul, div_shift) : -1;
    int32_t token[32];
#pragma unroll
    for (int r = 0; r < 32; r++)
        token[r] = __builtin_amdgcn_readlane(mine, r);
    if (strip >= nstrips)
        return;
    const uint64_t n0 = (uint64_t)strip * NB;
    uint32_t v[32][NW];
#pragma unroll
    for (int r = 0; r < 32; r++) {
        const int32_t tok = token[r];
        const uint16_t *p = x + (uint64_t)(tok < 0 ? 0 : tok) * N + n0;
        if constexpr (NB == 4) {
            const u32x2_t d = *reinterpret_cast<const u32x2_t *>(p);
            v[r][0] = tok < 0 ? 0u : d.x;
            v[r][1] = tok < 0 ? 0u : d.y;
        } else if constexpr (NB == 2) {
            v[r][0] = tok < 0 ? 0u : *reinterpret_cast<const uint32_t *>(p);
        } else {
            v[r][0] = tok < 0 ? 0u : *p;
        }
    }

    uint32_t e[NB];
    float s[NB];
    bool special = false;
#pragma unroll
    for (int h = 0; h < NW; h++) {
        uint32_t m = 0;
#pragma unroll
        for (int r = 0; r < 32; r++)
            m = pk_max_u16(m, v[r][h] & 0x7FFF7FFFu);
#pragma unroll
        for (int q = 0; q < 2 && 2 * h + q < NB; q++) {
            const uint32_t mag = half16(m, q);
            e[2 * h + q] = block_e8m0<IN>(mag, emax_bias);
            s[2 * h + q] = e8m0_to_scale(e[2 * h + q]);
            special |= mag > InfBits<IN>::value || e[2 * h + q] == 254u;
        }
    }
    constexpr int OW = OUT == kOutE2M1 ? NW : NB;
    uint32_t out[8][OW];
#pragma unroll
    for (int pr = 0; pr < 8; pr++) {
        uint32_t w[2 * NB];
#pragma unroll
        for (int b = 0; b < NB; b++) {
            const int h = b / 2, q = b & 1;
            w[2 * b] = half16(v[4 * pr][h], q) | half16(v[4 * pr + 1][h], q) << 16;
            w[2 * b + 1] = half16(v[4 * pr + 2][h], q) | half16(v[4 * pr + 3][h], q) << 16;
        }
        if constexpr (OUT == kOutE2M1) {
#pragma unroll
            for (int h = 0; h < NW; h++) {
                out[pr][h] = fp4_container<IN, 0>(0u, w[4 * h], w[4 * h + 1], s[2 * h]);
                if constexpr (NB > 1)
                    out[pr][h] = fp4_container<IN, 1>(out[pr][h], w[4 * h + 2], w[4 * h + 3], s[2 * h + 1]);
            }
        } else {
#pragma unroll
            for (int b = 0; b < NB; b++)
                out[pr][b] = fp8x4<IN, OUT>(w[2 * b], w[2 * b + 1], s[b]);
        }
        if (special)
            fix_special_codes<IN, OUT, NB>(w, e, out[pr]);
    }
#pragma unroll
    for (int pr = 0; pr < 8; pr++)
        store_bytes<LANE_BYTES, 1>(data + ((uint64_t)band * 8u + pr) * N * (LANE_BYTES / NB) +
                                       n0 * (LANE_BYTES / NB), out[pr]);
    const uint64_t slot = dense ? (uint64_t)band : (uint64_t)(band & 3u) + 32u * (uint64_t)(band >> 2);
    uint32_t packed[1] = {0};
#pragma unroll
    for (int b = 0; b < NB; b++)
        packed[0] |= e[b] << (8 * b);
    store_bytes<NB, 1>(scale + slot * N + n0, packed);
}

} // namespace mxq
