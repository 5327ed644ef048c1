// moe.cu -- routing of tokens to experts and back: exl3_moe_sort,
// exl3_moe_gather, exl3_moe_combine, exl3_moe_combine_grad.
//
// With ids[t, j] the j-th expert of token t (a choice), e's rows are
// [offsets[e], offsets[e + 1]) and a choice's row is
//     positions[t, j] = offsets[id] + #{earlier choices (in (t, j) order) with the same id},
// a stable counting sort; a choice whose id is outside [0, experts) has no row
// (position -1).  Then
//     gather        xs[positions[t, j]] = x[t]
//     combine       y[t] = sum_j weights[t, j] ys[positions[t, j]]
//     combine_grad  dys[positions[t, j]] = weights[t, j] dy[t],
//                   dweights[t, j] = <dy[t], ys[positions[t, j]]>
// and the gradient of gather is combine without weights.  Every sum runs in
// fp32 in a fixed order, and no kernel uses a floating-point atomic, so
// results are deterministic.
#include <type_traits>

#include "dtypes.cuh"
#include "exl3_device.cuh"
#include "exl3_host.h"

namespace exl3 {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxExperts = 1024;
constexpr int kSortMaxChunks = 128;
constexpr size_t kSyncArea = 64 * 1024;  // status word and counters of the matmul calls: never touched here

// ------------------------------------------------------------------ sort ---

// Choices per chunk (one CTA each): a multiple of the block, so that at most
// kSortMaxChunks chunks exist and the second launch reads a bounded table.
static int64_t sort_chunk(int64_t n)
{
    const int64_t per = (n + kSortMaxChunks - 1) / kSortMaxChunks;
    return (per + kSortThreads - 1) / kSortThreads * kSortThreads;
}

// counts[c][e] = choices of chunk c that go to expert e.
__global__ void __launch_bounds__(kSortThreads) moe_count_kernel(const int32_t *__restrict__ ids, int64_t n,
                                                                 int64_t chunk, int experts,
                                                                 int32_t *__restrict__ counts)
{
    __shared__ int32_t sum[kSortMaxExperts];
    grid_dep_wait();
    for (int e = threadIdx.x; e < experts; e += kSortThreads)
        sum[e] = 0;
    __syncthreads();
    const int64_t i0 = blockIdx.x * chunk, i1 = i0 + chunk < n ? i0 + chunk : n;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kSortThreads) {
        const uint32_t e = (uint32_t)ids[i];
        if (e < (uint32_t)experts)
            atomicAdd(&sum[e], 1);  // integers: the order does not matter
    }
    __syncthreads();
    for (int e = threadIdx.x; e < experts; e += kSortThreads)
        counts[(int64_t)blockIdx.x * experts + e] = sum[e];
}

// Latency-bound: 8 x 8 choices in 3.3 us (one launch), 8192 x 8 in 2.8 + 7.2 us.
// Positions of one chunk's choices; chunk 0 also writes the offsets.  With
// one chunk (counts == nullptr) it is the whole sort.  A rank is the sum of
// the expert's offset, the choices of earlier chunks and of earlier rounds of
// this chunk (base[e], shared), of earlier warps of this round (per-warp
// counts, prefix-summed over the warps) and of earlier lanes (match_any).
__global__ void __launch_bounds__(kSortThreads) moe_place_kernel(const int32_t *__restrict__ ids, int64_t n,
                                                                 int64_t chunk, int experts, int chunks,
                                                                 const int32_t *__restrict__ counts,
                                                                 int32_t *__restrict__ offsets,
                                                                 int32_t *__restrict__ positions)
{
    extern __shared__ uint16_t per_warp[];  // [kSortWarps][experts]
    __shared__ int32_t base[kSortMaxExperts];
    __shared__ int32_t warp_sum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_wait();
    const int64_t i0 = blockIdx.x * chunk, i1 = i0 + chunk < n ? i0 + chunk : n;

    // each thread owns one expert (experts <= threads): its total and what
    // earlier chunks hold of it
    int32_t total = 0, before = 0;
    if (counts) {
        if (tid < experts) {
#pragma unroll 8
            for (int c = 0; c < chunks; ++c) {
                const int32_t v = counts[(int64_t)c * experts + tid];
                total += v;
                before += c < (int)blockIdx.x ? v : 0;
            }
        }
    } else {
        base[tid] = 0;
        __syncthreads();
        for (int64_t i = i0 + tid; i < i1; i += kSortThreads) {
            const uint32_t e = (uint32_t)ids[i];
            if (e < (uint32_t)experts)
                atomicAdd(&base[e], 1);
        }
        __syncthreads();
        total = tid < experts ? base[tid] : 0;
    }
    // exclusive scan of the totals over the experts
    int32_t incl = total;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        incl += lane >= d ? o : 0;
    }
    if (lane == 31)
        warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int32_t v = warp_sum[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t o = __shfl_up_sync(0xffffffffu, v, d);
            v += lane >= d ? o : 0;
        }
        warp_sum[lane] = v;
    }
    __syncthreads();
    incl += warp ? warp_sum[warp - 1] : 0;
    if (tid < experts)
        base[tid] = incl - total + before;
    if (blockIdx.x == 0) {
        if (tid < experts)
            offsets[tid + 1] = incl;
        if (tid == 0)
            offsets[0] = 0;
    }

    for (int64_t r0 = i0; r0 < i1; r0 += kSortThreads) {
        const int64_t i = r0 + tid;
        const uint32_t e = i < i1 ? (uint32_t)ids[i] : 0xffffffffu;
        const bool chosen = e < (uint32_t)experts;
        for (int j = tid; j < kSortWarps * experts; j += kSortThreads)
            per_warp[j] = 0;
        __syncthreads();
        const uint32_t same = __match_any_sync(0xffffffffu, chosen ? e : 0xffffffffu);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (chosen && rank == 0)
            per_warp[warp * experts + e] = (uint16_t)__popc(same);
        __syncthreads();
        int32_t sum = 0;
        if (tid < experts)
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const int32_t c = per_warp[w * experts + tid];
                per_warp[w * experts + tid] = (uint16_t)sum;
                sum += c;
            }
        __syncthreads();
        if (i < i1)
            positions[i] = chosen ? base[e] + (int32_t)per_warp[warp * experts + e] + rank : -1;
        __syncthreads();
        if (tid < experts)
            base[tid] += sum;
    }
}

// ------------------------------------------------------ gather, combine ---

// V elements (16 bytes, or one element), loaded and unpacked in two steps, so
// that several loads can be in flight as bits.
template <typename T, int V>
using Raw = typename std::conditional<V == 1, T, uint4>::type;

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T *p)
{
    return *reinterpret_cast<const Raw<T, V> *>(p);
}

// The same for rows that are read once: they need not stay in the caches.
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> load_once(const T *p)
{
    if constexpr (V == 1)
        return *p;
    else
        return __ldcs(reinterpret_cast<const uint4 *>(p));
}

template <typename T, int V>
__device__ __forceinline__ void unpack_raw(const Raw<T, V> &raw, float (&v)[V])
{
    if constexpr (V == 1)
        v[0] = to_f32(raw);
    else
        unpack16<T>(raw, v);
}

constexpr int kAhead = 4;  // rows or vectors whose loads a thread keeps in flight

// 8192 tokens x 8 rows of 8 KB: blocks of 128 threads 96 us, of 256 105 us (2 and
// 8 loads in flight instead of 4: 113 and 109 us).
constexpr int kCombineThreads = 128;

template <typename T, int V>
__device__ __forceinline__ void store_vec(T *p, const float (&v)[V])
{
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (V == Vec<T>::N) {
        *reinterpret_cast<uint4 *>(p) = pack16<T>(v);
    } else {
        // 4 fp32 sums to 8 bytes
        static_assert(V == 4 && sizeof(T) == 2, "narrowing store");
        T e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            e[i] = from_f32<T>(v[i]);
        uint2 raw;
        memcpy(&raw, e, 8);
        *reinterpret_cast<uint2 *>(p) = raw;
    }
}

// A row number read from the caller's tensor: -1 (no row) unless it is one of
// `rows`.
__device__ __forceinline__ int64_t row_or_none(int32_t p, int64_t rows)
{
    return p >= 0 && (int64_t)p < rows ? (int64_t)p : -1;
}

// Bound by the copies' bytes: 8192 x 8 rows of 8 KB in 93 us, 6.5 TB/s.
// A thread per unit of the row (16 bytes, or the element itself where a row is
// no multiple of 16 bytes) and a block row per token: x[t] is read once and
// written to each of the token's rows.
template <typename U>
__global__ void __launch_bounds__(256) moe_gather_kernel(const U *__restrict__ x, const int32_t *__restrict__ positions,
                                                         int64_t tokens, int topk, int64_t units, int64_t rows,
                                                         U *__restrict__ out)
{
    grid_dep_wait();
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        const int32_t *pos = positions + t * topk;
        for (int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; c < units; c += (int64_t)gridDim.y * blockDim.x) {
            const U v = x[t * units + c];
            for (int j = 0; j < topk; ++j) {
                const int64_t p = row_or_none(pos[j], rows);
                if (p >= 0)
                    out[p * units + c] = v;
            }
        }
    }
}

// Bound by the rows' bytes: 8192 tokens x 8 rows of 8 KB in 97 us, 6.2 TB/s.
template <typename T, typename O, int V>
__global__ void __launch_bounds__(kCombineThreads) moe_combine_kernel(const T *__restrict__ ys, const int32_t *__restrict__ positions,
                                                          const float *__restrict__ weights, int64_t tokens, int topk,
                                                          int64_t h, int64_t rows, O *__restrict__ y)
{
    grid_dep_wait();
    const int64_t cols = h / V;
    for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
        const int32_t *pos = positions + t * topk;
        for (int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; c < cols; c += (int64_t)gridDim.y * blockDim.x) {
            float acc[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                acc[i] = 0.f;
            // kAhead rows' loads in flight, added in the order of j
            for (int j0 = 0; j0 < topk; j0 += kAhead) {
                int64_t p[kAhead];
                float w[kAhead];
                Raw<T, V> raw[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    p[j] = j0 + j < topk ? row_or_none(pos[j0 + j], rows) : -1;
                    w[j] = weights && j0 + j < topk ? weights[t * topk + j0 + j] : 1.f;
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (p[j] >= 0)
                        raw[j] = load_once<T, V>(ys + p[j] * h + c * V);
#pragma unroll
                for (int j = 0; j < kAhead; ++j)
                    if (p[j] >= 0) {
                        float v[V];
                        unpack_raw<T, V>(raw[j], v);
#pragma unroll
                        for (int i = 0; i < V; ++i)
                            acc[i] = fmaf(w[j], v[i], acc[i]);
                    }
            }
            store_vec<O, V>(y + t * h + c * V, acc);
        }
    }
}

// Bound by the rows' bytes: 4096 x 4 rows of 8 KB in 46 us, 6.4 TB/s.
// A warp per choice: dys row = weight * dy row, and the dot product of dy with
// the expert's output row (each lane sums its columns in order, then a fixed
// butterfly over the lanes).  dys and dweights may each be null.
template <typename T, int V>
__global__ void __launch_bounds__(256) moe_combine_grad_kernel(const T *__restrict__ dy, const T *__restrict__ ys,
                                                               const int32_t *__restrict__ positions,
                                                               const float *__restrict__ weights, int64_t choices,
                                                               int topk, int64_t h, int64_t rows, T *__restrict__ dys,
                                                               float *__restrict__ dweights)
{
    grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < choices; i += warps) {
        const int64_t p = row_or_none(positions[i], rows);
        float dot = 0.f;
        if (p >= 0) {
            const float w = weights ? weights[i] : 1.f;
            const T *g = dy + (i / topk) * h;
            const T *f = ys + p * h;
            T *out = dys + p * h;
            for (int64_t c0 = (int64_t)lane * V; c0 < h; c0 += 32 * V * kAhead) {
                Raw<T, V> ra[kAhead], rb[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int64_t c = c0 + j * 32 * V;
                    if (c < h) {
                        ra[j] = load_raw<T, V>(g + c);
                        if (dweights)
                            rb[j] = load_raw<T, V>(f + c);
                    }
                }
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int64_t c = c0 + j * 32 * V;
                    if (c < h) {
                        float a[V], b[V];
                        unpack_raw<T, V>(ra[j], a);
                        if (dweights) {
                            unpack_raw<T, V>(rb[j], b);
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                dot = fmaf(a[e], b[e], dot);
                        }
                        if (dys) {
#pragma unroll
                            for (int e = 0; e < V; ++e)
                                b[e] = w * a[e];
                            store_vec<T, V>(out + c, b);
                        }
                    }
                }
            }
        }
        if (dweights) {
#pragma unroll
            for (int d = 16; d; d >>= 1)
                dot += __shfl_xor_sync(0xffffffffu, dot, d);
            if (lane == 0)
                dweights[i] = dot;
        }
    }
}

// Grid of the row kernels: a block row per token (at most 65536, the rest by
// striding) and enough block columns for the row.
static dim3 row_grid(int64_t tokens, int64_t cols, int threads = 256)
{
    const int64_t gx = tokens < 65536 ? tokens : 65536;
    int64_t gy = (cols + threads - 1) / threads;
    gy = gy < 64 ? gy : 64;
    return dim3((unsigned)gx, (unsigned)gy);
}

static size_t dtype_bytes(int dtype)
{
    return dtype == EXL3_F32 ? 4 : 2;
}

static bool valid_dtype(int dtype)
{
    return dtype == EXL3_F16 || dtype == EXL3_BF16 || dtype == EXL3_F32;
}

static bool valid_route(int64_t tokens, int64_t topk, int64_t h, int64_t rows, int dtype)
{
    return valid_dtype(dtype) && tokens >= 0 && tokens <= (int64_t)1 << 24 && topk >= 1 && topk <= 1024 && h >= 1 &&
           h <= (int64_t)1 << 22 && rows >= 0 && rows <= (int64_t)1 << 31;
}

template <typename T, typename O, int V>
static exl3_status launch_combine_v(const void *ys, const int32_t *positions, const float *weights, int64_t tokens,
                                    int64_t topk, int64_t h, int64_t rows, void *y, cudaStream_t s)
{
    if (launch_kernel(moe_combine_kernel<T, O, V>, row_grid(tokens, h / V, kCombineThreads), dim3(kCombineThreads), 0, s, (const T *)ys, positions,
                      weights, tokens, (int)topk, h, rows, (O *)y) != cudaSuccess)
        return EXL3_ERR_CUDA;
    return launch_status();
}

template <typename T, typename O>
static exl3_status launch_combine(const void *ys, const int32_t *positions, const float *weights, int64_t tokens,
                                  int64_t topk, int64_t h, int64_t rows, void *y, cudaStream_t s)
{
    return h * sizeof(T) % 16 == 0
               ? launch_combine_v<T, O, Vec<T>::N>(ys, positions, weights, tokens, topk, h, rows, y, s)
               : launch_combine_v<T, O, 1>(ys, positions, weights, tokens, topk, h, rows, y, s);
}

template <typename T, int V>
static exl3_status launch_combine_grad(const void *dy, const void *ys, const int32_t *positions, const float *weights,
                                       int64_t tokens, int64_t topk, int64_t h, int64_t rows, void *dys, float *dw,
                                       cudaStream_t s)
{
    const int64_t choices = tokens * topk;
    int64_t grid = (choices + 7) / 8;
    grid = grid < 148 * 64 ? grid : 148 * 64;
    if (launch_kernel(moe_combine_grad_kernel<T, V>, dim3((unsigned)grid), dim3(256), 0, s, (const T *)dy,
                      (const T *)ys, positions, weights, choices, (int)topk, h, rows, (T *)dys, dw) != cudaSuccess)
        return EXL3_ERR_CUDA;
    return launch_status();
}

}  // namespace exl3

extern "C" size_t exl3_moe_sort_workspace_size(int64_t tokens, int64_t topk, int64_t experts)
{
    using namespace exl3;
    if (tokens < 0 || tokens > (int64_t)1 << 24 || topk < 1 || topk > 1024 || experts < 1 || experts > kSortMaxExperts ||
        tokens * topk >= (int64_t)1 << 31)
        return 0;
    return kSyncArea + (size_t)kSortMaxChunks * (size_t)experts * 4;
}

extern "C" exl3_status exl3_moe_sort(const int32_t *ids, int64_t tokens, int64_t topk, int64_t experts,
                                     int32_t *offsets, int32_t *positions, void *workspace, size_t workspace_bytes,
                                     void *stream)
{
    using namespace exl3;
    const size_t need = exl3_moe_sort_workspace_size(tokens, topk, experts);
    if (need == 0)
        return EXL3_ERR_INVALID_ARG;
    const int64_t n = tokens * topk;
    if (!offsets || !aligned16(offsets) || (n && (!ids || !positions || !aligned16(ids) || !aligned16(positions))))
        return EXL3_ERR_INVALID_ARG;
    const size_t nb = (size_t)n * 4, ob = (size_t)(experts + 1) * 4;
    if (n && (ranges_overlap(ids, nb, positions, nb) || ranges_overlap(ids, nb, offsets, ob) ||
              ranges_overlap(positions, nb, offsets, ob)))
        return EXL3_ERR_INVALID_ARG;
    if (!workspace || !aligned16(workspace) || workspace_bytes < need)
        return EXL3_ERR_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t chunk = n ? sort_chunk(n) : kSortThreads;
    const int chunks = n ? (int)((n + chunk - 1) / chunk) : 1;
    int32_t *counts = chunks > 1 ? (int32_t *)((unsigned char *)workspace + kSyncArea) : nullptr;
    if (counts && (launch_kernel(moe_count_kernel, dim3(chunks), dim3(kSortThreads), 0, s, ids, n, chunk, (int)experts,
                                 counts) != cudaSuccess ||
                   launch_status() != EXL3_OK))
        return EXL3_ERR_CUDA;
    const size_t smem = (size_t)kSortWarps * (size_t)experts * 2;
    if (cudaFuncSetAttribute(moe_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSortWarps * kSortMaxExperts * 2) != cudaSuccess)
        return EXL3_ERR_CUDA;
    if (launch_kernel(moe_place_kernel, dim3(chunks), dim3(kSortThreads), smem, s, ids, n, chunk, (int)experts, chunks,
                      (const int32_t *)counts, offsets, positions) != cudaSuccess)
        return EXL3_ERR_CUDA;
    return launch_status();
}

extern "C" exl3_status exl3_moe_gather(const void *x, int dtype, const int32_t *positions, int64_t tokens,
                                       int64_t topk, int64_t h, int64_t rows, void *xs, void *stream)
{
    using namespace exl3;
    if (!valid_route(tokens, topk, h, rows, dtype))
        return EXL3_ERR_INVALID_ARG;
    if (tokens == 0 || rows == 0)
        return EXL3_OK;
    if (!x || !positions || !xs || !aligned16(x) || !aligned16(positions) || !aligned16(xs))
        return EXL3_ERR_INVALID_ARG;
    const size_t row = (size_t)h * dtype_bytes(dtype);
    if (ranges_overlap(x, (size_t)tokens * row, xs, (size_t)rows * row) ||
        ranges_overlap(positions, (size_t)(tokens * topk) * 4, xs, (size_t)rows * row))
        return EXL3_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (row % 16 == 0)
        e = launch_kernel(moe_gather_kernel<uint4>, row_grid(tokens, (int64_t)(row / 16)), dim3(256), 0, s,
                          (const uint4 *)x, positions, tokens, (int)topk, (int64_t)(row / 16), rows, (uint4 *)xs);
    else if (dtype_bytes(dtype) == 4)
        e = launch_kernel(moe_gather_kernel<uint32_t>, row_grid(tokens, h), dim3(256), 0, s, (const uint32_t *)x,
                          positions, tokens, (int)topk, h, rows, (uint32_t *)xs);
    else
        e = launch_kernel(moe_gather_kernel<uint16_t>, row_grid(tokens, h), dim3(256), 0, s, (const uint16_t *)x,
                          positions, tokens, (int)topk, h, rows, (uint16_t *)xs);
    return e == cudaSuccess ? launch_status() : EXL3_ERR_CUDA;
}

extern "C" exl3_status exl3_moe_combine(const void *ys, int dtype, const int32_t *positions, const float *weights,
                                        int64_t tokens, int64_t topk, int64_t h, int64_t rows, void *y, int y_dtype,
                                        void *stream)
{
    using namespace exl3;
    if (!valid_route(tokens, topk, h, rows, dtype) || !valid_dtype(y_dtype) || (y_dtype != dtype && dtype != EXL3_F32))
        return EXL3_ERR_INVALID_ARG;
    if (tokens == 0)
        return EXL3_OK;
    if ((rows && (!ys || !aligned16(ys))) || !positions || !y || !aligned16(positions) || !aligned16(y) ||
        (weights && !aligned16(weights)))
        return EXL3_ERR_INVALID_ARG;
    const size_t row = (size_t)h * dtype_bytes(dtype), yb = (size_t)(tokens * h) * dtype_bytes(y_dtype), cb = (size_t)(tokens * topk) * 4;
    if ((rows && ranges_overlap(ys, (size_t)rows * row, y, yb)) || ranges_overlap(positions, cb, y, yb) ||
        (weights && ranges_overlap(weights, cb, y, yb)))
        return EXL3_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (dtype == EXL3_F16)
        return launch_combine<__half, __half>(ys, positions, weights, tokens, topk, h, rows, y, s);
    if (dtype == EXL3_BF16)
        return launch_combine<__nv_bfloat16, __nv_bfloat16>(ys, positions, weights, tokens, topk, h, rows, y, s);
    switch (y_dtype) {
    case EXL3_F16: return launch_combine<float, __half>(ys, positions, weights, tokens, topk, h, rows, y, s);
    case EXL3_BF16: return launch_combine<float, __nv_bfloat16>(ys, positions, weights, tokens, topk, h, rows, y, s);
    default: return launch_combine<float, float>(ys, positions, weights, tokens, topk, h, rows, y, s);
    }
}

extern "C" exl3_status exl3_moe_combine_grad(const void *dy, const void *ys, int dtype, const int32_t *positions,
                                             const float *weights, int64_t tokens, int64_t topk, int64_t h,
                                             int64_t rows, void *dys, float *dweights, void *stream)
{
    using namespace exl3;
    if (!valid_route(tokens, topk, h, rows, dtype) || (!dys && !dweights))
        return EXL3_ERR_INVALID_ARG;
    if (tokens == 0)
        return EXL3_OK;
    if (!dy || !positions || !aligned16(dy) || !aligned16(positions) || (weights && !aligned16(weights)) ||
        (rows && dweights && (!ys || !aligned16(ys))) || (dys && !aligned16(dys)) || (dweights && !aligned16(dweights)))
        return EXL3_ERR_INVALID_ARG;
    const size_t row = (size_t)h * dtype_bytes(dtype), cb = (size_t)(tokens * topk) * 4, rb = (size_t)rows * row;
    const void *in[4] = {dy, dweights ? ys : nullptr, positions, weights};
    const size_t in_bytes[4] = {(size_t)tokens * row, rb, cb, cb};
    for (int i = 0; i < 4; ++i)
        if (in[i] && ((dys && ranges_overlap(in[i], in_bytes[i], dys, rb)) ||
                      (dweights && ranges_overlap(in[i], in_bytes[i], dweights, cb))))
            return EXL3_ERR_INVALID_ARG;
    if (dys && dweights && ranges_overlap(dys, rb, dweights, cb))
        return EXL3_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    const bool vec = row % 16 == 0;
    switch (dtype) {
    case EXL3_F16:
        return vec ? launch_combine_grad<__half, 8>(dy, ys, positions, weights, tokens, topk, h, rows, dys, dweights, s)
                   : launch_combine_grad<__half, 1>(dy, ys, positions, weights, tokens, topk, h, rows, dys, dweights, s);
    case EXL3_BF16:
        return vec ? launch_combine_grad<__nv_bfloat16, 8>(dy, ys, positions, weights, tokens, topk, h, rows, dys, dweights, s)
                   : launch_combine_grad<__nv_bfloat16, 1>(dy, ys, positions, weights, tokens, topk, h, rows, dys, dweights, s);
    default:
        return vec ? launch_combine_grad<float, 4>(dy, ys, positions, weights, tokens, topk, h, rows, dys, dweights, s)
                   : launch_combine_grad<float, 1>(dy, ys, positions, weights, tokens, topk, h, rows, dys, dweights, s);
    }
}
