// mx4.cu -- exl3_mx4_quantize and exl3_mx4_dequantize: the 4-bit microscaled
// format (mx4.cuh) from fp16/bf16/fp32 rows and back.
//
// Quantisation of 32 values v (after x' = H128(x .* signs)/sqrt(128) if asked
// for): e = floor(log2(max |v|)) - 2, clamped to [-127, 127], so that the
// largest magnitude lies in [4, 8) 2^e; each code is v 2^-e rounded to the
// nearest code, ties to the even one, magnitudes over 6 taken to 6.  A block
// that holds an infinity or a NaN gets the scale byte 255 and codes 0.
//
// The scaling by a power of two is exact, so without the rotation every code is
// that of the product with the sign (mx4_quantize.cuh).  With it a sum that fp32 rounds across a border of the
// 4-bit rounding would put its code off by a whole step of the format, and two
// ways to the same sum would disagree by that step.  So the rotation runs in
// fp32 with a bound on its error, and where a value (or a block's largest)
// lies within the bound of a border its warp repeats it in fp64, whose sums are
// exact for 128 fp16 values and good to 2^-46 of the largest for bf16 and fp32
// ones.  (A rotated zero has the code of +0.)
#include "dtypes.cuh"
#include "exl3_device.cuh"
#include "exl3_host.h"
#include "mx4.cuh"
#include "mx4_quantize.cuh"

namespace exl3 {

// Row and column group of group g of a matrix with `groups` a row (64-bit
// division costs ten times the 32-bit one, which nearly every matrix allows).
__device__ __forceinline__ void split_group(int64_t g, int groups, int64_t &row, int &c)
{
    if ((uint64_t)g >> 32) {
        row = g / groups;
        c = (int)(g - row * groups);
    } else {
        const uint32_t r = (uint32_t)g / (uint32_t)groups;
        row = r;
        c = (int)((uint32_t)g - r * (uint32_t)groups);
    }
}

// Codes and scale byte of this thread's 8 columns of a block of 32 (4 lanes).
__device__ __forceinline__ uint32_t quantize8(const float (&v)[8], int *byte)
{
    uint32_t top = 0;  // magnitudes order like their bits, NaN above infinity
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int b = scale_byte32(top);
    *byte = b;
    if (b == 255)
        return 0u;
    const float inv = inverse_scale32(b);
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r[i] = v[i] * inv;
    return codes8(r);
}

// The same in fp64, for products with the signs that fp32 does not hold.
template <typename T>
__device__ __forceinline__ uint32_t quantize8_products(const T *x, const __half *signs, int *byte)
{
    double v[8];
    uint64_t top = products8<T>(x, signs, v);
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        const uint64_t o = __shfl_xor_sync(0xffffffffu, (unsigned long long)top, m);
        top = o > top ? o : top;
    }
    const int b = scale_byte64(top);
    *byte = b;
    return b == 255 ? 0u : codes8(v, b);
}

struct Mx4QuantParams {
    const void *x;
    const __half *signs;
    const int32_t *positions;  // row r goes to rows positions[r topk ..] (null: to row r)
    uint8_t *codes, *scales;
    int64_t rows, out_rows;
    int blocks;                // k / 32
    int topk, stride;          // stride: bytes of a row of scales
};

// Calls f with each of the rows that row `row` goes to.
template <typename F>
__device__ __forceinline__ void for_each_row(const Mx4QuantParams &p, int64_t row, F f)
{
    if (!p.positions) {
        f(row);
        return;
    }
    for (int j = 0; j < p.topk; ++j) {
        const int64_t to = p.positions[row * p.topk + j];
        if (to >= 0 && to < p.out_rows)
            f(to);
    }
}

// Scale of block b of a row; behind the last block also the unused bytes.
__device__ __forceinline__ void store_scale(const Mx4QuantParams &p, int64_t row, int b, int byte)
{
    uint8_t *s = p.scales + row * p.stride + b;
    *s = (uint8_t)byte;
    if (b + 1 == p.blocks)
        for (int i = b + 1; i < p.stride; ++i)
            *++s = 0;
}

// Bound by the bytes: 14336 x 4096 fp32 in 50 us, 5.3 TB/s.
// Without rotation: a thread takes 8 consecutive columns, 4 threads a block; a
// warp 32 consecutive groups of the matrix read as one long row (a row is a
// multiple of 32 columns, so no block straddles two).
// WIDE: there are signs, and a product may be more than fp32 holds: a warp that
// meets one takes its groups in fp64.  4096 x 8192 bf16 / fp32, us, in a graph behind
// an L2 flush: no signs 30.7 / 34.8, signs of +-1 34.8 / 37.0, other signs 57 / 57.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const Mx4QuantParams p)
{
    grid_dep_wait();
    grid_dep_launch();
    const int groups = p.blocks * 4;
    const int64_t total = p.rows * groups;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    // rounded up to whole warps: every lane takes part in the shuffles
    for (int64_t g0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x - (threadIdx.x & 31); g0 < total; g0 += stride) {
        const int64_t g = g0 + (threadIdx.x & 31);
        const bool live = g < total;
        int64_t row = 0;
        int c = 0;
        if (live)
            split_group(g, groups, row, c);
        const T *const x = (const T *)p.x + (row * groups + c) * 8;
        float v[8];
        load8<T>(x, v);
        uint32_t other = 0;
        if (p.signs) {
            const uint4 raw = *reinterpret_cast<const uint4 *>(p.signs + c * 8);
            float s[8];
            unpack16<__half>(raw, s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] *= s[i];
            other = WIDE ? other_than_ones(raw) : 0u;
        }
        int byte;
        uint32_t code = quantize8(v, &byte);
        if (WIDE && __any_sync(0xffffffffu, other != 0))
            code = quantize8_products<T>(x, p.signs + c * 8, &byte);
        if (!live)
            continue;
        for_each_row(p, row, [&](int64_t to) {
            reinterpret_cast<uint32_t *>(p.codes)[to * groups + c] = code;
            if ((c & 3) == 0)
                store_scale(p, to, c >> 2, byte);
        });
    }
}

// A lane per block of 32, 4 lanes a rotation (mx4_quantize.cuh).
// 2048 x 8192 fp16 in 22 us (2.0 TB/s; its bytes take 6.5 us, its 680 instructions a
// warp and 1024 values 10 us of issue): bound by latency.  126 registers leave 4
// warps a scheduler, each with one block's chain of loads, butterflies and shuffles
// in flight and, now and then, the fp64 repeat; they issue on half of the cycles.
template <typename T>
__global__ void __launch_bounds__(128) mx4_rotate_quantize_kernel(const Mx4QuantParams p)
{
    grid_dep_wait();
    grid_dep_launch();
    const int64_t total = p.rows * p.blocks;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t g0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x - (threadIdx.x & 31); g0 < total; g0 += stride) {
        const int64_t g = g0 + (threadIdx.x & 31);
        const bool live = g < total;
        int64_t row = 0;
        int c = (int)(threadIdx.x & 3);
        if (live)
            split_group(g, p.blocks, row, c);
        const T *const x = (const T *)p.x + (row * p.blocks + c) * 32;
        const __half *const signs = p.signs ? p.signs + c * 32 : nullptr;
        int byte;
        const uint4 code = quantize_block_rotated<T>(x, signs, &byte);
        if (!live)
            continue;
        for_each_row(p, row, [&](int64_t to) {
            reinterpret_cast<uint4 *>(p.codes)[to * p.blocks + c] = code;
            store_scale(p, to, c, byte);
        });
    }
}

// ------------------------------------------------------------ dequantise ---

// Magnitudes and signs of 8 codes (exact in fp16, through which the conversion goes).
__device__ __forceinline__ void decode8(uint32_t code, float (&v)[8])
{
    uint32_t h[4];
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "mov.b32 {b0, b1, b2, b3}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(code));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 p;
        memcpy(&p, &h[i], 4);
        const float2 f = __half22float2(p);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

// 8 fp32 values in one 32-byte store.
__device__ __forceinline__ void store8(float *p, const float (&v)[8])
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

constexpr int kDequantAhead = 4;  // groups of 8 values whose loads a thread keeps in flight

// Bound by the values' bytes: 14336 x 4096 to fp32 in 42 us, 6.4 TB/s.  A thread writes 8 consecutive values (16 or 32
// bytes) of each of 4 groups that lie a grid apart; `wide`: fp32 rows start on
// 32 bytes, as the 32-byte store needs.
template <typename T>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint32_t *__restrict__ codes,
                                                             const uint8_t *__restrict__ scales, int64_t rows,
                                                             int groups, int stride, bool wide, T *__restrict__ w)
{
    grid_dep_wait();
    grid_dep_launch();
    const int64_t total = rows * groups;
    const int64_t threads = (int64_t)gridDim.x * blockDim.x;
    for (int64_t g0 = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; g0 < total; g0 += threads * kDequantAhead) {
        uint32_t code[kDequantAhead];
        int byte[kDequantAhead];
#pragma unroll
        for (int j = 0; j < kDequantAhead; ++j) {
            const int64_t g = g0 + j * threads;
            if (g < total) {
                int64_t row;
                int c;
                split_group(g, groups, row, c);
                code[j] = codes[g];
                byte[j] = scales[row * stride + (c >> 2)];
            }
        }
#pragma unroll
        for (int j = 0; j < kDequantAhead; ++j) {
            const int64_t g = g0 + j * threads;
            if (g >= total)
                break;
            const int b = byte[j];
            const float s = b == 255 ? __uint_as_float(0x7fc00000u)
                                     : (b ? __uint_as_float((uint32_t)b << 23) : __uint_as_float(0x00400000u));
            float v[8];
            decode8(code[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] *= s;
            if constexpr (sizeof(T) == 2) {
                *reinterpret_cast<uint4 *>(w + g * 8) = pack16<T>(v);
            } else if (wide) {
                store8(w + g * 8, v);
            } else {
                *reinterpret_cast<float4 *>(w + g * 8) = make_float4(v[0], v[1], v[2], v[3]);
                *reinterpret_cast<float4 *>(w + g * 8 + 4) = make_float4(v[4], v[5], v[6], v[7]);
            }
        }
    }
}

static unsigned mx4_grid(int64_t threads, int block)
{
    const int64_t blocks = (threads + block - 1) / block;
    return (unsigned)(blocks < 148 * 32 ? blocks : 148 * 32);
}

template <typename T>
static exl3_status launch_quantize(const Mx4QuantParams &p, bool rotate, cudaStream_t s)
{
    const dim3 grid(rotate ? mx4_grid(p.rows * p.blocks, 128) : mx4_grid(p.rows * p.blocks * 4, 256));
    const bool wide = !kExactProducts<T> && p.signs;
    const cudaError_t e = rotate ? launch_kernel(mx4_rotate_quantize_kernel<T>, grid, dim3(128), 0, s, p)
                          : wide ? launch_kernel(mx4_quantize_kernel<T, !kExactProducts<T>>, grid, dim3(256), 0, s, p)
                                 : launch_kernel(mx4_quantize_kernel<T, false>, grid, dim3(256), 0, s, p);
    if (e != cudaSuccess)
        return EXL3_ERR_CUDA;
    return launch_status();
}

}  // namespace exl3

extern "C" int64_t exl3_mx4_scale_stride(int64_t k)
{
    return exl3::valid_mx4_k(k) ? exl3::mx4_scale_stride(k) : 0;
}

extern "C" exl3_status exl3_mx4_quantize(const void *x, int dtype, const void *signs, int rotate,
                                         const int32_t *positions, int64_t topk, int64_t out_rows, uint8_t *codes,
                                         uint8_t *scales, int64_t rows, int64_t k, void *stream)
{
    using namespace exl3;
    if (!valid_mx4_k(k) || !valid_mx4_rows(rows) || (rotate && k % 128) ||
        (dtype != EXL3_F16 && dtype != EXL3_BF16 && dtype != EXL3_F32))
        return EXL3_ERR_INVALID_ARG;
    if (positions && (topk < 1 || topk > 1024 || !valid_mx4_rows(out_rows) || !aligned16(positions)))
        return EXL3_ERR_INVALID_ARG;
    const int64_t to_rows = positions ? out_rows : rows;
    if (rows == 0 || to_rows == 0)
        return EXL3_OK;
    if (!x || !codes || !scales || !aligned16(x) || !aligned16(codes) || !aligned16(scales) ||
        (signs && !aligned16(signs)))
        return EXL3_ERR_INVALID_ARG;
    const size_t xb = (size_t)rows * (size_t)k * (dtype == EXL3_F32 ? 4 : 2);
    const size_t cb = (size_t)to_rows * (size_t)(k / 2), sb = (size_t)(to_rows * mx4_scale_stride(k));
    const void *in[3] = {x, signs, positions};
    const size_t in_bytes[3] = {xb, (size_t)k * 2, (size_t)rows * (size_t)topk * 4};
    for (int i = 0; i < 3; ++i)
        if (in[i] && (ranges_overlap(in[i], in_bytes[i], codes, cb) || ranges_overlap(in[i], in_bytes[i], scales, sb)))
            return EXL3_ERR_INVALID_ARG;
    if (ranges_overlap(codes, cb, scales, sb))
        return EXL3_ERR_INVALID_ARG;
    Mx4QuantParams p;
    p.x = x;
    p.signs = (const __half *)signs;
    p.positions = positions;
    p.codes = codes;
    p.scales = scales;
    p.rows = rows;
    p.out_rows = to_rows;
    p.blocks = (int)(k / 32);
    p.topk = positions ? (int)topk : 1;
    p.stride = (int)mx4_scale_stride(k);
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
    case EXL3_F16: return launch_quantize<__half>(p, rotate != 0, s);
    case EXL3_BF16: return launch_quantize<__nv_bfloat16>(p, rotate != 0, s);
    default: return launch_quantize<float>(p, rotate != 0, s);
    }
}

extern "C" exl3_status exl3_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, void *w, int dtype,
                                           int64_t rows, int64_t k, void *stream)
{
    using namespace exl3;
    if (!valid_mx4_k(k) || !valid_mx4_rows(rows) || (dtype != EXL3_F16 && dtype != EXL3_BF16 && dtype != EXL3_F32))
        return EXL3_ERR_INVALID_ARG;
    if (rows == 0)
        return EXL3_OK;
    if (!w || !codes || !scales || !aligned16(w) || !aligned16(codes) || !aligned16(scales))
        return EXL3_ERR_INVALID_ARG;
    const size_t wb = (size_t)rows * (size_t)k * (dtype == EXL3_F32 ? 4 : 2);
    if (ranges_overlap(codes, (size_t)rows * (size_t)(k / 2), w, wb) ||
        ranges_overlap(scales, (size_t)(rows * mx4_scale_stride(k)), w, wb))
        return EXL3_ERR_INVALID_ARG;
    const int groups = (int)(k / 8), stride = (int)mx4_scale_stride(k);
    const dim3 grid(mx4_grid((rows * groups + kDequantAhead - 1) / kDequantAhead, 256)), block(256);
    const bool wide = ((uintptr_t)w & 31u) == 0;
    cudaStream_t s = (cudaStream_t)stream;
    const uint32_t *c = (const uint32_t *)codes;
    cudaError_t e;
    switch (dtype) {
    case EXL3_F16:
        e = launch_kernel(mx4_dequantize_kernel<__half>, grid, block, 0, s, c, scales, rows, groups, stride, wide, (__half *)w);
        break;
    case EXL3_BF16:
        e = launch_kernel(mx4_dequantize_kernel<__nv_bfloat16>, grid, block, 0, s, c, scales, rows, groups, stride,
                          wide, (__nv_bfloat16 *)w);
        break;
    default:
        e = launch_kernel(mx4_dequantize_kernel<float>, grid, block, 0, s, c, scales, rows, groups, stride, wide, (float *)w);
    }
    return e == cudaSuccess ? launch_status() : EXL3_ERR_CUDA;
}
