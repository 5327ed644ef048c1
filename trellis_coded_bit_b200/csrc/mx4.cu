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
// the definition's.  With it a sum that fp32 rounds across a border of the
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

namespace exl3 {

// 8 consecutive elements.
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8])
{
    if constexpr (sizeof(T) == 2) {
        unpack16<T>(*reinterpret_cast<const uint4 *>(p), v);
    } else {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        const float4 b = *reinterpret_cast<const float4 *>(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
}

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

// Codes of 8 scaled values, the first in the lowest 4 bits (round to nearest
// even, saturating).
__device__ __forceinline__ uint32_t codes8(const float (&r)[8])
{
    uint32_t out;
    asm("{\n.reg .b8 b0, b1, b2, b3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        "mov.b32 %0, {b0, b1, b2, b3};\n}\n"
        : "=r"(out)
        : "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]));
    return out;
}

// The scale byte for a block whose largest magnitude has fp64 bits `bits`.
__device__ __forceinline__ int scale_byte64(uint64_t bits)
{
    const int e = (int)(bits >> 52);  // the sign is clear
    if (e == 2047)
        return 255;
    const int b = e - 1023 - 2 + 127;
    return b < 0 ? 0 : (b > 254 ? 254 : b);
}

__device__ __forceinline__ int scale_byte32(uint32_t bits)
{
    const int e = (int)(bits >> 23);
    if (e == 255)
        return 255;
    return e < 2 ? 0 : e - 2;
}

// 2^(127 - byte) as fp32 (byte 254 gives the subnormal 2^-127).
__device__ __forceinline__ float inverse_scale32(int byte)
{
    return byte >= 254 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(254 - byte) << 23);
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

// Without rotation: a thread takes 8 consecutive columns, 4 threads a block; a
// warp 32 consecutive groups of the matrix read as one long row (a row is a
// multiple of 32 columns, so no block straddles two).
template <typename T>
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
        float v[8];
        load8<T>((const T *)p.x + (row * groups + c) * 8, v);
        if (p.signs) {
            float s[8];
            load8<__half>(p.signs + c * 8, s);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] *= s[i];
        }
        int byte;
        const uint32_t code = quantize8(v, &byte);
        if (!live)
            continue;
        for_each_row(p, row, [&](int64_t to) {
            reinterpret_cast<uint32_t *>(p.codes)[to * groups + c] = code;
            if ((c & 3) == 0)
                store_scale(p, to, c >> 2, byte);
        });
    }
}

// ------------------------------------------------------ with the rotation ---
//
// 4 lanes take the 128 columns of a rotation and end with a block of 32 each (no
// exchange for its largest magnitude, one 16-byte store of codes).  Lane l loads
// columns 32 p + 8 l .. + 7 of the four blocks p, so that 4 lanes read 64
// contiguous bytes; five butterfly stages run over what a lane holds (the low 3
// and high 2 bits of the column), then the lanes exchange halves so that block
// p = l is theirs, and the two stages of the middle bits follow in registers.
// That is 32 shuffles; with a block per lane from the start the same two stages
// took 64, the loads touched four times the lines, and both share one pipe.

// 32-point Sylvester Hadamard in registers, then over the lanes 1 and 2 apart.
template <typename F>
__device__ __forceinline__ void rotate32x4(F (&v)[32])
{
#pragma unroll
    for (int h = 1; h < 32; h <<= 1)
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if ((i & h) == 0) {
                const F a = v[i], b = v[i + h];
                v[i] = a + b;
                v[i + h] = a - b;
            }
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        const F sign = (threadIdx.x & m) ? F(-1) : F(1);
#pragma unroll
        for (int i = 0; i < 32; ++i)
            v[i] = fma(sign, v[i], __shfl_xor_sync(0xffffffffu, v[i], m));  // v + o, or o - v
    }
}

// fp32 arithmetic on two values an instruction.
struct F2 {
    uint64_t v;
};

__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void unpack(F2 p, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}

__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// The rotation of the 128 columns of 4 lanes: v[4p + r/2] holds columns
// 32p + 8l + r, r + 1 before, block l's columns 8p + r, r + 1 after.
__device__ __forceinline__ void rotate32x4(F2 (&v)[16])
{
    const F2 minus = f2(-1.f, -1.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float a, b;
        unpack(v[i], a, b);
        v[i] = f2(a + b, a - b);
    }
#pragma unroll
    for (int h = 1; h < 16; h <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if ((i & h) == 0) {
                const F2 a = v[i], b = v[i + h];
                v[i] = add2(a, b);
                v[i + h] = fma2(b, minus, a);
            }
    // lane bit m <-> bit 4m of i: keep the half whose bit equals the lane's
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        const bool upper = (threadIdx.x & m) != 0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if ((i & (4 * m)) == 0) {
                F2 &lo = v[i], &hi = v[i + 4 * m];
                float a, b;
                unpack(upper ? lo : hi, a, b);
                const F2 got = f2(__shfl_xor_sync(0xffffffffu, a, m), __shfl_xor_sync(0xffffffffu, b, m));
                lo = upper ? got : lo;
                hi = upper ? hi : got;
            }
    }
#pragma unroll
    for (int h = 4; h < 16; h <<= 1)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if ((i & h) == 0) {
                const F2 a = v[i], b = v[i + h];
                v[i] = add2(a, b);
                v[i + h] = fma2(b, minus, a);
            }
}

// Codes of zero magnitude without their sign.
__device__ __forceinline__ uint32_t unsigned_zeros(uint32_t code)
{
    const uint32_t m = code & 0x77777777u;
    const uint32_t some = (m | m >> 1 | m >> 2) & 0x11111111u;
    return m | (code & (some << 3));
}

// A double as the fp32 value that rounds to 4 bits the same way: truncated,
// with the last bit set if anything was cut off, so that a value beside a
// border or a tie stays beside it.
__device__ __forceinline__ float sticky32(double v)
{
    const float f = __double2float_rz(v);
    return (double)f == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// A block in fp64, read again (x, signs: the thread's 32 columns).  A call of
// its own: about one warp in 70 of normal data comes here.
template <typename T>
__device__ __noinline__ uint4 quantize_block_fp64(const T *x, const __half *signs, int *byte)
{
    double v[32];
#pragma unroll
    for (int c = 0; c < 32; c += 8) {
        float f[8];
        load8<T>(x + c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[c + i] = (double)f[i];
        if (signs) {
            load8<__half>(signs + c, f);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[c + i] *= (double)f[i];
        }
    }
    rotate32x4(v);
    uint64_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        v[i] *= 0.088388347648318440550;  // 1/sqrt(128)
        const uint64_t a = (uint64_t)__double_as_longlong(v[i]) & 0x7fffffffffffffffull;
        top = a > top ? a : top;
    }
    const int b = scale_byte64(top);
    *byte = b;
    if (b == 255)
        return make_uint4(0u, 0u, 0u, 0u);
    const double inv = __longlong_as_double((long long)(1023 + 127 - b) << 52);
    uint32_t out[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            r[i] = sticky32(v[8 * c + i] * inv);
        out[c] = unsigned_zeros(codes8(r));
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// Columns 32 p + 8 l .. + 7, p = 0 .. 3, of the 128 from x (x and signs: at column
// 8 l) times their signs.  Signs of exactly +-1 (the usual ones) flip the
// sign bits of 16-bit values in place, a third of the instructions of
// converting and multiplying them.
template <typename T>
__device__ __forceinline__ void load_signed(const T *x, const __half *signs, F2 (&v)[16])
{
    if constexpr (sizeof(T) == 2) {
        uint4 raw[4], sg[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            raw[i] = *reinterpret_cast<const uint4 *>(x + 32 * i);
        if (signs) {
            uint32_t other = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                sg[i] = *reinterpret_cast<const uint4 *>(signs + 32 * i);
                other |= ((sg[i].x ^ 0x3c003c00u) | (sg[i].y ^ 0x3c003c00u) | (sg[i].z ^ 0x3c003c00u) | (sg[i].w ^ 0x3c003c00u)) &
                         0x7fff7fffu;
            }
            if (other == 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    raw[i].x ^= sg[i].x & 0x80008000u;
                    raw[i].y ^= sg[i].y & 0x80008000u;
                    raw[i].z ^= sg[i].z & 0x80008000u;
                    raw[i].w ^= sg[i].w & 0x80008000u;
                }
                signs = nullptr;
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[8];
            unpack16<T>(raw[i], f);
            if (signs) {
                float s[8];
                unpack16<__half>(sg[i], s);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[j] *= s[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[4 * i + j] = f2(f[2 * j], f[2 * j + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[8];
            load8<T>(x + 32 * i, f);
            if (signs) {
                float s[8];
                load8<__half>(signs + 32 * i, s);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    f[j] *= s[j];
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[4 * i + j] = f2(f[2 * j], f[2 * j + 1]);
        }
    }
}

// Error bound.  Each of the 7 stages rounds values whose magnitudes, over the
// tree of one output, add up to at most S = sum |x .* signs| (128 values), by
// 2^-24 each: 7 2^-24 S, and 2^-24 S for the products with the signs.  The
// factor 1/sqrt(128) 2^-e and the product with it are off by 2^-24 of a result
// below 8 each: 2^-20.  Together, in units of the scale,
//     |r - exact| <= 2^-21 S 2^-e / sqrt(128) + 2^-20,
// and `slack` is 2^-8 more than that, for the roundings of S and of itself.
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
        F2 v[16];
        const int shift = 24 * (int)(threadIdx.x & 3);  // from column 32 l to column 8 l
        load_signed(x - shift, signs ? signs - shift : nullptr, v);
        float sum = 0.f, top = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a, b;
            unpack(v[i], a, b);
            sum += fabsf(a) + fabsf(b);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        rotate32x4(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float a, b;
            unpack(v[i], a, b);
            top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
        }
        const float s = 0.08838834764831845f;  // 1/sqrt(128)
        int byte = scale_byte32(__float_as_uint(top * s));
        uint4 code = make_uint4(0u, 0u, 0u, 0u);
        // zeros are exact; what leaves fp32's range or the scales' takes fp64
        bool sure = sum == 0.f;
        if (!sure && byte >= 1 && byte <= 253 && sum < 1e38f) {
            const float inv = inverse_scale32(byte) * s;
            const float slack = fmaf(0x1.01p-21f * sum, inv, 0x1.01p-20f);
            const float most = top * inv;
            const F2 inv2 = f2(inv, inv);
            uint32_t out[4], differ = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float lo[8], hi[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    unpack(fma2(v[4 * i + j], inv2, f2(-slack, -slack)), lo[2 * j], lo[2 * j + 1]);
                    unpack(fma2(v[4 * i + j], inv2, f2(slack, slack)), hi[2 * j], hi[2 * j + 1]);
                }
                const uint32_t a = codes8(lo);
                differ |= (a ^ codes8(hi)) & 0x77777777u;  // equal magnitudes above 0 have equal signs
                out[i] = unsigned_zeros(a);
            }
            code = make_uint4(out[0], out[1], out[2], out[3]);
            sure = differ == 0 && most > 4.f + slack && most < 8.f - slack;
        }
        if (!__all_sync(0xffffffffu, sure))
            code = quantize_block_fp64<T>(x, signs, &byte);
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

// Bound by the values' bytes.  A thread writes 8 consecutive values (16 or 32
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
    const cudaError_t e =
        rotate ? launch_kernel(mx4_rotate_quantize_kernel<T>, dim3(mx4_grid(p.rows * p.blocks, 128)), dim3(128), 0, s, p)
               : launch_kernel(mx4_quantize_kernel<T>, dim3(mx4_grid(p.rows * p.blocks * 4, 256)), dim3(256), 0, s, p);
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
