// mx4_quantize.cuh -- 4-bit microscaled quantisation of blocks of 32 values, with
// and without the 128-point rotation: shared by the quantiser (mx4.cu) and by the
// product of a token or two, which quantises its own activations (mx4_gemm.cu).
//
// The definition: e = floor(log2(max |v|)) - 2, clamped to [-127, 127]; codes are
// v 2^-e rounded to nearest, ties to the even code, magnitudes over 6 taken to 6;
// a block with an infinity or a NaN has the scale byte 255 and codes 0.
//
// v is x or x .* signs, the exact products: fp32 holds them for fp16 x (22 bits,
// 2^-48 .. 2^32) and for signs of +-1; otherwise (fp32 products of 35 bits, bf16
// products outside fp32's range) a block is taken in fp64.
#pragma once

#include <type_traits>

#include "dtypes.cuh"
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

// 2^(127 - byte) as fp64.
__device__ __forceinline__ double inverse_scale64(int byte)
{
    return __longlong_as_double((long long)(1023 + 127 - byte) << 52);
}

// A double as the fp32 value that rounds to 4 bits the same way: truncated,
// with the last bit set if anything was cut off, so that a value beside a
// border or a tie stays beside it.
__device__ __forceinline__ float sticky32(double v)
{
    const float f = __double2float_rz(v);
    return (double)f == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Nonzero bits where 8 signs are not +-1.
__device__ __forceinline__ uint32_t other_than_ones(uint4 s)
{
    return ((s.x ^ 0x3c003c00u) | (s.y ^ 0x3c003c00u) | (s.z ^ 0x3c003c00u) | (s.w ^ 0x3c003c00u)) & 0x7fff7fffu;
}

// Whether fp32 holds the products of any T with any fp16.
template <typename T>
constexpr bool kExactProducts = std::is_same<T, __half>::value;

// 8 exact products and their largest magnitude's bits (NaN above infinity).
template <typename T>
__device__ __forceinline__ uint64_t products8(const T *x, const __half *signs, double (&v)[8])
{
    float f[8], s[8];
    load8<T>(x, f);
    load8<__half>(signs, s);
    uint64_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = (double)f[i] * (double)s[i];
        const uint64_t a = (uint64_t)__double_as_longlong(v[i]) & 0x7fffffffffffffffull;
        top = a > top ? a : top;
    }
    return top;
}

__device__ __forceinline__ uint32_t codes8(const double (&v)[8], int byte)
{
    const double inv = inverse_scale64(byte);
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r[i] = sticky32(v[i] * inv);
    return codes8(r);
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

// A block in fp64, read again (x, signs: the thread's 32 columns), where its
// scale is in doubt or out of fp32's range.
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
    const double inv = inverse_scale64(b);
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

// The codes in doubt alone (`differ`: nonzero nibbles), each from the exact sum:
// every group of 4 lanes takes its first one in turn, a lane summing its 32
// columns with the signs of that row of the Hadamard matrix,
// (-1)^popcount(row & column).  A call of its own: about one warp in 30 of normal
// data comes here, nearly always with one code.
template <typename T>
__device__ __noinline__ uint4 settle_codes(const T *x, const __half *signs, uint4 code, uint4 differ, int byte)
{
    const int lane = threadIdx.x & 31, l = lane & 3, group0 = lane & ~3;
    for (;;) {
        const bool mine = (differ.x | differ.y | differ.z | differ.w) != 0;
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        if (who == 0)
            return code;
        // the group's first lane in doubt, its first code and its scale
        const uint32_t in_group = (who >> group0) & 15u;
        const int src = in_group ? __ffs((int)in_group) - 1 : 0;
        const uint32_t word = differ.x ? differ.x : differ.y ? differ.y : differ.z ? differ.z : differ.w;
        const int index = differ.x ? 0 : differ.y ? 1 : differ.z ? 2 : 3;
        const int first = 8 * index + (word ? (__ffs((int)word) - 1) / 4 : 0);
        const int e = __shfl_sync(0xffffffffu, first, group0 + src);
        // bit j: the sign of column j of a block in row e (within a block)
        uint32_t row = 0;
        row ^= (e & 1) ? 0xaaaaaaaau : 0u;
        row ^= (e & 2) ? 0xccccccccu : 0u;
        row ^= (e & 4) ? 0xf0f0f0f0u : 0u;
        row ^= (e & 8) ? 0xff00ff00u : 0u;
        row ^= (e & 16) ? 0xffff0000u : 0u;
        row ^= (__popc(src & l) & 1) ? 0xffffffffu : 0u;
        // neighbours first, as the butterflies of quantize_block_fp64 add: the same
        // roundings where the sums are not exact
        double part[4];
#pragma unroll
        for (int c = 0; c < 32; c += 8) {
            float f[8], s[8];
            double v[8];
            load8<T>(x + c, f);
            if (signs)
                load8<__half>(signs + c, s);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = signs ? (double)f[j] * (double)s[j] : (double)f[j];
                v[j] = (row >> (c + j) & 1u) ? -v[j] : v[j];
            }
            part[c / 8] = ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        double sum = (part[0] + part[1]) + (part[2] + part[3]);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (mine && l == src) {
            sum *= 0.088388347648318440550;  // 1/sqrt(128)
            float r[8] = {sticky32(sum * inverse_scale64(byte)), 0.f, 0.f, 0.f,
                          0.f, 0.f, 0.f, 0.f};
            const uint32_t q = unsigned_zeros(codes8(r)) & 15u;
            const int shift = 4 * (e & 7);
            const uint32_t keep = ~(15u << shift);
            uint32_t *const c = index == 0 ? &code.x : index == 1 ? &code.y : index == 2 ? &code.z : &code.w;
            *c = (*c & keep) | (q << shift);
            differ.x &= index == 0 ? keep : 0xffffffffu;
            differ.y &= index == 1 ? keep : 0xffffffffu;
            differ.z &= index == 2 ? keep : 0xffffffffu;
            differ.w &= index == 3 ? keep : 0xffffffffu;
        }
    }
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
                other |= other_than_ones(sg[i]);
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
// A product with a sign that fp32 holds only below its normal numbers is off by
// 2^-150 instead: 128 of them, 2^-143, or with kFp32Byte, whose scale is 2^-111,
// 2^-35 of the scale, which the 2^-8 covers (they are at least 2^-27 of it).
constexpr int kFp32Byte = 16;

// The block of 32 columns at x (signs: its signs, or null) with the 128-point
// rotation: codes and scale byte.  The whole warp calls it, 4 consecutive lanes
// on the consecutive blocks of 128 columns.  SETTLE: only the codes in doubt are
// summed again (a tenth of the code to fetch, which is what a single call waits
// for; over many blocks the whole warp's repeat in fp64 is quicker, 21.5 us
// against 23.3 for 2048 x 8192 fp16).
template <typename T, bool SETTLE = false>
__device__ __forceinline__ uint4 quantize_block_rotated(const T *x, const __half *signs, int *out_byte)
{
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
    bool sure = sum == 0.f;  // of the scale
    uint32_t differ[4] = {0u, 0u, 0u, 0u};
    if (!sure && byte >= kFp32Byte && byte <= 253 && sum < 1e38f) {
        const float inv = inverse_scale32(byte) * s;
        const float slack = fmaf(0x1.01p-21f * sum, inv, 0x1.01p-20f);
        const float most = top * inv;
        const F2 inv2 = f2(inv, inv);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo[8], hi[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                unpack(fma2(v[4 * i + j], inv2, f2(-slack, -slack)), lo[2 * j], lo[2 * j + 1]);
                unpack(fma2(v[4 * i + j], inv2, f2(slack, slack)), hi[2 * j], hi[2 * j + 1]);
            }
            const uint32_t a = codes8(lo);
            differ[i] = (a ^ codes8(hi)) & 0x77777777u;  // equal magnitudes above 0 have equal signs
            out[i] = unsigned_zeros(a);
        }
        code = make_uint4(out[0], out[1], out[2], out[3]);
        sure = most > 4.f + slack && most < 8.f - slack;
    }
    if (!SETTLE)
        sure = sure && (differ[0] | differ[1] | differ[2] | differ[3]) == 0;
    if (!__all_sync(0xffffffffu, sure))
        code = quantize_block_fp64<T>(x, signs, &byte);
    else if (SETTLE && __any_sync(0xffffffffu, (differ[0] | differ[1] | differ[2] | differ[3]) != 0))
        code = settle_codes<T>(x, signs, code, make_uint4(differ[0], differ[1], differ[2], differ[3]), byte);
    *out_byte = byte;
    return code;
}

// The block of 32 columns at x times the signs there, in fp64.
template <typename T>
__device__ __forceinline__ uint4 quantize_block_products(const T *x, const __half *signs, int *out_byte)
{
    uint64_t top = 0;
    double v[8];
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        const uint64_t t = products8<T>(x + i, signs + i, v);
        top = t > top ? t : top;
    }
    const int byte = scale_byte64(top);
    *out_byte = byte;
    if (byte == 255)
        return make_uint4(0u, 0u, 0u, 0u);
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        products8<T>(x + 8 * i, signs + 8 * i, v);
        out[i] = codes8(v, byte);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// The same without rotation, each lane by itself.
template <typename T>
__device__ __forceinline__ uint4 quantize_block(const T *x, const __half *signs, int *out_byte)
{
    float v[32];
    uint32_t top = 0;  // magnitudes order like their bits, NaN above infinity
    uint32_t other = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        float f[8];
        load8<T>(x + i, f);
        if (signs) {
            const uint4 raw = *reinterpret_cast<const uint4 *>(signs + i);
            float s[8];
            unpack16<__half>(raw, s);
            other |= kExactProducts<T> ? 0u : other_than_ones(raw);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                f[j] *= s[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[i + j] = f[j];
            top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
        }
    }
    if (!kExactProducts<T> && other)
        return quantize_block_products<T>(x, signs, out_byte);
    const int byte = scale_byte32(top);
    *out_byte = byte;
    if (byte == 255)
        return make_uint4(0u, 0u, 0u, 0u);
    const float inv = inverse_scale32(byte);
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            r[j] = v[8 * i + j] * inv;
        out[i] = codes8(r);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

}  // namespace exl3
