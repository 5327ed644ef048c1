// mx4.cuh -- the 4-bit microscaled format, shared by its quantiser and its
// matmul kernels.
//
// A matrix of r rows and k columns (k, a multiple of 32, runs along the sums
// of a matmul) is stored as
//   codes   uint8 [r][k/2]: column c's code is the low (c even) or high half
//           of byte c/2; a code is sign, 2 exponent bits, 1 mantissa bit
//           (e2m1): magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6;
//   scales  uint8 [r][mx4_scale_stride(k)]: byte b scales columns 32b .. 32b+31
//           by 2^(byte - 127) (e8m0; 255 is NaN).
#pragma once

#include <stdint.h>

namespace exl3 {

constexpr int kMx4Block = 32;

// Bytes of a row of scales: rows start on 16 bytes, so that a thread can take
// 16 scales (512 columns) in one load.
__host__ __device__ inline int64_t mx4_scale_stride(int64_t k)
{
    return (k + 511) / 512 * 16;
}

inline bool valid_mx4_k(int64_t k)
{
    return k >= kMx4Block && k % kMx4Block == 0 && k <= (int64_t)1 << 22;
}

inline bool valid_mx4_rows(int64_t rows)
{
    return rows >= 0 && rows <= (int64_t)1 << 30;
}

}  // namespace exl3
