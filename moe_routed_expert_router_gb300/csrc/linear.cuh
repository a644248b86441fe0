// What the two kernels of the 4-bit product of a few tokens share.
#pragma once

#include "rows.cuh"

namespace moe {

// The power of two that brings values whose largest finite magnitude has exponent e to [2^7, 2^8), in two factors, and
// what undoes it; e is -127 where all are subnormals or zeros.
__device__ __forceinline__ int exponent_of(float amax) { return (int)(__float_as_uint(amax) >> 23) - 127; }
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }    // -126 to 127
__device__ __forceinline__ float scale_up(int e) { return power_of_two(min(7 - e, 127)); }
__device__ __forceinline__ float scale_more(int e) { return power_of_two(max(0, 7 - e - 127)); }
__device__ __forceinline__ float scale_down(int e) { return power_of_two(max(e - 7, -126)) * power_of_two(min(0, e - 7 + 126)); }

// A tensor scale's power of two and the rest.  The power goes back into the sums together with the tokens' own, so that a
// sum passes fp32's range only where the result does: all of a power that makes sums larger, and of one that makes them
// smaller 2^-28, for 65536 products of 2^128 * 2688 are below 2^156.  (Any more would only round results below fp32's
// smallest normal number more than once.)
struct TensorScale {
    int power;                   // -28 to 126
    float rest;
};
__device__ __forceinline__ TensorScale split_scale(float ts) {
    const int e = exponent_of(fabsf(ts));
    const int power = e > 127 ? 0 : max(-28, min(e, 126));           // 128: an infinity or a NaN
    return {power, ts * power_of_two(-power)};
}
// 2^c as two factors, for any sum of those two powers: below 2^-200 no product of a sum is left.
__device__ __forceinline__ float first_factor(int c) { return power_of_two(max(-126, min(c, 127))); }
__device__ __forceinline__ float second_factor(int c) { return power_of_two(max(c, -200) - max(-126, min(c, 127))); }

// A call, checked.
struct LinearCall {
    const void *x;
    int64_t x_stride;
    const uint8_t *codes, *scales;
    const float *ts;             // null: MXFP4
    int T, N, K;
    int dtype, out_dtype;
    void *out, *workspace;
};

// Bytes of workspace of the block-scaled tensor-core kernel; 0: the call is not for it.
size_t linear_tc_workspace(bool mx, bool f16, int T, int N, int K);
cudaError_t launch_linear_tc(const LinearCall &c, cudaStream_t st);

}  // namespace moe
