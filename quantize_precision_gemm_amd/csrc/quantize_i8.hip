// quantize_i8.hip -- symmetric 8-bit integer quantisation of the rows of a
// bf16 matrix: one fp32 scale per row (a token of an activation, an output
// channel of a weight).
//
//   amax_r = max_k |x[r, k]|,  scale_r = amax_r / 127,
//   code[r, k] = rint(127 x[r, k] / amax_r), ties to even, in [-127, 127].
// 127 x is exact in fp32 for a bf16 x and the quotient is rounded once, so a
// code is the one that exact arithmetic gives: with significands X and A of 8
// bits, 127 X / (A 2^d) that is no tie differs from one by at least
// 1 / (2 A 2^d), that is 1 / (254 X) > 2^-16 of its value, and fp32 rounds by
// 2^-24 of it.
//
// Bound by HBM traffic: 2 bytes read and 1 written per element.
#include "internal.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// Factor that keeps 127 x below fp32's maximum (a power of two on both sides
// of the quotient leaves it as it is).
__device__ __forceinline__ float headroom(float amax) { return amax >= 0x1p120f ? 0x1p-8f : 1.0f; }

__device__ __forceinline__ uint32_t code_of(float x, float amax_s)
{
    const float y = (x * 127.0f) / amax_s;
    return (uint32_t)(int)__builtin_rintf(__builtin_fminf(__builtin_fmaxf(y, -127.0f), 127.0f)) & 0xFFu;
}

}  // namespace

// One workgroup per row: the maximum, then the codes (the row's second read
// comes from the cache).
__global__ __launch_bounds__(kThreads) void k_i8_quant(const uint16_t* __restrict__ x, int64_t cols, int64_t ld,
                                                       int8_t* __restrict__ codes, int64_t ld_codes,
                                                       float* __restrict__ scales)
{
    __shared__ uint32_t part[kThreads / 64];
    const int64_t row = blockIdx.x;
    const uint16_t* src = x + row * ld;
    uint32_t top = 0;
    for (int64_t k = 8 * (int64_t)threadIdx.x; k < cols; k += 8 * kThreads) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    }
    top = wave_max_u32(top);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(part[0], part[1]), max(part[2], part[3]));
    const float amax = __uint_as_float(top << 16);
    if (threadIdx.x == 0) scales[row] = amax / 127.0f;
    const float f = headroom(amax);
    const float amax_s = amax > 0.0f ? amax * f : 1.0f;
    int8_t* dst = codes + row * ld_codes;
    for (int64_t k = 8 * (int64_t)threadIdx.x; k < cols; k += 8 * kThreads) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + k);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t lo = code_of(__uint_as_float(w[j] << 16) * f, amax_s);
            const uint32_t hi = code_of(__uint_as_float(w[j] & 0xFFFF0000u) * f, amax_s);
            o[j >> 1] |= (lo | (hi << 8)) << (16 * (j & 1));
        }
        *reinterpret_cast<uint2*>(dst + k) = make_uint2(o[0], o[1]);
    }
}

void launch_i8_quant(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes, int64_t ld_codes,
                     float* scales, hipStream_t s)
{
    if (rows == 0) return;
    hipLaunchKernelGGL(k_i8_quant, dim3((uint32_t)rows), dim3(kThreads), 0, s, x, cols, ld, codes, ld_codes, scales);
}

}  // namespace nvfp4
