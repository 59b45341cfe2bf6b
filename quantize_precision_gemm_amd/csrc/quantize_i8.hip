// quantize_i8.hip -- symmetric 8-bit integer quantisation of the rows of a
// bf16 matrix: one fp32 scale per row (a token of an activation, an output
// channel of a weight).
//
//   amax_r = max_k |x[r, k]|,  scale_r = amax_r / 127,
//   code[r, k] = rint(127 x[r, k] / amax_r), ties to even, in [-127, 127].
// A row whose maximum is not finite keeps that as its scale; its codes are 0
// (the factor is 0, and an element that is not finite times 0 is NaN).
// 127 x is exact in fp32 for a bf16 x and the quotient is rounded once, so a
// code is the one that exact arithmetic gives: with significands X and A of 8
// bits, 127 X / (A 2^d) that is no tie differs from one by at least
// 1 / (2 A 2^d), that is 1 / (254 X) > 2^-16 of its value, and fp32 rounds by
// 2^-24 of it.
//
// A true division of every element would bind the kernel to its arithmetic
// (37 us for 8192 x 5120): y = x (127 / amax), two roundings, lies within
// 2^-23 of the quotient, and rounding y to 18 bits makes a tie a tie again
// (it has 8 bits) without carrying any other quotient across one.
//
// Bound by HBM traffic: 2 bytes read and 1 written per element (8192 x 5120
// 22.2 us, 5.7 TB/s with its inputs partly in the last-level cache); one short
// row takes 2.2 us.
#include "internal.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kHeld = 4;  // 16-byte pieces that a lane keeps between the maximum and the codes

__device__ __forceinline__ uint32_t max_of(uint32_t top, const uint4& v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    return top;
}

__device__ __forceinline__ uint32_t code_of(float x, float scale)
{
    const float y = x * scale;
    const float t = y * 65.0f;              // y to 18 bits: 24 - 6
    const float y18 = t - (t - y);
    // the instruction takes NaN as 0, a C++ conversion leaves it undefined (a
    // mask that clears such a row first cost 20.8 -> 21.1 us for 8192 x 5120)
    uint32_t code;
    asm("v_cvt_i32_f32 %0, %1" : "=v"(code) : "v"(__builtin_rintf(y18)));
    return code & 0xFFu;
}

__device__ __forceinline__ uint2 codes_of(const uint4& v, float lift, float scale)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t lo = code_of(__uint_as_float(w[j] << 16) * lift, scale);
        const uint32_t hi = code_of(__uint_as_float(w[j] & 0xFFFF0000u) * lift, scale);
        o[j >> 1] |= (lo | (hi << 8)) << (16 * (j & 1));
    }
    return make_uint2(o[0], o[1]);
}

}  // namespace

// kWaves waves per row (4: a workgroup of one row; 1: a workgroup of 4 rows).
template <int kWaves>
__global__ __launch_bounds__(256) void k_i8_quant(const uint16_t* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                                                  int8_t* __restrict__ codes, int64_t ld_codes,
                                                  float* __restrict__ scales)
{
    constexpr int kLanes = 64 * kWaves, kRows = 4 / kWaves;
    __shared__ uint32_t part[4];
    const int lane = kWaves == 4 ? threadIdx.x : threadIdx.x & 63;
    for (int64_t row = (int64_t)blockIdx.x * kRows + (kWaves == 4 ? 0 : threadIdx.x >> 6); row < rows;
         row += (int64_t)gridDim.x * kRows) {
        const uint16_t* src = x + row * ld;
        uint4 held[kHeld];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int64_t k = 8 * (lane + (int64_t)kLanes * i);
            held[i] = k < cols ? *reinterpret_cast<const uint4*>(src + k) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) top = max_of(top, held[i]);
        for (int64_t k = 8 * (lane + (int64_t)kLanes * kHeld); k < cols; k += 8 * kLanes)
            top = max_of(top, *reinterpret_cast<const uint4*>(src + k));
        top = wave_max_u32(top);
        if constexpr (kWaves == 4) {
            if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
            __syncthreads();
            top = max(max(part[0], part[1]), max(part[2], part[3]));
            __syncthreads();  // part is written again for the next row
        }
        const float amax = __uint_as_float(top << 16);
        if (lane == 0) scales[row] = amax / 127.0f;  // infinity or NaN if amax is
        // a power of two on both sides of the quotient keeps 127 / amax finite
        const float lift = amax < 0x1p-100f ? 0x1p64f : 1.0f;
        const float scale = amax > 0.0f ? 127.0f / (amax * lift) : 0.0f;
        int8_t* dst = codes + row * ld_codes;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int64_t k = 8 * (lane + (int64_t)kLanes * i);
            if (k < cols) *reinterpret_cast<uint2*>(dst + k) = codes_of(held[i], lift, scale);
        }
        for (int64_t k = 8 * (lane + (int64_t)kLanes * kHeld); k < cols; k += 8 * kLanes)
            *reinterpret_cast<uint2*>(dst + k) = codes_of(*reinterpret_cast<const uint4*>(src + k), lift, scale);
    }
}

void launch_i8_quant(const uint16_t* x, int64_t rows, int64_t cols, int64_t ld, int8_t* codes, int64_t ld_codes,
                     float* scales, hipStream_t s)
{
    if (rows == 0) return;
    // A wave a row / a workgroup a row (us): 16384 x 512 8.0 / 19.2, 1024 x 1024
    // 2.83 / 3.47, 1 x 512 2.2 / 2.4; 8192 x 2048 10.3 / 12.7 but 256 x 2048
    // 3.1 / 2.8 (600 rows: equal); beyond the 2048 columns that a wave holds
    // 4096 x 3584 11.4 / 9.5, 8192 x 5120 27.9 / 22.2 (5.7 TB/s), 1 x 5120 4.7 / 2.6.
    const int64_t most = int64_t(1) << 22;  // workgroups; each takes more rows beyond that
    if (cols <= 256 * kHeld || (cols <= 512 * kHeld && rows > 512))
        hipLaunchKernelGGL(k_i8_quant<1>, dim3((uint32_t)(rows < 4 * most ? (rows + 3) / 4 : most)), dim3(256), 0, s, x,
                           rows, cols, ld, codes, ld_codes, scales);
    else
        hipLaunchKernelGGL(k_i8_quant<4>, dim3((uint32_t)(rows < most ? rows : most)), dim3(256), 0, s, x, rows, cols, ld,
                           codes, ld_codes, scales);
}

}  // namespace nvfp4
