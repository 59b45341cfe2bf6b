// wave.hpp -- sums and maxima over the lanes of a wave by DPP lane moves, which
// stay inside the vector unit, and the 8-element pieces that the row kernels
// move.  Every sum has one fixed order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "nvfp4_device.hpp"

namespace nvfp4 {

typedef __bf16 wave_bf16x2_t __attribute__((ext_vector_type(2)));
typedef float wave_f32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((wave_f32x2_t{a, b}), wave_bf16x2_t));
}

// The index of this wave in its workgroup, in a scalar register.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }

// v of the lane that a DPP control names (rows of 16 lanes), `none` where there is none.
template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ int lane_move(int none, int v)
{
    return __builtin_amdgcn_update_dpp(none, v, kCtrl, kRows, 0xF, false);
}

template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ float lane_move(float none, float v)
{
    return __int_as_float(lane_move<kCtrl, kRows>(__float_as_int(none), __float_as_int(v)));
}

// v of a lane that there always is (rotations and mirrors); the move becomes
// part of the instruction that takes its result.
template <int kCtrl>
__device__ __forceinline__ int lane_turn(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, kCtrl, 0xF, 0xF, true);
}

// op over all 64 lanes, the same value in each (a scalar register): within rows
// of 16 by 1, 2, 4, 8 lanes, then the last lane of a row into the next.
template <class Op>
__device__ __forceinline__ float wave_all(float v, float none, const Op& op)
{
    v = op(v, lane_move<0x111>(none, v));
    v = op(v, lane_move<0x112>(none, v));
    v = op(v, lane_move<0x114>(none, v));
    v = op(v, lane_move<0x118>(none, v));
    v = op(v, lane_move<0x142, 0xA>(none, v));
    v = op(v, lane_move<0x143, 0xC>(none, v));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ float wave_sum(float v)
{
    return wave_all(v, 0.0f, [](float a, float b) { return a + b; });
}

// The largest of non-negative values; NaN counts as the largest.
__device__ __forceinline__ float wave_top(float v)
{
    return wave_all(v, 0.0f, [](float a, float b) {
        return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
    });
}

// The register pair that exchanging v's rows of 16 lanes (kLanes 16) or its halves
// (32) with itself gives: v of this lane and v of the one kLanes away.
template <int kLanes>
__device__ __forceinline__ uint2 both_of(uint32_t v)
{
    typedef uint32_t Pair __attribute__((ext_vector_type(2)));
    Pair p;
    if constexpr (kLanes == 16) p = __builtin_bit_cast(Pair, __builtin_amdgcn_permlane16_swap(v, v, false, false));
    else p = __builtin_bit_cast(Pair, __builtin_amdgcn_permlane32_swap(v, v, false, false));
    return make_uint2(p.x, p.y);
}

template <int kLanes>
__device__ __forceinline__ float sum_of_halves(float v)
{
    const uint2 p = both_of<kLanes>(__float_as_uint(v));
    return __uint_as_float(p.x) + __uint_as_float(p.y);
}

// Sums (and the largest of non-negative values, NaN the largest) over groups of
// kLanes neighbours (16, 32 or 64), the same in each lane of a group.
template <int kLanes>
__device__ __forceinline__ float group_sum(float v)
{
    if constexpr (kLanes == 64) return wave_sum(v);
    v += __int_as_float(lane_turn<0x128>(__float_as_int(v)));
    v += __int_as_float(lane_turn<0x124>(__float_as_int(v)));
    v += __int_as_float(lane_turn<0x122>(__float_as_int(v)));
    v += __int_as_float(lane_turn<0x121>(__float_as_int(v)));
    return kLanes == 32 ? sum_of_halves<16>(v) : v;
}

template <int kLanes>
__device__ __forceinline__ float group_top(float v)
{
    if constexpr (kLanes == 64) return wave_top(v);
    uint32_t t = __float_as_uint(v);
    t = max(t, (uint32_t)lane_turn<0x128>((int)t));
    t = max(t, (uint32_t)lane_turn<0x124>((int)t));
    t = max(t, (uint32_t)lane_turn<0x122>((int)t));
    t = max(t, (uint32_t)lane_turn<0x121>((int)t));
    if constexpr (kLanes == 32) {
        const uint2 p = both_of<16>(t);
        t = max(p.x, p.y);
    }
    return __uint_as_float(t);
}

// 8 neighbouring elements as fp32.
struct Piece {
    float v[8];
};

// The same as they lie in memory: bf16 in `a`, fp32 in both.
struct RawPiece {
    uint4 a, b;
};

__device__ __forceinline__ RawPiece load_raw(const void* p, int64_t at, bool f32)
{
    RawPiece r;
    if (f32) {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
        r.a = s[0];
        r.b = s[1];
    } else {
        r.a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
        r.b = make_uint4(0, 0, 0, 0);
    }
    return r;
}

__device__ __forceinline__ Piece widen(const RawPiece& r, bool f32)
{
    const uint32_t a[4] = {r.a.x, r.a.y, r.a.z, r.a.w}, b[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
    Piece o;
    if (f32) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o.v[j] = __uint_as_float(a[j]);
            o.v[4 + j] = __uint_as_float(b[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            o.v[2 * j] = bf16_lo(a[j]);
            o.v[2 * j + 1] = bf16_hi(a[j]);
        }
    }
    return o;
}

__device__ __forceinline__ Piece load_piece(const void* p, int64_t at, bool f32) { return widen(load_raw(p, at, f32), f32); }

// Rounded to nearest even where the output is bf16.
__device__ __forceinline__ void store_piece(void* p, int64_t at, const Piece& o, bool f32)
{
    if (f32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
        d[0] = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
        d[1] = make_float4(o.v[4], o.v[5], o.v[6], o.v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
            make_uint4(pack_bf16(o.v[0], o.v[1]), pack_bf16(o.v[2], o.v[3]), pack_bf16(o.v[4], o.v[5]),
                       pack_bf16(o.v[6], o.v[7]));
    }
}

// e^x for x <= 0 (also minus infinity: 0), to about 2^-23 of its value: the
// product with log2 e is taken in two parts, so that its rounding does not
// grow with x.
__device__ __forceinline__ float exp_neg(float x)
{
    x = __builtin_fmaxf(x, -150.0f);
    const float t = x * 1.44269504f;
    float r = __builtin_fmaf(x, 1.44269504f, -t);
    r = __builtin_fmaf(x, 1.92596299e-8f, r);  // log2 e - 1.44269504 as fp32 holds it
    const float p = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(p, r * 0.693147181f, p);
}

}  // namespace nvfp4
