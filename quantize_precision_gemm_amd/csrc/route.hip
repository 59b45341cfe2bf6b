// route.hip -- routing tokens to experts: scores, the choice of k experts a
// token, their weights, and the order of the rows by expert.
//
//   s = softmax(l) or 1 / (1 + e^-l) of a token's E logits; c = s + bias.
//   With fewer groups kept than there are, a group of E / G neighbours counts
//   the sum of its two largest c, and only the best groups' experts stay.
//   Chosen are the k largest c (without a bias: the k largest l, which is the
//   same order), equal ones from the lowest index on, and
//   w = scale s, or scale s / (sum of the chosen s).
//   Place of slot (t, j): the slots sorted by expert, then token.
//
// A choice is a comparison, and two implementations that round differently
// choose differently when two values lie close.  Here every choice is the one
// that 64-bit arithmetic makes: what is compared is held as whole numbers of a
// bounded error, and a token for which two values that a decision compares lie
// within that bound is done again in 64 bits by the whole wave, unless they are made of equal
// logits and biases, as all others within the bound of theirs are.  Ordinary
// logits have a few such tokens in a thousand; if all are such, 16384 x 256 take 33
// us (softmax; sigmoid with a bias 43, with groups 60) instead of 15 to 16.  The bound
// grows with the largest finite bias, of whatever sign: one of -100 16 us (groups 22), -1e4 38
// (51), -1e9 all of them; one of minus infinity costs nothing.
//
// The whole numbers carry the expert's index in their low bits, so no two of a
// token are equal and the k largest come out in order, ties by the lowest
// index, with neither a search nor a removal: the next one is the largest of
// key - last, as unsigned numbers (those from `last` on wrap to small values).
// That is 1.5 instructions a logit and round; finding and removing the largest
// took 5 (16384 x 128, k 8: 13.2 us in all, 17.9).
//
// Weights: renormalised ones are a softmax over the chosen logits (sigmoid:
// with factors of 1 / (1 + e^-|l|)), scaled by the largest, so that no sum of
// them vanishes.
//
// Bound by instructions, not bytes: 16384 x 128 softmax 6.4 us for the choice (8.4
// MB of logits are 1.6) and 5.2 for the places, each 2.5 us of starting and
// ending; 16384 x 256 with groups and a bias 13 and 5.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "internal.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

constexpr int kChunk = kRouteChunk;
constexpr int kThreads = 1024;
constexpr int kMostExperts = kRouteMostExperts, kMostGroups = kRouteMostGroups;

// op over groups of L lanes (16: a DPP row, or the wave), the same in each.
template <int L, class Op>
__device__ __forceinline__ int over_lanes(int v, const Op& op)
{
    v = op(v, lane_turn<0x128>(v));  // rotations within the row by 8, 4, 2, 1
    v = op(v, lane_turn<0x124>(v));
    v = op(v, lane_turn<0x122>(v));
    v = op(v, lane_turn<0x121>(v));
    if constexpr (L == 64) {
        const int a = op(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16));
        return op(a, op(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
    }
    return v;
}

template <int L, class Op>
__device__ __forceinline__ float over_lanes(float v, const Op& op)
{
    return __int_as_float(over_lanes<L>(__float_as_int(v), [&](int a, int b) {
        return __float_as_int(op(__int_as_float(a), __int_as_float(b)));
    }));
}

// v of the lane that a DPP control names.
template <int kCtrl>
__device__ __forceinline__ double lane_move64(double v)
{
    const int64_t b = __double_as_longlong(v);
    const uint32_t lo = lane_turn<kCtrl>((int)b), hi = lane_turn<kCtrl>((int)(b >> 32));
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

__device__ __forceinline__ double lane_value(double v, int lane)
{
    const int64_t b = __double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)b, lane), hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}

template <class Op>
__device__ __forceinline__ double over_wave(double v, const Op& op)
{
    v = op(v, lane_move64<0x128>(v));
    v = op(v, lane_move64<0x124>(v));
    v = op(v, lane_move64<0x122>(v));
    v = op(v, lane_move64<0x121>(v));
    return op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
}

struct Add {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
// The instructions themselves (the compiler adds one to each, for signalling NaNs; there are none here).
__device__ __forceinline__ float max_of(float a, float b)
{
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float max_of(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float min_of(float a, float b)
{
    float r;
    asm("v_min_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ __forceinline__ float middle_of(float a, float b, float c)
{
    float r;
    asm("v_med3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

struct Max {
    __device__ __forceinline__ float operator()(float a, float b) const { return max_of(a, b); }
    __device__ __forceinline__ double operator()(double a, double b) const { return a > b ? a : b; }
};
struct Min {
    __device__ __forceinline__ float operator()(float a, float b) const { return min_of(a, b); }
};
struct MaxUnsigned {
    __device__ __forceinline__ int operator()(int a, int b) const { return (int)max((uint32_t)a, (uint32_t)b); }
};

// The bits of a ballot that belong to this lane's group of L lanes.
template <int L>
__device__ __forceinline__ uint64_t own_bits(uint64_t ballot)
{
    if constexpr (L == 64) return ballot;
    return ballot >> (threadIdx.x & 48) & 0xFFFF;
}

// v of one lane, in scalar registers.
__device__ __forceinline__ int64_t uniform_of(int64_t v, int lane)
{
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)v, lane) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32);
}

__device__ __forceinline__ float logit_at(const RouteArgs& a, int64_t at)
{
    if (a.f32) return static_cast<const float*>(a.logits)[at];
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[at] << 16);
}

// P values e0 .. e0 + P - 1 of the E of a row, `beyond` from E on.  One branch
// for the type and one for the alignment; what is beyond E is read from the
// row's end, so that no load has a branch of its own.
template <int P>
__device__ __forceinline__ void load_values(const void* p, bool f32, bool vec, int64_t row, int e0, int E, float beyond,
                                            float (&l)[P])
{
    if (f32) {
        const float* src = static_cast<const float*>(p) + row;
        if (P >= 4 && vec && e0 + P <= E) {
#pragma unroll
            for (int i = 0; i + 4 <= P; i += 4) {
                const float4 v = *reinterpret_cast<const float4*>(src + e0 + i);
                l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
            }
            asm volatile("");  // (without it both branches may become the other one's single loads)
            return;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) l[i] = src[min(e0 + i, E - 1)];
    } else {
        const uint16_t* src = static_cast<const uint16_t*>(p) + row;
        if (P >= 8 && vec && e0 + P <= E) {
#pragma unroll
            for (int i = 0; i + 8 <= P; i += 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(src + e0 + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) l[i + 2 * j] = bf16_lo(w[j]), l[i + 2 * j + 1] = bf16_hi(w[j]);
            }
            return;
        }
        if (P == 4 && vec && e0 + P <= E) {
#pragma unroll
            for (int i = 0; i + 4 <= P; i += 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(src + e0 + i);
                l[i] = bf16_lo(v.x), l[i + 1] = bf16_hi(v.x), l[i + 2] = bf16_lo(v.y), l[i + 3] = bf16_hi(v.y);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) l[i] = __uint_as_float((uint32_t)src[min(e0 + i, E - 1)] << 16);
    }
#pragma unroll
    for (int i = 0; i < P; ++i) l[i] = e0 + i < E ? l[i] : beyond;
}

template <int P>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int e0, float (&l)[P])
{
    load_values<P>(a.logits, a.f32, a.vec, row, e0, a.E, -INFINITY, l);
}

// Minus infinity for what is no number to choose by; whether there was one
// that is not minus infinity itself.
template <int P>
__device__ __forceinline__ bool drop_not_finite(float (&l)[P])
{
    bool bad = false;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const bool off = !(l[i] < INFINITY);
        bad |= off;
        l[i] = off ? -INFINITY : l[i];
    }
    return bad;
}

// The largest logit of a row, 0 where it has none.
template <int L, int P>
__device__ __forceinline__ float top_of(const float (&l)[P])
{
    float m = l[0];
#pragma unroll
    for (int i = 1; i + 1 < P; i += 2) m = max_of(m, l[i], l[i + 1]);
    if (P % 2 == 0) m = max_of(m, l[P - 1]);
    m = over_lanes<L>(m, Max());
    return m > -INFINITY ? m : 0.0f;
}

// Softmax's sum.
template <int L, int P>
__device__ __forceinline__ float sum_of(const float (&l)[P], float top)
{
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) s += exp_neg(l[i] - top);
    return over_lanes<L>(s, Add());
}

// Sum of the two largest values of a group, as far as there are two; in fp32 half of it, which does not overflow.
__device__ __forceinline__ float pair_sum(float one, float two)
{
    one *= 0.5f;
    return two > -INFINITY ? __builtin_fmaf(two, 0.5f, one) : one;
}
__device__ __forceinline__ double pair_sum(double one, double two) { return two > -INFINITY ? one + two : one; }

// v among the two largest so far (one >= two): the new second is the middle of the three.
__device__ __forceinline__ void take(float v, float& one, float& two)
{
    two = middle_of(v, one, two);
    one = max_of(v, one);
}

__device__ __forceinline__ void take(double v, double& one, double& two)
{
    two = v > one ? one : v > two ? v : two;
    one = v > one ? v : one;
}

// The two largest over the lanes that share a group (2^n neighbours): pairs of
// lanes, quads, and then whole quads and halves by mirroring.
template <int kCtrl>
__device__ __forceinline__ void take_from(float& one, float& two)
{
    const float a = __int_as_float(lane_turn<kCtrl>(__float_as_int(one))), b = __int_as_float(lane_turn<kCtrl>(__float_as_int(two)));
    take(a, one, two);
    take(b, one, two);
}

// Drops the experts (c = minus infinity) of all but the a.kept best groups of
// each row.  Returns whether fp32 may have taken another group than exact values
// would, each c being off by `error` at most.  buf: this row's LDS, E + G values.
template <int L, int P>
__device__ __forceinline__ bool drop_groups(const RouteArgs& a, float (&c)[P], float error, float* buf)
{
    const int sub = threadIdx.x & (L - 1), e0 = sub * P, G = a.groups, per = a.per_group;
    float* value = buf + a.E;
    const int lanes = per / P;  // of a group
    int g = e0 / per;
    const bool whole = L == 16 && lanes * P == per && (lanes & (lanes - 1)) == 0 && lanes <= 16;  // uniform
    if (whole) {
        float one = -INFINITY, two = -INFINITY;
#pragma unroll
        for (int i = 0; i < P; ++i) take(c[i], one, two);
        if (lanes > 1) take_from<0xB1>(one, two);   // the lane's neighbour in its pair
        if (lanes > 2) take_from<0x4E>(one, two);   // in its quad
        if (lanes > 4) take_from<0x141>(one, two);  // the other quad of 8
        if (lanes > 8) take_from<0x140>(one, two);  // the other half of 16
        if (sub % lanes == 0 && g < G) value[g] = pair_sum(one, two);
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (e0 + i < a.E) buf[e0 + i] = c[i];
        __builtin_amdgcn_wave_barrier();
        for (int h = sub; h < G; h += L) {
            float one = -INFINITY, two = -INFINITY;
            int at = sub % per;  // lanes begin at different banks
            for (int i = 0; i < per; ++i) {
                take(buf[h * per + at], one, two);
                at = at + 1 == per ? 0 : at + 1;
            }
            value[h] = pair_sum(one, two);
        }
    }
    __builtin_amdgcn_wave_barrier();
    uint64_t kept = 0;
    float least = INFINITY, most = -INFINITY;  // of the groups kept, and of the others
    for (int q = 0; q < G; q += L) {
        const int h = q + sub;
        const float v = h < G ? value[h] : -INFINITY;
        int before = 0;
#pragma unroll 8
        for (int i = 0; i < G; ++i) {
            const float u = value[i];
            before += u > v || (u == v && i < h);
        }
        const bool keep = h < G && before < a.kept && v > -INFINITY;
        if (keep) least = v < least ? v : least;
        else if (h < G) most = v > most ? v : most;
        kept |= own_bits<L>(__ballot(keep)) << q;
    }
    least = over_lanes<L>(least, Min());
    most = over_lanes<L>(most, Max());
    if (whole) {
        const bool keep = kept >> (g & 63) & 1;
#pragma unroll
        for (int i = 0; i < P; ++i) c[i] = keep ? c[i] : -INFINITY;
    } else {
        int in = e0 - g * per;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (!(kept >> (g & 63) & 1)) c[i] = -INFINITY;
            if (++in == per) in = 0, ++g;
        }
    }
    __builtin_amdgcn_wave_barrier();  // buf is written again for the next row
    // (half a sum is off by as much as a c, and rounds by no more; infinity where nothing is dropped)
    return least - most <= 4 * error;
}

// A float as a whole number, truncated, what is below 0 (and NaN) as 0: the instruction's rule.
__device__ __forceinline__ uint32_t whole_of(float v)
{
    uint32_t r;
    asm("v_cvt_u32_f32 %0, %1" : "=v"(r) : "v"(v));
    return r;
}

// The largest key of a row below `last` (0: the largest of all).
template <int L, int P>
__device__ __forceinline__ uint32_t key_below(const uint32_t (&key)[P], uint32_t last)
{
    uint32_t top = key[0] - last;
#pragma unroll
    for (int i = 1; i < P; ++i) top = max(top, key[i] - last);
    return (uint32_t)over_lanes<L>((int)top, MaxUnsigned()) + last;
}

// The k + 1 largest of a row's keys, (value << kBits) + (2^kBits - 1 - index),
// a value of 0: never.  Lane j of the row gets the j-th one's index (-1: there
// is none left), `last` the last one's key.  Returns (in every lane of the
// row) whether values no further apart than `near` decided, other than those of equal
// logits (the row's, in LDS) and biases: among the candidates each with the next one, since
// values that lie between two near ones are near to both; and where the k-th and the
// next one are equal, the k-th with all that are left.
template <int L, int P>
__device__ __forceinline__ bool pick(const RouteArgs& a, const float* logits, const uint32_t (&key)[P], uint32_t near,
                                     int& mine, uint32_t& last)
{
    constexpr int kBits = __builtin_ctz(L * P);
    constexpr uint32_t kMask = (1u << kBits) - 1;
    const int sub = threadIdx.x & (L - 1);
    uint32_t own = 0;
    last = 0;
    for (int r = 0; r <= a.k; ++r) {
        last = key_below<L, P>(key, last);
        own = sub == r ? last : own;
    }
    // each with the next one (lane j + 1's; a 17th has no lane)
    uint32_t next = (uint32_t)lane_move<0x101>((int)last, (int)own);
    if (sub == a.k - 1) next = last;
    const int e = (int)(kMask - (own & kMask)), after = (int)(kMask - (next & kMask));
    bool close = false;
    if (sub < a.k && next > kMask && (own >> kBits) - (next >> kBits) <= near)  // equal logits and biases make equal values
        close = logits[e] != logits[after] || (a.bias && a.bias[e] != a.bias[after]);
    mine = own > kMask ? e : -1;
    const bool border = sub == a.k - 1 && !close && next > kMask && (own >> kBits) - (next >> kBits) <= near;
    if (__ballot(border)) {  // (rare but for rows of few values)
        const uint32_t edge = (uint32_t)__shfl((int)own, a.k - 1, L);
        const int at = (int)(kMask - (edge & kMask)), e0 = sub * P;
        uint32_t left = 0;
#pragma unroll
        for (int i = 0; i < P; ++i)
            left |= key[i] < last && key[i] > kMask && (edge >> kBits) - (key[i] >> kBits) <= near ? 1u << i : 0u;
        for (; left && !close; left &= left - 1) {
            const int i = e0 + __builtin_ctz(left);
            close |= logits[i] != logits[at] || (a.bias && a.bias[i] != a.bias[at]);
        }
    }
    return own_bits<L>(__ballot(close)) != 0;
}

__device__ __forceinline__ double sigmoid64(float l)
{
    const double e = exp(-__builtin_fabs((double)l));
    return (l < 0 ? e : 1.0) / (1.0 + e);
}

// The k + 1 candidates of each row (lane j: the j-th, -1: none) in the order of
// their sigmoid scores and biases in 64 bits, one exponential a lane, by their ranks.
__device__ __forceinline__ int sort_exactly(const RouteArgs& a, const float* logits, int mine)
{
    const int sub = threadIdx.x & 15;
    const bool there = sub <= a.k && mine >= 0;
    const double c = there ? sigmoid64(logits[mine]) + (double)a.bias[mine] : -INFINITY;
    int rank = 0;
    for (int i = 0; i <= a.k; ++i) {
        const double other = __shfl(c, i, 16);
        const int e = __shfl(mine, i, 16);
        rank += other > c || (other == c && (e < mine || (e == mine && i < sub)));
    }
    if (sub > a.k) rank = sub;
    return __builtin_amdgcn_ds_permute(((threadIdx.x & 48) + rank) << 2, mine);
}

// Bound on the error of c as fp32 computes it.  Softmax, relative to the
// largest score: e^x 2e-7, x's own rounding 6e-8 |x| e^-|x| <= 2.2e-8, the sum
// 22 additions of 6e-8, the reciprocal and the product 1.2e-7.  Sigmoid, as
// 1 / (1 + 2^(-l log2 e)): a quarter of the power's 1.2e-7, the rounding of its
// argument 6e-8 |l| s (1 - s) <= 1.4e-8 twice, 6e-8 for the sum and 1.2e-7 for the
// reciprocal.  The sum with the bias rounds by 6e-8 of itself.
__device__ __forceinline__ float choice_error(const RouteArgs& a, float largest, float most_bias)
{
    return (a.sigmoid ? 2.5e-7f : 2e-6f * largest) + 6.2e-8f * (1.0f + most_bias);
}

// The experts of a row in 64 bits, by the whole wave: lane j gets the j-th.
// kMode as for k_route.
template <int P, int kMode>
__device__ __forceinline__ int choose_exactly(const RouteArgs& a, int64_t row, double* buf)
{
    float l[P];
    double c[P];
    const int lane = threadIdx.x & 63, e0 = lane * P;
    load_logits<P>(a, row, e0, l);
    drop_not_finite(l);
    if constexpr (kMode == 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) c[i] = l[i];
    } else {
        const double top = top_of<64, P>(l);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            c[i] = exp(a.sigmoid ? -__builtin_fabs((double)l[i]) : (double)l[i] - top);
            sum += c[i];
        }
        if (!a.sigmoid) sum = over_wave(sum, Add());
#pragma unroll
        for (int i = 0; i < P; ++i) {
            double v = a.sigmoid ? (l[i] < 0 ? c[i] : 1.0) / (1.0 + c[i]) : c[i] / sum;
            if (a.bias && e0 + i < a.E) v += (double)a.bias[e0 + i];
            c[i] = l[i] > -INFINITY && v - v == 0 ? v : -INFINITY;
        }
    }
    if constexpr (kMode == 2) {
        const int G = a.groups, per = a.per_group;
        double* value = buf + a.E;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (e0 + i < a.E) buf[e0 + i] = c[i];
        __builtin_amdgcn_wave_barrier();
        if (lane < G) {
            double one = -INFINITY, two = -INFINITY;
#pragma unroll 8
            for (int i = 0; i < per; ++i) take(buf[lane * per + i], one, two);
            value[lane] = pair_sum(one, two);
        }
        __builtin_amdgcn_wave_barrier();
        bool keep = false;
        if (lane < G) {
            const double v = value[lane];
            int before = 0;
#pragma unroll 8
            for (int i = 0; i < G; ++i) before += value[i] > v || (value[i] == v && i < lane);
            keep = before < a.kept && v > -INFINITY;
        }
        const uint64_t kept = __ballot(keep);
        int g = e0 / per, in = e0 - g * per;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            // without a bias the order within the groups is the logits'
            c[i] = !(kept >> (g & 63) & 1) || !(c[i] > -INFINITY) ? -INFINITY : a.bias ? c[i] : (double)l[i];
            if (++in == per) in = 0, ++g;
        }
        __builtin_amdgcn_wave_barrier();
    }
    int mine = -1;
    for (int r = 0; r < a.k; ++r) {
        double top = c[0];
#pragma unroll
        for (int i = 1; i < P; ++i) top = c[i] > top ? c[i] : top;
        const double best = over_wave(top, Max());
        if (!(best > -INFINITY)) break;
        const int winner = __builtin_ctzll(__ballot(top == best));  // (lanes hold their experts in order)
        int e = 0;
#pragma unroll
        for (int i = P - 1; i >= 0; --i) e = c[i] == best ? e0 + i : e;
        e = __builtin_amdgcn_readlane(e, winner);
#pragma unroll
        for (int i = 0; i < P; ++i) c[i] = e == e0 + i ? -INFINITY : c[i];
        if (lane == r) mine = e;
    }
    return mine;
}

// The weight of the expert that lane j of a row chose, of logit l (minus infinity
// and a weight of 0 where it has none).
template <int L>
__device__ __forceinline__ float weight_of(const RouteArgs& a, float l, int mine, float top, float inverse)
{
    const float neg = l < 0.0f ? l : 0.0f;  // 1 / (1 + e^-l) = e^neg / (1 + e^-|l|)
    float q = 1.0f;
    if (a.sigmoid) q = 1.0f / (1.0f + exp_neg(-__builtin_fabsf(l)));
    if (!a.renorm) return a.scale * (a.sigmoid ? q * exp_neg(neg) : exp_neg(l - top) * inverse);
    const float x = a.sigmoid ? neg : l;
    float m = over_lanes<L>(mine >= 0 ? x : -INFINITY, Max());
    m = m > -INFINITY ? m : 0.0f;
    q = mine >= 0 ? q * exp_neg(x - m) : 0.0f;
    const float all = over_lanes<L>(q, Add());
    return all > 0.0f ? a.scale * (q / all) : 0.0f;
}

// Inclusive sums over the workgroup's threads; all: the sum of them all.
__device__ __forceinline__ int group_scan(int v, int* waves, int& all)
{
    const int wave = wave_index();
    v += lane_move<0x111>(0, v);
    v += lane_move<0x112>(0, v);
    v += lane_move<0x114>(0, v);
    v += lane_move<0x118>(0, v);
    v += lane_move<0x142, 0xA>(0, v);
    v += lane_move<0x143, 0xC>(0, v);
    if ((threadIdx.x & 63) == 63) waves[wave] = v;
    __syncthreads();
    int before = 0;
    all = 0;
    for (int w = 0; w < (int)blockDim.x / 64; ++w) {
        before += w < wave ? waves[w] : 0;
        all += waves[w];
    }
    return v + before;
}

}  // namespace

// Chunks of 64 tokens, one a workgroup: L lanes hold a token's logits, P each.
// kMode 0: the logits themselves are compared; 1: scores with a bias; 2: groups are dropped.
// An expert's tokens of the chunk are a 64-bit mask in LDS, so that a slot's
// place among them is a count of bits, in token order, with no atomic whose
// order could show.  One chunk: the places are written here; otherwise its
// counts, one byte each, and k_route_place writes them.
// 16 lanes a token up to 256 experts: four tokens share a lane move or a scalar step
// (4096 x 256: 11.7 us, a wave a token 18.5; 65536 x 256: 46 and 71).
template <int L, int P, int kMode>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a)
{
    constexpr int kRows = kThreads / L, kWaves = kThreads / 64;
    constexpr int kExact = L == 64 ? P : P > 4 ? P / 4 : 1;         // experts a lane, for a row held by the wave
    constexpr int kBuf = (L == 64 ? 8 : 16) * (L * P + kMostGroups);  // bytes of a wave: rows in fp32, or one in 64 bits
    constexpr int kBits = __builtin_ctz(L * P);
    // values of keys go from kLeast to kMost + kLeast, with room for roundings of 2^-24 kMost (16 at most) on both sides
    constexpr float kMost = (float)((1u << (32 - kBits)) - (1u << 9)), kLeast = 64.0f;
    __shared__ unsigned long long mask[L * P];
    __shared__ int waves[kWaves], start[L * P];
    __shared__ int16_t picked[kChunk * kRouteMostK];
    __shared__ __attribute__((aligned(16))) uint8_t bufs[kWaves * kBuf];
    const int tid = threadIdx.x, sub = tid & (L - 1), e0 = sub * P;
    const int64_t first = (int64_t)blockIdx.x * kChunk;
    const int tokens = (int)min((int64_t)kChunk, a.T - first);
    uint8_t* buf = bufs + wave_index() * kBuf;
    for (int e = tid; e < L * P; e += kThreads) mask[e] = 0;
    __syncthreads();
#pragma unroll 1
    for (int t0 = 0; t0 < (kRows == kChunk ? 1 : tokens); t0 += kRows) {
        const int in = t0 + tid / L;
        const bool live = in < tokens;
        if (!__ballot(live)) break;  // (a wave without tokens)
        const int64_t t = first + (live ? in : tokens - 1), row = t * a.ld;
        float l[P];
        load_logits<P>(a, row, e0, l);
        float bias[P], most_bias = 0.0f;
        if constexpr (kMode != 0) {
#pragma unroll
            for (int i = 0; i < P; ++i) bias[i] = 0.0f;
            if (a.bias) {
                load_values<P>(a.bias, true, a.vec_bias, 0, e0, a.E, 0.0f, bias);  // (not finite: never chosen)
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float size = __builtin_fabsf(bias[i]);
                    const bool fine = size < INFINITY;
                    most_bias = fine && size > most_bias ? size : most_bias;
                    bias[i] = fine ? bias[i] : -INFINITY;
                }
                most_bias = over_lanes<L>(most_bias, Max());
            }
        }
        const bool bad = own_bits<L>(__ballot(drop_not_finite(l))) != 0;
        const bool by_bias = kMode != 0 && a.bias;
        const bool softmax = !a.sigmoid && (kMode != 0 || !a.renorm || a.scores);
        float top = 0.0f, inverse = 1.0f;
        if (softmax || !by_bias) top = top_of<L, P>(l);
        if (softmax) {
            const float sum = sum_of<L, P>(l, top);
            inverse = sum > 0.0f ? 1.0f / sum : 0.0f;  // (a padded token: scores of 0)
        }
        if (a.scores && live) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float e = exp_neg(a.sigmoid ? -__builtin_fabsf(l[i]) : l[i] - top);
                const float s = a.sigmoid ? (l[i] < 0.0f ? e : 1.0f) / (1.0f + e) : e * inverse;
                if (e0 + i < a.E) a.scores[t * a.E + e0 + i] = bad ? NAN : s;
            }
        }
        bool close = false;
        float c[P], error = 0.0f;
        float* own = reinterpret_cast<float*>(buf) + (L == 64 ? 0 : (tid >> 4 & 3) * (L * P + kMostGroups));  // the row's
        if constexpr (kMode != 0) {
            if (a.sigmoid) {
#pragma unroll
                for (int i = 0; i < P; ++i)
                    c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -1.44269504f));
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) c[i] = exp_neg(l[i] - top) * inverse;
            }
#pragma unroll
            for (int i = 0; i < P; ++i) c[i] = l[i] > -INFINITY ? c[i] + bias[i] : -INFINITY;
            error = choice_error(a, inverse, most_bias);
            if constexpr (kMode == 2) close = drop_groups<L, P>(a, c, error, own);
        }
        // Whole numbers of what is compared: c from -most_bias to 1 + most_bias,
        // or logits down to 16 below the largest (rounding keeps their order, as
        // far as they stay apart); minus infinity becomes 0.
        uint32_t key[P], near = 0;
        float unit, offset;
        if (by_bias) {
            unit = kMost / (1.0f + 2.0f * most_bias);
            offset = __builtin_fmaf(most_bias, unit, kLeast);
            // (each of two values is rounded once to 24 bits, and they are truncated)
            near = (uint32_t)(2.0f * error * unit + kMost * 0x1p-23f + 1.0f);
        } else {
            float least = INFINITY;
#pragma unroll
            for (int i = 0; i < P; ++i) least = min_of(l[i] > -INFINITY ? l[i] : INFINITY, least);
            least = over_lanes<L>(least, Min());
            const float range = min_of(max_of(top - least, 1e-30f), 16.0f);
            unit = kMost / range;
            offset = kMost + kLeast;
#pragma unroll
            for (int i = 0; i < P; ++i) {  // (a difference that overflows is far down, not nothing)
                const bool may = (kMode == 0 ? l[i] : c[i]) > -INFINITY;
                c[i] = may ? max_of(l[i] - top, -range) : -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i)
            key[i] = (whole_of(__builtin_fmaf(c[i], unit, offset)) << kBits | ((1u << kBits) - P - e0)) | (P - 1 - i);
        // the row's logits, for the comparisons of equals and the weights
#pragma unroll
        for (int i = 0; i < P; ++i) own[e0 + i] = l[i];
        __builtin_amdgcn_wave_barrier();
        int mine;
        uint32_t last;
        bool swapped = pick<L, P>(a, own, key, near, mine, last);
        if constexpr (L == 16 && kMode != 0) {
            // Values of neighbours in the order alone: the candidates are put in order in 64 bits
            // (unless the last of them and what comes next lie close, too).
            if (a.sigmoid && a.bias && a.k < 16 && __ballot(swapped)) {
                const uint32_t next = key_below<L, P>(key, last);
                const bool more = next >> kBits && (last >> kBits) - (next >> kBits) <= near;
                const int sorted = sort_exactly(a, own, mine);
                mine = swapped ? sorted : mine;
                swapped = swapped && more;
            }
        }
        close |= swapped;
        if (sub >= a.k) mine = -1;
        float chosen = mine >= 0 ? own[mine] : -INFINITY;
        uint64_t again = __ballot(close && live);
        while (again) {
            const int lane = __builtin_ctzll(again);
            const int64_t that = uniform_of(row, lane);
            const int exact = choose_exactly<kExact, kMode>(a, that, reinterpret_cast<double*>(buf));
            const int moved = __shfl(exact, sub, 64);
            if (L == 64 || (tid & 63) / L == lane / L) {
                mine = moved;
                chosen = mine >= 0 ? logit_at(a, row + mine) : -INFINITY;
            }
            again &= L == 64 ? 0 : ~(0xFFFFull << (lane & 48));
        }
        const float w = weight_of<L>(a, chosen, mine, top, inverse);
        if (live && sub < a.k) {
            a.experts[t * a.k + sub] = mine;
            a.weights[t * a.k + sub] = bad ? NAN : w;
            picked[in * a.k + sub] = (int16_t)mine;
            if (mine >= 0) atomicOr(&mask[mine], 1ull << in);
        }
    }
    if (!a.ends) return;
    __syncthreads();
    const int count = tid < a.E ? __popcll(mask[tid]) : 0;
    if (gridDim.x > 1) {
        if (tid < a.pitch) a.counts[(int64_t)blockIdx.x * a.pitch + tid] = (uint8_t)count;
        return;
    }
    int all;
    const int upto = group_scan(count, waves, all);
    if (tid < a.E) {
        a.ends[tid] = upto;
        start[tid] = upto - count;
    }
    __syncthreads();
    if (tid < tokens * a.k) {
        const int e = picked[tid];
        a.rows[tid] = e < 0 ? -1 : start[e] + __popcll(mask[e] & ((1ull << tid / a.k) - 1));
    }
}

// The places of a chunk's slots.  Each workgroup adds up all chunks' counts
// (256 chunks of 256 experts are 64 KB, in the L2), those before its own and
// all of them, 16 experts a lane in pairs of 16 bits (256 chunks of 64 tokens fit); or
// k_route_sums has done so (sums).
__global__ __launch_bounds__(kThreads) void k_route_place(RouteArgs a, int chunks, const int* __restrict__ sums)
{
    constexpr int kWaves = kThreads / 64;
    __shared__ unsigned long long mask[kMostExperts];
    __shared__ int start[kMostExperts], waves[kWaves];
    __shared__ uint32_t part[kWaves][kMostExperts / 16][17];
    const int tid = threadIdx.x, chunk = blockIdx.x;
    const int64_t first = (int64_t)chunk * kChunk;
    const int slots = (int)(min((int64_t)kChunk, a.T - first) * a.k);
    const int slot = tid, e = slot < slots ? a.experts[first * a.k + slot] : -1, t = slot / a.k;
    for (int i = tid; i < a.E; i += kThreads) mask[i] = 0;
    int mine = 0, all = 0;  // this thread's expert: its rows in earlier chunks, and in all
    if (sums) {
        if (tid < a.E) {
            mine = sums[(int64_t)chunk * a.E + tid];
            all = sums[(int64_t)chunks * a.E + tid];
        }
    } else {
        const int lanes = a.pitch / 16, at = tid & (lanes - 1), slices = kThreads / lanes;
        uint32_t n[16] = {};  // words 0 to 7: before; 8 to 15: all; even and odd bytes of the four words
#pragma unroll 4
        for (int c = tid / lanes; c < chunks; c += slices) {
            const uint4 v = *reinterpret_cast<const uint4*>(a.counts + (int64_t)c * a.pitch + 16 * at);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w}, earlier = c < chunk ? 0x00FF00FFu : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                n[8 + 2 * j] += w[j] & 0x00FF00FFu;
                n[9 + 2 * j] += w[j] >> 8 & 0x00FF00FFu;
                n[2 * j] += w[j] & earlier;
                n[2 * j + 1] += w[j] >> 8 & earlier;
            }
        }
        for (int d = lanes; d < 8; d <<= 1)  // (up to 64 experts)
#pragma unroll
            for (int j = 0; j < 16; ++j) n[j] += (uint32_t)__shfl_xor((int)n[j], d, 64);
        if (lanes <= 8)
#pragma unroll
            for (int j = 0; j < 16; ++j) n[j] += (uint32_t)lane_turn<0x128>((int)n[j]);
        if (lanes <= 16)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint2 both = both_of<16>(n[j]);
                n[j] = both.x + both.y;
            }
        if (lanes <= 32)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint2 both = both_of<32>(n[j]);
                n[j] = both.x + both.y;
            }
        if ((tid & 63) < lanes) {
#pragma unroll
            for (int j = 0; j < 16; ++j) part[wave_index()][at][j] = n[j];
        }
        __syncthreads();
        if (tid < a.E) {
            const int word = tid % 16 / 4 * 2 + (tid & 1), shift = tid & 2 ? 16 : 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                mine += part[w][tid / 16][word] >> shift & 0xFFFF;
                all += part[w][tid / 16][8 + word] >> shift & 0xFFFF;
            }
        }
    }
    int sum;
    const int upto = group_scan(all, waves, sum);
    if (tid < a.E) {
        start[tid] = upto - all + mine;
        if (chunk == 0) a.ends[tid] = upto;
    }
    const bool there = e >= 0 && e < a.E;
    if (there) atomicOr(&mask[e], 1ull << t);
    __syncthreads();
    if (slot < slots)
        a.rows[first * a.k + slot] = there ? start[e] + __popcll(mask[e] & ((1ull << t) - 1)) : -1;
}

// Many chunks: the sums of the counts before each chunk, expert by expert, and
// a last row of totals.  A workgroup takes 16 experts, 64 runs of the chunks.
__global__ __launch_bounds__(kThreads) void k_route_sums(const uint8_t* __restrict__ counts, int pitch, int chunks, int E,
                                                         int* __restrict__ sums)
{
    __shared__ int part[64][17];
    const int i = threadIdx.x & 15, s = threadIdx.x >> 4, e = blockIdx.x * 16 + i;
    const int64_t from = (int64_t)chunks * s / 64, to = (int64_t)chunks * (s + 1) / 64;
    int n = 0;
    if (e < E)
        for (int64_t c = from; c < to; ++c) n += counts[c * pitch + e];
    part[s][i] = n;
    __syncthreads();
    int at = 0;
    for (int j = 0; j < s; ++j) at += part[j][i];
    if (e >= E) return;
    for (int64_t c = from; c < to; ++c) {
        sums[c * E + e] = at;
        at += counts[c * pitch + e];
    }
    if (s == 63) sums[(int64_t)chunks * E + e] = at;
}

// Gradients of the logits, L lanes a row, P experts each.  With g = scale dw
// over the chosen and d the gradients of the scores:
//   renormalised, p the chosen scores over their sum:
//     softmax  p (g - sum g p),   sigmoid  p (g - sum g p) (1 - s)
//   otherwise: softmax  s (g - sum g s),   sigmoid  g s (1 - s)
//   and of d: softmax  s (d - sum d s),   sigmoid  d s (1 - s).
// The chosen's part is added in LDS, slot by slot (a repeated expert adds up
// in order).  Only what the form needs is read: renormalised weights need the
// chosen logits alone.  16384 x 256, softmax not renormalised: 11.6 us for 34.6 MB (6.8 at a
// copy's rate), 489 instructions a wave beside them.
template <int L, int P>
__global__ __launch_bounds__(256) void k_route_backward(RouteBackArgs a)
{
    __shared__ __attribute__((aligned(16))) float parts[256 * P];
    const int tid = threadIdx.x, sub = tid & (L - 1), e0 = sub * P;
    float* part = parts + (tid / L) * (L * P);
    const bool softmax = !a.f.sigmoid, whole = a.dscores || (softmax && !a.f.renorm);
    const int64_t step = (int64_t)gridDim.x * (256 / L);
    for (int64_t t0 = (int64_t)blockIdx.x * (256 / L); t0 < a.f.T; t0 += step) {
        const bool live = t0 + tid / L < a.f.T;
        const int64_t t = live ? t0 + tid / L : a.f.T - 1, row = t * a.f.ld;
        const int e = sub < a.f.k ? a.f.experts[t * a.f.k + sub] : -1;
        const bool there = e >= 0 && e < a.f.E;
        const float g = there ? a.f.scale * a.dweights[t * a.f.k + sub] : 0.0f;
        // all scores, where the form needs them: softmax s, sigmoid s (1 - s)
        float s[P], mine = 0.0f;
        bool bad = false;
        if (whole) {
            load_logits<P>(a.f, row, e0, s);
            bad = own_bits<L>(__ballot(drop_not_finite(s))) != 0;
            if (softmax) {
                const float top = top_of<L, P>(s);
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    s[i] = exp_neg(s[i] - top);
                    sum += s[i];
                }
                sum = over_lanes<L>(sum, Add());
                const float inverse = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
                for (int i = 0; i < P; ++i) s[i] *= inverse;
                if (!a.f.renorm) {
                    __builtin_amdgcn_wave_barrier();  // (the last row's reads)
#pragma unroll
                    for (int i = 0; i < P; ++i) part[e0 + i] = s[i];
                    __builtin_amdgcn_wave_barrier();
                    mine = there ? part[e] : 0.0f;
                }
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const float p = exp_neg(-__builtin_fabsf(s[i])), h = 1.0f / (1.0f + p);
                    s[i] = p * h * h;
                }
            }
        }
        // the chosen: d their gradient, or (softmax, not renormalised) what it has beside s times the mean
        float d, dot = 0.0f;
        if (softmax && !a.f.renorm) {
            d = g * mine;
            dot = over_lanes<L>(d, Add());
        } else {
            const float l = there ? logit_at(a.f, row + e) : -INFINITY;
            const float neg = l < 0.0f ? l : 0.0f, half = 1.0f / (1.0f + exp_neg(-__builtin_fabsf(l)));
            const float rest = exp_neg(l > 0.0f ? -l : 0.0f) * half;  // 1 - 1 / (1 + e^-l)
            if (a.f.renorm) {
                const float x = a.f.sigmoid ? neg : l;
                float m = over_lanes<L>(there ? x : -INFINITY, Max());
                m = m > -INFINITY ? m : 0.0f;
                const float q = there ? exp_neg(x - m) * (a.f.sigmoid ? half : 1.0f) : 0.0f;
                const float all = over_lanes<L>(q, Add());
                const float p = all > 0.0f ? q / all : 0.0f;
                const float mean = over_lanes<L>(there ? g * p : 0.0f, Add());
                d = p * (g - mean) * (a.f.sigmoid ? rest : 1.0f);
            } else {
                d = g * (exp_neg(neg) * half) * rest;
            }
        }
        float o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = 0.0f;
        if (whole) {
            float ds[P], along = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) ds[i] = 0.0f;
            if (a.dscores) {
                load_values<P>(a.dscores, true, a.vec_scores, t * a.f.E, e0, a.f.E, 0.0f, ds);
                if (softmax) {
#pragma unroll
                    for (int i = 0; i < P; ++i) along = __builtin_fmaf(ds[i], s[i], along);
                    along = over_lanes<L>(along, Add());
                }
            }
            along += dot;
#pragma unroll
            for (int i = 0; i < P; ++i) o[i] = bad ? NAN : s[i] * (ds[i] - along);
        }
        __builtin_amdgcn_wave_barrier();  // (reads of the last row's, or of the scores)
#pragma unroll
        for (int i = 0; i < P; ++i) part[e0 + i] = o[i];
        __builtin_amdgcn_wave_barrier();
        for (int j = 0; j < a.f.k; ++j) {
            if (sub == j && there) part[e] += d;
            __builtin_amdgcn_wave_barrier();
        }
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = part[e0 + i];
        if (!live) continue;  // (no lane moves follow in this round of the loop)
        const int64_t at = t * a.ld_out + e0;
        const bool wide = P >= 4 && a.vec_out && e0 + P <= a.f.E;
        if (a.out_f32) {
            float* dst = static_cast<float*>(a.out) + at;
            if (wide) {
#pragma unroll
                for (int i = 0; i + 4 <= P; i += 4)
                    *reinterpret_cast<float4*>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if (e0 + i < a.f.E) dst[i] = o[i];
            }
        } else {
            uint16_t* dst = static_cast<uint16_t*>(a.out) + at;
            if (wide) {
#pragma unroll
                for (int i = 0; i + 4 <= P; i += 4)
                    *reinterpret_cast<uint2*>(dst + i) = make_uint2(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]));
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if (e0 + i < a.f.E) dst[i] = (uint16_t)pack_bf16(o[i], 0.0f);
            }
        }
    }
}

namespace {

template <int L, int P>
void launch_route_rows(const RouteArgs& a, uint32_t grid, hipStream_t s)
{
    if (a.kept < a.groups)
        hipLaunchKernelGGL((k_route<L, P, 2>), dim3(grid), dim3(kThreads), 0, s, a);
    else if (a.bias)
        hipLaunchKernelGGL((k_route<L, P, 1>), dim3(grid), dim3(kThreads), 0, s, a);
    else
        hipLaunchKernelGGL((k_route<L, P, 0>), dim3(grid), dim3(kThreads), 0, s, a);
}

template <int L, int P>
void launch_route_back_rows(const RouteBackArgs& a, hipStream_t s)
{
    const int64_t blocks = (a.f.T + 256 / L - 1) / (256 / L), most = int64_t(1) << 22;
    hipLaunchKernelGGL((k_route_backward<L, P>), dim3((uint32_t)(blocks < most ? blocks : most)), dim3(256), 0, s, a);
}

// Beyond 256 chunks one more launch adds up the counts, which each workgroup does
// for itself up to there.  (16384 x 256, 256 chunks: 15.6 us, by the launch 17.7; 32768 x 256: 26.0
// without it, 25.8 by it; 65536 x 64: 30.2 and 27.1; 65536 x 256: 57 and 46.)
bool sums_apart(int64_t chunks) { return chunks > 256; }

// Bytes of a chunk's counts: 16 experts a lane, a power of two of lanes.
int64_t count_pitch(int64_t E)
{
    int64_t pitch = 16;
    while (pitch < E) pitch *= 2;
    return pitch;
}

}  // namespace

int64_t route_workspace(int64_t T, int64_t E)
{
    const int64_t chunks = (T + kChunk - 1) / kChunk;
    if (chunks <= 1) return 0;
    return chunks * count_pitch(E) + (sums_apart(chunks) ? (chunks + 1) * E * (int64_t)sizeof(int) : 0);
}

void launch_route(const RouteArgs& a0, hipStream_t s)
{
    RouteArgs a = a0;
    a.pitch = (int)count_pitch(a.E);
    a.per_group = a.E / a.groups;
    const int64_t chunks = (a.T + kChunk - 1) / kChunk;
    if (chunks == 0 && !a.ends) return;
    const uint32_t grid = (uint32_t)std::max<int64_t>(chunks, 1);  // (no tokens: ends of 0)
    if (a.E <= 16) launch_route_rows<16, 1>(a, grid, s);
    else if (a.E <= 32) launch_route_rows<16, 2>(a, grid, s);
    else if (a.E <= 64) launch_route_rows<16, 4>(a, grid, s);
    else if (a.E <= 128) launch_route_rows<16, 8>(a, grid, s);
    else if (a.E <= 256) launch_route_rows<16, 16>(a, grid, s);
    else if (a.E <= 512) launch_route_rows<64, 8>(a, grid, s);
    else launch_route_rows<64, 16>(a, grid, s);
    if (!a.ends || chunks <= 1) return;
    int* sums = nullptr;
    if (sums_apart(chunks)) {
        sums = reinterpret_cast<int*>(a.counts + chunks * a.pitch);
        hipLaunchKernelGGL(k_route_sums, dim3((uint32_t)((a.E + 15) / 16)), dim3(kThreads), 0, s, a.counts, a.pitch,
                           (int)chunks, a.E, sums);
    }
    hipLaunchKernelGGL(k_route_place, dim3(grid), dim3(kThreads), 0, s, a, (int)chunks, sums);
}

void launch_route_backward(const RouteBackArgs& a, hipStream_t s)
{
    const int E = a.f.E;
    if (a.f.T == 0) return;
    if (E <= 16) launch_route_back_rows<16, 1>(a, s);
    else if (E <= 32) launch_route_back_rows<16, 2>(a, s);
    else if (E <= 64) launch_route_back_rows<16, 4>(a, s);
    else if (E <= 128) launch_route_back_rows<16, 8>(a, s);
    else if (E <= 256) launch_route_back_rows<16, 16>(a, s);
    else if (E <= 512) launch_route_back_rows<64, 8>(a, s);
    else launch_route_back_rows<64, 16>(a, s);
}

}  // namespace nvfp4
