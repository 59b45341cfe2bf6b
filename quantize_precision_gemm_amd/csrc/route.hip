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
// that 64-bit arithmetic makes: c is computed in fp32 with a bound on its
// error, and a token for which two values that a decision compares lie within
// that bound is done again in 64 bits by the whole wave (about one in a
// thousand).  Without bias and groups the logits themselves are compared,
// which is exact.
//
// Weights: renormalised ones are a softmax over the chosen logits (sigmoid:
// with factors of 1 / (1 + e^-|l|)), scaled by the largest, so that no sum of
// them vanishes.
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

// A value that compares as a signed integer; +0 and -0 are one.
__device__ __forceinline__ int key_of(float v)
{
    const int b = __float_as_int(v + 0.0f);
    return b ^ ((b >> 31) & 0x7FFFFFFF);
}

__device__ __forceinline__ int64_t key_of(double v)
{
    const int64_t b = __double_as_longlong(v + 0.0);
    return b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFFll);
}

__device__ __forceinline__ float value_of(int key) { return __int_as_float(key ^ ((key >> 31) & 0x7FFFFFFF)); }
__device__ __forceinline__ double value_of(int64_t key)
{
    return __longlong_as_double(key ^ ((key >> 63) & 0x7FFFFFFFFFFFFFFFll));
}

// What is never chosen: below the key of every finite value.
template <class Key>
constexpr Key kNever = sizeof(Key) == 4 ? (Key)0x80000000 : (Key)0x8000000000000000ull;

// op over groups of L lanes (16: a DPP row, or the wave), the same in each.
template <int L, class Op>
__device__ __forceinline__ float over_lanes(float v, const Op& op)
{
    v = op(v, lane_move<0x128>(v, v));  // rotations within the row by 8, 4, 2, 1
    v = op(v, lane_move<0x124>(v, v));
    v = op(v, lane_move<0x122>(v, v));
    v = op(v, lane_move<0x121>(v, v));
    if constexpr (L == 64) {
        v = op(v, __shfl_xor(v, 16, 64));
        v = op(v, __shfl_xor(v, 32, 64));
    }
    return v;
}

template <int L, class Op>
__device__ __forceinline__ int over_lanes(int v, const Op& op)
{
    return __float_as_int(over_lanes<L>(__int_as_float(v), [&](float a, float b) {
        return __int_as_float(op(__float_as_int(a), __float_as_int(b)));
    }));
}

template <int L, class Op>
__device__ __forceinline__ int64_t over_lanes(int64_t v, const Op& op)
{
#pragma unroll
    for (int d = 1; d < L; d <<= 1) v = op(v, (int64_t)__shfl_xor((long long)v, d, 64));
    return v;
}

template <int L, class Op>
__device__ __forceinline__ double over_lanes(double v, const Op& op)
{
#pragma unroll
    for (int d = 1; d < L; d <<= 1) v = op(v, __shfl_xor(v, d, 64));
    return v;
}

struct Add {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
};
struct Min {
    template <class T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a < b ? a : b; }
};

// The bits of a ballot that belong to this lane's group of L lanes.
template <int L>
__device__ __forceinline__ uint64_t own_bits(uint64_t ballot)
{
    if constexpr (L == 64) return ballot;
    return ballot >> (threadIdx.x & 48) & 0xFFFF;
}

__device__ __forceinline__ float exp_any(float x) { return exp_neg(x); }
__device__ __forceinline__ double exp_any(double x) { return exp(x); }

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

// The logits of experts e0 .. e0 + P - 1 of a row, minus infinity beyond E.
template <int P>
__device__ __forceinline__ void load_logits(const RouteArgs& a, int64_t row, int e0, float (&l)[P])
{
    if constexpr (P >= 4) {
        if (a.vec) {  // rows 16 (fp32) or 8 (bf16) bytes aligned
#pragma unroll
            for (int i = 0; i < P; i += 4) {
                if (e0 + i + 4 <= a.E) {
                    if (a.f32) {
                        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + row + e0 + i);
                        l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + row + e0 + i);
                        l[i] = bf16_lo(v.x), l[i + 1] = bf16_hi(v.x), l[i + 2] = bf16_lo(v.y), l[i + 3] = bf16_hi(v.y);
                    }
                } else {
#pragma unroll
                    for (int j = i; j < i + 4; ++j) l[j] = e0 + j < a.E ? logit_at(a, row + e0 + j) : -INFINITY;
                }
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) l[i] = e0 + i < a.E ? logit_at(a, row + e0 + i) : -INFINITY;
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

// Softmax's largest logit (0 where a row has none) and sum.
template <int L, int P, class Num>
__device__ __forceinline__ void softmax_of(const float (&l)[P], float& top, Num& sum)
{
    float m = l[0];
#pragma unroll
    for (int i = 1; i < P; ++i) m = l[i] > m ? l[i] : m;
    m = over_lanes<L>(m, Max());
    top = m > -INFINITY ? m : 0.0f;
    Num s = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) s += exp_any((Num)l[i] - (Num)top);
    sum = over_lanes<L>(s, Add());
}

// The k experts of a row held by L lanes, P a lane: those with the largest c
// (minus infinity: never), without a bias those with the largest l, equal ones
// from the lowest index on.  Lane j of the row gets the j-th (-1: there is
// none left).  kGuard: true is returned if two values that a decision compares
// may be in another order than their exact ones, each c being off by `error`
// at most.  buf: this row's LDS, E + G values (kGroups).
template <int L, int P, bool kGroups, bool kGuard, class Num>
__device__ __forceinline__ bool choose(const RouteArgs& a, int64_t row, const float (&l)[P], Num (&c)[P], Num error, Num* buf,
                                       int& mine)
{
    typedef typename std::conditional<sizeof(Num) == 4, int, int64_t>::type Key;
    const int sub = threadIdx.x & (L - 1), e0 = sub * P;
    bool close = false;
    if constexpr (kGroups) {
        const int G = a.groups, per = a.E / G;
        Num* value = buf + a.E;
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (e0 + i < a.E) buf[e0 + i] = c[i];
        __builtin_amdgcn_wave_barrier();
        for (int g = sub; g < G; g += L) {
            Num one = -INFINITY, two = -INFINITY;
            int at = sub % per;  // lanes begin at different banks
            for (int i = 0; i < per; ++i) {
                const Num v = buf[g * per + at];
                two = v > one ? one : v > two ? v : two;
                one = v > one ? v : one;
                at = at + 1 == per ? 0 : at + 1;
            }
            value[g] = two > -INFINITY ? one + two : one;
        }
        __builtin_amdgcn_wave_barrier();
        uint64_t kept = 0;
        Num least = INFINITY, most = -INFINITY;  // of the groups kept, and of the others
        for (int q = 0; q < G; q += L) {
            const int g = q + sub;
            bool keep = false;
            if (g < G) {
                const Num v = value[g];
                int before = 0;
                for (int h = 0; h < G; ++h) {
                    const Num u = value[h];
                    before += u > v || (u == v && h < g);
                }
                keep = before < a.kept && v > -INFINITY;
                if (keep) least = v < least ? v : least;
                else most = v > most ? v : most;
            }
            kept |= own_bits<L>(__ballot(keep)) << q;
        }
        if constexpr (kGuard) {  // (infinity where nothing is dropped; the sums round, too)
            least = over_lanes<L>(least, Min());
            most = over_lanes<L>(most, Max());
            close = least - most <= 6 * error;
        }
        int g = e0 / per, in = e0 - g * per;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (!(kept >> (g & 63) & 1)) c[i] = -INFINITY;
            if (++in == per) in = 0, ++g;
        }
        __builtin_amdgcn_wave_barrier();  // buf is written again for the next row
    }
    Key key[P];
#pragma unroll
    for (int i = 0; i < P; ++i) key[i] = c[i] > -INFINITY ? key_of(a.bias ? c[i] : (Num)l[i]) : kNever<Key>;
    mine = -1;
    Key last = kNever<Key>;
    int last_e = -1;
    const bool guard = kGuard && a.bias;
    const int rounds = a.k + (guard ? 1 : 0);  // the guard compares with the first that is left out, too
    for (int r = 0; r < rounds; ++r) {
        Key top = key[0];
#pragma unroll
        for (int i = 1; i < P; ++i) top = key[i] > top ? key[i] : top;
        const Key best = over_lanes<L>(top, Max());
        const uint64_t who = own_bits<L>(__ballot(top == best));
        const bool winner = sub == __builtin_ctzll(who | 1ull << 63);
        int e = -1;
#pragma unroll
        for (int i = P - 1; i >= 0; --i) e = key[i] == best ? e0 + i : e;
        if (!winner || best == kNever<Key>) e = -1;
#pragma unroll
        for (int i = 0; i < P; ++i) key[i] = e == e0 + i ? kNever<Key> : key[i];
        e = over_lanes<L>(e, Max());
        if (guard) {
            if (r > 0 && e >= 0) {
                const Num gap = value_of(last) - value_of(best);
                if (gap <= 2 * error)  // equal logits and biases make equal values: their order is the index's
                    close |= logit_at(a, row + last_e) != logit_at(a, row + e) || a.bias[last_e] != a.bias[e];
            }
            last = best;
            last_e = e;
        }
        if (sub == r && r < a.k) mine = e;
    }
    return close;
}

// Bound on the error of c as fp32 computes it.  Softmax, relative to the
// largest score: e^x 2e-7, x's own rounding 6e-8 |x| e^-|x| <= 2.2e-8, the sum
// 22 additions of 6e-8, the reciprocal and the product 1.2e-7.  Sigmoid: a
// quarter of 2e-7, then 6e-8 for the sum, 1.2e-7 for the reciprocal and 6e-8
// for the product.  The sum with the bias rounds by 6e-8 of itself.
__device__ __forceinline__ float choice_error(const RouteArgs& a, float largest, float most_bias)
{
    return (a.sigmoid ? 4e-7f : 4e-6f * largest) + 1.2e-7f * (1.0f + most_bias);
}

// The experts of a row in 64 bits, by the whole wave.
template <int P, bool kGroups>
__device__ __forceinline__ int choose_exactly(const RouteArgs& a, int64_t row, double* buf)
{
    float l[P];
    double c[P];
    const int e0 = (threadIdx.x & 63) * P;
    load_logits<P>(a, row, e0, l);
    drop_not_finite(l);
    float top = 0.0f;
    double sum = 1.0;
    if (!a.sigmoid) softmax_of<64, P>(l, top, sum);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        double v;
        if (a.sigmoid) {
            const double e = exp(-__builtin_fabs((double)l[i]));
            v = (l[i] < 0 ? e : 1.0) / (1.0 + e);
        } else {
            v = exp((double)l[i] - (double)top) / sum;
        }
        if (a.bias && e0 + i < a.E) v += (double)a.bias[e0 + i];
        c[i] = l[i] > -INFINITY && v - v == 0 ? v : -INFINITY;
    }
    int mine;
    choose<64, P, kGroups, false, double>(a, row, l, c, 0.0, buf, mine);
    return mine;
}

// The weight of the expert that lane j of a row chose (lanes without one: 0).
template <int L>
__device__ __forceinline__ float weight_of(const RouteArgs& a, int64_t row, int mine, float top, float inverse)
{
    const float l = mine >= 0 ? logit_at(a, row + mine) : -INFINITY;
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
// counts, and k_route_place writes them.
template <int L, int P, int kMode>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a)
{
    constexpr int kRows = kThreads / L, kPasses = kChunk / kRows, kWaves = kThreads / 64;
    constexpr int kExact = L == 64 ? P : P > 4 ? P / 4 : 1;         // experts a lane, for a row held by the wave
    constexpr int kBuf = (L == 64 ? 8 : 16) * (L * P + kMostGroups);  // bytes of a wave: rows in fp32, or one in 64 bits
    __shared__ unsigned long long mask[L * P];
    __shared__ int waves[kWaves];
    __shared__ __attribute__((aligned(16))) uint8_t bufs[kMode == 2 ? kWaves * kBuf : 16];
    const int tid = threadIdx.x, sub = tid & (L - 1), e0 = sub * P;
    const int64_t first = (int64_t)blockIdx.x * kChunk;
    uint8_t* buf = bufs + (kMode == 2 ? wave_index() * kBuf : 0);
    for (int e = tid; e < L * P; e += kThreads) mask[e] = 0;
    __syncthreads();
    int chosen[kPasses];
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
        chosen[pass] = -1;
        const int64_t t0 = first + pass * kRows;
        if (t0 >= a.T) break;
        const int64_t t = t0 + tid / L;
        const bool live = t < a.T;
        const int64_t row = (live ? t : a.T - 1) * a.ld;
        float l[P];
        load_logits<P>(a, row, e0, l);
        const bool bad = own_bits<L>(__ballot(drop_not_finite(l))) != 0;
        float top = 0.0f, sum = 1.0f;
        const bool stats = !a.sigmoid && (kMode != 0 || !a.renorm || a.scores);
        if (stats) softmax_of<L, P>(l, top, sum);
        const float inverse = sum > 0.0f ? 1.0f / sum : 0.0f;  // (a padded token: scores of 0)
        const auto score = [&](float x) {
            if (!a.sigmoid) return exp_neg(x - top) * inverse;
            const float e = exp_neg(-__builtin_fabsf(x));
            return (x < 0.0f ? e : 1.0f) * __builtin_amdgcn_rcpf(1.0f + e);
        };
        if (a.scores && live) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (e0 + i < a.E) a.scores[t * a.E + e0 + i] = bad ? NAN : score(l[i]);
        }
        int mine;
        if constexpr (kMode == 0) {
            float c[P];
#pragma unroll
            for (int i = 0; i < P; ++i) c[i] = l[i];
            choose<L, P, false, false, float>(a, row, l, c, 0.0f, nullptr, mine);
        } else {
            float c[P], most_bias = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float v = score(l[i]);
                if (a.bias) {
                    const float b = e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
                    v += b;
                    const float size = __builtin_fabsf(b);
                    most_bias = size < INFINITY && size > most_bias ? size : most_bias;
                }
                c[i] = l[i] > -INFINITY && v - v == 0.0f ? v : -INFINITY;
            }
            if (a.bias) most_bias = over_lanes<L>(most_bias, Max());
            bool close = choose<L, P, kMode == 2, true, float>(
                a, row, l, c, choice_error(a, inverse, most_bias),
                reinterpret_cast<float*>(buf) + (L == 64 ? 0 : (tid >> 4 & 3) * (L * P + kMostGroups)), mine);
            uint64_t again = __ballot(close && live);
            while (again) {
                const int lane = __builtin_ctzll(again);
                const int64_t that = uniform_of(row, lane);
                const int exact = choose_exactly<kExact, kMode == 2>(a, that, reinterpret_cast<double*>(buf));
                const int moved = __shfl(exact, sub, 64);
                if (L == 64 || (tid & 63) / L == lane / L) mine = moved;
                again &= L == 64 ? 0 : ~(0xFFFFull << (lane & 48));
            }
        }
        const float w = weight_of<L>(a, row, mine, top, inverse);
        if (live && sub < a.k) {
            a.experts[t * a.k + sub] = mine;
            a.weights[t * a.k + sub] = bad ? NAN : w;
            if (mine >= 0) atomicOr(&mask[mine], 1ull << (t - first));
        }
        chosen[pass] = live && sub < a.k ? mine : -1;
    }
    if (!a.ends) return;
    __syncthreads();
    const int count = tid < a.E ? __popcll(mask[tid]) : 0;
    if (gridDim.x > 1) {
        if (tid < a.E) a.counts[(int64_t)blockIdx.x * a.E + tid] = count;
        return;
    }
    __shared__ int start[L * P];
    int all;
    const int upto = group_scan(count, waves, all);
    if (tid < a.E) {
        a.ends[tid] = upto;
        start[tid] = upto - count;
    }
    __syncthreads();
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
        const int64_t t = first + pass * kRows + tid / L;
        if (t >= a.T || sub >= a.k) continue;
        const int e = chosen[pass];
        a.rows[t * a.k + sub] = e < 0 ? -1 : start[e] + __popcll(mask[e] & ((1ull << (t - first)) - 1));
    }
}

// The places of a chunk's slots.  Each workgroup adds up all chunks' counts
// (they lie in the L2: 256 chunks of 256 experts are 256 KB), those before its
// own and all of them, unless k_route_sums has done so (summed).
__global__ __launch_bounds__(kThreads) void k_route_place(RouteArgs a, int chunks, bool summed)
{
    __shared__ unsigned long long mask[kMostExperts];
    __shared__ int start[kMostExperts], waves[kThreads / 64], before[kThreads], total[kThreads];
    const int tid = threadIdx.x, chunk = blockIdx.x;
    const int64_t first = (int64_t)chunk * kChunk;
    const int slots = (int)(min((int64_t)kChunk, a.T - first) * a.k);
    const int slot = tid, e = slot < slots ? a.experts[first * a.k + slot] : -1, t = slot / a.k;
    for (int i = tid; i < a.E; i += kThreads) mask[i] = 0;
    int mine = 0, all = 0;  // this thread's expert: its rows in earlier chunks, and in all
    if (summed) {
        if (tid < a.E) {
            mine = a.counts[(int64_t)chunk * a.E + tid];
            all = a.counts[(int64_t)chunks * a.E + tid];
        }
        __syncthreads();
    } else {
        // slices of the chunks, E threads each
        const int slices = kThreads / a.E, s = tid / a.E, i = tid - s * a.E;
        int b = 0, n = 0;
        if (s < slices) {
            for (int c = s; c < chunks; c += slices) {
                const int v = a.counts[(int64_t)c * a.E + i];
                n += v;
                b += c < chunk ? v : 0;
            }
        }
        before[tid] = b;
        total[tid] = n;
        __syncthreads();
        if (tid < a.E)
            for (int j = 0; j < slices; ++j) {
                mine += before[j * a.E + tid];
                all += total[j * a.E + tid];
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

// Many chunks: their counts become the sums of those before, expert by expert,
// and a last row of totals.  A workgroup takes 16 experts, 64 runs of the chunks.
__global__ __launch_bounds__(kThreads) void k_route_sums(int* __restrict__ counts, int chunks, int E)
{
    __shared__ int part[64][17];
    const int i = threadIdx.x & 15, s = threadIdx.x >> 4, e = blockIdx.x * 16 + i;
    const int64_t from = (int64_t)chunks * s / 64, to = (int64_t)chunks * (s + 1) / 64;
    int n = 0;
    if (e < E)
        for (int64_t c = from; c < to; ++c) n += counts[c * E + e];
    part[s][i] = n;
    __syncthreads();
    int at = 0;
    for (int j = 0; j < s; ++j) at += part[j][i];
    if (e >= E) return;
    for (int64_t c = from; c < to; ++c) {
        const int v = counts[c * E + e];
        counts[c * E + e] = at;
        at += v;
    }
    if (s == 63) counts[(int64_t)chunks * E + e] = at;
}

// Gradients of the logits, L lanes a row, P experts each.  With g = scale dw
// over the chosen and d the gradients of the scores:
//   renormalised, p the chosen scores over their sum:
//     softmax  p (g - sum g p),   sigmoid  p (g - sum g p) (1 - s)
//   otherwise: softmax  s (g - sum g s),   sigmoid  g s (1 - s)
//   and of d: softmax  s (d - sum d s),   sigmoid  d s (1 - s).
// The chosen's part is added in LDS, slot by slot (a repeated expert adds up
// in order).  Only what the form needs is read: renormalised weights need the
// chosen logits alone.
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
        float s[P], top = 0.0f, inverse = 1.0f;
        bool bad = false;
        if (whole) {
            load_logits<P>(a.f, row, e0, s);
            bad = own_bits<L>(__ballot(drop_not_finite(s))) != 0;
            if (softmax) {
                float sum;
                softmax_of<L, P>(s, top, sum);
                inverse = sum > 0.0f ? 1.0f / sum : 0.0f;
            }
        }
        // the chosen
        const int e = sub < a.f.k ? a.f.experts[t * a.f.k + sub] : -1;
        const bool there = e >= 0 && e < a.f.E;
        const float l = there ? logit_at(a.f, row + e) : -INFINITY;
        const float g = there ? a.f.scale * a.dweights[t * a.f.k + sub] : 0.0f;
        const float neg = l < 0.0f ? l : 0.0f, half = 1.0f / (1.0f + exp_neg(-__builtin_fabsf(l)));
        const float rest = exp_neg(l > 0.0f ? -l : 0.0f) * half;  // 1 - 1 / (1 + e^-l)
        float d, dot = 0.0f;
        if (a.f.renorm) {
            const float x = a.f.sigmoid ? neg : l;
            float m = over_lanes<L>(there ? x : -INFINITY, Max());
            m = m > -INFINITY ? m : 0.0f;
            const float q = there ? exp_neg(x - m) * (a.f.sigmoid ? half : 1.0f) : 0.0f;
            const float all = over_lanes<L>(q, Add());
            const float p = all > 0.0f ? q / all : 0.0f;
            const float mean = over_lanes<L>(there ? g * p : 0.0f, Add());
            d = p * (g - mean) * (a.f.sigmoid ? rest : 1.0f);
        } else if (a.f.sigmoid) {
            d = g * (exp_neg(neg) * half) * rest;
        } else {
            d = g * (exp_neg(l - top) * inverse);
            dot = over_lanes<L>(there ? d : 0.0f, Add());
        }
        if (!there) d = 0.0f;
        __builtin_amdgcn_wave_barrier();  // (the last row's reads)
#pragma unroll
        for (int i = 0; i < P; ++i) part[e0 + i] = 0.0f;
        __builtin_amdgcn_wave_barrier();
        for (int j = 0; j < a.f.k; ++j) {
            if (sub == j && there) part[e] += d;
            __builtin_amdgcn_wave_barrier();
        }
        float o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = part[e0 + i];
        if (whole) {
            float ds[P], along = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                ds[i] = a.dscores && e0 + i < a.f.E ? a.dscores[t * a.f.E + e0 + i] : 0.0f;
                if (softmax) {
                    s[i] = exp_neg(s[i] - top) * inverse;
                    along = __builtin_fmaf(ds[i], s[i], along);
                } else {
                    const float h = 1.0f / (1.0f + exp_neg(-__builtin_fabsf(s[i])));
                    s[i] = exp_neg(-__builtin_fabsf(s[i])) * h * h;  // s (1 - s)
                }
            }
            if (softmax) along = (a.dscores ? over_lanes<L>(along, Add()) : 0.0f) + dot;
#pragma unroll
            for (int i = 0; i < P; ++i) o[i] = bad ? NAN : __builtin_fmaf(s[i], ds[i] - along, o[i]);
        }
        if (!live) continue;  // (no lane moves follow in this round of the loop)
        const int64_t at = t * a.ld_out + e0;
        if (P >= 4 && a.vec_out) {
#pragma unroll
            for (int i = 0; i < P; i += 4) {
                if (e0 + i + 4 <= a.f.E) {
                    if (a.out_f32)
                        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at + i) =
                            make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    else
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at + i) =
                            make_uint2(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]));
                } else {
#pragma unroll
                    for (int j = i; j < i + 4; ++j)
                        if (e0 + j < a.f.E) {
                            if (a.out_f32) static_cast<float*>(a.out)[at + j] = o[j];
                            else static_cast<uint16_t*>(a.out)[at + j] = (uint16_t)pack_bf16(o[j], 0.0f);
                        }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (e0 + i < a.f.E) {
                    if (a.out_f32) static_cast<float*>(a.out)[at + i] = o[i];
                    else static_cast<uint16_t*>(a.out)[at + i] = (uint16_t)pack_bf16(o[i], 0.0f);
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

bool sums_apart(int64_t chunks) { return chunks > 256; }

}  // namespace

int64_t route_workspace(int64_t T, int64_t E)
{
    const int64_t chunks = (T + kChunk - 1) / kChunk;
    return chunks > 1 ? (chunks + (sums_apart(chunks) ? 1 : 0)) * E * (int64_t)sizeof(int) : 0;
}

void launch_route(const RouteArgs& a, hipStream_t s)
{
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
    const bool apart = sums_apart(chunks);
    if (apart)
        hipLaunchKernelGGL(k_route_sums, dim3((uint32_t)((a.E + 15) / 16)), dim3(kThreads), 0, s, a.counts, (int)chunks, a.E);
    hipLaunchKernelGGL(k_route_place, dim3(grid), dim3(kThreads), 0, s, a, (int)chunks, apart);
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
