// adamw.hip -- one AdamW step over many tensors on gfx950, with the two
// moments held in fp32 or in 8 bits.
//
// With the gradient g (times the optional device factor grad_scale):
//   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
//   p = p (1 - lr decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
// all in fp32, every operation rounded once (the factors that depend on the
// step alone are rounded from double on the host).
//
// 8-bit states: m and r = sqrt(v) are OCP E4M3 values times one fp32 power of
// two per block of 128 elements, the smallest for which no value passes 448;
// the root needs half the exponent range of v.  A root that is not zero is
// held as at least the smallest E4M3 value (2^-9 of its scale), so that an
// element with a first moment is never divided by eps alone.  The update uses
// m and r before they are rounded to 8 bits.  The next step squares r: its
// scale goes up to 2^55, (448 * 2^55)^2 = 0.77 * 2^128.  An element that is
// NaN or infinite, or whose v has overflowed, does not count for its block's
// scales: its neighbours keep theirs.
//
// Every element is read and written once: the step is bound by HBM traffic
// (30 bytes an element with fp32 states, fp32 gradients and a bf16 copy,
// 18.1 with 8-bit states).  Stores go past the caches, and loads too where a
// launch moves more than the last-level cache holds twice (512 MB): 139.8M
// elements in 32 bits 747 -> 693 us (6.05 TB/s), 106.2M in 8 bits 328 -> 311 us
// (6.2 TB/s); of 405 MB that the cache does hold, such loads cost 9 us of 58.
#include <type_traits>

#include "internal.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 4;  // elements of one workgroup

__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

// Whole accesses, past the caches if kStream.
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

template <bool kStream, class V>
__device__ __forceinline__ V load_vec(const void* p)
{
    return kStream ? __builtin_nontemporal_load(static_cast<const V*>(p)) : *static_cast<const V*>(p);
}

template <class V>
__device__ __forceinline__ void store_vec(V v, void* p)
{
    __builtin_nontemporal_store(v, static_cast<V*>(p));
}

// 4 elements from element i; those past n read as zero.
template <bool kStream>
__device__ __forceinline__ void load4(float (&y)[4], const void* base, int64_t i, int64_t n, bool vec, float)
{
    const float* p = static_cast<const float*>(base) + i;
    if (vec && i + 4 <= n) {
        const f32x4_t v = load_vec<kStream, f32x4_t>(p);
        y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = i + k < n ? p[k] : 0.0f;
    }
}

template <bool kStream>
__device__ __forceinline__ void load4(float (&y)[4], const void* base, int64_t i, int64_t n, bool vec, uint16_t)
{
    const uint16_t* p = static_cast<const uint16_t*>(base) + i;
    if (vec && i + 4 <= n) {
        const u32x2_t v = load_vec<kStream, u32x2_t>(p);
        y[0] = __uint_as_float(v.x << 16), y[1] = __uint_as_float(v.x & 0xFFFF0000u);
        y[2] = __uint_as_float(v.y << 16), y[3] = __uint_as_float(v.y & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = i + k < n ? bf16_to_f32(p[k]) : 0.0f;
    }
}

__device__ __forceinline__ void store4(const float (&y)[4], void* base, int64_t i, int64_t n, bool vec, float)
{
    float* p = static_cast<float*>(base) + i;
    if (vec && i + 4 <= n) {
        store_vec(f32x4_t{y[0], y[1], y[2], y[3]}, p);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[k] = y[k];
    }
}

__device__ __forceinline__ void store4(const float (&y)[4], void* base, int64_t i, int64_t n, bool vec, uint16_t)
{
    uint16_t* p = static_cast<uint16_t*>(base) + i;
    const uint32_t w[2] = {bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3])};
    if (vec && i + 4 <= n) {
        store_vec(u32x2_t{w[0], w[1]}, p);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
    }
}

// 4 E4M3 codes from element i (past n: zero).
template <bool kStream>
__device__ __forceinline__ uint32_t load_codes(const void* base, int64_t i, int64_t n, bool vec)
{
    const uint8_t* p = static_cast<const uint8_t*>(base) + i;
    if (vec && i + 4 <= n) return load_vec<kStream, uint32_t>(p);
    uint32_t w = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (i + k < n) w |= (uint32_t)p[k] << (8 * k);
    return w;
}

__device__ __forceinline__ void store_codes(uint32_t w, void* base, int64_t i, int64_t n, bool vec)
{
    uint8_t* p = static_cast<uint8_t*>(base) + i;
    if (vec && i + 4 <= n) {
        store_vec(w, p);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + k < n) p[k] = (uint8_t)(w >> (8 * k));
    }
}

__device__ __forceinline__ void decode4(float (&y)[4], uint32_t w, float scale)
{
    y[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0) * scale;
    y[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * scale;
    y[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * scale;
    y[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * scale;
}

// Max over the 32 lanes that hold one block of 128 elements.
__device__ __forceinline__ uint32_t block_max(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, true));   // lanes ^ 1
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, true));   // lanes ^ 2
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, true));  // mirror in 8
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, true));  // mirror in 16
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return max((uint32_t)r[0], (uint32_t)r[1]);
}

// Bits of the largest values that an 8-bit state holds without saturating:
// 448 * 2^55 for roots, 448 * 2^119 for first moments.
template <bool kRoot>
constexpr uint32_t kMost = kRoot ? 0x5F600000u : 0x7F600000u;

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t largest(const float (&y)[4])
{
    return max(max(magnitude(y[0]), magnitude(y[1])), max(magnitude(y[2]), magnitude(y[3])));
}

// The 4 values y (the roots r themselves if kRoot, else the first moments) as
// E4M3 codes and their block's scale: 2^j, j the smallest for which
// max |y| <= 448 * 2^j (a mantissa above 1.75 takes the next power), from -126
// to 55 for roots and 119 for first moments.  The maximum is over the elements
// whose y and r are finite.  Larger finite values and infinite roots
// (overflowed squares of finite gradients) are held as the largest code, so that the
// next steps stay finite; other infinities and NaN as NaN.  kPlain: there are
// none of these in the wave (checking every element cost 310 -> 316 us over
// 106.2M, checking the wave nothing).
template <bool kRoot, bool kPlain>
__device__ __forceinline__ uint32_t encode4(const float (&y)[4], const float (&r)[4], float& scale)
{
    constexpr uint32_t kInf = 0x7F800000u;
    uint32_t top = 0;
    if (kPlain) {
        top = largest(y);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (magnitude(y[k]) < kInf && magnitude(r[k]) < kInf) top = max(top, magnitude(y[k]));
    }
    top = min(block_max(top), kMost<kRoot>);
    const int e = max((int)((top + 0x1FFFFFu) >> 23) - 8, 1);
    scale = __uint_as_float((uint32_t)e << 23);
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
    float q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float t = y[k] * inv;
        if (kRoot) t = t > 0.0f ? __builtin_fmaxf(t, 0x1p-9f) : t;
        if (!kPlain && __builtin_fabsf(t) > 448.0f)
            t = !kRoot && magnitude(y[k]) == kInf ? __uint_as_float(0x7FC00000u) : __builtin_copysignf(448.0f, t);
        q[k] = t;
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    return (uint32_t)w;
}

// The factor of the gradients; false: it is not finite, the step is left out.
__device__ __forceinline__ bool gradient_scale(const AdamWStep& a, float& gs)
{
    gs = a.grad_scale ? *a.grad_scale : 1.0f;
    return (__float_as_uint(gs) & 0x7F800000u) != 0x7F800000u;
}

// A workgroup's 1024 elements, the chunk-th of tensor t.
template <class P, class G, bool k8, bool kStream>
__device__ __forceinline__ void update(const AdamWStep& a, float gs, const AdamWTensor& t, uint32_t chunk)
{
    const int lane = threadIdx.x & 63;
    const int64_t n = t.n;
    const bool vec = t.vec != 0;
    const int64_t i = (int64_t)chunk * kChunk + 4 * threadIdx.x;

    float p[4], g[4], m[4], v[4], r[4];
    load4<kStream>(p, t.p, i, n, vec, P());
    load4<kStream>(g, t.g, i, n, vec, G());
    const int64_t nb = (n + 127) >> 7, b = i >> 7;
    if constexpr (k8) {
        const uint32_t cm = load_codes<kStream>(t.m, i, n, vec), cv = load_codes<kStream>(t.v, i, n, vec);
        const float sm = b < nb ? t.m_scale[b] : 0.0f, sv = b < nb ? t.v_scale[b] : 0.0f;
        decode4(m, cm, sm);
        decode4(r, cv, sv);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = r[k] * r[k];
    } else {
        load4<kStream>(m, t.m, i, n, vec, float());
        load4<kStream>(v, t.v, i, n, vec, float());
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float gk = g[k] * gs;
        m[k] = a.beta1 * m[k] + a.rest1 * gk;
        v[k] = a.beta2 * v[k] + a.rest2 * (gk * gk);
        r[k] = sqrtf(v[k]);
        p[k] = p[k] * a.keep - a.rate * (m[k] / (r[k] * a.root_corr + a.eps));
    }
    store4(p, t.p, i, n, vec, P());
    if (t.copy) store4(p, t.copy, i, n, vec, uint16_t());
    if constexpr (k8) {
        float sm, sv;
        uint32_t cm, cv;
        if (__all(largest(m) <= kMost<false> && largest(r) <= kMost<true>)) {
            cm = encode4<false, true>(m, r, sm);
            cv = encode4<true, true>(r, r, sv);
        } else {
            cm = encode4<false, false>(m, r, sm);
            cv = encode4<true, false>(r, r, sv);
        }
        store_codes(cm, t.m, i, n, vec);
        store_codes(cv, t.v, i, n, vec);
        if ((lane & 31) == 0 && b < nb) {
            t.m_scale[b] = sm;
            t.v_scale[b] = sv;
        }
    } else {
        store4(m, t.m, i, n, vec, float());
        store4(v, t.v, i, n, vec, float());
    }
}

}  // namespace

// One workgroup updates one chunk of one tensor; the tensor is found from the
// first chunk of each, held in the kernel's arguments.
template <class P, class G, bool k8, bool kStream>
__global__ __launch_bounds__(kThreads) void k_adamw(AdamWArgs a)
{
    float gs;
    if (!gradient_scale(a.step, gs)) return;
    const int lane = threadIdx.x & 63;
    const uint32_t mine = a.first[min(lane, a.count)];
    const int at = __builtin_amdgcn_readfirstlane(
        (int)__popcll(__ballot(lane < a.count && mine <= blockIdx.x)) - 1);
    update<P, G, k8, kStream>(a.step, gs, a.t[at], blockIdx.x - a.first[at]);
}

// The same for more tensors than the arguments hold, in one launch (96 small
// tensors 8.5 -> 4.9 us, 1000 of 100000 elements 626 -> 443).  The wave looks at 64 tensors, evenly
// spaced, at a time (96 tensors: twice, 4097: three times).
template <class P, class G, bool k8, bool kStream>
__global__ __launch_bounds__(kThreads) void k_adamw_table(AdamWStep step, const AdamWTensor* __restrict__ t,
                                                          const uint32_t* __restrict__ first, int count)
{
    float gs;
    if (!gradient_scale(step, gs)) return;
    const int lane = threadIdx.x & 63;
    int at = 0;  // the chunk's tensor is one of at .. at + len - 1
    for (int len = count; len > 1;) {
        const int stride = (len + 63) / 64, off = lane * stride;
        const bool past = off < len && first[at + off] <= blockIdx.x;
        const int k = (__builtin_amdgcn_readfirstlane((int)__popcll(__ballot(past))) - 1) * stride;
        at += k;
        len = min(stride, len - k);
    }
    update<P, G, k8, kStream>(step, gs, t[at], blockIdx.x - first[at]);
}

namespace {

// launch(kernel's types): the update past the caches if it moves more than they hold.
template <class P, class G, bool k8, class Launch>
void launch_bits(uint32_t chunks, const Launch& launch)
{
    const int64_t bytes = 2 * sizeof(P) + sizeof(G) + (k8 ? 4 : 16);
    if ((int64_t)chunks * kChunk * bytes > (int64_t)512 << 20)
        launch(P(), G(), std::integral_constant<bool, k8>(), std::true_type());
    else
        launch(P(), G(), std::integral_constant<bool, k8>(), std::false_type());
}

template <class P, class G, class Launch>
void launch_types(uint32_t chunks, bool eight, const Launch& launch)
{
    if (eight) launch_bits<P, G, true>(chunks, launch);
    else launch_bits<P, G, false>(chunks, launch);
}

template <class Launch>
void launch_kind(uint32_t chunks, bool p_bf16, bool g_bf16, bool eight, const Launch& launch)
{
    if (chunks == 0) return;
    if (p_bf16 && g_bf16) launch_types<uint16_t, uint16_t>(chunks, eight, launch);
    else if (p_bf16) launch_types<uint16_t, float>(chunks, eight, launch);
    else if (g_bf16) launch_types<float, uint16_t>(chunks, eight, launch);
    else launch_types<float, float>(chunks, eight, launch);
}

}  // namespace

int64_t adamw_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

void launch_adamw(const AdamWArgs& a, bool p_bf16, bool g_bf16, bool eight, hipStream_t s)
{
    const uint32_t chunks = a.first[a.count];
    launch_kind(chunks, p_bf16, g_bf16, eight, [&](auto p, auto g, auto k8, auto stream) {
        hipLaunchKernelGGL((k_adamw<decltype(p), decltype(g), decltype(k8)::value, decltype(stream)::value>), dim3(chunks),
                           dim3(kThreads), 0, s, a);
    });
}

void launch_adamw_table(const AdamWStep& step, const AdamWTensor* t, const uint32_t* first, int64_t count,
                        uint32_t chunks, bool p_bf16, bool g_bf16, bool eight, hipStream_t s)
{
    launch_kind(chunks, p_bf16, g_bf16, eight, [&](auto p, auto g, auto k8, auto stream) {
        hipLaunchKernelGGL((k_adamw_table<decltype(p), decltype(g), decltype(k8)::value, decltype(stream)::value>),
                           dim3(chunks), dim3(kThreads), 0, s, step, t, first, (int)count);
    });
}

}  // namespace nvfp4
