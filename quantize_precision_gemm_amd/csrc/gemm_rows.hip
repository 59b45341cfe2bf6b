// gemm_rows.hip -- GEMMs over rows of 16-byte pieces on gfx950: products
// grouped by expert in bf16, and the 8-bit integer product.
//
// Grouped products (a linear layer whose tokens are split among experts,
// sorted by expert): for the rows t of expert e
//   fprop  Y[t, n]  = sum_k X[t, k] W[e, n, k]
//   dgrad  dX[t, k] = sum_n dY[t, n] W[e, n, k]
//   wgrad  dW[e, n, k] = sum_{t in e} dY[t, n] X[t, k]
// Integer product: Y[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k].
//
// v_mfma_f32_16x16x32_bf16 and v_mfma_i32_16x16x64_i8 both take 16 bytes of
// a row per lane, so one loop serves both types: lane l supplies row l % 16
// and the 16-byte piece l / 16 of a 64-byte step, and accumulator j of lane l
// is row 4 (l / 16) + j of the first operand, column l % 16 of the second.
// The output's columns are passed as the first operand, so that a lane holds
// 4 neighbouring columns of one output row.
#include <type_traits>

#include "internal.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

__device__ __forceinline__ f32x4_t mma(uint4 a, uint4 b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
}

__device__ __forceinline__ i32x4_t mma(uint4 a, uint4 b, i32x4_t c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c,
                                                 0, 0, 0);
}

// One product of a launch, in elements: rows x K operands (element (r, k) at
// r * ld + k), or with kT rows (K x rows, element (r, k) at k * ld + r).
struct View {
    const uint8_t* p;
    int64_t ld;    // bytes from row to row (or from k to k)
    int64_t rows;  // rows there are
};

// This launch's share of a grouped product.
struct Slice {
    int64_t e;             // expert; E: the rows that belong to none
    int64_t begin, end;    // its rows
    int64_t tile;          // this workgroup's tile of them
};

// Tile `tile` of the experts' row tiles of `rows` rows each, counted expert
// by expert, the rows behind the last expert as one more; false past them
// all.  Each wave scans the ends, 64 at a time.
__device__ __forceinline__ bool find_slice(const int32_t* __restrict__ ends, int64_t E, int64_t T, int rows, int64_t tile,
                                           Slice& s)
{
    const int lane = threadIdx.x & 63;
    int prev = 0;        // end of the experts before this chunk
    int64_t before = 0;  // tiles of those
    for (int64_t e0 = 0; e0 <= E; e0 += 64) {
        const int64_t e = e0 + lane;
        int end = e < E ? min(max(ends[e], 0), (int)T) : (int)T;
        end = max(end, prev);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(end, o, 64);
            if (lane >= o) end = max(end, u);
        }
        int begin = __shfl_up(end, 1, 64);
        if (lane == 0) begin = prev;
        int tiles = e <= E ? (end - begin + rows - 1) / rows : 0;
        const int own = tiles;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(tiles, o, 64);
            if (lane >= o) tiles += u;
        }
        const unsigned long long past = __ballot(before + tiles > tile);
        if (past) {
            const int l = __builtin_ctzll(past);
            s.e = e0 + l;
            s.begin = __shfl(begin, l, 64);
            s.end = __shfl(end, l, 64);
            s.tile = tile - (before + __shfl(tiles - own, l, 64));
            return true;
        }
        prev = __shfl(end, 63, 64);
        before += __shfl(tiles, 63, 64);
    }
    return false;
}

// The rows of expert e (wgrad), as find_slice sees them.
__device__ __forceinline__ void expert_rows(const int32_t* __restrict__ ends, int64_t e, int64_t T, int64_t& begin,
                                            int64_t& end)
{
    const int lane = threadIdx.x & 63;
    int b = 0;  // the largest end before e
    for (int64_t i = lane; i < e; i += 64) b = max(b, ends[i]);
    b = (int)wave_max_u32((uint32_t)max(b, 0));
    b = min(b, (int)T);
    begin = b;
    end = max(b, min(max(ends[e], 0), (int)T));
}

// 16 bytes (one MFMA operand piece) of row r from byte kb of its K; bytes
// from kend on read as zero (kb and kend multiples of 16).
template <bool kT>
__device__ __forceinline__ uint4 piece(const View& v, int64_t r, int64_t kb, int64_t kend)
{
    if constexpr (!kT) {
        return kb < kend ? *reinterpret_cast<const uint4*>(v.p + r * v.ld + kb) : make_uint4(0, 0, 0, 0);
    } else {  // bf16 only: 8 values, one from each k row
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t k = (kb >> 1) + j;
            if (2 * k < kend) w[j >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(v.p + k * v.ld + 2 * r) << (16 * (j & 1));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// 4 neighbouring columns of an output row.
template <bool kF32>
__device__ __forceinline__ void store_cols(void* c, int64_t at, int64_t n, int64_t N, const float (&y)[4])
{
    if constexpr (kF32) {
        float* d = static_cast<float*>(c) + at;
        if (n + 4 <= N) {
            *reinterpret_cast<float4*>(d) = make_float4(y[0], y[1], y[2], y[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < N) d[j] = y[j];
        }
    } else {
        uint16_t* d = static_cast<uint16_t*>(c) + at;
        const uint32_t w[2] = {bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3])};
        if (n + 4 <= N) {
            *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (n + j < N) d[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
        }
    }
}

// ---------------------------------------------------------------------------
// Few rows: a workgroup of 4 waves computes 16 kM rows x 16 kN columns, each
// wave a quarter of the contraction (128-byte steps dealt in turn), straight
// from memory to registers; the parts are added in wave order in LDS.
// ---------------------------------------------------------------------------
template <class Acc, bool kTA, bool kTB, int kM, int kN, class Out>
__device__ __forceinline__ void thin_tile(const View& A, const View& B, int64_t kend, int64_t m0, int64_t n0,
                                          f32x4_t* lds, const Out& out)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    Acc acc[kM][kN] = {};
    for (int64_t k0 = 128 * wave; k0 < kend; k0 += 512) {
        const int64_t kb = k0 + 32 * g;
        uint4 a[kM][2], b[kN][2];
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) b[j][h] = piece<kTB>(B, min(n0 + 16 * j + r, B.rows - 1), kb + 16 * h, kend);
#pragma unroll
        for (int i = 0; i < kM; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) a[i][h] = piece<kTA>(A, min(m0 + 16 * i + r, A.rows - 1), kb + 16 * h, kend);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < kM; ++i)
#pragma unroll
                for (int j = 0; j < kN; ++j) acc[i][j] = mma(b[j][h], a[i][h], acc[i][j]);
    }
    Acc* part = reinterpret_cast<Acc*>(lds);
#pragma unroll
    for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < kN; ++j) part[(wave * kM * kN + i * kN + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int t = wave; t < kM * kN; t += 4) {
        Acc sum = part[t * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) sum += part[(w * kM * kN + t) * 64 + lane];
        const int64_t m = m0 + 16 * (t / kN) + r, n = n0 + 16 * (t % kN) + 4 * g;
        if (m < A.rows && n < B.rows) out(m, n, sum);
    }
}

constexpr int kThinM = 2, kThinN = 2;

}  // namespace

template <int kPass, bool kF32>
__global__ __launch_bounds__(256) void k_grouped_thin(GroupedArgs g)
{
    __shared__ f32x4_t lds[4 * kThinM * kThinN * 64];
    const int64_t cols = kPass == 0 ? g.N : g.K;
    const int64_t tn = (cols + 16 * kThinN - 1) / (16 * kThinN);
    View A, B;
    int64_t m0, n0, kend, row0;
    int64_t c_at = 0;
    if constexpr (kPass == 2) {
        const int64_t tm = (g.N + 16 * kThinM - 1) / (16 * kThinM);
        const int64_t e = blockIdx.x / (tm * tn), in = blockIdx.x % (tm * tn);
        int64_t begin, end;
        expert_rows(g.ends, e, g.T, begin, end);
        A = View{reinterpret_cast<const uint8_t*>(g.a + begin * g.lda), 2 * g.lda, g.N};
        B = View{reinterpret_cast<const uint8_t*>(g.b + begin * g.ldb), 2 * g.ldb, g.K};
        m0 = in / tn * 16 * kThinM;
        n0 = in % tn * 16 * kThinN;
        kend = 2 * (end - begin);
        row0 = 0;
        c_at = e * g.c_expert;
    } else {
        Slice s;
        if (!find_slice(g.ends, g.E, g.T, 16 * kThinM, blockIdx.x / tn, s)) return;
        A = View{reinterpret_cast<const uint8_t*>(g.a + s.begin * g.lda), 2 * g.lda, s.end - s.begin};
        const int64_t e = s.e < g.E ? s.e : 0;
        B = View{reinterpret_cast<const uint8_t*>(g.b + e * g.b_expert), 2 * g.ldb, cols};
        m0 = s.tile * 16 * kThinM;
        n0 = blockIdx.x % tn * 16 * kThinN;
        kend = s.e < g.E ? 2 * (kPass == 0 ? g.K : g.N) : 0;  // rows of no expert: zeros
        row0 = s.begin;
    }
    thin_tile<f32x4_t, kPass == 2, kPass != 0, kThinM, kThinN>(
        A, B, kend, m0, n0, lds, [&](int64_t m, int64_t n, f32x4_t v) {
            const float y[4] = {v[0], v[1], v[2], v[3]};
            store_cols<kF32>(g.c, c_at + (row0 + m) * g.ldc + n, n, B.rows, y);
        });
}

template <bool kF32>
__global__ __launch_bounds__(256) void k_i8_thin(const int8_t* __restrict__ a, int64_t lda, const float* __restrict__ sa,
                                                 const int8_t* __restrict__ b, int64_t ldb, const float* __restrict__ sb,
                                                 int64_t M, int64_t N, int64_t K, void* __restrict__ c, int64_t ldc)
{
    __shared__ f32x4_t lds[4 * kThinM * kThinN * 64];
    const int64_t tn = (N + 16 * kThinN - 1) / (16 * kThinN);
    const View A{reinterpret_cast<const uint8_t*>(a), lda, M}, B{reinterpret_cast<const uint8_t*>(b), ldb, N};
    thin_tile<i32x4_t, false, false, kThinM, kThinN>(
        A, B, K, blockIdx.x / tn * 16 * kThinM, blockIdx.x % tn * 16 * kThinN, lds,
        [&](int64_t m, int64_t n, i32x4_t v) {
            const float s = sa[m];
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = ((float)v[j] * s) * sb[min(n + j, N - 1)];
            store_cols<kF32>(c, m * ldc + n, n, N, y);
        });
}

void launch_i8_gemm(const int8_t* a, int64_t lda, const float* sa, const int8_t* b, int64_t ldb, const float* sb,
                    int64_t M, int64_t N, int64_t K, void* c, int64_t ldc, bool out_fp32, hipStream_t s)
{
    if (M == 0 || N == 0) return;
    const int64_t grid = (M + 16 * kThinM - 1) / (16 * kThinM) * ((N + 16 * kThinN - 1) / (16 * kThinN));
    if (out_fp32)
        hipLaunchKernelGGL(k_i8_thin<true>, dim3((uint32_t)grid), dim3(256), 0, s, a, lda, sa, b, ldb, sb, M, N, K, c, ldc);
    else
        hipLaunchKernelGGL(k_i8_thin<false>, dim3((uint32_t)grid), dim3(256), 0, s, a, lda, sa, b, ldb, sb, M, N, K, c, ldc);
}

namespace {

template <int kPass>
void launch_grouped_thin(const GroupedArgs& g, bool out_fp32, hipStream_t s)
{
    const int64_t tm = 16 * kThinM, tn = 16 * kThinN;
    const int64_t cols = ((kPass == 0 ? g.N : g.K) + tn - 1) / tn;
    // every expert, and the rows of none, can have one partial row tile
    const int64_t rows = kPass == 2 ? g.E * ((g.N + tm - 1) / tm) : g.T / tm + g.E + 1;
    if (out_fp32)
        hipLaunchKernelGGL((k_grouped_thin<kPass, true>), dim3((uint32_t)(rows * cols)), dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL((k_grouped_thin<kPass, false>), dim3((uint32_t)(rows * cols)), dim3(256), 0, s, g);
}

}  // namespace

void launch_grouped(int pass, const GroupedArgs& g, bool out_fp32, hipStream_t s)
{
    const int64_t rows = pass == 2 ? g.E * g.N : g.T, cols = pass == 0 ? g.N : g.K;
    if (rows == 0 || cols == 0) return;  // (an empty contraction still writes zeros)
    if (pass == 0) launch_grouped_thin<0>(g, out_fp32, s);
    else if (pass == 1) launch_grouped_thin<1>(g, out_fp32, s);
    else launch_grouped_thin<2>(g, out_fp32, s);
}

}  // namespace nvfp4
