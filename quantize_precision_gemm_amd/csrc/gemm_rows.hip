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
// The bf16 and the int8 matrix instructions (16 x 16 and 32 x 32 outputs) take
// 16 bytes of a row per lane and give one accumulator layout, so the loops
// serve both types: in a 16 x 16 instruction lane l supplies row l % 16 and
// the 16-byte piece l / 16 of 64 bytes, and accumulator j of lane l is row
// 4 (l / 16) + j of the first operand, column l % 16 of the second; in a
// 32 x 32 one row l % 32 and piece l / 32 of 32 bytes, and accumulator j is
// row 8 (j / 4) + 4 (l / 32) + j % 4, column l % 32.  The output's columns are
// passed as the first operand, so that a lane holds 4 neighbouring columns of
// one output row.
//
// Three kernels, chosen from estimates of their time (see choose()): thin
// tiles (few rows, bound by the weights' bytes), 128 x 128 tiles (fewer of
// them than compute units: bound by latency, with their contraction split
// when it is long) and 256 x 256 tiles (bound by the matrix and LDS pipes).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "internal.hpp"
#include "nvfp4_device.hpp"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b)
{
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32);
}

__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p)
{
    return reinterpret_cast<const uint8_t*>(uniform((int64_t)reinterpret_cast<uintptr_t>(p)));
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

__device__ __forceinline__ f32x16_t mma(uint4 a, uint4 b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   c, 0, 0, 0);
}

__device__ __forceinline__ i32x16_t mma(uint4 a, uint4 b, i32x16_t c)
{
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c,
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
    uint32_t tile;         // this workgroup's tile of them
};

// Inclusive scans over the wave, by lane moves inside the vector unit (a row
// of 16 by 1, 2, 4, 8 lanes, then the last lane of each row into the next).
template <class Op>
__device__ __forceinline__ int wave_scan(int v, int none, const Op& op)
{
    v = op(v, __builtin_amdgcn_update_dpp(none, v, 0x111, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(none, v, 0x112, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(none, v, 0x114, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(none, v, 0x118, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(none, v, 0x142, 0xA, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(none, v, 0x143, 0xC, 0xF, false));
    return v;
}

// Rows [begin, end) of the experts e0 + lane, in order and range whatever the
// ends hold; the rows behind the last expert count as expert E's.  prev: the
// end before e0's rows, and then the last lane's.
__device__ __forceinline__ void lane_rows(const int32_t* __restrict__ ends, int64_t E, int64_t T, int64_t e0, int& prev,
                                          int& begin, int& end)
{
    const int64_t e = e0 + (threadIdx.x & 63);
    end = e < E ? min(max(ends[e], 0), (int)T) : (int)T;
    end = wave_scan(max(end, prev), 0, [](int x, int y) { return max(x, y); });
    begin = __builtin_amdgcn_update_dpp(prev, end, 0x138, 0xF, 0xF, false);  // the lane before's end
    prev = __builtin_amdgcn_readlane(end, 63);
}

// One of the tiles of kRows rows of all experts, each row tile counting
// `cols` times, expert by expert: the one that order(total, at) chooses.
// False if it chooses none.  Each wave scans the ends, 64 at a time.
template <int kRows, class Order>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ ends, int64_t E, int64_t T, int cols,
                                          const Order& order, Slice& s)
{
    const auto add = [](int x, int y) { return x + y; };
    const bool once = E < 64;
    uint32_t total = 0, at = 0;
    for (int pass = once ? 1 : 0; pass < 2; ++pass) {  // the count, then the search
        int prev = 0, begin, end;
        uint32_t before = 0;  // tiles of the experts before this chunk
        for (int64_t e0 = 0; e0 <= E; e0 += 64) {
            lane_rows(ends, E, T, e0, prev, begin, end);
            const int own = (end - begin + kRows - 1) / kRows * cols;
            const int upto = wave_scan(own, 0, add);
            const int all = __builtin_amdgcn_readlane(upto, 63);
            if (once && !order((uint32_t)all, at)) return false;
            const unsigned long long past = pass ? __ballot(before + upto > at) : 0;
            if (past) {
                const int l = __builtin_ctzll(past);
                s.e = e0 + l;
                s.begin = __builtin_amdgcn_readlane(begin, l);
                s.end = __builtin_amdgcn_readlane(end, l);
                s.tile = at - (before + __builtin_amdgcn_readlane(upto - own, l));
                return true;
            }
            before += all;
        }
        total = before;
        if (pass == 0 && !order(total, at)) return false;
    }
    return false;
}

// The rows of expert e (wgrad), as find_tile sees them.
__device__ __forceinline__ void expert_rows(const int32_t* __restrict__ ends, uint32_t e, int64_t T, int64_t& begin,
                                            int64_t& end)
{
    const uint32_t lane = threadIdx.x & 63;
    int b = 0;  // the largest end before e
    for (uint32_t i = lane; i < e; i += 64) b = max(b, ends[i]);
    b = __builtin_amdgcn_readfirstlane((int)wave_max_u32((uint32_t)max(b, 0)));
    b = min(b, (int)T);
    begin = b;
    end = max(b, min(max(ends[e], 0), (int)T));
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
// Few rows: bound by the weights' bytes.  A workgroup of 4 waves computes
// 16 kM rows x 16 kN columns (rows x K operands only), each wave a quarter of
// the contraction, 128-byte steps dealt in turn, straight from memory to
// registers with kU steps in flight; the parts are added in wave order in LDS.
// One token through 5120 -> 20480 in int8: 18.1 us, 5.8 TB/s of the weight.
// ---------------------------------------------------------------------------
template <class Acc, int kM, int kN, int kU, class Out>
__device__ __forceinline__ void thin_tile(const View& A, const View& B, int64_t kend, int64_t m0, int64_t n0,
                                          f32x4_t* lds, const Out& out)
{
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int r = lane & 15, g = lane >> 4;
    const uint8_t *pa[kM], *pb[kN];
#pragma unroll
    for (int i = 0; i < kM; ++i) pa[i] = A.p + min(m0 + 16 * i + r, A.rows - 1) * A.ld + 16 * g;
#pragma unroll
    for (int j = 0; j < kN; ++j) pb[j] = B.p + min(n0 + 16 * j + r, B.rows - 1) * B.ld + 16 * g;
    Acc acc[kM][kN] = {};
    auto steps = [&](int64_t k0, auto count, auto whole) {
        constexpr int kSteps = count.value;
        uint4 a[kSteps][kM][2], b[kSteps][kN][2];
        auto piece = [&](const uint8_t* p, int64_t k) {  // pieces past K: zeros
            return whole.value || k + 16 * g < kend ? *reinterpret_cast<const uint4*>(p + k) : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = k0 + 512 * u + 64 * h;
#pragma unroll
                for (int j = 0; j < kN; ++j) b[u][j][h] = piece(pb[j], k);
#pragma unroll
                for (int i = 0; i < kM; ++i) a[u][i][h] = piece(pa[i], k);
            }
        __builtin_amdgcn_sched_barrier(0);  // every load before the first MFMA
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < kM; ++i)
#pragma unroll
                    for (int j = 0; j < kN; ++j) acc[i][j] = mma(b[u][j][h], a[u][i][h], acc[i][j]);
    };
    int64_t k0 = 128 * wave;
    for (; k0 + 512 * (kU - 1) + 128 <= kend; k0 += 512 * kU)
        steps(k0, std::integral_constant<int, kU>(), std::true_type());
    for (; k0 < kend; k0 += 512) steps(k0, std::integral_constant<int, 1>(), std::false_type());
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

// ---------------------------------------------------------------------------
// Many rows: a workgroup of 8 waves computes 256 x 256 outputs in steps of
// 128 bytes of K (64 bf16, 128 int8).
//
// Two LDS buffers of 64 KB each hold a step's A and B tile in halves of 128
// rows (16 KB).  The halves come straight from memory by LDS DMA, 16 bytes a
// lane, and the DMA writes LDS in lane order; so the places are permuted by
// choosing what each lane reads:
//   rows x K  (N): 128 rows of 128 bytes, piece c of row r at place
//     c ^ (r / 2) % 8: the 16 rows of a fragment read, 128 bytes apart, then
//     cover all banks;
//   K x rows  (T): 64 k rows of 256 bytes, 32-byte block b of k row r at
//     b ^ 2 (r % 4): a transposing read takes two neighbouring blocks of 4 k
//     rows, 256 bytes apart, per 32 lanes, which then lie in 8 bank groups.
// Pieces past the operand's K are read from a page of zeros, rows past its
// end from its last row (their products are not stored).
//
// Wave (wm, wn) of 2 x 4 owns rows 64 wm .. +63 of each A half and columns
// 32 wn .. +31 of each B half: four quadrants of two 32 x 32 MFMA tiles.  A
// step has four phases, each of a memory part and 8 MFMAs, between barriers:
//   phase  reads from LDS         multiplies   starts the DMA of
//     0    A0 (8 x 16 B a lane)   A0 B0        A1 of step t + 1
//     1    B1 (4)                 A0 B1        B0 of step t + 2
//     2    A1 (8)                 A1 B1        A0 of step t + 2
//     3    B0 of step t + 1 (4)   A1 B0        B1 of step t + 2
// Waves 4-7 run one barrier behind waves 0-3 (the other wave of each SIMD),
// so one wave's memory part lies beside the other's MFMAs.  A wave's reads of
// a phase have come back before the barrier that ends its MFMAs; a half is
// refilled two phases after its read, which is behind that barrier for every
// wave.  It is next read 5 phases after that, and every memory part ends with
// a wait for all but the last 10 DMA instructions, those of the last 5 phases.
//
// What bounds it: reading LDS (192 KB a step) and the DMA's writes (64 KB)
// keep the LDS busy for about as long as the MFMAs take, and under full load
// the power limit lowers the clock (1.5 to 1.7 GHz): 16384 rows of 8 experts,
// N = K = 5120, 710 to 760 us (1130 to 1210 TFLOP/s, MFMAs 0.70 of the cycles), int8
// 8192 x 20480 x 5120 690 to 735 us (2340 to 2490 TOP/s).  A tile alone: 1.15 us a step and 9
// us for its start and end.
// ---------------------------------------------------------------------------
constexpr int kHalfBytes = 128 * 128;
constexpr int kLdsBytes = 9 * kHalfBytes;

__device__ __attribute__((aligned(16))) const uint8_t kZeros[16] = {0};

// 16 bytes a lane from `src` to LDS byte `lds` + 16 * lane.  (m0 is written
// and read within the statement; the compiler reserves it and warns of its name in a
// clobber list, which changes no instruction here.  Its own uses, LDS DMA by
// builtins, indexed registers and messages, must not be added to these kernels.)
__device__ __forceinline__ void dma16(const uint8_t* src, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory");
}

// The same from `base` (one for the wave) + off.
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
                 : "memory");
}

template <int kLeft>
__device__ __forceinline__ void wait_dma()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ void barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Where one thread's DMA pieces of an operand tile of kHalves x 128 rows come
// from in a workgroup of kThreads: instruction j of half h of a step at the
// step's base + off[kLoads h + j].  Steps that lie wholly inside K take the
// short way (a scalar base and a 32-bit offset; the loops spend more of their
// time on such overhead than on the transfers); the others check each piece.
template <bool kT, int kThreads, int kHalves>
struct Source {
    static constexpr int kLoads = kHalfBytes / (16 * kThreads);  // instructions of a half
    const uint8_t* p;
    uint32_t off[kHalves * kLoads];
    int64_t K, advance;  // K in bytes (N) or k rows (T); bytes from step to step

    // the tile's first row r0; second: whether half 1 is used (if not, its
    // lanes all read one place).  kPairs (N): half h holds the rows 32 h ..
    // 32 h + 31 of every 64, so that a wave's two 32-column pieces are neighbours.
    template <bool kPairs = false>
    __device__ __forceinline__ void set(const View& v, int64_t r0, int64_t K_, bool second)
    {
        const int tid = threadIdx.x;
        const int64_t ld = uniform(v.ld);
        K = uniform(K_);
        advance = kT ? 64 * ld : 128;
        p = uniform(v.p + (kT ? 2 * r0 : r0 * ld));
        const int last = (int)min(v.rows - (kT ? 8 : 1) - r0, (int64_t)255);
#pragma unroll
        for (int i = 0; i < kHalves * kLoads; ++i) {
            if constexpr (!kT) {
                const int r = kThreads / 8 * i + (tid >> 3);  // half r / 128
                const int row = kPairs ? (r >> 5 & 3) * 64 + (r >> 7) * 32 + (r & 31) : r;
                off[i] = (uint32_t)min(row, last) * (uint32_t)ld + 16 * ((tid & 7) ^ ((tid >> 4) & 7));
            } else {
                const int kr = kThreads / 16 * (i % kLoads) + (tid >> 4);
                const int block = ((tid & 15) >> 1) ^ (kr & 3) << 1;
                off[i] = (uint32_t)kr * (uint32_t)ld +
                         2 * min(128 * (i / kLoads) + 16 * block + 8 * (tid & 1), last);
            }
            if (i >= kLoads && !second) off[i] = 0;
        }
    }

    // half `h` of step t, which lies wholly inside K, into LDS at `lds`;
    // base: p + t * advance
    __device__ __forceinline__ void fetch(int h, const uint8_t* base, uint32_t lds) const
    {
        const uint32_t at = lds + wave_id() * 1024;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) dma16(base, off[kLoads * h + j], at + 16 * kThreads * j);
    }

    // the same of any step: zeros for the pieces past K
    __device__ __forceinline__ void fetch_checked(int h, int t, uint32_t lds) const
    {
        const uint32_t at = lds + wave_id() * 1024;
        const uint8_t* base = p + t * advance;
        const int tid = threadIdx.x;
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int64_t k = kT ? (int64_t)t * 64 + kThreads / 16 * j + (tid >> 4)
                                 : (int64_t)t * 128 + 16 * ((tid & 7) ^ ((tid >> 4) & 7));
            dma16(k < K ? base + off[kLoads * h + j] : kZeros, at + 16 * kThreads * j);
        }
    }

    __device__ __forceinline__ int whole() const { return (int)(K >> (kT ? 6 : 7)); }
};

// A lane's fragments of 32-row tiles of one half: kTiles tiles from tile
// `first` (a multiple of kTiles), the four 32-byte sub-steps of each.
template <bool kT, int kTiles>
struct Fragments {
    int at, block;  // N: the lane's row, its piece in sub-step 0; T: its k row and column, its block in tile 0

    __device__ __forceinline__ explicit Fragments(int first)
    {
        const int lane = threadIdx.x & 63;
        if constexpr (!kT) {
            const int r = lane & 31;
            at = (32 * first + r) * 128;
            block = ((lane >> 5) ^ (r >> 1 & 7)) << 4;
        } else {
            const int r = lane & 15, g = lane >> 4;
            at = (8 * (g >> 1) + (r >> 2)) * 256 + 8 * (r & 3);
            block = ((2 * first + (g & 1)) ^ (r >> 2) << 1) << 5;
        }
    }

    __device__ __forceinline__ void read(uint4 (&f)[kTiles][4], const uint8_t* half) const
    {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                if constexpr (!kT) {
                    f[i][s] = *reinterpret_cast<const uint4*>(half + at + (block ^ (s << 5)) + 4096 * i);
                } else {
                    typedef short short4_t __attribute__((ext_vector_type(4)));
                    typedef __attribute__((address_space(3))) short4_t lds_short4;
                    const uint8_t* a = half + at + (block ^ (i << 6)) + 4096 * s;
                    const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_short4*)(__attribute__((address_space(3))) uint8_t*)a);
                    const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                        (lds_short4*)(__attribute__((address_space(3))) uint8_t*)(a + 1024));
                    const uint2 l = __builtin_bit_cast(uint2, lo), u = __builtin_bit_cast(uint2, hi);
                    f[i][s] = make_uint4(l.x, l.y, u.x, u.y);
                }
            }
    }
};

// First column, within the tile, of wave wn's part of B half h.
template <bool kTB>
__device__ __forceinline__ int column0(int wn, int h)
{
    return kTB ? 128 * h + 32 * wn : 64 * wn + 32 * h;
}

// The 256 x 256 products of A rows m0 .. and B rows n0 ..; K in bytes of a
// row, or with kTA (then kTB too, or B alone) the k rows: see Source.
// acc[half of A][half of B][tile of A].  Rows from mend on are not wanted.
template <class Acc, bool kTA, bool kTB>
__device__ __forceinline__ void big_tile(const View& A, const View& B, int64_t m0, int64_t n0, int64_t Ka, int64_t Kb,
                                         int64_t mend, int steps, uint8_t* lds, Acc (&acc)[2][2][2])
{
    const int wave = wave_id(), wm = wave >> 2, wn = wave & 3;
    Source<kTA, 512, 2> sa;
    Source<kTB, 512, 2> sb;
    sa.set(A, m0, Ka, m0 + 128 < mend);
    sb.template set<!kTB>(B, n0, Kb, kTB ? n0 + 128 < B.rows : n0 + 32 < B.rows);
    // a wave's quadrants beyond the rows or columns are left out
    const bool rows0 = m0 + 64 * wm < mend, rows1 = m0 + 128 + 64 * wm < mend;
    const int64_t n = n0 + column0<kTB>(wn, 0);
    const bool cols0 = n < B.rows, cols1 = n0 + column0<kTB>(wn, 1) < B.rows;
    const Fragments<kTA, 2> fa(2 * wm);
    const Fragments<kTB, 1> fb(wn);
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    // A's halves of both buffers, then B's: every place is within a 16-bit
    // offset of its operand's first
    constexpr int kA0 = 0, kA1 = kHalfBytes, kB0 = 4 * kHalfBytes, kB1 = 5 * kHalfBytes, kNext = 2 * kHalfBytes;

    sb.fetch_checked(0, 0, base + kB0);
    sa.fetch_checked(0, 0, base + kA0);
    sb.fetch_checked(1, 0, base + kB1);
    sa.fetch_checked(1, 0, base + kA1);
    sb.fetch_checked(0, 1, base + kNext + kB0);
    sa.fetch_checked(0, 1, base + kNext + kA0);
    sb.fetch_checked(1, 1, base + kNext + kB1);
    uint4 a[2][4], b[2][1][4];
    wait_dma<10>();
    barrier();
    fb.read(b[0], lds + kB0);
    wait_lds();
    barrier();
    if (wm == 1) barrier();

    auto multiply = [&](Acc(&c)[2], const uint4(&bf)[1][4], bool used) {
        if (used) {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) c[i] = mma(bf[0][s], a[i][s], c[i]);
            __builtin_amdgcn_s_setprio(0);
        }
        wait_lds();
        barrier();
    };
    auto between = [&]() {  // the memory part ends
        wait_dma<10>();
        barrier();
    };
    // One step from buffer `buf`; b0 holds its B half 0, b1 takes its half 1
    // and then the next step's half 0.  pa1, pa2, pb2: the operands' bases of
    // steps t + 1 and t + 2, used if those lie wholly inside K.
    const uint8_t *pa1 = sa.p + sa.advance, *pb2 = sb.p + 2 * sb.advance;
    auto step = [&](int t, int buf, uint4(&b0)[1][4], uint4(&b1)[1][4], auto whole) {
        const uint8_t* cur = lds + buf * kNext;
        const uint8_t* nxt = lds + (buf ^ 1) * kNext;
        const uint32_t fill = base + buf * kNext, other = base + (buf ^ 1) * kNext;
        const uint8_t* pa2 = pa1 + sa.advance;
        if (rows0) fa.read(a, cur + kA0);
        if constexpr (whole.value) sa.fetch(1, pa1, other + kA1);
        else sa.fetch_checked(1, t + 1, other + kA1);
        between();
        multiply(acc[0][0], b0, rows0 && cols0);
        fb.read(b1, cur + kB1);
        if constexpr (whole.value) sb.fetch(0, pb2, fill + kB0);
        else sb.fetch_checked(0, t + 2, fill + kB0);
        between();
        multiply(acc[0][1], b1, rows0 && cols1);
        if (rows1) fa.read(a, cur + kA1);
        if constexpr (whole.value) sa.fetch(0, pa2, fill + kA0);
        else sa.fetch_checked(0, t + 2, fill + kA0);
        between();
        multiply(acc[1][1], b1, rows1 && cols1);
        fb.read(b1, nxt + kB0);
        if constexpr (whole.value) sb.fetch(1, pb2, fill + kB1);
        else sb.fetch_checked(1, t + 2, fill + kB1);
        between();
        multiply(acc[1][0], b0, rows1 && cols0);
        pa1 = pa2;
        pb2 += sb.advance;
    };
    const int whole = min(sa.whole(), sb.whole());
    int t = 0;
    for (; t + 3 < whole; t += 2) {
        step(t, 0, b[0], b[1], std::true_type());
        step(t + 1, 1, b[1], b[0], std::true_type());
    }
    for (; t < steps; t += 2) {
        step(t, 0, b[0], b[1], std::false_type());
        if (t + 1 < steps) step(t + 1, 1, b[1], b[0], std::false_type());
    }
    if (wm == 0) barrier();
    wait_dma<0>();
    barrier();  // nothing is on its way into LDS or being read any more
}

// ---------------------------------------------------------------------------
// Fewer tiles than compute units: a workgroup of 4 waves computes 128 x 128
// outputs, with the same places in LDS.  Four buffers of 32 KB hold steps t
// to t + 3, because a tile that has a compute unit to itself waits for memory
// (a step's latency is 1.0 to 1.4 us, its MFMAs take 0.25): the DMA of step
// t + 4 starts when every wave's reads of step t have come back.  Wave
// (wm, wn) of 2 x 2 owns 64 x 64; it reads the fragments of the next step
// while it multiplies those of this one.  0.47 us a step (int8, 64 x 5120 x
// 5120: 20.6 us, by 256 x 256 tiles 25.4).
// ---------------------------------------------------------------------------
template <class Acc, bool kTA, bool kTB>
__device__ __forceinline__ void mid_tile(const View& A, const View& B, int64_t m0, int64_t n0, int64_t Ka, int64_t Kb,
                                         int64_t mend, int steps, uint8_t* lds, Acc (&acc)[2][2])
{
    const int wave = wave_id(), wm = wave >> 1, wn = wave & 1;
    Source<kTA, 256, 1> sa;
    Source<kTB, 256, 1> sb;
    sa.set(A, m0, Ka, true);
    sb.set(B, n0, Kb, true);
    const bool used = m0 + 64 * wm < mend && n0 + 64 * wn < B.rows;
    const Fragments<kTA, 2> fa(2 * wm);
    const Fragments<kTB, 2> fb(2 * wn);
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    constexpr int kB = 4 * kHalfBytes;  // B's buffers lie behind A's
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        sa.fetch_checked(0, t, base + t * kHalfBytes);
        sb.fetch_checked(0, t, base + t * kHalfBytes + kB);
    }
    uint4 a[2][2][4], b[2][2][4];
    wait_dma<24>();
    barrier();
    if (used) {
        fa.read(a[0], lds);
        fb.read(b[0], lds + kB);
    }
    const uint8_t *pa = sa.p + 4 * sa.advance, *pb = sb.p + 4 * sb.advance;  // the operands' bases of step t + 4
    // buf: t % 4
    auto step = [&](int t, int buf, auto whole) {
        wait_lds();
        wait_dma<16>();  // all but steps t + 2 and t + 3
        barrier();
        const int cur = buf & 1, next = ((buf + 1) & 3) * kHalfBytes, fill = buf * kHalfBytes;
        if (used) {
            fa.read(a[cur ^ 1], lds + next);
            fb.read(b[cur ^ 1], lds + next + kB);
        }
        auto multiply = [&](int s) {
            if (!used) return;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[j][i] = mma(b[cur][j][s], a[cur][i][s], acc[j][i]);
        };
        multiply(0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (whole.value) sa.fetch(0, pa, base + fill);
        else sa.fetch_checked(0, t + 4, base + fill);
        multiply(1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (whole.value) sb.fetch(0, pb, base + fill + kB);
        else sb.fetch_checked(0, t + 4, base + fill + kB);
        multiply(2);
        multiply(3);
        pa += sa.advance;
        pb += sb.advance;
    };
    const int whole = min(sa.whole(), sb.whole());
    int t = 0;
    for (; t + 7 < whole; t += 4) {
        step(t, 0, std::true_type());
        step(t + 1, 1, std::true_type());
        step(t + 2, 2, std::true_type());
        step(t + 3, 3, std::true_type());
    }
    for (; t < steps; t += 4) {
        step(t, 0, std::false_type());
        if (t + 1 < steps) step(t + 1, 1, std::false_type());
        if (t + 2 < steps) step(t + 2, 2, std::false_type());
        if (t + 3 < steps) step(t + 3, 3, std::false_type());
    }
    wait_lds();
    wait_dma<0>();
    barrier();  // nothing is on its way into LDS or being read any more
}

// The 128 x 256 products of a 256 x 256 tile of which no more rows are
// wanted: the same loop with the 8 waves of the big tile, 2 x 4 of 64 x 64
// outputs each, and three buffers of 48 KB.  0.72 us a step, 1.15 for the whole
// tile (int8, 777 x 5120 x 5120, 80 tiles as halves: 36.3 us back to back,
// 37.2 behind its quantiser).
template <class Acc, bool kTA, bool kTB>
__device__ __forceinline__ void wide_tile(const View& A, const View& B, int64_t m0, int64_t n0, int64_t Ka, int64_t Kb,
                                          int64_t mend, int steps, uint8_t* lds, Acc (&acc)[2][2])
{
    const int wave = wave_id(), wm = wave >> 2, wn = wave & 3;
    Source<kTA, 512, 1> sa;
    Source<kTB, 512, 2> sb;
    sa.set(A, m0, Ka, true);
    sb.set(B, n0, Kb, n0 + 128 < B.rows);
    const bool used = m0 + 64 * wm < mend && n0 + 64 * wn < B.rows;
    const Fragments<kTA, 2> fa(2 * wm);
    const Fragments<kTB, 2> fb(2 * (wn & 1));
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
    constexpr int kBuf = 3 * kHalfBytes, kB = kHalfBytes;  // a buffer: A, then B's halves
    const int b_half = kB + (wn >> 1) * kHalfBytes;        // the wave's columns
#pragma unroll
    for (int t = 0; t < 3; ++t) {
        sa.fetch_checked(0, t, base + t * kBuf);
        sb.fetch_checked(0, t, base + t * kBuf + kB);
        sb.fetch_checked(1, t, base + t * kBuf + kB + kHalfBytes);
    }
    uint4 a[2][2][4], b[2][2][4];
    wait_dma<12>();
    barrier();
    if (used) {
        fa.read(a[0], lds);
        fb.read(b[0], lds + b_half);
    }
    const uint8_t *pa = sa.p + 3 * sa.advance, *pb = sb.p + 3 * sb.advance;  // the operands' bases of step t + 3
    int buf = 0;                                                             // the buffer of step t
    auto step = [&](int t, auto parity, auto whole) {
        constexpr int cur = parity.value;
        wait_lds();
        wait_dma<6>();  // all but step t + 2
        barrier();
        const int next = buf == 2 * kBuf ? 0 : buf + kBuf;
        if (used) {
            fa.read(a[cur ^ 1], lds + next);
            fb.read(b[cur ^ 1], lds + next + b_half);
        }
        auto multiply = [&](int s) {
            if (!used) return;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[j][i] = mma(b[cur][j][s], a[cur][i][s], acc[j][i]);
        };
        multiply(0);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (whole.value) sa.fetch(0, pa, base + buf);
        else sa.fetch_checked(0, t + 3, base + buf);
        multiply(1);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (whole.value) {
            sb.fetch(0, pb, base + buf + kB);
            sb.fetch(1, pb, base + buf + kB + kHalfBytes);
        } else {
            sb.fetch_checked(0, t + 3, base + buf + kB);
            sb.fetch_checked(1, t + 3, base + buf + kB + kHalfBytes);
        }
        multiply(2);
        multiply(3);
        pa += sa.advance;
        pb += sb.advance;
        buf = next;
    };
    typedef std::integral_constant<int, 0> Even;
    typedef std::integral_constant<int, 1> Odd;
    const int whole = min(sa.whole(), sb.whole());
    int t = 0;
    for (; t + 4 < whole; t += 2) {
        step(t, Even(), std::true_type());
        step(t + 1, Odd(), std::true_type());
    }
    for (; t < steps; t += 2) {
        step(t, Even(), std::false_type());
        if (t + 1 < steps) step(t + 1, Odd(), std::false_type());
    }
    wait_lds();
    wait_dma<0>();
    barrier();  // nothing is on its way into LDS or being read any more
}

template <bool kStream>
__device__ __forceinline__ void store16(void* d, uint4 v, bool stream)
{
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    if (kStream && stream)
        __builtin_nontemporal_store(u32x4_t{v.x, v.y, v.z, v.w}, static_cast<u32x4_t*>(d));
    else
        *static_cast<uint4*>(d) = v;
}

// 64 x 64 outputs of a wave: rows row0 .., columns col[0] .. + 31 and
// col[1] .. + 31; value(i, k, e): accumulator e of row tile i and column tile
// k as a float.  The wave stages 64 rows of 128 bytes in its own 8 KB of LDS
// (16-byte piece c of row r at c ^ r % 8, and the 8-byte halves of the bf16
// pieces of every other 8 rows exchanged: the writes, a row per lane, then
// meet no bank twice within the 128 bytes that the LDS takes at a time) and
// stores 8 row pieces of 128 bytes at a time.
template <bool kF32, bool kStream, class Value>
__device__ __forceinline__ void store_wave(uint8_t* stage, int64_t row0, const int64_t (&col)[2], int64_t mend, int64_t N,
                                           void* c, int64_t c_at, int64_t ldc, const Value& value)
{
    const int lane = threadIdx.x & 63, g = lane >> 5;
    const bool wide = (reinterpret_cast<uintptr_t>(c) & 15) == 0 && (kF32 || ((ldc | c_at) & 7) == 0);
    const bool stream = kStream && ((reinterpret_cast<uintptr_t>(c) | (c_at | ldc) * (kF32 ? 4 : 2)) & 127) == 0;
    constexpr int kUnits = kF32 ? 2 : 1;  // stagings for the 64 columns
    if (row0 >= mend) return;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = 32 * i + (lane & 31);
#pragma unroll
            for (int k = kF32 ? u : 0; k < (kF32 ? u + 1 : 2); ++k)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[j] = value(i, k, 4 * q + j);
                    uint8_t* row = stage + 128 * r;
                    if constexpr (kF32)
                        *reinterpret_cast<float4*>(row + (((2 * q + g) ^ (r & 7)) << 4)) =
                            make_float4(y[0], y[1], y[2], y[3]);
                    else
                        *reinterpret_cast<uint2*>(row + (((4 * k + q) ^ (r & 7)) << 4) + 8 * (g ^ (r >> 3 & 1))) =
                            make_uint2(bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3]));
                }
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int it = 0; it < 8; ++it) {
            const int r = 8 * it + (lane >> 3), p = lane & 7;
            uint4 v = *reinterpret_cast<const uint4*>(stage + 128 * r + ((p ^ (r & 7)) << 4));
            if (!kF32 && (it & 1)) v = make_uint4(v.z, v.w, v.x, v.y);
            const int64_t m = row0 + r;
            const int64_t n = kF32 ? col[u] + 4 * p : (p < 4 ? col[0] : col[1]) + 8 * (p & 3);
            if (m >= mend || n >= N) continue;
            const int64_t at = c_at + m * ldc + n;
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if constexpr (kF32) {
                float* d = static_cast<float*>(c) + at;
                if (n + 4 <= N) {
                    store16<kStream>(d, v, stream);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (n + j < N) d[j] = __uint_as_float(w[j]);
                }
            } else {
                uint16_t* d = static_cast<uint16_t*>(c) + at;
                if (wide && n + 8 <= N) {
                    store16<kStream>(d, v, stream);
                } else {  // rows are 8-byte aligned at least
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (n + 4 * h + 4 <= N) {
                            *reinterpret_cast<uint2*>(d + 4 * h) = make_uint2(w[2 * h], w[2 * h + 1]);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (n + 4 * h + j < N) d[4 * h + j] = (uint16_t)(w[2 * h + (j >> 1)] >> (16 * (j & 1)));
                        }
                    }
                }
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Sums as they are.
struct Plain {
    __device__ __forceinline__ void row(int, int64_t) {}
    __device__ __forceinline__ void columns(int, int64_t, int) {}
    __device__ __forceinline__ float operator()(float v, int, int, int) const { return v; }
};

// Integer sums times the scales of their row and column.
struct Scaled {
    const float *sa, *sb;
    int64_t M, N;
    float rows[2], cols[2][16];

    __device__ __forceinline__ Scaled(const float* sa_, const float* sb_, int64_t M_, int64_t N_)
        : sa(sa_), sb(sb_), M(M_), N(N_)
    {
    }
    __device__ __forceinline__ void row(int i, int64_t m) { rows[i] = sa[min(m, M - 1)]; }
    // columns n + first + 8 (e / 4) + e % 4 of accumulators e
    __device__ __forceinline__ void columns(int k, int64_t n, int first)
    {
        const int64_t at = min(n, N - 1);
        const int last = (int)min(N - 1 - at, (int64_t)31);
#pragma unroll
        for (int e = 0; e < 16; ++e) cols[k][e] = (sb + at)[min(first + 8 * (e >> 2) + (e & 3), last)];
    }
    __device__ __forceinline__ float operator()(int v, int i, int k, int e) const
    {
        return ((float)v * rows[i]) * cols[k][e];
    }
};

// The products of one tile (kBig: 256 x 256 by 8 waves, else 128 x 128 by 4)
// and their way into memory.
template <bool kBig, class Acc, bool kTA, bool kTB, bool kF32, bool kStream, class Convert>
__device__ __forceinline__ void tile(const View& A, const View& B, int64_t m0, int64_t n0, int64_t Ka, int64_t Kb,
                                     int64_t mend, int steps, uint8_t* lds, void* c, int64_t c_at, int64_t ldc,
                                     Convert convert)
{
    const int lane = threadIdx.x & 63, wave = wave_id();
    const int wm = kBig ? wave >> 2 : wave >> 1, wn = kBig ? wave & 3 : wave & 1;
    if constexpr (kBig) {
        if (m0 + 128 < mend) {
            Acc acc[2][2][2] = {};  // [half of A][half of B][32 rows]
            if (steps > 0) big_tile<Acc, kTA, kTB>(A, B, m0, n0, Ka, Kb, mend, steps, lds, acc);
            const int64_t col[2] = {n0 + column0<kTB>(wn, 0), n0 + column0<kTB>(wn, 1)};
#pragma unroll
            for (int k = 0; k < 2; ++k) convert.columns(k, col[k], 4 * (lane >> 5));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t row0 = m0 + 128 * h + 64 * wm;
#pragma unroll
                for (int i = 0; i < 2; ++i) convert.row(i, row0 + 32 * i + (lane & 31));
                store_wave<kF32, kStream>(lds + 8192 * wave, row0, col, mend, B.rows, c, c_at, ldc,
                                          [&](int i, int k, int e) { return convert(acc[h][k][i][e], i, k, e); });
            }
            return;
        }
    }
    Acc acc[2][2] = {};  // [32 columns][32 rows]
    if (steps > 0) {
        if constexpr (kBig) wide_tile<Acc, kTA, kTB>(A, B, m0, n0, Ka, Kb, mend, steps, lds, acc);
        else mid_tile<Acc, kTA, kTB>(A, B, m0, n0, Ka, Kb, mend, steps, lds, acc);
    }
    const int64_t row0 = m0 + 64 * wm, col[2] = {n0 + 64 * wn, n0 + 64 * wn + 32};
#pragma unroll
    for (int k = 0; k < 2; ++k) convert.columns(k, col[k], 4 * (lane >> 5));
#pragma unroll
    for (int i = 0; i < 2; ++i) convert.row(i, row0 + 32 * i + (lane & 31));
    store_wave<kF32, kStream>(lds + 8192 * wave, row0, col, mend, B.rows, c, c_at, ldc,
                              [&](int i, int k, int e) { return convert(acc[k][i][e], i, k, e); });
}

// Tile `in` of a product of tm x tn tiles, walked in groups of 8 tile rows,
// column by column, so that tiles that run together share panels.
__device__ __forceinline__ void grouped_order(int in, int tm, int tn, int& m, int& n)
{
    const int group = in / (8 * tn), first = 8 * group, rows = min(8, tm - first), at = in - group * 8 * tn;
    m = first + at % rows;
    n = at / rows;
}

// Workgroups are dealt to the 8 XCDs in turn: the hw-th of `total` pieces of
// work such that each XCD gets neighbouring ones, the first total % 8 XCDs
// one more.  False: none left.  (Tile numbers have 32 bits, here and below: a
// launch has fewer than 2^30 tiles, and 64-bit divisions before the first load
// cost 0.5 to 1.5 %: dgrad of 16 experts 229.8 -> 228.7 us, int8 of 777 rows
// 42.8 -> 42.1.)
__device__ __forceinline__ bool xcd_order(uint32_t hw, uint32_t total, uint32_t& at)
{
    const uint32_t x = hw % 8, each = total / 8, more = total % 8;
    at = x * each + min(x, more) + hw / 8;
    return hw < total;
}

// The hw-th tile of `total`, and which of its row halves (-1: both).  Whole
// rounds of one tile per compute unit come first, each round dealt so that an
// XCD gets neighbouring tiles of it (dealt over all rounds at once, the XCD of
// the largest experts would finish last: 468 against 354 us for a wgrad of 16
// uneven experts, 8192 x 2560 x 5120).  If what
// remains is at most half the compute units, its tiles are done as two halves
// of 128 rows each (a step of up to 160 halves takes 0.71 us, of 256 about
// 1.0, a whole tile's 1.15 to 1.6).
template <bool kBig>
__device__ __forceinline__ bool tile_order(uint32_t hw, uint32_t total, uint32_t cus, uint32_t& at, int& half)
{
    const uint32_t rest = total % cus, full = total - rest;
    half = -1;
    if (hw < full) {
        if (!xcd_order(hw % cus, cus, at)) return false;
        at += hw - hw % cus;
        return true;
    }
    const bool split = kBig && 2 * rest <= cus;
    if (!xcd_order(hw - full, split ? 2 * rest : rest, at)) return false;
    if (split) {
        half = (int)(at & 1);
        at >>= 1;
    }
    at += full;
    return true;
}

// Columns / 16 of a thin tile, and the steps a wave has in flight.  One token
// through 5120 -> 20480 in int8: 1 and 2 22.4 us, 1 and 4 23.0, 1 and 8 25.0,
// 2 and 2 24.4 (more waves on a compute unit do more than more loads in one).
constexpr int kThinN = 1, kThinU = 2;

// One tile of a grouped product: its operands, place and steps.
struct Place {
    View A, B;
    int64_t m0, n0, mend, Ka, Kb, c_at;
    uint32_t at;
    int steps;
};

// The hw-th tile's; false: there is none.
template <bool kBig, int kPass>
__device__ __forceinline__ bool place_tile(const GroupedArgs& g, uint32_t hw, Place& t)
{
    constexpr int kTile = kBig ? 256 : 128;
    const int64_t cols = kPass == 0 ? g.N : g.K;
    const int tn = (int)((cols + kTile - 1) / kTile);
    int im, in_, half;
    if constexpr (kPass == 2) {
        const int tm = (int)((g.N + kTile - 1) / kTile);
        if (!tile_order<kBig>(hw, (uint32_t)g.E * tm * tn, g.cus, t.at, half)) return false;
        const uint32_t e = t.at / (uint32_t)(tm * tn);
        grouped_order((int)(t.at - e * (tm * tn)), tm, tn, im, in_);
        int64_t begin, end;
        expert_rows(g.ends, e, g.T, begin, end);
        t.A = View{reinterpret_cast<const uint8_t*>(g.a + begin * g.lda), 2 * g.lda, g.N};
        t.B = View{reinterpret_cast<const uint8_t*>(g.b + begin * g.ldb), 2 * g.ldb, g.K};
        t.Ka = t.Kb = end - begin;
        t.steps = (int)((end - begin + 63) / 64);
        t.c_at = e * g.c_expert;
    } else {
        Slice s;
        const auto order = [&](uint32_t total, uint32_t& tile) {
            if (!tile_order<kBig>(hw, total, g.cus, tile, half)) return false;
            t.at = tile;
            return true;
        };
        if (!find_tile<kTile>(g.ends, g.E, g.T, tn, order, s)) return false;
        grouped_order((int)s.tile, (int)((s.end - s.begin + kTile - 1) / kTile), tn, im, in_);
        const bool none = s.e >= g.E;  // rows of no expert: zeros
        t.A = View{reinterpret_cast<const uint8_t*>(g.a + s.begin * g.lda), 2 * g.lda, s.end - s.begin};
        t.B = View{reinterpret_cast<const uint8_t*>(g.b + (none ? 0 : s.e) * g.b_expert), 2 * g.ldb, cols};
        const int64_t K = none ? 0 : kPass == 0 ? g.K : g.N;
        t.Ka = 2 * K;
        t.Kb = kPass == 0 ? 2 * K : K;
        t.steps = (int)((K + 63) / 64);
        t.c_at = s.begin * g.ldc;
    }
    t.m0 = (int64_t)kTile * im + (half == 1 ? 128 : 0);
    t.n0 = (int64_t)kTile * in_;
    t.mend = half >= 0 ? min(t.m0 + 128, t.A.rows) : t.A.rows;
    return t.m0 < t.mend;
}

constexpr int kPart = 128 * 128;  // floats of a partial tile

}  // namespace

template <bool kBig, int kPass, bool kF32>
__global__ __launch_bounds__(kBig ? 512 : 256, kBig ? 2 : 1) void k_grouped(GroupedArgs g)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLdsBytes];
    Place t;
    if (!place_tile<kBig, kPass>(g, blockIdx.x, t)) return;
    tile<kBig, f32x16_t, kPass == 2, kPass != 0, kF32, kPass == 2 && kF32>(t.A, t.B, t.m0, t.n0, t.Ka, t.Kb, t.mend, t.steps, lds,
                                                                   g.c, t.c_at, g.ldc, Plain());
}

// Few tiles and a long contraction: g.split workgroups per 128 x 128 tile,
// each over an equal run of the tile's steps, leave fp32 partial tiles in the
// workspace; k_grouped_join adds them in order.  (Whole -> split, us: wgrad of
// 16384 tokens and one expert of 1280 x 1280, 100 tiles, 123 -> 75, of 4096
// and 512 x 512 34.7 -> 24.0; dgrad of 300 tokens, 1280 of 5120, 42.4 -> 21.0;
// fprop of 128 tokens, 1024 of 4096, 32.7 -> 16.9.  The partial tiles are 64 KB
// each way for 4 steps of 32 KB or more.)
template <int kPass>
__global__ __launch_bounds__(256, 1) void k_grouped_part(GroupedArgs g)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLdsBytes];
    Place t;
    if (!place_tile<false, kPass>(g, blockIdx.x / g.split, t)) return;
    const int part = blockIdx.x % g.split;
    const int first = (int)((int64_t)t.steps * part / g.split), last = (int)((int64_t)t.steps * (part + 1) / g.split);
    // a step is 128 bytes of a row, or 64 k rows
    const auto cut = [&](View& v, int64_t& K, bool k_rows) {
        const int64_t unit = k_rows ? 64 : 128;
        v.p += k_rows ? first * unit * v.ld : first * unit;
        K = min(K, last * unit) - first * unit;
    };
    cut(t.A, t.Ka, kPass == 2);
    cut(t.B, t.Kb, kPass != 0);
    tile<false, f32x16_t, kPass == 2, kPass != 0, true, false>(t.A, t.B, t.m0, t.n0, t.Ka, t.Kb, t.mend, last - first, lds,
                                                               g.ws, (t.at * g.split + part) * kPart - t.m0 * 128 - t.n0,
                                                               128, Plain());
}

constexpr int kJoinRows = 8;  // rows of a tile that one workgroup joins

template <int kPass, bool kF32>
__global__ __launch_bounds__(256) void k_grouped_join(GroupedArgs g)
{
    Place t;
    if (!place_tile<false, kPass>(g, blockIdx.x / (128 / kJoinRows), t)) return;
    const int r = blockIdx.x % (128 / kJoinRows) * kJoinRows + (threadIdx.x >> 5), c = 4 * (threadIdx.x & 31);
    const int64_t m = t.m0 + r, n = t.n0 + c;
    if (m >= t.mend || n >= t.B.rows) return;
    const float* part = g.ws + t.at * g.split * kPart + r * 128 + c;
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < g.split; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)i * kPart);
        y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
    }
    store_cols<kF32>(g.c, t.c_at + m * g.ldc + n, n, t.B.rows, y);
}

template <bool kBig, bool kF32>
__global__ __launch_bounds__(kBig ? 512 : 256, kBig ? 2 : 1) void k_i8(
    const int8_t* __restrict__ a, int64_t lda, const float* __restrict__ sa, const int8_t* __restrict__ b, int64_t ldb,
    const float* __restrict__ sb, int64_t M, int64_t N, int64_t K, void* __restrict__ c, int64_t ldc, int cus)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLdsBytes];
    constexpr int kTile = kBig ? 256 : 128;
    const int tm = (int)((M + kTile - 1) / kTile), tn = (int)((N + kTile - 1) / kTile);
    uint32_t at;
    int im, in_, half;
    if (!tile_order<kBig>(blockIdx.x, (uint32_t)tm * tn, cus, at, half)) return;
    grouped_order((int)at, tm, tn, im, in_);
    const View A{reinterpret_cast<const uint8_t*>(a), lda, M}, B{reinterpret_cast<const uint8_t*>(b), ldb, N};
    const int64_t m0 = (int64_t)kTile * im + (half == 1 ? 128 : 0), n0 = (int64_t)kTile * in_;
    const int64_t mend = half >= 0 ? min(m0 + 128, M) : M;
    if (m0 >= mend) return;
    tile<kBig, i32x16_t, false, false, kF32, false>(A, B, m0, n0, K, K, mend, (int)((K + 127) / 128), lds, c, 0, ldc,
                                                    Scaled(sa, sb, M, N));
}

// fprop
template <int kM, bool kF32>
__global__ __launch_bounds__(256) void k_grouped_thin(GroupedArgs g)
{
    __shared__ f32x4_t lds[4 * kM * kThinN * 64];
    const int64_t tn = (g.N + 16 * kThinN - 1) / (16 * kThinN);
    Slice s;
    const auto order = [&](uint32_t total, uint32_t& at) { return xcd_order(blockIdx.x, total, at); };
    if (!find_tile<16 * kM>(g.ends, g.E, g.T, (int)tn, order, s)) return;
    const bool none = s.e >= g.E;  // rows of no expert: zeros
    const View A{reinterpret_cast<const uint8_t*>(g.a + s.begin * g.lda), 2 * g.lda, s.end - s.begin};
    const View B{reinterpret_cast<const uint8_t*>(g.b + (none ? 0 : s.e) * g.b_expert), 2 * g.ldb, g.N};
    const int64_t c_at = s.begin * g.ldc;
    // the row tiles of the same columns lie side by side: they share the weights
    const int tm = (int)((s.end - s.begin + 16 * kM - 1) / (16 * kM));
    thin_tile<f32x4_t, kM, kThinN, kThinU>(
        A, B, none ? 0 : 2 * g.K, s.tile % tm * 16 * kM, s.tile / tm * 16 * kThinN, lds,
        [&](int64_t m, int64_t n, f32x4_t v) {
            const float y[4] = {v[0], v[1], v[2], v[3]};
            store_cols<kF32>(g.c, c_at + m * g.ldc + n, n, g.N, y);
        });
}

template <int kM, bool kF32>
__global__ __launch_bounds__(256) void k_i8_thin(const int8_t* __restrict__ a, int64_t lda, const float* __restrict__ sa,
                                                 const int8_t* __restrict__ b, int64_t ldb, const float* __restrict__ sb,
                                                 int64_t M, int64_t N, int64_t K, void* __restrict__ c, int64_t ldc)
{
    __shared__ f32x4_t lds[4 * kM * kThinN * 64];
    const int64_t tm = (M + 16 * kM - 1) / (16 * kM);
    const View A{reinterpret_cast<const uint8_t*>(a), lda, M}, B{reinterpret_cast<const uint8_t*>(b), ldb, N};
    thin_tile<i32x4_t, kM, kThinN, kThinU>(
        A, B, K, blockIdx.x % tm * 16 * kM, blockIdx.x / tm * 16 * kThinN, lds, [&](int64_t m, int64_t n, i32x4_t v) {
            const float s = sa[m];
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = ((float)v[j] * s) * sb[min(n + j, N - 1)];
            store_cols<kF32>(c, m * ldc + n, n, N, y);
        });
}

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

enum class Tiles { kThin, kMid, kBig };

// The kernel that takes the least time, by what each was measured to take (us
// on 256 compute units, int8 and bf16 alike):
//   thin  6 and its traffic from the caches at 8.5 TB/s (`traffic` bytes; none: 0)
//   mid   1.5, and 4 and 0.47 per step for each round of its tiles
//   big   1.5, and 9 and 1.15 per step for each round (7 and 0.72 to 1.0 in a
//         last round of halves)
// For example int8 (products alone, back to back), N = K = 5120: 16 rows 10.9 /
// 19.9 / 24.0, 64 rows 24.4 / 20.6 / 25.4 (where thin is taken: the estimate is
// 3 us short of its time), 777 rows - / 44.6 / 36.3, 2048 rows - / 71.6 / 53.7;
// N = 1024, K = 2048, 256 rows 6.6 / 12.0 / 17.5.
// thin_grid, mid_grid: their workgroups; a grid holds fewer than 2^32 threads.
Tiles choose(double traffic, int64_t thin_grid, double mid, int64_t mid_grid, double big, double steps, int cus,
             double* time = nullptr)
{
    constexpr int64_t most = int64_t(1) << 24;  // workgroups of 256 threads
    const double thin = traffic > 0 && thin_grid < most ? 6.0 + traffic / 8.5e6 : 1e30;
    const double m = mid_grid < most ? 1.5 + std::ceil(mid / cus) * (4.0 + 0.47 * steps) : 1e30;
    const double whole = std::floor(big / cus), rest = big - whole * cus;
    const double b = 1.5 + whole * (9.0 + 1.15 * steps) +
                     (rest == 0 ? 0.0 : 2 * rest <= cus ? 7.0 + (8 * rest <= 3 * cus ? 0.72 : 1.0) * steps : 9.0 + 1.15 * steps);
    if (time) *time = std::min(thin, std::min(m, b));
    return thin <= m && thin <= b ? Tiles::kThin : m <= b ? Tiles::kMid : Tiles::kBig;
}

template <bool kBig, bool kF32>
void launch_i8_tiles(const int8_t* a, int64_t lda, const float* sa, const int8_t* b, int64_t ldb, const float* sb,
                     int64_t M, int64_t N, int64_t K, void* c, int64_t ldc, int cus, hipStream_t s)
{
    const int64_t t = kBig ? 256 : 128, tiles = ceil_div(M, t) * ceil_div(N, t);
    const dim3 grid((uint32_t)(tiles + (kBig ? cus : 0)));  // the remainder may be done in halves
    hipLaunchKernelGGL((k_i8<kBig, kF32>), grid, dim3(kBig ? 512 : 256), 0, s, a, lda, sa, b, ldb, sb, M, N, K, c, ldc,
                       cus);
}

// Workgroups of a grouped launch: every expert, and the rows of none, can
// have one partial row tile.
template <int kPass>
int64_t grouped_grid(const GroupedArgs& g, int64_t row_tile, int64_t col_tile)
{
    const int64_t rows = kPass == 2 ? g.E * ceil_div(g.N, row_tile) : g.T / row_tile + g.E + 1;
    return rows * ceil_div(kPass == 0 ? g.N : g.K, col_tile);
}

template <bool kBig, int kPass>
void launch_grouped_tiles(const GroupedArgs& g, bool out_fp32, hipStream_t s)
{
    const int64_t t = kBig ? 256 : 128;
    const dim3 grid((uint32_t)(grouped_grid<kPass>(g, t, t) + (kBig ? g.cus : 0)));  // (halves of the remainder)
    if (out_fp32)
        hipLaunchKernelGGL((k_grouped<kBig, kPass, true>), grid, dim3(kBig ? 512 : 256), 0, s, g);
    else
        hipLaunchKernelGGL((k_grouped<kBig, kPass, false>), grid, dim3(kBig ? 512 : 256), 0, s, g);
}

// Row tiles of a thin product of about `rows` rows: 16, 32 or 64.  (int8,
// N = K = 5120, us with 16 / 32 / 64: one row 7.5 / 8.6 / 11.0, 16 rows 10.8 /
// 12.1 / 14.4, 24 rows 15.9 / 13.7 / 16.1, 33 rows 18.6 / 22.3 / 17.8, 48 rows
// 20.4 / 22.3 / 21.0.)  A grouped product takes the mean load for it, since the
// host does not see the routing: 256 rows of one expert, 5120 -> 2560, take
// 24.6 us alone and 41.7 among 64 experts.
int thin_rows(double rows) { return rows <= 16.0 ? 1 : rows <= 32.0 ? 2 : 4; }

template <int kM>
void launch_grouped_thin(const GroupedArgs& g, bool out_fp32, hipStream_t s)
{
    const dim3 grid((uint32_t)grouped_grid<0>(g, 16 * kM, 16 * kThinN));
    if (out_fp32)
        hipLaunchKernelGGL((k_grouped_thin<kM, true>), grid, dim3(256), 0, s, g);
    else
        hipLaunchKernelGGL((k_grouped_thin<kM, false>), grid, dim3(256), 0, s, g);
}

template <int kM>
void launch_i8_thin(const int8_t* a, int64_t lda, const float* sa, const int8_t* b, int64_t ldb, const float* sb,
                    int64_t M, int64_t N, int64_t K, void* c, int64_t ldc, bool out_fp32, hipStream_t s)
{
    const dim3 grid((uint32_t)(ceil_div(M, 16 * kM) * ceil_div(N, 16 * kThinN)));
    if (out_fp32)
        hipLaunchKernelGGL((k_i8_thin<kM, true>), grid, dim3(256), 0, s, a, lda, sa, b, ldb, sb, M, N, K, c, ldc);
    else
        hipLaunchKernelGGL((k_i8_thin<kM, false>), grid, dim3(256), 0, s, a, lda, sa, b, ldb, sb, M, N, K, c, ldc);
}

// How a grouped product is done: its kernel, the rows / 16 of a thin tile, and
// in how many parts the contraction is taken (1: whole).
struct Plan {
    Tiles tiles;
    int m, split;
};

template <int kPass>
Plan plan_grouped(const GroupedArgs& g)
{
    const int64_t cols = kPass == 0 ? g.N : g.K;
    const double T = (double)g.T, experts = (double)std::max<int64_t>(1, std::min(g.E, g.T)), each = T / experts;
    const int m = thin_rows(each);
    // row tiles of t rows: half of an expert's last one is taken as empty
    const auto row_tiles = [&](double t) {
        return kPass == 2 ? (double)(g.E * ceil_div(g.N, (int64_t)t)) : std::max(experts, T / t + experts / 2);
    };
    const auto tiles = [&](int64_t t) { return row_tiles((double)t) * ceil_div(cols, t); };
    const double K = kPass == 0 ? (double)g.K : kPass == 1 ? (double)g.N : each, steps = std::ceil(K / 64);
    // (thin: not below 2.4 ns per element of the contraction at 64 rows, its
    // loads' latency; a workgroup takes the whole of it)
    const double traffic =
        kPass == 0 ? std::max(row_tiles(16.0 * m) * ceil_div(cols, 16) * (std::min(each, 16.0 * m) + 16) * 2,
                              0.6e-3 * 8.5e6 * m) * K : 0.0;
    const int64_t grid = grouped_grid<kPass>(g, 128, 128);
    double time;
    const Tiles t = choose(traffic, grouped_grid<kPass>(g, 16 * m, 16 * kThinN), tiles(128), grid, tiles(256), steps, g.cus,
                           &time);
    // parts of 4 steps at least, a compute unit for each; 7 us to join them
    const int split = (int)std::min(std::min(32.0, std::floor((double)g.cus / grid)), std::floor(steps / 4));
    if (split > 1 && 1.5 + 4.0 + 0.47 * std::ceil(steps / split) + 7.0 < time) return Plan{Tiles::kMid, m, split};
    return Plan{t, m, 1};
}

template <int kPass>
int64_t plan_bytes(const GroupedArgs& g)
{
    const int split = plan_grouped<kPass>(g).split;
    return split > 1 ? grouped_grid<kPass>(g, 128, 128) * split * kPart * (int64_t)sizeof(float) : 0;
}

template <int kPass>
void launch_grouped_pass(const GroupedArgs& g0, int64_t ws_bytes, bool out_fp32, hipStream_t s)
{
    GroupedArgs g = g0;
    Plan p = plan_grouped<kPass>(g);
    const int64_t grid = grouped_grid<kPass>(g, 128, 128);
    if (p.split > 1 && g.ws && ws_bytes >= plan_bytes<kPass>(g)) {
        g.split = p.split;
        hipLaunchKernelGGL(k_grouped_part<kPass>, dim3((uint32_t)(grid * p.split)), dim3(256), 0, s, g);
        const dim3 join((uint32_t)(grid * (128 / kJoinRows)));
        if (out_fp32)
            hipLaunchKernelGGL((k_grouped_join<kPass, true>), join, dim3(256), 0, s, g);
        else
            hipLaunchKernelGGL((k_grouped_join<kPass, false>), join, dim3(256), 0, s, g);
        return;
    }
    if (kPass == 0 && p.tiles == Tiles::kThin)
        return p.m == 1 ? launch_grouped_thin<1>(g, out_fp32, s)
               : p.m == 2 ? launch_grouped_thin<2>(g, out_fp32, s) : launch_grouped_thin<4>(g, out_fp32, s);
    if (p.tiles == Tiles::kBig)
        launch_grouped_tiles<true, kPass>(g, out_fp32, s);
    else
        launch_grouped_tiles<false, kPass>(g, out_fp32, s);
}

}  // namespace

int64_t grouped_workspace(int pass, const GroupedArgs& g)
{
    const int64_t rows = pass == 2 ? g.E * g.N : g.T, cols = pass == 0 ? g.N : g.K;
    if (rows == 0 || cols == 0) return 0;
    return pass == 0 ? plan_bytes<0>(g) : pass == 1 ? plan_bytes<1>(g) : plan_bytes<2>(g);
}

void launch_i8_gemm(const int8_t* a, int64_t lda, const float* sa, const int8_t* b, int64_t ldb, const float* sb,
                    int64_t M, int64_t N, int64_t K, void* c, int64_t ldc, bool out_fp32, int cus, hipStream_t s)
{
    if (M == 0 || N == 0) return;
    const int m = thin_rows((double)M);
    const double traffic =
        (double)ceil_div(M, 16 * m) * ceil_div(N, 16) * (std::min(M, (int64_t)16 * m) + 16) * std::max<int64_t>(K, 1);
    const auto tiles = [&](int64_t t) { return (double)ceil_div(M, t) * ceil_div(N, t); };
    const Tiles t = choose(traffic, ceil_div(M, 16 * m) * ceil_div(N, 16 * kThinN), tiles(128),
                           ceil_div(M, 128) * ceil_div(N, 128), tiles(256), (double)ceil_div(K, 128), cus);
    if (t == Tiles::kThin) {
        const auto thin = m == 1 ? launch_i8_thin<1> : m == 2 ? launch_i8_thin<2> : launch_i8_thin<4>;
        return thin(a, lda, sa, b, ldb, sb, M, N, K, c, ldc, out_fp32, s);
    }
    const bool big = t == Tiles::kBig;
    const auto launch = big ? (out_fp32 ? launch_i8_tiles<true, true> : launch_i8_tiles<true, false>)
                            : (out_fp32 ? launch_i8_tiles<false, true> : launch_i8_tiles<false, false>);
    launch(a, lda, sa, b, ldb, sb, M, N, K, c, ldc, cus, s);
}

void launch_grouped(int pass, const GroupedArgs& g, int64_t ws_bytes, bool out_fp32, hipStream_t s)
{
    const int64_t rows = pass == 2 ? g.E * g.N : g.T, cols = pass == 0 ? g.N : g.K;
    if (rows == 0 || cols == 0) return;  // (an empty contraction still writes zeros)
    if (pass == 0) launch_grouped_pass<0>(g, ws_bytes, out_fp32, s);
    else if (pass == 1) launch_grouped_pass<1>(g, ws_bytes, out_fp32, s);
    else launch_grouped_pass<2>(g, ws_bytes, out_fp32, s);
}

}  // namespace nvfp4
