// norm.hip -- root-mean-square norm of rows with the residual's addition.
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   int8: scale = max|y| / 127, code = rint(127 y / max|y|), ties to even
//   backward, u = dy w:  dx = rstd (u - h rstd^2 mean(u h)) + dh,
//                        dw = sum over rows of dy h rstd
// h is written rounded to its type and normalised unrounded, in fp32; an int8
// code is rounded from the unrounded y.  A row whose largest |y| is not finite
// keeps that as its scale, and its codes are 0.
//
// Bound by the bytes of x, r, h and y (backward dy, h, dh, dx): a row is read
// once and stays in registers between its sum and its outputs.  8192 x 5120 in bf16
// (336 MB): forward 59 to 62 us, int8 58 to 60, backward 65 and 4 for dw's second
// launch; a copy of as many bytes 65.6.
#include <algorithm>

#include "internal.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

constexpr int64_t kMostBlocks = int64_t(1) << 21;  // of a launch (a grid has fewer than 2^32 threads); each takes more rows beyond that
constexpr int kHeld = 2;                           // pieces of 8 columns that a lane keeps

__device__ __forceinline__ Piece sum_of(const NormArgs& a, int64_t row, int64_t c)
{
    const RawPiece x = load_raw(a.x, row * a.ld_x + c, a.x_f32);
    Piece h = widen(x, a.x_f32);
    if (a.residual) {
        const Piece r = load_piece(a.residual, row * a.ld_r + c, a.s_f32);
#pragma unroll
        for (int e = 0; e < 8; ++e) h.v[e] += r.v[e];
    }
    return h;
}

// h rstd w in place; the largest |y| so far.
__device__ __forceinline__ void scale_piece(const NormArgs& a, int64_t c, float rstd, Piece& h, float& top)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) h.v[e] *= rstd;
    if (a.weight) {
        const Piece w = load_piece(a.weight, c, a.w_f32);
#pragma unroll
        for (int e = 0; e < 8; ++e) h.v[e] *= w.v[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(h.v[e]) & 0x7FFFFFFFu));
}

// Codes of 8 values; the instruction takes NaN as 0.
__device__ __forceinline__ uint2 codes_of(const Piece& y, float lift, float factor)
{
    uint32_t o[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        uint32_t code;
        asm("v_cvt_i32_f32 %0, %1" : "=v"(code) : "v"(__builtin_rintf(y.v[e] * lift * factor)));
        o[e >> 2] |= (code & 0xFFu) << (8 * (e & 3));
    }
    return make_uint2(o[0], o[1]);
}

}  // namespace

// kLanes 16 or 32: so many lanes a row (of up to 128 or 256 columns), 256 / kLanes
// rows a workgroup.  0: a workgroup a row, as many waves as its columns fill (16 at most).
// (65536 x 128, a head's norm: 16 lanes a row 13 us, 32 14.6, a wave 28; 32768 x 256:
// 32 lanes 13, a wave 16; 16384 x 512: a wave a workgroup 12.5, four in one 12.7.)
template <int kLanes, bool kI8>
__global__ __launch_bounds__(kLanes ? 256 : 1024) void k_norm(NormArgs a)
{
    constexpr bool kSolo = kLanes > 0;
    constexpr int kHeld = kSolo ? 1 : nvfp4::kHeld, kRows = kSolo ? 256 / kLanes : 1;
    __shared__ float part[2][16];
    const int lanes = kSolo ? kLanes : blockDim.x, lane = kSolo ? threadIdx.x & (kLanes - 1) : threadIdx.x;
    const int wave = wave_index(), waves = lanes / 64;
    const float each = 1.0f / (float)a.cols;
    // (all lanes go through the lane moves: rows beyond the last one are its copies, not written)
    const int64_t rows = kSolo ? (a.rows + kRows - 1) / kRows * kRows : a.rows;
    for (int64_t at = kSolo ? (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes : blockIdx.x; at < rows;
         at += (int64_t)gridDim.x * kRows) {
        const bool live = at < a.rows;
        const int64_t row = live ? at : a.rows - 1;
        Piece h[kHeld];
        float sum = 0.0f;
        const auto square = [&](const Piece& p) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(p.v[e], p.v[e], sum);
        };
        {
            RawPiece x[kHeld], r[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int64_t c = 8 * (lane + (int64_t)lanes * i);
                x[i] = r[i] = RawPiece{};
                if (c < a.cols) {
                    x[i] = load_raw(a.x, row * a.ld_x + c, a.x_f32);
                    if (a.residual) r[i] = load_raw(a.residual, row * a.ld_r + c, a.s_f32);
                }
            }
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int64_t c = 8 * (lane + (int64_t)lanes * i);
                h[i] = widen(x[i], a.x_f32);
                const Piece d = widen(r[i], a.s_f32);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i].v[e] += d.v[e];
                square(h[i]);
                if (a.h && c < a.cols && live) store_piece(a.h, row * a.ld_h + c, h[i], a.s_f32);
            }
        }
        const int64_t rest = 8 * (lane + (int64_t)lanes * kHeld);  // what is not kept is read again
        for (int64_t c = rest; c < a.cols; c += 8 * lanes) square(sum_of(a, row, c));
        sum = group_sum<kSolo ? kLanes : 64>(sum);
        if constexpr (!kSolo) {
            if ((threadIdx.x & 63) == 0) part[0][wave] = sum;
            __syncthreads();
            sum = part[0][0];
            for (int v = 1; v < waves; ++v) sum += part[0][v];
        }
        const float rstd = 1.0f / __builtin_sqrtf(sum * each + a.eps);
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int64_t c = 8 * (lane + (int64_t)lanes * i);
            if (c >= a.cols) continue;
            scale_piece(a, c, rstd, h[i], top);
            if (a.y && live) store_piece(a.y, row * a.ld_y + c, h[i], false);
        }
        for (int64_t c = rest; c < a.cols; c += 8 * lanes) {
            Piece p = sum_of(a, row, c);
            if (a.h && !kI8) store_piece(a.h, row * a.ld_h + c, p, a.s_f32);  // (h may lie where r does)
            scale_piece(a, c, rstd, p, top);
            if (a.y) store_piece(a.y, row * a.ld_y + c, p, false);
        }
        if constexpr (kI8) {
            top = group_top<kSolo ? kLanes : 64>(top);
            if constexpr (!kSolo) {
                if ((threadIdx.x & 63) == 0) part[1][wave] = top;
                __syncthreads();
                uint32_t most = 0;
                for (int v = 0; v < waves; ++v) most = max(most, __float_as_uint(part[1][v]));
                top = __uint_as_float(most);
            }
            if (lane == 0 && live) a.scales[row] = top / 127.0f;
            // a power of two on both sides of the quotient keeps 127 / max finite
            const float lift = top < 0x1p-100f ? 0x1p64f : 1.0f;
            const float factor = top > 0.0f ? 127.0f / (top * lift) : 0.0f;
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int64_t c = 8 * (lane + (int64_t)lanes * i);
                if (c < a.cols && live) *reinterpret_cast<uint2*>(a.codes + row * a.ld_codes + c) = codes_of(h[i], lift, factor);
            }
            for (int64_t c = rest; c < a.cols; c += 8 * lanes) {
                Piece p = sum_of(a, row, c);
                if (a.h) store_piece(a.h, row * a.ld_h + c, p, a.s_f32);
                scale_piece(a, c, rstd, p, top);
                *reinterpret_cast<uint2*>(a.codes + row * a.ld_codes + c) = codes_of(p, lift, factor);
            }
        } else if constexpr (!kSolo) {
            __syncthreads();  // part[0] is written again for the next row
        }
    }
}

namespace {

// How the backward pass goes through rows of `cols` columns: pieces of 8 a
// lane, waves a row, rows that a workgroup takes at a time (teams), and workgroups.
struct BackPlan {
    int lanes;  // 16 or 32: so many a row; 64: its waves'
    int held, waves, teams;
    int64_t blocks;
};

BackPlan back_plan(int64_t rows, int64_t cols, int cus)
{
    const int64_t pieces = (cols + 7) / 8;
    const int held = pieces <= 64 ? 1 : 2, lanes = pieces <= 16 ? 16 : pieces <= 32 ? 32 : 64;
    const int waves = (int)std::max<int64_t>(1, (pieces + 64 * held - 1) / (64 * held)), teams = 16 / waves * (64 / lanes);
    // up to two rows a team: one workgroup, whose sums are dweight (6 x 5120: 7.2 us, with a
    // second launch 7.9; 9 x 5120, three rows a team: 9.0 and 8.0)
    // (two or more otherwise: on a host without a device the answer is one for two units)
    const int64_t turns = (rows + teams - 1) / teams;
    return BackPlan{lanes, held, waves, teams, turns <= 2 ? std::min<int64_t>(turns, 1) : std::min<int64_t>(turns, std::max(cus, 2))};
}

}  // namespace

// A workgroup takes `teams` rows at a time, each by `waves` waves (kLanes 16 or
// 32: by so many lanes, 64 or 32 rows), and keeps its columns' sums of dy h rstd in
// registers; the teams' sums are added in LDS, in order, and the workgroups' by
// k_column_sums.  Many rows at a time keep loads in flight while others are added
// up; more than one workgroup of 16 waves on a compute unit adds more sums than it
// hides (16384 x 512: one 16.7 us, two 20.5).  8192 x 5120, us: 3 rows at a time 67
// (with the sums' kernel), one 79, one with the next's loads in flight 80 to 85.
// One piece a lane up to 512 columns (1000 x 512: 8.5, two a lane and half the teams 8.9).
template <int kBackHeld, int kLanes, bool kDyF32, bool kSF32>
__global__ __launch_bounds__(1024) void k_norm_backward(NormArgs a, int waves, int teams)
{
    __shared__ float part[2][2][16];
    __shared__ __attribute__((aligned(16))) float sums[kNormMostCols];
    const int wave = wave_index(), team = kLanes < 64 ? threadIdx.x / kLanes : wave / waves;
    const int lanes = kLanes < 64 ? kLanes : 64 * waves, lane = (int)threadIdx.x - team * lanes;
    const float each = 1.0f / (float)a.cols;
    Piece w[kBackHeld], dw[kBackHeld];
    bool in[kBackHeld];
#pragma unroll
    for (int i = 0; i < kBackHeld; ++i) {
        const int64_t c = 8 * (lane + (int64_t)lanes * i);
        in[i] = c < a.cols;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[i].v[e] = 1.0f, dw[i].v[e] = 0.0f;
        if (a.weight && in[i]) w[i] = load_piece(a.weight, c, a.w_f32);
    }
    int turn = 0;
    for (int64_t base = (int64_t)blockIdx.x * teams; base < a.rows; base += (int64_t)gridDim.x * teams, turn ^= 1) {
        const int64_t row = base + team;
        const bool live = row < a.rows;
        RawPiece dy[kBackHeld], h[kBackHeld], dh[kBackHeld];
#pragma unroll
        for (int i = 0; i < kBackHeld; ++i) {
            const int64_t c = 8 * (lane + (int64_t)lanes * i);
            dy[i] = h[i] = dh[i] = RawPiece{};
            if (in[i] && live) {
                dy[i] = load_raw(a.x, row * a.ld_x + c, kDyF32);
                h[i] = load_raw(a.h, row * a.ld_h + c, kSF32);
                if (a.residual) dh[i] = load_raw(a.residual, row * a.ld_r + c, kSF32);
            }
        }
        float squares = 0.0f, along = 0.0f;
#pragma unroll
        for (int i = 0; i < kBackHeld; ++i) {
            const Piece d = widen(dy[i], kDyF32), x = widen(h[i], kSF32);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                squares = __builtin_fmaf(x.v[e], x.v[e], squares);
                along = __builtin_fmaf(d.v[e] * w[i].v[e], x.v[e], along);
            }
        }
        squares = group_sum<kLanes>(squares);
        along = group_sum<kLanes>(along);
        if (waves > 1) {
            if ((threadIdx.x & 63) == 0) {
                part[turn][0][wave] = squares;
                part[turn][1][wave] = along;
            }
            __syncthreads();  // (the other turn's are read before the next barrier)
            squares = along = 0.0f;
            for (int v = team * waves; v < (team + 1) * waves; ++v) {
                squares += part[turn][0][v];
                along += part[turn][1][v];
            }
        }
        const float rstd = 1.0f / __builtin_sqrtf(squares * each + a.eps);
        const float mean = along * each * rstd * rstd;
        if (!live) continue;
#pragma unroll
        for (int i = 0; i < kBackHeld; ++i) {
            const int64_t c = 8 * (lane + (int64_t)lanes * i);
            const Piece d = widen(dy[i], kDyF32), x = widen(h[i], kSF32), r = widen(dh[i], kSF32);
            Piece o;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                dw[i].v[e] = __builtin_fmaf(d.v[e] * rstd, x.v[e], dw[i].v[e]);
                o.v[e] = __builtin_fmaf(rstd, __builtin_fmaf(-mean, x.v[e], d.v[e] * w[i].v[e]), r.v[e]);
            }
            if (in[i]) store_piece(a.dx, row * a.ld_dx + c, o, a.dx_f32);
        }
    }
    if (!a.dweight) return;
    if constexpr (kLanes < 64) {  // the rows of a wave: the first one's lanes get their sums
#pragma unroll
        for (int i = 0; i < kBackHeld; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (kLanes == 16) dw[i].v[e] = sum_of_halves<16>(dw[i].v[e]);
                dw[i].v[e] = sum_of_halves<32>(dw[i].v[e]);
            }
    }
    const int parts = kLanes < 64 ? 16 : teams, own = kLanes < 64 ? wave : team;
    for (int k = 0; k < parts; ++k) {
        __syncthreads();
        if (own != k || (kLanes < 64 && (threadIdx.x & 63) >= kLanes)) continue;
#pragma unroll
        for (int i = 0; i < kBackHeld; ++i) {
            const int64_t c = 8 * (lane + (int64_t)lanes * i);
            if (!in[i]) continue;
            if (k > 0) {
                const Piece before = load_piece(sums, c, true);
#pragma unroll
                for (int e = 0; e < 8; ++e) dw[i].v[e] += before.v[e];
            }
            if (k + 1 < parts) store_piece(sums, c, dw[i], true);
            else store_piece(a.parts, (int64_t)blockIdx.x * a.cols + c, dw[i], true);
        }
    }
}

// Column sums of `parts` (groups x cols) in the order of the groups: 32
// columns a workgroup, 32 runs of the groups.  (256 x 5120: 4.8 us, the launch.)
__global__ __launch_bounds__(256) void k_column_sums(const float* __restrict__ parts, int64_t groups, int64_t cols,
                                                     float* __restrict__ out)
{
    __shared__ float4 part[32][8];
    const int q = threadIdx.x & 7, s = threadIdx.x >> 3;
    const int64_t c = 32 * (int64_t)blockIdx.x + 4 * q;
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < cols)
#pragma unroll 8
        for (int64_t g = groups * s / 32, to = groups * (s + 1) / 32; g < to; ++g) {
            const float4 v = *reinterpret_cast<const float4*>(parts + g * cols + c);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
    part[s][q] = sum;
    __syncthreads();
    if (s != 0 || c >= cols) return;
    for (int j = 1; j < 32; ++j) {
        const float4 v = part[j][q];
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    *reinterpret_cast<float4*>(out + c) = sum;
}

namespace {

template <int kLanes>
void launch_norm_of(const NormArgs& a, hipStream_t s)
{
    const int64_t waves = std::min<int64_t>(16, (a.cols / 8 + 64 * kHeld - 1) / (64 * kHeld));
    const int64_t each = kLanes ? 256 / std::max(kLanes, 1) : 1, blocks = (a.rows + each - 1) / each;
    const dim3 grid((uint32_t)std::min(blocks, kMostBlocks)), block((uint32_t)(kLanes ? 256 : 64 * waves));
    if (a.scales) hipLaunchKernelGGL((k_norm<kLanes, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((k_norm<kLanes, false>), grid, block, 0, s, a);
}

}  // namespace

void launch_norm(const NormArgs& a, hipStream_t s)
{
    if (a.rows == 0) return;
    if (a.cols <= 128) launch_norm_of<16>(a, s);
    else if (a.cols <= 256) launch_norm_of<32>(a, s);
    else launch_norm_of<0>(a, s);
}

int64_t norm_backward_workspace(int64_t rows, int64_t cols, int cus)
{
    const int64_t blocks = back_plan(rows, cols, cus).blocks;
    return blocks > 1 ? blocks * cols * (int64_t)sizeof(float) : 0;
}

namespace {

template <bool kDyF32, bool kSF32>
void launch_norm_backward_of(const BackPlan& p, const NormArgs& a, hipStream_t s)
{
    const dim3 grid((uint32_t)p.blocks), block((uint32_t)(p.lanes * p.waves * p.teams));
    if (p.lanes == 16) hipLaunchKernelGGL((k_norm_backward<1, 16, kDyF32, kSF32>), grid, block, 0, s, a, p.waves, p.teams);
    else if (p.lanes == 32) hipLaunchKernelGGL((k_norm_backward<1, 32, kDyF32, kSF32>), grid, block, 0, s, a, p.waves, p.teams);
    else if (p.held == 1) hipLaunchKernelGGL((k_norm_backward<1, 64, kDyF32, kSF32>), grid, block, 0, s, a, p.waves, p.teams);
    else hipLaunchKernelGGL((k_norm_backward<2, 64, kDyF32, kSF32>), grid, block, 0, s, a, p.waves, p.teams);
}

}  // namespace

void launch_norm_backward(const NormArgs& args, hipStream_t s)
{
    NormArgs a = args;
    const BackPlan p = back_plan(a.rows, a.cols, a.cus);
    if (p.blocks == 1) a.parts = a.dweight;
    if (p.blocks > 0) {
        if (a.x_f32) {
            if (a.s_f32) launch_norm_backward_of<true, true>(p, a, s);
            else launch_norm_backward_of<true, false>(p, a, s);
        } else {
            if (a.s_f32) launch_norm_backward_of<false, true>(p, a, s);
            else launch_norm_backward_of<false, false>(p, a, s);
        }
    }
    if (a.dweight && a.cols > 0 && p.blocks != 1)  // (no rows: zeros)
        hipLaunchKernelGGL(k_column_sums, dim3((uint32_t)((a.cols + 31) / 32)), dim3(256), 0, s, a.parts, p.blocks, a.cols,
                           a.dweight);
}

}  // namespace nvfp4
