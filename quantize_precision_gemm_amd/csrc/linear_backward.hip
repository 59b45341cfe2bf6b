// linear_backward.hip -- gradients through the epilogue of a linear layer's
// forward product: dpre = dy act'(pre), dbias = sum of dpre over the rows (of
// each expert).
//
// Bound by the bytes of dy, pre and dpre (8192 x 5120, 252 MB: 47 to 48 us, squared ReLU;
// SiLU and GELU, 20 to 30 instructions an element, 52 and 56 with the sums).  A wave takes 512 columns of a run of
// rows and keeps their sums in registers; where the run passes from one expert
// to the next it writes them down.  Run c's sums for expert e go to line c + e
// of the workspace: going along the rows, c or e grows from one to the next,
// so no line is used twice and runs + experts lines hold them all, whatever
// the routing.  A second kernel adds an expert's lines in order.
#include <algorithm>

#include "activation.hpp"
#include "internal.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

// Rows of a run: 4096 waves where there are as many rows (of 8192 rows of 5120: 52 us,
// 2048 waves 59, 8192 53), and no run shorter than the 4 rows that a wave has in
// flight (64 rows of 5120: 9 us, 8 a run 14, 16 a run 23; each run costs 4 bytes a
// column, its rows 24).  4 rows are one run: without experts its sums are dbias.
int64_t run_rows(int64_t T, int64_t N)
{
    const int64_t units = std::max<int64_t>(1, (N + 511) / 512), runs = std::max<int64_t>(1, 4096 / units);
    return std::max<int64_t>(4, (T + runs - 1) / runs);
}

int64_t run_count(int64_t T, int64_t N) { return (T + run_rows(T, N) - 1) / run_rows(T, N); }

// The first expert from `e` on whose rows reach beyond row r (its end is then
// the largest so far, whatever the ends before hold); E: none.
__device__ __forceinline__ int64_t expert_at(const int32_t* __restrict__ ends, int64_t E, int64_t e, int64_t r)
{
    for (int64_t e0 = e; e0 < E; e0 += 64) {
        const int64_t i = e0 + (threadIdx.x & 63);
        const uint64_t past = __ballot(i < E && ends[i < E ? i : 0] > r);
        if (past) return e0 + __builtin_ctzll(past);
    }
    return E;
}

}  // namespace

template <bool kSums>
__global__ __launch_bounds__(256) void k_linear_backward(LinearBackArgs a, int64_t each)
{
    constexpr int kAhead = 4;
    const int64_t run = (int64_t)blockIdx.x * 4 + wave_index();
    const int64_t c = 512 * (int64_t)blockIdx.y + 8 * (threadIdx.x & 63);
    const bool in = c < a.N;
    int64_t r = run * each, e = 0;
    const int64_t stop = min(r + each, a.T);
    while (r < stop) {
        int64_t end = stop;
        if (a.ends) {
            e = expert_at(a.ends, a.E, e, r);
            if (e >= a.E) break;  // rows of no expert: left as they are
            end = min((int64_t)__builtin_amdgcn_readfirstlane(a.ends[e]), stop);
        }
        Piece sum;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum.v[i] = 0.0f;
        for (; r < end; r += kAhead) {
            RawPiece dy[kAhead], z[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                dy[u].a = dy[u].b = z[u].a = z[u].b = make_uint4(0, 0, 0, 0);
                if (in && r + u < end) {
                    dy[u] = load_raw(a.dy, (r + u) * a.ld_dy + c, a.dy_f32);
                    if (a.pre) z[u] = load_raw(a.pre, (r + u) * a.ld_pre + c, false);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (r + u >= end) break;
                Piece d = widen(dy[u], a.dy_f32);
                if (a.pre) {
                    const Piece p = widen(z[u], false);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d.v[i] *= activation_slope(a.act, p.v[i]);
                    if (in) store_piece(a.dpre, (r + u) * a.ld_dpre + c, d, false);
                }
                if constexpr (kSums) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum.v[i] += d.v[i];
                }
            }
        }
        r = end;
        if (kSums && in) store_piece(a.parts, (run + e) * a.N + c, sum, true);
    }
}

// dbias of one expert: its lines in order, 64 columns a workgroup, kRuns runs of
// the lines: 64 from 256 lines an expert on, else 16.  (65536 rows of 512, 4096 lines for 8
// workgroups: 54 us in all, with 16 runs 61; 777 of 5120, 195 lines: 12.9 and 12.5; 8192
// of 5120 for 8 experts, 51 lines: 62.9 and 60.7.)
template <int kRuns>
__global__ __launch_bounds__(16 * kRuns) void k_bias_sums(LinearBackArgs a, int64_t each)
{
    __shared__ float4 part[kRuns][16];
    const int q = threadIdx.x & 15, s = threadIdx.x >> 4;
    const int64_t e = blockIdx.y, c = 64 * (int64_t)blockIdx.x + 4 * q;
    int64_t begin = 0, end = a.T;
    if (a.ends) {
        int b = 0;
        for (int64_t i = threadIdx.x & 63; i < e; i += 64) b = max(b, a.ends[i]);
        b = (int)wave_max_u32((uint32_t)b);
        begin = min((int64_t)__builtin_amdgcn_readfirstlane(b), a.T);
        end = min((int64_t)__builtin_amdgcn_readfirstlane(a.ends[e]), a.T);
    }
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (end > begin && c < a.N) {
        const int64_t first = begin / each, count = (end - 1) / each - first + 1;
#pragma unroll 4
        for (int64_t i = first + count * s / kRuns, to = first + count * (s + 1) / kRuns; i < to; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(a.parts + (i + e) * a.N + c);
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
    }
    part[s][q] = sum;
    // the runs' sums: kJoin at a time, and those
    constexpr int kJoin = kRuns == 64 ? 8 : 4;
    const auto join = [&](int step) {
        __syncthreads();
        if (s % (kJoin * step)) return;
#pragma unroll
        for (int j = 1; j < kJoin; ++j) {
            const float4 v = part[s + j * step][q];
            sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
    };
    join(1);
    if (s % kJoin == 0) part[s][q] = sum;
    join(kJoin);
    if (s == 0 && c < a.N) *reinterpret_cast<float4*>(a.dbias + e * a.N + c) = sum;
}

int64_t linear_backward_workspace(int64_t E, int64_t T, int64_t N)
{
    return T == 0 || N == 0 || E == 0 ? 0 : (run_count(T, N) + E) * N * (int64_t)sizeof(float);
}

bool linear_backward_one_run(const int32_t* ends, int64_t T, int64_t N) { return !ends && T > 0 && run_count(T, N) == 1; }

void launch_linear_backward(const LinearBackArgs& args, hipStream_t s)
{
    LinearBackArgs a = args;
    if (a.N == 0) return;
    const bool whole = linear_backward_one_run(a.ends, a.T, a.N);
    if (whole) a.parts = a.dbias;
    const int64_t each = run_rows(a.T, a.N), runs = run_count(a.T, a.N);
    if (a.T > 0 && a.E > 0) {
        const dim3 grid((uint32_t)((runs + 3) / 4), (uint32_t)((a.N + 511) / 512));
        if (a.dbias) hipLaunchKernelGGL(k_linear_backward<true>, grid, dim3(256), 0, s, a, each);
        else hipLaunchKernelGGL(k_linear_backward<false>, grid, dim3(256), 0, s, a, each);
    }
    if (a.dbias && a.E > 0 && !whole) {
        const dim3 grid((uint32_t)((a.N + 63) / 64), (uint32_t)a.E);
        if (runs >= 256 * a.E) hipLaunchKernelGGL(k_bias_sums<64>, grid, dim3(1024), 0, s, a, each);
        else hipLaunchKernelGGL(k_bias_sums<16>, grid, dim3(256), 0, s, a, each);
    }
}

}  // namespace nvfp4
