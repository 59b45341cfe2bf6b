// move_rows.hip -- tokens into the experts' order and back.
//
//   dispatch   o[rows[t, j]] = x[t]
//   combine    y[t] = r[t] + sum_j w[t, j] o[rows[t, j]]
//   backward   do[rows[t, j]] = w[t, j] dy[t],  dw[t, j] = sum_c dy[t, c] o[rows[t, j], c]
// Dispatch's backward is combine without weights.  A place outside the rows
// there are stands for a row of zeros that nobody reads.
//
// All three go token by token: a token's k places are scalar loads, its own
// row moves once, and the experts' rows are whole row pieces wherever they
// lie.  Sums run over j in order, so no atomic and no order of workgroups
// shows in a result.  Bound by the bytes of the experts' rows: 8192 tokens of 5120
// columns, 4 rows each, take 82 us to dispatch (420 MB, 5.1 TB/s), 98 to combine
// with a residual (503 MB), 155 backward (755 MB, 4.9 TB/s); a copy reaches 5.1 TB/s.
#include <algorithm>

#include "internal.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

constexpr int64_t kMostBlocks = int64_t(1) << 21;  // of a launch (a grid has fewer than 2^32 threads); each takes more tokens beyond that

__device__ __forceinline__ bool inside(int64_t place, int64_t R) { return (uint64_t)place < (uint64_t)R; }

}  // namespace

// A workgroup takes one unit of columns of four tokens, a wave each; workgroups
// that follow each other take the units of the same tokens, so that whole rows
// are in flight together.  (8192 tokens, 8 rows of 2048: combine 67 us, with all
// tokens' first unit before the second 85; dispatch 54 and 61.)
struct Turn {
    int64_t unit, token, step;
    __device__ __forceinline__ Turn(const MoveArgs& a, int width)
    {
        const uint32_t units = (uint32_t)((a.cols + width - 1) / width), first = blockIdx.x / units;
        unit = blockIdx.x - first * units;
        token = 4 * (int64_t)first + wave_index();
        step = 4 * (int64_t)(gridDim.x / units);
    }
};

// A wave moves two pieces of 16 bytes a lane.  (8192 tokens of 5120 columns to 4
// rows: 82 us, one piece 86, four 87.)
__global__ __launch_bounds__(256) void k_dispatch(MoveArgs a)
{
    constexpr int kPieces = 2;
    const Turn turn(a, 512 * kPieces);
    const int64_t c0 = 512 * kPieces * turn.unit + 8 * (threadIdx.x & 63);
    for (int64_t t = turn.token; t < a.T; t += turn.step) {
        const uint16_t* src = static_cast<const uint16_t*>(a.tokens) + t * a.ld_tokens;
        uint4 v[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int64_t c = c0 + 512 * i;
            v[i] = c < a.cols ? *reinterpret_cast<const uint4*>(src + c) : make_uint4(0, 0, 0, 0);
        }
        for (int j = 0; j < a.k; ++j) {
            const int64_t place = a.rows[t * a.k + j];
            if (!inside(place, a.R)) continue;
            uint16_t* dst = static_cast<uint16_t*>(a.out) + place * a.ld_out;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int64_t c = c0 + 512 * i;
                if (c < a.cols) *reinterpret_cast<uint4*>(dst + c) = v[i];
            }
        }
    }
}

// A wave adds up 512 columns of one token, four of its rows in flight.  (1024
// columns, or eight rows, hold more registers than they hide latency: 8192
// tokens of 4 rows of 5120 103 us, 105, 122.)
__global__ __launch_bounds__(256) void k_combine(MoveArgs a)
{
    constexpr int kAhead = 4;
    const Turn turn(a, 512);
    const int64_t c = 512 * turn.unit + 8 * (threadIdx.x & 63);
    for (int64_t t = turn.token; t < a.T; t += turn.step) {
        Piece sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += kAhead) {
            RawPiece raw[kAhead];
            float w[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const bool in = j0 + u < a.k;
                const int64_t slot = t * a.k + (in ? j0 + u : j0);
                const int64_t place = a.rows[slot];
                w[u] = !in ? 0.0f : a.weights ? a.weights[slot] : 1.0f;
                raw[u] = RawPiece{};
                if (in && inside(place, a.R) && c < a.cols) raw[u] = load_raw(a.from, place * a.ld_from + c, a.from_f32);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const Piece o = widen(raw[u], a.from_f32);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum.v[e] = __builtin_fmaf(w[u], o.v[e], sum.v[e]);
            }
        }
        if (c >= a.cols) continue;
        if (a.tokens) {
            const Piece r = load_piece(a.tokens, t * a.ld_tokens + c, a.out_f32);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum.v[e] += r.v[e];
        }
        store_piece(a.out, t * a.ld_out + c, sum, a.out_f32);
    }
}

// A token's waves hold two pieces of dy a lane while its rows pass by, four of
// them in flight; each wave adds its dot products up by lane moves, and the
// waves' are added in order.  kSolo: up to 1024 columns, a wave a token, four a
// workgroup; otherwise a workgroup a token, as many waves as its columns fill.  (16384
// tokens of 2 rows of 1024: 27.1 us, a wave a workgroup 27.4; 16384 of 4 of 768: 35.2, 36.0.
// 4001 of 6 of 2568: 58.7; one piece 65, eight rows in flight 61.)
template <bool kDyF32, bool kOF32, bool kSolo>
__global__ __launch_bounds__(kSolo ? 256 : 1024) void k_combine_backward(MoveArgs a)
{
    constexpr int kHeld = 2, kAhead = 4;
    __shared__ float part[16][kMoveMostK];
    const int lanes = kSolo ? 64 : blockDim.x, lane = kSolo ? threadIdx.x & 63 : threadIdx.x, wave = wave_index();
    const int64_t each = kSolo ? 4 : 1;
    for (int64_t t = (int64_t)blockIdx.x * each + (kSolo ? wave : 0); t < a.T; t += (int64_t)gridDim.x * each) {
        for (int64_t c0 = 0; c0 == 0 || c0 < a.cols; c0 += 8 * kHeld * lanes) {  // (one turn, but for the longest rows)
            Piece dy[kHeld];
            bool in[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; ++i) {
                const int64_t c = c0 + 8 * (lane + (int64_t)lanes * i);
                in[i] = c < a.cols;
                RawPiece r = {};
                if (in[i]) r = load_raw(a.tokens, t * a.ld_tokens + c, kDyF32);
                dy[i] = widen(r, kDyF32);
            }
            for (int j0 = 0; j0 < a.k; j0 += kAhead) {
                int64_t place[kAhead];
                RawPiece o[kAhead][kHeld];
                float w[kAhead], dot[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int64_t slot = t * a.k + min(j0 + u, a.k - 1);
                    place[u] = j0 + u < a.k ? a.rows[slot] : -1;
                    w[u] = a.weights[slot];
#pragma unroll
                    for (int i = 0; i < kHeld; ++i) {
                        o[u][i] = RawPiece{};
                        if (in[i] && inside(place[u], a.R))
                            o[u][i] = load_raw(a.from, place[u] * a.ld_from + c0 + 8 * (lane + (int64_t)lanes * i), kOF32);
                    }
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    dot[u] = 0.0f;
#pragma unroll
                    for (int i = 0; i < kHeld; ++i) {
                        const Piece v = widen(o[u][i], kOF32);
                        Piece g;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            dot[u] = __builtin_fmaf(dy[i].v[e], v.v[e], dot[u]);
                            g.v[e] = w[u] * dy[i].v[e];
                        }
                        if (in[i] && inside(place[u], a.R))
                            store_piece(a.out, place[u] * a.ld_out + c0 + 8 * (lane + (int64_t)lanes * i), g, false);
                    }
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    // (an empty slot's row of zeros: 0, whatever dy holds)
                    const float sum = inside(place[u], a.R) ? wave_sum(dot[u]) : 0.0f;
                    if ((threadIdx.x & 63) == 0 && j0 + u < a.k) part[wave][j0 + u] = c0 == 0 ? sum : part[wave][j0 + u] + sum;
                }
            }
        }
        if constexpr (kSolo) {
            __builtin_amdgcn_wave_barrier();
            if (lane < a.k) a.dweights[t * a.k + lane] = part[wave][lane];
            __builtin_amdgcn_wave_barrier();
        } else {
            __syncthreads();
            if (lane < a.k) {
                float sum = part[0][lane];
                for (int v = 1; v < (int)blockDim.x / 64; ++v) sum += part[v][lane];
                a.dweights[t * a.k + lane] = sum;
            }
            __syncthreads();  // part is written again for the next token
        }
    }
}

namespace {

void launch_turns(void (*kernel)(MoveArgs), int width, const MoveArgs& a, hipStream_t s)
{
    const int64_t units = (a.cols + width - 1) / width, blocks = std::min((a.T + 3) / 4, std::max<int64_t>(1, kMostBlocks / units));
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(blocks * units)), dim3(256), 0, s, a);
}

}  // namespace

void launch_dispatch(const MoveArgs& a, hipStream_t s) { launch_turns(k_dispatch, 1024, a, s); }

void launch_combine(const MoveArgs& a, hipStream_t s) { launch_turns(k_combine, 512, a, s); }

namespace {

template <bool kDyF32, bool kOF32>
void launch_combine_backward_of(const MoveArgs& a, hipStream_t s)
{
    const int64_t pieces = (a.cols + 7) / 8, waves = std::max<int64_t>(1, std::min<int64_t>(16, (pieces + 127) / 128));
    if (waves == 1) {
        const int64_t blocks = (a.T + 3) / 4;
        hipLaunchKernelGGL((k_combine_backward<kDyF32, kOF32, true>), dim3((uint32_t)std::min(blocks, kMostBlocks)), dim3(256),
                           0, s, a);
    } else {
        hipLaunchKernelGGL((k_combine_backward<kDyF32, kOF32, false>), dim3((uint32_t)std::min(a.T, kMostBlocks)),
                           dim3((uint32_t)(64 * waves)), 0, s, a);
    }
}

}  // namespace

void launch_combine_backward(const MoveArgs& a, hipStream_t s)
{
    const auto launch = a.tokens_f32 ? (a.from_f32 ? launch_combine_backward_of<true, true> : launch_combine_backward_of<true, false>)
                                     : (a.from_f32 ? launch_combine_backward_of<false, true> : launch_combine_backward_of<false, false>);
    launch(a, s);
}

}  // namespace nvfp4
