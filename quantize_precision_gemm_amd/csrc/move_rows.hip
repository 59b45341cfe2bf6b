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
// shows in a result.  Bound by the bytes of the experts' rows.
#include <algorithm>

#include "internal.hpp"
#include "wave.hpp"

namespace nvfp4 {

namespace {

constexpr int64_t kMostBlocks = int64_t(1) << 21;  // of a launch (a grid has fewer than 2^32 threads); each takes more tokens beyond that

__device__ __forceinline__ bool inside(int64_t place, int64_t R) { return (uint64_t)place < (uint64_t)R; }

}  // namespace

// A wave moves kPieces x 64 pieces of 16 bytes of one token.
template <int kPieces>
__global__ __launch_bounds__(256) void k_dispatch(MoveArgs a)
{
    const int lane = threadIdx.x & 63;
    const int64_t c0 = 8 * ((int64_t)blockIdx.y * 64 * kPieces + lane);
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave_index(); t < a.T; t += (int64_t)gridDim.x * 4) {
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

// A wave adds up kPieces x 64 pieces of 8 columns of one token, four of its
// rows in flight.
template <int kPieces>
__global__ __launch_bounds__(256) void k_combine(MoveArgs a)
{
    constexpr int kAhead = 4;
    const int lane = threadIdx.x & 63;
    const int64_t c0 = 8 * ((int64_t)blockIdx.y * 64 * kPieces + lane);
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave_index(); t < a.T; t += (int64_t)gridDim.x * 4) {
        Piece sum[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[i].v[e] = 0.0f;
        for (int j0 = 0; j0 < a.k; j0 += kAhead) {
            RawPiece raw[kAhead][kPieces];
            float w[kAhead];
            bool there[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const bool in = j0 + u < a.k;
                const int64_t slot = t * a.k + (in ? j0 + u : j0);
                const int64_t place = a.rows[slot];
                there[u] = in && inside(place, a.R);
                w[u] = !in ? 0.0f : a.weights ? a.weights[slot] : 1.0f;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int64_t c = c0 + 512 * i;
                    raw[u][i].a = raw[u][i].b = make_uint4(0, 0, 0, 0);
                    if (there[u] && c < a.cols) raw[u][i] = load_raw(a.from, place * a.ld_from + c, a.from_f32);
                }
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const Piece o = widen(raw[u][i], a.from_f32);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[i].v[e] = __builtin_fmaf(w[u], o.v[e], sum[i].v[e]);
                }
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int64_t c = c0 + 512 * i;
            if (c >= a.cols) continue;
            if (a.tokens) {
                const Piece r = load_piece(a.tokens, t * a.ld_tokens + c, a.out_f32);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[i].v[e] += r.v[e];
            }
            store_piece(a.out, t * a.ld_out + c, sum[i], a.out_f32);
        }
    }
}

// A token's waves hold two pieces of dy a lane while its rows pass by, four of
// them in flight; each wave adds its dot products up by lane moves, and the
// waves' are added in order.  kSolo: a wave a token, four a workgroup;
// otherwise a workgroup a token, as many waves as its columns fill.
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

template <class Kernel>
void launch_pieces(Kernel kernel, int pieces, const MoveArgs& a, hipStream_t s)
{
    const int64_t blocks = (a.T + 3) / 4, units = (a.cols / 8 + 64 * pieces - 1) / (64 * pieces);
    const int64_t most = kMostBlocks / units > 0 ? kMostBlocks / units : 1;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(blocks < most ? blocks : most), (uint32_t)units), dim3(256), 0, s, a);
}

}  // namespace

void launch_dispatch(const MoveArgs& a, hipStream_t s)
{
    if (a.cols > 512)
        launch_pieces(k_dispatch<2>, 2, a, s);
    else
        launch_pieces(k_dispatch<1>, 1, a, s);
}

void launch_combine(const MoveArgs& a, hipStream_t s)
{
    if (a.cols > 512)
        launch_pieces(k_combine<2>, 2, a, s);
    else
        launch_pieces(k_combine<1>, 1, a, s);
}

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
