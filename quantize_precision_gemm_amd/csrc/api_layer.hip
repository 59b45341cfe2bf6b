// api_layer.hip -- the C ABI of the operators around the expert products
// (include/nvfp4.h): routing, dispatch and combine, the norm, and the linear
// layer with its epilogue.  Every check runs on the host before anything is
// enqueued; a failed check returns a negative status and launches nothing.
#include <stdint.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "nvfp4.h"
#include "api_common.hpp"
#include "internal.hpp"

namespace {

using nvfp4::aligned;
using nvfp4::device_cus;
using nvfp4::holds;
using nvfp4::launch_status;

constexpr int64_t kRowLimit = int64_t(1) << 31;
constexpr int64_t kColLimit = int64_t(1) << 24;  // columns of a row kernel: its grid counts units of 512 in 16 bits

bool known(int32_t dtype) { return dtype == NVFP4_OUT_BF16 || dtype == NVFP4_OUT_FP32; }

// A matrix whose rows move in pieces of 16 bytes: its pitch, then its alignment.
int check_rows(const void* p, int64_t ld, int64_t cols, int32_t dtype)
{
    if (ld < cols) return NVFP4_ERR_SHAPE;
    return aligned(p, 16) && ld % (dtype == NVFP4_OUT_FP32 ? 4 : 8) == 0 ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// What nvfp4_route and its gradient have in common.
int check_route(const void* logits, int32_t l_dtype, int64_t ld, int64_t T, int64_t E, int64_t k, int32_t score,
                int32_t renormalise, float scale)
{
    if (!known(l_dtype) || (score != NVFP4_SOFTMAX && score != NVFP4_SIGMOID) || (renormalise != 0 && renormalise != 1) ||
        !std::isfinite(scale))
        return NVFP4_ERR_MODE;
    if (T < 0 || T > (int64_t(1) << 27) || E < 1 || E > nvfp4::kRouteMostExperts || k < 1 || k > nvfp4::kRouteMostK ||
        k > E || T * k >= kRowLimit || ld < E)
        return NVFP4_ERR_SHAPE;
    if (T > 0 && !logits) return NVFP4_ERR_NULL;
    return aligned(logits, l_dtype == NVFP4_OUT_FP32 ? 4 : 2) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

nvfp4::RouteArgs route_args(const void* logits, int32_t l_dtype, int64_t ld, int64_t T, int64_t E, int64_t k,
                            int32_t score, int32_t renormalise, float scale)
{
    nvfp4::RouteArgs a{};
    a.logits = logits;
    a.T = T;
    a.ld = ld;
    a.E = (int)E;
    a.k = (int)k;
    a.groups = a.kept = 1;
    a.f32 = l_dtype == NVFP4_OUT_FP32;
    a.vec = ld % (a.f32 ? 4 : 8) == 0 && aligned(logits, 16);
    a.sigmoid = score == NVFP4_SIGMOID;
    a.renorm = renormalise != 0;
    a.scale = scale;
    return a;
}

// Sizes of dispatch and combine.
int check_move(const int32_t* rows, int64_t T, int64_t k, int64_t cols, int64_t R)
{
    if (T < 0 || k < 1 || k > nvfp4::kMoveMostK || T >= kRowLimit || R < 0 || R >= kRowLimit || cols < 0 || cols % 8 ||
        cols > kColLimit)
        return NVFP4_ERR_SHAPE;
    if (T > 0 && !rows) return NVFP4_ERR_NULL;
    return aligned(rows, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// Sizes, types and eps of the norm and its gradient.
int check_norm(int64_t rows, int64_t cols, int32_t x_dtype, int32_t s_dtype, int32_t w_dtype, double eps,
               const void* weight)
{
    if (!known(x_dtype) || !known(s_dtype) || !known(w_dtype) || !(eps >= 0.0) || !std::isfinite(eps))
        return NVFP4_ERR_MODE;
    if (rows < 0 || rows >= kRowLimit || cols < 0 || cols >= kRowLimit || cols % 8) return NVFP4_ERR_SHAPE;
    return aligned(weight, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// Sizes of a linear layer's gradients: the sums of the biases take a workgroup
// of 256 threads for 64 columns of an expert, in one grid.
bool fits_linear_backward(int64_t E, int64_t T, int64_t N)
{
    return E >= 0 && E <= 65535 && T >= 0 && T < kRowLimit && N >= 0 && N % 8 == 0 && N <= kColLimit &&
           E * ((N + 63) / 64) < (int64_t(1) << 24);
}

float norm_eps(double eps)
{
    const float e = (float)eps;
    return eps > 0.0 && e == 0.0f ? FLT_TRUE_MIN : e;  // a row of zeros stays one
}

}  // namespace

extern "C" {

int nvfp4_route_workspace(int64_t T, int64_t E, int64_t* bytes)
{
    if (!bytes) return NVFP4_ERR_NULL;
    if (T < 0 || T > (int64_t(1) << 27) || E < 1 || E > nvfp4::kRouteMostExperts) return NVFP4_ERR_SHAPE;
    *bytes = nvfp4::route_workspace(T, E);
    return NVFP4_OK;
}

int nvfp4_route(const void* logits, int32_t l_dtype, int64_t ld, int64_t T, int64_t E, int64_t k, const float* bias,
                int64_t groups, int64_t groups_kept, int32_t score, int32_t renormalise, float scale,
                int32_t* experts, float* weights, int32_t* rows, int32_t* ends, float* scores, void* workspace,
                int64_t workspace_bytes, void* stream)
{
    const int st = check_route(logits, l_dtype, ld, T, E, k, score, renormalise, scale);
    if (st != NVFP4_OK) return st;
    if (groups < 1 || groups > nvfp4::kRouteMostGroups || E % groups || groups_kept < 1 || groups_kept > groups ||
        k > E / groups * groups_kept || workspace_bytes < 0)
        return NVFP4_ERR_SHAPE;
    if (T > 0 && (!rows != !ends || !experts || !weights)) return NVFP4_ERR_NULL;
    if (!aligned(bias, 4) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(rows, 4) || !aligned(ends, 4) ||
        !aligned(scores, 4) || !aligned(workspace, 16))
        return NVFP4_ERR_ALIGN;
    const int64_t need = ends ? nvfp4::route_workspace(T, E) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
    nvfp4::RouteArgs a = route_args(logits, l_dtype, ld, T, E, k, score, renormalise, scale);
    a.bias = bias;
    a.vec_bias = aligned(bias, 16);
    a.groups = (int)groups;
    a.kept = (int)groups_kept;
    a.experts = experts;
    a.weights = weights;
    a.rows = rows;
    a.ends = ends;
    a.scores = scores;
    a.counts = static_cast<uint8_t*>(workspace);
    nvfp4::launch_route(a, static_cast<hipStream_t>(stream));
    return launch_status();
}

int nvfp4_route_backward(const void* logits, int32_t l_dtype, int64_t ld, int64_t T, int64_t E, int64_t k,
                         const int32_t* experts, const float* dweights, const float* dscores, int32_t score,
                         int32_t renormalise, float scale, void* dlogits, int64_t ld_out, int32_t out_dtype,
                         void* stream)
{
    const int st = check_route(logits, l_dtype, ld, T, E, k, score, renormalise, scale);
    if (st != NVFP4_OK) return st;
    if (!known(out_dtype)) return NVFP4_ERR_MODE;
    if (ld_out < E) return NVFP4_ERR_SHAPE;
    if (T > 0 && (!experts || !dweights || !dlogits)) return NVFP4_ERR_NULL;
    const bool f32 = out_dtype == NVFP4_OUT_FP32;
    if (!aligned(experts, 4) || !aligned(dweights, 4) || !aligned(dscores, 4) || !aligned(dlogits, f32 ? 4 : 2))
        return NVFP4_ERR_ALIGN;
    nvfp4::RouteBackArgs a{};
    a.f = route_args(logits, l_dtype, ld, T, E, k, score, renormalise, scale);
    a.f.experts = const_cast<int32_t*>(experts);
    a.dweights = dweights;
    a.dscores = dscores;
    a.out = dlogits;
    a.ld_out = ld_out;
    a.out_f32 = f32;
    a.vec_scores = E % 4 == 0 && aligned(dscores, 16);
    a.vec_out = ld_out % 4 == 0 && aligned(dlogits, f32 ? 16 : 8);
    nvfp4::launch_route_backward(a, static_cast<hipStream_t>(stream));
    return launch_status();
}

int nvfp4_dispatch(const void* x, int64_t ld_x, const int32_t* rows, int64_t T, int64_t k, int64_t cols, int64_t R,
                   void* out, int64_t ld_out, void* stream)
{
    int st = check_move(rows, T, k, cols, R);
    if (st == NVFP4_OK) st = check_rows(x, ld_x, cols, NVFP4_OUT_BF16);
    if (st == NVFP4_OK) st = check_rows(out, ld_out, cols, NVFP4_OUT_BF16);
    if (st != NVFP4_OK) return st;
    if (T == 0 || cols == 0) return NVFP4_OK;
    if (!x || (R > 0 && !out)) return NVFP4_ERR_NULL;
    nvfp4::MoveArgs a{};
    a.rows = rows;
    a.T = T;
    a.R = R;
    a.k = (int)k;
    a.cols = cols;
    a.tokens = x;
    a.ld_tokens = ld_x;
    a.out = out;
    a.ld_out = ld_out;
    nvfp4::launch_dispatch(a, static_cast<hipStream_t>(stream));
    return launch_status();
}

int nvfp4_combine(const void* o, int32_t o_dtype, int64_t ld_o, int64_t R, const int32_t* rows, const float* weights,
                  int64_t T, int64_t k, int64_t cols, const void* residual, int64_t ld_r, void* y, int64_t ld_y,
                  int32_t y_dtype, void* stream)
{
    if (!known(o_dtype) || !known(y_dtype)) return NVFP4_ERR_MODE;
    int st = check_move(rows, T, k, cols, R);
    if (st == NVFP4_OK) st = check_rows(o, ld_o, cols, o_dtype);
    if (st == NVFP4_OK) st = check_rows(y, ld_y, cols, y_dtype);
    if (st == NVFP4_OK && residual) st = check_rows(residual, ld_r, cols, y_dtype);
    if (st != NVFP4_OK) return st;
    if (!aligned(weights, 4)) return NVFP4_ERR_ALIGN;
    if (T == 0 || cols == 0) return NVFP4_OK;
    if (!y || (R > 0 && !o)) return NVFP4_ERR_NULL;
    nvfp4::MoveArgs a{};
    a.rows = rows;
    a.T = T;
    a.R = R;
    a.k = (int)k;
    a.cols = cols;
    a.weights = weights;
    a.tokens = residual;
    a.ld_tokens = ld_r;
    a.from = o;
    a.ld_from = ld_o;
    a.from_f32 = o_dtype == NVFP4_OUT_FP32;
    a.out = y;
    a.ld_out = ld_y;
    a.out_f32 = y_dtype == NVFP4_OUT_FP32;
    nvfp4::launch_combine(a, static_cast<hipStream_t>(stream));
    return launch_status();
}

int nvfp4_combine_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* o, int32_t o_dtype,
                           int64_t ld_o, int64_t R, const int32_t* rows, const float* weights, int64_t T, int64_t k,
                           int64_t cols, void* d_o, int64_t ld_do, float* dweights, void* stream)
{
    if (!known(dy_dtype) || !known(o_dtype)) return NVFP4_ERR_MODE;
    int st = check_move(rows, T, k, cols, R);
    if (st == NVFP4_OK) st = check_rows(dy, ld_dy, cols, dy_dtype);
    if (st == NVFP4_OK) st = check_rows(o, ld_o, cols, o_dtype);
    if (st == NVFP4_OK) st = check_rows(d_o, ld_do, cols, NVFP4_OUT_BF16);
    if (st != NVFP4_OK) return st;
    if (!aligned(weights, 4) || !aligned(dweights, 4)) return NVFP4_ERR_ALIGN;
    if (T == 0) return NVFP4_OK;
    if (!weights || !dweights || (cols > 0 && (!dy || (R > 0 && (!o || !d_o))))) return NVFP4_ERR_NULL;
    nvfp4::MoveArgs a{};
    a.rows = rows;
    a.T = T;
    a.R = R;
    a.k = (int)k;
    a.cols = cols;
    a.weights = weights;
    a.tokens = dy;
    a.ld_tokens = ld_dy;
    a.tokens_f32 = dy_dtype == NVFP4_OUT_FP32;
    a.from = o;
    a.ld_from = ld_o;
    a.from_f32 = o_dtype == NVFP4_OUT_FP32;
    a.out = d_o;
    a.ld_out = ld_do;
    a.dweights = dweights;
    nvfp4::launch_combine_backward(a, static_cast<hipStream_t>(stream));
    return launch_status();
}

int nvfp4_rmsnorm(const void* x, int32_t x_dtype, int64_t ld_x, const void* residual, int64_t ld_r, int32_t s_dtype,
                  const void* weight, int32_t w_dtype, double eps, int64_t rows, int64_t cols, void* h, int64_t ld_h,
                  void* y, int64_t ld_y, int8_t* codes, int64_t ld_codes, float* scales, void* stream)
{
    int st = check_norm(rows, cols, x_dtype, s_dtype, w_dtype, eps, weight);
    if (st != NVFP4_OK) return st;
    const bool some = rows > 0 && cols > 0, int8 = scales != nullptr;  // (rows of no columns have scales of 0)
    if (int8 && cols % 16) return NVFP4_ERR_SHAPE;
    if ((codes && !int8) || (some && (!x || (int8 ? !codes : !y)))) return NVFP4_ERR_NULL;
    st = check_rows(x, ld_x, cols, x_dtype);
    if (st == NVFP4_OK && residual) st = check_rows(residual, ld_r, cols, s_dtype);
    if (st == NVFP4_OK && h) st = check_rows(h, ld_h, cols, s_dtype);
    if (st == NVFP4_OK && y) st = check_rows(y, ld_y, cols, NVFP4_OUT_BF16);
    if (st != NVFP4_OK) return st;
    if (int8 && ld_codes < cols) return NVFP4_ERR_SHAPE;
    if (int8 && (!aligned(codes, 16) || ld_codes % 16 || !aligned(scales, 4))) return NVFP4_ERR_ALIGN;
    nvfp4::NormArgs a{};
    a.rows = rows;
    a.cols = cols;
    a.x = x;
    a.ld_x = ld_x;
    a.residual = residual;
    a.ld_r = ld_r;
    a.weight = weight;
    a.x_f32 = x_dtype == NVFP4_OUT_FP32;
    a.s_f32 = s_dtype == NVFP4_OUT_FP32;
    a.w_f32 = w_dtype == NVFP4_OUT_FP32;
    a.eps = norm_eps(eps);
    a.h = h;
    a.ld_h = ld_h;
    a.y = static_cast<uint16_t*>(y);
    a.ld_y = ld_y;
    a.codes = codes;
    a.ld_codes = ld_codes;
    a.scales = scales;
    nvfp4::launch_norm(a, static_cast<hipStream_t>(stream));
    return launch_status();
}

int nvfp4_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes)
{
    if (!bytes) return NVFP4_ERR_NULL;
    if (rows < 0 || rows >= kRowLimit || cols < 0 || cols % 8 || cols > nvfp4::kNormMostCols) return NVFP4_ERR_SHAPE;
    *bytes = nvfp4::norm_backward_workspace(rows, cols, std::max(device_cus(), 1));
    return NVFP4_OK;
}

int nvfp4_rmsnorm_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* h, int64_t ld_h,
                           const void* dh, int64_t ld_dh, int32_t s_dtype, const void* weight, int32_t w_dtype,
                           double eps, int64_t rows, int64_t cols, void* dx, int64_t ld_dx, int32_t dx_dtype,
                           float* dweight, void* workspace, int64_t workspace_bytes, void* stream)
{
    int st = check_norm(rows, cols, dy_dtype, s_dtype, w_dtype, eps, weight);
    if (st != NVFP4_OK) return st;
    if (!known(dx_dtype)) return NVFP4_ERR_MODE;
    if (cols > nvfp4::kNormMostCols || workspace_bytes < 0) return NVFP4_ERR_SHAPE;
    if (rows > 0 && cols > 0 && (!dy || !h || !dx)) return NVFP4_ERR_NULL;
    st = check_rows(dy, ld_dy, cols, dy_dtype);
    if (st == NVFP4_OK) st = check_rows(h, ld_h, cols, s_dtype);
    if (st == NVFP4_OK && dh) st = check_rows(dh, ld_dh, cols, s_dtype);
    if (st == NVFP4_OK) st = check_rows(dx, ld_dx, cols, dx_dtype);
    if (st != NVFP4_OK) return st;
    if (!aligned(dweight, 16) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    const int cus = std::max(device_cus(), 1);
    const int64_t need = dweight ? nvfp4::norm_backward_workspace(rows, cols, cus) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
    nvfp4::NormArgs a{};
    a.rows = rows;
    a.cols = cols;
    a.x = dy;
    a.ld_x = ld_dy;
    a.residual = dh;
    a.ld_r = ld_dh;
    a.weight = weight;
    a.x_f32 = dy_dtype == NVFP4_OUT_FP32;
    a.s_f32 = s_dtype == NVFP4_OUT_FP32;
    a.w_f32 = w_dtype == NVFP4_OUT_FP32;
    a.eps = norm_eps(eps);
    a.h = const_cast<void*>(h);
    a.ld_h = ld_h;
    a.dx = dx;
    a.ld_dx = ld_dx;
    a.dx_f32 = dx_dtype == NVFP4_OUT_FP32;
    a.dweight = dweight;
    a.parts = static_cast<float*>(workspace);
    a.cus = cus;
    nvfp4::launch_norm_backward(a, static_cast<hipStream_t>(stream));
    return launch_status();
}

int nvfp4_bf16_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t stride_w, const int32_t* ends,
                      int64_t E, int64_t T, int64_t N, int64_t K, const void* bias, int64_t stride_bias,
                      int32_t bias_dtype, int32_t act, const void* residual, int64_t ld_r, void* pre, int64_t ld_pre,
                      void* c, int64_t ldc, int32_t c_dtype, void* workspace, int64_t workspace_bytes, void* stream)
{
    if (!known(c_dtype) || !known(bias_dtype) || act < NVFP4_ACT_NONE || act > NVFP4_ACT_GELU) return NVFP4_ERR_MODE;
    const int st = nvfp4::check_grouped(NVFP4_FPROP, E, T, N, K);
    if (st != NVFP4_OK) return st;
    if ((!ends && E != 1 && E != 0) || workspace_bytes < 0) return NVFP4_ERR_SHAPE;
    if ((T > 0 && K > 0 && !x) || (E > 0 && N > 0 && K > 0 && !w) || (T > 0 && N > 0 && !c) || (E > 0 && !ends && E != 1))
        return NVFP4_ERR_NULL;
    const bool f32 = c_dtype == NVFP4_OUT_FP32;
    if (!aligned(x, 16) || !aligned(w, 16) || ldx % 8 || ldw % 8 || stride_w % 8 || !aligned(ends, 4)) return NVFP4_ERR_ALIGN;
    if (!aligned(c, f32 ? 16 : 8) || ldc % 4 || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    if (!aligned(bias, bias_dtype == NVFP4_OUT_FP32 ? 16 : 8) || stride_bias % 4) return NVFP4_ERR_ALIGN;
    if (residual && (!aligned(residual, f32 ? 16 : 8) || ld_r % 4)) return NVFP4_ERR_ALIGN;
    if (pre && (!aligned(pre, 8) || ld_pre % 4)) return NVFP4_ERR_ALIGN;
    if (ldx < K || ldw < K || ldc < N || (residual && ld_r < N) || (pre && ld_pre < N)) return NVFP4_ERR_SHAPE;
    if (E > 1 && !holds(stride_w, N, ldw, K)) return NVFP4_ERR_SHAPE;
    if (bias && E > 1 && stride_bias < N) return NVFP4_ERR_SHAPE;
    const int64_t span = int64_t(1) << 22;  // a tile's 256 rows are addressed with 32-bit offsets
    if (ldx >= span || ldw >= span) return NVFP4_ERR_SHAPE;
    const nvfp4::GroupedArgs g{static_cast<const uint16_t*>(x), ldx, static_cast<const uint16_t*>(w), ldw, stride_w, ends,
                               E, T, N, K, c, ldc, 0, std::max(device_cus(), 1), static_cast<float*>(workspace), 1};
    const nvfp4::Epilogue e{bias, stride_bias, bias_dtype == NVFP4_OUT_FP32, act, residual, ld_r,
                            static_cast<uint16_t*>(pre), ld_pre};
    nvfp4::launch_linear(g, e, workspace_bytes, f32, static_cast<hipStream_t>(stream));
    return launch_status();
}

int nvfp4_bf16_linear_backward_workspace(int64_t E, int64_t T, int64_t N, int64_t* bytes)
{
    if (!bytes) return NVFP4_ERR_NULL;
    if (!fits_linear_backward(E, T, N)) return NVFP4_ERR_SHAPE;
    *bytes = nvfp4::linear_backward_workspace(E, T, N);
    return NVFP4_OK;
}

int nvfp4_bf16_linear_backward(const void* dy, int32_t dy_dtype, int64_t ld_dy, const void* pre, int64_t ld_pre,
                               int32_t act, const int32_t* ends, int64_t E, int64_t T, int64_t N, void* dpre,
                               int64_t ld_dpre, float* dbias, void* workspace, int64_t workspace_bytes, void* stream)
{
    if (!known(dy_dtype) || act < NVFP4_ACT_NONE || act > NVFP4_ACT_GELU) return NVFP4_ERR_MODE;
    if (!pre && act != NVFP4_ACT_NONE && T > 0 && N > 0) return NVFP4_ERR_NULL;
    if (!fits_linear_backward(E, T, N) || workspace_bytes < 0) return NVFP4_ERR_SHAPE;
    if (!ends && E > 1) return NVFP4_ERR_NULL;
    if (T > 0 && N > 0 && E > 0 && (!dy || (pre && !dpre) || (!pre && !dbias))) return NVFP4_ERR_NULL;
    int st = check_rows(dy, ld_dy, N, dy_dtype);
    if (st == NVFP4_OK && pre) st = check_rows(pre, ld_pre, N, NVFP4_OUT_BF16);
    if (st == NVFP4_OK && pre) st = check_rows(dpre, ld_dpre, N, NVFP4_OUT_BF16);
    if (st != NVFP4_OK) return st;
    if (!aligned(ends, 4) || !aligned(dbias, 16) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    const int64_t need =
        dbias && !nvfp4::linear_backward_one_run(ends, T, N) ? nvfp4::linear_backward_workspace(E, T, N) : 0;
    if (need > 0 && (!workspace || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
    const nvfp4::LinearBackArgs a{dy, ld_dy, dy_dtype == NVFP4_OUT_FP32, static_cast<const uint16_t*>(pre), ld_pre,
                                  static_cast<uint16_t*>(dpre), ld_dpre, ends, E, T, N, act, dbias,
                                  static_cast<float*>(workspace)};
    nvfp4::launch_linear_backward(a, static_cast<hipStream_t>(stream));
    return launch_status();
}

}  // extern "C"
