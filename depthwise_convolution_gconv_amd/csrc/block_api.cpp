// block_api.cpp -- C entry points of the recurrent block's operators (gated linear
// recurrence, group norm, product in 8-bit integers): validation, plans and launches.  Host code only.
#include <hip/hip_runtime.h>

#include "block.hpp"
#include "gconv.h"
#include "seq_host.hpp"

namespace {

using namespace gconv::host;

// ---------------------------------------------------------------- gated recurrence

gconv_status_t gated_shape(const int64_t *shape, gconv_dtype_t dtype)
{
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    const int64_t B = shape[0], T = shape[1], C = shape[2];
    if (B < 0 || T < 0 || C < 1)
        return fail(GCONV_ERR_INVALID_ARG, "gated recurrence: B, T >= 0 and C >= 1 are needed");
    if (B > kMax || T > kMax - 65536 || C > kMax / 8 || (double)B * (double)T * (double)C >= kCells / 8)
        return fail(GCONV_ERR_UNSUPPORTED, "gated recurrence: sizes exceed the library's index range");
    return GCONV_OK;
}

// Strides whose products with the sizes stay in 64 bits.
gconv_status_t reach(const int64_t *strides, int n, int64_t B, int64_t T)
{
    const gconv_status_t st = check_strides(strides, n);
    if (st != GCONV_OK) return st;
    for (int i = 0; i < n; ++i)
        if ((double)strides[i] * (double)(i % 2 ? T : B) >= kCells / 8)
            return fail(GCONV_ERR_UNSUPPORTED, "stride %d exceeds the library's index range", i);
    return GCONV_OK;
}

gconv_status_t gated_check(const gconv::GatedArgs &a, const gconv::GatedPlan &g, bool backward)
{
    if (!gconv::gated_fits(a, g, backward))
        return fail(GCONV_ERR_UNSUPPORTED, "gated recurrence: the sizes or token strides exceed what a launch takes");
    return GCONV_OK;
}

// ---------------------------------------------------------------- group norm

gconv_status_t gn_shape(const int64_t *shape, gconv_act_t act, gconv_dtype_t dtype)
{
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (act != GCONV_ACT_NONE && act != GCONV_ACT_SILU)
        return fail(GCONV_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    const int64_t N = shape[0], P = shape[1], C = shape[2], G = shape[3];
    if (N < 0 || P < 0 || C < 1 || G < 1)
        return fail(GCONV_ERR_INVALID_ARG, "group norm: N, P >= 0 and C, G >= 1 are needed");
    if (C % G != 0)
        return fail(GCONV_ERR_SHAPE, "group norm: %lld channels do not divide into %lld groups", (long long)C, (long long)G);
    if (C > int64_t(1) << 20 || N > kMax || P > kMax - 65536 || (double)N * (double)P * (double)C >= kCells / 8)
        return fail(GCONV_ERR_UNSUPPORTED, "group norm: at most 2^20 channels, 2^31 - 1 samples and positions");
    return GCONV_OK;
}

gconv_status_t gn_check(const gconv::GroupNormArgs &a, const gconv::GroupNormPlan &g)
{
    if (!gconv::gn_fits(a, g))
        return fail(GCONV_ERR_UNSUPPORTED, "group norm: the sizes or position strides exceed what a launch takes");
    return GCONV_OK;
}

}  // namespace

extern "C" {

gconv_status_t gconv_gated_recurrence_workspace(const int64_t *shape, gconv_dtype_t dtype, int32_t backward, size_t *bytes)
{
    gconv::set_last_error("");
    if (!bytes) return fail(GCONV_ERR_INVALID_ARG, "NULL bytes");
    const gconv_status_t st = gated_shape(shape, dtype);
    if (st != GCONV_OK) return st;
    const gconv::GatedPlan g = gconv::gated_plan(shape[0], shape[1], shape[2], (int)dtype, backward != 0);
    *bytes = gconv::gated_workspace(g, shape[0], shape[2], backward != 0);
    return GCONV_OK;
}

gconv_status_t gconv_gated_recurrence(const void *x, const void *r, const void *i, const float *log_decay, void *h,
                                      const int64_t *shape, const int64_t *strides, const float *initial_state,
                                      float *final_state, const int32_t *lengths, gconv_dtype_t dtype, void *workspace,
                                      size_t workspace_bytes, void *hip_stream)
{
    gconv::set_last_error("");
    gconv_status_t st = gated_shape(shape, dtype);
    if (st != GCONV_OK) return st;
    const int64_t B = shape[0], T = shape[1], C = shape[2];
    if ((st = reach(strides, 6, B, T)) != GCONV_OK) return st;
    if (!log_decay) return fail(GCONV_ERR_INVALID_ARG, "NULL log_decay");
    if (B > 0 && T > 0 && (!x || !r || !i || !h)) return fail(GCONV_ERR_INVALID_ARG, "NULL x, r, i or h");
    const gconv::GatedPlan g = gconv::gated_plan(B, T, C, (int)dtype, false);
    const size_t need = gconv::gated_workspace(g, B, C, false), es = elem(dtype), ns = 4 * (size_t)(B * C);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GCONV_OK) return st;
    const Range ranges[] = {
        {"h", h, es * (size_t)(B * T * C), true},
        {"final_state", final_state, ns, true},
        {"workspace", workspace, need, true},
        {"x", x, extent(B, strides[0], T, strides[1], 1, 0, C, es), false},
        {"r", r, extent(B, strides[2], T, strides[3], 1, 0, C, es), false},
        {"i", i, extent(B, strides[4], T, strides[5], 1, 0, C, es), false},
        {"log_decay", log_decay, 4 * (size_t)C, false},
        {"initial_state", initial_state, ns, false},
        {"lengths", lengths, 4 * (size_t)B, false},
    };
    if ((st = check_ranges(ranges, sizeof(ranges) / sizeof(ranges[0]))) != GCONV_OK) return st;
    gconv::GatedArgs a = {};
    a.x = x; a.r = r; a.i = i; a.log_decay = log_decay; a.s0 = initial_state; a.lengths = lengths;
    a.h = h; a.sf = final_state; a.ws = (float *)workspace;
    a.B = B; a.T = T; a.C = C;
    a.xsb = strides[0]; a.xst = strides[1]; a.rsb = strides[2]; a.rst = strides[3]; a.isb = strides[4]; a.ist = strides[5];
    a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    if ((st = gated_check(a, g, false)) != GCONV_OK) return st;
    if (B == 0 || (T == 0 && !final_state)) return done(hipSuccess, "");
    const char *kname = "";
    const hipError_t err = gconv::launch_gated(a, g, &kname);
    return done(err, kname);
}

gconv_status_t gconv_gated_recurrence_backward(const void *x, const void *r, const void *i, const float *log_decay, const void *h,
                                               const void *dh, void *dx, void *dr, void *di, float *dlog_decay,
                                               const int64_t *shape, const int64_t *strides, const float *initial_state,
                                               const float *dfinal, float *dinitial, const int32_t *lengths,
                                               gconv_dtype_t dtype, void *workspace, size_t workspace_bytes, void *hip_stream)
{
    gconv::set_last_error("");
    gconv_status_t st = gated_shape(shape, dtype);
    if (st != GCONV_OK) return st;
    const int64_t B = shape[0], T = shape[1], C = shape[2];
    if ((st = reach(strides, 10, B, T)) != GCONV_OK) return st;
    if (!log_decay || !dlog_decay) return fail(GCONV_ERR_INVALID_ARG, "NULL log_decay or its gradient");
    if (B > 0 && T > 0 && (!x || !r || !i || !h || !dh || !dx || !dr || !di))
        return fail(GCONV_ERR_INVALID_ARG, "NULL x, r, i, h, dh, dx, dr or di");
    if (dinitial && !initial_state)
        return fail(GCONV_ERR_INVALID_ARG, "gated recurrence: dinitial goes with an initial state");
    const gconv::GatedPlan g = gconv::gated_plan(B, T, C, (int)dtype, true);
    const size_t need = gconv::gated_workspace(g, B, C, true), es = elem(dtype), ns = 4 * (size_t)(B * C),
                 all = es * (size_t)(B * T * C);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GCONV_OK) return st;
    auto view = [&](int k) { return extent(B, strides[2 * k], T, strides[2 * k + 1], 1, 0, C, es); };
    const Range ranges[] = {
        {"dx", dx, all, true},
        {"dr", dr, all, true},
        {"di", di, all, true},
        {"dlog_decay", dlog_decay, 4 * (size_t)C, true},
        {"dinitial", dinitial, ns, true},
        {"workspace", workspace, need, true},
        {"x", x, view(0), false},
        {"r", r, view(1), false},
        {"i", i, view(2), false},
        {"h", h, view(3), false},
        {"dh", dh, view(4), false},
        {"log_decay", log_decay, 4 * (size_t)C, false},
        {"initial_state", initial_state, ns, false},
        {"dfinal", dfinal, ns, false},
        {"lengths", lengths, 4 * (size_t)B, false},
    };
    if ((st = check_ranges(ranges, sizeof(ranges) / sizeof(ranges[0]))) != GCONV_OK) return st;
    gconv::GatedArgs a = {};
    a.x = x; a.r = r; a.i = i; a.log_decay = log_decay; a.s0 = initial_state; a.lengths = lengths;
    a.h = const_cast<void *>(h); a.dh = dh; a.dsf = dfinal; a.dx = dx; a.dr = dr; a.di = di; a.dlog = dlog_decay; a.ds0 = dinitial;
    a.ws = (float *)workspace;
    a.B = B; a.T = T; a.C = C;
    a.xsb = strides[0]; a.xst = strides[1]; a.rsb = strides[2]; a.rst = strides[3]; a.isb = strides[4]; a.ist = strides[5];
    a.hsb = strides[6]; a.hst = strides[7]; a.dsb = strides[8]; a.dst = strides[9];
    a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    if ((st = gated_check(a, g, true)) != GCONV_OK) return st;
    const char *kname = "";
    const hipError_t err = gconv::launch_gated_bwd(a, g, &kname);
    return done(err, kname);
}

gconv_status_t gconv_gated_recurrence_step(const void *x, const void *r, const void *i, const float *log_decay, float *state,
                                           void *h, const int64_t *shape, const int64_t *strides, const int32_t *slots,
                                           gconv_dtype_t dtype, void *hip_stream)
{
    gconv::set_last_error("");
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    const int64_t B = shape[0], C = shape[1], n = shape[2], whole[3] = {B, 1, C};
    gconv_status_t st = gated_shape(whole, dtype);
    if (st != GCONV_OK || (st = check_strides(strides, 3)) != GCONV_OK) return st;
    for (int k = 0; k < 3; ++k)
        if ((double)strides[k] * (double)B >= kCells / 8)
            return fail(GCONV_ERR_UNSUPPORTED, "stride %d exceeds the library's index range", k);
    if (n < 0) return fail(GCONV_ERR_INVALID_ARG, "gated recurrence step: n >= 0 states are needed");
    if (!slots && n < B)
        return fail(GCONV_ERR_SHAPE, "gated recurrence step: %lld states for %lld sequences without slots", (long long)n,
                    (long long)B);
    if ((double)n * (double)C >= kCells / 8)
        return fail(GCONV_ERR_UNSUPPORTED, "gated recurrence step: sizes exceed the library's index range");
    if (!log_decay) return fail(GCONV_ERR_INVALID_ARG, "NULL log_decay");
    if (B == 0) return done(hipSuccess, "");
    if (!x || !r || !i || !h || (!state && n > 0)) return fail(GCONV_ERR_INVALID_ARG, "NULL x, r, i, h or state");
    const size_t es = elem(dtype);
    const Range ranges[] = {
        {"h", h, es * (size_t)(B * C), true},
        {"state", state, 4 * (size_t)(n * C), true},
        {"x", x, extent(B, strides[0], 1, 0, 1, 0, C, es), false},
        {"r", r, extent(B, strides[1], 1, 0, 1, 0, C, es), false},
        {"i", i, extent(B, strides[2], 1, 0, 1, 0, C, es), false},
        {"log_decay", log_decay, 4 * (size_t)C, false},
        {"slots", slots, 4 * (size_t)B, false},
    };
    if ((st = check_ranges(ranges, sizeof(ranges) / sizeof(ranges[0]))) != GCONV_OK) return st;
    gconv::GatedStepArgs a = {};
    a.x = x; a.r = r; a.i = i; a.log_decay = log_decay; a.state = state; a.h = h; a.slots = slots;
    a.B = B; a.C = C; a.n = n; a.xs = strides[0]; a.rs = strides[1]; a.is = strides[2];
    a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    if (!gconv::gated_step_fits(a))
        return fail(GCONV_ERR_UNSUPPORTED, "gated recurrence step: the call needs more threads than a launch takes");
    const char *kname = "";
    const hipError_t err = gconv::launch_gated_step(a, &kname);
    return done(err, kname);
}

// ---------------------------------------------------------------- group norm

gconv_status_t gconv_group_norm_workspace(const int64_t *shape, gconv_dtype_t dtype, int32_t backward, size_t *bytes)
{
    gconv::set_last_error("");
    if (!bytes) return fail(GCONV_ERR_INVALID_ARG, "NULL bytes");
    const gconv_status_t st = gn_shape(shape, GCONV_ACT_NONE, dtype);
    if (st != GCONV_OK) return st;
    const gconv::GroupNormPlan g = gconv::gn_plan(shape[0], shape[1], shape[2], shape[3], (int)dtype, backward != 0);
    *bytes = gconv::gn_workspace(g, shape[0], shape[2], shape[3], backward != 0);
    return GCONV_OK;
}

gconv_status_t gconv_group_norm(const void *x, const void *weight, const void *bias, void *y, float *stats, const int64_t *shape,
                                const int64_t *strides, const int32_t *lengths, float eps, gconv_act_t activation,
                                gconv_dtype_t dtype, void *workspace, size_t workspace_bytes, void *hip_stream)
{
    gconv::set_last_error("");
    gconv_status_t st = gn_shape(shape, activation, dtype);
    if (st != GCONV_OK) return st;
    const int64_t N = shape[0], P = shape[1], C = shape[2], G = shape[3];
    if ((st = reach(strides, 2, N, P)) != GCONV_OK) return st;
    if (!(eps >= 0.0f)) return fail(GCONV_ERR_INVALID_ARG, "group norm: eps must be >= 0");
    if (!weight) return fail(GCONV_ERR_INVALID_ARG, "NULL weight");
    if (N > 0 && P > 0 && (!x || !y)) return fail(GCONV_ERR_INVALID_ARG, "NULL x or y");
    const gconv::GroupNormPlan g = gconv::gn_plan(N, P, C, G, (int)dtype, false);
    const size_t need = gconv::gn_workspace(g, N, C, G, false), es = elem(dtype);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GCONV_OK) return st;
    const Range ranges[] = {
        {"y", y, es * (size_t)(N * P * C), true},
        {"stats", stats, 8 * (size_t)(N * G), true},
        {"workspace", workspace, need, true},
        {"x", x, extent(N, strides[0], P, strides[1], 1, 0, C, es), false},
        {"weight", weight, es * (size_t)C, false},
        {"bias", bias, es * (size_t)C, false},
        {"lengths", lengths, 4 * (size_t)N, false},
    };
    if ((st = check_ranges(ranges, sizeof(ranges) / sizeof(ranges[0]))) != GCONV_OK) return st;
    gconv::GroupNormArgs a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.stats_out = stats; a.lengths = lengths; a.ws = workspace;
    a.N = N; a.P = P; a.C = C; a.G = G; a.xsb = strides[0]; a.xst = strides[1];
    a.eps = eps; a.silu = activation == GCONV_ACT_SILU; a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    if ((st = gn_check(a, g)) != GCONV_OK) return st;
    if (N == 0 || (P == 0 && !stats)) return done(hipSuccess, "");
    const char *kname = "";
    const hipError_t err = gconv::launch_group_norm(a, g, &kname);
    return done(err, kname);
}

gconv_status_t gconv_group_norm_backward(const void *dy, const void *x, const void *weight, const void *bias, const float *stats,
                                         void *dx, void *dw, void *db, const int64_t *shape, const int64_t *strides,
                                         const int32_t *lengths, gconv_act_t activation, gconv_dtype_t dtype, void *workspace,
                                         size_t workspace_bytes, void *hip_stream)
{
    gconv::set_last_error("");
    gconv_status_t st = gn_shape(shape, activation, dtype);
    if (st != GCONV_OK) return st;
    const int64_t N = shape[0], P = shape[1], C = shape[2], G = shape[3];
    if ((st = reach(strides, 4, N, P)) != GCONV_OK) return st;
    if (!weight || !dw) return fail(GCONV_ERR_INVALID_ARG, "NULL weight or dw");
    if ((bias != nullptr) != (db != nullptr)) return fail(GCONV_ERR_INVALID_ARG, "group norm: db goes with a bias");
    if (N > 0 && !stats) return fail(GCONV_ERR_INVALID_ARG, "NULL stats");
    if (N > 0 && P > 0 && (!x || !dy || !dx)) return fail(GCONV_ERR_INVALID_ARG, "NULL x, dy or dx");
    const gconv::GroupNormPlan g = gconv::gn_plan(N, P, C, G, (int)dtype, true);
    const size_t need = gconv::gn_workspace(g, N, C, G, true), es = elem(dtype);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GCONV_OK) return st;
    const Range ranges[] = {
        {"dx", dx, es * (size_t)(N * P * C), true},
        {"dw", dw, es * (size_t)C, true},
        {"db", db, es * (size_t)C, true},
        {"workspace", workspace, need, true},
        {"dy", dy, extent(N, strides[0], P, strides[1], 1, 0, C, es), false},
        {"x", x, extent(N, strides[2], P, strides[3], 1, 0, C, es), false},
        {"stats", stats, 8 * (size_t)(N * G), false},
        {"weight", weight, es * (size_t)C, false},
        {"bias", bias, es * (size_t)C, false},
        {"lengths", lengths, 4 * (size_t)N, false},
    };
    if ((st = check_ranges(ranges, sizeof(ranges) / sizeof(ranges[0]))) != GCONV_OK) return st;
    gconv::GroupNormArgs a = {};
    a.x = x; a.dy = dy; a.weight = weight; a.bias = bias; a.stats = stats; a.y = dx; a.dw = dw; a.db = db; a.lengths = lengths;
    a.ws = workspace;
    a.N = N; a.P = P; a.C = C; a.G = G; a.dsb = strides[0]; a.dst = strides[1]; a.xsb = strides[2]; a.xst = strides[3];
    a.silu = activation == GCONV_ACT_SILU; a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    if ((st = gn_check(a, g)) != GCONV_OK) return st;
    const char *kname = "";
    const hipError_t err = gconv::launch_group_norm_bwd(a, g, &kname);
    return done(err, kname);
}

// ---------------------------------------------------------------- product in 8-bit integers

static gconv_status_t int8_shape(int64_t M, int64_t N, int64_t K, gconv_dtype_t dtype)
{
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (M < 0 || N < 1 || K < 1) return fail(GCONV_ERR_INVALID_ARG, "int8 product: M >= 0 and N, K >= 1 are needed");
    if (M > kMax - 65536 || N > kMax - 65536)
        return fail(GCONV_ERR_UNSUPPORTED, "int8 product: sizes exceed the library's index range");
    return GCONV_OK;
}

gconv_status_t gconv_quantize_int8(const void *x, int8_t *q, float *scales, int64_t rows, int64_t K, int64_t x_stride,
                                   gconv_dtype_t dtype, void *hip_stream)
{
    gconv::set_last_error("");
    gconv_status_t st = int8_shape(rows, 1, K, dtype);
    if (st != GCONV_OK || (st = check_strides(&x_stride, 1)) != GCONV_OK) return st;
    if (K > int64_t(1) << 30 || (double)rows * (double)(K > x_stride ? K : x_stride) >= kCells / 8)
        return fail(GCONV_ERR_UNSUPPORTED, "int8 rows: sizes exceed the library's index range");
    if (rows == 0) return done(hipSuccess, "");
    if (!x || !q || !scales) return fail(GCONV_ERR_INVALID_ARG, "NULL x, q or scales");
    const Range ranges[] = {
        {"q", q, (size_t)(rows * K), true},
        {"scales", scales, 4 * (size_t)rows, true},
        {"x", x, extent(rows, x_stride, 1, 0, 1, 0, K, elem(dtype)), false},
    };
    if ((st = check_ranges(ranges, sizeof(ranges) / sizeof(ranges[0]))) != GCONV_OK) return st;
    if (!gconv::quantize_fits(rows))
        return fail(GCONV_ERR_UNSUPPORTED, "int8 rows: the call needs more threads than a launch takes");
    const gconv::QuantizeArgs a = {x, q, scales, rows, K, x_stride, (int)dtype, (hipStream_t)hip_stream};
    const char *kname = "";
    const hipError_t err = gconv::launch_quantize(a, &kname);
    return done(err, kname);
}

gconv_status_t gconv_matmul_int8(const int8_t *q, const float *scales, const int8_t *w, const float *w_scales, const void *bias,
                                 void *y, const int64_t *shape, gconv_dtype_t dtype, void *hip_stream)
{
    gconv::set_last_error("");
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    const int64_t M = shape[0], N = shape[1], K = shape[2];
    gconv_status_t st = int8_shape(M, N, K, dtype);
    if (st != GCONV_OK) return st;
    if (K > gconv::kInt8MaxK)
        return fail(GCONV_ERR_UNSUPPORTED, "int8 product: K = %lld, sums of at most %lld products stay in 32 bits", (long long)K,
                    (long long)gconv::kInt8MaxK);
    if (M == 0) return done(hipSuccess, "");
    if (!q || !scales || !w || !w_scales || !y) return fail(GCONV_ERR_INVALID_ARG, "NULL q, scales, w, w_scales or y");
    const Range ranges[] = {
        {"y", y, elem(dtype) * (size_t)(M * N), true},
        {"q", q, (size_t)(M * K), false},
        {"scales", scales, 4 * (size_t)M, false},
        {"w", w, (size_t)(N * K), false},
        {"w_scales", w_scales, 4 * (size_t)N, false},
        {"bias", bias, elem(dtype) * (size_t)N, false},
    };
    if ((st = check_ranges(ranges, sizeof(ranges) / sizeof(ranges[0]))) != GCONV_OK) return st;
    if (!gconv::matmul_int8_fits(M, N))
        return fail(GCONV_ERR_UNSUPPORTED, "int8 product: the call needs more threads than a launch takes");
    const gconv::MatmulInt8Args a = {q, w, scales, w_scales, bias, y, M, N, K, (int)dtype, (hipStream_t)hip_stream};
    const char *kname = "";
    const hipError_t err = gconv::launch_matmul_int8(a, &kname);
    return done(err, kname);
}

}  // extern "C"
