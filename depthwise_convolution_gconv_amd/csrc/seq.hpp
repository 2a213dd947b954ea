// seq.hpp -- host-validated calls of the sequence operators next to the convolutions:
// RMS norm and the causal depthwise conv1d.
#pragma once

#include "common.hpp"

namespace gconv {

struct RmsArgs {
    const void *x, *residual, *weight;   // residual may be nullptr
    void *y;                             // dtype, or e4m3 bytes with scales != nullptr
    void *h;                             // x + residual, or nullptr (no residual)
    float *scales;
    int64_t rows, C, xs, rs;             // xs, rs: row strides of x and residual
    int32_t block;                       // columns for each scale; 0: the row
    float eps;
    int dtype;
    hipStream_t stream;
};
hipError_t launch_rms_norm(const RmsArgs &a, const char **kname);

struct RmsBwdArgs {
    const void *dy, *h, *weight, *dh;    // dh may be nullptr
    void *dx, *dw;
    float *ws;
    int64_t rows, C, dys, hs, dhs;
    float eps;
    int dtype;
    hipStream_t stream;
};
size_t rms_bwd_workspace(int64_t rows, int64_t C, int dtype);
hipError_t launch_rms_norm_bwd(const RmsBwdArgs &a, const char **kname);

struct CausalArgs {
    const void *x, *w, *bias, *s0;       // bias, s0 may be nullptr
    void *y, *sf;                        // sf may be nullptr
    const void *dy, *dsf;                // backward: dsf may be nullptr
    void *dx, *dw, *db, *ds0;            // db, ds0 may be nullptr
    float *ws;
    const int32_t *lengths;              // [B] or nullptr: T
    int64_t B, T, C, K, xsb, xst, dysb, dyst;
    int32_t silu;
    int dtype;
    hipStream_t stream;
};
// (fits: whether the launches of a call take it)
bool causal_fits(const CausalArgs &a);
hipError_t launch_causal(const CausalArgs &a, const char **kname);
size_t causal_bwd_workspace(int64_t B, int64_t T, int64_t C, int64_t K);
bool causal_bwd_fits(const CausalArgs &a);
hipError_t launch_causal_bwd(const CausalArgs &a, const char **kname);

struct CausalStepArgs {
    const void *x, *w, *bias;
    void *y, *state;
    const int32_t *slots;
    int64_t B, C, K, n, xsb;
    int32_t silu;
    int dtype;
    hipStream_t stream;
};
bool causal_step_fits(const CausalStepArgs &a);
hipError_t launch_causal_step(const CausalStepArgs &a, const char **kname);

// The thread's error text and last kernel name, held by api.cpp.
void set_last_error(const char *text);
void set_last_kernel(const char *name);

constexpr int kCausalMaxK = 64;
constexpr int64_t kNormMaxRows = (int64_t(1) << 31) - 1;

}  // namespace gconv
