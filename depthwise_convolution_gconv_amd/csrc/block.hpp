// block.hpp -- host-validated calls of the recurrent block's operators: gated linear
// recurrence, group norm with an activation, product in 8-bit integers.
#pragma once

#include "common.hpp"

namespace gconv {

// h_t = a_t h_(t-1) + sqrt(1 - a_t^2) sigmoid(i_t) x_t,  a_t = exp(log_decay sigmoid(r_t)).
struct GatedArgs {
    const void *x, *r, *i;               // [B][T][C], channels contiguous
    const float *log_decay;              // [C]
    const float *s0;                     // [B][C] or nullptr
    const int32_t *lengths;              // [B] or nullptr: T
    void *h;                             // forward: written; backward: read, [B][T][C] contiguous
    float *sf;                           // final state or nullptr; backward: its gradient
    const void *dh;                      // backward from here on
    const float *dsf;                    // gradient of the final state or nullptr
    void *dx, *dr, *di;                  // contiguous
    float *ds0;                          // or nullptr
    float *dlog;                         // [C]
    int64_t B, T, C;
    int64_t xsb, xst, rsb, rst, isb, ist, hsb, hst, dsb, dst;   // element strides: batch, token
    float *ws;
    int dtype;
    hipStream_t stream;
};
// How a call is laid out over workgroups.
struct GatedPlan {
    int32_t lanes;                       // lanes that share a row, 8 bytes each
    int32_t waves;                       // of a workgroup
    int32_t nseg;                        // segments of a sequence
    int64_t seg_len;                     // tokens of a segment
};
GatedPlan gated_plan(int64_t B, int64_t T, int64_t C, int dtype, bool backward);
size_t gated_workspace(const GatedPlan &g, int64_t B, int64_t C, bool backward);
// Whether the launches and 32-bit offsets of a call take it.
bool gated_fits(const GatedArgs &a, const GatedPlan &g, bool backward);
hipError_t launch_gated(const GatedArgs &a, const GatedPlan &g, const char **kname);
hipError_t launch_gated_bwd(const GatedArgs &a, const GatedPlan &g, const char **kname);

struct GatedStepArgs {
    const void *x, *r, *i;
    const float *log_decay;
    float *state;
    void *h;
    const int32_t *slots;
    int64_t B, C, n, xs, rs, is;
    int dtype;
    hipStream_t stream;
};
bool gated_step_fits(const GatedStepArgs &a);
hipError_t launch_gated_step(const GatedStepArgs &a, const char **kname);

// y = act(weight (x - mean) rstd + bias) with the statistics of a sample's group.
struct GroupNormArgs {
    const void *x;                       // [N][P][C], channels contiguous
    const void *weight, *bias;           // [C]; bias may be nullptr
    void *y;                             // [N][P][C] contiguous; backward: dx
    const void *dy;                      // backward: [N][P][C], channels contiguous
    void *dw, *db;                       // backward: [C]; db may be nullptr
    const float *stats;                  // backward: (mean, rstd) [N][G][2]
    float *stats_out;                    // forward: the same, or nullptr
    const int32_t *lengths;              // [N] or nullptr: P
    void *ws;
    int64_t N, P, C, G;
    int64_t xsb, xst, dsb, dst;          // element strides: sample, position
    float eps;
    int32_t silu;
    int dtype;
    hipStream_t stream;
};
// How a call is laid out: threads of a workgroup, channels of a vector (V), groups and vectors
// of a row of its slab, positions of a thread (K), chunks of a sample's positions, parts of a
// group too wide for one workgroup, samples that a gradients' workgroup takes one after the other;
// whole: a workgroup holds all positions of its sample, and one launch does.
struct GroupNormPlan {
    int32_t whole, threads, V, kg, cols, K, chunks, chunk_rows, parts;
    int64_t range;
};
GroupNormPlan gn_plan(int64_t N, int64_t P, int64_t C, int64_t G, int dtype, bool backward);
size_t gn_chunk_bytes(const GroupNormPlan &g, int64_t N, int64_t G);
size_t gn_workspace(const GroupNormPlan &g, int64_t N, int64_t C, int64_t G, bool backward);
bool gn_fits(const GroupNormArgs &a, const GroupNormPlan &g);
hipError_t launch_group_norm(const GroupNormArgs &a, const GroupNormPlan &g, const char **kname);
hipError_t launch_group_norm_bwd(const GroupNormArgs &a, const GroupNormPlan &g, const char **kname);

// q = rint(x / scale), scale = max|row| / 127.
struct QuantizeArgs {
    const void *x;                       // [M][K], row stride xs
    int8_t *q;                           // [M][K]
    float *scales;                       // [M]
    int64_t M, K, xs;
    int dtype;
    hipStream_t stream;
};
bool quantize_fits(int64_t M);
hipError_t launch_quantize(const QuantizeArgs &a, const char **kname);

// y = (q w^T) qs ws + bias
struct MatmulInt8Args {
    const int8_t *q, *w;                 // [M][K], [N][K]
    const float *qs, *ws;                // [M], [N]
    const void *bias;                    // [N] in the dtype, or nullptr
    void *y;                             // [M][N]
    int64_t M, N, K;
    int dtype;                           // of y and bias
    hipStream_t stream;
};
constexpr int64_t kInt8MaxK = 131071;    // 2^7 2^7 K stays below 2^31
bool matmul_int8_fits(int64_t M, int64_t N);
hipError_t launch_matmul_int8(const MatmulInt8Args &a, const char **kname);

}  // namespace gconv
