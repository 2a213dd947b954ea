// linattn.hpp -- the one pass that every direction of linear attention is made of.
//
// With lam = exp(log_decay[head]) and logical token index u = 0 .. n-1,
//
//     out_u = p_scale * sum_{s <= u} lam^(u-s) (a_u . b_s) c_s  +  inter_scale * lam^(u+e0) a_u R_0
//     R_n   = upd_scale * sum_s lam^(n-s-e0) b_s c_s^T  +  lam^n R_0
//
// forward      a = q,  b = k,  c = v,  out = o,  R_0 = initial state, e0 = 1
// gradient dq  a = do, b = v,  c = k,  out = dq, R_0 = initial state transposed, e0 = 1
// gradient dv  a = k,  b = q,  c = do, out = dv, tokens reversed, R_0 = the final state's gradient, e0 = 0
// gradient dk  a = v,  b = do, c = q,  out = dk, the same with the states transposed
//
// R_n of the third line is the initial state's gradient.  In a reversed pass u counts
// from the sequence's last token.
#pragma once

#include "common.hpp"

namespace gconv {

struct LinWalk {
    const void *a, *b, *c;
    void *out;
    int64_t asb, ast, ash, bsb, bst, bsh, csb, cst, csh, osb, ost, osh;   // element strides: batch, token, head
    int32_t ra, rb, rc;          // value heads for each head of a, b, c
    int32_t B, T, H, Da, Dc;     // a, b have Da columns, c and out Dc
    const float *log_decay;      // [H]
    const int32_t *lengths;      // [B] or nullptr: T
    const float *s0;             // state before the first token, or nullptr: zero
    int64_t s0b, s0h, s0r, s0c;  // its element strides: batch, head, row (a's column), column (c's)
    float *sf;                   // state after the last token, or nullptr
    int64_t sfb, sfh, sfr, sfc;
    float *ws;                   // [B*H][nseg] states of Da x Dc
    float *wst;                  // their transposes for another walk (written with them), or nullptr
    float p_scale, inter_scale, upd_scale;
    int32_t e0, reverse;
    int32_t nseg, seg_len;       // segments of seg_len tokens (a multiple of 64), walked by one workgroup each
    int32_t rep;                 // value heads for each key head
    int dtype;                   // of a, b, c
    int out_f32;                 // out is fp32 (partial gradients of a shared head) rather than dtype
    hipStream_t stream;
};

__device__ __forceinline__ double lin_pow64(float g, int e) { return e == 0 ? 1.0 : exp((double)g * e); }
__device__ __forceinline__ float lin_pow(float g, int e) { return (float)lin_pow64(g, e); }

// Length of sequence b.
__device__ __forceinline__ int lin_len(const LinWalk &p, int b)
{
    if (!p.lengths) return p.T;
    const int n = p.lengths[b];
    return n < 0 ? 0 : n > p.T ? p.T : n;
}

// Token of logical index u; indices past the length stand for the padding tokens.
__device__ __forceinline__ int lin_token(const LinWalk &p, int u, int n)
{
    return p.reverse && u < n ? n - 1 - u : u;
}

// Walks that one launch makes together: they share B, T, H, dtype, nseg, seg_len and stream.
constexpr int kMaxWalks = 3;
struct LinWalks {
    LinWalk w[kMaxWalks];
    int32_t count;
    int32_t ndv;                 // column tiles of c
    int64_t blocks;              // workgroups
};

// The kernel of a walk: columns of a and b it holds (64, 128 or 256) and waves of 32 columns of
// c.  Two waves where 64 columns are all there are, but for the widest rows: their staging is
// shared by four, or in 16 bits by eight, which then fill their compute unit as two workgroups
// of four would, with the rows staged once (4 x 11 heads of 198 x 170 over 7984 tokens in bf16:
// 847 us with one workgroup of four waves, 450 with eight; 2 x 2 of 219 x 219 over 4571 in fp16,
// gradients: 213 and 156).
inline int lin_wide(int64_t Da) { return Da <= 64 ? 64 : Da <= 128 ? 128 : 256; }
inline int lin_waves(int64_t Da, int64_t Dc, int dtype)
{
    if (Da > 128) return Dc > 128 && dtype != DT_F32 ? 8 : 4;
    return Dc <= 64 ? 2 : 4;
}
inline int64_t lin_tiles(int64_t Da, int64_t Dc, int dtype) { return ceil_div(Dc, 32 * lin_waves(Da, Dc, dtype)); }

// Walks that one launch can make: one kernel, and one number of workgroups for each.
inline bool lin_alike(int64_t Da, int64_t Dc, int64_t Ea, int64_t Ec, int dtype)
{
    return lin_wide(Da) == lin_wide(Ea) && lin_waves(Da, Dc, dtype) == lin_waves(Ea, Ec, dtype) &&
           lin_tiles(Da, Dc, dtype) == lin_tiles(Ea, Ec, dtype);
}

// The walks of all segments, outputs (full) or local states only, for each dtype; all alike.
hipError_t run_lin_walks_f32(const LinWalks &all, bool full);
hipError_t run_lin_walks_f16(const LinWalks &all, bool full);
hipError_t run_lin_walks_bf16(const LinWalks &all, bool full);

// Workgroups of a walk (Da, Dc) for outputs that a compute unit holds at once.
int lin_held_f32(int64_t Da, int64_t Dc);
int lin_held_f16(int64_t Da, int64_t Dc);
int lin_held_bf16(int64_t Da, int64_t Dc);

// Up to this many segments, each walk adds up the local states before its own, and the last
// one writes sf: a mean of half as many reads as there are segments, and no scan.
constexpr int kFoldSegs = 8;
constexpr int kMaxSeg = 1024;    // segments of a sequence at most

// The segment states (nseg > 1): local sums into ws, the first with what is left of s0, then
// past kFoldSegs the scan that turns them into the states before each segment but the first
// and writes sf.  The first `summed` walks have states of their own, the others' are the
// transposes that those write.
hipError_t launch_lin_states(const LinWalks &all, int summed, const char **kname);
// The outputs (up to kFoldSegs also sf).
hipError_t launch_lin_walks(const LinWalks &all, const char **kname);
// Scan alone (T == 0: sf = s0), and whether a launch takes it.
hipError_t launch_lin_scan(const LinWalks &all);
bool lin_scan_fits(int64_t count, int64_t heads, int64_t cells);
// out[b,t,g,:] = sum over j < r of part[b,t,g*r+j,:] (contiguous), rounded to dtype; ost: out's
// element strides (batch, token, head).  In as many launches as it takes.
hipError_t launch_lin_group_sum(const float *part, void *out, const int64_t *ost, int64_t B, int64_t T, int Hk, int r,
                                int D, int dtype, hipStream_t stream);

struct LinStep {
    const void *q, *k, *v;
    void *o;
    float *state;
    const float *log_decay;
    const int32_t *slots;
    int64_t qsb, qsh, ksb, ksh, vsb, vsh, osb, osh;
    int64_t n;                   // states in the pool
    int32_t B, Hk, H, Dk, Dv;
    float scale;
    int dtype;
    hipStream_t stream;
};
hipError_t launch_lin_step(const LinStep &p, const char **kname);

}  // namespace gconv
