// rmsnorm.hip -- root-mean-square norm with the residual's addition, in the tensor's
// dtype or as e4m3 with scales, and its gradient.
//
//     h = round(x + residual),   y = weight * h / sqrt(mean(h^2) + eps)
//     e4m3:  s = max(max|y|, 2^-100) / 448 over a row or a block of columns,  q = y / s
//     dx = r (w dy - h r^2 mean(w dy h)) + dh,  r = 1 / sqrt(mean(h^2) + eps)
//     dw = sum over rows of dy h r
//
// A row is read once: TPR threads hold it in registers (8 or 16 elements each, 16-byte
// loads at any alignment) between the sum of squares and the output, so the kernels move
// each input and output once and are bound by HBM.  Rows of up to 128 / 512 / 4096 /
// 16384 columns take 16 / 64 / 256 / 1024 threads (8192 rows of 4096 in bf16 with a residual
// and an e4m3 output: 44 us, 5.3 TB/s; the gradient of 16384 rows of 2048: 46 us and 5 us for
// the sum of 1024 partial rows, 5.3 TB/s together); longer rows are read again for each
// pass (rms_norm_long).  Squares and sums are fp32; h is rounded to the dtype before it is
// squared because it is what the next layer sees as its residual.
#include <algorithm>

#include "seq.hpp"
#include "vecio.hpp"

namespace gconv {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-100f;

__device__ __forceinline__ float sum_lanes(float v, int width)
{
    for (int o = width / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Largest magnitude as bits: as integers NaN > infinity > every number, so a NaN stays.
__device__ __forceinline__ uint32_t max_lanes(uint32_t v, int width)
{
    for (int o = width / 2; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    return v;
}

// Sum over the TPR threads of a row; red: one slot for each wave (TPR > 64).
template <int TPR> __device__ __forceinline__ float sum_row(float v, float *red)
{
    v = sum_lanes(v, TPR < 64 ? TPR : 64);
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += red[i];
    }
    return v;
}

__device__ __forceinline__ float abs_bits_max(uint32_t amax)
{
    const float a = __builtin_bit_cast(float, amax);
    return a < kAmaxFloor ? kAmaxFloor : a;     // NaN stays
}

// VE values divided by the scale, clamped, as e4m3 (round to nearest even), at any byte alignment.
// A quotient, not a product with 1 / scale: values on a border between two e4m3 numbers, which
// rows of few distinct values have many of, would go to the other side.
template <int VE> __device__ __forceinline__ void store_e4m3(uint8_t *dst, int valid, const float (&y)[VE], float scale)
{
    uint32_t w[VE / 4];
#pragma unroll
    for (int e = 0; e < VE / 4; ++e) {
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = y[4 * e + i] / scale;
            f[i] = v > kE4m3Max ? kE4m3Max : v < -kE4m3Max ? -kE4m3Max : v;   // NaN stays
        }
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
        w[e] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], v, true);
    }
    if (valid >= VE) {
        if constexpr (VE == 8) {
            typedef uint32_t bytes8 __attribute__((ext_vector_type(2), aligned(1)));
            bytes8 b;
            b[0] = w[0]; b[1] = w[1];
            *reinterpret_cast<bytes8 *>(dst) = b;
        } else {
            typedef uint32_t bytes4 __attribute__((aligned(1)));
            *reinterpret_cast<bytes4 *>(dst) = w[0];
        }
    } else {
#pragma unroll
        for (int e = 0; e < VE; ++e)
            if (e < valid) dst[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
    }
}

// VE: elements of a 16-byte load; a thread holds NV of them, at columns (v * TPR + its index) * VE.
template <typename T, int TPR, int NV, bool RES, bool Q8>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
rms_norm_rows(const RmsArgs a)
{
    constexpr int VE = 16 / sizeof(T), RPW = TPR < 256 ? 256 / TPR : 1;
    __shared__ float red[TPR > 64 ? TPR / 64 : 1];
    __shared__ uint32_t redq[TPR > 64 ? TPR / 64 : 1];
    const int sub = threadIdx.x % TPR, C = (int)a.C;
    const int64_t row = (int64_t)blockIdx.x * RPW + threadIdx.x / TPR;
    if (RPW > 1 && row >= a.rows) return;      // whole lane groups of a wave, no barrier follows
    const T *xp = (const T *)a.x + row * a.xs;
    const T *wp = (const T *)a.weight;
    float f[NV][VE];
    Run<T, VE> w[NV];
    float ss = 0.0f;
    {
        Run<T, VE> xr[NV], rr[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) xr[v] = load_raw<T, VE>(xp + (v * TPR + sub) * VE, C - (v * TPR + sub) * VE);
        if constexpr (RES) {
            const T *rp = (const T *)a.residual + row * a.rs;
#pragma unroll
            for (int v = 0; v < NV; ++v) rr[v] = load_raw<T, VE>(rp + (v * TPR + sub) * VE, C - (v * TPR + sub) * VE);
        }
#pragma unroll
        for (int v = 0; v < NV; ++v) w[v] = load_raw<T, VE>(wp + (v * TPR + sub) * VE, C - (v * TPR + sub) * VE);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if constexpr (RES) {
#pragma unroll
                for (int e = 0; e < VE; ++e) xr[v].v[e] = from_f32<T>(to_f32(xr[v].v[e]) + to_f32(rr[v].v[e]));
                store_raw<T, VE>((T *)a.h + row * a.C + (v * TPR + sub) * VE, C - (v * TPR + sub) * VE, xr[v]);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                f[v][e] = to_f32(xr[v].v[e]);
                ss = fmaf(f[v][e], f[v][e], ss);
            }
        }
    }
    const float rstd = 1.0f / sqrtf(sum_row<TPR>(ss, red) / (float)C + a.eps);
    uint32_t amax = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            f[v][e] = f[v][e] * rstd * to_f32(w[v].v[e]);
            if constexpr (Q8)     // columns past C count as zero even where rstd is not finite
                if ((v * TPR + sub) * VE + e >= C) f[v][e] = 0.0f;
        }
    if constexpr (!Q8) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            store_run<T, VE>((T *)a.y + row * a.C + (v * TPR + sub) * VE, C - (v * TPR + sub) * VE, f[v]);
    } else {
        uint8_t *qp = (uint8_t *)a.y + row * a.C;
        if (a.block == 0) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < VE; ++e) amax = max(amax, __builtin_bit_cast(uint32_t, f[v][e]) & 0x7fffffffu);
            amax = max_lanes(amax, TPR < 64 ? TPR : 64);
            if constexpr (TPR > 64) {
                if ((threadIdx.x & 63) == 0) redq[threadIdx.x >> 6] = amax;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < TPR / 64; ++i) amax = max(amax, redq[i]);
            }
            const float s = abs_bits_max(amax) / kE4m3Max;
            if (sub == 0) a.scales[row] = s;
#pragma unroll
            for (int v = 0; v < NV; ++v) store_e4m3<VE>(qp + (v * TPR + sub) * VE, C - (v * TPR + sub) * VE, f[v], s);
        } else {
            // A block of columns is held by block / VE neighbouring lanes (a block wider than the row by all of them).
            const int group = min(a.block / VE, TPR < 64 ? TPR : 64);
            const int nb = (C + a.block - 1) / a.block;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                uint32_t am = 0;
#pragma unroll
                for (int e = 0; e < VE; ++e) am = max(am, __builtin_bit_cast(uint32_t, f[v][e]) & 0x7fffffffu);
                am = max_lanes(am, group);
                const int col = (v * TPR + sub) * VE;
                const float s = abs_bits_max(am) / kE4m3Max;
                if (col % a.block == 0 && col < C) a.scales[row * nb + col / a.block] = s;
                store_e4m3<VE>(qp + col, C - col, f[v], s);
            }
        }
    }
}

// Rows beyond 16384 columns: one workgroup reads its row again for each pass.
template <typename T, bool Q8>
__global__ void __launch_bounds__(1024)
rms_norm_long(const RmsArgs a)
{
    constexpr int VE = 16 / sizeof(T), NT = 1024;
    __shared__ float red[NT / 64];
    __shared__ uint32_t redq[NT / 64];
    const int64_t row = blockIdx.x;
    const T *xp = (const T *)a.x + row * a.xs, *wp = (const T *)a.weight;
    const T *rp = a.residual ? (const T *)a.residual + row * a.rs : nullptr;
    auto load = [&](int64_t col, float (&f)[VE]) {
        const int left = (int)min(a.C - col, (int64_t)VE);
        load_run<T, VE>(xp + col, left, f);
        if (rp) {
            float r[VE];
            load_run<T, VE>(rp + col, left, r);
#pragma unroll
            for (int e = 0; e < VE; ++e) f[e] = to_f32(from_f32<T>(f[e] + r[e]));
        }
    };
    float ss = 0.0f, f[VE], w[VE];
    for (int64_t col = threadIdx.x * VE; col < a.C; col += NT * VE) {
        load(col, f);
        if (rp) store_run<T, VE>((T *)a.h + row * a.C + col, (int)min(a.C - col, (int64_t)VE), f);
#pragma unroll
        for (int e = 0; e < VE; ++e) ss = fmaf(f[e], f[e], ss);
    }
    const float rstd = 1.0f / sqrtf(sum_row<NT>(ss, red) / (float)a.C + a.eps);
    auto norm = [&](int64_t col) {
        load(col, f);
        load_run<T, VE>(wp + col, (int)min(a.C - col, (int64_t)VE), w);
#pragma unroll
        for (int e = 0; e < VE; ++e) f[e] = col + e < a.C ? f[e] * rstd * w[e] : 0.0f;
    };
    if constexpr (!Q8) {
        for (int64_t col = threadIdx.x * VE; col < a.C; col += NT * VE) {
            norm(col);
            store_run<T, VE>((T *)a.y + row * a.C + col, (int)min(a.C - col, (int64_t)VE), f);
        }
    } else {
        uint8_t *qp = (uint8_t *)a.y + row * a.C;
        uint32_t amax = 0;
        float s = 0.0f;
        if (a.block == 0) {
            for (int64_t col = threadIdx.x * VE; col < a.C; col += NT * VE) {
                norm(col);
#pragma unroll
                for (int e = 0; e < VE; ++e) amax = max(amax, __builtin_bit_cast(uint32_t, f[e]) & 0x7fffffffu);
            }
            amax = max_lanes(amax, 64);
            if ((threadIdx.x & 63) == 0) redq[threadIdx.x >> 6] = amax;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NT / 64; ++i) amax = max(amax, redq[i]);
            s = abs_bits_max(amax) / kE4m3Max;
            if (threadIdx.x == 0) a.scales[row] = s;
        }
        const int64_t nb = a.block ? (a.C + a.block - 1) / a.block : 1;
        // Whole waves stay in the loop: a block's lanes exchange their maxima.
        for (int64_t c0 = 0; c0 < a.C; c0 += NT * VE) {
            const int64_t col = c0 + threadIdx.x * VE;
#pragma unroll
            for (int e = 0; e < VE; ++e) f[e] = 0.0f;
            if (col < a.C) norm(col);
            if (a.block) {
                uint32_t am = 0;
#pragma unroll
                for (int e = 0; e < VE; ++e) am = max(am, __builtin_bit_cast(uint32_t, f[e]) & 0x7fffffffu);
                am = max_lanes(am, a.block / VE);
                s = abs_bits_max(am) / kE4m3Max;
                if (col % a.block == 0 && col < a.C) a.scales[row * nb + col / a.block] = s;
            }
            if (col < a.C) store_e4m3<VE>(qp + col, (int)min(a.C - col, (int64_t)VE), f, s);
        }
    }
}

// ---------------------------------------------------------------- gradient

constexpr int kBwdGroups = 1024;   // workgroups, each with one row of partial weight gradients

// Workgroups walk rows with a stride; the weight gradient of a thread's columns stays in
// its registers over all of them and leaves once, as one row of fp32 partial sums.  1024 threads
// have 128 registers each: with 16 fp32 columns a thread 12 go to scratch memory (16-bit: 2), and
// 2000 rows of 12000 with dh take 94 us in fp32, 4.1 TB/s.
template <typename T, int TPR, int NV>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
rms_bwd_rows(const RmsBwdArgs a)
{
    constexpr int VE = 16 / sizeof(T), RPW = TPR < 256 ? 256 / TPR : 1, NW = TPR > 64 ? TPR / 64 : 1;
    __shared__ float red[2][2][NW];
    __shared__ float part[RPW > 1 ? RPW : 1][RPW > 1 ? TPR * NV * VE : 1];
    const int sub = threadIdx.x % TPR, C = (int)a.C, slot = threadIdx.x / TPR;
    float w[NV][VE], dw[NV][VE];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        load_run<T, VE>((const T *)a.weight + (v * TPR + sub) * VE, C - (v * TPR + sub) * VE, w[v]);
#pragma unroll
        for (int e = 0; e < VE; ++e) dw[v][e] = 0.0f;
    }
    int flip = 0;
    for (int64_t row0 = (int64_t)blockIdx.x * RPW; row0 < a.rows; row0 += (int64_t)gridDim.x * RPW) {
        const int64_t row = row0 + slot;
        const bool ok = row < a.rows;          // every lane stays in the loop for the exchanges
        Run<T, VE> hr[NV], dr[NV], er[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = (v * TPR + sub) * VE, left = ok ? C - col : 0;
            hr[v] = load_raw<T, VE>((const T *)a.h + row * a.hs + col, left);
            dr[v] = load_raw<T, VE>((const T *)a.dy + row * a.dys + col, left);
        }
        if (a.dh) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int col = (v * TPR + sub) * VE;
                er[v] = load_raw<T, VE>((const T *)a.dh + row * a.dhs + col, ok ? C - col : 0);
            }
        }
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float h = to_f32(hr[v].v[e]);
                s1 = fmaf(h, h, s1);
                s2 = fmaf(w[v][e] * to_f32(dr[v].v[e]), h, s2);
            }
        s1 = sum_lanes(s1, TPR < 64 ? TPR : 64);
        s2 = sum_lanes(s2, TPR < 64 ? TPR : 64);
        if constexpr (TPR > 64) {
            // Two buffers in turn: a wave a row ahead does not overwrite what others still read.
            if ((threadIdx.x & 63) == 0) {
                red[flip][0][threadIdx.x >> 6] = s1;
                red[flip][1][threadIdx.x >> 6] = s2;
            }
            __syncthreads();
            s1 = s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                s1 += red[flip][0][i];
                s2 += red[flip][1][i];
            }
            flip ^= 1;
        }
        const float r = 1.0f / sqrtf(s1 / (float)C + a.eps), k = r * r * (s2 / (float)C);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int col = (v * TPR + sub) * VE;
            float dx[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float h = to_f32(hr[v].v[e]), d = to_f32(dr[v].v[e]);
                dx[e] = r * (w[v][e] * d - h * k);
                if (a.dh) dx[e] += to_f32(er[v].v[e]);
                if (ok) dw[v][e] = fmaf(d, h * r, dw[v][e]);
            }
            if (ok) store_run<T, VE>((T *)a.dx + row * a.C + col, C - col, dx);
        }
    }
    float *out = a.ws + (int64_t)blockIdx.x * a.C;
    if constexpr (RPW > 1) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VE; ++e) part[slot][(v * TPR + sub) * VE + e] = dw[v][e];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += 256) {
            float s = part[0][c];
            for (int i = 1; i < RPW; ++i) s += part[i][c];
            out[c] = s;
        }
    } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) store_run<float, 4>(out + (v * TPR + sub) * VE, C - (v * TPR + sub) * VE, *(float(*)[4])&dw[v][0]);
        if constexpr (VE == 8) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
                store_run<float, 4>(out + (v * TPR + sub) * VE + 4, C - (v * TPR + sub) * VE - 4, *(float(*)[4])&dw[v][4]);
        }
    }
}

// Rows beyond 16384 columns: dx row by row, the row's factor r to ws; then the weight
// gradient's partial sums with threads along columns.
template <typename T>
__global__ void __launch_bounds__(1024)
rms_bwd_long(const RmsBwdArgs a, float *rs)
{
    constexpr int VE = 16 / sizeof(T), NT = 1024;
    __shared__ float red[2][NT / 64];
    const int64_t row = blockIdx.x;
    const T *hp = (const T *)a.h + row * a.hs, *dp = (const T *)a.dy + row * a.dys, *wp = (const T *)a.weight;
    float s1 = 0.0f, s2 = 0.0f, h[VE], d[VE], w[VE];
    for (int64_t col = threadIdx.x * VE; col < a.C; col += NT * VE) {
        const int left = (int)min(a.C - col, (int64_t)VE);
        load_run<T, VE>(hp + col, left, h);
        load_run<T, VE>(dp + col, left, d);
        load_run<T, VE>(wp + col, left, w);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            s1 = fmaf(h[e], h[e], s1);
            s2 = fmaf(w[e] * d[e], h[e], s2);
        }
    }
    s1 = sum_row<NT>(s1, red[0]);
    s2 = sum_row<NT>(s2, red[1]);
    const float r = 1.0f / sqrtf(s1 / (float)a.C + a.eps), k = r * r * (s2 / (float)a.C);
    if (threadIdx.x == 0) rs[row] = r;
    for (int64_t col = threadIdx.x * VE; col < a.C; col += NT * VE) {
        const int left = (int)min(a.C - col, (int64_t)VE);
        float e[VE];
        load_run<T, VE>(hp + col, left, h);
        load_run<T, VE>(dp + col, left, d);
        load_run<T, VE>(wp + col, left, w);
        if (a.dh) load_run<T, VE>((const T *)a.dh + row * a.dhs + col, left, e);
#pragma unroll
        for (int i = 0; i < VE; ++i) h[i] = r * (w[i] * d[i] - h[i] * k) + (a.dh ? e[i] : 0.0f);
        store_run<T, VE>((T *)a.dx + row * a.C + col, left, h);
    }
}

template <typename T>
__global__ void __launch_bounds__(256)
rms_bwd_long_dw(const RmsBwdArgs a, const float *rs, int groups)
{
    const int64_t cblocks = (a.C + 255) / 256, g = blockIdx.x / cblocks;
    const int64_t c = blockIdx.x % cblocks * 256 + threadIdx.x;
    if (c >= a.C) return;
    float s = 0.0f;
    for (int64_t row = g; row < a.rows; row += groups)
        s = fmaf(to_f32(((const T *)a.dy)[row * a.dys + c]), to_f32(((const T *)a.h)[row * a.hs + c]) * rs[row], s);
    a.ws[g * a.C + c] = s;
}

// dw from `groups` rows of partial sums: 16 columns and 64 slices of the rows for each
// workgroup, added in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024)
rms_bwd_reduce(const float *__restrict__ ws, T *__restrict__ dw, int64_t C, int groups)
{
    __shared__ float part[64][17];
    const int col = threadIdx.x & 15, slice = threadIdx.x >> 4;
    const int64_t c = (int64_t)blockIdx.x * 16 + col;
    float s = 0.0f;
    if (c < C) {
        int g = slice;
        for (; g + 192 < groups; g += 256) {
            const float v0 = ws[(int64_t)g * C + c], v1 = ws[(int64_t)(g + 64) * C + c];
            const float v2 = ws[(int64_t)(g + 128) * C + c], v3 = ws[(int64_t)(g + 192) * C + c];
            s += (v0 + v1) + (v2 + v3);
        }
        for (; g < groups; g += 64) s += ws[(int64_t)g * C + c];
    }
    part[slice][col] = s;
    __syncthreads();
    if (slice >= 4) return;      // 4 sums of 16 slices, then their sum by lanes
    s = 0.0f;
    for (int i = 0; i < 16; ++i) s += part[slice + 4 * i][col];
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (slice == 0 && c < C) dw[c] = from_f32<T>(s);
}

// A launch of more than 2^32 - 1 threads would silently lose some: rows go in pieces that fit.
// one(piece) launches the rows of `piece`.
int64_t rows_of_launch(int rows_each, int threads) { return ((int64_t(1) << 32) - 1) / threads * rows_each; }

template <typename T, typename F> hipError_t in_pieces(const RmsArgs &a, int64_t most, F one)
{
    const int64_t nb = a.block ? ceil_div(a.C, a.block) : 1;
    for (int64_t r = 0; r < a.rows; r += most) {
        RmsArgs p = a;
        p.rows = std::min(most, a.rows - r);
        p.x = (const T *)a.x + r * a.xs;
        if (a.residual) {
            p.residual = (const T *)a.residual + r * a.rs;
            p.h = (T *)a.h + r * a.C;
        }
        p.y = (char *)a.y + r * a.C * (a.scales ? 1 : (int64_t)sizeof(T));
        if (a.scales) p.scales = a.scales + r * nb;
        const hipError_t err = one(p);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

template <typename T, int TPR, int NV> hipError_t run_some_rows(const RmsArgs &a)
{
    constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
    const dim3 grid((unsigned)ceil_div(a.rows, RPW)), block(TPR < 256 ? 256 : TPR);
    if (a.scales) {
        if (a.residual) hipLaunchKernelGGL((rms_norm_rows<T, TPR, NV, true, true>), grid, block, 0, a.stream, a);
        else hipLaunchKernelGGL((rms_norm_rows<T, TPR, NV, false, true>), grid, block, 0, a.stream, a);
    } else {
        if (a.residual) hipLaunchKernelGGL((rms_norm_rows<T, TPR, NV, true, false>), grid, block, 0, a.stream, a);
        else hipLaunchKernelGGL((rms_norm_rows<T, TPR, NV, false, false>), grid, block, 0, a.stream, a);
    }
    return hipGetLastError();
}

template <typename T, int TPR, int NV> hipError_t run_rows(const RmsArgs &a)
{
    constexpr int NT = TPR < 256 ? 256 : TPR;
    return in_pieces<T>(a, rows_of_launch(NT / TPR, NT), run_some_rows<T, TPR, NV>);
}

template <typename T> hipError_t run_norm(const RmsArgs &a, const char **kname)
{
    constexpr int VE = 16 / sizeof(T), X = 8 / VE;   // X: 1 (16-bit) or 2 (fp32)
    *kname = "rms_norm_rows";
    // A scale's columns have to lie in one load of a row's lanes: 16 lanes hold 64 fp32 columns in one, 64 lanes 256.
    if (a.C <= 128 && (X == 1 || a.block <= 16 * VE)) return run_rows<T, 16, X>(a);
    if (a.C <= 512) return run_rows<T, 64, X>(a);
    if (a.C <= 2048) return run_rows<T, 256, X>(a);
    if (a.C <= 4096) return run_rows<T, 256, 2 * X>(a);
    if (a.C <= 8192) return run_rows<T, 1024, X>(a);
    if (a.C <= 16384) return run_rows<T, 1024, 2 * X>(a);
    *kname = "rms_norm_long";
    return in_pieces<T>(a, rows_of_launch(1, 1024), [](const RmsArgs &p) {
        const dim3 grid((unsigned)p.rows), block(1024);
        if (p.scales) hipLaunchKernelGGL((rms_norm_long<T, true>), grid, block, 0, p.stream, p);
        else hipLaunchKernelGGL((rms_norm_long<T, false>), grid, block, 0, p.stream, p);
        return hipGetLastError();
    });
}

// Rows of partial weight gradients a call makes.
int bwd_groups(int64_t rows, int64_t C)
{
    const int64_t rpw = C <= 128 ? 16 : C <= 512 ? 4 : 1;
    // Past 16384 columns a launch has a thread for each of a group's columns: fewer groups from 2^22 columns on.
    const int64_t most = ((int64_t(1) << 32) - 1) / (256 * ceil_div(C, 256));
    return (int)std::min<int64_t>({ceil_div(rows, rpw), kBwdGroups, most});
}

template <typename T, int TPR, int NV> hipError_t run_bwd_rows(const RmsBwdArgs &a, int groups)
{
    hipLaunchKernelGGL((rms_bwd_rows<T, TPR, NV>), dim3((unsigned)groups), dim3(TPR < 256 ? 256 : TPR), 0, a.stream, a);
    return hipGetLastError();
}

template <typename T> hipError_t run_bwd(const RmsBwdArgs &a, const char **kname)
{
    constexpr int X = 8 / (16 / (int)sizeof(T));
    const int groups = bwd_groups(a.rows, a.C);
    *kname = "rms_bwd_rows";
    hipError_t err = hipSuccess;
    if (a.rows > 0) {
        if (a.C <= 128) err = run_bwd_rows<T, 16, X>(a, groups);
        else if (a.C <= 512) err = run_bwd_rows<T, 64, X>(a, groups);
        else if (a.C <= 2048) err = run_bwd_rows<T, 256, X>(a, groups);
        else if (a.C <= 4096) err = run_bwd_rows<T, 256, 2 * X>(a, groups);
        else if (a.C <= 8192) err = run_bwd_rows<T, 1024, X>(a, groups);
        else if (a.C <= 16384) err = run_bwd_rows<T, 1024, 2 * X>(a, groups);
        else {
            *kname = "rms_bwd_long";
            float *rs = a.ws + (int64_t)groups * a.C;
            const int64_t most = rows_of_launch(1, 1024);
            for (int64_t r = 0; r < a.rows; r += most) {
                RmsBwdArgs p = a;
                p.dy = (const T *)a.dy + r * a.dys;
                p.h = (const T *)a.h + r * a.hs;
                if (a.dh) p.dh = (const T *)a.dh + r * a.dhs;
                p.dx = (T *)a.dx + r * a.C;
                hipLaunchKernelGGL((rms_bwd_long<T>), dim3((unsigned)std::min(most, a.rows - r)), dim3(1024), 0, a.stream,
                                   p, rs + r);
                if ((err = hipGetLastError()) != hipSuccess) return err;
            }
            hipLaunchKernelGGL((rms_bwd_long_dw<T>), dim3((unsigned)(ceil_div(a.C, 256) * groups)), dim3(256), 0,
                               a.stream, a, rs, groups);
            err = hipGetLastError();
        }
    }
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((rms_bwd_reduce<T>), dim3((unsigned)ceil_div(a.C, 16)), dim3(1024), 0, a.stream, a.ws,
                       (T *)a.dw, a.C, groups);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const RmsArgs &a, const char **kname)
{
    switch (a.dtype) {
    case DT_F32: return run_norm<float>(a, kname);
    case DT_F16: return run_norm<_Float16>(a, kname);
    default: return run_norm<__bf16>(a, kname);
    }
}

size_t rms_bwd_workspace(int64_t rows, int64_t C, int)
{
    return sizeof(float) * ((size_t)bwd_groups(rows, C) * (size_t)C + (C > 16384 ? (size_t)rows : 0));
}

hipError_t launch_rms_norm_bwd(const RmsBwdArgs &a, const char **kname)
{
    switch (a.dtype) {
    case DT_F32: return run_bwd<float>(a, kname);
    case DT_F16: return run_bwd<_Float16>(a, kname);
    default: return run_bwd<__bf16>(a, kname);
    }
}

}  // namespace gconv
