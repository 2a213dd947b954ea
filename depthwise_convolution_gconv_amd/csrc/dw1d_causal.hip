// dw1d_causal.hip -- causal depthwise conv1d over (batch, steps, channels) that carries
// its state: prompts, gradients and single tokens.
//
//     z[b,t,c] = bias[c] + sum_k w[c,0,k] xs[b, t-(K-1)+k, c],   y = z or z / (1 + exp(-z))
//
// where xs[b, -1 .. -(K-1)] are the K-1 inputs before the first token (the state, or
// zeros).  The state after n tokens is xs[b, n-(K-1) .. n-1].  Tokens from lengths[b] on
// are padding: their y is zero, and neither the state nor a gradient depends on them.
//
// causal_run<T, K>: K <= 4.  Lanes run along channels in 16-byte loads, a thread slides
//   its K taps down kRun tokens in registers.  Bound by HBM: 79 us for 2 x 8192 x 6144 in
//   bf16, 403 MB, 5.1 TB/s.
// causal_tile<T>: any K <= 64.  64 channels x 64 tokens and the K-1 inputs before them in
//   LDS as fp32; a thread takes 16 tokens of a channel and goes through the taps 4 at a
//   time, so 19 LDS reads feed 64 multiplications.
// causal_bwd_tile<T, NT>: one tile of the gradients, 32 channels x 64 tokens: z is computed
//   again, dz = dy act'(z) goes to LDS with the K-1 rows behind the tile, then dx is the
//   correlation of dz with the reversed taps and dw, db are the tile's sums, which a second
//   kernel adds over the tiles in a fixed order.  Bound by vector instructions: 32 us by kernel
//   trace, and 4 for the sum, for 8 x 1024 x 512 in fp32 with 31 taps (about 1500 a wave, 950 of
//   them the products; 50 MB take 8 us).  64 channels a tile, two workgroups a compute unit, took 41 us.
// causal_step<T, KS>: one token; the state moves up by one row in place.
#include <algorithm>

#include "seq.hpp"
#include "vecio.hpp"

namespace gconv {
namespace {

constexpr int kThreads = 256;

// 1 / (1 + exp(-z)).  16-bit tensors take the hardware's exponential and reciprocal (relative
// error 2^-21 at |z| = 8, far below half a step).  fp32 ones carry what the product z log2(e)
// loses, exp(-z) = 2^t (1 + ln2 err), and give the reciprocal a Newton step: a few ulp, at half
// the instructions of the library's exponential and a division.
template <typename T> __device__ __forceinline__ float sigmoid(float z)
{
    if constexpr (sizeof(T) == 4) {
        constexpr float hi = 1.44269502f, lo = 1.92596303e-8f, ln2 = 0.693147182f;     // log2(e) = hi + lo
        const float t = -z * hi, err = fmaf(-z, lo, fmaf(-z, hi, -t));
        const float e = __builtin_amdgcn_exp2f(t), d = 1.0f + (fabsf(t) < 126.0f ? fmaf(e, ln2 * err, e) : e);
        const float r = __builtin_amdgcn_rcpf(d);
        return d > 0x1p126f ? r : fmaf(r, fmaf(-d, r, 1.0f), r);     // the step would make NaN of infinity
    } else {
        return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    }
}

template <typename T> __device__ __forceinline__ float silu(float z) { return z * sigmoid<T>(z); }

// d silu(z) / dz
template <typename T> __device__ __forceinline__ float silu_grad(float z)
{
    const float s = sigmoid<T>(z);
    return s * (1.0f + z * (1.0f - s));
}

__device__ __forceinline__ int seq_len(const int32_t *lengths, int64_t b, int64_t T)
{
    if (!lengths) return (int)T;
    const int n = lengths[b];
    return n < 0 ? 0 : n > T ? (int)T : n;
}

// Pointer to xs[b, t, c] (t >= -(K-1)): an input, a state row, or nullptr for a zero.
template <typename T>
__device__ __forceinline__ const T *xs_at(const CausalArgs &a, int64_t b, int64_t t, int64_t c)
{
    if (t >= 0) return (const T *)a.x + b * a.xsb + t * a.xst + c;
    return a.s0 ? (const T *)a.s0 + (b * (a.K - 1) + t + a.K - 1) * a.C + c : nullptr;
}

constexpr int kRun = 16;    // tokens for each thread of causal_run (2 x 8192 x 6144: 82.3 us a call, 83.3 with 24, 87.5 with 32)

template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
causal_run(const CausalArgs a, int cx, int cblocks, int tblocks)
{
    constexpr int VE = 16 / sizeof(T);
    const int ty = threadIdx.x / cx;                       // cx channel runs by 256 / cx token runs
    int64_t id = blockIdx.x;
    const int cb = (int)(id % cblocks);
    id /= cblocks;
    const int tb = (int)(id % tblocks);
    const int64_t b = id / tblocks;
    const int64_t c = ((int64_t)cb * cx + threadIdx.x % cx) * VE;
    const int t0 = (tb * (kThreads / cx) + ty) * kRun, T_in = (int)a.T;
    if (c >= a.C) return;
    const int left = (int)min(a.C - c, (int64_t)VE), n = seq_len(a.lengths, b, a.T);

    if (t0 == 0 && a.sf) {   // the state after the sequence
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const T *src = xs_at<T>(a, b, (int64_t)n - (K - 1) + j, c);
            const Run<T, VE> r = load_raw<T, VE>(src, src ? left : 0);
            store_raw<T, VE>((T *)a.sf + (b * (K - 1) + j) * a.C + c, left, r);
        }
    }
    if (t0 >= T_in) return;
    float w[VE * K], z0[VE];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        float f[VE];
        load_run<T, VE>((const T *)a.w + c * K + j * VE, left * K - j * VE, f);
#pragma unroll
        for (int e = 0; e < VE; ++e) w[j * VE + e] = f[e];
    }
    load_run<T, VE>((const T *)a.bias + c, a.bias ? left : 0, z0);

    float win[K][VE];        // xs of the K tokens up to the current one
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
        const T *src = xs_at<T>(a, b, (int64_t)t0 - (K - 1) + j, c);
        load_run<T, VE>(src, src ? left : 0, win[j]);
    }
    const T *xp = (const T *)a.x + b * a.xsb + (int64_t)t0 * a.xst + c;
    T *yp = (T *)a.y + (b * a.T + t0) * a.C + c;
    constexpr int U = 8;     // rows in flight
#pragma unroll
    for (int t1 = 0; t1 < kRun; t1 += U) {
        Run<T, VE> xr[U];
#pragma unroll
        for (int u = 0; u < U; ++u) xr[u] = load_raw<T, VE>(xp + (int64_t)(t1 + u) * a.xst, t0 + t1 + u < T_in ? left : 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t1 + u;
            float y[VE];
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                win[K - 1][e] = to_f32(xr[u].v[e]);
                float z = z0[e];
#pragma unroll
                for (int j = 0; j < K; ++j) z = fmaf(w[e * K + j], win[j][e], z);
                y[e] = t0 + t < n ? (a.silu ? silu<T>(z) : z) : 0.0f;
            }
            if (t0 + t < T_in) store_run<T, VE>(yp + (int64_t)t * a.C, left, y);
#pragma unroll
            for (int j = 0; j < K - 1; ++j)
#pragma unroll
                for (int e = 0; e < VE; ++e) win[j][e] = win[j + 1][e];
        }
    }
}

constexpr int kCT = 64;     // channels of a tile (lanes)
constexpr int kTT = 64;     // tokens of a tile
constexpr int kWaves = kThreads / 64;

// acc[r] += sum over N taps from k on of w[k] xs[row0 + r + k], through a register window.
template <int R, bool REV, int S, int C, int N>
__device__ __forceinline__ void taps_of(const float *xs, const float *ws, int K, int k, int lane, float (&acc)[R])
{
    float x[R + N - 1], w[N];
#pragma unroll
    for (int i = 0; i < R + N - 1; ++i) x[i] = xs[(k + i) * S + lane];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = ws[(REV ? K - 1 - k - i : k + i) * C + lane];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = fmaf(x[r + i], w[i], acc[r]);
}

// The same over all K taps, 4 at a time, for R rows of the staged inputs (stride S) and
// filters (stride C); REV reads the taps from the end.
template <int R, bool REV, int S = kCT, int C = kCT>
__device__ __forceinline__ void taps(const float *xs, const float *ws, int K, int lane, float (&acc)[R])
{
    int k = 0;
    for (; k + 4 <= K; k += 4) taps_of<R, REV, S, C, 4>(xs, ws, K, k, lane, acc);
    if (K - k == 3) taps_of<R, REV, S, C, 3>(xs, ws, K, k, lane, acc);
    else if (K - k == 2) taps_of<R, REV, S, C, 2>(xs, ws, K, k, lane, acc);
    else if (K - k == 1) taps_of<R, REV, S, C, 1>(xs, ws, K, k, lane, acc);
}

// Stages `rows` rows of 64 channels from row(r) (nullptr: zeros) as fp32.  T elements go in
// runs of VE; UN runs of a thread are in flight together.
template <typename T, typename F>
__device__ __forceinline__ void stage(float *dst, int rows, int64_t c0, int64_t C, F row)
{
    constexpr int VE = 16 / sizeof(T), PR = kCT / VE, UN = 4;
    for (int base = 0; base < rows * PR; base += UN * kThreads) {
        Run<T, VE> v[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int i = base + u * kThreads + (int)threadIdx.x, r = i / PR;
            const int64_t c = c0 + i % PR * VE;
            const T *src = i < rows * PR ? row(r) : nullptr;
            v[u] = load_raw<T, VE>(src + c, src ? (int)max((int64_t)0, min(C - c, (int64_t)VE)) : 0);
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int i = base + u * kThreads + (int)threadIdx.x;
            if (i < rows * PR) {
#pragma unroll
                for (int e = 0; e < VE; ++e) dst[i / PR * kCT + i % PR * VE + e] = to_f32(v[u].v[e]);
            }
        }
    }
}

// The same with ROWS known: the loads, then what they brought, so that several stagings wait
// together.
template <typename T, int ROWS, int CT, int S> struct Staged {
    static constexpr int VE = 16 / sizeof(T), PR = CT / VE, NR = (ROWS * PR + kThreads - 1) / kThreads;
    RunVec<T, VE> v[NR];
    // all: every one of the ROWS rows exists, row r at first + r * stride.
    template <typename F>
    __device__ __forceinline__ void load(int64_t c0, int64_t C, bool all, const T *first, int64_t stride, F row)
    {
        const int64_t c = c0 + threadIdx.x % PR * VE;
        const int left = (int)min(C - c, (int64_t)VE);
        if (all && c0 + CT <= C) {
            const T *p = first + (int64_t)(threadIdx.x / PR) * stride + c;
#pragma unroll
            for (int u = 0; u < NR; ++u)
                if ((u + 1) * kThreads <= ROWS * PR || u * kThreads + (int)threadIdx.x < ROWS * PR)
                    v[u] = *reinterpret_cast<const RunVec<T, VE> *>(p + u * (kThreads / PR) * stride);
        } else {
#pragma unroll
            for (int u = 0; u < NR; ++u) v[u] = RunVec<T, VE>{};
#pragma unroll
            for (int u = 0; u < NR; ++u) {
                const T *src = row((u * kThreads + (int)threadIdx.x) / PR);
                if (src && left > 0) v[u] = load_words<T, VE>(src + c, left);
            }
        }
    }
    __device__ __forceinline__ void put(float *dst) const
    {
#pragma unroll
        for (int u = 0; u < NR; ++u) {
            const int r = (u * kThreads + (int)threadIdx.x) / PR;
            if (r >= ROWS) break;
            const Run<T, VE> x = __builtin_bit_cast(Run<T, VE>, v[u]);
            float *p = dst + r * S + threadIdx.x % PR * VE;
#pragma unroll
            for (int e = 0; e < VE; e += 4)
                *reinterpret_cast<float4 *>(p + e) = float4{to_f32(x.v[e]), to_f32(x.v[e + 1]), to_f32(x.v[e + 2]), to_f32(x.v[e + 3])};
        }
    }
};

// Filters of CT channels as [K][CT], K <= KM: the loads, then what they brought.
template <typename T, int CT, int KM> struct StagedTaps {
    static constexpr int NR = (CT * KM + kThreads - 1) / kThreads;
    T v[NR];
    __device__ __forceinline__ void load(const CausalArgs &a, int64_t c0)
    {
        const int total = (int)min(a.C - c0, (int64_t)CT) * (int)a.K;
#pragma unroll
        for (int u = 0; u < NR; ++u) {
            const int i = u * kThreads + threadIdx.x;
            v[u] = (T)0.0f;
            if (i < total) v[u] = ((const T *)a.w)[c0 * a.K + i];
        }
    }
    __device__ __forceinline__ void put(float *ws, int K) const
    {
        const uint32_t inv = ((1u << 19) + K - 1) / K;     // i / K = i inv >> 19 for i < 2^12, K <= 64
#pragma unroll
        for (int u = 0; u < NR; ++u) {
            const int i = u * kThreads + threadIdx.x, c = (int)(i * inv >> 19);
            if (c < CT) ws[(i - c * K) * CT + c] = to_f32(v[u]);
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
causal_tile(const CausalArgs a, int cblocks, int tblocks)
{
    constexpr int R = kTT / kWaves;
    extern __shared__ float sm[];
    const int K = (int)a.K, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float *xs = sm, *ws = sm + (kTT + K - 1) * kCT;
    int64_t id = blockIdx.x;
    const int64_t c0 = id % cblocks * kCT;
    id /= cblocks;
    const int t0 = (int)(id % tblocks) * kTT, T_in = (int)a.T;
    const int64_t b = id / tblocks, c = c0 + lane;
    const int n = seq_len(a.lengths, b, a.T);
    StagedTaps<T, kCT, kCausalMaxK> tp;
    tp.load(a, c0);
    stage<T>(xs, kTT + K - 1, c0, a.C, [&](int r) -> const T * {
        const int t = t0 - (K - 1) + r;
        return t < n ? xs_at<T>(a, b, t, 0) : nullptr;
    });
    tp.put(ws, K);
    __syncthreads();
    if (t0 == 0 && a.sf && c < a.C)
        for (int j = wave; j < K - 1; j += kWaves) {
            const T *src = xs_at<T>(a, b, (int64_t)n - (K - 1) + j, c);
            ((T *)a.sf)[(b * (K - 1) + j) * a.C + c] = src ? *src : (T)0.0f;
        }
    if (c >= a.C) return;
    const float b0 = a.bias ? to_f32(((const T *)a.bias)[c]) : 0.0f;
    float acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = b0;
    taps<R, false>(xs + wave * R * kCT, ws, K, lane, acc);
    T *yp = (T *)a.y + (b * a.T + t0 + wave * R) * a.C + c;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int t = t0 + wave * R + r;
        if (t < T_in) store_nt(yp + (int64_t)r * a.C, from_f32<T>(t < n ? (a.silu ? silu<T>(acc[r]) : acc[r]) : 0.0f));
    }
}

// The gradients' tile: 32 channels x 64 tokens, a wave holds two groups of rows.  Half as
// wide as the forward one so that four workgroups share a compute unit: its three passes
// alternate between LDS and arithmetic.  Rows lie kBS apart: groups 8, 24, 40 or 72 rows apart
// (8 modulo 16) then read the two halves of the 64 banks.
constexpr int kBT = 32, kBS = 36;

// Tile of rows s0 .. s0 + 63 of the inputs with their state (s = -(K-1) .. T-1).
// NT: taps for each wave (K <= 4 NT).
template <typename T, int NT>
__global__ void __launch_bounds__(kThreads)
causal_bwd_tile(const CausalArgs a, int cblocks, int tblocks, int64_t blocks)
{
    constexpr int RZ = NT <= 4 ? 10 : NT == 8 ? 12 : 18;      // rows of z for each group of lanes (8 groups)
    constexpr int R = kTT / 8, NX = 8 * RZ + 4 * NT, ND = 8 * RZ;
    __shared__ __attribute__((aligned(16))) float xs[NX * kBS];   // x at s0 - (K-1) ..
    __shared__ __attribute__((aligned(16))) float dz[ND * kBS];   // dz at s0 ..
    __shared__ float ws[4 * NT * kBT];
    const int K = (int)a.K, lane = threadIdx.x & 31, half = threadIdx.x >> 5 & 1, wave = threadIdx.x >> 6;
    // A contiguous run of tiles on each XCD: neighbours share lines of 16-bit rows, and halo rows.
    int64_t id = (int64_t)(blockIdx.x & 7) * ((blocks + 7) / 8) + (blockIdx.x >> 3);
    if (id >= blocks) return;
    const int64_t c0 = id % cblocks * kBT;
    id /= cblocks;
    const int tb = (int)(id % tblocks), s0 = tb * kTT - (a.s0 ? K - 1 : 0);
    const int64_t b = id / tblocks, c = c0 + lane;
    const int n = seq_len(a.lengths, b, a.T), rows_dz = kTT + K - 1;
    const bool cok = c < a.C;
    const float b0 = a.bias && cok ? to_f32(((const T *)a.bias)[c]) : 0.0f;

    // Rows past what the tile needs are zeroed: the weight sums read them beside zero dz.
    {
        Staged<T, NX, kBT, kBS> sx;
        Staged<T, ND, kBT, kBS> sd;
        StagedTaps<T, kBT, 4 * NT> tp;
        const int x0 = s0 - (K - 1);
        sx.load(c0, a.C, x0 >= 0 && x0 + NX <= n, (const T *)a.x + b * a.xsb + x0 * a.xst, a.xst, [&](int r) -> const T * {
            const int t = s0 - (K - 1) + r;
            return t < n && t >= -(K - 1) && r < rows_dz + K - 1 ? xs_at<T>(a, b, t, 0) : nullptr;
        });
        sd.load(c0, a.C, s0 >= 0 && s0 + ND <= n, (const T *)a.dy + b * a.dysb + s0 * a.dyst, a.dyst, [&](int r) -> const T * {
            const int t = s0 + r;
            return t >= 0 && t < n && r < rows_dz ? (const T *)a.dy + b * a.dysb + (int64_t)t * a.dyst : nullptr;
        });
        tp.load(a, c0);
        sx.put(xs);
        sd.put(dz);
        tp.put(ws, K);
    }
    __syncthreads();

    if (a.silu) {   // dz = dy silu'(z), each element by the thread that reads it here
        const int r0 = NT == 8 ? (wave >> 1) * 4 * RZ + (wave & 1) * RZ + half * 2 * RZ : half * 4 * RZ + wave * RZ;
        float z[RZ];
#pragma unroll
        for (int r = 0; r < RZ; ++r) z[r] = b0;
        taps<RZ, false, kBS, kBT>(xs + r0 * kBS, ws, K, lane, z);
        if (s0 >= 0 && s0 + 8 * RZ <= n) {     // rows past rows_dz are not read
#pragma unroll
            for (int r = 0; r < RZ; ++r) dz[(r0 + r) * kBS + lane] *= silu_grad<T>(z[r]);
        } else {
#pragma unroll
            for (int r = 0; r < RZ; ++r) {
                const int t = s0 + r0 + r;
                if (r0 + r < rows_dz && t >= 0 && t < n) dz[(r0 + r) * kBS + lane] *= silu_grad<T>(z[r]);
            }
        }
        __syncthreads();
    }

    // dx[s] = sum_j dz[s + j] w[K-1-j], and the gradient of the final state's inputs.
    {
        const int r0 = wave * 2 * R + half * R;
        float acc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = 0.0f;
        taps<R, true, kBS, kBT>(dz + r0 * kBS, ws, K, lane, acc);
        // Inside the sequence and away from the final state's inputs a row is its sum.
        if (s0 >= 0 && s0 + kTT <= n - (K - 1)) {
            T *p = (T *)a.dx + (b * a.T + s0 + r0) * a.C + c;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (cok) p[r * a.C] = from_f32<T>(acc[r]);
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int s = s0 + r0 + r;
                if (s >= a.T || !cok) continue;
                float v = s < n ? acc[r] : 0.0f;
                if (a.dsf && s < n && s >= n - (K - 1))
                    v += to_f32(((const T *)a.dsf)[(b * (K - 1) + s - n + K - 1) * a.C + c]);
                if (s >= 0) ((T *)a.dx)[(b * a.T + s) * a.C + c] = from_f32<T>(v);
                else if (a.ds0) ((T *)a.ds0)[(b * (K - 1) + s + K - 1) * a.C + c] = from_f32<T>(v);
            }
        }
    }

    // dw[k] = sum over the tile's tokens of dz[t] xs[t-(K-1)+k]: wave g takes the taps from
    // g NT on, the halves every other eight tokens.  Row i of xs is input s0 - (K-1) + i, so
    // token s0 + i meets tap k at row i + k.
    float acc[NT], accb = 0.0f;
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = 0.0f;
    for (int t = half * 8; t < kTT; t += 16) {
        float x[7 + NT], d[8];
#pragma unroll
        for (int i = 0; i < 7 + NT; ++i) x[i] = xs[(t + wave * NT + i) * kBS + lane];
#pragma unroll
        for (int u = 0; u < 8; ++u) d[u] = dz[(t + u) * kBS + lane];   // zero outside [0, n)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            accb += d[u];
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[j] = fmaf(d[u], x[u + j], acc[j]);
        }
    }
    accb += __shfl_xor(accb, 32);
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] += __shfl_xor(acc[j], 32);
    if (!cok || half) return;
    float *pt = a.ws + (b * tblocks + tb) * (int64_t)(K + 1) * a.C + c;
#pragma unroll
    for (int j = 0; j < NT; ++j)
        if (wave * NT + j < K) pt[(int64_t)(wave * NT + j) * a.C] = acc[j];
    if (wave == 0) pt[(int64_t)K * a.C] = accb;
}

// dw[c,0,k] and db[c] from the tiles' sums: 64 columns of the (K+1) x C sums and 16 slices
// of the tiles for each workgroup, added in a fixed order.
template <typename T>
__global__ void __launch_bounds__(1024)
causal_bwd_reduce(const float *__restrict__ ws, T *__restrict__ dw, T *__restrict__ db, int64_t tiles, int64_t C, int K)
{
    __shared__ float part[16][64];
    const int lane = threadIdx.x & 63, slice = threadIdx.x >> 6;
    const int64_t cols = (K + 1) * C, x = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (x < cols) {
        int64_t g = slice;
        for (; g + 48 < tiles; g += 64) {
            const float v0 = ws[g * cols + x], v1 = ws[(g + 16) * cols + x];
            const float v2 = ws[(g + 32) * cols + x], v3 = ws[(g + 48) * cols + x];
            s += (v0 + v1) + (v2 + v3);
        }
        for (; g < tiles; g += 16) s += ws[g * cols + x];
    }
    part[slice][lane] = s;
    __syncthreads();
    if (slice != 0 || x >= cols) return;
    for (int i = 1; i < 16; ++i) s += part[i][lane];
    const int64_t k = x / C, c = x - k * C;
    if (k < K) dw[c * K + k] = from_f32<T>(s);
    else if (db) db[c] = from_f32<T>(s);
}

// One token for each sequence: 4 channels for each thread.  KS: the number of taps where it
// is small enough for a channel run's filters to be loaded as they lie (0: any number).
template <typename T, int KS>
__global__ void __launch_bounds__(kThreads)
causal_step(const CausalStepArgs a, int cblocks)
{
    constexpr int VE = 4;
    const int64_t b = blockIdx.x / cblocks;
    const int64_t c = ((int64_t)(blockIdx.x % cblocks) * kThreads + threadIdx.x) * VE;
    if (c >= a.C) return;
    const int left = (int)min(a.C - c, (int64_t)VE), K = KS ? KS : (int)a.K;
    const int64_t slot = a.slots ? a.slots[b] : b;
    T *yp = (T *)a.y + b * a.C + c;
    float x[VE], z[VE];
    const T *wp = (const T *)a.w + c * K;
    load_run<T, VE>((const T *)a.x + b * a.xsb + c, left, x);
    load_run<T, VE>((const T *)a.bias + c, a.bias ? left : 0, z);
    float wk[KS ? KS * VE : 1];
    if constexpr (KS > 0) {
#pragma unroll
        for (int j = 0; j < KS; ++j) load_run<T, VE>(wp + j * VE, left * KS - j * VE, *(float(*)[VE])&wk[j * VE]);
    }
    if (slot < 0 || slot >= a.n) {   // no state: nothing to update, the token's output is zero
#pragma unroll
        for (int e = 0; e < VE; ++e) z[e] = 0.0f;
        store_run<T, VE>(yp, left, z);
        return;
    }
    T *sp = (T *)a.state + slot * (K - 1) * a.C + c;
    constexpr int U = 4;     // state rows in flight
#pragma unroll 1
    for (int j0 = 0; j0 < K; j0 += U) {
        Run<T, VE> row[U];
        float w[U][VE];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u;
            row[u] = load_raw<T, VE>(sp + (int64_t)j * a.C, j < K - 1 ? left : 0);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if constexpr (KS > 0) w[u][e] = u < KS ? wk[e * KS + u] : 0.0f;
                else w[u][e] = j < K && e < left ? to_f32(wp[e * K + j]) : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = j0 + u;
            if (j >= K) continue;
            if (j == K - 1) {
#pragma unroll
                for (int e = 0; e < VE; ++e) row[u].v[e] = from_f32<T>(x[e]);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) z[e] = fmaf(w[u][e], to_f32(row[u].v[e]), z[e]);
            if (j > 0) store_raw<T, VE>(sp + (int64_t)(j - 1) * a.C, left, row[u]);
        }
    }
    if (a.silu) {
#pragma unroll
        for (int e = 0; e < VE; ++e) z[e] = silu<T>(z[e]);
    }
    store_run<T, VE>(yp, left, z);
}

// The grid of a call: workgroups along channels and along tokens; cx (up to 4 taps): channel runs
// of a workgroup.
struct Plan {
    int64_t cblocks, tblocks, blocks;
    int cx;
};
Plan plan_fwd(const CausalArgs &a)
{
    Plan p = {};
    if (a.K <= 4) {
        const int64_t runs = ceil_div(a.C, a.dtype == DT_F32 ? 4 : 8);
        for (p.cx = 8; p.cx < kThreads && p.cx < runs;) p.cx *= 2;
        p.cblocks = ceil_div(runs, p.cx);
        p.tblocks = ceil_div(a.T, (int64_t)(kThreads / p.cx) * kRun);
    } else {
        p.cblocks = ceil_div(a.C, kCT);
        p.tblocks = ceil_div(a.T, kTT);
    }
    p.tblocks = std::max<int64_t>(1, p.tblocks);
    p.blocks = a.B * p.cblocks * p.tblocks;
    return p;
}

template <typename T, int K> hipError_t run_short(const CausalArgs &a)
{
    const Plan p = plan_fwd(a);
    hipLaunchKernelGGL((causal_run<T, K>), dim3((unsigned)p.blocks), dim3(kThreads), 0, a.stream, a, p.cx, (int)p.cblocks,
                       (int)p.tblocks);
    return hipGetLastError();
}

template <typename T> hipError_t run_fwd(const CausalArgs &a, const char **kname)
{
    *kname = "causal_run";
    switch (a.K) {
    case 1: return run_short<T, 1>(a);
    case 2: return run_short<T, 2>(a);
    case 3: return run_short<T, 3>(a);
    case 4: return run_short<T, 4>(a);
    default: break;
    }
    *kname = "causal_tile";
    const Plan p = plan_fwd(a);
    hipLaunchKernelGGL((causal_tile<T>), dim3((unsigned)p.blocks), dim3(kThreads),
                       (unsigned)((kTT + 2 * a.K - 1) * kCT * sizeof(float)), a.stream, a, (int)p.cblocks, (int)p.tblocks);
    return hipGetLastError();
}

template <typename T, int NT> hipError_t run_bwd_tile(const CausalArgs &a, const Plan &p)
{
    hipLaunchKernelGGL((causal_bwd_tile<T, NT>), dim3((unsigned)(8 * ceil_div(p.blocks, 8))), dim3(kThreads), 0, a.stream,
                       a, (int)p.cblocks, (int)p.tblocks, p.blocks);
    return hipGetLastError();
}

// Tiles along the sequence: its tokens and, for the state's gradient, the K-1 before them.
int64_t bwd_tblocks(int64_t T, int64_t K) { return ceil_div(T + K - 1, kTT); }

Plan plan_bwd(const CausalArgs &a)
{
    Plan p = {};
    p.cblocks = ceil_div(a.C, kBT);
    p.tblocks = a.s0 ? bwd_tblocks(a.T, a.K) : ceil_div(a.T, kTT);
    p.blocks = a.B * p.tblocks * p.cblocks;
    return p;
}
int64_t reduce_blocks(const CausalArgs &a) { return ceil_div((a.K + 1) * a.C, 64); }

template <typename T> hipError_t run_bwd(const CausalArgs &a, const char **kname)
{
    *kname = "causal_bwd_tile";
    const Plan p = plan_bwd(a);
    hipError_t err = hipSuccess;
    if (p.blocks > 0) {
        if (a.K <= 4) err = run_bwd_tile<T, 1>(a, p);
        else if (a.K <= 8) err = run_bwd_tile<T, 2>(a, p);
        else if (a.K <= 16) err = run_bwd_tile<T, 4>(a, p);
        else if (a.K <= 32) err = run_bwd_tile<T, 8>(a, p);
        else err = run_bwd_tile<T, 16>(a, p);
    }
    if (err != hipSuccess) return err;
    hipLaunchKernelGGL((causal_bwd_reduce<T>), dim3((unsigned)reduce_blocks(a)), dim3(1024), 0, a.stream, a.ws, (T *)a.dw,
                       (T *)a.db, a.B * p.tblocks, a.C, (int)a.K);
    return hipGetLastError();
}

int64_t step_cblocks(const CausalStepArgs &a) { return ceil_div(a.C, kThreads * 4); }

template <typename T> hipError_t run_step(const CausalStepArgs &a)
{
    const int64_t cblocks = step_cblocks(a);
    const dim3 grid((unsigned)(a.B * cblocks)), block(kThreads);
    switch (a.K) {
    case 2: hipLaunchKernelGGL((causal_step<T, 2>), grid, block, 0, a.stream, a, (int)cblocks); break;
    case 3: hipLaunchKernelGGL((causal_step<T, 3>), grid, block, 0, a.stream, a, (int)cblocks); break;
    case 4: hipLaunchKernelGGL((causal_step<T, 4>), grid, block, 0, a.stream, a, (int)cblocks); break;
    default: hipLaunchKernelGGL((causal_step<T, 0>), grid, block, 0, a.stream, a, (int)cblocks); break;
    }
    return hipGetLastError();
}

}  // namespace

bool causal_fits(const CausalArgs &a) { return grid_fits(plan_fwd(a).blocks, kThreads); }
bool causal_bwd_fits(const CausalArgs &a)
{
    return grid_fits(8 * ceil_div(plan_bwd(a).blocks, 8), kThreads) && grid_fits(reduce_blocks(a), 1024);
}
bool causal_step_fits(const CausalStepArgs &a) { return grid_fits(a.B * step_cblocks(a), kThreads); }

hipError_t launch_causal(const CausalArgs &a, const char **kname)
{
    switch (a.dtype) {
    case DT_F32: return run_fwd<float>(a, kname);
    case DT_F16: return run_fwd<_Float16>(a, kname);
    default: return run_fwd<__bf16>(a, kname);
    }
}

size_t causal_bwd_workspace(int64_t B, int64_t T, int64_t C, int64_t K)
{
    return sizeof(float) * (size_t)(B * bwd_tblocks(T, K) * (K + 1) * C);
}

hipError_t launch_causal_bwd(const CausalArgs &a, const char **kname)
{
    switch (a.dtype) {
    case DT_F32: return run_bwd<float>(a, kname);
    case DT_F16: return run_bwd<_Float16>(a, kname);
    default: return run_bwd<__bf16>(a, kname);
    }
}

hipError_t launch_causal_step(const CausalStepArgs &a, const char **kname)
{
    *kname = "causal_step";
    switch (a.dtype) {
    case DT_F32: return run_step<float>(a);
    case DT_F16: return run_step<_Float16>(a);
    default: return run_step<__bf16>(a);
    }
}

}  // namespace gconv
