// int8.hip -- product in 8-bit integers with a scale for each token and each output channel, and
// the tokens' quantiser:
//     scale_m = max(max|x_m|, 2^-100) / 127,   q = rint(x / scale_m)
//     y[m][n] = (sum over k of q[m][k] w[n][k]) scale_m wscale_n + bias_n
// The sum is exact in int32 (K <= 131071).  It is rounded to fp32, and so is its product with the
// token's scale; that times the channel's scale plus the bias is one fused operation, rounded once,
// and the result is rounded to the dtype.
//
// Two kernels, by the number of tokens:
//   mm_tile  tiles of tokens x channels on the matrix cores (v_mfma_i32_32x32x32_i8), both operands
//            staged 64 bytes of K at a time by loads that go straight to LDS, three stages on their
//            way while one is multiplied;
//   mm_rows  up to 32 tokens: bound by the weights' one read.  A workgroup takes 16 channels, its
//            waves share K, every wave has all its weights' loads in flight at once
//            (v_mfma_i32_16x16x64_i8).
#include <algorithm>

#include "block.hpp"
#include "vecio.hpp"

namespace gconv {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t any16 __attribute__((ext_vector_type(4), aligned(1)));

// ---------------------------------------------------------------- quantiser

constexpr float kTopFloor = 7.888609052210118e-31f;     // 2^-100

// Largest magnitude as bits: NaN is above infinity, so that it is kept.
__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7fffffffu; }

template <typename T, int V> __device__ __forceinline__ uint32_t top_of(const Run<T, V> &r, uint32_t top)
{
#pragma unroll
    for (int k = 0; k < V; ++k) top = max(top, magnitude(to_f32(r.v[k])));
    return top;
}

// x / scale, rounded to fp32 and then to an integer.  x times inv = 1 / scale is off by at most 2^-22 of
// itself, 3.1e-5 for quotients up to 127: where it lies further than that from a border between two integers
// its integer is the quotient's, and only next to one (one vector in some hundred) the quotient is taken.
// 8192 x 4096 in bf16: 21 us, with a division for every value 27.
template <typename T, int V> __device__ __forceinline__ void store_q(int8_t *dst, int valid, const Run<T, V> &r, float scale, float inv)
{
    float v[V], far = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const float t = to_f32(r.v[k]) * inv;
        v[k] = rintf(t);
        far = fmaxf(far, fabsf(t - v[k]));
    }
    if (far >= 0.5f - 4e-5f)
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = rintf(to_f32(r.v[k]) / scale);
    uint32_t w[V / 4] = {};
#pragma unroll
    for (int k = 0; k < V; ++k) w[k / 4] |= ((uint32_t)(int32_t)v[k] & 0xffu) << 8 * (k % 4);
    if (valid >= V) {
        if constexpr (V == 8) {
            typedef uint32_t two __attribute__((ext_vector_type(2), aligned(1)));
            *reinterpret_cast<two *>(dst) = two{w[0], w[1]};
        } else {
            typedef uint32_t one __attribute__((aligned(1)));
            *reinterpret_cast<one *>(dst) = w[0];
        }
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < valid) dst[k] = (int8_t)(w[k / 4] >> 8 * (k % 4));
    }
}

// TPR threads take a row, 256 / TPR rows a workgroup.  NV vectors of a thread stay in registers;
// what a longer row has beyond them is read a second time.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(256) void int8_rows(const T *__restrict__ x, int8_t *__restrict__ q, float *__restrict__ scales,
                                                 int64_t M, int64_t K, int64_t xs)
{
    constexpr int V = 16 / sizeof(T);
    __shared__ uint32_t tops[4];
    const int t = threadIdx.x % TPR;
    const int64_t m = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
    const bool on = m < M;
    const T *const row = x + (on ? m : M - 1) * xs;
    Run<T, V> keep[NV];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t at = ((int64_t)j * TPR + t) * V, left = K - at;
        if (left > 0) {
            keep[j] = load_raw<T, V>(row + at, left < V ? (int)left : V);
            top = top_of<T, V>(keep[j], top);
        }
    }
    for (int64_t at = ((int64_t)NV * TPR + t) * V; at < K; at += TPR * V)
        top = top_of<T, V>(load_raw<T, V>(row + at, K - at < V ? (int)(K - at) : V), top);
#pragma unroll
    for (int d = 32; d; d /= 2) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    if constexpr (TPR == 256) {
        if (threadIdx.x % 64 == 0) tops[threadIdx.x / 64] = top;
        __syncthreads();
        top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
    }
    const float high = __builtin_bit_cast(float, top), scale = (high < kTopFloor ? kTopFloor : high) / 127.0f, inv = 1.0f / scale;
    if (!on) return;
    if (t == 0) scales[m] = scale;
    int8_t *const out = q + m * K;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int64_t at = ((int64_t)j * TPR + t) * V, left = K - at;
        if (left > 0) store_q<T, V>(out + at, left < V ? (int)left : V, keep[j], scale, inv);
    }
    for (int64_t at = ((int64_t)NV * TPR + t) * V; at < K; at += TPR * V) {
        const int valid = K - at < V ? (int)(K - at) : V;
        store_q<T, V>(out + at, valid, load_raw<T, V>(row + at, valid), scale, inv);
    }
}

// ---------------------------------------------------------------- product

struct Mm {
    const int8_t *q, *w;
    const float *qs, *ws;
    const void *bias;                    // [N] in the output's dtype, or nullptr
    void *y;
    int32_t M, N, K;
    int32_t mt, nt;                      // tiles
};

template <typename T> __device__ __forceinline__ float bias_of(const Mm &p, int n)
{
    return p.bias ? to_f32(static_cast<const T *>(p.bias)[n]) : 0.0f;
}

// The sum, scaled: three roundings, written out so that they do not depend on what the compiler contracts.
__device__ __forceinline__ float scaled(int32_t sum, float qs, float ws, float bias)
{
#pragma clang fp contract(off)
    const float t = (float)sum * qs;
    return fmaf(t, ws, bias);
}

// 16 bytes of a row from byte k on; those past K are zero.  Rows of any alignment.
__device__ __forceinline__ uint4 load16(const int8_t *row, int k, int K)
{
    if (k + 16 <= K) return __builtin_bit_cast(uint4, *reinterpret_cast<const any16 *>(row + k));
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (k + i < K) w[i / 4] |= (uint32_t)(uint8_t)row[k + i] << 8 * (i % 4);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kStage = 64;               // bytes of K in a stage
constexpr int kStages = 4;               // stages in LDS: one being read, three on their way
constexpr uint32_t kNowhere = 0x80000000u;

// Tile BM x BN, waves WM x WN of it.  ALIGNED: K a multiple of 16 and rows on 16 bytes; else
// the stages go through registers.
//
// Bound by the matrix cores, at the clock that they leave (1.7 GHz over a row of calls; busy 67% of it),
// and for short K by what stands before and behind the stages of a tile, some 11 us.  8192 x 6144 x 4096
// takes 190 - 215 us (a library's product of that size without scales 187), 8192^3 464 (460).  Measured
// on the way: 2 stages of 128 bytes 250, 4 of 64 bytes 243, rows that leave in whole lines 216.
//
// LDS holds a stage's rows one after the other, 4 pieces of 16 bytes each, piece c of row r at place
// c ^ (r / 4 & 3): a wave reads one piece of 32 rows at a time, and any 16 rows next to each other
// then lie in different banks.
template <typename T, int BM, int BN, int WM, int WN, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN, BM * BN > 128 * 128 ? 1 : 2) void mm_tile(const Mm p)
{
    constexpr int NWAVES = WM * WN, UA = BM * 4 / 64 / NWAVES, UB = BN * 4 / 64 / NWAVES;   // loads of a wave
    constexpr int FM = BM / WM / 32, FN = BN / WN / 32;
    __shared__ uint4 s0[(BM + BN) * 4], s1[(BM + BN) * 4], s2[(BM + BN) * 4], s3[(BM + BN) * 4];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), l32 = lane % 32, hf = lane / 32;
    const int wm = wave / WN, wn = wave % WN;
    // Each XCD takes tiles next to each other: bands of 8 tiles of tokens, channel tile after channel tile.
    const int64_t tiles = (int64_t)p.mt * p.nt, per = (tiles + 7) / 8, id = (int64_t)(blockIdx.x % 8) * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || id >= tiles) return;
    const int band = (int)(id / (8 * (int64_t)p.nt)), rows_of_band = min(8, p.mt - band * 8);
    const int in_band = (int)(id - (int64_t)band * 8 * p.nt);
    const int m0 = (band * 8 + in_band % rows_of_band) * BM, n0 = in_band / rows_of_band * BN;
    const int rows = min(BM, p.M - m0), cols = min(BN, p.N - n0);
    const int8_t *const A = p.q + (int64_t)m0 * p.K, *const B = p.w + (int64_t)n0 * p.K;

    i32x16 acc[FM][FN] = {};
    const __amdgpu_buffer_rsrc_t ar = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(A), (short)0, rows * p.K, 0x00020000);
    const __amdgpu_buffer_rsrc_t br = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(B), (short)0, cols * p.K, 0x00020000);
    // A load fills 16 rows: the lane's row of them, and the piece that goes to its place.
    const int lrow = lane / 4, piece = lane % 4 ^ lrow / 4;
    uint4 held[ALIGNED ? 1 : kStages][UA + UB];      // through registers: four stages on their way

    // Stage k0: straight to LDS (past K: zeros), or into registers.
    auto fetch = [&](uint4 *to, int slot, int k0) {
        const int k = 16 * piece;
        if constexpr (ALIGNED) {
            const bool in = k0 + k < p.K;
#pragma unroll
            for (int i = 0; i < UA; ++i) {
                const int r = (wave * UA + i) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ar, (__attribute__((address_space(3))) void *)(to + r * 4), 16,
                                                         in ? (uint32_t)((r + lrow) * p.K + k) : kNowhere, k0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < UB; ++i) {
                const int r = (wave * UB + i) * 16;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(br, (__attribute__((address_space(3))) void *)(to + (BM + r) * 4), 16,
                                                         in ? (uint32_t)((r + lrow) * p.K + k) : kNowhere, k0, 0, 0);
            }
        } else {
            auto piece16 = [&](const int8_t *row) {
                return k0 + kStage <= p.K ? __builtin_bit_cast(uint4, *reinterpret_cast<const any16 *>(row + k0 + k))
                       : k0 < p.K         ? load16(row, k0 + k, p.K)
                                          : make_uint4(0, 0, 0, 0);
            };
#pragma unroll
            for (int i = 0; i < UA; ++i) held[slot][i] = piece16(A + (int64_t)min((wave * UA + i) * 16 + lrow, rows - 1) * p.K);
#pragma unroll
            for (int i = 0; i < UB; ++i) held[slot][UA + i] = piece16(B + (int64_t)min((wave * UB + i) * 16 + lrow, cols - 1) * p.K);
        }
    };
    auto put = [&](uint4 *to, int slot) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < UA; ++i) to[(wave * UA + i) * 64 + lane] = held[slot][i];
#pragma unroll
            for (int i = 0; i < UB; ++i) to[BM * 4 + (wave * UB + i) * 64 + lane] = held[slot][UA + i];
        }
    };
    // Every wave's next stage is in LDS, and its reads of this one are done.
    auto meet = [&] {
        if constexpr (ALIGNED) {
            static_assert(UA + UB == 4 || UA + UB == 2, "two stages' loads may stay on their way");
            if constexpr (UA + UB == 4) asm volatile("s_waitcnt vmcnt(8) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        } else {
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    // Operands of 32 bytes of K, in two sets: one is read while the other is multiplied.
    uint4 a[2][FM], b[2][FN];
    auto read = [&](const uint4 *from, int kk) {
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const int r = (wn * FN + j) * 32 + l32;
            b[kk][j] = from[(BM + r) * 4 + ((2 * kk + hf) ^ (r / 4 & 3))];
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            const int r = (wm * FM + i) * 32 + l32;
            a[kk][i] = from[r * 4 + ((2 * kk + hf) ^ (r / 4 & 3))];
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto multiply = [&](int kk) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, b[kk][j]), __builtin_bit_cast(i32x4, a[kk][i]),
                                                                  acc[i][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    };
    // One stage out of `now`: its last operands are in registers before the waves meet; behind that the
    // stage four later may come into its place, and the next one's first operands are read under its last
    // products.  Through registers: the stage two later goes to `second`, its slot takes the one six later.
    auto stage = [&](uint4 *now, uint4 *next, uint4 *second, int slot, int k0) {
        read(now, 1);
        multiply(0);
        put(second, slot);
        meet();
        fetch(now, slot, k0 + (ALIGNED ? 4 : 6) * kStage);
        read(next, 0);
        multiply(1);
    };

    // Stages in fours, one buffer each; those past K hold zeros.
    fetch(s0, 0, 0);
    put(s0, 0);
    fetch(s1, 0, kStage);
    put(s1, 0);
    fetch(s2, 0, 2 * kStage);
    fetch(s3, 1, 3 * kStage);
    if constexpr (!ALIGNED) {
        fetch(s0, 2, 4 * kStage);
        fetch(s0, 3, 5 * kStage);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    } else if constexpr (UA + UB == 4) {
        asm volatile("s_waitcnt vmcnt(12)\n\ts_barrier" ::: "memory");
    } else {
        asm volatile("s_waitcnt vmcnt(6)\n\ts_barrier" ::: "memory");
    }
    read(s0, 0);
    for (int k0 = 0; k0 < p.K; k0 += kStages * kStage) {
        stage(s0, s1, s2, 0, k0);
        stage(s1, s2, s3, 1, k0 + kStage);
        stage(s2, s3, s0, 2, k0 + 2 * kStage);
        stage(s3, s0, s1, 3, k0 + 3 * kStage);
    }

    // What is still on its way is zeros for LDS that nobody reads as operands.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

    // Channels are the rows of a block of products: a lane has token l32, channels 8 (r / 4) + 4 hf + r % 4.
    // 32 tokens at a time go through the wave's own piece of LDS, so that rows leave in whole lines; 16-byte
    // unit u of token t's row lies at u ^ t.
    constexpr int CW = FN * 32, UPR = CW * (int)sizeof(T) / 16, PER = (BM + BN) * 4 / (32 * UPR);
    static_assert(PER * 2 >= NWAVES, "the waves' pieces lie in two stages");
    uint4 *const rowsout = (wave < PER ? s0 : s1) + wave % PER * (32 * UPR);
    T *const y = static_cast<T *>(p.y);
    const int nw = n0 + wn * CW;                    // the wave's first channel
    if (nw >= p.N) return;
    const bool whole = nw + CW <= p.N;
    float ws[FN][16], bias[FN][16];
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int n = min(nw + j * 32 + 8 * (r / 4) + 4 * hf + r % 4, p.N - 1);
            ws[j][r] = p.ws[n];
            bias[j][r] = bias_of<T>(p, n);
        }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int mw = m0 + (wm * FM + i) * 32;
        const float qs = p.qs[min(mw + l32, p.M - 1)];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                Run<T, 4> v;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v.v[k] = from_f32<T>(scaled(acc[i][j][4 * g + k], qs, ws[j][4 * g + k], bias[j][4 * g + k]));
                const int byte = (j * 32 + 8 * g + 4 * hf) * (int)sizeof(T);
                char *const to = (char *)(rowsout + l32 * UPR + ((byte / 16) ^ (l32 & (UPR - 1)))) + byte % 16;
                if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(to) = __builtin_bit_cast(uint4, v);
                else *reinterpret_cast<uint2 *>(to) = __builtin_bit_cast(uint2, v);
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the wave's own writes, by any lane
#pragma unroll
        for (int h = 0; h < UPR / 2; ++h) {
            const int at = h * 64 + lane, t = at / UPR, u = at % UPR, m = mw + t;
            const uint4 w = rowsout[t * UPR + (u ^ (t & (UPR - 1)))];
            if (m >= p.M) continue;
            T *const to = y + (int64_t)m * p.N + nw + u * (16 / (int)sizeof(T));
            if (whole) {
                typedef uint32_t out16 __attribute__((ext_vector_type(4), aligned(2)));
                *reinterpret_cast<out16 *>(to) = __builtin_bit_cast(out16, w);
            } else {
                typedef Run<T, 16 / (int)sizeof(T)> Piece;
                const Piece v = __builtin_bit_cast(Piece, w);
#pragma unroll
                for (int k = 0; k < 16 / (int)sizeof(T); ++k)
                    if (nw + u * (16 / (int)sizeof(T)) + k < p.N) to[k] = v.v[k];
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // read before the next 32 tokens are written
    }
}

// MB blocks of 16 tokens, NW waves that share K.
template <typename T, int MB, int NW>
__global__ __launch_bounds__(64 * NW) void mm_rows(const Mm p)
{
    constexpr int UNROLL = 8;
    __shared__ i32x4 sums[NW][MB][64];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), r = lane % 16, g = lane / 16;
    const int n0 = blockIdx.x * 16;
    const int8_t *const w = p.w + (int64_t)min(n0 + r, p.N - 1) * p.K;
    const int8_t *q[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) q[b] = p.q + (int64_t)min(16 * b + r, p.M - 1) * p.K;
    const int steps = (p.K + 63) / 64, each = (steps + NW - 1) / NW, from = wave * each, to = min(from + each, steps);
    i32x4 acc[MB] = {};
    int s = from;
    for (; s + UNROLL <= to && (s + UNROLL) * 64 <= p.K; s += UNROLL) {
        uint4 wv[UNROLL], qv[UNROLL][MB];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            wv[u] = __builtin_bit_cast(uint4, *reinterpret_cast<const any16 *>(w + (s + u) * 64 + 16 * g));
#pragma unroll
            for (int b = 0; b < MB; ++b) qv[u][b] = __builtin_bit_cast(uint4, *reinterpret_cast<const any16 *>(q[b] + (s + u) * 64 + 16 * g));
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int b = 0; b < MB; ++b)
                acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wv[u]), __builtin_bit_cast(i32x4, qv[u][b]), acc[b],
                                                               0, 0, 0);
    }
    for (; s < to; ++s) {
        const uint4 wv = load16(w, s * 64 + 16 * g, p.K);
#pragma unroll
        for (int b = 0; b < MB; ++b)
            acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wv),
                                                           __builtin_bit_cast(i32x4, load16(q[b], s * 64 + 16 * g, p.K)), acc[b], 0, 0, 0);
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) sums[wave][b][lane] = acc[b];
    __syncthreads();
    // Lane: token r, channels 4 g + i.
    for (int b = wave; b < MB; b += NW) {
        i32x4 v = sums[0][b][lane];
#pragma unroll
        for (int k = 1; k < NW; ++k) v += sums[k][b][lane];
        const int m = 16 * b + r;
        if (m >= p.M) continue;
        const float qs = p.qs[m];
        T *const y = static_cast<T *>(p.y) + (int64_t)m * p.N;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 4 * g + i;
            if (n < p.N) y[n] = from_f32<T>(scaled(v[i], qs, p.ws[n], bias_of<T>(p, n)));
        }
    }
}

template <int N> struct Int { static constexpr int value = N; };

template <typename F> hipError_t with_type(int dtype, F &&f)
{
    if (dtype == DT_F32) return f(float{});
    if (dtype == DT_F16) return f(_Float16{});
    return f(__bf16{});
}

}  // namespace

bool quantize_fits(int64_t M) { return grid_fits(M, 256); }

hipError_t launch_quantize(const QuantizeArgs &a, const char **kname)
{
    *kname = "int8_rows";
    const int64_t V = a.dtype == DT_F32 ? 4 : 8;
    return with_type(a.dtype, [&](auto t) {
        typedef decltype(t) E;
        auto run = [&](auto tpr, auto nv) {
            constexpr int R = 256 / tpr.value;
            int8_rows<E, tpr.value, nv.value><<<(unsigned)ceil_div(a.M, R), 256, 0, a.stream>>>((const E *)a.x, a.q, a.scales, a.M, a.K, a.xs);
            return hipGetLastError();
        };
        const int64_t vecs = ceil_div(a.K, V);
        if (vecs <= 128) return run(Int<64>{}, Int<2>{});
        return vecs <= 512 ? run(Int<256>{}, Int<2>{}) : run(Int<256>{}, Int<8>{});
    });
}

namespace {

template <int BM, int BN, int WM, int WN, bool ALIGNED> hipError_t run_tile(Mm p, int dtype, hipStream_t stream)
{
    p.mt = (int32_t)ceil_div(p.M, BM);
    p.nt = (int32_t)ceil_div(p.N, BN);
    const unsigned grid = (unsigned)(8 * ceil_div((int64_t)p.mt * p.nt, 8));
    return with_type(dtype, [&](auto t) {
        mm_tile<decltype(t), BM, BN, WM, WN, ALIGNED><<<grid, 64 * WM * WN, 0, stream>>>(p);
        return hipGetLastError();
    });
}

template <int MB, int NW> hipError_t run_rows(const Mm &p, int dtype, hipStream_t stream)
{
    return with_type(dtype, [&](auto t) {
        mm_rows<decltype(t), MB, NW><<<(unsigned)ceil_div(p.N, 16), 64 * NW, 0, stream>>>(p);
        return hipGetLastError();
    });
}

}  // namespace

bool matmul_int8_fits(int64_t M, int64_t N)
{
    return grid_fits(8 * ceil_div(ceil_div(M, 64) * ceil_div(N, 64), 8), 256) && grid_fits(ceil_div(N, 16), 1024);
}

hipError_t launch_matmul_int8(const MatmulInt8Args &a, const char **kname)
{
    Mm p = {};
    p.q = a.q; p.w = a.w; p.qs = a.qs; p.ws = a.ws; p.bias = a.bias; p.y = a.y;
    p.M = (int32_t)a.M; p.N = (int32_t)a.N; p.K = (int32_t)a.K;
    // Few tokens: 16 x 12288 x 4096 14 us; from 17 on tiles overtake where there are channel tiles enough
    // (32 x 12288 x 4096 21 us and 13, 64 x 12288 x 4096 32 and 13, 32 x 4096 x 4096 8.9 and 9.8).
    if (a.M <= 16 || (a.M <= 32 && a.N < 8192)) {
        *kname = "mm_rows";
        const bool few = ceil_div(a.N, 16) < 512;       // channel groups: more waves share K
        if (a.M <= 16) return few ? run_rows<1, 16>(p, a.dtype, a.stream) : run_rows<1, 4>(p, a.dtype, a.stream);
        return few ? run_rows<2, 8>(p, a.dtype, a.stream) : run_rows<2, 4>(p, a.dtype, a.stream);
    }
    *kname = "mm_tile";
    const bool aligned = a.K % 16 == 0 && (uintptr_t)a.q % 16 == 0 && (uintptr_t)a.w % 16 == 0;
    // Larger tiles where they nearly fill the card.  K = 4096, in bf16: 224 tiles of 256 (3584 x 4096) 60 us and 80
    // in tiles of 128, 128 of them (2048 x 4096) 53 and 45; 192 tiles of 128 (1536 x 2048) 22 us and 27 in tiles
    // of 64, 128 of them (1024 x 2048) 21 and 18.  Unaligned rows: 224 tiles of 128 36 and 41, 192 35 and 31.
    auto tiles = [&](int64_t bm, int64_t bn) { return ceil_div(a.M, bm) * ceil_div(a.N, bn); };
    if (!aligned)
        return tiles(128, 128) >= 208 ? run_tile<128, 128, 2, 2, false>(p, a.dtype, a.stream)
                                      : run_tile<64, 64, 2, 2, false>(p, a.dtype, a.stream);
    if (tiles(256, 256) >= 224) return run_tile<256, 256, 2, 4, true>(p, a.dtype, a.stream);
    return tiles(128, 128) >= 160 ? run_tile<128, 128, 2, 2, true>(p, a.dtype, a.stream) : run_tile<64, 64, 2, 2, true>(p, a.dtype, a.stream);
}

}  // namespace gconv
