// gated_rec.hip -- gated linear recurrence over (batch, steps, channels):
//     a_t = exp(log_decay[c] sigmoid(r_t)),   h_t = a_t h_(t-1) + sqrt(1 - a_t^2) sigmoid(i_t) x_t,
// its gradients and its form for single tokens.
//
// A recurrence h_t = a_t h_(t-1) + u_t is a composition of affine maps: over any run of tokens
// it is h_out = A h_in + E with A the product of the a_t and E the run's own result from zero.
// A workgroup walks the tokens of one sequence for a stripe of channels, tile after tile: each
// lane takes a run of consecutive tokens for two channels, keeps its a_t and u_t in registers,
// and (A, E) of the runs are joined by lane exchanges within a wave and through LDS across the
// waves.  Then each lane knows the state before its run and writes its h_t.  So the inputs are
// read once and one barrier is needed for a tile; the next tile's loads are in flight meanwhile.
// Where stripes alone do not fill the card a sequence is cut into segments: (A, E) of each come
// first (gated_states), and a walk folds those before its own.
//
// Bound by HBM and, nearly as much, by vector instructions: six of quarter rate (three
// exponentials, two reciprocals, a root) and about 30 others for the 8 bytes of an element.
#include <algorithm>

#include "block.hpp"

namespace gconv {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// Two neighbouring channels as they are stored.
template <typename T> struct Two {
    typedef uint32_t raw;
    typedef uint32_t mem __attribute__((aligned(2)));
    typedef uint16_t one;
};
template <> struct Two<float> {
    typedef uint2 raw;
    typedef uint32_t mem __attribute__((ext_vector_type(2), aligned(4)));
    typedef uint32_t one;
};

__device__ __forceinline__ uint32_t alone(uint32_t v, uint32_t) { return v; }
__device__ __forceinline__ uint2 alone(uint32_t v, uint2) { return make_uint2(v, 0); }
__device__ __forceinline__ uint32_t second(uint32_t w) { return w >> 16; }
__device__ __forceinline__ uint2 second(uint2 w) { return make_uint2(w.y, 0); }

// What a stripe of channels is: whole; the one that C ends in (a pair past the end is read from the
// last pair that exists, its only channel from the second of that); the one channel of C = 1.
enum { kWhole = 0, kEdge = 1, kSingle = 2 };

struct Cols {
    uint32_t at;           // byte offset that is read
    uint32_t to;           // and that is written
    bool has_lo, has_hi;   // which of the two exist
};

template <typename T, int MODE>
__device__ __forceinline__ typename Two<T>::raw load2(const char *base, uint32_t row, const Cols &c)
{
    typedef typename Two<T>::raw raw;
    if constexpr (MODE == kSingle)
        return alone(*reinterpret_cast<const typename Two<T>::one *>(base + (row + c.at)), raw{});
    else
        return __builtin_bit_cast(raw, *reinterpret_cast<const typename Two<T>::mem *>(base + (row + c.at)));
}

template <typename T> __device__ __forceinline__ void split2(uint32_t w, float (&f)[2])
{
    f[0] = to_f32(__builtin_bit_cast(T, (uint16_t)w));
    f[1] = to_f32(__builtin_bit_cast(T, (uint16_t)(w >> 16)));
}
template <> __device__ __forceinline__ void split2<__bf16>(uint32_t w, float (&f)[2])
{
    f[0] = __builtin_bit_cast(float, w << 16);
    f[1] = __builtin_bit_cast(float, w & 0xffff0000u);
}
template <typename T> __device__ __forceinline__ void split2(uint2 w, float (&f)[2])
{
    f[0] = __builtin_bit_cast(float, w.x);
    f[1] = __builtin_bit_cast(float, w.y);
}
template <typename T, int MODE, typename RAW> __device__ __forceinline__ void values(RAW w, const Cols &c, float (&f)[2])
{
    split2<T>(MODE == kEdge && !c.has_hi ? second(w) : w, f);
}

template <typename T, int MODE>
__device__ __forceinline__ void store2(char *base, uint32_t row, const Cols &c, float lo, float hi)
{
    if constexpr (MODE != kWhole) {
        if (c.has_lo) *reinterpret_cast<T *>(base + (row + c.to)) = from_f32<T>(lo);
        if (c.has_hi) *reinterpret_cast<T *>(base + (row + c.to + (uint32_t)sizeof(T))) = from_f32<T>(hi);
    } else {
        typedef T pair __attribute__((ext_vector_type(2)));
        const pair v = {from_f32<T>(lo), from_f32<T>(hi)};
        *reinterpret_cast<typename Two<T>::mem *>(base + (row + c.to)) = __builtin_bit_cast(typename Two<T>::mem, v);
    }
}

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ __forceinline__ float rcp_fast(float v) { return __builtin_amdgcn_rcpf(v); }
__device__ __forceinline__ float sigmoid(float z) { return rcp_fast(1.0f + exp2_fast(-kLog2e * z)); }

// a and 1 - a^2 for a = 2^l, l <= 0.  Near a = 1 the difference is taken by the series of
// 1 - e^w, w = 2 ln(a): up to w = -1/2 seven terms leave 2^-22 of it, and the difference
// itself, from there on, as much.
__device__ __forceinline__ void decay(float l, float &a, float &m)
{
    a = exp2_fast(l);
    const float w = 2.0f * kLn2 * l;
    float s = fmaf(w, 1.0f / 5040, 1.0f / 720);
    s = fmaf(w, s, 1.0f / 120);
    s = fmaf(w, s, 1.0f / 24);
    s = fmaf(w, s, 1.0f / 6);
    s = fmaf(w, s, 0.5f);
    s = fmaf(w, s, 1.0f);
    m = w > -0.5f ? -w * s : fmaf(-a, a, 1.0f);
}

// Tokens of a lane's run: what fits in registers with the next tile's loads beside it.
template <typename T> constexpr int run_len() { return sizeof(T) == 4 ? 4 : 8; }
template <typename T> constexpr int run_len_bwd() { return sizeof(T) == 4 ? 2 : 4; }

// A run's map joined with the one before it.
__device__ __forceinline__ void join_maps(float &A, float &E, float Ab, float Eb)
{
    E = fmaf(A, Eb, E);
    A *= Ab;
}

// Maps of the runs of a wave (64 / LR of them, LR lanes each) -> the map before each run, and in
// its last run's lanes that of the wave.
template <int LR>
__device__ __forceinline__ void scan_wave(int lane, float (&A)[2], float (&E)[2], float (&Ab)[2], float (&Eb)[2])
{
#pragma unroll
    for (int d = LR; d < 64; d *= 2)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float pa = __shfl_up(A[k], d), pe = __shfl_up(E[k], d);
            if (lane >= d) join_maps(A[k], E[k], pa, pe);
        }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float pa = __shfl_up(A[k], LR), pe = __shfl_up(E[k], LR);
        Ab[k] = lane >= LR ? pa : 1.0f;
        Eb[k] = lane >= LR ? pe : 0.0f;
    }
}

struct Walk {
    int64_t B, T, C, seg_len, blocks;
    int32_t nseg, tiles;                 // segments of a sequence, stripes of channels
    const char *x, *r, *i, *dh;
    const char *h_in;
    char *h, *dx, *dr, *di;
    const float *log_decay, *s0;
    float *sf;
    float *maps;                         // (A, E) [B][nseg][C][2]
    float *part;                         // shares of the gradient of log_decay [B * nseg][C]
    const int32_t *lengths;
    int64_t xsb, xst, rsb, rst, isb, ist, hsb, hst, dsb, dst;   // bytes
};

// Workgroup -> (stripe, segment, sequence); neighbouring stripes, which share lines, on one XCD.
__device__ __forceinline__ bool place(const Walk &p, int nseg, int &ct, int &seg, int64_t &b)
{
    const int64_t per = (p.blocks + 7) / 8, id = (int64_t)(blockIdx.x % 8) * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || id >= p.blocks) return false;
    ct = (int)(id % p.tiles);
    const int64_t rest = id / p.tiles;
    seg = (int)(rest % nseg);
    b = rest / nseg;
    return true;
}

__device__ __forceinline__ int64_t live_tokens(const Walk &p, int64_t b)
{
    if (!p.lengths) return p.T;
    const int64_t n = p.lengths[b];
    return n < 0 ? 0 : n > p.T ? p.T : n;
}

template <typename T, int LR>
__device__ __forceinline__ Cols columns(const Walk &p, int ct, int lane, int64_t &c)
{
    c = (int64_t)ct * 2 * LR + 2 * (lane % LR);
    Cols k;
    k.has_lo = c < p.C;
    k.has_hi = c + 1 < p.C;
    k.to = (uint32_t)(c * sizeof(T));
    k.at = (uint32_t)(max((int64_t)0, min(c, p.C - 2)) * sizeof(T));
    return k;
}

// A stride that the compiler does not multiply out in advance: products for every row of a tile
// would fill the scalar registers.
__device__ __forceinline__ int64_t fresh(int64_t v)
{
    asm volatile("" : "+s"(v));
    return v;
}

// State before a segment: the first one's, through the maps of the segments before it.
__device__ __forceinline__ float fold(const Walk &p, int64_t b, int seg, int64_t c, float h)
{
    for (int s = 0; s < seg; ++s) {
        const float2 m = *reinterpret_cast<const float2 *>(p.maps + 2 * ((b * p.nseg + s) * p.C + c));
        h = fmaf(m.x, h, m.y);
    }
    return h;
}

// ---------------------------------------------------------------- forward

template <typename T, int L> struct RawIn { typename Two<T>::raw x[L], r[L], i[L]; };

template <typename T, int MODE, int L>
__device__ __forceinline__ void load_in(const Walk &p, const char *const (&base)[3], int64_t t0, int64_t live, int run, int TS,
                                        const uint32_t (&step)[3], const Cols &col, RawIn<T, L> &raw)
{
    const char *x = base[0] + t0 * p.xst, *r = base[1] + t0 * p.rst, *i = base[2] + t0 * p.ist;
    if (t0 + TS <= live) {
#pragma unroll
        for (int l = 0; l < L; ++l) {
            raw.x[l] = load2<T, MODE>(x, step[0], col);
            raw.r[l] = load2<T, MODE>(r, step[1], col);
            raw.i[l] = load2<T, MODE>(i, step[2], col);
            x += fresh(p.xst);
            r += fresh(p.rst);
            i += fresh(p.ist);
        }
    } else {        // rows past the end are read from the last one
        const int last = (int)(live - 1 - t0);
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const uint32_t row = (uint32_t)min(run * L + l, last);
            raw.x[l] = load2<T, MODE>(x, row * (uint32_t)p.xst, col);
            raw.r[l] = load2<T, MODE>(r, row * (uint32_t)p.rst, col);
            raw.i[l] = load2<T, MODE>(i, row * (uint32_t)p.ist, col);
        }
    }
}

template <typename T, int MODE, int L>
__device__ __forceinline__ void gates(const RawIn<T, L> &raw, const Cols &col, const float (&ld)[2], int live_rows, float (&a)[L][2], float (&u)[L][2])
{
#pragma unroll
    for (int l = 0; l < L; ++l) {
        float x[2], r[2], i[2];
        values<T, MODE>(raw.x[l], col, x);
        values<T, MODE>(raw.r[l], col, r);
        values<T, MODE>(raw.i[l], col, i);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float m;
            decay(ld[k] * sigmoid(r[k]), a[l][k], m);
            u[l][k] = __builtin_amdgcn_sqrtf(m) * (x[k] * sigmoid(i[k]));
        }
        __builtin_amdgcn_sched_barrier(0);      // one token after the other: temporaries of all at once do not fit
    }
    if (live_rows < L)      // tokens that do not exist leave the state alone, whatever was read
#pragma unroll
        for (int l = 0; l < L; ++l)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                a[l][k] = l < live_rows ? a[l][k] : 1.0f;
                u[l][k] = l < live_rows ? u[l][k] : 0.0f;
            }
}

template <typename T, int LR, int NW, int MODE>
__device__ __forceinline__ void walk_body(const Walk &p, int ct, int seg, int64_t b, float4 (*agg)[NW][LR])
{
    constexpr int RW = 64 / LR, L = run_len<T>(), TS = NW * RW * L;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int run = wave * RW + lane / LR;
    int64_t c;
    const Cols col = columns<T, LR>(p, ct, lane, c);
    const int64_t n = live_tokens(p, b), begin = seg * p.seg_len, end = min(begin + p.seg_len, p.T), live = min(end, n);
    const char *const base[3] = {p.x + b * p.xsb, p.r + b * p.rsb, p.i + b * p.isb};
    const uint32_t step[3] = {(uint32_t)(run * L * p.xst), (uint32_t)(run * L * p.rst), (uint32_t)(run * L * p.ist)};
    const uint32_t hrow = (uint32_t)(p.C * sizeof(T));
    char *const out = p.h + b * p.T * (int64_t)hrow;

    RawIn<T, L> raw;
    if (begin < live) load_in<T, MODE, L>(p, base, begin, live, run, TS, step, col, raw);
    float ld[2], carry[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int64_t ck = min(c + k, p.C - 1);
        ld[k] = p.log_decay[ck] * kLog2e;
        carry[k] = fold(p, b, seg, ck, p.s0 ? p.s0[b * p.C + ck] : 0.0f);
    }
    int buf = 0;
    for (int64_t t0 = begin; t0 < live; t0 += TS, buf ^= 1) {
        RawIn<T, L> next;
        if (t0 + TS < live) load_in<T, MODE, L>(p, base, t0 + TS, live, run, TS, step, col, next);
        const bool full = t0 + TS <= live;
        const int rows = full ? L : (int)min((int64_t)L, max((int64_t)0, live - t0 - run * L));
        float a[L][2], u[L][2];
        gates<T, MODE, L>(raw, col, ld, rows, a, u);
        float A[2] = {1.0f, 1.0f}, E[2] = {0.0f, 0.0f}, Ab[2], Eb[2];
#pragma unroll
        for (int l = 0; l < L; ++l)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                A[k] *= a[l][k];
                E[k] = fmaf(a[l][k], E[k], u[l][k]);
            }
        scan_wave<LR>(lane, A, E, Ab, Eb);
        if (lane >= 64 - LR) agg[buf][wave][lane - (64 - LR)] = make_float4(A[0], E[0], A[1], E[1]);
        __syncthreads();
        float h[2] = {carry[0], carry[1]};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float4 m = agg[buf][w][lane % LR];
            h[0] = w == wave ? carry[0] : h[0];
            h[1] = w == wave ? carry[1] : h[1];
            carry[0] = fmaf(m.x, carry[0], m.y);
            carry[1] = fmaf(m.z, carry[1], m.w);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) h[k] = fmaf(Ab[k], h[k], Eb[k]);
        char *o = out + t0 * (int64_t)hrow;
        const uint32_t first = (uint32_t)(run * L) * hrow;
        if (full) {
#pragma unroll
            for (int l = 0; l < L; ++l) {
#pragma unroll
                for (int k = 0; k < 2; ++k) h[k] = fmaf(a[l][k], h[k], u[l][k]);
                store2<T, MODE>(o, first, col, h[0], h[1]);
                o += fresh(hrow);
            }
        } else {
#pragma unroll
            for (int l = 0; l < L; ++l) {
#pragma unroll
                for (int k = 0; k < 2; ++k) h[k] = fmaf(a[l][k], h[k], u[l][k]);
                if (l < rows) store2<T, MODE>(o, first, col, h[0], h[1]);
                o += fresh(hrow);
            }
        }
        raw = next;
    }
    for (int64_t t = max(begin, n) + run; t < end; t += NW * RW)
        store2<T, MODE>(out + t * (int64_t)hrow, 0, col, 0.0f, 0.0f);
    if (p.sf && seg == p.nseg - 1 && threadIdx.x < LR)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (c + k < p.C) p.sf[b * p.C + c + k] = carry[k];
}

template <typename T, int LR, int NW, bool SINGLE>
__global__ __launch_bounds__(64 * NW) void gated_walk(const Walk p)
{
    __shared__ float4 agg[2][NW][LR];
    int ct, seg;
    int64_t b;
    if (!place(p, p.nseg, ct, seg, b)) return;
    if constexpr (SINGLE) walk_body<T, LR, NW, kSingle>(p, ct, seg, b, agg);
    else if ((int64_t)(ct + 1) * 2 * LR <= p.C) walk_body<T, LR, NW, kWhole>(p, ct, seg, b, agg);
    else walk_body<T, LR, NW, kEdge>(p, ct, seg, b, agg);
}

// ---------------------------------------------------------------- (A, E) of segments

// Each run of lanes takes a stretch of the segment of its own; no joins until its end.  Forward:
// maps of h.  Backward (from the sequence's end): maps of c_t = a_t (dh_t + c_(t+1)).
template <typename T, int LR, int NW, bool BWD, int MODE>
__device__ __forceinline__ void states_body(const Walk &p, int ct, int seg, int64_t b, float4 (*agg)[LR])
{
    constexpr int RW = 64 / LR, L = 8;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int run = wave * RW + lane / LR;
    int64_t c;
    const Cols col = columns<T, LR>(p, ct, lane, c);
    const int64_t n = live_tokens(p, b), stretch = p.seg_len / (NW * RW);
    // Positions count from the start of the walk: token q forward, n - 1 - q backward.
    const int64_t first = seg * p.seg_len + run * stretch, past = min(first + stretch, n);
    float ld[2], A[2] = {1.0f, 1.0f}, E[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 2; ++k) ld[k] = p.log_decay[min(c + k, p.C - 1)] * kLog2e;
    for (int64_t q = first; q < past; q += L) {
        typename Two<T>::raw r[L], x[L], i[L];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int64_t at = min(q + l, past - 1), t = BWD ? n - 1 - at : at;
            r[l] = load2<T, MODE>(p.r + b * p.rsb + t * p.rst, 0, col);
            x[l] = BWD ? load2<T, MODE>(p.dh + b * p.dsb + t * p.dst, 0, col) : load2<T, MODE>(p.x + b * p.xsb + t * p.xst, 0, col);
            if constexpr (!BWD) i[l] = load2<T, MODE>(p.i + b * p.isb + t * p.ist, 0, col);
        }
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float rf[2], xf[2], jf[2];
            values<T, MODE>(r[l], col, rf);
            values<T, MODE>(x[l], col, xf);
            if constexpr (!BWD) values<T, MODE>(i[l], col, jf);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float a, m, u;
                const float s = ld[k] * sigmoid(rf[k]);
                if constexpr (BWD) {
                    a = exp2_fast(s);
                    u = a * xf[k];
                } else {
                    decay(s, a, m);
                    u = __builtin_amdgcn_sqrtf(m) * (xf[k] * sigmoid(jf[k]));
                }
                if (q + l < past) {
                    A[k] *= a;
                    E[k] = fmaf(a, E[k], u);
                }
            }
        }
    }
    float Ab[2], Eb[2];
    scan_wave<LR>(lane, A, E, Ab, Eb);
    if (lane >= 64 - LR) agg[wave][lane - (64 - LR)] = make_float4(A[0], E[0], A[1], E[1]);
    __syncthreads();
    if (threadIdx.x >= LR) return;
    float4 m = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
    for (int w = 0; w < NW; ++w) {
        const float4 v = agg[w][lane];
        m.y = fmaf(v.x, m.y, v.y);
        m.x *= v.x;
        m.w = fmaf(v.z, m.w, v.w);
        m.z *= v.z;
    }
    float2 *const o = reinterpret_cast<float2 *>(p.maps) + (b * p.nseg + seg) * p.C + c;
    if (col.has_lo) o[0] = make_float2(m.x, m.y);
    if (col.has_hi) o[1] = make_float2(m.z, m.w);
}

template <typename T, int LR, int NW, bool BWD, bool SINGLE>
__global__ __launch_bounds__(64 * NW) void gated_states(const Walk p)
{
    __shared__ float4 agg[NW][LR];
    int ct, seg;
    int64_t b;
    if (!place(p, p.nseg - 1, ct, seg, b)) return;     // nothing follows the last segment
    if constexpr (SINGLE) states_body<T, LR, NW, BWD, kSingle>(p, ct, seg, b, agg);
    else if ((int64_t)(ct + 1) * 2 * LR <= p.C) states_body<T, LR, NW, BWD, kWhole>(p, ct, seg, b, agg);
    else states_body<T, LR, NW, BWD, kEdge>(p, ct, seg, b, agg);
}

// ---------------------------------------------------------------- backward

// From the sequence's end, c_t = a_t G_t with G_t = dh_t + c_(t+1) the gradient of h_t itself:
//     dx = G s i',  di = G s x i'(1 - i'),  dla = a G h_(t-1) - (a^2 / s) G i' x,
//     dr = dla log_decay r'(1 - r'),  dlog_decay = sum of dla r'      (s = sqrt(1 - a^2))
// so each gradient is G times a factor of the token alone.  Where s is 0 (r' underflows, or a
// log_decay of 0) the root has no derivative, and its term is left out.
template <typename T, int L> struct RawBwd { typename Two<T>::raw x[L], r[L], i[L], h[L], d[L]; };

// Row l of a lane: token t0 - l (tokens fall), its h one token before.
template <typename T, int MODE, int L>
__device__ __forceinline__ void load_bwd(const Walk &p, const char *const (&base)[5], int64_t t0, int run, int TS, const Cols &col,
                                         RawBwd<T, L> &raw)
{
    // t0: the newest token of the tile; the oldest is t0 - TS + 1.
    const int64_t low = t0 - TS + 1;
    if (low >= 1) {
        const uint32_t up = (uint32_t)(TS - L - run * L);      // the lane's oldest token, from low
        const uint32_t ox = up * (uint32_t)p.xst, orr = up * (uint32_t)p.rst, oi = up * (uint32_t)p.ist, oh = up * (uint32_t)p.hst,
                       od = up * (uint32_t)p.dst;
        const char *x = base[0] + low * p.xst, *r = base[1] + low * p.rst, *i = base[2] + low * p.ist,
                   *h = base[3] + (low - 1) * p.hst, *d = base[4] + low * p.dst;
#pragma unroll
        for (int l = L - 1; l >= 0; --l) {
            raw.r[l] = load2<T, MODE>(r, orr, col);
            raw.d[l] = load2<T, MODE>(d, od, col);
            raw.x[l] = load2<T, MODE>(x, ox, col);
            raw.i[l] = load2<T, MODE>(i, oi, col);
            raw.h[l] = load2<T, MODE>(h, oh, col);
            x += fresh(p.xst);
            r += fresh(p.rst);
            i += fresh(p.ist);
            h += fresh(p.hst);
            d += fresh(p.dst);
        }
    } else {        // tokens before the first are read from it
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int64_t t = max((int64_t)0, t0 - run * L - l);
            raw.r[l] = load2<T, MODE>(base[1] + t * p.rst, 0, col);
            raw.d[l] = load2<T, MODE>(base[4] + t * p.dst, 0, col);
            raw.x[l] = load2<T, MODE>(base[0] + t * p.xst, 0, col);
            raw.i[l] = load2<T, MODE>(base[2] + t * p.ist, 0, col);
            raw.h[l] = load2<T, MODE>(base[3] + max((int64_t)0, t - 1) * p.hst, 0, col);
        }
    }
}

template <typename T, int LR, int NW, int MODE>
__device__ __forceinline__ void bwd_body(const Walk &p, int ct, int seg, int64_t b, float4 (*agg)[NW][LR])
{
    constexpr int RW = 64 / LR, L = run_len_bwd<T>(), TS = NW * RW * L;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int run = wave * RW + lane / LR;
    int64_t c;
    const Cols col = columns<T, LR>(p, ct, lane, c);
    // Segments count from the sequence's end.
    const int64_t n = live_tokens(p, b), top = n - 1 - seg * p.seg_len, bottom = max((int64_t)0, n - (seg + 1) * p.seg_len);
    const char *const base[5] = {p.x + b * p.xsb, p.r + b * p.rsb, p.i + b * p.isb, p.h_in + b * p.hsb, p.dh + b * p.dsb};
    const uint32_t orow = (uint32_t)(p.C * sizeof(T));
    const int64_t ob = b * p.T * (int64_t)orow;

    RawBwd<T, L> raw;
    if (top >= bottom) load_bwd<T, MODE, L>(p, base, top, run, TS, col, raw);
    float ld[2], carry[2], before[2], share[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int64_t ck = min(c + k, p.C - 1);
        ld[k] = p.log_decay[ck];
        carry[k] = fold(p, b, seg, ck, p.sf ? p.sf[b * p.C + ck] : 0.0f);
        before[k] = p.s0 ? p.s0[b * p.C + ck] : 0.0f;
    }
    int buf = 0;
    for (int64_t t0 = top; t0 >= bottom; t0 -= TS, buf ^= 1) {
        RawBwd<T, L> next;
        if (t0 - TS >= bottom) load_bwd<T, MODE, L>(p, base, t0 - TS, run, TS, col, next);
        const bool full = t0 - TS + 1 >= bottom;
        const int rows = full ? L : (int)min((int64_t)L, max((int64_t)0, t0 - run * L - bottom + 1));
        float a[L][2], g[L][2], fx[L][2], fi[L][2], fr[L][2], fd[L][2];
        float A[2] = {1.0f, 1.0f}, E[2] = {0.0f, 0.0f}, Ab[2], Eb[2];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float x[2], r[2], i[2], h[2];
            values<T, MODE>(raw.x[l], col, x);
            values<T, MODE>(raw.r[l], col, r);
            values<T, MODE>(raw.i[l], col, i);
            values<T, MODE>(raw.h[l], col, h);
            values<T, MODE>(raw.d[l], col, g[l]);
            const bool start = t0 - run * L - l == 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float sr = sigmoid(r[k]), si = sigmoid(i[k]), la = ld[k] * sr;
                float m;
                decay(kLog2e * la, a[l][k], m);
                // 1 / s and s from one root.
                const float inv = m > 0.0f ? __builtin_amdgcn_rsqf(m) : 0.0f, xi = x[k] * si;
                const float hp = start ? before[k] : h[k];
                fx[l][k] = m * inv * si;
                fi[l][k] = m * inv * xi * (1.0f - si);
                const float f = a[l][k] * (hp - a[l][k] * inv * xi);
                fd[l][k] = f * sr;
                fr[l][k] = f * la * (1.0f - sr);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (rows < L)
#pragma unroll
            for (int l = 0; l < L; ++l)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    a[l][k] = l < rows ? a[l][k] : 1.0f;
                    g[l][k] = l < rows ? g[l][k] : 0.0f;
                    fd[l][k] = l < rows ? fd[l][k] : 0.0f;
                }
#pragma unroll
        for (int l = 0; l < L; ++l)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                A[k] *= a[l][k];
                E[k] = a[l][k] * (g[l][k] + E[k]);
            }
        scan_wave<LR>(lane, A, E, Ab, Eb);
        if (lane >= 64 - LR) agg[buf][wave][lane - (64 - LR)] = make_float4(A[0], E[0], A[1], E[1]);
        __syncthreads();
        float cc[2] = {carry[0], carry[1]};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float4 m = agg[buf][w][lane % LR];
            cc[0] = w == wave ? carry[0] : cc[0];
            cc[1] = w == wave ? carry[1] : cc[1];
            carry[0] = fmaf(m.x, carry[0], m.y);
            carry[1] = fmaf(m.z, carry[1], m.w);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) cc[k] = fmaf(Ab[k], cc[k], Eb[k]);
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float G[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                G[k] = g[l][k] + cc[k];
                cc[k] = a[l][k] * G[k];
                // A token that does not exist adds nothing, whatever G is.
                share[k] = l < rows ? fmaf(G[k], fd[l][k], share[k]) : share[k];
            }
            if (full || l < rows) {
                const int64_t at = ob + (t0 - run * L - l) * (int64_t)orow;
                store2<T, MODE>(p.dx + at, 0, col, G[0] * fx[l][0], G[1] * fx[l][1]);
                store2<T, MODE>(p.dr + at, 0, col, G[0] * fr[l][0], G[1] * fr[l][1]);
                store2<T, MODE>(p.di + at, 0, col, G[0] * fi[l][0], G[1] * fi[l][1]);
            }
        }
        raw = next;
    }
    // Tokens that do not exist: this segment's part of [n, T).
    for (int64_t t = n + (int64_t)seg * NW * RW + run; t < p.T; t += (int64_t)p.nseg * NW * RW) {
        const int64_t at = ob + t * (int64_t)orow;
        store2<T, MODE>(p.dx + at, 0, col, 0.0f, 0.0f);
        store2<T, MODE>(p.dr + at, 0, col, 0.0f, 0.0f);
        store2<T, MODE>(p.di + at, 0, col, 0.0f, 0.0f);
    }
    if (p.h && seg == p.nseg - 1 && threadIdx.x < LR)      // p.h: the first state's gradient, fp32
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (c + k < p.C) reinterpret_cast<float *>(p.h)[b * p.C + c + k] = carry[k];
    // Shares of log_decay's gradient: over the runs of a wave, then over the waves.
#pragma unroll
    for (int d = LR; d < 64; d *= 2)
#pragma unroll
        for (int k = 0; k < 2; ++k) share[k] += __shfl_xor(share[k], d);
    __syncthreads();
    if (lane < LR) agg[0][wave][lane] = make_float4(share[0], share[1], 0.0f, 0.0f);
    __syncthreads();
    if (threadIdx.x >= LR) return;
    float sum[2] = {0.0f, 0.0f};
    for (int w = 0; w < NW; ++w) {
        sum[0] += agg[0][w][lane].x;
        sum[1] += agg[0][w][lane].y;
    }
    float *const o = p.part + (b * p.nseg + seg) * p.C + c;
    if (col.has_lo) o[0] = sum[0];
    if (col.has_hi) o[1] = sum[1];
}

template <typename T, int LR, int NW, bool SINGLE>
__global__ __launch_bounds__(64 * NW) void gated_bwd_walk(const Walk p)
{
    __shared__ float4 agg[2][NW][LR];
    int ct, seg;
    int64_t b;
    if (!place(p, p.nseg, ct, seg, b)) return;
    if constexpr (SINGLE) bwd_body<T, LR, NW, kSingle>(p, ct, seg, b, agg);
    else if ((int64_t)(ct + 1) * 2 * LR <= p.C) bwd_body<T, LR, NW, kWhole>(p, ct, seg, b, agg);
    else bwd_body<T, LR, NW, kEdge>(p, ct, seg, b, agg);
}

// Sum over sequences and segments, in order: 16 rows at a time, then those 16.
__global__ __launch_bounds__(256) void gated_share_sum(const float *__restrict__ part, float *__restrict__ out, int64_t rows,
                                                       int64_t C)
{
    __shared__ float s[16][17];
    const int col = threadIdx.x % 16, row = threadIdx.x / 16;
    const int64_t c = (int64_t)blockIdx.x * 16 + col;
    float v = 0.0f;
    if (c < C)
        for (int64_t r = row; r < rows; r += 16) v += part[r * C + c];
    s[row][col] = v;
    __syncthreads();
    if (row == 0 && c < C) {
        for (int r = 1; r < 16; ++r) v += s[r][col];
        out[c] = v;
    }
}

// ---------------------------------------------------------------- single tokens

template <typename T>
__global__ __launch_bounds__(256) void gated_step(const T *__restrict__ x, const T *__restrict__ r, const T *__restrict__ i,
                                                  const float *__restrict__ log_decay, float *__restrict__ state, T *__restrict__ h,
                                                  const int32_t *__restrict__ slots, int64_t B, int64_t C, int64_t n, int64_t xs,
                                                  int64_t rs, int64_t is)
{
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, b = at / C, c = at - b * C;
    if (b >= B) return;
    const int64_t slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= n) {
        h[b * C + c] = from_f32<T>(0.0f);
        return;
    }
    float a, m;
    decay(kLog2e * log_decay[c] * sigmoid(to_f32(r[b * rs + c])), a, m);
    const float v = fmaf(a, state[slot * C + c], __builtin_amdgcn_sqrtf(m) * (to_f32(x[b * xs + c]) * sigmoid(to_f32(i[b * is + c]))));
    state[slot * C + c] = v;
    h[b * C + c] = from_f32<T>(v);
}

int tile_steps(const GatedPlan &g, int dtype, bool backward)
{
    const int run = dtype == DT_F32 ? (backward ? run_len_bwd<float>() : run_len<float>())
                                    : (backward ? run_len_bwd<__bf16>() : run_len<__bf16>());
    return g.waves * (64 / g.lanes) * run;
}

Walk make_walk(const GatedArgs &a, const GatedPlan &g)
{
    const int64_t es = a.dtype == DT_F32 ? 4 : 2;
    Walk p = {};
    p.B = a.B; p.T = a.T; p.C = a.C; p.seg_len = g.seg_len; p.nseg = g.nseg;
    p.tiles = (int32_t)ceil_div(a.C, 2 * g.lanes);
    p.blocks = a.B * g.nseg * p.tiles;
    p.x = (const char *)a.x; p.r = (const char *)a.r; p.i = (const char *)a.i;
    p.log_decay = a.log_decay; p.s0 = a.s0; p.lengths = a.lengths;
    p.maps = a.ws;
    p.xsb = a.xsb * es; p.xst = a.xst * es; p.rsb = a.rsb * es; p.rst = a.rst * es; p.isb = a.isb * es; p.ist = a.ist * es;
    p.hsb = a.hsb * es; p.hst = a.hst * es; p.dsb = a.dsb * es; p.dst = a.dst * es;
    return p;
}

size_t map_bytes(const GatedPlan &g, int64_t B, int64_t C)
{
    return g.nseg > 1 ? (sizeof(float2) * (size_t)(B * g.nseg * C) + 255) & ~(size_t)255 : 0;
}

template <typename F> hipError_t with_type(int dtype, F &&f)
{
    if (dtype == DT_F32) return f(float{});
    if (dtype == DT_F16) return f(_Float16{});
    return f(__bf16{});
}

template <int N> struct Int { static constexpr int value = N; };

// The kernels that exist: (lanes, waves, one channel).
template <typename F> hipError_t with_shape(const GatedPlan &g, int64_t C, F &&f)
{
    constexpr Int<0> more{};
    if (C == 1) return f(Int<16>{}, Int<4>{}, Int<1>{});
    if (g.lanes == 16)
        return g.waves == 16 ? f(Int<16>{}, Int<16>{}, more) : g.waves == 8 ? f(Int<16>{}, Int<8>{}, more) : f(Int<16>{}, Int<4>{}, more);
    return g.waves == 16 ? f(Int<8>{}, Int<16>{}, more) : g.waves == 8 ? f(Int<8>{}, Int<8>{}, more) : f(Int<8>{}, Int<4>{}, more);
}

template <bool BWD> hipError_t launch_states(Walk p, const GatedPlan &g, int dtype, hipStream_t stream)
{
    p.blocks = p.B * (g.nseg - 1) * p.tiles;
    const dim3 grid((unsigned)(8 * ceil_div(p.blocks, 8)));
    return with_type(dtype, [&](auto t) {
        return with_shape(g, p.C, [&](auto lanes, auto waves, auto one) {
            gated_states<decltype(t), lanes.value, waves.value, BWD, one.value><<<grid, 64 * waves.value, 0, stream>>>(p);
            return hipGetLastError();
        });
    });
}

}  // namespace

GatedPlan gated_plan(int64_t B, int64_t T, int64_t C, int dtype, bool backward)
{
    GatedPlan g = {16, C == 1 ? 4 : 8, 1, std::max<int64_t>(T, 1)};
    const int64_t stripes = std::max<int64_t>(1, B * ceil_div(C, 32));
    const int64_t ts = tile_steps(g, dtype, backward), tiles = ceil_div(std::max<int64_t>(T, 1), ts);
    g.nseg = (int32_t)std::max<int64_t>(1, std::min<int64_t>({512 / stripes, tiles / 2, 256}));
    const int64_t each = ceil_div(tiles, (int64_t)g.nseg);
    g.nseg = (int32_t)ceil_div(tiles, each);
    g.seg_len = each * ts;
    return g;
}

size_t gated_workspace(const GatedPlan &g, int64_t B, int64_t C, bool backward)
{
    return map_bytes(g, B, C) + (backward ? sizeof(float) * (size_t)(B * g.nseg * C) : 0);
}

bool gated_fits(const GatedArgs &a, const GatedPlan &g, bool backward)
{
    const int64_t es = a.dtype == DT_F32 ? 4 : 2, ts = tile_steps(g, a.dtype, backward), top = (int64_t(1) << 31) - 1;
    for (int64_t st : {a.xst, a.rst, a.ist, a.C, backward ? a.hst : 0, backward ? a.dst : 0})
        if (ts * es > top / std::max<int64_t>(st, 1)) return false;
    return grid_fits(8 * ceil_div(a.B * g.nseg * ceil_div(a.C, 2 * g.lanes), 8), 64 * g.waves);
}

hipError_t launch_gated(const GatedArgs &a, const GatedPlan &g, const char **kname)
{
    Walk p = make_walk(a, g);
    p.h = (char *)a.h;
    p.sf = a.sf;
    *kname = "gated_walk";
    if (g.nseg > 1) {
        const hipError_t err = launch_states<false>(p, g, a.dtype, a.stream);
        if (err != hipSuccess) return err;
    }
    const dim3 grid((unsigned)(8 * ceil_div(p.blocks, 8)));
    return with_type(a.dtype, [&](auto t) {
        return with_shape(g, a.C, [&](auto lanes, auto waves, auto one) {
            gated_walk<decltype(t), lanes.value, waves.value, one.value><<<grid, 64 * waves.value, 0, a.stream>>>(p);
            return hipGetLastError();
        });
    });
}

hipError_t launch_gated_bwd(const GatedArgs &a, const GatedPlan &g, const char **kname)
{
    Walk p = make_walk(a, g);
    p.h_in = (const char *)a.h;
    p.dh = (const char *)a.dh;
    p.sf = const_cast<float *>(a.dsf);
    p.h = (char *)a.ds0;
    p.dx = (char *)a.dx; p.dr = (char *)a.dr; p.di = (char *)a.di;
    p.part = a.ws + map_bytes(g, a.B, a.C) / sizeof(float);
    *kname = "gated_bwd_walk";
    if (p.blocks > 0) {
        if (g.nseg > 1) {
            const hipError_t err = launch_states<true>(p, g, a.dtype, a.stream);
            if (err != hipSuccess) return err;
        }
        const dim3 grid((unsigned)(8 * ceil_div(p.blocks, 8)));
        const hipError_t err = with_type(a.dtype, [&](auto t) {
            return with_shape(g, a.C, [&](auto lanes, auto waves, auto one) {
                gated_bwd_walk<decltype(t), lanes.value, waves.value, one.value><<<grid, 64 * waves.value, 0, a.stream>>>(p);
                return hipGetLastError();
            });
        });
        if (err != hipSuccess) return err;
    }
    gated_share_sum<<<(unsigned)ceil_div(a.C, 16), 256, 0, a.stream>>>(p.part, a.dlog, a.B * g.nseg, a.C);
    return hipGetLastError();
}

bool gated_step_fits(const GatedStepArgs &a) { return grid_fits(ceil_div(a.B * a.C, 256), 256); }

hipError_t launch_gated_step(const GatedStepArgs &a, const char **kname)
{
    *kname = "gated_step";
    const dim3 grid((unsigned)ceil_div(a.B * a.C, 256));
    return with_type(a.dtype, [&](auto t) {
        typedef decltype(t) E;
        gated_step<E><<<grid, 256, 0, a.stream>>>((const E *)a.x, (const E *)a.r, (const E *)a.i, a.log_decay, a.state, (E *)a.h,
                                                  a.slots, a.B, a.C, a.n, a.xs, a.rs, a.is);
        return hipGetLastError();
    });
}

}  // namespace gconv
