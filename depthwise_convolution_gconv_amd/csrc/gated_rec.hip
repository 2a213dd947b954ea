// gated_rec.hip -- gated linear recurrence over (batch, steps, channels):
//     a_t = exp(log_decay[c] sigmoid(r_t)),   h_t = a_t h_(t-1) + sqrt(1 - a_t^2) sigmoid(i_t) x_t,
// its gradients and its form for single tokens.
//
// A recurrence h_t = a_t h_(t-1) + u_t is a composition of affine maps: over any run of tokens
// it is h_out = A h_in + E with A the product of the a_t and E the run's own result from zero.
// A workgroup walks the tokens of one sequence for a stripe of channels, tile after tile: each
// lane takes a run of consecutive tokens for 8 bytes of channels, keeps its a_t and u_t in registers,
// and (A, E) of the runs are joined by lane exchanges within a wave and through LDS across the
// waves.  Then each lane knows the state before its run and writes its h_t.  So the inputs are
// read once and one barrier is needed for a tile; the next tile's loads are in flight meanwhile.
// Where stripes alone do not fill the card a sequence is cut into segments: (A, E) of each come
// first (gated_states), and a walk folds those before its own.
//
// Bound by HBM and, nearly as much, by vector instructions: six of quarter rate (three
// exponentials, two reciprocals, a root) and about 30 others for the 8 bytes of an element.  In bf16
// 8 x 4096 x 4096 takes 224 us (1.07 GB, 4.8 TB/s), 1 x 32768 x 4096, where stripes of 32 bytes fill the
// card, 385 - 420; gradients of 4 x 4096 x 2560 take 191 us: 48 for the segments' maps, 139 for the walk
// (0.67 GB, 4.8 TB/s, 200 registers, two waves a SIMD) and 5 for the sum of log_decay's shares.  Tokens of
// 64 x 4096 take 3 us in gated_step.
//
// One pass with a workgroup waiting for its predecessor's state would save the cut's second read; it took
// 442 us where the narrow stripes take 400.
#include <algorithm>

#include "block.hpp"

namespace gconv {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// A lane's channels: 8 bytes of a row.
typedef uint32_t lane_mem __attribute__((ext_vector_type(2), aligned(2)));
template <typename T> constexpr int lane_channels() { return 8 / (int)sizeof(T); }

// What a stripe of channels is: whole; the one that C ends in (a lane that reaches past the end
// reads the last 8 bytes of the row and shifts them down); all of a row shorter than 8 bytes.
enum { kWhole = 0, kEdge = 1, kShort = 2 };

struct Cols {
    uint32_t at;           // byte offset that is read
    uint32_t to;           // and that is written
    int shift;             // bits by which what is read lies too high
    int have;              // channels of the lane that exist
};

template <typename T, int MODE>
__device__ __forceinline__ uint2 load_lane(const char *base, uint32_t row, const Cols &c)
{
    if constexpr (MODE == kShort) {
        uint64_t w = 0;
        for (int k = 0; k < c.have; ++k) {
            if constexpr (sizeof(T) == 2)
                w |= (uint64_t) * reinterpret_cast<const uint16_t *>(base + (row + c.at + 2 * k)) << 16 * k;
            else
                w |= (uint64_t) * reinterpret_cast<const uint32_t *>(base + (row + c.at + 4 * k)) << 32 * k;
        }
        return __builtin_bit_cast(uint2, w);
    } else {
        return __builtin_bit_cast(uint2, *reinterpret_cast<const lane_mem *>(base + (row + c.at)));
    }
}

template <typename T, int MODE, int V>
__device__ __forceinline__ void values(uint2 w, const Cols &c, float (&f)[V])
{
    if constexpr (MODE == kEdge) w = __builtin_bit_cast(uint2, __builtin_bit_cast(uint64_t, w) >> c.shift);
    if constexpr (sizeof(T) == 4) {
        f[0] = __builtin_bit_cast(float, w.x);
        f[1] = __builtin_bit_cast(float, w.y);
    } else if constexpr (__is_same(T, __bf16)) {
        f[0] = __builtin_bit_cast(float, w.x << 16);
        f[1] = __builtin_bit_cast(float, w.x & 0xffff0000u);
        f[2] = __builtin_bit_cast(float, w.y << 16);
        f[3] = __builtin_bit_cast(float, w.y & 0xffff0000u);
    } else {
        typedef T quad __attribute__((ext_vector_type(4)));
        const quad q = __builtin_bit_cast(quad, w);
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = to_f32(q[k]);
    }
}

template <typename T, int MODE, int V>
__device__ __forceinline__ void store_lane(char *base, uint32_t row, const Cols &c, const float (&f)[V])
{
    if constexpr (MODE != kWhole) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < c.have) *reinterpret_cast<T *>(base + (row + c.to + k * (uint32_t)sizeof(T))) = from_f32<T>(f[k]);
    } else {
        typedef T vec __attribute__((ext_vector_type(V)));
        vec v;
#pragma unroll
        for (int k = 0; k < V; ++k) v[k] = from_f32<T>(f[k]);
        *reinterpret_cast<lane_mem *>(base + (row + c.to)) = __builtin_bit_cast(lane_mem, v);
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
template <typename T> constexpr int run_len() { return 4; }
template <typename T> constexpr int run_len_bwd() { return sizeof(T) == 4 ? 4 : 2; }

// A run's map joined with the one before it.
__device__ __forceinline__ void join_maps(float &A, float &E, float Ab, float Eb)
{
    E = fmaf(A, Eb, E);
    A *= Ab;
}

// Maps of the runs of a wave (64 / LR of them, LR lanes each) -> the map before each run, and in
// its last run's lanes that of the wave.
template <int LR, int V>
__device__ __forceinline__ void scan_wave(int lane, float (&A)[V], float (&E)[V], float (&Ab)[V], float (&Eb)[V])
{
#pragma unroll
    for (int d = LR; d < 64; d *= 2)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float pa = __shfl_up(A[k], d), pe = __shfl_up(E[k], d);
            if (lane >= d) join_maps(A[k], E[k], pa, pe);
        }
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const float pa = __shfl_up(A[k], LR), pe = __shfl_up(E[k], LR);
        Ab[k] = lane >= LR ? pa : 1.0f;
        Eb[k] = lane >= LR ? pe : 0.0f;
    }
}

// Maps of the waves of a tile, two channels in 16 bytes.
template <int NW, int LR, int V> struct Maps { float4 m[V / 2][NW][LR]; };

template <int NW, int LR, int V>
__device__ __forceinline__ void put_maps(Maps<NW, LR, V> &to, int wave, int at, const float (&A)[V], const float (&E)[V])
{
#pragma unroll
    for (int k = 0; k < V / 2; ++k) to.m[k][wave][at] = make_float4(A[2 * k], E[2 * k], A[2 * k + 1], E[2 * k + 1]);
}

// The state after the tile, and (h) that before the wave.
template <int NW, int LR, int V>
__device__ __forceinline__ void through_waves(const Maps<NW, LR, V> &maps, int wave, int at, float (&carry)[V], float (&h)[V])
{
    asm volatile("" : "+s"(wave));      // compared here, not once for all tiles in 2 NW scalar registers
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float4 m = maps.m[k / 2][w][at];
            h[k] = w == wave ? carry[k] : h[k];
            h[k + 1] = w == wave ? carry[k + 1] : h[k + 1];
            carry[k] = fmaf(m.x, carry[k], m.y);
            carry[k + 1] = fmaf(m.z, carry[k + 1], m.w);
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
    constexpr int V = lane_channels<T>();
    c = ((int64_t)ct * LR + lane % LR) * V;
    const int64_t read = max((int64_t)0, min(c, p.C - V));
    Cols k;
    k.have = (int)max((int64_t)0, min((int64_t)V, p.C - c));
    k.to = (uint32_t)(c * sizeof(T));
    k.at = (uint32_t)(read * sizeof(T));
    k.shift = 8 * (int)sizeof(T) * (int)min(c - read, (int64_t)(V - 1));
    return k;
}

// A stride that the compiler does not multiply out in advance: products for every row of a tile
// would fill the scalar registers.
__device__ __forceinline__ int64_t fresh(int64_t v)
{
    asm volatile("" : "+s"(v));
    return v;
}

// carry: the state before the first segment -> before this one, through the maps of those between, shared
// among the workgroup's runs as a tile's tokens are: 2 x 15147 x 256 in bf16, 79 segments, 43 us; every lane
// all of them by itself 69 us.
template <int NW, int LR, int V>
__device__ __forceinline__ void enter_segment(const Walk &p, int64_t b, int seg, int64_t c, int wave, int lane, Maps<NW, LR, V> &maps,
                                              float (&carry)[V])
{
    if (seg == 0) return;
    constexpr int RUNS = NW * (64 / LR);
    const int each = (seg + RUNS - 1) / RUNS, from = min(seg, (wave * (64 / LR) + lane / LR) * each), to = min(seg, from + each);
    float A[V], E[V], Ab[V], Eb[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        A[k] = 1.0f;
        E[k] = 0.0f;
    }
    for (int s = from; s < to; ++s)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float2 m = *reinterpret_cast<const float2 *>(p.maps + 2 * ((b * p.nseg + s) * p.C + min(c + k, p.C - 1)));
            E[k] = fmaf(m.x, E[k], m.y);
            A[k] *= m.x;
        }
    scan_wave<LR>(lane, A, E, Ab, Eb);
    if (lane >= 64 - LR) put_maps(maps, wave, lane - (64 - LR), A, E);
    __syncthreads();
    through_waves(maps, wave, lane % LR, carry, Ab);
}

// ---------------------------------------------------------------- forward

template <int L> struct RawIn { uint2 x[L], r[L], i[L]; };

// step: byte offsets of the lane's run in x, r and i.
template <typename T, int MODE>
__device__ __forceinline__ void load_in(const Walk &p, const char *const (&base)[3], int64_t t0, int64_t live, int run, int TS,
                                        const uint32_t (&step)[3], const Cols &col, RawIn<run_len<T>()> &raw)
{
    constexpr int kRun = run_len<T>();
    const char *x = base[0] + t0 * p.xst, *r = base[1] + t0 * p.rst, *i = base[2] + t0 * p.ist;
    if (t0 + TS <= live) {
#pragma unroll
        for (int l = 0; l < kRun; ++l) {
            raw.x[l] = load_lane<T, MODE>(x, step[0], col);
            raw.r[l] = load_lane<T, MODE>(r, step[1], col);
            raw.i[l] = load_lane<T, MODE>(i, step[2], col);
            x += fresh(p.xst);
            r += fresh(p.rst);
            i += fresh(p.ist);
        }
    } else {        // rows past the end are read from the last one
        const int last = (int)(live - 1 - t0);
#pragma unroll
        for (int l = 0; l < kRun; ++l) {
            const uint32_t row = (uint32_t)min(run * kRun + l, last);
            raw.x[l] = load_lane<T, MODE>(x, row * (uint32_t)p.xst, col);
            raw.r[l] = load_lane<T, MODE>(r, row * (uint32_t)p.rst, col);
            raw.i[l] = load_lane<T, MODE>(i, row * (uint32_t)p.ist, col);
        }
    }
}

template <typename T, int MODE, int V>
__device__ __forceinline__ void gates(const RawIn<run_len<T>()> &raw, const Cols &col, const float (&ld)[V], int rows, float (&a)[run_len<T>()][V],
                                      float (&u)[run_len<T>()][V])
{
    constexpr int kRun = run_len<T>();
#pragma unroll
    for (int l = 0; l < kRun; ++l) {
        float x[V], r[V], i[V];
        values<T, MODE>(raw.x[l], col, x);
        values<T, MODE>(raw.r[l], col, r);
        values<T, MODE>(raw.i[l], col, i);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            float m;
            decay(ld[k] * sigmoid(r[k]), a[l][k], m);
            u[l][k] = __builtin_amdgcn_sqrtf(m) * (x[k] * sigmoid(i[k]));
        }
        __builtin_amdgcn_sched_barrier(0);      // one token after the other: temporaries of all at once do not fit
    }
    if (rows < kRun)        // tokens that do not exist leave the state alone, whatever was read
#pragma unroll
        for (int l = 0; l < kRun; ++l)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                a[l][k] = l < rows ? a[l][k] : 1.0f;
                u[l][k] = l < rows ? u[l][k] : 0.0f;
            }
}

template <typename T, int LR, int NW, int MODE>
__device__ __forceinline__ void walk_body(const Walk &p, int ct, int seg, int64_t b, Maps<NW, LR, lane_channels<T>()> *maps)
{
    constexpr int V = lane_channels<T>(), RW = 64 / LR, kRun = run_len<T>(), TS = NW * RW * kRun;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int run = wave * RW + lane / LR;
    int64_t c;
    const Cols col = columns<T, LR>(p, ct, lane, c);
    const int64_t n = live_tokens(p, b), begin = seg * p.seg_len, end = min(begin + p.seg_len, p.T), live = min(end, n);
    const char *const base[3] = {p.x + b * p.xsb, p.r + b * p.rsb, p.i + b * p.isb};
    const uint32_t step[3] = {(uint32_t)(run * kRun * p.xst), (uint32_t)(run * kRun * p.rst), (uint32_t)(run * kRun * p.ist)};
    const uint32_t hrow = (uint32_t)(p.C * sizeof(T)), first = (uint32_t)(run * kRun) * hrow;
    char *const out = p.h + b * p.T * (int64_t)hrow;

    RawIn<kRun> raw;
    if (begin < live) load_in<T, MODE>(p, base, begin, live, run, TS, step, col, raw);
    float ld[V], carry[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int64_t ck = min(c + k, p.C - 1);
        ld[k] = p.log_decay[ck] * kLog2e;
        carry[k] = p.s0 ? p.s0[b * p.C + ck] : 0.0f;
    }
    enter_segment(p, b, seg, c, wave, lane, maps[1], carry);
    int buf = 0;
    for (int64_t t0 = begin; t0 < live; t0 += TS, buf ^= 1) {
        RawIn<kRun> next;
        if (t0 + TS < live) load_in<T, MODE>(p, base, t0 + TS, live, run, TS, step, col, next);
        const bool full = t0 + TS <= live;
        const int rows = full ? kRun : (int)min((int64_t)kRun, max((int64_t)0, live - t0 - run * kRun));
        float a[kRun][V], u[kRun][V], A[V], E[V], Ab[V], Eb[V], h[V];
        gates<T, MODE>(raw, col, ld, rows, a, u);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            A[k] = a[0][k];
            E[k] = u[0][k];
        }
#pragma unroll
        for (int l = 1; l < kRun; ++l)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                A[k] *= a[l][k];
                E[k] = fmaf(a[l][k], E[k], u[l][k]);
            }
        scan_wave<LR>(lane, A, E, Ab, Eb);
        if (lane >= 64 - LR) put_maps(maps[buf], wave, lane - (64 - LR), A, E);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < V; ++k) h[k] = carry[k];
        through_waves(maps[buf], wave, lane % LR, carry, h);
#pragma unroll
        for (int k = 0; k < V; ++k) h[k] = fmaf(Ab[k], h[k], Eb[k]);
        char *o = out + t0 * (int64_t)hrow;
        if (full) {
#pragma unroll
            for (int l = 0; l < kRun; ++l) {
#pragma unroll
                for (int k = 0; k < V; ++k) h[k] = fmaf(a[l][k], h[k], u[l][k]);
                store_lane<T, MODE>(o, first, col, h);
                o += fresh(hrow);
            }
        } else {
#pragma unroll
            for (int l = 0; l < kRun; ++l) {
#pragma unroll
                for (int k = 0; k < V; ++k) h[k] = fmaf(a[l][k], h[k], u[l][k]);
                if (l < rows) store_lane<T, MODE>(o, first, col, h);
                o += fresh(hrow);
            }
        }
        raw = next;
    }
    const float zero[V] = {};
    for (int64_t t = max(begin, n) + run; t < end; t += NW * RW) store_lane<T, MODE>(out + t * (int64_t)hrow, 0, col, zero);
    if (p.sf && seg == p.nseg - 1 && threadIdx.x < LR)
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < col.have) p.sf[b * p.C + c + k] = carry[k];
}

// Whole, last and only stripe of a row.
#define GATED_BODY(body, ...)                                                             \
    if constexpr (SHORT) body<__VA_ARGS__, kShort>(p, ct, seg, b, maps);                  \
    else if ((int64_t)(ct + 1) * LR * lane_channels<T>() <= p.C) body<__VA_ARGS__, kWhole>(p, ct, seg, b, maps); \
    else body<__VA_ARGS__, kEdge>(p, ct, seg, b, maps)

template <typename T, int LR, int NW, bool SHORT>
__global__ __launch_bounds__(64 * NW) void gated_walk(const Walk p)
{
    __shared__ Maps<NW, LR, lane_channels<T>()> maps[2];
    int ct, seg;
    int64_t b;
    if (!place(p, p.nseg, ct, seg, b)) return;
    GATED_BODY(walk_body, T, LR, NW);
}

// ---------------------------------------------------------------- (A, E) of segments

// Each run of lanes takes a stretch of the segment of its own; no joins until its end.  Forward:
// maps of h.  Backward (from the sequence's end): maps of c_t = a_t (dh_t + c_(t+1)).
template <typename T, int LR, int NW, bool BWD, int MODE>
__device__ __forceinline__ void states_body(const Walk &p, int ct, int seg, int64_t b, Maps<NW, LR, lane_channels<T>()> &maps)
{
    constexpr int V = lane_channels<T>(), RW = 64 / LR, L = 4;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int run = wave * RW + lane / LR;
    int64_t c;
    const Cols col = columns<T, LR>(p, ct, lane, c);
    const int64_t n = live_tokens(p, b), stretch = p.seg_len / (NW * RW);
    // Positions count from the start of the walk: token q forward, n - 1 - q backward.
    const int64_t first = seg * p.seg_len + run * stretch, past = min(first + stretch, n);
    float ld[V], A[V], E[V], Ab[V], Eb[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        ld[k] = p.log_decay[min(c + k, p.C - 1)] * kLog2e;
        A[k] = 1.0f;
        E[k] = 0.0f;
    }
    for (int64_t q = first; q < past; q += L) {
        uint2 r[L], x[L], i[L];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            const int64_t at = min(q + l, past - 1), t = BWD ? n - 1 - at : at;
            r[l] = load_lane<T, MODE>(p.r + b * p.rsb + t * p.rst, 0, col);
            x[l] = BWD ? load_lane<T, MODE>(p.dh + b * p.dsb + t * p.dst, 0, col) : load_lane<T, MODE>(p.x + b * p.xsb + t * p.xst, 0, col);
            if constexpr (!BWD) i[l] = load_lane<T, MODE>(p.i + b * p.isb + t * p.ist, 0, col);
        }
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float rf[V], xf[V], jf[V];
            values<T, MODE>(r[l], col, rf);
            values<T, MODE>(x[l], col, xf);
            if constexpr (!BWD) values<T, MODE>(i[l], col, jf);
#pragma unroll
            for (int k = 0; k < V; ++k) {
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
    scan_wave<LR>(lane, A, E, Ab, Eb);
    if (lane >= 64 - LR) put_maps(maps, wave, lane - (64 - LR), A, E);
    __syncthreads();
    if (threadIdx.x >= LR) return;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        A[k] = 1.0f;
        E[k] = 0.0f;
    }
    for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float4 v = maps.m[k / 2][w][lane];
            E[k] = fmaf(v.x, E[k], v.y);
            A[k] *= v.x;
            E[k + 1] = fmaf(v.z, E[k + 1], v.w);
            A[k + 1] *= v.z;
        }
    float2 *const o = reinterpret_cast<float2 *>(p.maps) + (b * p.nseg + seg) * p.C + c;
#pragma unroll
    for (int k = 0; k < V; ++k)
        if (k < col.have) o[k] = make_float2(A[k], E[k]);
}

template <typename T, int LR, int NW, bool BWD, bool SHORT>
__global__ __launch_bounds__(64 * NW) void gated_states(const Walk p)
{
    __shared__ Maps<NW, LR, lane_channels<T>()> maps;
    int ct, seg;
    int64_t b;
    if (!place(p, p.nseg - 1, ct, seg, b)) return;     // nothing follows the last segment
    GATED_BODY(states_body, T, LR, NW, BWD);
}

// ---------------------------------------------------------------- backward

// From the sequence's end, c_t = a_t G_t with G_t = dh_t + c_(t+1) the gradient of h_t itself:
//     dx = G s i',  di = G s x i'(1 - i'),  dla = a G h_(t-1) - (a^2 / s) G i' x,
//     dr = dla log_decay r'(1 - r'),  dlog_decay = sum of dla r'      (s = sqrt(1 - a^2))
// so each gradient is G times a factor of the token alone.  Where s is 0 (r' underflows, or a
// log_decay of 0) the root has no derivative, and its term is left out; so it is where 1 - a^2
// lies below fp32's smallest normal number, 2^-126, which the forward pass's root takes as 0 too.
template <int L> struct RawBwd { uint2 x[L], r[L], i[L], h[L], d[L]; };

// Row l of a lane: token t0 - run run_len_bwd<T>() - l (tokens fall), its h one token before.
// step: byte offsets of the lane's oldest token from the tile's.
template <typename T, int MODE>
__device__ __forceinline__ void load_bwd(const Walk &p, const char *const (&base)[5], int64_t t0, int run, int TS,
                                         const uint32_t (&step)[5], const Cols &col, RawBwd<run_len_bwd<T>()> &raw)
{
    const int64_t low = t0 - TS + 1;
    if (low >= 1) {
        const char *x = base[0] + low * p.xst, *r = base[1] + low * p.rst, *i = base[2] + low * p.ist,
                   *h = base[3] + (low - 1) * p.hst, *d = base[4] + low * p.dst;
#pragma unroll
        for (int l = run_len_bwd<T>() - 1; l >= 0; --l) {
            raw.r[l] = load_lane<T, MODE>(r, step[1], col);
            raw.d[l] = load_lane<T, MODE>(d, step[4], col);
            raw.x[l] = load_lane<T, MODE>(x, step[0], col);
            raw.i[l] = load_lane<T, MODE>(i, step[2], col);
            raw.h[l] = load_lane<T, MODE>(h, step[3], col);
            x += fresh(p.xst);
            r += fresh(p.rst);
            i += fresh(p.ist);
            h += fresh(p.hst);
            d += fresh(p.dst);
        }
    } else {        // tokens before the first are read from it
#pragma unroll
        for (int l = 0; l < run_len_bwd<T>(); ++l) {
            const int64_t t = max((int64_t)0, t0 - run * run_len_bwd<T>() - l);
            raw.r[l] = load_lane<T, MODE>(base[1] + t * p.rst, 0, col);
            raw.d[l] = load_lane<T, MODE>(base[4] + t * p.dst, 0, col);
            raw.x[l] = load_lane<T, MODE>(base[0] + t * p.xst, 0, col);
            raw.i[l] = load_lane<T, MODE>(base[2] + t * p.ist, 0, col);
            raw.h[l] = load_lane<T, MODE>(base[3] + max((int64_t)0, t - 1) * p.hst, 0, col);
        }
    }
}

template <typename T, int LR, int NW, int MODE>
__device__ __forceinline__ void bwd_body(const Walk &p, int ct, int seg, int64_t b, Maps<NW, LR, lane_channels<T>()> *maps)
{
    constexpr int V = lane_channels<T>(), RW = 64 / LR, L = run_len_bwd<T>(), TS = NW * RW * L;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int run = wave * RW + lane / LR;
    int64_t c;
    const Cols col = columns<T, LR>(p, ct, lane, c);
    // Segments count from the sequence's end.
    const int64_t n = live_tokens(p, b), top = n - 1 - seg * p.seg_len, bottom = max((int64_t)0, n - (seg + 1) * p.seg_len);
    const char *const base[5] = {p.x + b * p.xsb, p.r + b * p.rsb, p.i + b * p.isb, p.h_in + b * p.hsb, p.dh + b * p.dsb};
    const int up = TS - L - run * L;
    const uint32_t step[5] = {(uint32_t)(up * p.xst), (uint32_t)(up * p.rst), (uint32_t)(up * p.ist), (uint32_t)(up * p.hst),
                              (uint32_t)(up * p.dst)};
    const uint32_t orow = (uint32_t)(p.C * sizeof(T)), oldest = (uint32_t)up * orow;
    const int64_t ob = b * p.T * (int64_t)orow;

    RawBwd<L> raw;
    if (top >= bottom) load_bwd<T, MODE>(p, base, top, run, TS, step, col, raw);
    float ld[V], carry[V], before[V], share[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int64_t ck = min(c + k, p.C - 1);
        ld[k] = p.log_decay[ck];
        carry[k] = p.sf ? p.sf[b * p.C + ck] : 0.0f;
        before[k] = p.s0 ? p.s0[b * p.C + ck] : 0.0f;
        share[k] = 0.0f;
    }
    enter_segment(p, b, seg, c, wave, lane, maps[1], carry);
    int buf = 0;
    for (int64_t t0 = top; t0 >= bottom; t0 -= TS, buf ^= 1) {
        RawBwd<L> next;
        if (t0 - TS >= bottom) load_bwd<T, MODE>(p, base, t0 - TS, run, TS, step, col, next);
        const bool full = t0 - TS + 1 >= bottom;
        const int rows = full ? L : (int)min((int64_t)L, max((int64_t)0, t0 - run * L - bottom + 1));
        float a[L][V], g[L][V], fx[L][V], fi[L][V], fr[L][V], fd[L][V], A[V], E[V], Ab[V], Eb[V], cc[V];
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float x[V], r[V], i[V], h[V];
            values<T, MODE>(raw.x[l], col, x);
            values<T, MODE>(raw.r[l], col, r);
            values<T, MODE>(raw.i[l], col, i);
            values<T, MODE>(raw.h[l], col, h);
            values<T, MODE>(raw.d[l], col, g[l]);
            const bool start = t0 - run * L - l == 0;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float sr = sigmoid(r[k]), si = sigmoid(i[k]), la = ld[k] * sr;
                float m;
                decay(kLog2e * la, a[l][k], m);
                // 1 / s and s from one root, which takes a denormal number as zero: its inverse would be infinite.
                const float inv = m >= 0x1p-126f ? __builtin_amdgcn_rsqf(m) : 0.0f, xi = x[k] * si;
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
                for (int k = 0; k < V; ++k) {
                    a[l][k] = l < rows ? a[l][k] : 1.0f;
                    g[l][k] = l < rows ? g[l][k] : 0.0f;
                }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            A[k] = a[0][k];
            E[k] = a[0][k] * g[0][k];
        }
#pragma unroll
        for (int l = 1; l < L; ++l)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                A[k] *= a[l][k];
                E[k] = a[l][k] * (g[l][k] + E[k]);
            }
        scan_wave<LR>(lane, A, E, Ab, Eb);
        if (lane >= 64 - LR) put_maps(maps[buf], wave, lane - (64 - LR), A, E);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < V; ++k) cc[k] = carry[k];
        through_waves(maps[buf], wave, lane % LR, carry, cc);
#pragma unroll
        for (int k = 0; k < V; ++k) cc[k] = fmaf(Ab[k], cc[k], Eb[k]);
        // The tile's oldest token is t0 - TS + 1, which a tile that is not full may have below 0.
        const int64_t at = ob + (t0 - TS + 1) * (int64_t)orow;
#pragma unroll
        for (int l = 0; l < L; ++l) {
            float ox[V], oi[V], orr[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float G = g[l][k] + cc[k];
                cc[k] = a[l][k] * G;
                ox[k] = G * fx[l][k];
                oi[k] = G * fi[l][k];
                orr[k] = G * fr[l][k];
                // A token that does not exist adds nothing, whatever its factors are.
                share[k] = l < rows ? fmaf(G, fd[l][k], share[k]) : share[k];
            }
            if (full || l < rows) {
                const int64_t o = at + (L - 1 - l) * (int64_t)orow;
                store_lane<T, MODE>(p.dx + o, oldest, col, ox);
                store_lane<T, MODE>(p.dr + o, oldest, col, orr);
                store_lane<T, MODE>(p.di + o, oldest, col, oi);
            }
        }
        raw = next;
    }
    // Tokens that do not exist: this segment's part of [n, T).
    const float zero[V] = {};
    for (int64_t t = n + (int64_t)seg * NW * RW + run; t < p.T; t += (int64_t)p.nseg * NW * RW) {
        const int64_t o = ob + t * (int64_t)orow;
        store_lane<T, MODE>(p.dx + o, 0, col, zero);
        store_lane<T, MODE>(p.dr + o, 0, col, zero);
        store_lane<T, MODE>(p.di + o, 0, col, zero);
    }
    if (p.h && seg == p.nseg - 1 && threadIdx.x < LR)      // p.h: the first state's gradient, fp32
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (k < col.have) reinterpret_cast<float *>(p.h)[b * p.C + c + k] = carry[k];
    // Shares of log_decay's gradient: over the runs of a wave, then over the waves.
#pragma unroll
    for (int dist = LR; dist < 64; dist *= 2)
#pragma unroll
        for (int k = 0; k < V; ++k) share[k] += __shfl_xor(share[k], dist);
    __syncthreads();
    if (lane < LR) put_maps(maps[0], wave, lane, share, share);
    __syncthreads();
    if (threadIdx.x >= LR) return;
    float *const o = p.part + (b * p.nseg + seg) * p.C + c;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        float sum = 0.0f;
        for (int w = 0; w < NW; ++w) sum += k % 2 ? maps[0].m[k / 2][w][lane].z : maps[0].m[k / 2][w][lane].x;
        if (k < col.have) o[k] = sum;
    }
}

template <typename T, int LR, int NW, bool SHORT>
__global__ __launch_bounds__(64 * NW) void gated_bwd_walk(const Walk p)
{
    __shared__ Maps<NW, LR, lane_channels<T>()> maps[2];
    int ct, seg;
    int64_t b;
    if (!place(p, p.nseg, ct, seg, b)) return;
    GATED_BODY(bwd_body, T, LR, NW);
}

// Sum over sequences and segments, in order: 64 rows at a time, then those 64.
constexpr int kShareCols = 16, kShareThreads = 64 * kShareCols;
__global__ __launch_bounds__(kShareThreads) void gated_share_sum(const float *__restrict__ part, float *__restrict__ out,
                                                                 int64_t rows, int64_t C)
{
    __shared__ float s[64][kShareCols + 1];
    const int col = threadIdx.x % kShareCols, row = threadIdx.x / kShareCols;
    const int64_t c = (int64_t)blockIdx.x * kShareCols + col;
    float v = 0.0f;
    if (c < C)
        for (int64_t r = row; r < rows; r += 64) v += part[r * C + c];
    s[row][col] = v;
    __syncthreads();
    if (row == 0 && c < C) {
        for (int r = 1; r < 64; ++r) v += s[r][col];
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

// Channels of a stripe, and tokens of a tile.
int stripe(const GatedPlan &g, int dtype) { return g.lanes * (dtype == DT_F32 ? 2 : 4); }
int tile_steps(const GatedPlan &g, int dtype, bool backward)
{
    return g.waves * (64 / g.lanes) * (dtype == DT_F32 ? (backward ? run_len_bwd<float>() : run_len<float>())
                                                    : (backward ? run_len_bwd<__bf16>() : run_len<__bf16>()));
}

Walk make_walk(const GatedArgs &a, const GatedPlan &g)
{
    const int64_t es = a.dtype == DT_F32 ? 4 : 2;
    Walk p = {};
    p.B = a.B; p.T = a.T; p.C = a.C; p.seg_len = g.seg_len; p.nseg = g.nseg;
    p.tiles = (int32_t)ceil_div(a.C, stripe(g, a.dtype));
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

// The kernels that exist: (lanes, waves, rows shorter than a lane's 8 bytes).
bool short_rows(int64_t C, int dtype) { return C < (dtype == DT_F32 ? 2 : 4); }
template <typename F> hipError_t with_shape(const GatedPlan &g, int64_t C, int dtype, F &&f)
{
    constexpr Int<0> whole{};
    if (short_rows(C, dtype)) return f(Int<32>{}, Int<4>{}, Int<1>{});
    if (g.lanes == 4) return f(Int<4>{}, Int<8>{}, whole);
    if (g.lanes == 8) return f(Int<8>{}, Int<8>{}, whole);
    if (g.lanes == 16) return f(Int<16>{}, Int<8>{}, whole);
    return g.waves == 8 ? f(Int<32>{}, Int<8>{}, whole) : f(Int<32>{}, Int<4>{}, whole);
}

template <bool BWD> hipError_t launch_states(Walk p, const GatedPlan &g, int dtype, hipStream_t stream)
{
    p.blocks = p.B * (g.nseg - 1) * p.tiles;
    const dim3 grid((unsigned)(8 * ceil_div(p.blocks, 8)));
    return with_type(dtype, [&](auto t) {
        return with_shape(g, p.C, dtype, [&](auto lanes, auto waves, auto one) {
            constexpr bool planned = lanes.value == 32 && (!BWD || waves.value == 4);      // of cut sequences
            if constexpr (planned) gated_states<decltype(t), lanes.value, waves.value, BWD, one.value><<<grid, 64 * waves.value, 0, stream>>>(p);
            return planned ? hipGetLastError() : hipErrorInvalidValue;
        });
    });
}

}  // namespace

// Up to 256 tokens: the shape whose tiles take the least time.  A workgroup's tile takes `alone` us where
// each has a compute unit to itself and `each` us for every one that a compute unit gets, nearly
// whatever part of the tile the tokens fill: 5 x 16 x 3840 in bf16 took 5.5 us in stripes of 32 lanes on
// four waves, 13.2 us of 8 and 20.5 us of 4 lanes on eight (gradients 8.8, 23 and 41), 5 x 256 x 3840
// 21, 15 and 23 us (41, 37 and 47).
GatedPlan short_plan(int64_t B, int64_t T, int64_t C, int dtype, bool backward)
{
    const int64_t lanes = ceil_div(C, dtype == DT_F32 ? 2 : 4);
    GatedPlan best = {};
    double least = 0.0;
    for (int L : {32, 16, 8, 4}) {
        if (backward && L == 16) continue;
        const GatedPlan g = {L, L == 32 ? 4 : 8, 1, std::max<int64_t>(T, 1)};
        const bool four = g.waves == 4;
        const double start = backward ? 6.5 : 4.0, alone = four ? 2.2 : 3.4,
                     each = four ? (backward ? 2.4 : 1.8) : backward ? 7.6 : 3.6;
        const double loads = (double)(std::max<int64_t>(B, 1) * ceil_div(lanes, L)) / 256;
        const double us = start + (double)ceil_div(std::max<int64_t>(T, 1), tile_steps(g, dtype, backward)) * std::max(alone, each * loads);
        if (least == 0.0 || us < least) {
            least = us;
            best = g;
        }
    }
    return best;
}

// Longer: stripes as wide as fill the card without cuts, or cut sequences.  A narrow stripe costs more for each
// lane: rows of 256, 128, 64 and 32 bytes took 225, 281, 323 and 364 us for 8 x 4096 x 4096 in bf16
// (factors 1, 1.25, 1.43 and 1.62), since neighbours that share lines are not in step.  A cut reads three of
// four tensors twice (1.65, and a launch worth 6500 lane-tokens; gradients two of eight, 1.17 and 5000).  With
// narrow stripes uncut, and cut, in bf16: 1 x 4096 x 4096 40 and 54 us, 2 x 8192 x 4096 151 and 190, 6 x 1021 x 1350
// 24 and 43, 1 x 32768 x 4096 397 and 382, 1 x 32768 x 2048 367 and 203; gradients of 4 x 4096 x 2560 334 and 192,
// of 8 x 1024 x 512 28 both.  The costs were fitted when a cut's fold was dearer, and are off by up to a quarter
// where both sides are near: 1 x 32768 x 4096 stays uncut (397), 6 x 5545 x 1024 and 5 x 2360 x 64 are cut (100 and
// 25 us; uncut 89 and 21).
GatedPlan gated_plan(int64_t B, int64_t T, int64_t C, int dtype, bool backward)
{
    GatedPlan g = {32, backward ? 4 : 8, 1, std::max<int64_t>(T, 1)};
    if (T <= 256 && !short_rows(C, dtype)) return short_plan(B, T, C, dtype, backward);
    const int64_t lanes = ceil_div(C, dtype == DT_F32 ? 2 : 4);      // of a row
    const double each = std::max(1.0, (double)std::max<int64_t>(B, 1) * lanes / 256);
    bool cut = true;
    if (short_rows(C, dtype)) {
        g.waves = 4;
    } else {
        double least = 0.0;
        for (int L : {32, 16, 8, 4}) {
            if (backward && (L == 32 || L == 16)) continue;
            const double factor = L == 32 ? 1.0 : L == 16 ? 1.25 : L == 8 ? 1.43 : 1.62;
            const double cost = (double)ceil_div(std::max<int64_t>(B, 1) * ceil_div(lanes, L), 256) * L * factor;
            if (least == 0.0 || cost < least) {
                least = cost;
                g.lanes = L;
            }
        }
        cut = (backward ? 1.17 : 1.65) * each * T + (backward ? 5000 : 6500) < least * T;
        if (cut) g.lanes = 32;
        else if (backward || g.lanes < 32) g.waves = 8;
    }
    if (!cut) return g;
    const int64_t stripes = std::max<int64_t>(1, B * ceil_div(C, stripe(g, dtype)));
    const int64_t ts = tile_steps(g, dtype, backward), tiles = ceil_div(std::max<int64_t>(T, 1), ts);
    g.nseg = (int32_t)std::max<int64_t>(1, std::min<int64_t>({512 / stripes, tiles / 2, 256}));
    const int64_t per = ceil_div(tiles, (int64_t)g.nseg);
    g.nseg = (int32_t)ceil_div(tiles, per);
    g.seg_len = per * ts;
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
    if (backward && !grid_fits(ceil_div(a.C, kShareCols), kShareThreads)) return false;
    return grid_fits(8 * ceil_div(a.B * g.nseg * ceil_div(a.C, stripe(g, a.dtype)), 8), 64 * g.waves);
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
        return with_shape(g, a.C, a.dtype, [&](auto lanes, auto waves, auto one) {
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
            return with_shape(g, a.C, a.dtype, [&](auto lanes, auto waves, auto one) {
                constexpr bool planned = lanes.value < 16 || waves.value == 4;
                if constexpr (planned) gated_bwd_walk<decltype(t), lanes.value, waves.value, one.value><<<grid, 64 * waves.value, 0, a.stream>>>(p);
                return planned ? hipGetLastError() : hipErrorInvalidValue;
            });
        });
        if (err != hipSuccess) return err;
    }
    gated_share_sum<<<(unsigned)ceil_div(a.C, kShareCols), kShareThreads, 0, a.stream>>>(p.part, a.dlog, a.B * g.nseg, a.C);
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
