// group_norm.hip -- group norm with an activation over channels-last tensors [N][P][C]:
//     y = act(w (x - mean) rstd + b),   mean and rstd = 1 / sqrt(var + eps) of a sample's group
// (its positions that exist times C / G channels), and its gradients.
//
// A workgroup takes a slab: the positions of one sample (or a chunk of them) times a bundle of
// whole groups.  A thread keeps one vector of V channels, all of one group, for every R-th
// position in registers.  Where a sample's bundle fits (up to 256 KB of registers) everything
// happens in one launch, x is read once and y written once; else one launch takes the statistics
// of chunks and a second one joins them and reads x again, which the last-level cache holds for
// tensors up to its 256 MB.
//
// Statistics: a thread's sum, and its squares about its own mean; joined exactly,
//     M2 = sum over threads of M2_t + n_t (mean_t - mean)^2,
// so an offset much larger than the spread does not cancel in the variance: it enters only by the square of
// a mean's rounding (a mean is off by a few 2^-24 of the offset).  The order of addition is fixed.
//
// Gradients: with xhat = (x - mean) rstd, dz = dy act'(w xhat + b), m = positions times channels,
//     dx = rstd (w dz - S1 / m - xhat S2 / m),  S1 = sum of w dz,  S2 = sum of w dz xhat,
//     dw = sum of dz xhat,  db = sum of dz  over samples and positions.
// dw and db leave each workgroup as fp32 partial sums; a last launch adds them in order.
//
// Bound by HBM; with silu two quarter-rate instructions an element, four in gradients.  64 x 784 x 2048
// in fp16 with silu takes 102 us (0.41 GB, 4.0 TB/s: a workgroup's load, statistics and stores follow one
// another, two workgroups of 1024 threads share a compute unit); a workgroup that stays and loads its next
// slab early holds two slabs in registers and took 133 us.  Gradients of 8 x 20480 x 256 in bf16: 47 us for
// the sums (0.17 GB, 3.6 TB/s), 44 for dx (0.25 GB, 5.7 TB/s), 5 for dw and db.
#include <algorithm>

#include "block.hpp"

namespace gconv {
namespace {

template <int BYTES> struct Words;
template <> struct Words<2> { typedef uint16_t type; };
template <> struct Words<4> { typedef uint32_t type __attribute__((aligned(2))); };
template <> struct Words<8> { typedef uint32_t type __attribute__((ext_vector_type(2), aligned(2))); };
template <> struct Words<16> { typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2))); };
template <typename T, int V> struct Vec { T v[V]; };

template <typename T, int V> __device__ __forceinline__ Vec<T, V> load_vec(const char *p)
{
    typedef typename Words<V * sizeof(T)>::type W;
    return __builtin_bit_cast(Vec<T, V>, *reinterpret_cast<const W *>(p));
}
template <typename T, int V> __device__ __forceinline__ void store_vec(char *p, const float (&f)[V])
{
    typedef typename Words<V * sizeof(T)>::type W;
    Vec<T, V> r;
#pragma unroll
    for (int k = 0; k < V; ++k) r.v[k] = from_f32<T>(f[k]);
    *reinterpret_cast<W *>(p) = __builtin_bit_cast(W, r);
}

__device__ __forceinline__ float sigmoid(float z)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * z));
}

// One position after the other: the temporaries of all at once would not fit beside the data.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// What a second pass over the registers computes it computes again: kept from the first, the fp32
// values of 16-bit data would take twice their registers.
template <typename T, int V, int K> __device__ __forceinline__ void forget(Vec<T, V> (&raw)[K])
{
    typedef typename Words<V * sizeof(T)>::type W;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if constexpr (sizeof(W) > 4) {
            W w = __builtin_bit_cast(W, raw[j]);
#pragma unroll
            for (int i = 0; i < (int)sizeof(W) / 4; ++i) {
                uint32_t u = w[i];
                asm volatile("" : "+v"(u));
                w[i] = u;
            }
            raw[j] = __builtin_bit_cast(Vec<T, V>, w);
        } else {
            uint32_t u = (uint32_t)__builtin_bit_cast(W, raw[j]);
            asm volatile("" : "+v"(u));
            raw[j] = __builtin_bit_cast(Vec<T, V>, (W)u);
        }
    }
}

struct Norm {
    const char *x, *dy, *w, *b;          // b may be nullptr
    char *y;                             // or dx
    const float *stats;                  // backward: (mean, rstd) [N][G][2]
    float *stats_out;                    // forward: the same, or nullptr
    float2 *chunk;                       // of chunks: (mean, M2), or (S1, S2) [N][G][chunks * parts]
    float *part;                         // (dw, db) [rows][2][C]
    const int32_t *lengths;
    int64_t N, P, C, blocks, rows, range;   // rows of `part`, samples of each
    int64_t xsb, xst, dsb, dst;          // bytes
    int32_t G, cg, kg, bundles, cols, R, parts, chunks, chunk_rows;
    int32_t join;                        // lanes that add up a group: a power of two up to 64
    float eps;
    int32_t silu;
};

constexpr int kMaxThreads = 1024;

// For each thread two pairs (one of its own, one of a group) and the cells of column sums.  As much as
// the workgroup uses: workgroups of a wave with room for 1024 threads, three to a compute unit, took 250 us
// for the gradients of 8192 x 4096 in bf16.
extern __shared__ float2 lds[];
constexpr size_t lds_bytes(int threads, int cells) { return (size_t)threads * (2 * sizeof(float2) + sizeof(float) * cells); }

struct Slab {
    int64_t n;             // sample (backward: the first of a range)
    int32_t chunk, bundle, part;
    int32_t first;         // position
    int32_t rows;          // positions that the chunk has
    int32_t c0;            // channel of the slab
    int32_t cols;          // vectors of a row
    int32_t groups;
};

__device__ __forceinline__ void slab_of(const Norm &p, int64_t id, Slab &s)
{
    const int64_t rest = id / p.bundles;
    const int at = (int)(id - rest * p.bundles);
    s.part = at % p.parts;
    s.bundle = at / p.parts;
    s.n = rest / p.chunks;
    s.chunk = (int)(rest - s.n * p.chunks);
    s.first = s.chunk * p.chunk_rows;
    s.rows = (int)min((int64_t)p.chunk_rows, p.P - s.first);
}

// A workgroup's slab: neighbouring bundles, which may share lines, on one XCD.
__device__ __forceinline__ bool find_slab(const Norm &p, Slab &s)
{
    const int64_t per = (p.blocks + 7) / 8, id = (int64_t)(blockIdx.x % 8) * per + blockIdx.x / 8;
    if (blockIdx.x / 8 >= per || id >= p.blocks) return false;
    slab_of(p, id, s);
    return true;
}

template <int V> __device__ __forceinline__ void slab_columns(const Norm &p, Slab &s)
{
    s.groups = min(p.kg, p.G - s.bundle * p.kg);
    s.c0 = s.bundle * p.kg * p.cg + s.part * p.cols * V;
    s.cols = p.parts > 1 ? min(p.cols, p.cg / V - s.part * p.cols) : s.groups * (p.cg / V);
}

__device__ __forceinline__ int live_rows(const Norm &p, int64_t n, const Slab &s)
{
    int64_t live = p.P;
    if (p.lengths) live = max((int64_t)0, min(p.P, (int64_t)p.lengths[n]));
    return (int)max((int64_t)0, min((int64_t)s.rows, live - s.first));
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
    return v;
}

// Sum over aligned runs of `lanes` (a power of two).
__device__ __forceinline__ float lanes_sum(float v, int lanes)
{
    for (int d = lanes / 2; d; d /= 2) v += __shfl_xor(v, d);
    return v;
}

// Threads of a group, in the order in which its lanes take them: lane, lane + lanes, ...
struct Members {
    int r, j, dr, dj, width, R;
    __device__ Members(int lane, int lanes, int width, int R) : width(width), R(R)
    {
        r = lane / width; j = lane - r * width;
        dr = lanes / width; dj = lanes - dr * width;
    }
    __device__ bool on() const { return r < R; }
    __device__ void next()
    {
        r += dr; j += dj;
        if (j >= width) { j -= width; ++r; }
    }
};

// Elements of a thread that starts at row r of `live` rows, R apart.
__device__ __forceinline__ float count_of(int r, int live, int R, int V) { return r < live ? (float)(V * ((live - 1 - r) / R + 1)) : 0.0f; }

// Sums of two values over the threads of each group: written to out[group] by the first of its lanes.
template <int V>
__device__ __forceinline__ void group_sums(const Norm &p, const Slab &s, int tid, float a, float b, float2 *mine, float2 *out)
{
    mine[tid] = make_float2(a, b);
    __syncthreads();
    const int lane = tid % p.join, width = p.parts > 1 ? s.cols : p.cg / V;
    for (int g = tid / p.join; g < s.groups; g += blockDim.x / p.join) {
        float sa = 0.0f, sb = 0.0f;
        for (Members m(lane, p.join, width, p.R); m.on(); m.next()) {
            const float2 v = mine[m.r * p.cols + g * width + m.j];
            sa += v.x;
            sb += v.y;
        }
        sa = lanes_sum(sa, p.join);
        sb = lanes_sum(sb, p.join);
        if (lane == 0) out[g] = make_float2(sa, sb);
    }
    __syncthreads();
}

// ---------------------------------------------------------------- forward

// Statistics of each group from its threads' sums and squares about their own means, of `live` rows:
// done(group, mean, M2) in one lane.
template <int V, typename F>
__device__ __forceinline__ void join_threads(const Norm &p, const Slab &s, int tid, int live, float2 own, float2 *mine, F &&done)
{
    mine[tid] = own;
    __syncthreads();
    const int lane = tid % p.join, width = p.parts > 1 ? s.cols : p.cg / V;
    const float total = fmaxf((float)live * (width * V), 1.0f);
    for (int g = tid / p.join; g < s.groups; g += blockDim.x / p.join) {
        float a = 0.0f, q = 0.0f;
        for (Members m(lane, p.join, width, p.R); m.on(); m.next()) a += mine[m.r * p.cols + g * width + m.j].x;
        const float mean = lanes_sum(a, p.join) / total;
        for (Members m(lane, p.join, width, p.R); m.on(); m.next()) {
            const float2 v = mine[m.r * p.cols + g * width + m.j];
            const float n = count_of(m.r, live, p.R, V);
            if (n > 0.0f) {
                const float d = v.x / n - mean;
                q += fmaf(n * d, d, v.y);
            }
        }
        q = lanes_sum(q, p.join);
        if (lane == 0) done(g, mean, q);
    }
}

// Sum, and squares about its own mean, of what a thread holds: rows r0, r0 + R, ... below `live`.
template <typename T, int V, int K>
__device__ __forceinline__ float2 own_stats(Vec<T, V> (&raw)[K], bool on, int r0, int R, int live)
{
    float sum = 0.0f, m2 = 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (on && r0 + j * R < live)
#pragma unroll
            for (int k = 0; k < V; ++k) sum += to_f32(raw[j].v[k]);
    forget<T, V, K>(raw);
    const float own = on ? sum / fmaxf(count_of(r0, live, R, V), 1.0f) : 0.0f;
#pragma unroll
    for (int j = 0; j < K; ++j) {
        if (on && r0 + j * R < live)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float d = to_f32(raw[j].v[k]) - own;
                m2 = fmaf(d, d, m2);
            }
        keep_order();
    }
    forget<T, V, K>(raw);
    return make_float2(sum, m2);
}

template <typename T, int V>
__device__ __forceinline__ void normed(const Norm &p, const Vec<T, V> &x, float2 st, const Vec<T, V> &w, const Vec<T, V> &b, bool live,
                                       char *to)
{
    float f[V];
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = fmaf(to_f32(x.v[k]) - st.x, st.y * to_f32(w.v[k]), to_f32(b.v[k]));
    if (p.silu)     // one branch for all: the channels' exponentials overlap
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] *= sigmoid(f[k]);
    if (!live)
#pragma unroll
        for (int k = 0; k < V; ++k) f[k] = 0.0f;
    store_vec<T, V>(to, f);
}

// Positions of a tile: K for each thread.  A chunk is a row of tiles, the next one's loads under way
// while one is worked on.
template <typename T, int V, int K>
__device__ __forceinline__ void load_tile(const char *base, int64_t st, uint32_t from, bool on, int r0, int R, int first, int live,
                                          Vec<T, V> (&raw)[K])
{
    const char *const x = base + first * st;
#pragma unroll
    for (int j = 0; j < K; ++j)
        if (on && first + r0 + j * R < live) raw[j] = load_vec<T, V>(x + j * (R * st) + from);
}

// The whole sample in registers; of single positions several samples, one after the other, the next
// one's loads under way.
template <typename T, int V, int K>
__global__ __launch_bounds__(kMaxThreads) void gn_forward(const Norm p)
{
    float2 *const mine = lds;
    float2 *const out = lds + blockDim.x;
    Slab s;
    if (!find_slab(p, s)) return;
    slab_columns<V>(p, s);
    const int tid = threadIdx.x, r0 = tid / p.cols, col = tid - r0 * p.cols, width = p.cg / V;
    const bool on = r0 < p.R && col < s.cols;
    const uint32_t here = (uint32_t)(col * V * sizeof(T)), from = (uint32_t)r0 * (uint32_t)p.xst + here;
    const int64_t c = s.c0 + (int64_t)col * V, row = p.C * (int64_t)sizeof(T);
    const uint32_t to = (uint32_t)r0 * (uint32_t)row + here;
    const int64_t past = K == 1 ? min((s.n + 1) * p.range, p.N) : s.n + 1;
    const int g = on ? col / width : 0;
    Vec<T, V> raw[K], next[1], w, b = {};
    const auto affine = [&] {
        w = load_vec<T, V>(p.w + c * (int64_t)sizeof(T));
        if (p.b) b = load_vec<T, V>(p.b + c * (int64_t)sizeof(T));
    };
    int64_t n = K == 1 ? s.n * p.range : s.n;
    int live = live_rows(p, n, s);
    const char *x = p.x + n * p.xsb + s.c0 * (int64_t)sizeof(T);
    load_tile<T, V, K>(x, p.xst, from, on, r0, p.R, 0, live, raw);
    if (K == 1 && on) affine();
    while (true) {
        int after = 0;
        if constexpr (K == 1)
            if (n + 1 < past) {
                x += p.xsb;
                after = live_rows(p, n + 1, s);
                load_tile<T, V, K>(x, p.xst, from, on, r0, p.R, 0, after, next);
            }
        const float total = fmaxf((float)live * p.cg, 1.0f);
        join_threads<V>(p, s, tid, live, own_stats<T, V, K>(raw, on, r0, p.R, live), mine, [&](int of, float mean, float q) {
            const float2 v = make_float2(mean, 1.0f / sqrtf(q / total + p.eps));
            out[of] = v;
            if (p.stats_out) reinterpret_cast<float2 *>(p.stats_out)[n * p.G + s.bundle * p.kg + of] = v;
        });
        __syncthreads();
        if (on) {
            const float2 st = out[g];
            if (K > 1) affine();
            char *const y = p.y + (n * p.P * p.C + s.c0) * (int64_t)sizeof(T);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                const int r = r0 + j * p.R;
                if (r < s.rows) normed<T, V>(p, raw[j], st, w, b, r < live, y + j * (p.R * row) + to);
                keep_order();
            }
        }
        if constexpr (K > 1) return;
        if (++n >= past) return;
        raw[0] = next[0];
        live = after;
    }
}

constexpr int64_t kPartRows = 1024;
constexpr int kTile = 4, kTileBwd = 2;

template <typename T, int V>
__global__ __launch_bounds__(kMaxThreads) void gn_chunk_stats(const Norm p)
{
    constexpr int K = kTile;
    float2 *const mine = lds;
    Slab s;
    if (!find_slab(p, s)) return;
    slab_columns<V>(p, s);
    const int tid = threadIdx.x, r0 = tid / p.cols, col = tid - r0 * p.cols, live = live_rows(p, s.n, s);
    const bool on = r0 < p.R && col < s.cols;
    const char *const x = p.x + s.n * p.xsb + s.first * p.xst + s.c0 * (int64_t)sizeof(T);
    const uint32_t from = (uint32_t)r0 * (uint32_t)p.xst + (uint32_t)(col * V * sizeof(T));
    Vec<T, V> raw[K], next[K];
    load_tile<T, V, K>(x, p.xst, from, on, r0, p.R, 0, live, raw);
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    for (int first = 0; first < live; first += p.R * K) {
        load_tile<T, V, K>(x, p.xst, from, on, r0, p.R, first + p.R * K, live, next);
        const float2 own = own_stats<T, V, K>(raw, on, r0, p.R, min(live - first, p.R * K));
        const float nb = on ? count_of(r0, min(live - first, p.R * K), p.R, V) : 0.0f;
        if (nb > 0.0f) {
            const float d = own.x / nb - mean, all = n + nb, part = nb / all;
            mean = fmaf(d, part, mean);
            m2 += fmaf(d * d, n * part, own.y);
            n = all;
        }
#pragma unroll
        for (int j = 0; j < K; ++j) raw[j] = next[j];
    }
    join_threads<V>(p, s, tid, live, make_float2(mean * n, m2), mine, [&](int g, float all, float q) {
        p.chunk[(s.n * p.G + s.bundle * p.kg + g) * (p.chunks * p.parts) + s.chunk * p.parts + s.part] = make_float2(all, q);
    });
}

template <typename T, int V>
__global__ __launch_bounds__(kMaxThreads) void gn_chunk_apply(const Norm p)
{
    constexpr int K = kTile;
    float2 *const out = lds;
    Slab s;
    if (!find_slab(p, s)) return;
    slab_columns<V>(p, s);
    const int tid = threadIdx.x, lane = tid % 64, r0 = tid / p.cols, col = tid - r0 * p.cols, live = live_rows(p, s.n, s);
    const bool on = r0 < p.R && col < s.cols;
    const int64_t c = s.c0 + (int64_t)col * V;
    const char *const x = p.x + s.n * p.xsb + s.first * p.xst + s.c0 * (int64_t)sizeof(T);
    const uint32_t from = (uint32_t)r0 * (uint32_t)p.xst + (uint32_t)(col * V * sizeof(T));
    Vec<T, V> raw[K], next[K], w = {}, b = {};
    load_tile<T, V, K>(x, p.xst, from, on, r0, p.R, 0, live, raw);
    if (on) {
        w = load_vec<T, V>(p.w + c * (int64_t)sizeof(T));
        if (p.b) b = load_vec<T, V>(p.b + c * (int64_t)sizeof(T));
    }
    // Statistics of the chunks, joined as those of threads are.
    int64_t all = p.P;
    if (p.lengths) all = max((int64_t)0, min(p.P, (int64_t)p.lengths[s.n]));
    const int slots = p.chunks * p.parts;
    const float total = fmaxf((float)all * p.cg, 1.0f);
    auto size = [&](int i) {        // elements of slot i
        const int ch = i / p.parts, pt = i - ch * p.parts;
        const int64_t first = (int64_t)ch * p.chunk_rows;
        const int64_t r = max((int64_t)0, min(min((int64_t)p.chunk_rows, p.P - first), all - first));
        return (float)r * (p.parts > 1 ? min(p.cols * V, p.cg - pt * p.cols * V) : p.cg);
    };
    for (int g = tid / 64; g < s.groups; g += blockDim.x / 64) {
        const int64_t at = s.n * p.G + s.bundle * p.kg + g;
        const float2 *const of = p.chunk + at * slots;
        float a = 0.0f, q = 0.0f;
        for (int i = lane; i < slots; i += 64) a = fmaf(size(i), of[i].x, a);
        const float mean = wave_sum(a) / total;
        for (int i = lane; i < slots; i += 64) {
            const float2 v = of[i];
            const float d = v.x - mean;
            q += fmaf(size(i) * d, d, v.y);
        }
        q = wave_sum(q);
        if (lane == 0) {
            const float2 v = make_float2(mean, 1.0f / sqrtf(q / total + p.eps));
            out[g] = v;
            if (p.stats_out && s.chunk == 0 && s.part == 0) reinterpret_cast<float2 *>(p.stats_out)[at] = v;
        }
    }
    __syncthreads();
    if (!on) return;
    const float2 st = out[p.parts > 1 ? 0 : col / (p.cg / V)];
    const int64_t row = p.C * (int64_t)sizeof(T);
    char *const y = p.y + (s.n * p.P + s.first) * row + s.c0 * (int64_t)sizeof(T);
    const uint32_t to = (uint32_t)r0 * (uint32_t)row + (uint32_t)(col * V * sizeof(T));
    for (int first = 0; first < s.rows; first += p.R * K) {
        load_tile<T, V, K>(x, p.xst, from, true, r0, p.R, first + p.R * K, live, next);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int r = first + r0 + j * p.R;
            if (r < s.rows) normed<T, V>(p, raw[j], st, w, b, r < live, y + first * row + j * (p.R * row) + to);
            keep_order();
        }
#pragma unroll
        for (int j = 0; j < K; ++j) raw[j] = next[j];
    }
}

// ---------------------------------------------------------------- backward

// d = x - mean and dz = dy act'(z), z = a d + b with a = w rstd.
template <typename T, int V>
__device__ __forceinline__ void slopes(const Vec<T, V> &x, const Vec<T, V> &dy, const float (&a)[V], const float (&b)[V], float mean,
                                       int silu, float (&d)[V], float (&dz)[V])
{
#pragma unroll
    for (int k = 0; k < V; ++k) {
        d[k] = to_f32(x.v[k]) - mean;
        dz[k] = to_f32(dy.v[k]);
    }
    if (silu)       // one branch for all: the channels' exponentials overlap
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const float z = fmaf(d[k], a[k], b[k]), sg = sigmoid(z);
            dz[k] *= fmaf(z * sg, 1.0f - sg, sg);
        }
}

// Sums of each column's values over the rows of threads: col_sums[0..cols V) of `out`, for the
// thread's own V values.
template <int V>
__device__ __forceinline__ void column_sums(const Norm &p, const Slab &s, int tid, int r0, int col, const float (&v)[V], float *mine,
                                            float *out)
{
    const int W = s.cols * V, step = p.cols * V;
    __syncthreads();
    if (r0 < p.R && col < s.cols)
#pragma unroll
        for (int k = 0; k < V; ++k) mine[r0 * step + col * V + k] = v[k];
    __syncthreads();
    // The rows in `parts` interleaved shares, then the shares.
    const int parts = min(p.R, max(1, (int)blockDim.x / W));
    for (int u = tid; u < W * parts; u += blockDim.x) {
        const int part = u / W, c = u - part * W;
        float a = 0.0f;
        for (int r = part; r < p.R; r += parts) a += mine[r * step + c];
        mine[part * step + c] = a;      // this thread's own first row
    }
    __syncthreads();
    for (int c = tid; c < W; c += blockDim.x) {
        float a = 0.0f;
        for (int r = 0; r < parts; ++r) a += mine[r * step + c];
        out[c] = a;
    }
}

// A thread's weights and biases.
template <typename T, int V>
__device__ __forceinline__ void load_affine(const Norm &p, bool on, int64_t c, float (&w)[V], float (&b)[V])
{
    Vec<T, V> wr = {}, br = {};
    if (on) {
        wr = load_vec<T, V>(p.w + c * (int64_t)sizeof(T));
        if (p.b) br = load_vec<T, V>(p.b + c * (int64_t)sizeof(T));
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
        w[k] = to_f32(wr.v[k]);
        b[k] = to_f32(br.v[k]);
    }
}

// What a thread's vector adds to its sums of dz d and of dz.  (dw, db, and S1, S2 of its group all
// follow from those.)
template <typename T, int V>
__device__ __forceinline__ void add_sums(const Norm &p, const Vec<T, V> &x, const Vec<T, V> &dy, const float (&a)[V], const float (&b)[V],
                                         float mean, float (&sd)[V], float (&sz)[V])
{
    float d[V], dz[V];
    slopes<T, V>(x, dy, a, b, mean, p.silu, d, dz);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        sd[k] = fmaf(dz[k], d[k], sd[k]);
        sz[k] += dz[k];
    }
}

// dx = a dz - rstd S1 / m - d rstd^2 S2 / m: c1 = rstd S1 / m, c2 = rstd^2 S2 / m.
template <typename T, int V>
__device__ __forceinline__ void input_slope(const Norm &p, const Vec<T, V> &x, const Vec<T, V> &dy, const float (&a)[V], const float (&b)[V],
                                            float mean, float c1, float c2, bool live, char *to)
{
    float d[V], dz[V], f[V];
    slopes<T, V>(x, dy, a, b, mean, p.silu, d, dz);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = live ? fmaf(a[k], dz[k], -fmaf(d[k], c2, c1)) : 0.0f;
    store_vec<T, V>(to, f);
}

__device__ __forceinline__ float per_element(const Norm &p, int64_t n)
{
    int64_t all = p.P;
    if (p.lengths) all = max((int64_t)0, min(p.P, (int64_t)p.lengths[n]));
    return 1.0f / fmaxf((float)all * p.cg, 1.0f);
}

// (mean, rstd) of a group for the sums over its `live` rows.  Without rows the sums are zero, and rstd, which
// is infinite where eps is zero, must not multiply them.
__device__ __forceinline__ float2 group_stats(const Norm &p, int64_t at, int live)
{
    float2 st = reinterpret_cast<const float2 *>(p.stats)[at];
    if (live == 0) st.y = 0.0f;
    return st;
}

// Whole samples in registers: a range of them, their dw and db added up on the way.
//
// With more than four vectors of 16 bytes a thread the sample's x and dy do not fit the 128 registers of a
// workgroup of 1024 threads: 136 (fp32) to 176 bytes a lane go to scratch memory, and 64 x 784 x 2048 in fp16
// takes 296 us for the 94 of its bytes.  Eight 16-bit channels in up to four vectors keep 12 bytes there.
template <typename T, int V, int K>
__global__ __launch_bounds__(kMaxThreads) void gn_backward(const Norm p)
{
    float2 *const mine = lds;
    float2 *const out = lds + blockDim.x;
    float *const cells = (float *)(lds + 2 * blockDim.x);
    Slab s;
    if (!find_slab(p, s)) return;
    slab_columns<V>(p, s);
    const int tid = threadIdx.x, r0 = tid / p.cols, col = tid - r0 * p.cols;
    const bool on = r0 < p.R && col < s.cols;
    const int64_t c = s.c0 + (int64_t)col * V, row = p.C * (int64_t)sizeof(T);
    const int g = on ? col / (p.cg / V) : 0;
    const uint32_t at0 = (uint32_t)(col * V * sizeof(T)), xat = (uint32_t)r0 * (uint32_t)p.xst + at0,
                   dat = (uint32_t)r0 * (uint32_t)p.dst + at0, to = (uint32_t)r0 * (uint32_t)row + at0;
    // Sums over samples: with more than one position a thread in LDS, its registers hold the sample.
    float b[V], dw[V] = {}, db[V] = {};
    if constexpr (K > 1)
#pragma unroll
        for (int k = 0; k < 2 * V; ++k) cells[k * blockDim.x + tid] = 0.0f;
    // Of single positions the next sample's loads are under way.
    const int64_t from = s.n * p.range, past = min(from + p.range, p.N);
    Vec<T, V> xr[K], dr[K], xn[1], dn[1];
    int live = 0, after = 0;
    float2 st = {}, stn = {};
    float weight[V];
    const auto load = [&](int64_t n, int &live, float2 &st, auto &xr, auto &dr) {
        live = live_rows(p, n, s);
        load_tile<T, V, K>(p.x + n * p.xsb + s.c0 * (int64_t)sizeof(T), p.xst, xat, on, r0, p.R, 0, live, xr);
        load_tile<T, V, K>(p.dy + n * p.dsb + s.c0 * (int64_t)sizeof(T), p.dst, dat, on, r0, p.R, 0, live, dr);
        st = group_stats(p, n * p.G + s.bundle * p.kg + g, live);
    };
    if constexpr (K == 1)
        if (from < past) {
            load(from, after, stn, xn, dn);
            load_affine<T, V>(p, on, c, weight, b);
        }
    for (int64_t n = from; n < past; ++n) {
        float a[V], sd[V] = {}, sz[V] = {}, s1 = 0.0f, s2 = 0.0f;
        if constexpr (K == 1) {
            xr[0] = xn[0]; dr[0] = dn[0];
            live = after; st = stn;
            if (n + 1 < past) load(n + 1, after, stn, xn, dn);
#pragma unroll
            for (int k = 0; k < V; ++k) a[k] = weight[k];
        } else {
            load(n, live, st, xr, dr);
            load_affine<T, V>(p, on, c, a, b);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) a[k] *= st.y;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (on && r0 + j * p.R < live) add_sums<T, V>(p, xr[j], dr[j], a, b, st.x, sd, sz);
            keep_order();
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (K > 1) {
                cells[k * blockDim.x + tid] = fmaf(sd[k], st.y, cells[k * blockDim.x + tid]);
                cells[(V + k) * blockDim.x + tid] += sz[k];
            } else {
                dw[k] = fmaf(sd[k], st.y, dw[k]);
                db[k] += sz[k];
            }
            s1 = fmaf(a[k], sz[k], s1);      // rstd S1
            s2 = fmaf(a[k], sd[k], s2);
        }
        group_sums<V>(p, s, tid, s1, s2, mine, out);
        forget<T, V, K>(xr);
        forget<T, V, K>(dr);
        const float inv = per_element(p, n), c1 = out[g].x * inv, c2 = out[g].y * inv * st.y * st.y;
        char *const dx = p.y + (n * p.P * p.C + s.c0) * (int64_t)sizeof(T);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int r = r0 + j * p.R;
            if (on && r < s.rows) input_slope<T, V>(p, xr[j], dr[j], a, b, st.x, c1, c2, r < live, dx + j * (p.R * row) + to);
            keep_order();
        }
        // `out` is written next behind the barrier that the next sample's pairs wait at.
    }
    if constexpr (K > 1)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            dw[k] = cells[k * blockDim.x + tid];
            db[k] = cells[(V + k) * blockDim.x + tid];
        }
    float *const o = p.part + s.n * 2 * p.C + s.c0;
    column_sums<V>(p, s, tid, r0, col, dw, cells, o);
    column_sums<V>(p, s, tid, r0, col, db, cells, o + p.C);
}

// Chunks: S1, S2 and the partial dw, db first, then dx.  RANGES: a chunk is a whole sample, and a workgroup takes
// a range of samples one after the other, so that they share a row of partial sums (16-bit vectors of 8 channels
// then keep some 36 bytes a lane in scratch memory).
template <typename T, int V, bool RANGES>
__global__ __launch_bounds__(kMaxThreads) void gn_chunk_sums(const Norm p)
{
    constexpr int K = kTileBwd;
    float2 *const mine = lds;
    float2 *const out = lds + blockDim.x;
    float *const cells = (float *)(lds + 2 * blockDim.x);
    Slab s;
    if (!find_slab(p, s)) return;
    slab_columns<V>(p, s);
    const int tid = threadIdx.x, r0 = tid / p.cols, col = tid - r0 * p.cols;
    const bool on = r0 < p.R && col < s.cols;
    const int64_t c = s.c0 + (int64_t)col * V, past = min((s.n + 1) * p.range, p.N);
    const uint32_t at0 = (uint32_t)(col * V * sizeof(T)), xat = (uint32_t)r0 * (uint32_t)p.xst + at0, dat = (uint32_t)r0 * (uint32_t)p.dst + at0;
    float dw[V] = {}, db[V] = {};
    int64_t n = RANGES ? s.n * p.range : s.n;
    do {
        const int live = live_rows(p, n, s);
        const int64_t at = n * p.G + s.bundle * p.kg;
        const char *const x = p.x + n * p.xsb + s.first * p.xst + s.c0 * (int64_t)sizeof(T);
        const char *const dy = p.dy + n * p.dsb + s.first * p.dst + s.c0 * (int64_t)sizeof(T);
        Vec<T, V> xr[K], dr[K], xn[K], dn[K];
        load_tile<T, V, K>(x, p.xst, xat, on, r0, p.R, 0, live, xr);
        load_tile<T, V, K>(dy, p.dst, dat, on, r0, p.R, 0, live, dr);
        float a[V], b[V], sd[V] = {}, sz[V] = {}, s1 = 0.0f, s2 = 0.0f;
        load_affine<T, V>(p, on, c, a, b);
        const float2 st = group_stats(p, at + (on && p.parts == 1 ? col / (p.cg / V) : 0), live);
#pragma unroll
        for (int k = 0; k < V; ++k) a[k] *= st.y;
        for (int first = 0; first < live; first += p.R * K) {
            load_tile<T, V, K>(x, p.xst, xat, on, r0, p.R, first + p.R * K, live, xn);
            load_tile<T, V, K>(dy, p.dst, dat, on, r0, p.R, first + p.R * K, live, dn);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                if (on && first + r0 + j * p.R < live) add_sums<T, V>(p, xr[j], dr[j], a, b, st.x, sd, sz);
                keep_order();
            }
#pragma unroll
            for (int j = 0; j < K; ++j) {
                xr[j] = xn[j];
                dr[j] = dn[j];
            }
        }
        load_affine<T, V>(p, on, c, a, b);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            sd[k] *= st.y;
            dw[k] = RANGES ? dw[k] + sd[k] : sd[k];
            db[k] = RANGES ? db[k] + sz[k] : sz[k];
            s1 = fmaf(a[k], sz[k], s1);
            s2 = fmaf(a[k], sd[k], s2);
        }
        group_sums<V>(p, s, tid, s1, s2, mine, out);
        // `out` is written next behind the barrier that the next sample's pairs wait at.
        for (int g = tid; g < s.groups; g += blockDim.x) p.chunk[(at + g) * (p.chunks * p.parts) + s.chunk * p.parts + s.part] = out[g];
    } while (RANGES && ++n < past);
    float *const o = p.part + (s.n * p.chunks + s.chunk) * 2 * p.C + s.c0;
    column_sums<V>(p, s, tid, r0, col, dw, cells, o);
    column_sums<V>(p, s, tid, r0, col, db, cells, o + p.C);
}

template <typename T, int V>
__global__ __launch_bounds__(kMaxThreads) void gn_chunk_slopes(const Norm p)
{
    constexpr int K = kTileBwd;
    float2 *const out = lds;
    Slab s;
    if (!find_slab(p, s)) return;
    slab_columns<V>(p, s);
    const int tid = threadIdx.x, lane = tid % 64, r0 = tid / p.cols, col = tid - r0 * p.cols, live = live_rows(p, s.n, s);
    const bool on = r0 < p.R && col < s.cols;
    const int64_t c = s.c0 + (int64_t)col * V, at = s.n * p.G + s.bundle * p.kg, row = p.C * (int64_t)sizeof(T);
    const uint32_t at0 = (uint32_t)(col * V * sizeof(T)), xat = (uint32_t)r0 * (uint32_t)p.xst + at0,
                   dat = (uint32_t)r0 * (uint32_t)p.dst + at0, to = (uint32_t)r0 * (uint32_t)row + at0;
    const char *const x = p.x + s.n * p.xsb + s.first * p.xst + s.c0 * (int64_t)sizeof(T);
    const char *const dy = p.dy + s.n * p.dsb + s.first * p.dst + s.c0 * (int64_t)sizeof(T);
    Vec<T, V> xr[K], dr[K], xn[K], dn[K];
    load_tile<T, V, K>(x, p.xst, xat, on, r0, p.R, 0, live, xr);
    load_tile<T, V, K>(dy, p.dst, dat, on, r0, p.R, 0, live, dr);
    float a[V], b[V];
    load_affine<T, V>(p, on, c, a, b);
    const int slots = p.chunks * p.parts;
    for (int k = tid / 64; k < s.groups; k += blockDim.x / 64) {
        float s1 = 0.0f, s2 = 0.0f;
        for (int i = lane; i < slots; i += 64) {
            const float2 v = p.chunk[(at + k) * slots + i];
            s1 += v.x;
            s2 += v.y;
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if (lane == 0) out[k] = make_float2(s1, s2);
    }
    __syncthreads();
    if (!on) return;
    const int g = p.parts > 1 ? 0 : col / (p.cg / V);
    const float2 st = reinterpret_cast<const float2 *>(p.stats)[at + g];
    const float inv = per_element(p, s.n) * st.y, c1 = out[g].x * inv, c2 = out[g].y * inv * st.y;
#pragma unroll
    for (int k = 0; k < V; ++k) a[k] *= st.y;
    char *const dx = p.y + (s.n * p.P + s.first) * row + s.c0 * (int64_t)sizeof(T);
    for (int first = 0; first < s.rows; first += p.R * K) {
        load_tile<T, V, K>(x, p.xst, xat, true, r0, p.R, first + p.R * K, live, xn);
        load_tile<T, V, K>(dy, p.dst, dat, true, r0, p.R, first + p.R * K, live, dn);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const int r = first + r0 + j * p.R;
            if (r < s.rows) input_slope<T, V>(p, xr[j], dr[j], a, b, st.x, c1, c2, r < live, dx + first * row + j * (p.R * row) + to);
            keep_order();
        }
#pragma unroll
        for (int j = 0; j < K; ++j) {
            xr[j] = xn[j];
            dr[j] = dn[j];
        }
    }
}

// Partial sums [rows][2][C] -> dw [C], db [C] (or nullptr), in order: 64 rows at a time, eight of a
// thread's loads at once, then those 64.
template <typename T>
__global__ __launch_bounds__(1024) void gn_param_sum(const float *__restrict__ part, T *__restrict__ dw, T *__restrict__ db, int64_t rows,
                                                     int64_t C)
{
    __shared__ float s[64][17];
    const int col = threadIdx.x % 16, row = threadIdx.x / 16;
    const int64_t c = (int64_t)blockIdx.x * 16 + col;
    float v = 0.0f;
    if (c < 2 * C) {
        int64_t r = row;
        for (; r + 7 * 64 < rows; r += 8 * 64) {
            float a[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = part[(r + 64 * i) * 2 * C + c];
#pragma unroll
            for (int i = 0; i < 8; ++i) v += a[i];
        }
        for (; r < rows; r += 64) v += part[r * 2 * C + c];
    }
    s[row][col] = v;
    __syncthreads();
    if (row == 0 && c < 2 * C) {
        for (int r = 1; r < 64; ++r) v += s[r][col];
        if (c < C) dw[c] = from_f32<T>(v);
        else if (db) db[c - C] = from_f32<T>(v);
    }
}

// ---------------------------------------------------------------- plans and launches

template <int N> struct Int { static constexpr int value = N; };

template <typename F> hipError_t with_vec(int dtype, int V, F &&f)
{
    auto by = [&](auto t) {
        if constexpr (sizeof(t) == 2)
            if (V == 8) return f(t, Int<8>{});
        return V == 4 ? f(t, Int<4>{}) : V == 2 ? f(t, Int<2>{}) : f(t, Int<1>{});
    };
    return dtype == DT_F32 ? by(float{}) : dtype == DT_F16 ? by(_Float16{}) : by(__bf16{});
}
template <typename F> void with_rows(int K, F &&f)
{
    if (K <= 1) f(Int<1>{});
    else if (K <= 4) f(Int<4>{});
    else if (K <= 8) f(Int<8>{});
    else f(Int<16>{});
}

// f(kernel type, vector) of a call; the kernels of whole samples also by K.
template <typename F> hipError_t launch_with(const Norm &p, const GroupNormArgs &a, const GroupNormPlan &g, F &&f)
{
    const dim3 grid((unsigned)(8 * ceil_div(p.blocks, 8)));
    return with_vec(a.dtype, g.V, [&](auto t, auto v) {
        f(t, v, grid);
        return hipGetLastError();
    });
}

Norm make_norm(const GroupNormArgs &a, const GroupNormPlan &g)
{
    const int64_t es = a.dtype == DT_F32 ? 4 : 2;
    Norm p = {};
    p.x = (const char *)a.x; p.dy = (const char *)a.dy; p.w = (const char *)a.weight; p.b = (const char *)a.bias; p.y = (char *)a.y;
    p.stats = a.stats; p.stats_out = a.stats_out; p.lengths = a.lengths;
    p.N = a.N; p.P = a.P; p.C = a.C; p.G = (int32_t)a.G; p.cg = (int32_t)(a.C / a.G);
    p.xsb = a.xsb * es; p.xst = a.P > 1 ? a.xst * es : 0; p.dsb = a.dsb * es; p.dst = a.P > 1 ? a.dst * es : 0;
    p.kg = g.kg; p.cols = g.cols; p.R = g.threads / g.cols; p.parts = g.parts; p.chunks = g.chunks; p.chunk_rows = g.chunk_rows;
    p.bundles = (int32_t)ceil_div(a.G, g.kg) * g.parts;
    // All groups at once where a workgroup has that many lanes: one wave took 32 groups of two threads one after
    // the other in 26 us.
    p.join = 64;
    while (p.join > 1 && p.join * g.kg > g.threads) p.join /= 2;
    p.range = g.range;
    p.blocks = ceil_div(a.N, g.range) * g.chunks * p.bundles;
    p.rows = ceil_div(a.N, g.range) * g.chunks;
    p.eps = a.eps; p.silu = a.silu;
    p.chunk = (float2 *)a.ws;
    p.part = (float *)((char *)a.ws + gn_chunk_bytes(g, a.N, a.G));
    return p;
}

}  // namespace

size_t gn_chunk_bytes(const GroupNormPlan &g, int64_t N, int64_t G)
{
    return g.whole ? 0 : (sizeof(float2) * (size_t)(N * G * g.chunks * g.parts) + 255) & ~(size_t)255;
}

GroupNormPlan gn_plan(int64_t N, int64_t P, int64_t C, int64_t G, int dtype, bool backward)
{
    const int es = dtype == DT_F32 ? 4 : 2;
    const int64_t cg = C / G;
    GroupNormPlan g = {};
    g.V = 16 / es;
    while (cg % g.V) g.V /= 2;
    const int64_t cgv = cg / g.V;
    const int most = backward ? 8 : 16;      // vectors of a thread, of each tensor
    g.parts = (int32_t)ceil_div(cgv, kMaxThreads);
    g.range = 1;
    g.chunks = 1;
    g.chunk_rows = (int32_t)P;
    if (g.parts == 1) {
        // Rows of a line (128 bytes) at least, and a wave's worth of vectors.
        for (int64_t bytes : {int64_t(128), int64_t(64), cg * es}) {
            int64_t kg = std::min(G, std::max(ceil_div(bytes, cg * es), ceil_div(64, cgv * std::max<int64_t>(P, 1))));
            kg = std::max<int64_t>(1, std::min(kg, kMaxThreads / cgv));
            const int64_t cols = kg * cgv;
            for (int want : {backward ? 4 : 8, most})
                for (int t = 64; t <= kMaxThreads; t *= 2) {
                    if (t < cols || (want == most && t < kMaxThreads)) continue;
                    const int64_t R = t / cols, K = ceil_div(std::max<int64_t>(P, 1), R);
                    if (K > want) continue;
                    g.whole = 1; g.kg = (int32_t)kg; g.cols = (int32_t)cols; g.threads = t; g.K = (int32_t)K;
                    // Samples of a workgroup: twice the workgroups that the card holds at once (forward, single
                    // positions: 5092 x 6656 in fp32 154 us in one workgroup for each sample, 104 and 89 us in as
                    // many as it holds and in twice as many), and for gradients no more than it holds, and up to
                    // kPartRows rows of partial sums (20000 x 512 in fp16: 95 us with 512, 57 with 1024; 3063 x 512
                    // in bf16: 23, 22 and with 2048 23 us).
                    const int64_t blocks = N * ceil_div(G, kg), held = 256 * (2048 / t);
                    if (backward) g.range = std::max(ceil_div(blocks, held), ceil_div(N, kPartRows));
                    else if (K == 1) g.range = ceil_div(blocks, 2 * held);
                    g.range = std::max<int64_t>(1, g.range);
                    return g;
                }
        }
    }
    // Chunks of positions: rows as wide as 64 lanes take, 512 workgroups (gradients of 8 x 20480 x 256 in bf16:
    // sums 48.7 and dx 44.0 us, with 1024 52.8 and 45.4).
    g.kg = g.parts > 1 ? 1 : (int32_t)std::max<int64_t>(1, std::min(G, 64 / cgv));
    g.cols = (int32_t)(g.parts > 1 ? ceil_div(cgv, g.parts) : g.kg * cgv);
    g.threads = (int32_t)std::max<int64_t>(512, 64 * ceil_div(g.cols, 64));
    if (g.threads > 512) g.threads = kMaxThreads;
    g.K = backward ? kTileBwd : kTile;
    const int64_t tile = g.threads / g.cols * g.K, tiles = ceil_div(std::max<int64_t>(P, 1), tile);
    const int64_t bundles = ceil_div(G, g.kg) * g.parts, want = std::max<int64_t>(1, 512 / std::max<int64_t>(1, N * bundles));
    g.chunk_rows = (int32_t)(tile * ceil_div(tiles, want));
    g.chunks = (int32_t)ceil_div(std::max<int64_t>(P, 1), g.chunk_rows);
    // Partial sums of dw and db: up to 2 kPartRows rows a sample each, beyond that ranges of samples of 64 positions
    // in all, whose row of sums is a sixteenth of their x in 16 bits.  16384 rows of 16384 channels in one group in
    // fp32: 4080 us and 2.1 GB of sums with a row a sample, 2050 us and 0.13 GB; 2050 x 3000 x 64 in bf16 786 us,
    // in ranges of two samples 825.
    if (backward && g.chunks == 1) g.range = std::max<int64_t>(1, std::min(N / kPartRows, ceil_div(64, std::max<int64_t>(P, 1))));
    return g;
}

size_t gn_workspace(const GroupNormPlan &g, int64_t N, int64_t C, int64_t G, bool backward)
{
    return gn_chunk_bytes(g, N, G) + (backward ? sizeof(float) * 2 * (size_t)(ceil_div(N, g.range) * g.chunks * C) : 0);
}

bool gn_fits(const GroupNormArgs &a, const GroupNormPlan &g)
{
    // A thread's first position lies within 2^31 bytes of its workgroup's.
    const int64_t es = a.dtype == DT_F32 ? 4 : 2, top = ((int64_t(1) << 31) - 1) / es / 2, R = g.threads / g.cols;
    for (int64_t st : {a.P > 1 ? a.xst : 0, a.P > 1 ? a.dst : 0, a.C})
        if (st > top / R) return false;
    const int64_t samples = g.whole ? ceil_div(a.N, g.range) : a.N;      // (of the launch that has most workgroups)
    return grid_fits(8 * ceil_div(samples * g.chunks * ceil_div(a.G, g.kg) * g.parts, 8), g.threads);
}

hipError_t launch_group_norm(const GroupNormArgs &a, const GroupNormPlan &g, const char **kname)
{
    const Norm p = make_norm(a, g);
    if (g.whole) {
        *kname = "gn_forward";
        return launch_with(p, a, g, [&](auto t, auto v, dim3 grid) {
            with_rows(g.K, [&](auto k) {
                gn_forward<decltype(t), v.value, k.value><<<grid, g.threads, lds_bytes(g.threads, 0), a.stream>>>(p);
            });
        });
    }
    *kname = "gn_chunk_apply";
    const hipError_t err = launch_with(p, a, g, [&](auto t, auto v, dim3 grid) {
        gn_chunk_stats<decltype(t), v.value><<<grid, g.threads, lds_bytes(g.threads, 0), a.stream>>>(p);
    });
    return err != hipSuccess ? err : launch_with(p, a, g, [&](auto t, auto v, dim3 grid) {
        gn_chunk_apply<decltype(t), v.value><<<grid, g.threads, lds_bytes(g.threads, 0), a.stream>>>(p);
    });
}

hipError_t launch_group_norm_bwd(const GroupNormArgs &a, const GroupNormPlan &g, const char **kname)
{
    const Norm p = make_norm(a, g);
    *kname = g.whole ? "gn_backward" : "gn_chunk_slopes";
    if (p.blocks > 0) {
        hipError_t err;
        if (g.whole) {
            err = launch_with(p, a, g, [&](auto t, auto v, dim3 grid) {
                with_rows(g.K, [&](auto k) {
                    const size_t bytes = lds_bytes(g.threads, v.value * (k.value > 1 ? 2 : 1));
                    if constexpr (k.value <= 8) gn_backward<decltype(t), v.value, k.value><<<grid, g.threads, bytes, a.stream>>>(p);
                });
            });
        } else {
            err = launch_with(p, a, g, [&](auto t, auto v, dim3 grid) {
                const size_t bytes = lds_bytes(g.threads, v.value);
                if (g.range > 1) gn_chunk_sums<decltype(t), v.value, true><<<grid, g.threads, bytes, a.stream>>>(p);
                else gn_chunk_sums<decltype(t), v.value, false><<<grid, g.threads, bytes, a.stream>>>(p);
            });
            Norm each = p;      // a workgroup for each sample's chunk
            each.range = 1;
            each.blocks = a.N * g.chunks * p.bundles;
            if (err == hipSuccess)
                err = launch_with(each, a, g, [&](auto t, auto v, dim3 grid) {
                    gn_chunk_slopes<decltype(t), v.value><<<grid, g.threads, lds_bytes(g.threads, 0), a.stream>>>(each);
                });
        }
        if (err != hipSuccess) return err;
    }
    const unsigned grid = (unsigned)ceil_div(2 * a.C, 16);
    return with_vec(a.dtype, 1, [&](auto t, auto) {
        typedef decltype(t) E;
        gn_param_sum<E><<<grid, 1024, 0, a.stream>>>(p.part, (E *)a.dw, (E *)a.db, p.rows, a.C);
        return hipGetLastError();
    });
}

}  // namespace gconv
