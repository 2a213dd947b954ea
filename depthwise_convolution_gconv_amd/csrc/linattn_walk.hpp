// linattn_walk.hpp -- the chunked pass of linear attention on the bf16 matrix cores, for
// every dtype; one translation unit for each dtype instantiates it.
//
// The pass (linattn.hpp) walks a sequence in chunks of L tokens.  With R the state before
// the chunk and i, j token indices inside it,
//
//     out_i = inter_scale lam^(i+e0) a_i R  +  p_scale sum_{j <= i} lam^(i-j) (a_i . b_j) c_j
//     R'    = lam^m R + upd_scale sum_j lam^(m-j-e0) b_j c_j^T          (m tokens in the chunk)
//
// so a token costs 2 (Da + Dc) L + 4 Da Dc operations instead of the T Da of the quadratic
// form, all of them matrix products.  A workgroup owns one (batch, head, segment) and 32
// columns of c for each wave.  A sequence that gives too few workgroups is cut into
// segments: their local states are summed first (FULL = false), a scan turns them into the
// states before each segment, and then every segment is walked on its own.  That reads b
// and c a second time.
//
// Operands.  A 16-bit matrix product takes 8 or 11 bits of each factor, so a value is
// carried as a sum of bf16 parts, which keep fp32's range: one part for bf16 inputs, two
// for fp16 (exact), three for fp32 (exact).  Products of two parts below the last bit that
// the result can show are left out.  The weighted rows lam^(m-j-e0) c_j of the state's
// update always have three parts (24 bits), so the state is the fp32 sum it would be on a
// vector unit.  Scores and the state that meets a_i have two parts in 16 bits and three in
// fp32: they lose 2^-16 (2^-24) of a term, below what an output of the inputs' type shows, and
// both stay fp32 in their accumulators.
//
// Nothing but the inputs goes through LDS.  Products run transposed (columns of the
// accumulators are tokens i, rows are j or columns of c): scores and the state leave the
// matrix cores with four consecutive rows in a lane (rows 4h .. 4h+3 and 8+4h .. 8+4h+3 of
// each 16 for the lane's half h), and as the order of a reduction is free, the other
// operand is read in that same order: for the scores by reading c's rows so, for the state
// by taking b's columns of each 16 in the order 0-3, 8-11, 4-7, 12-15, so that a lane's
// eight rows stand for eight neighbours of a.  A wave keeps the state of its 32 columns in
// accumulators for the whole walk.
//
// What bounds it (bf16, 128 x 128 heads): HBM, and beside it the products.  65536 tokens x 16
// heads take 442 us: 1.07 GB for the outputs' walk, 0.54 GB for the local states', and the scan.
// One part for the scores and the state that meets a_i took 390 us where two took 432, with
// 2.4e-3 of error beside the 1.7e-3 of the outputs' own rounding, and 249 instead of 284 us for
// the gradients of 4 x 4096 tokens x 16 heads; the scale in 64 bits and the search for values that
// are not finite took the rest.  32 tokens rather than 64: half the registers for what is on
// its way, so three workgroups on a compute unit instead of two, and no off-diagonal tile of
// scores (504 -> 486 us, and 447 with the segments that three workgroups call for, all with one
// part).  Two parts instead of three in the update took 403 instead of 421 us and left the state
// with 2.5e-6 of error instead of 1e-7.  fp16 and fp32 pay for their parts (3 and 6 products for
// one) and are bound by those: 40 us for 5 x 1021 tokens x 12 heads of 96 x 80 in fp16, 67 us for
// the three walks of 8 x 1024 tokens x 8 heads of 64 in fp32.
#pragma once

#include "linattn.hpp"
#include "vecio.hpp"

namespace gconv {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <typename T> constexpr int kParts = sizeof(T) == 4 ? 3 : 2;
template <> constexpr int kParts<__bf16> = 1;
constexpr int kUpdParts = 3;
// Of scores, and of the state that meets a_i.
template <typename T> constexpr int kMidParts = sizeof(T) == 4 ? 3 : 2;
constexpr int kLen = 32;     // tokens in a chunk

// A tile of D columns in LDS, laid out so that the 16-byte reads of 16 rows and the transposing
// reads of 4 rows x 64 bytes both cover all 64 banks: groups of four rows four banks apart, and
// within each four the 64-byte blocks that one read takes on different banks, by padding, or for
// 64 columns (where that is half the tile again) by swapping the two blocks of every other pair.
template <int D> struct Tile {
    static constexpr int row = D == 64 ? 64 : D == 128 ? 160 : 288;
    static constexpr int group = D == 64 ? 264 : D == 128 ? 648 : 1160;
    static constexpr int size = kLen / 4 * group;
    static __device__ __forceinline__ int row_at(int j) { return (j >> 2) * group + (j & 3) * row; }
    // where block q (32 columns) of row j is in it
    static __device__ __forceinline__ int block(int q, int j) { return (D == 64 ? q ^ (j >> 1 & 1) : q) * 32; }
    static __device__ __forceinline__ int at(int j, int d) { return row_at(j) + block(d / 32, j) + d % 32; }
};

template <int NP> struct Part8 { bf16x8 p[NP]; };

// x as a sum of NP bf16 parts, each the rounding of what the earlier ones leave.
template <int NP> __device__ __forceinline__ Part8<NP> split8(const float (&x)[8])
{
    Part8<NP> r;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        f32x2 left = {x[e], x[e + 1]};
#pragma unroll
        for (int q = 0; q < NP; ++q) {
            const bf16x2 two = __builtin_convertvector(left, bf16x2);   // one instruction
            r.p[q][e] = two[0];
            r.p[q][e + 1] = two[1];
            if (q + 1 < NP) {
                const uint32_t bits = __builtin_bit_cast(uint32_t, two);
                left[0] -= __builtin_bit_cast(float, bits << 16);
                left[1] -= __builtin_bit_cast(float, bits & 0xffff0000u);
            }
        }
    }
    return r;
}

// acc += a b over the pairs of parts p + q <= TOP, the smallest first.
template <int TOP, int NA, int NB>
__device__ __forceinline__ f32x16 mma(const Part8<NA> &a, const Part8<NB> &b, f32x16 acc)
{
#pragma unroll
    for (int s = TOP; s >= 0; --s)
#pragma unroll
        for (int q = 0; q < NA; ++q)
            if (s - q >= 0 && s - q < NB)
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.p[q], b.p[s - q], acc, 0, 0, 0);
    return acc;
}

// 8 neighbours of a row (16-byte aligned).
template <int D, int NP> __device__ __forceinline__ Part8<NP> read_row(const __bf16 *t, int at)
{
    Part8<NP> r;
#pragma unroll
    for (int q = 0; q < NP; ++q) r.p[q] = *reinterpret_cast<const bf16x8 *>(t + q * Tile<D>::size + at);
    return r;
}

// Rows 4h .. 4h+3 and 8+4h .. of a column each lane: two transposing reads.  Of 16 lanes,
// lane t names row t / 4 and the t % 4-th four columns, and gets its column of all four rows.
template <int D, int NP> __device__ __forceinline__ Part8<NP> read_col(const __bf16 *t, int at)
{
    typedef __attribute__((address_space(3))) s16x4 lds4;
    Part8<NP> r;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const __bf16 *x = t + q * Tile<D>::size + at;
        const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)x));
        const bf16x4 hi =
            __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(x + 2 * Tile<D>::group)));
        r.p[q] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
}

// 8 elements on their way from memory to LDS, in loads of 16 bytes.
template <typename T> struct Raw8 {
    static constexpr int N = 16 / sizeof(T);     // elements of a load
    RunVec<T, N> w[8 / N];
};

// Where a row ends inside a load, the load ends with the row instead (rows of N columns or
// more): offset of its address from the block's first column, and later the shift that puts
// its elements in their places and zeros after them.  Both take the columns left from the
// block's first one on; a load past the row's end reads the one before it.
template <typename T> __device__ __forceinline__ int load_at(int left, int i)
{
    constexpr int N = Raw8<T>::N;
    if (left <= N * i) i = 0;
    return N * i + min(left - N * i - N, 0);
}
template <typename T> __device__ __forceinline__ void shift_tail(Raw8<T> &r, int left)
{
    constexpr int N = Raw8<T>::N;
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) {
        const int sh = min(max(N * i + N - left, 0), N) * (128 / N);
        typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
        u64x2 v = __builtin_bit_cast(u64x2, r.w[i]);
        const uint64_t lo = sh & 63 ? v[0] >> (sh & 63) | v[1] << (64 - (sh & 63)) : v[0], hi = v[1] >> (sh & 63);
        v[0] = sh < 64 ? lo : sh < 128 ? hi : 0;
        v[1] = sh < 64 ? hi : 0;
        r.w[i] = __builtin_bit_cast(RunVec<T, N>, v);
    }
}

// Their parts, and those to their tiles.
template <typename T> __device__ __forceinline__ Part8<kParts<T>> parts8(const Raw8<T> &v)
{
    constexpr int NP = kParts<T>;
    Part8<NP> r;
    if constexpr (NP == 1) {
        r.p[0] = __builtin_bit_cast(bf16x8, v);
    } else {
        const Run<T, 8> x = __builtin_bit_cast(Run<T, 8>, v);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = to_f32(x.v[e]);
        r = split8<NP>(f);
    }
    return r;
}
template <int D, int NP> __device__ __forceinline__ void put8(__bf16 *t, int at, const Part8<NP> &r)
{
#pragma unroll
    for (int q = 0; q < NP; ++q) *reinterpret_cast<bf16x8 *>(t + q * Tile<D>::size + at) = r.p[q];
}

// x plus zero times every value of a run: NaN if one is not finite.
__device__ __forceinline__ float taint(bf16x8 v, float x)
{
    const bf16x2 zero = {(__bf16)0.0f, (__bf16)0.0f};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const bf16x2 two = {v[i], v[i + 1]};
        x = __builtin_amdgcn_fdot2_f32_bf16(two, zero, x, false);
    }
    return x;
}
constexpr int kNoToken = 0x7fffffff;

// A thread's share of a tile of kLen tokens by D columns: NR runs of 8 of one column block,
// every STEP tokens.  Blocks past the last column are neither read nor staged.
template <typename T, int D, int NTH> struct Share {
    static constexpr int NR = kLen * D / 8 / NTH, STEP = NTH / (D / 8), N = Raw8<T>::N;
    Raw8<T> r[NR];
    const T *p;              // its first run of the next chunk
    int64_t step, chunk;     // elements from token to token of the walk, from chunk to chunk
    int j, left;             // first token; columns from its block on
    __device__ __forceinline__ void init(const T *base, int64_t stride, int cols, int u0, int du, int n, int reverse)
    {
        const int d = threadIdx.x % (D / 8) * 8;
        j = threadIdx.x / (D / 8);
        left = cols - d;
        step = reverse ? -stride : stride;
        chunk = du * step;
        p = base + d + (int64_t)(reverse ? n - 1 - u0 - j : u0 + j) * stride;
    }
    // A whole chunk of a row of N columns or more.
    __device__ __forceinline__ void fetch()
    {
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int e = 0; e < 8 / N; ++e)
                    r[i].w[e] = *reinterpret_cast<const RunVec<T, N> *>(p + i * STEP * step + load_at<T>(left, e));
        }
        p += chunk;
    }
    // The chunk's first `live` tokens; narrow: a row of fewer columns, element by element.
    __device__ __forceinline__ void fetch(int live, bool narrow)
    {
#pragma unroll
        for (int i = 0; i < NR; ++i) r[i] = Raw8<T>{};
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if (left <= 0 || j + i * STEP >= live) continue;
#pragma unroll
            for (int e = 0; e < 8 / N; ++e) {
                if (!narrow) r[i].w[e] = *reinterpret_cast<const RunVec<T, N> *>(p + i * STEP * step + load_at<T>(left, e));
                else if (e == 0) r[i].w[e] = load_words<T, N>(p + i * STEP * step, left);
            }
        }
        p += chunk;
    }
    // shift: row ends inside a load have to be moved (not for narrow rows).  bad: for c, whose
    // values that are not finite a product would take to all tokens (0 x NaN where a score is
    // masked).  They become zeros, and each column keeps the first of its tokens, counted from the
    // chunk's first u0 on, that had one: bad[0] tells whether any has, bad[1 + column] is that
    // token.  Outputs from there on become NaN after the walk (in it, a test a chunk took 14 of 442
    // us over 65536 tokens x 16 heads in bf16; finding the values takes 5).
    __device__ __forceinline__ void stage(__bf16 *t, bool shift, int *bad = nullptr, int u0 = 0)
    {
        if (left <= 0) return;
        const int d = threadIdx.x % (D / 8) * 8;
        if (shift) {
#pragma unroll
            for (int i = 0; i < NR; ++i) shift_tail<T>(r[i], left);
        }
        float tainted = 0.0f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const Part8<kParts<T>> x = parts8<T>(r[i]);
            put8<D>(t, Tile<D>::at(j + i * STEP, d), x);
            if (bad) tainted = taint(x.p[0], tainted);
        }
        if (bad && tainted != tainted) drop_bad(t, bad, u0);
    }
    __device__ __forceinline__ void drop_bad(__bf16 *t, int *bad, int u0)
    {
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));     // addresses are made here, not kept for the whole walk
        const int d = tid % (D / 8) * 8;
        bad[0] = 1;
#pragma unroll 1
        for (int row = tid / (D / 8); row < kLen; row += STEP)
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
                __bf16 *p = t + Tile<D>::at(row, d) + e;     // in the same block of columns
                const __bf16 x = *p;
                if ((__builtin_bit_cast(uint16_t, x) & 0x7fff) < 0x7f80) continue;
                atomicMin(&bad[1 + d + e], u0 + row);
                for (int q = 0; q < kParts<T>; ++q) p[q * Tile<D>::size] = (__bf16)0.0f;
            }
    }
};

// A lane's 16 values of a token: four columns of every eight.  Of two 16-bit runs the lane
// gives one to the other half's lane and takes the rest of the other, so stores are 16 bytes.
template <typename TO> __device__ __forceinline__ void store_tile(TO *o, int half, int left, const f32x16 &acc)
{
    if constexpr (sizeof(TO) == 4) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float f[4] = {acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
            const int at = 8 * g + 4 * half;
            if (left > at) store_run<TO, 4>(o + at, left - at, f);
        }
    } else {
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
            union { Run<TO, 8> v; uint32_t w[4]; } x;
#pragma unroll
            for (int e = 0; e < 8; ++e) x.v.v[e] = from_f32<TO>(acc[4 * g + e]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto y = __builtin_amdgcn_permlane32_swap(x.w[i], x.w[2 + i], false, false);
                x.w[i] = y[0];
                x.w[2 + i] = y[1];
            }
            const int at = 8 * g + 8 * half;
            if (left > at) store_raw<TO, 8>(o + at, left - at, x.v);
        }
    }
}

// A value that all lanes of a wave have, in scalar registers.
__device__ __forceinline__ double wave_value(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

template <typename T, int DK, int NW, bool FULL> struct WalkLds {
    static constexpr int NP = kParts<T>;
    static constexpr int tiles = 2 * NP * ((FULL ? 2 : 1) * Tile<DK>::size + Tile<32 * NW>::size) + (FULL ? 0 : 16);
    __bf16 a[FULL ? NP * Tile<DK>::size : 8];
    __bf16 b[NP * Tile<DK>::size];
    __bf16 c[NP * Tile<32 * NW>::size];
    float diag[FULL ? 16 * 64 : 4];     // weights of a tile of scores, [r / 4][lane][r % 4]
    uint32_t mask[FULL ? 8 * 64 : 4];   // halves of ones for the pairs of them with j <= i, [r / 8][lane][r / 2 % 4]
    float upd[kLen];                    // upd_scale lam^(m-j-e0)
    float pw[kLen + 1];                 // lam^0 .. lam^kLen
    double fade;                        // lam^kLen
    int bad[FULL ? 1 + 32 * NW : 1];    // see drop_bad
};

// Waves of a SIMD that registers are kept for: two or three workgroups share a compute unit.
// The output walks over 129 to 256 columns of a and b keep some addresses in scratch memory for
// it: 23 registers in bf16 with four waves, 6 in fp16 with eight, 3 in fp32 (and 3 those of local
// states; bf16 over 128 columns with four waves: 1).  The first with one wave a SIMD, without
// any: 140 -> 159 us for 4 x 4096 tokens x 8 heads of 256 x 128, 83 -> 114 for 2 x 3000 x 16 of 192
// x 64, but 109 -> 81 for 16 x 512 x 16 of 256 x 128, and gradients 368 -> 363, 221 -> 220, 223 ->
// 218.
template <typename T, int DK, int NW>
constexpr int kWavesPerSimd = DK == 256 ? (kParts<T> == 3 ? 1 : 2) : kParts<T> == 1 && DK / NW <= 32 ? 3 : 2;

// Kernels that have registers to spare before their loop (the others would spill into it).
template <typename T, int DK> constexpr bool kRoomy = DK == 64 ? kParts<T> > 1 : DK == 128 && kParts<T> == 3;

template <typename T, int DK, int NW, bool FULL>
__global__ void __launch_bounds__(64 * NW, (kWavesPerSimd<T, DK, NW>))
lin_walk(const LinWalks all)
{
    constexpr int NP = kParts<T>, NM = kMidParts<T>, L = kLen, NT = 32 * NW, NTH = 64 * NW;
    typedef WalkLds<T, DK, NW, FULL> Lds;
    constexpr int NX = DK / 32, NS = DK / 16, NG = L / 16;          // state tiles, steps along columns, along tokens
    __shared__ __attribute__((aligned(16))) Lds sm;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, l32 = lane & 31, half = lane >> 5;

    // Workgroups go round the 8 XCDs, a contiguous run of ids on each.  Neighbours read the same
    // rows: column tiles, a launch's walks, the value heads of a key head.
    const int64_t per = (all.blocks + 7) / 8;
    int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (id >= all.blocks) return;
    auto next = [&](int count) {
        const int x = (int)(id % count);
        id /= count;
        return x;
    };
    const int dv = next(all.ndv);
    const LinWalk &p = all.w[next(all.count)];
    const int hr = next(p.rep), seg = next(p.nseg), h = next(p.H / p.rep) * p.rep + hr, bi = (int)id;
    const int64_t bh = (int64_t)bi * p.H + h;
    const int n = lin_len(p, bi), n0 = dv * NT;
    const int useg = seg * p.seg_len;
    // Tokens [useg, utop) of this workgroup; useg + seg_len may pass 2^31.
    const int top = FULL ? p.T : n, utop = top - useg > p.seg_len ? useg + p.seg_len : top;
    const int ulive = min(n, utop);
    // Outputs go from the first chunk on.  Local states go from the last one back: each chunk
    // then adds its tokens with their weights at the segment's end, the state itself is never
    // scaled, and what was read last, the segments' first halves, is what the outputs' walk
    // finds in the last-level cache.
    const int nchunk = (utop - useg + L - 1) / L, ufirst = FULL ? useg : useg + (nchunk - 1) * L, du = FULL ? L : -L;
    const bool mine = n0 + wave * 32 < p.Dc;                  // this wave has columns
    // Row ends inside a load, and rows shorter than one.
    constexpr int N = Raw8<T>::N;
    const bool narrow_ab = p.Da < N, narrow_c = p.Dc < N, narrow = narrow_ab || narrow_c;
    const bool shift_ab = p.Da % 8 != 0 && !narrow_ab, shift_c = p.Dc % 8 != 0 && !narrow_c;

    Share<T, DK, NTH> sa, sb;
    Share<T, NT, NTH> sc;
    if constexpr (FULL)
        sa.init((const T *)p.a + bi * p.asb + (h / p.ra) * p.ash, p.ast, p.Da, ufirst, du, n, p.reverse);
    sb.init((const T *)p.b + bi * p.bsb + (h / p.rb) * p.bsh, p.bst, p.Da, ufirst, du, n, p.reverse);
    sc.init((const T *)p.c + bi * p.csb + (h / p.rc) * p.csh + n0, p.cst, p.Dc - n0, ufirst, du, n, p.reverse);
    auto fetch = [&](int u0) {
        const int live = ulive - u0;
        if (live >= L && !narrow) {
            if constexpr (FULL) sa.fetch();
            sb.fetch();
            sc.fetch();
        } else {
            if constexpr (FULL) sa.fetch(live, narrow_ab);
            sb.fetch(live, narrow_ab);
            sc.fetch(live, narrow_c);
        }
    };
    {   // columns past the last stay zero
        u32x4 *z = reinterpret_cast<u32x4 *>(&sm);
        for (int e = tid; e < Lds::tiles / 16; e += NTH) z[e] = u32x4{0, 0, 0, 0};
    }
    if constexpr (FULL) {
        if (tid < NT) sm.bad[1 + tid] = kNoToken;
        if (tid == 0) sm.bad[0] = 0;
    }
    if (tid <= L) {
        const double power = lin_pow64(p.log_decay[h], tid);
        sm.pw[tid] = (float)power;
        if (tid == L) sm.fade = power;
    }

    if (kRoomy<T, DK> && nchunk > 0) fetch(ufirst);

    // The state: column scol, rows 4 half + 32 x + 8 (r / 4) + r % 4 of the tiles, which stand
    // for the columns of b that d_of gives.
    const int scol = n0 + wave * 32 + l32;
    auto d_of = [](int x, int r) { return 32 * x + 16 * (r / 8) + 4 * (r / 4 % 2) + r % 4; };     // + 8 half
    f32x16 st[NX];
    // st = keep st + gain *sp, whose rows are sr apart.  The loads of two tiles are in flight
    // together where registers allow.
    constexpr int TB = kRoomy<T, DK> ? 2 : 1;
    auto read_state = [&](const float *sp, int sr, int sc, float keep, float gain) {
#pragma unroll
        for (int x0 = 0; x0 < NX; x0 += TB) {
            int d0 = 8 * half;
            asm volatile("" : "+v"(d0));     // the offsets are made here, not kept from call to call
            float v[TB][16];
#pragma unroll
            for (int x = 0; x < TB; ++x)
#pragma unroll
                for (int r = 0; r < 16; ++r)     // rows past the last read that one
                    v[x][r] = sp[min(d0 + d_of(x0 + x, r), p.Da - 1) * sr + scol * sc];
#pragma unroll
            for (int x = 0; x < TB; ++x)
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    asm volatile("" : "+v"(v[x][r]));     // a load inside the condition would wait for each
                    st[x0 + x][r] = d0 + d_of(x0 + x, r) < p.Da ? fmaf(keep, st[x0 + x][r], gain * v[x][r]) : 0.0f;
                }
        }
    };
#pragma unroll
    for (int x = 0; x < NX; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) st[x][r] = 0.0f;
    const bool fold = p.nseg <= kFoldSegs, ends = FULL && fold && p.sf && seg + 1 == p.nseg;
    const float *s0 = p.s0 ? p.s0 + bi * p.s0b + h * p.s0h : nullptr;
    auto tokens_of = [&](int g) { return max(0, min(n - g * p.seg_len, p.seg_len)); };
    if (FULL && scol < p.Dc && (seg > 0 || s0)) {
        // The state before the first segment; or the local ones up to this, of which the first
        // holds that state's rest; or what the scan made of them.
        const bool first = seg == 0;
#pragma unroll 1
        for (int g = first || fold ? 0 : seg; g < (first || !fold ? seg + 1 : seg); ++g)
            read_state(first ? s0 : p.ws + (bh * p.nseg + g) * (int64_t)p.Da * p.Dc, (int)(first ? p.s0r : p.Dc),
                       (int)(first ? p.s0c : 1), fold && g > 0 ? lin_pow(p.log_decay[h], tokens_of(g)) : 0.0f, 1.0f);
    }

    if (!kRoomy<T, DK> && nchunk > 0) fetch(ufirst);
    __syncthreads();     // the powers
    if constexpr (FULL) {
        for (int e = tid; e < 16 * 64; e += NTH) {
            const int i = e / 4 % 32, j = 8 * (e / 256) + 4 * (e / 128 % 2) + e % 4;
            sm.diag[e] = j <= i ? p.p_scale * sm.pw[i - j] : 0.0f;
        }
        for (int e = tid; e < 8 * 64; e += NTH) {
            const int i = e / 4 % 32, j = 16 * (e / 256) + 8 * (e / 2 % 2) + 4 * (e / 128 % 2) + e % 2 * 2;
            sm.mask[e] = (j <= i ? 0xffffu : 0u) | (j + 1 <= i ? 0xffff0000u : 0u);
        }
    }
    const int row0 = Tile<DK>::row_at(l32) + 8 * half;
    auto row_at = [&](int s) { return row0 + Tile<DK>::block(s / 2, l32) + s % 2 * 16; };      // columns 16 s + 8 half ..
    // Columns over rows: the lane's row of its group, and its four columns (b's in the order
    // 0-3, 8-11, 4-7, 12-15).
    const int col_row = 4 * half + ((lane & 15) >> 2);
    const int bcol0 = Tile<DK>::row_at(col_row) + (lane & 16) + (lane & 1) * 8 + (lane & 2) * 2;
    auto bcol_at = [&](int g, int x) { return bcol0 + Tile<DK>::block(x, col_row) + 4 * g * Tile<DK>::group; };
    const int ccol0 = Tile<NT>::row_at(col_row) + Tile<NT>::block(wave, col_row) + (lane & 16) + (lane & 3) * 4;
    auto ccol_at = [&](int g) { return ccol0 + 4 * g * Tile<NT>::group; };

    // Outputs: the state is scale times its registers, so that it need not be scaled for every
    // chunk's decay.  Local states: scale is the weight of the next chunk's last token.  In 64
    // bits (one for the wave): every chunk multiplies it by the same power, whose rounding to fp32
    // would add up to 2^-25 a chunk (918 u after 65536 tokens with a log decay of -4e-8).
    double scale64 = 1.0;
    for (int k = 0; k < nchunk; ++k) {
        const int u0 = ufirst + k * du;
        const int m = max(0, min(ulive - u0, L));
        const double faded64 = wave_value(scale64 * (m == L ? sm.fade : (double)sm.pw[m]));
        const float scale = (float)scale64, faded = (float)faded64;
        const bool settle = FULL && !(faded >= 0x1p-10f && faded <= 0x1p10f);   // registers take the scale
        // The previous chunk's readers are done (barrier at the loop's end).
        if constexpr (FULL) sa.stage(sm.a, shift_ab);
        sb.stage(sm.b, shift_ab);
        sc.stage(sm.c, shift_c, FULL ? sm.bad : nullptr, u0);
        if (tid < L)
            sm.upd[tid] = p.upd_scale * sm.pw[max(m - tid - p.e0, 0)] * (!FULL ? scale : settle ? 1.0f : 1.0f / faded);
        __syncthreads();
        if (k + 1 < nchunk) fetch(u0 + du);

        if (FULL && mine) {
            f32x16 acc;
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
            if (m > 0) {
                // a_i R and the scores a_i . b_j share the reads of a.
                f32x16 sco;
#pragma unroll
                for (int r = 0; r < 16; ++r) sco[r] = 0.0f;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const Part8<NP> aq = read_row<DK, NP>(sm.a, row_at(s));
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = st[s / 2][s % 2 * 8 + e];
                    sco = mma<NP - 1>(read_row<DK, NP>(sm.b, row_at(s)), aq, sco);
                    acc = mma<NM - 1>(split8<NM>(f), aq, acc);
                }
                const float fi = scale * p.inter_scale * sm.pw[min(l32 + p.e0, L)];
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[r] *= fi;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 w = *reinterpret_cast<const float4 *>(&sm.diag[256 * (2 * g + e / 4) + 4 * lane]);
                        f[e] = sco[8 * g + e] * w.x;
                        f[e + 1] = sco[8 * g + e + 1] * w.y;
                        f[e + 2] = sco[8 * g + e + 2] * w.z;
                        f[e + 3] = sco[8 * g + e + 3] * w.w;
                    }
                    // Scores of later tokens are masked, not only multiplied by zero: they may be infinite.
                    Part8<NM> pr = split8<NM>(f);
                    const u32x4 mask = *reinterpret_cast<const u32x4 *>(&sm.mask[256 * g + 4 * lane]);
#pragma unroll
                    for (int q = 0; q < NM; ++q)
                        pr.p[q] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(u32x4, pr.p[q]) & mask);
                    acc = mma<NM - 1>(read_col<NT, NP>(sm.c, ccol_at(g)), pr, acc);
                }
            }
            if (m < L) {
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[r] = l32 < m ? acc[r] : 0.0f;
            }
            // Both lanes of a token store or neither: they hold each other's values.
            const int u = u0 + l32;
            if (u < utop) {
                const int64_t at = bi * p.osb + (int64_t)lin_token(p, u, n) * p.ost + h * p.osh + n0 + wave * 32;
                const int left = p.Dc - n0 - wave * 32;
                if (sizeof(T) == 4 || p.out_f32) store_tile<float>((float *)p.out + at, half, left, acc);
                else store_tile<T>((T *)p.out + at, half, left, acc);
            }
        }

        if (mine && m > 0 && (!FULL || k + 1 < nchunk || ends)) {
            if (settle) {
#pragma unroll
                for (int x = 0; x < NX; ++x)
#pragma unroll
                    for (int r = 0; r < 16; ++r) st[x][r] *= faded;
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const Part8<NP> cT = read_col<NT, NP>(sm.c, ccol_at(g));
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float v = (float)cT.p[NP - 1][e];
#pragma unroll
                    for (int q = NP - 2; q >= 0; --q) v += (float)cT.p[q][e];
                    f[e] = v * sm.upd[16 * g + 4 * half + 8 * (e / 4) + e % 4];
                }
                const Part8<kUpdParts> wc = split8<kUpdParts>(f);
#pragma unroll
                for (int x = 0; x < NX; ++x)
                    st[x] = mma<2>(read_col<DK, NP>(sm.b, bcol_at(g, x)), wc, st[x]);
            }
        }
        scale64 = settle ? 1.0 : faded64;
        __syncthreads();
    }
    const float scale = (float)scale64;
    if (FULL && sm.bad[0]) {     // behind the loop's last barrier, which orders these stores after its own
#pragma unroll 1
        for (int col = 0; col < min(NT, p.Dc - n0); ++col)
#pragma unroll 1
            for (int64_t u = (int64_t)sm.bad[1 + col] + tid; u < ulive; u += NTH) {
                const int64_t at = bi * p.osb + (int64_t)lin_token(p, (int)u, n) * p.ost + h * p.osh + n0 + col;
                if (sizeof(T) == 4 || p.out_f32) ((float *)p.out)[at] = __builtin_nanf("");
                else ((T *)p.out)[at] = from_f32<T>(__builtin_nanf(""));
            }
    }

    if (!FULL && seg == 0 && s0 && scol < p.Dc)
        read_state(s0, (int)p.s0r, (int)p.s0c, 1.0f, lin_pow(p.log_decay[h], tokens_of(0)));
    float *dp = nullptr, *tp = nullptr;
    int dr = p.Dc, dc = 1;       // a state's offsets stay below 2^16
    if (!FULL) {
        dp = p.ws + (bh * p.nseg + seg) * (int64_t)p.Da * p.Dc;
        if (p.wst) tp = p.wst + (bh * p.nseg + seg) * (int64_t)p.Da * p.Dc;
    } else if (ends) {
        dp = p.sf + bi * p.sfb + h * p.sfh;
        dr = (int)p.sfr; dc = (int)p.sfc;
    }
    if (dp && scol < p.Dc) {
        if (FULL && sm.bad[0] && sm.bad[1 + wave * 32 + l32] != kNoToken) {
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
                for (int r = 0; r < 16; ++r) st[x][r] = __builtin_nanf("");
        }
        int d0 = 8 * half;
        asm volatile("" : "+v"(d0));
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int d = d0 + d_of(x, r);
                if (d < p.Da) dp[d * dr + scol * dc] = FULL ? st[x][r] * scale : st[x][r];
            }
        if (!FULL && tp) {
#pragma unroll
            for (int x = 0; x < NX; ++x)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int d = d0 + d_of(x, r);
                    const float f[4] = {st[x][r], st[x][r + 1], st[x][r + 2], st[x][r + 3]};
                    if (d < p.Da) store_run<float, 4>(tp + scol * p.Da + d, p.Da - d, f);
                }
        }
    }
}

template <typename T, int DK, int NW, bool FULL> hipError_t run_walk_on(LinWalks all)
{
    const LinWalk &p = all.w[0];
    all.ndv = (int32_t)ceil_div(p.Dc, 32 * NW);
    all.blocks = (int64_t)all.count * p.B * p.H * p.nseg * all.ndv;
    hipLaunchKernelGGL((lin_walk<T, DK, NW, FULL>), dim3((unsigned)(8 * ceil_div(all.blocks, 8))), dim3(64 * NW), 0, p.stream, all);
    return hipGetLastError();
}

// f of the kernel for a walk (Da, Dc).
template <int DK_, int NW_> struct Kernel {
    static constexpr int DK = DK_, NW = NW_;
};
template <typename T, typename F> auto on_kernel(int64_t Da, int64_t Dc, int dtype, F f)
{
    const int waves = lin_waves(Da, Dc, dtype);
    switch (lin_wide(Da)) {
    case 64: return waves == 2 ? f(Kernel<64, 2>{}) : f(Kernel<64, 4>{});
    case 128: return waves == 2 ? f(Kernel<128, 2>{}) : f(Kernel<128, 4>{});
    default:
        if constexpr (kParts<T> < 3)
            if (waves == 8) return f(Kernel<256, 8>{});
        return f(Kernel<256, 4>{});
    }
}

// The walks of `all` are alike.
template <typename T, bool FULL> hipError_t run_walks(const LinWalks &all)
{
    const LinWalk &p = all.w[0];
    return on_kernel<T>(p.Da, p.Dc, p.dtype, [&](auto k) { return run_walk_on<T, decltype(k)::DK, decltype(k)::NW, FULL>(all); });
}

// Workgroups of the outputs' kernel that a compute unit holds: by the registers it is built for
// and by its LDS.
template <typename T> int held_walks(int64_t Da, int64_t Dc, int dtype)
{
    return on_kernel<T>(Da, Dc, dtype, [](auto k) {
        constexpr int DK = decltype(k)::DK, NW = decltype(k)::NW;
        constexpr int regs = 4 * kWavesPerSimd<T, DK, NW> / NW, lds = 160 * 1024 / (int)sizeof(WalkLds<T, DK, NW, true>);
        return regs < lds ? regs : lds;
    });
}

}  // namespace
}  // namespace gconv
