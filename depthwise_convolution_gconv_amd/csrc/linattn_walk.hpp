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
// vector unit.  Scores and the state that meets a_i are rounded to as many parts as the
// inputs have: their error stays at one rounding of the output's own type (2^-9 of a term
// in bf16, 2^-18 in fp16, 2^-25 in fp32), and both stay fp32 in their accumulators.
//
// Nothing but the inputs goes through LDS.  Products run transposed (columns of the
// accumulators are tokens i, rows are j or columns of c): scores and the state leave the
// matrix cores with four consecutive rows in a lane, and as the order of a reduction is
// free, the other operand is read in that same order (rows 4h .. 4h+3 and 8+4h .. 8+4h+3
// of each 16 for the lane's half h).  A wave keeps the state of its 32 columns in
// accumulators for the whole walk.
#pragma once

#include "linattn.hpp"
#include "vecio.hpp"

namespace gconv {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <typename T> constexpr int kParts = sizeof(T) == 4 ? 3 : 2;
template <> constexpr int kParts<__bf16> = 1;
constexpr int kUpdParts = 3;
// Tokens in a chunk: more parts take more LDS, more columns more registers.
template <typename T, int DK, int NW> constexpr int kLen = kParts<T> == 1 && DK / NW <= 32 ? 64 : 32;

// A tile of D columns in LDS: rows 16 banks apart within each four and groups of four two
// banks apart, so the 32 rows of an operand read (8 bytes each) and the 4 rows x 64 bytes
// of a transposing read both cover all 64 banks.
template <int D> struct Tile {
    static constexpr int row = D == 64 ? 96 : D == 128 ? 160 : 288;
    static constexpr int group = D == 64 ? 388 : D == 128 ? 644 : 1156;
    static __device__ __forceinline__ int at(int j, int d) { return (j >> 2) * group + (j & 3) * row + d; }
    static constexpr int size(int rows) { return rows / 4 * group; }
};

template <int NP> struct Part8 { bf16x8 p[NP]; };

// x as a sum of NP bf16 parts, each the rounding of what the earlier ones leave.
template <int NP> __device__ __forceinline__ Part8<NP> split8(const float (&x)[8])
{
    Part8<NP> r;
    float left[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) left[e] = x[e];
#pragma unroll
    for (int q = 0; q < NP; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            r.p[q][e] = (__bf16)left[e];
            if (q + 1 < NP) left[e] -= (float)r.p[q][e];
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

// 8 values of row j at columns d + 4h .. and d + 8 + 4h .. (the caller's d holds 4h).
template <int D, int NP>
__device__ __forceinline__ Part8<NP> read_rows(const __bf16 *t, int size, int at)
{
    Part8<NP> r;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const bf16x4 lo = *reinterpret_cast<const bf16x4 *>(t + q * size + at);
        const bf16x4 hi = *reinterpret_cast<const bf16x4 *>(t + q * size + at + 8);
        r.p[q] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
}

// The same of column (lane) over rows: two transposing reads of 4 rows each, `at` and
// two groups of rows further.
template <int D, int NP>
__device__ __forceinline__ Part8<NP> read_cols(const __bf16 *t, int size, int at)
{
    typedef __attribute__((address_space(3))) s16x4 lds4;
    Part8<NP> r;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        const bf16x4 lo = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(t + q * size + at)));
        const bf16x4 hi = __builtin_bit_cast(
            bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(t + q * size + at + 2 * Tile<D>::group)));
        r.p[q] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
    return r;
}

// 8 elements on their way from memory to LDS.
template <typename T> struct Raw8 { RunVec<T, 16 / (int)sizeof(T)> w[sizeof(T) / 2]; };

template <typename T> __device__ __forceinline__ Raw8<T> load8(const T *src, int valid)
{
    constexpr int N = 16 / sizeof(T);
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < 8 / N; ++i) r.w[i] = load_words<T, N>(src + N * i, valid - N * i);
    return r;
}

// They go to their parts' tiles.
template <typename T, int NP> __device__ __forceinline__ void stage8(__bf16 *t, int size, int at, const Raw8<T> &v)
{
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
#pragma unroll
    for (int q = 0; q < NP; ++q) {
        *reinterpret_cast<bf16x4 *>(t + q * size + at) = __builtin_shufflevector(r.p[q], r.p[q], 0, 1, 2, 3);
        *reinterpret_cast<bf16x4 *>(t + q * size + at + 4) = __builtin_shufflevector(r.p[q], r.p[q], 4, 5, 6, 7);
    }
}

template <typename T, int DK, int NW, bool FULL> struct WalkLds {
    static constexpr int NP = kParts<T>, L = kLen<T, DK, NW>, NT = 32 * NW;
    static constexpr int AB = Tile<DK>::size(L), C = Tile<NT>::size(L);
    __bf16 a[FULL ? NP * AB : 4];
    __bf16 b[NP * AB];
    __bf16 c[NP * C];
    float pw[L + 1];         // lam^0 .. lam^L
    float upd[L];            // upd_scale lam^(m-j-e0)
    float off[32];           // lam^(32-j)
};

// Two workgroups of four waves share a compute unit where their registers and LDS allow.
template <typename T, int DK, int NW> constexpr int kWavesPerSimd = DK == 256 || kParts<T> == 3 ? 1 : 2;

template <typename T, typename TO, int DK, int NW, bool FULL>
__global__ void __launch_bounds__(64 * NW, (kWavesPerSimd<T, DK, NW>))
lin_walk(const LinWalk p)
{
    constexpr int NP = kParts<T>, L = kLen<T, DK, NW>, NT = 32 * NW, NTH = 64 * NW;
    typedef WalkLds<T, DK, NW, FULL> Lds;
    constexpr int NBR = L * DK / 8 / NTH, NCR = L * NT / 8 / NTH;   // staging runs of 8 for each thread
    constexpr int NX = DK / 32, NS = DK / 16, NG = L / 16;          // state tiles, steps along columns, along tokens
    __shared__ __attribute__((aligned(16))) Lds sm;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, l32 = lane & 31, half = lane >> 5;

    // Workgroups go round the 8 XCDs; a contiguous run of ids on one XCD keeps the column
    // tiles and heads that share a's and b's rows on one L2.
    const int64_t per = (p.blocks + 7) / 8;
    int64_t id = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (id >= p.blocks) return;
    const int dv = (int)(id % p.ndv);
    id /= p.ndv;
    const int seg = (int)(id % p.nseg);
    const int64_t bh = id / p.nseg;
    const int h = (int)(bh % p.H), bi = (int)(bh / p.H);
    const int n = lin_len(p, bi), n0 = dv * NT;
    const int useg = seg * p.seg_len;
    const int utop = min(useg + p.seg_len, FULL ? p.T : n);   // tokens [useg, utop) of this workgroup
    const int ulive = min(n, utop);
    const bool mine = n0 + wave * 32 < p.Dc;                  // this wave has columns

    for (int e = tid; e <= L; e += NTH) sm.pw[e] = lin_pow(p.log_decay[h], e);
    if (tid < 32) sm.off[tid] = lin_pow(p.log_decay[h], 32 - tid);
    const T *ab = (const T *)p.a + bi * p.asb + (h / p.ra) * p.ash;
    const T *bb = (const T *)p.b + bi * p.bsb + (h / p.rb) * p.bsh;
    const T *cb = (const T *)p.c + bi * p.csb + (h / p.rc) * p.csh + n0;

    // The state: column n0 + 32 wave + l32, rows 32x + 8 (r / 4) + 4 half + r % 4.
    const int scol = n0 + wave * 32 + l32;
    f32x16 st[NX];
    const float *sp = nullptr;
    int64_t sr = 0, sc = 0;
    if (FULL && p.nseg > 1) {
        sp = p.ws + (bh * p.nseg + seg) * (int64_t)p.Da * p.Dc;
        sr = p.wsr; sc = p.wsc;
    } else if (FULL && p.s0) {
        sp = p.s0 + bi * p.s0b + h * p.s0h;
        sr = p.s0r; sc = p.s0c;
    }
    if (sp && scol < p.Dc) {
        sp += scol * sc;
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
            for (int r = 0; r < 16; ++r) {     // rows past the last read that one
                const int d = 32 * x + 8 * (r / 4) + 4 * half + r % 4;
                const float v = sp[min(d, p.Da - 1) * sr];
                st[x][r] = d < p.Da ? v : 0.0f;
            }
    } else {
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
            for (int r = 0; r < 16; ++r) st[x][r] = 0.0f;
    }

    Raw8<T> ar[FULL ? NBR : 1], br[NBR], cr[NCR];
    auto fetch = [&](int u0) {
#pragma unroll
        for (int i = 0; i < NBR; ++i) {
            const int x = tid + i * NTH, j = x / (DK / 8), d = x % (DK / 8) * 8, u = u0 + j;
            const int left = u < ulive ? p.Da - d : 0;
            const int64_t tok = lin_token(p, u, n);
            if constexpr (FULL) ar[i] = load8<T>(ab + tok * p.ast + d, left);
            br[i] = load8<T>(bb + tok * p.bst + d, left);
        }
#pragma unroll
        for (int i = 0; i < NCR; ++i) {
            const int x = tid + i * NTH, j = x / (NT / 8), d = x % (NT / 8) * 8, u = u0 + j;
            cr[i] = load8<T>(cb + (int64_t)lin_token(p, u, n) * p.cst + d, u < ulive ? p.Dc - n0 - d : 0);
        }
    };
    fetch(useg);
    __syncthreads();     // the powers

    const int row_at = Tile<DK>::at(l32, 4 * half);                                   // row l32
    const int col_row = 4 * half + ((lane & 15) >> 2), col_d = (lane & 16) + (lane & 3) * 4;
    const int bcol_at = Tile<DK>::at(col_row, col_d), ccol_at = Tile<NT>::at(col_row, 32 * wave + col_d);

    int mset = -1;
    for (int u0 = useg; u0 < utop; u0 += L) {
        const int m = max(0, min(n - u0, L));
        // The previous chunk's readers are done (barrier at the loop's end).
#pragma unroll
        for (int i = 0; i < NBR; ++i) {
            const int x = tid + i * NTH, at = Tile<DK>::at(x / (DK / 8), x % (DK / 8) * 8);
            if constexpr (FULL) stage8<T, NP>(sm.a, Lds::AB, at, ar[i]);
            stage8<T, NP>(sm.b, Lds::AB, at, br[i]);
        }
#pragma unroll
        for (int i = 0; i < NCR; ++i) {
            const int x = tid + i * NTH;
            stage8<T, NP>(sm.c, Lds::C, Tile<NT>::at(x / (NT / 8), x % (NT / 8) * 8), cr[i]);
        }
        if (m != mset) {
            if (tid < L) sm.upd[tid] = p.upd_scale * sm.pw[max(m - tid - p.e0, 0)];
            mset = m;
        }
        __syncthreads();
        if (u0 + L < utop) fetch(u0 + L);

        if (mine && m > 0) {
            auto cols_c = [&](int g) { return read_cols<NT, NP>(sm.c, Lds::C, ccol_at + 4 * g * Tile<NT>::group); };
            if constexpr (FULL) {
                // Rolled: the copies would keep each other's operands alive.
#pragma unroll 1
                for (int it = 0; 32 * it < m; ++it) {
                    const int a_at = row_at + it * 8 * Tile<DK>::group;
                    f32x16 acc, sc;
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[r] = sc[r] = 0.0f;
                    // a_i R, and the scores of the tile on the diagonal.
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const Part8<NP> aq = read_rows<DK, NP>(sm.a, Lds::AB, a_at + 16 * s);
                        float f[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) f[e] = st[s / 2][s % 2 * 8 + e];
                        acc = mma<NP - 1>(split8<NP>(f), aq, acc);
                        sc = mma<NP - 1>(read_rows<DK, NP>(sm.b, Lds::AB, a_at + 16 * s), aq, sc);
                    }
                    const float fi = p.inter_scale * sm.pw[min(it * 32 + l32 + p.e0, L)];
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int j = 8 * (r / 4) + 4 * half + r % 4;
                        acc[r] *= fi;
                        // Scores of later tokens are dropped, not multiplied by zero: they may be infinite.
                        sc[r] = j <= l32 ? sc[r] * (p.p_scale * sm.pw[max(l32 - j, 0)]) : 0.0f;
                    }
                    auto add = [&](int jt) {
#pragma unroll
                        for (int g = 0; g < 2; ++g) {
                            float f[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) f[e] = sc[8 * g + e];
                            acc = mma<NP - 1>(cols_c(2 * jt + g), split8<NP>(f), acc);
                        }
                    };
                    add(it);
                    if (L > 32 && it > 0) {   // the tile before it
#pragma unroll
                        for (int r = 0; r < 16; ++r) sc[r] = 0.0f;
#pragma unroll
                        for (int s = 0; s < NS; ++s)
                            sc = mma<NP - 1>(read_rows<DK, NP>(sm.b, Lds::AB, row_at + 16 * s),
                                             read_rows<DK, NP>(sm.a, Lds::AB, a_at + 16 * s), sc);
                        const float fs = p.p_scale * sm.pw[l32];
#pragma unroll
                        for (int r = 0; r < 16; ++r) sc[r] *= fs * sm.off[8 * (r / 4) + 4 * half + r % 4];
                        add(0);
                    }
                    const int i = it * 32 + l32, u = u0 + i;
                    if (u < utop) {
                        TO *op = (TO *)p.out + bi * p.osb + (int64_t)lin_token(p, u, n) * p.ost + h * p.osh + n0 +
                                 wave * 32 + 4 * half;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            float f[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) f[e] = i < m ? acc[4 * g + e] : 0.0f;
                            const int left = p.Dc - n0 - wave * 32 - 4 * half - 8 * g;
                            if (left > 0) store_run<TO, 4>(op + 8 * g, left, f);
                        }
                    }
                }
            }

            if (!FULL || u0 + L < utop || (p.nseg == 1 && p.sf)) {
                const float lm = sm.pw[m];
#pragma unroll
                for (int x = 0; x < NX; ++x)
#pragma unroll
                    for (int r = 0; r < 16; ++r) st[x][r] *= lm;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    if (16 * g >= m) break;
                    const Part8<NP> cT = cols_c(g);
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
                        st[x] = mma<2>(read_cols<DK, NP>(sm.b, Lds::AB, bcol_at + 4 * g * Tile<DK>::group + 32 * x), wc, st[x]);
                }
            }
        }
        if (FULL && mine) {
            // Tokens past the sequence's end, in 32-token tiles that held none that exist: zeros.
#pragma unroll
            for (int it = 0; it < L / 32; ++it) {
                const int u = u0 + it * 32 + l32;
                if (32 * it < m || u >= utop) continue;
                TO *op = (TO *)p.out + bi * p.osb + (int64_t)u * p.ost + h * p.osh + n0 + wave * 32 + 4 * half;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const int left = p.Dc - n0 - wave * 32 - 4 * half - 8 * g;
                    if (left > 0) store_run<TO, 4>(op + 8 * g, left, z);
                }
            }
        }
        __syncthreads();
    }

    float *dp = nullptr;
    int64_t dr = 0, dc = 0;
    if (!FULL) {
        dp = p.ws + (bh * p.nseg + seg) * (int64_t)p.Da * p.Dc;
        dr = p.wsr; dc = p.wsc;
    } else if (p.nseg == 1 && p.sf) {
        dp = p.sf + bi * p.sfb + h * p.sfh;
        dr = p.sfr; dc = p.sfc;
    }
    if (dp && scol < p.Dc) {
        int d0 = 4 * half;
        asm("" : "+v"(d0));      // the addresses are made here, not kept through the walk
        dp += d0 * dr + scol * dc;
#pragma unroll
        for (int x = 0; x < NX; ++x)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int d = 32 * x + 8 * (r / 4) + r % 4;
                if (d0 + d < p.Da) dp[d * dr] = st[x][r];
            }
    }
}

template <typename T, typename TO, int DK, bool FULL>
hipError_t run_walk_waves(const LinWalk &p0)
{
    LinWalk p = p0;
    const int nw = p.Dc <= 64 ? 2 : 4;
    p.ndv = (int32_t)ceil_div(p.Dc, 32 * nw);
    p.blocks = (int64_t)p.B * p.H * p.nseg * p.ndv;
    const int64_t grid = 8 * ceil_div(p.blocks, 8);
    if (grid >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    if (nw == 2) hipLaunchKernelGGL((lin_walk<T, TO, DK, 2, FULL>), dim3((unsigned)grid), dim3(128), 0, p.stream, p);
    else hipLaunchKernelGGL((lin_walk<T, TO, DK, 4, FULL>), dim3((unsigned)grid), dim3(256), 0, p.stream, p);
    return hipGetLastError();
}

template <typename T, typename TO, bool FULL> hipError_t run_walk(const LinWalk &p)
{
    if (p.Da <= 64) return run_walk_waves<T, TO, 64, FULL>(p);
    if (p.Da <= 128) return run_walk_waves<T, TO, 128, FULL>(p);
    return run_walk_waves<T, TO, 256, FULL>(p);
}

}  // namespace
}  // namespace gconv
