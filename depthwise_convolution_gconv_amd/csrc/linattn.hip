// linattn.hip -- linear attention with a decay for each head: chunked pass on the fp32
// matrix cores (any dtype), the scan over segment states, and the single-token step.
//
// The pass (linattn.hpp) walks a sequence in chunks of L = 64 tokens.  With R the state
// before the chunk and i, j token indices inside it,
//
//     out_i = inter_scale lam^(i+e0) a_i R  +  p_scale sum_{j <= i} lam^(i-j) (a_i . b_j) c_j
//     R'    = lam^m R + upd_scale sum_j lam^(m-j-e0) b_j c_j^T          (m tokens in the chunk)
//
// so a token costs 2 (Da + Dc) L + 4 Da Dc operations instead of the T Da of the quadratic
// form, all of them matrix products.  A workgroup owns one (batch, head, segment) and 64
// columns of c; R stays in its accumulators and a copy in LDS.  A sequence that gives too
// few workgroups is cut into segments: their local states are summed first
// (lin_walk_f32<..., false>), a scan turns them into the states before each segment, and
// then every segment is walked on its own.  That reads b and c a second time.
//
// Products run transposed (columns of the accumulators are tokens i): decay and mask of
// a token are then one scalar for each lane, and the scores leave the matrix cores in
// the layout the next product takes them in.
#include <algorithm>

#include "linattn.hpp"
#include "vecio.hpp"

namespace gconv {
namespace {

constexpr int kThreads = 256;
constexpr int kL = 64;       // tokens in a chunk
constexpr int kNT = 64;      // columns of c for each workgroup
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mfma_f32(float a, float b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
}

// Row strides keep 16-byte reads of 16 neighbouring rows on distinct LDS banks.
template <int DK> struct LdsF32 {
    float b[kL][DK + 4];
    float c[kL][kNT + 4];
    float s[DK][kNT + 4];
    float pw[kL + 1];        // lam^0 .. lam^64
};

template <typename T, typename TO, int DK, bool FULL>
__global__ void __launch_bounds__(kThreads)
lin_walk_f32(const LinWalk p)
{
    constexpr int NBR = kL * DK / 4 / kThreads;    // staging runs of 4 elements of b for each thread
    constexpr int NCR = kL * kNT / 4 / kThreads;
    constexpr int NST = DK / 64;                   // 32x32 state tiles for each wave
    __shared__ LdsF32<DK> sm;
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
    const int n = lin_len(p, bi), n0 = dv * kNT;
    const int useg = seg * p.seg_len;
    const int utop = min(useg + p.seg_len, FULL ? p.T : n);   // tokens [useg, utop) of this workgroup

    if (tid <= kL) sm.pw[tid] = lin_pow(p.log_decay[h], tid);
    const T *ab = (const T *)p.a + bi * p.asb + (h / p.ra) * p.ash;
    const T *bb = (const T *)p.b + bi * p.bsb + (h / p.rb) * p.bsh;
    const T *cb = (const T *)p.c + bi * p.csb + (h / p.rc) * p.csh + n0;
    TO *ob = (TO *)p.out + bi * p.osb + h * p.osh + n0;

    // The state, as accumulators: wave w holds columns 32 (w & 1) .. and rows 32 ((w >> 1) + 2x) ..
    const int scol = (wave & 1) * 32 + l32, srow = (wave >> 1) * 32 + 4 * half;
    f32x16 st[NST];
    const float *sp = nullptr;
    int64_t sr = 0, sc = 0;
    if (FULL && p.nseg > 1) {
        sp = p.ws + (bh * p.nseg + seg) * (int64_t)p.Da * p.Dc;
        sr = p.wsr; sc = p.wsc;
    } else if (FULL && p.s0) {
        sp = p.s0 + bi * p.s0b + h * p.s0h;
        sr = p.s0r; sc = p.s0c;
    }
    bool have = sp != nullptr;   // a state that is not known to be zero
#pragma unroll
    for (int x = 0; x < NST; ++x)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int d = srow + 64 * x + 8 * (r / 4) + r % 4;
            st[x][r] = have && d < p.Da && n0 + scol < p.Dc ? sp[d * sr + (n0 + scol) * sc] : 0.0f;
        }

    Run<T, 4> br[NBR], cr[NCR];
    auto fetch = [&](int u0) {
#pragma unroll
        for (int i = 0; i < NBR; ++i) {
            const int x = tid + i * kThreads, j = x / (DK / 4), d = x % (DK / 4) * 4;
            br[i] = load_raw<T, 4>(bb + (int64_t)lin_token(p, u0 + j, n) * p.bst + d, u0 + j < min(n, utop) ? p.Da - d : 0);
        }
#pragma unroll
        for (int i = 0; i < NCR; ++i) {
            const int x = tid + i * kThreads, j = x / (kNT / 4), d = x % (kNT / 4) * 4;
            cr[i] = load_raw<T, 4>(cb + (int64_t)lin_token(p, u0 + j, n) * p.cst + d,
                                   u0 + j < min(n, utop) ? p.Dc - n0 - d : 0);
        }
    };
    fetch(useg);

    for (int u0 = useg; u0 < utop; u0 += kL) {
        const int m = max(0, min(n - u0, kL));
        // The previous chunk's readers are done with b, c and s (barrier at the loop's end).
#pragma unroll
        for (int i = 0; i < NBR; ++i) {
            const int x = tid + i * kThreads, j = x / (DK / 4), d = x % (DK / 4) * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) sm.b[j][d + e] = to_f32(br[i].v[e]);
        }
#pragma unroll
        for (int i = 0; i < NCR; ++i) {
            const int x = tid + i * kThreads, j = x / (kNT / 4), d = x % (kNT / 4) * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) sm.c[j][d + e] = to_f32(cr[i].v[e]);
        }
        if (FULL && have) {
#pragma unroll
            for (int x = 0; x < NST; ++x)
#pragma unroll
                for (int r = 0; r < 16; ++r) sm.s[srow + 64 * x + 8 * (r / 4) + r % 4][scol] = st[x][r];
        }
        __syncthreads();
        if (u0 + kL < utop) fetch(u0 + kL);

        if constexpr (FULL) {
            const int rb = wave >> 1, nh = (wave & 1) * 32;
            const int i = rb * 32 + l32;          // this lane's token
            const int u = u0 + i;
            const T *ap = ab + (int64_t)lin_token(p, u, n) * p.ast;
            float aq[DK / 8][4];                  // a_i at d = 8g + 4 half ..
#pragma unroll
            for (int g = 0; g < DK / 8; ++g) load_run<T, 4>(ap + 8 * g + 4 * half, i < m ? p.Da - 8 * g - 4 * half : 0, aq[g]);
            f32x16 acc;
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[r] = 0.0f;
            if (have) {
#pragma unroll
                for (int g = 0; g < DK / 8; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc = mfma_f32(sm.s[8 * g + 4 * half + e][nh + l32], aq[g][e], acc);
                const float f = p.inter_scale * sm.pw[i + p.e0];
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[r] *= f;
            }
            for (int jt = 0; jt <= rb && jt * 32 < m; ++jt) {
                f32x16 s;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = 0.0f;
#pragma unroll
                for (int g = 0; g < DK / 8; ++g) {
                    const float4 kv = *reinterpret_cast<const float4 *>(&sm.b[jt * 32 + l32][8 * g + 4 * half]);
                    s = mfma_f32(kv.x, aq[g][0], s);
                    s = mfma_f32(kv.y, aq[g][1], s);
                    s = mfma_f32(kv.z, aq[g][2], s);
                    s = mfma_f32(kv.w, aq[g][3], s);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int j = jt * 32 + 8 * (r / 4) + 4 * half + r % 4;
                    // Scores of later tokens are dropped, not multiplied by zero: they may be infinite.
                    const float w = j <= i ? s[r] * (sm.pw[max(i - j, 0)] * p.p_scale) : 0.0f;
                    acc = mfma_f32(sm.c[j][nh + l32], w, acc);
                }
            }
            if (u < utop) {
                TO *op = ob + (int64_t)lin_token(p, u, n) * p.ost + nh + 4 * half;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = i < m ? acc[4 * g + e] : 0.0f;
                    const int left = p.Dc - n0 - nh - 4 * half - 8 * g;
                    if (left > 0) store_run<TO, 4>(op + 8 * g, left, f);
                }
            }
        }

        if (m > 0 && (!FULL || u0 + kL < utop || (p.nseg == 1 && p.sf))) {
            const float lm = sm.pw[m];
#pragma unroll
            for (int x = 0; x < NST; ++x)
#pragma unroll
                for (int r = 0; r < 16; ++r) st[x][r] *= lm;
            for (int s = 0; 2 * s < m; ++s) {
                const int j = 2 * s + half;
                const float w = p.upd_scale * sm.pw[max(m - j - p.e0, 0)], cv = sm.c[j][scol];
#pragma unroll
                for (int x = 0; x < NST; ++x)
                    st[x] = mfma_f32(sm.b[j][(wave >> 1) * 32 + 64 * x + l32] * w, cv, st[x]);
            }
            have = true;
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
    if (dp && n0 + scol < p.Dc) {
#pragma unroll
        for (int x = 0; x < NST; ++x)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int d = srow + 64 * x + 8 * (r / 4) + r % 4;
                if (d < p.Da) dp[d * dr + (n0 + scol) * dc] = st[x][r];
            }
    }
}

// States before each segment from the segments' own sums, in place:
//     R_(g+1) = lam^(tokens of g) R_g + local_g,  R_0 = s0.
// One thread for each state element, 8 segments' loads in flight.
constexpr int kMaxSeg = 1024;
__global__ void __launch_bounds__(kThreads)
lin_scan(const LinWalk p)
{
    __shared__ float lam[kMaxSeg];
    const int tid = threadIdx.x;
    const int64_t cells = (int64_t)p.Da * p.Dc, tiles = (cells + kThreads - 1) / kThreads;
    const int64_t bh = blockIdx.x / tiles;
    const int h = (int)(bh % p.H), bi = (int)(bh / p.H);
    const int n = lin_len(p, bi);
    for (int g = tid; g < p.nseg; g += kThreads)
        lam[g] = lin_pow(p.log_decay[h], max(0, min(n - g * p.seg_len, p.seg_len)));
    __syncthreads();
    const int64_t x = (blockIdx.x % tiles) * kThreads + tid;
    if (x >= cells) return;
    const int64_t d = x / p.Dc, c = x % p.Dc;
    float r = p.s0 ? p.s0[bi * p.s0b + h * p.s0h + d * p.s0r + c * p.s0c] : 0.0f;
    float *w = p.ws + bh * p.nseg * cells + x;
    for (int g0 = 0; g0 < p.nseg; g0 += 8) {
        float loc[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) loc[g] = g0 + g < p.nseg ? w[(g0 + g) * cells] : 0.0f;
#pragma unroll
        for (int g = 0; g < 8; ++g)
            if (g0 + g < p.nseg) {
                w[(g0 + g) * cells] = r;
                r = fmaf(lam[g0 + g], r, loc[g]);
            }
    }
    if (p.sf) p.sf[bi * p.sfb + h * p.sfh + d * p.sfr + c * p.sfc] = r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
lin_group_sum(const float *__restrict__ part, T *__restrict__ out, int64_t sb, int64_t st, int64_t sh, int64_t total,
              int64_t T_in, int Hk, int r, int D)
{
    for (int64_t x = (int64_t)blockIdx.x * kThreads + threadIdx.x; x < total; x += (int64_t)gridDim.x * kThreads) {
        const int64_t g = x / D, bt = g / Hk;    // (batch, token, key head), (batch, token)
        const int d = (int)(x - g * D);
        const float *src = part + g * r * D + d;
        float s = src[0];
        for (int j = 1; j < r; ++j) s += src[(int64_t)j * D];
        out[bt / T_in * sb + bt % T_in * st + (g - bt * Hk) * sh + d] = from_f32<T>(s);
    }
}

template <typename T, typename TO, bool FULL>
hipError_t run_walk(const LinWalk &p0)
{
    LinWalk p = p0;
    p.ndv = (int32_t)ceil_div(p.Dc, kNT);
    p.blocks = (int64_t)p.B * p.H * p.nseg * p.ndv;
    const int64_t grid = 8 * ceil_div(p.blocks, 8);
    if (grid >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    if (p.Da <= 64)
        hipLaunchKernelGGL((lin_walk_f32<T, TO, 64, FULL>), dim3((unsigned)grid), dim3(kThreads), 0, p.stream, p);
    else if (p.Da <= 128)
        hipLaunchKernelGGL((lin_walk_f32<T, TO, 128, FULL>), dim3((unsigned)grid), dim3(kThreads), 0, p.stream, p);
    else
        hipLaunchKernelGGL((lin_walk_f32<T, TO, 256, FULL>), dim3((unsigned)grid), dim3(kThreads), 0, p.stream, p);
    return hipGetLastError();
}

template <bool FULL> hipError_t run_walk_typed(const LinWalk &p)
{
    switch (p.dtype) {
    case DT_F32: return run_walk<float, float, FULL>(p);
    case DT_F16: return FULL && p.out_f32 ? run_walk<_Float16, float, FULL>(p) : run_walk<_Float16, _Float16, FULL>(p);
    default: return FULL && p.out_f32 ? run_walk<__bf16, float, FULL>(p) : run_walk<__bf16, __bf16, FULL>(p);
    }
}

// ---------------------------------------------------------------- single tokens
//
// S <- lam S + k v^T in place, o = scale q S: one pass over the state, which is all the
// traffic there is (8 Dk Dv bytes a head).  One workgroup for each (token, head): lanes
// run along 4 columns each, thread rows take every RP-th row of the state, and the RP
// partial sums of o are added in a fixed order through LDS.
template <typename T, int CG>
__global__ void __launch_bounds__(kThreads)
lin_step(const LinStep p)
{
    constexpr int RP = kThreads / CG;
    __shared__ float red[RP][CG * 4];
    const int tid = threadIdx.x, c0 = tid % CG * 4, r0 = tid / CG;
    const int h = blockIdx.x % p.H, bi = blockIdx.x / p.H;
    const int left = p.Dv - c0;
    const int64_t slot = p.slots ? p.slots[bi] : bi;
    T *op = (T *)p.o + bi * p.osb + h * p.osh + c0;
    if (slot < 0 || slot >= p.n) {   // no state: nothing to update, the token's output is zero
        const float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (r0 == 0 && left > 0) store_run<T, 4>(op, left, z);
        return;
    }
    const int hk = h / (p.H / p.Hk);
    const T *qp = (const T *)p.q + bi * p.qsb + hk * p.qsh, *kp = (const T *)p.k + bi * p.ksb + hk * p.ksh;
    float v[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    load_run<T, 4>((const T *)p.v + bi * p.vsb + h * p.vsh + c0, left, v);
    const float lam = expf(p.log_decay[h]);
    float *sp = p.state + (slot * p.H + h) * (int64_t)p.Dk * p.Dv + c0;
    constexpr int U = 8;             // rows in flight for each thread
    for (int d0 = r0; d0 < p.Dk; d0 += RP * U) {
        float s[U][4], qv[U], kv[U];
#pragma unroll
        for (int x = 0; x < U; ++x) {
            const int d = d0 + x * RP;
            load_run<float, 4>(sp + (int64_t)d * p.Dv, d < p.Dk ? left : 0, s[x]);
            qv[x] = d < p.Dk ? to_f32(qp[d]) : 0.0f;
            kv[x] = d < p.Dk ? to_f32(kp[d]) : 0.0f;
        }
#pragma unroll
        for (int x = 0; x < U; ++x) {
            const int d = d0 + x * RP;
            if (d >= p.Dk || left <= 0) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[x][e] = fmaf(lam, s[x][e], kv[x] * v[e]);
                o[e] = fmaf(qv[x], s[x][e], o[e]);
            }
            store_run<float, 4>(sp + (int64_t)d * p.Dv, left, s[x]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) red[r0][c0 + e] = o[e];
    __syncthreads();
    if (r0 == 0 && left > 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            for (int r = 1; r < RP; ++r) o[e] += red[r][c0 + e];
            o[e] *= p.scale;
        }
        store_run<T, 4>(op, left, o);
    }
}

template <typename T> hipError_t run_step(const LinStep &p)
{
    const dim3 grid((unsigned)(p.B * p.H)), block(kThreads);
    if (p.Dv <= 64) hipLaunchKernelGGL((lin_step<T, 16>), grid, block, 0, p.stream, p);
    else if (p.Dv <= 128) hipLaunchKernelGGL((lin_step<T, 32>), grid, block, 0, p.stream, p);
    else hipLaunchKernelGGL((lin_step<T, 64>), grid, block, 0, p.stream, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_lin_scan(const LinWalk &p)
{
    const int64_t blocks = (int64_t)p.B * p.H * ceil_div((int64_t)p.Da * p.Dc, kThreads);
    if (blocks >= (int64_t(1) << 31) || p.nseg > kMaxSeg) return hipErrorInvalidValue;
    hipLaunchKernelGGL(lin_scan, dim3((unsigned)blocks), dim3(kThreads), 0, p.stream, p);
    return hipGetLastError();
}

hipError_t launch_lin_states(const LinWalk &p, const char **kname)
{
    *kname = "lin_walk_f32";
    const hipError_t err = run_walk_typed<false>(p);
    return err != hipSuccess ? err : launch_lin_scan(p);
}

hipError_t launch_lin_walk(const LinWalk &p, const char **kname)
{
    *kname = "lin_walk_f32";
    return run_walk_typed<true>(p);
}

hipError_t launch_lin_group_sum(const float *part, void *out, const int64_t *ost, int64_t B, int64_t T, int Hk, int r,
                                int D, int dtype, hipStream_t stream)
{
    const int64_t total = B * T * Hk * D;
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div(total, kThreads), 1 << 16)), block(kThreads);
    switch (dtype) {
    case DT_F32:
        hipLaunchKernelGGL((lin_group_sum<float>), grid, block, 0, stream, part, (float *)out, ost[0], ost[1], ost[2],
                           total, T, Hk, r, D);
        break;
    case DT_F16:
        hipLaunchKernelGGL((lin_group_sum<_Float16>), grid, block, 0, stream, part, (_Float16 *)out, ost[0], ost[1],
                           ost[2], total, T, Hk, r, D);
        break;
    default:
        hipLaunchKernelGGL((lin_group_sum<__bf16>), grid, block, 0, stream, part, (__bf16 *)out, ost[0], ost[1], ost[2],
                           total, T, Hk, r, D);
        break;
    }
    return hipGetLastError();
}

hipError_t launch_lin_step(const LinStep &p, const char **kname)
{
    *kname = "lin_step";
    switch (p.dtype) {
    case DT_F32: return run_step<float>(p);
    case DT_F16: return run_step<_Float16>(p);
    default: return run_step<__bf16>(p);
    }
}

}  // namespace gconv
