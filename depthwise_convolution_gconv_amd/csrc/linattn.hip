// linattn.hip -- linear attention with a decay for each head: the scan over segment
// states, the sum over a key head's value heads, and the single-token step.  The chunked
// pass is in linattn_walk.hpp.
#include <algorithm>

#include "linattn.hpp"
#include "vecio.hpp"

namespace gconv {
namespace {

constexpr int kThreads = 256;

// States before each segment but the first from the segments' own sums, in place:
//     R_1 = local_0,  R_(g+1) = lam^(tokens of g) R_g + local_g
// (local_0 holds what is left of s0).  Powers and the running state are fp64, rounded where a
// state leaves: a slowly fading state passes up to 1024 powers of one sign of rounding (fp32: 176
// half steps after 512 segments).  Two neighbouring elements for each thread, 8 segments' loads
// in flight: 20 us for 47 segments of 16 heads of 128 x 128, 100 MB, 5 TB/s.
constexpr int kScan = 2;
__global__ void __launch_bounds__(kThreads)
lin_scan(const LinWalks all)
{
    __shared__ double lam[kMaxSeg];
    const int tid = threadIdx.x;
    // Every walk's states have as many elements.
    const int64_t cells = (int64_t)all.w[0].Da * all.w[0].Dc, tiles = (cells + kScan * kThreads - 1) / (kScan * kThreads);
    const LinWalk &p = all.w[blockIdx.x / all.blocks];
    const int64_t bh = blockIdx.x % all.blocks / tiles;
    const int h = (int)(bh % p.H), bi = (int)(bh / p.H);
    const int n = lin_len(p, bi);
    for (int g = tid; g < p.nseg; g += kThreads)
        lam[g] = lin_pow64(p.log_decay[h], max(0, min(n - g * p.seg_len, p.seg_len)));
    __syncthreads();
    const int64_t x = ((blockIdx.x % all.blocks % tiles) * kThreads + tid) * kScan;
    const int left = (int)min(cells - x, (int64_t)kScan);
    if (left <= 0) return;
    double r[kScan];
#pragma unroll
    for (int e = 0; e < kScan; ++e) {
        const int64_t d = (x + e) / p.Dc, c = (x + e) % p.Dc;
        r[e] = p.nseg == 0 && p.s0 && e < left ? p.s0[bi * p.s0b + h * p.s0h + d * p.s0r + c * p.s0c] : 0.0f;
    }
    float *w = p.ws + bh * p.nseg * cells + x;
    for (int g0 = 0; g0 < p.nseg; g0 += 8) {
        float loc[8][kScan];
#pragma unroll
        for (int g = 0; g < 8; ++g) load_run<float, kScan>(w + (g0 + g) * cells, g0 + g < p.nseg ? left : 0, loc[g]);
#pragma unroll
        for (int g = 0; g < 8; ++g)
            if (g0 + g < p.nseg) {
                const float before[kScan] = {(float)r[0], (float)r[1]};
                if (g0 + g > 0) store_run<float, kScan>(w + (g0 + g) * cells, left, before);
#pragma unroll
                for (int e = 0; e < kScan; ++e) r[e] = fma(lam[g0 + g], r[e], (double)loc[g][e]);
            }
    }
    if (p.sf) {
#pragma unroll
        for (int e = 0; e < kScan; ++e) {
            const int64_t d = (x + e) / p.Dc, c = (x + e) % p.Dc;
            if (e < left) p.sf[bi * p.sfb + h * p.sfh + d * p.sfr + c * p.sfc] = (float)r[e];
        }
    }
}

// The value heads of a key head added up: workgroups of 256 columns of a token's Hk D.
template <typename T>
__global__ void __launch_bounds__(kThreads)
lin_group_sum(const float *__restrict__ part, T *__restrict__ out, int64_t sb, int64_t st, int64_t sh, int T_in, int Hk,
              int r, int D, int blocks, int64_t bt0)
{
    const int64_t bt = bt0 + blockIdx.x / blocks;      // (batch, token)
    const int x = (int)(blockIdx.x % blocks) * kThreads + threadIdx.x, g = x / D, d = x - g * D;
    if (g >= Hk) return;
    const float *src = part + (bt * Hk + g) * r * D + d;
    float s = src[0];
    for (int j = 1; j < r; ++j) s += src[j * D];
    out[bt / T_in * sb + bt % T_in * st + g * sh + d] = from_f32<T>(s);
}

// ---------------------------------------------------------------- single tokens
//
// S <- lam S + k v^T in place, o = scale q S: one pass over the state, which is all the
// traffic there is (8 Dk Dv bytes a head).  One workgroup for each (token, head): lanes run
// along 4 columns each, thread rows take every RP-th row of the state, U at a time, and the RP
// partial sums of o are added in a fixed order through LDS.
//
// Many heads: more waves beat more rows in flight (256 sequences x 16 heads of 128 x 128, 537
// MB: 114 us with 8 rows, 105 with 4, 97 with 2, 5.6 TB/s where a streaming copy reaches 6.5).
// Up to a head a compute unit, and more than 8 rows a thread: four times the threads and twice
// the rows in flight (6 heads of 178 x 225: 19 us became 9.7, 16 of 128 x 128: 7.4 became 5.9; 8 of
// 64 x 64: 4.4 would be 5.4).
template <typename T, int CG, int NT, int U>
__global__ void __launch_bounds__(NT)
lin_step(const LinStep p)
{
    constexpr int RP = NT / CG;
    __shared__ __attribute__((aligned(16))) float red[RP][CG * 4];
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
    for (int half = RP / 2; half > 0; half /= 2) {     // rows half .. 2 half - 1 to those before them
        if (r0 >= half && r0 < 2 * half) *reinterpret_cast<float4 *>(&red[r0][c0]) = float4{o[0], o[1], o[2], o[3]};
        __syncthreads();
        if (r0 < half) {
            const float4 x = *reinterpret_cast<const float4 *>(&red[r0 + half][c0]);
            o[0] += x.x; o[1] += x.y; o[2] += x.z; o[3] += x.w;
        }
    }
    if (r0 == 0 && left > 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= p.scale;
        store_run<T, 4>(op, left, o);
    }
}

template <typename T, int CG> hipError_t run_step_on(const LinStep &p)
{
    const int64_t heads = (int64_t)p.B * p.H;
    if (heads > 256 || p.Dk * CG <= 2048)
        hipLaunchKernelGGL((lin_step<T, CG, 256, 2>), dim3((unsigned)heads), dim3(256), 0, p.stream, p);
    else
        hipLaunchKernelGGL((lin_step<T, CG, 1024, 4>), dim3((unsigned)heads), dim3(1024), 0, p.stream, p);
    return hipGetLastError();
}

template <typename T> hipError_t run_step(const LinStep &p)
{
    if (p.Dv <= 64) return run_step_on<T, 16>(p);
    if (p.Dv <= 128) return run_step_on<T, 32>(p);
    return run_step_on<T, 64>(p);
}

}  // namespace

static int64_t scan_blocks(int64_t heads, int64_t cells) { return heads * ceil_div(cells, kScan * kThreads); }

bool lin_scan_fits(int64_t count, int64_t heads, int64_t cells)
{
    return grid_fits(count * scan_blocks(heads, cells), kThreads);
}

hipError_t launch_lin_scan(const LinWalks &walks)
{
    LinWalks all = walks;
    const LinWalk &p = all.w[0];
    all.blocks = scan_blocks((int64_t)p.B * p.H, (int64_t)p.Da * p.Dc);
    hipLaunchKernelGGL(lin_scan, dim3((unsigned)(all.count * all.blocks)), dim3(kThreads), 0, p.stream, all);
    return hipGetLastError();
}

// One launch for walks that are alike.
static hipError_t run_walks(const LinWalks &all, bool full)
{
    for (int i = 0; i < all.count; ++i) {
        LinWalks some = {};
        bool first = true;
        for (int j = 0; j < all.count; ++j)
            if (lin_alike(all.w[j].Da, all.w[j].Dc, all.w[i].Da, all.w[i].Dc, all.w[0].dtype)) {
                first = first && j >= i;
                some.w[some.count++] = all.w[j];
            }
        if (!first) continue;
        const hipError_t err = all.w[0].dtype == DT_F32   ? run_lin_walks_f32(some, full)
                               : all.w[0].dtype == DT_F16 ? run_lin_walks_f16(some, full)
                                                          : run_lin_walks_bf16(some, full);
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

hipError_t launch_lin_states(const LinWalks &all, int summed, const char **kname)
{
    *kname = "lin_walk";
    LinWalks some = all;
    some.count = summed;
    const hipError_t err = run_walks(some, false);
    return err != hipSuccess || all.w[0].nseg <= kFoldSegs ? err : launch_lin_scan(all);
}

hipError_t launch_lin_walks(const LinWalks &all, const char **kname)
{
    *kname = "lin_walk";
    return run_walks(all, true);
}

template <typename T>
static hipError_t run_group_sum(const float *part, T *out, const int64_t *ost, int64_t B, int64_t T_in, int Hk, int r, int D,
                                hipStream_t stream)
{
    const int blocks = (int)ceil_div((int64_t)Hk * D, kThreads);
    const int64_t most = ((int64_t(1) << 32) - 1) / kThreads / blocks;      // tokens of a launch
    for (int64_t bt0 = 0; bt0 < B * T_in; bt0 += most) {
        hipLaunchKernelGGL((lin_group_sum<T>), dim3((unsigned)(std::min(most, B * T_in - bt0) * blocks)), dim3(kThreads), 0,
                           stream, part, out, ost[0], ost[1], ost[2], (int)T_in, Hk, r, D, blocks, bt0);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
    }
    return hipSuccess;
}

hipError_t launch_lin_group_sum(const float *part, void *out, const int64_t *ost, int64_t B, int64_t T, int Hk, int r,
                                int D, int dtype, hipStream_t stream)
{
    switch (dtype) {
    case DT_F32: return run_group_sum(part, (float *)out, ost, B, T, Hk, r, D, stream);
    case DT_F16: return run_group_sum(part, (_Float16 *)out, ost, B, T, Hk, r, D, stream);
    default: return run_group_sum(part, (__bf16 *)out, ost, B, T, Hk, r, D, stream);
    }
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
