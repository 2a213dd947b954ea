// seq_api.cpp -- C entry points of the sequence operators (linear attention, RMS norm,
// causal depthwise conv1d): validation, plans and launches.  Host code only.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>

#include "gconv.h"
#include "linattn.hpp"
#include "seq.hpp"

namespace {

gconv_status_t fail(gconv_status_t s, const char *fmt, ...)
{
    char text[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    gconv::set_last_error(text);
    return s;
}

gconv_status_t done(hipError_t err, const char *kname)
{
    if (err != hipSuccess) return fail(GCONV_ERR_LAUNCH, "kernel launch failed: HIP error %d", (int)err);
    gconv::set_last_kernel(kname);
    return GCONV_OK;
}

bool bad_dtype(gconv_dtype_t d) { return d != GCONV_F32 && d != GCONV_F16 && d != GCONV_BF16; }
size_t elem(gconv_dtype_t d) { return d == GCONV_F32 ? 4 : 2; }

// Memory a call reads or writes.
struct Range {
    const char *name;
    const void *p;
    size_t bytes;
    bool out;
};

gconv_status_t check_ranges(const Range *r, int n)
{
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (i == j || !r[i].out || !r[i].p || !r[j].p || !r[i].bytes || !r[j].bytes) continue;
            const uintptr_t a = (uintptr_t)r[i].p, b = (uintptr_t)r[j].p;
            if (a < b + r[j].bytes && b < a + r[i].bytes)
                return fail(GCONV_ERR_INVALID_ARG, "%s overlaps %s", r[i].name, r[j].name);
        }
    return GCONV_OK;
}

// Bytes from the first to past the last element of a strided [n0][n1][n2][len] view.
size_t extent(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t len, size_t es)
{
    if (n0 == 0 || n1 == 0 || n2 == 0 || len == 0) return 0;
    return es * (size_t)((n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + len);
}

constexpr int64_t kMax = (int64_t(1) << 31) - 1;
constexpr double kCells = 4.0e18;   // element offsets stay in int64

// ---------------------------------------------------------------- linear attention

struct LinShape {
    int64_t B, T, Hk, H, Dk, Dv;
};

gconv_status_t lin_shape(const int64_t *shape, LinShape *s)
{
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    *s = LinShape{shape[0], shape[1], shape[2], shape[3], shape[4], shape[5]};
    if (s->B < 0 || s->T < 0 || s->Hk < 1 || s->H < 1 || s->Dk < 1 || s->Dv < 1)
        return fail(GCONV_ERR_INVALID_ARG, "linear attention: B, T >= 0 and Hk, H, Dk, Dv >= 1 are needed");
    if (s->H % s->Hk != 0)
        return fail(GCONV_ERR_SHAPE, "linear attention: %lld value heads are no multiple of %lld key heads",
                    (long long)s->H, (long long)s->Hk);
    if (s->Dk > 256 || s->Dv > 256)
        return fail(GCONV_ERR_UNSUPPORTED, "linear attention: Dk = %lld, Dv = %lld, at most 256 columns a head",
                    (long long)s->Dk, (long long)s->Dv);
    if (s->B > kMax || s->T > kMax - 4096 || s->H > 65536 || (double)s->B * s->H >= 1 << 24 ||
        (double)s->B * s->T * s->H * 256.0 >= kCells)
        return fail(GCONV_ERR_UNSUPPORTED, "linear attention: sizes exceed the library's index range");
    return GCONV_OK;
}

gconv_status_t check_strides(const int64_t *strides, int n)
{
    if (!strides) return fail(GCONV_ERR_INVALID_ARG, "NULL strides");
    for (int i = 0; i < n; ++i)
        if (strides[i] < 0) return fail(GCONV_ERR_INVALID_ARG, "stride %d is negative", i);
    return GCONV_OK;
}

// Segments of a sequence: as many workgroups as the 256 compute units hold at once of the
// outputs' kernel, counted for each launch of a call, while a segment keeps at least 2 chunks of
// 64 tokens (a cut sequence reads two of its three inputs again, and every segment sets up its
// tables and reads a state).  16 heads over 32768 tokens with as many workgroups as are held, and
// with a half more or less: fp16, 64 x 64 (1024): 138 us, 178 with 1536, 161 with 768; fp16, 64 x
// 128 (512): 236, 259 with 768, 321 with 256; fp32, 64 x 128 (512): 351, 396, 431; fp32, 128 x 64
// (512): 384, 455, 639; fp32, 64 x 64 (768): 230, 260 with 1024, 293 with 512; bf16, 128 x 128
// (768): 233, 272 with 1024, 238 with 512; bf16, 64 x 64 (1536): 107, 96 with 1024, 105 with 768.
// At least 64, 128 and 192 tokens in a segment: 16 heads of 128 over 2048 tokens in bf16 48, 44
// and 63 us, 8 heads of 64 over 1024, gradients, 31, 29 and 36; 12 heads of 96 x 80 over 5 x 1021
// in fp16 70, 68 and 68; few heads over few tokens gain from 64 (4 heads of 128 over 2 x 700: 32,
// 38 and 44 us).
constexpr int64_t kChunk = 64;

int64_t lin_slots(int64_t Da, int64_t Dc, gconv_dtype_t dtype)
{
    return 256 * (dtype == GCONV_F32   ? gconv::lin_held_f32(Da, Dc)
                  : dtype == GCONV_F16 ? gconv::lin_held_f16(Da, Dc)
                                       : gconv::lin_held_bf16(Da, Dc));
}

void lin_segments(const LinShape &s, bool backward, gconv_dtype_t dtype, int32_t *nseg, int32_t *seg_len)
{
    const int64_t chunks = std::max<int64_t>(1, gconv::ceil_div(s.T, kChunk)), heads = std::max<int64_t>(1, s.B * s.H);
    auto fit = [&](int64_t walks, int64_t Da, int64_t Dc) {
        return lin_slots(Da, Dc, dtype) / (walks * heads * gconv::lin_tiles(Da, Dc, (int)dtype));
    };
    // The output; or dv, and dq and dk, in one launch where they can be.
    int64_t n = !backward                                      ? fit(1, s.Dk, s.Dv)
                : gconv::lin_alike(s.Dk, s.Dv, s.Dv, s.Dk, (int)dtype) ? fit(3, s.Dk, s.Dv)
                                                               : std::min(fit(1, s.Dk, s.Dv), fit(2, s.Dv, s.Dk));
    n = std::max<int64_t>(1, std::min<int64_t>({n, chunks / 2, gconv::kMaxSeg}));
    const int64_t each = gconv::ceil_div(chunks, n);
    *nseg = (int32_t)gconv::ceil_div(chunks, each);
    *seg_len = (int32_t)(each * kChunk);
}

// Every launch of a call, before the first is made.  (The local states' launches are no larger
// than the outputs', and the sum over value heads goes in pieces.)
gconv_status_t lin_grids(const LinShape &s, bool backward, gconv_dtype_t dtype)
{
    int32_t nseg, len;
    lin_segments(s, backward, dtype, &nseg, &len);
    auto walks = [&](int64_t count, int64_t Da, int64_t Dc) {
        const int64_t blocks = count * s.B * s.H * nseg * gconv::lin_tiles(Da, Dc, (int)dtype);
        return gconv::grid_fits(8 * gconv::ceil_div(blocks, 8), 64 * gconv::lin_waves(Da, Dc, (int)dtype));
    };
    const bool alike = gconv::lin_alike(s.Dk, s.Dv, s.Dv, s.Dk, (int)dtype);
    const bool fits = s.T == 0   ? gconv::lin_scan_fits(1, s.B * s.H, s.Dk * s.Dv)
                      : !backward ? walks(1, s.Dk, s.Dv)
                      : alike     ? walks(3, s.Dk, s.Dv)
                                  : walks(1, s.Dk, s.Dv) && walks(2, s.Dv, s.Dk);
    if (!fits || (nseg > gconv::kFoldSegs && !gconv::lin_scan_fits(backward ? 3 : 1, s.B * s.H, s.Dk * s.Dv)))
        return fail(GCONV_ERR_UNSUPPORTED, "linear attention: %lld heads need more threads than a launch takes",
                    (long long)(s.B * s.H));
    return GCONV_OK;
}

// One set of segment states.
size_t lin_states_bytes(const LinShape &s, bool backward, gconv_dtype_t dtype)
{
    int32_t nseg, len;
    lin_segments(s, backward, dtype, &nseg, &len);
    return nseg > 1 ? sizeof(float) * (size_t)(s.B * s.H * nseg * s.Dk * s.Dv) : 0;
}

size_t lin_part_bytes(const LinShape &s)
{
    return s.H > s.Hk ? sizeof(float) * (size_t)(s.B * s.T * s.H * s.Dk) : 0;
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t lin_workspace(const LinShape &s, bool backward, gconv_dtype_t dtype)
{
    const size_t states = align256(lin_states_bytes(s, backward, dtype));
    return backward ? 3 * states + 2 * align256(lin_part_bytes(s)) : states;
}

// What every pass over these heads shares.
gconv::LinWalk lin_base(const LinShape &s, bool backward, const float *log_decay, const int32_t *lengths,
                        gconv_dtype_t dtype, void *stream)
{
    gconv::LinWalk p = {};
    p.B = (int32_t)s.B; p.T = (int32_t)s.T; p.H = (int32_t)s.H; p.rep = (int32_t)(s.H / s.Hk);
    p.log_decay = log_decay;
    p.lengths = lengths;
    p.dtype = (int)dtype;
    p.stream = (hipStream_t)stream;
    lin_segments(s, backward, dtype, &p.nseg, &p.seg_len);
    return p;
}

struct View {   // a [B][T][heads][D] tensor
    const void *p;
    const int64_t *st;
    int64_t heads;
    int64_t D;
};
void set_a(gconv::LinWalk &p, const View &v)
{
    p.a = v.p; p.asb = v.st[0]; p.ast = v.st[1]; p.ash = v.st[2];
    p.ra = (int32_t)(p.H / v.heads); p.Da = (int32_t)v.D;
}
void set_b(gconv::LinWalk &p, const View &v)
{
    p.b = v.p; p.bsb = v.st[0]; p.bst = v.st[1]; p.bsh = v.st[2];
    p.rb = (int32_t)(p.H / v.heads);
}
void set_c(gconv::LinWalk &p, const View &v)
{
    p.c = v.p; p.csb = v.st[0]; p.cst = v.st[1]; p.csh = v.st[2];
    p.rc = (int32_t)(p.H / v.heads); p.Dc = (int32_t)v.D;
}
// States as fp32 [B][H][Dk][Dv], read by row and column or transposed.
void set_s0(gconv::LinWalk &p, const float *s0, const LinShape &s, bool turned)
{
    p.s0 = s0;
    p.s0b = s.H * s.Dk * s.Dv; p.s0h = s.Dk * s.Dv;
    p.s0r = turned ? 1 : s.Dv; p.s0c = turned ? s.Dv : 1;
}
void set_sf(gconv::LinWalk &p, float *sf, const LinShape &s)
{
    p.sf = sf;
    p.sfb = s.H * s.Dk * s.Dv; p.sfh = s.Dk * s.Dv;
    p.sfr = s.Dv; p.sfc = 1;
}

gconv_status_t check_workspace(const void *ws, size_t have, size_t need)
{
    if (need > 0 && !ws) return fail(GCONV_ERR_INVALID_ARG, "NULL workspace");
    if (((uintptr_t)ws & 15) != 0) return fail(GCONV_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    if (have < need) return fail(GCONV_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", have, need);
    return GCONV_OK;
}

}  // namespace

extern "C" {

gconv_status_t gconv_linear_attention_workspace(const int64_t *shape, gconv_dtype_t dtype, int32_t backward,
                                                size_t *bytes)
{
    gconv::set_last_error("");
    if (!bytes) return fail(GCONV_ERR_INVALID_ARG, "NULL bytes");
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    LinShape s;
    gconv_status_t st = lin_shape(shape, &s);
    if (st != GCONV_OK || (st = lin_grids(s, backward != 0, dtype)) != GCONV_OK) return st;
    *bytes = lin_workspace(s, backward != 0, dtype);
    return GCONV_OK;
}

gconv_status_t gconv_linear_attention(const void *q, const void *k, const void *v, void *o, const int64_t *shape,
                                      const int64_t *strides, const float *log_decay, float scale,
                                      const float *initial_state, float *final_state, const int32_t *lengths,
                                      gconv_dtype_t dtype, void *workspace, size_t workspace_bytes, void *hip_stream)
{
    gconv::set_last_error("");
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    LinShape s;
    gconv_status_t st = lin_shape(shape, &s);
    if (st != GCONV_OK || (st = check_strides(strides, 12)) != GCONV_OK ||
        (st = lin_grids(s, false, dtype)) != GCONV_OK)
        return st;
    if (!log_decay) return fail(GCONV_ERR_INVALID_ARG, "NULL log_decay");
    if (s.B > 0 && s.T > 0 && (!q || !k || !v || !o)) return fail(GCONV_ERR_INVALID_ARG, "NULL q, k, v or o");
    const size_t need = lin_workspace(s, false, dtype), es = elem(dtype), ns = 4 * (size_t)(s.B * s.H * s.Dk * s.Dv);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GCONV_OK) return st;
    const Range r[] = {
        {"o", o, extent(s.B, strides[9], s.T, strides[10], s.H, strides[11], s.Dv, es), true},
        {"final_state", final_state, ns, true},
        {"workspace", workspace, need, true},
        {"q", q, extent(s.B, strides[0], s.T, strides[1], s.Hk, strides[2], s.Dk, es), false},
        {"k", k, extent(s.B, strides[3], s.T, strides[4], s.Hk, strides[5], s.Dk, es), false},
        {"v", v, extent(s.B, strides[6], s.T, strides[7], s.H, strides[8], s.Dv, es), false},
        {"initial_state", initial_state, ns, false},
        {"log_decay", log_decay, 4 * (size_t)s.H, false},
        {"lengths", lengths, 4 * (size_t)s.B, false},
    };
    if ((st = check_ranges(r, sizeof(r) / sizeof(r[0]))) != GCONV_OK) return st;
    if (s.B == 0) return done(hipSuccess, "");
    gconv::LinWalks all = {};
    all.count = 1;
    gconv::LinWalk &p = all.w[0];
    p = lin_base(s, false, log_decay, lengths, dtype, hip_stream);
    set_a(p, View{q, strides, s.Hk, s.Dk});
    set_b(p, View{k, strides + 3, s.Hk, s.Dk});
    set_c(p, View{v, strides + 6, s.H, s.Dv});
    p.out = o; p.osb = strides[9]; p.ost = strides[10]; p.osh = strides[11];
    set_s0(p, initial_state, s, false);
    set_sf(p, final_state, s);
    p.ws = (float *)workspace;
    p.p_scale = p.inter_scale = scale;
    p.upd_scale = 1.0f;
    p.e0 = 1;
    const char *kname = "lin_scan";
    if (s.T == 0) {   // no token: the state stays
        if (!final_state) return done(hipSuccess, "");
        p.nseg = 0;
        return done(gconv::launch_lin_scan(all), kname);
    }
    hipError_t err = hipSuccess;
    if (p.nseg > 1) err = gconv::launch_lin_states(all, 1, &kname);
    if (err == hipSuccess) err = gconv::launch_lin_walks(all, &kname);
    return done(err, kname);
}

gconv_status_t gconv_linear_attention_backward(const void *q, const void *k, const void *v, const void *d_o,
                                               void *dq, void *dk, void *dv, const int64_t *shape,
                                               const int64_t *strides, const float *log_decay, float scale,
                                               const float *initial_state, const float *dfinal, float *dinitial,
                                               const int32_t *lengths, gconv_dtype_t dtype, void *workspace,
                                               size_t workspace_bytes, void *hip_stream)
{
    gconv::set_last_error("");
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    LinShape s;
    gconv_status_t st = lin_shape(shape, &s);
    if (st != GCONV_OK || (st = check_strides(strides, 21)) != GCONV_OK ||
        (st = lin_grids(s, true, dtype)) != GCONV_OK)
        return st;
    if (!log_decay) return fail(GCONV_ERR_INVALID_ARG, "NULL log_decay");
    if (s.B > 0 && s.T > 0 && (!q || !k || !v || !d_o || !dq || !dk || !dv))
        return fail(GCONV_ERR_INVALID_ARG, "NULL q, k, v, d_o, dq, dk or dv");
    const size_t need = lin_workspace(s, true, dtype), es = elem(dtype), ns = 4 * (size_t)(s.B * s.H * s.Dk * s.Dv);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GCONV_OK) return st;
    auto ext = [&](int i, int64_t heads, int64_t D) {
        return extent(s.B, strides[3 * i], s.T, strides[3 * i + 1], heads, strides[3 * i + 2], D, es);
    };
    const Range r[] = {
        {"dq", dq, ext(4, s.Hk, s.Dk), true},    {"dk", dk, ext(5, s.Hk, s.Dk), true},
        {"dv", dv, ext(6, s.H, s.Dv), true},     {"dinitial", dinitial, ns, true},
        {"workspace", workspace, need, true},    {"q", q, ext(0, s.Hk, s.Dk), false},
        {"k", k, ext(1, s.Hk, s.Dk), false},     {"v", v, ext(2, s.H, s.Dv), false},
        {"d_o", d_o, ext(3, s.H, s.Dv), false},  {"initial_state", initial_state, ns, false},
        {"dfinal", dfinal, ns, false},           {"log_decay", log_decay, 4 * (size_t)s.H, false},
        {"lengths", lengths, 4 * (size_t)s.B, false},
    };
    if ((st = check_ranges(r, sizeof(r) / sizeof(r[0]))) != GCONV_OK) return st;
    if (s.B == 0) return done(hipSuccess, "");
    const View vq{q, strides, s.Hk, s.Dk}, vk{k, strides + 3, s.Hk, s.Dk}, vv{v, strides + 6, s.H, s.Dv},
        vdo{d_o, strides + 9, s.H, s.Dv};
    const int32_t rep = (int32_t)(s.H / s.Hk);
    const size_t nstates = align256(lin_states_bytes(s, true, dtype)), npart = align256(lin_part_bytes(s));
    float *ahead = (float *)workspace, *behind = (float *)((char *)workspace + nstates),
          *turned = (float *)((char *)workspace + 2 * nstates);
    char *part = (char *)workspace + 3 * nstates;
    const char *kname = "lin_scan";
    const gconv::LinWalk base = lin_base(s, true, log_decay, lengths, dtype, hip_stream);
    gconv::LinWalks all = {};
    all.count = 3;
    gconv::LinWalk &pv = all.w[0], &pq = all.w[1], &pk = all.w[2];

    // Gradients of later tokens: states of q do^T from the end, for dv and transposed for dk; their value before the first token is the initial state's gradient.
    pv = base;
    set_a(pv, vk);
    set_b(pv, vq);
    set_c(pv, vdo);
    set_s0(pv, dfinal, s, false);
    set_sf(pv, dinitial, s);
    pv.ws = behind;
    pv.wst = turned;
    pv.p_scale = pv.upd_scale = scale;
    pv.inter_scale = 1.0f;
    pv.e0 = 0;
    pv.reverse = 1;
    if (s.T == 0) {
        if (!dinitial) return done(hipSuccess, "");
        pv.nseg = 0;
        all.count = 1;
        return done(gconv::launch_lin_scan(all), kname);
    }
    pv.out = dv; pv.osb = strides[18]; pv.ost = strides[19]; pv.osh = strides[20];

    // Gradient of q: the forward states, transposed.
    pq = base;
    set_a(pq, vdo);
    set_b(pq, vv);
    set_c(pq, vk);
    set_s0(pq, initial_state, s, true);
    pq.ws = ahead;
    pq.p_scale = pq.inter_scale = scale;
    pq.upd_scale = 1.0f;
    pq.e0 = 1;

    pk = pv;
    set_a(pk, vv);
    set_b(pk, vdo);
    set_c(pk, vq);
    set_s0(pk, dfinal, s, true);
    pk.sf = nullptr;
    pk.ws = turned;
    pk.wst = nullptr;

    // A key head that serves several value heads: each writes its share in fp32, then the
    // shares are added and rounded once.
    auto key_grad = [&](gconv::LinWalk &w, void *out, const int64_t *st, float *shares) {
        w.out = out; w.osb = st[0]; w.ost = st[1]; w.osh = st[2];
        if (rep == 1) return;
        w.out = shares;
        w.osb = s.T * s.H * s.Dk; w.ost = s.H * s.Dk; w.osh = s.Dk;
        w.out_f32 = 1;
    };
    key_grad(pq, dq, strides + 12, (float *)part);
    key_grad(pk, dk, strides + 15, (float *)(part + npart));
    hipError_t err = hipSuccess;
    if (base.nseg > 1) err = gconv::launch_lin_states(all, 2, &kname);
    if (err == hipSuccess) err = gconv::launch_lin_walks(all, &kname);
    if (rep > 1) {
        auto sum = [&](const void *shares, void *out, const int64_t *st) {
            if (err == hipSuccess)
                err = gconv::launch_lin_group_sum((const float *)shares, out, st, s.B, s.T, (int)s.Hk, rep, (int)s.Dk,
                                                  (int)dtype, base.stream);
        };
        sum(part, dq, strides + 12);
        sum(part + npart, dk, strides + 15);
    }
    return done(err, kname);
}

gconv_status_t gconv_linear_attention_step(const void *q, const void *k, const void *v, void *o, float *state,
                                           const int64_t *shape, const int64_t *strides, const float *log_decay,
                                           float scale, const int32_t *slots, gconv_dtype_t dtype, void *hip_stream)
{
    gconv::set_last_error("");
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    const int64_t full[6] = {shape[0], 1, shape[1], shape[2], shape[3], shape[4]}, n = shape[5];
    LinShape s;
    gconv_status_t st = lin_shape(full, &s);
    if (st != GCONV_OK || (st = check_strides(strides, 8)) != GCONV_OK) return st;
    if (n < 0) return fail(GCONV_ERR_INVALID_ARG, "linear attention step: n >= 0 states are needed");
    if (!slots && n < s.B)
        return fail(GCONV_ERR_SHAPE, "linear attention step: %lld states for %lld sequences without slots",
                    (long long)n, (long long)s.B);
    if ((double)n * s.H * s.Dk * s.Dv >= kCells || s.B * s.H > kMax)
        return fail(GCONV_ERR_UNSUPPORTED, "linear attention step: sizes exceed the library's index range");
    if (!log_decay) return fail(GCONV_ERR_INVALID_ARG, "NULL log_decay");
    if (s.B == 0) return done(hipSuccess, "");
    if (!q || !k || !v || !o || (!state && n > 0)) return fail(GCONV_ERR_INVALID_ARG, "NULL q, k, v, o or state");
    const size_t es = elem(dtype);
    const Range r[] = {
        {"o", o, extent(s.B, strides[6], 1, 0, s.H, strides[7], s.Dv, es), true},
        {"state", state, 4 * (size_t)(n * s.H * s.Dk * s.Dv), true},
        {"q", q, extent(s.B, strides[0], 1, 0, s.Hk, strides[1], s.Dk, es), false},
        {"k", k, extent(s.B, strides[2], 1, 0, s.Hk, strides[3], s.Dk, es), false},
        {"v", v, extent(s.B, strides[4], 1, 0, s.H, strides[5], s.Dv, es), false},
        {"log_decay", log_decay, 4 * (size_t)s.H, false},
        {"slots", slots, 4 * (size_t)s.B, false},
    };
    if ((st = check_ranges(r, sizeof(r) / sizeof(r[0]))) != GCONV_OK) return st;
    gconv::LinStep p = {};
    p.q = q; p.k = k; p.v = v; p.o = o; p.state = state; p.log_decay = log_decay; p.slots = slots;
    p.qsb = strides[0]; p.qsh = strides[1]; p.ksb = strides[2]; p.ksh = strides[3];
    p.vsb = strides[4]; p.vsh = strides[5]; p.osb = strides[6]; p.osh = strides[7];
    p.n = n; p.B = (int32_t)s.B; p.Hk = (int32_t)s.Hk; p.H = (int32_t)s.H; p.Dk = (int32_t)s.Dk; p.Dv = (int32_t)s.Dv;
    p.scale = scale; p.dtype = (int)dtype; p.stream = (hipStream_t)hip_stream;
    const char *kname = "";
    const hipError_t err = gconv::launch_lin_step(p, &kname);
    return done(err, kname);
}

// ---------------------------------------------------------------- RMS norm

static gconv_status_t norm_check(int64_t rows, int64_t C, const int64_t *strides, int ns, float eps, gconv_dtype_t dtype)
{
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (rows < 0 || C < 1) return fail(GCONV_ERR_INVALID_ARG, "RMS norm: rows >= 0 and C >= 1 are needed");
    if (!(eps >= 0.0f)) return fail(GCONV_ERR_INVALID_ARG, "RMS norm: eps must be >= 0");
    if (C > int64_t(1) << 24 || rows > gconv::kNormMaxRows)
        return fail(GCONV_ERR_UNSUPPORTED, "RMS norm: at most 2^24 columns and 2^31 - 1 rows");
    return ns ? check_strides(strides, ns) : GCONV_OK;
}

static gconv_status_t norm_run(const void *x, const void *residual, const void *weight, void *y, float *scales, void *h,
                               int64_t rows, int64_t C, const int64_t *strides, float eps, int32_t block,
                               gconv_dtype_t dtype, void *hip_stream, bool e4m3)
{
    gconv::set_last_error("");
    gconv_status_t st = norm_check(rows, C, strides, 2, eps, dtype);
    if (st != GCONV_OK) return st;
    if (e4m3 && block != 0 && block != 32 && block != 64 && block != 128 && block != 256)
        return fail(GCONV_ERR_UNSUPPORTED, "RMS norm: %d columns a scale (0, 32, 64, 128 or 256 are run)", (int)block);
    if (!weight) return fail(GCONV_ERR_INVALID_ARG, "NULL weight");
    if (rows == 0) return done(hipSuccess, "");
    if (!x || !y || (e4m3 && !scales)) return fail(GCONV_ERR_INVALID_ARG, "NULL x, output or scales");
    if ((residual != nullptr) != (h != nullptr))
        return fail(GCONV_ERR_INVALID_ARG, "RMS norm: the h output goes with a residual");
    const size_t es = elem(dtype), n = (size_t)(rows * C);
    const Range r[] = {
        {e4m3 ? "q" : "y", y, n * (e4m3 ? 1 : es), true},
        {"scales", scales, e4m3 ? 4 * (size_t)(rows * (block ? gconv::ceil_div(C, block) : 1)) : 0, true},
        {"h", h, n * es, true},
        {"x", x, extent(rows, strides[0], 1, 0, 1, 0, C, es), false},
        {"residual", residual, extent(rows, strides[1], 1, 0, 1, 0, C, es), false},
        {"weight", weight, es * (size_t)C, false},
    };
    if ((st = check_ranges(r, sizeof(r) / sizeof(r[0]))) != GCONV_OK) return st;
    gconv::RmsArgs a = {};
    a.x = x; a.residual = residual; a.weight = weight; a.y = y; a.h = h; a.scales = e4m3 ? scales : nullptr;
    a.rows = rows; a.C = C; a.xs = strides[0]; a.rs = strides[1]; a.block = block; a.eps = eps;
    a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    const char *kname = "";
    const hipError_t err = gconv::launch_rms_norm(a, &kname);
    return done(err, kname);
}

gconv_status_t gconv_rms_norm(const void *x, const void *residual, const void *weight, void *y, void *h, int64_t rows,
                              int64_t C, const int64_t *strides, float eps, gconv_dtype_t dtype, void *hip_stream)
{
    return norm_run(x, residual, weight, y, nullptr, h, rows, C, strides, eps, 0, dtype, hip_stream, false);
}

gconv_status_t gconv_rms_norm_e4m3(const void *x, const void *residual, const void *weight, void *q, float *scales,
                                   void *h, int64_t rows, int64_t C, const int64_t *strides, float eps, int32_t block,
                                   gconv_dtype_t dtype, void *hip_stream)
{
    return norm_run(x, residual, weight, q, scales, h, rows, C, strides, eps, block, dtype, hip_stream, true);
}

gconv_status_t gconv_rms_norm_backward_workspace(int64_t rows, int64_t C, gconv_dtype_t dtype, size_t *bytes)
{
    gconv::set_last_error("");
    if (!bytes) return fail(GCONV_ERR_INVALID_ARG, "NULL bytes");
    const gconv_status_t st = norm_check(rows, C, nullptr, 0, 0.0f, dtype);
    if (st != GCONV_OK) return st;
    *bytes = gconv::rms_bwd_workspace(rows, C, (int)dtype);
    return GCONV_OK;
}

gconv_status_t gconv_rms_norm_backward(const void *dy, const void *h, const void *weight, const void *dh, void *dx,
                                       void *dw, int64_t rows, int64_t C, const int64_t *strides, float eps,
                                       gconv_dtype_t dtype, void *workspace, size_t workspace_bytes, void *hip_stream)
{
    gconv::set_last_error("");
    gconv_status_t st = norm_check(rows, C, strides, 3, eps, dtype);
    if (st != GCONV_OK) return st;
    const size_t need = gconv::rms_bwd_workspace(rows, C, (int)dtype), es = elem(dtype);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GCONV_OK) return st;
    if (!weight || !dw) return fail(GCONV_ERR_INVALID_ARG, "NULL weight or dw");
    if (rows > 0 && (!dy || !h || !dx)) return fail(GCONV_ERR_INVALID_ARG, "NULL dy, h or dx");
    const Range r[] = {
        {"dx", dx, es * (size_t)(rows * C), true},
        {"dw", dw, es * (size_t)C, true},
        {"workspace", workspace, need, true},
        {"dy", dy, extent(rows, strides[0], 1, 0, 1, 0, C, es), false},
        {"h", h, extent(rows, strides[1], 1, 0, 1, 0, C, es), false},
        {"dh", dh, extent(rows, strides[2], 1, 0, 1, 0, C, es), false},
        {"weight", weight, es * (size_t)C, false},
    };
    if ((st = check_ranges(r, sizeof(r) / sizeof(r[0]))) != GCONV_OK) return st;
    gconv::RmsBwdArgs a = {};
    a.dy = dy; a.h = h; a.weight = weight; a.dh = dh; a.dx = dx; a.dw = dw; a.ws = (float *)workspace;
    a.rows = rows; a.C = C; a.dys = strides[0]; a.hs = strides[1]; a.dhs = strides[2]; a.eps = eps;
    a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    const char *kname = "";
    const hipError_t err = gconv::launch_rms_norm_bwd(a, &kname);
    return done(err, kname);
}

// ---------------------------------------------------------------- causal depthwise conv1d

static const char kTooManyThreads[] = "causal conv1d: the call needs more threads than a launch takes";

static gconv_status_t causal_shape(int64_t B, int64_t T, int64_t C, int64_t K, gconv_act_t act, gconv_dtype_t dtype)
{
    if (bad_dtype(dtype)) return fail(GCONV_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (act != GCONV_ACT_NONE && act != GCONV_ACT_SILU)
        return fail(GCONV_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    if (B < 0 || T < 0 || C < 1 || K < 1)
        return fail(GCONV_ERR_INVALID_ARG, "causal conv1d: B, T >= 0 and C, K >= 1 are needed");
    if (K > gconv::kCausalMaxK)
        return fail(GCONV_ERR_UNSUPPORTED, "causal conv1d: %lld taps, at most %d are run", (long long)K,
                    gconv::kCausalMaxK);
    if (B > kMax || T > kMax - 4096 || C > kMax / 64 || (double)B * (double)(T + K) * (double)C >= kCells)
        return fail(GCONV_ERR_UNSUPPORTED, "causal conv1d: sizes exceed the library's index range");
    return GCONV_OK;
}

gconv_status_t gconv_dw1d_causal(const void *x, const void *w, const void *bias, void *y, const void *initial_state,
                                 void *final_state, const int32_t *lengths, const int64_t *shape,
                                 const int64_t *strides, gconv_act_t activation, gconv_dtype_t dtype, void *hip_stream)
{
    gconv::set_last_error("");
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    const int64_t B = shape[0], T = shape[1], C = shape[2], K = shape[3];
    gconv_status_t st = causal_shape(B, T, C, K, activation, dtype);
    if (st != GCONV_OK || (st = check_strides(strides, 2)) != GCONV_OK) return st;
    if (!w) return fail(GCONV_ERR_INVALID_ARG, "NULL w");
    if (B > 0 && T > 0 && (!x || !y)) return fail(GCONV_ERR_INVALID_ARG, "NULL x or y");
    const size_t es = elem(dtype), ns = es * (size_t)(B * (K - 1) * C);
    const Range r[] = {
        {"y", y, es * (size_t)(B * T * C), true},
        {"final_state", final_state, ns, true},
        {"x", x, extent(B, strides[0], T, strides[1], 1, 0, C, es), false},
        {"w", w, es * (size_t)(C * K), false},
        {"bias", bias, es * (size_t)C, false},
        {"initial_state", initial_state, ns, false},
        {"lengths", lengths, 4 * (size_t)B, false},
    };
    if ((st = check_ranges(r, sizeof(r) / sizeof(r[0]))) != GCONV_OK) return st;
    if (B == 0 || (T == 0 && (!final_state || K == 1))) return done(hipSuccess, "");
    gconv::CausalArgs a = {};
    a.x = x; a.w = w; a.bias = bias; a.y = y; a.s0 = initial_state; a.sf = K > 1 ? final_state : nullptr;
    a.lengths = lengths;
    a.B = B; a.T = T; a.C = C; a.K = K; a.xsb = strides[0]; a.xst = strides[1];
    a.silu = activation == GCONV_ACT_SILU;
    a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    if (!gconv::causal_fits(a)) return fail(GCONV_ERR_UNSUPPORTED, kTooManyThreads);
    const char *kname = "";
    const hipError_t err = gconv::launch_causal(a, &kname);
    return done(err, kname);
}

gconv_status_t gconv_dw1d_causal_backward_workspace(const int64_t *shape, gconv_dtype_t dtype, size_t *bytes)
{
    gconv::set_last_error("");
    if (!shape || !bytes) return fail(GCONV_ERR_INVALID_ARG, "NULL shape or bytes");
    const gconv_status_t st = causal_shape(shape[0], shape[1], shape[2], shape[3], GCONV_ACT_NONE, dtype);
    if (st != GCONV_OK) return st;
    *bytes = gconv::causal_bwd_workspace(shape[0], shape[1], shape[2], shape[3]);
    return GCONV_OK;
}

gconv_status_t gconv_dw1d_causal_backward(const void *x, const void *w, const void *bias, const void *dy,
                                          const void *initial_state, const void *dfinal, void *dx, void *dw, void *db,
                                          void *dinitial, const int32_t *lengths, const int64_t *shape,
                                          const int64_t *strides, gconv_act_t activation, gconv_dtype_t dtype,
                                          void *workspace, size_t workspace_bytes, void *hip_stream)
{
    gconv::set_last_error("");
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    const int64_t B = shape[0], T = shape[1], C = shape[2], K = shape[3];
    gconv_status_t st = causal_shape(B, T, C, K, activation, dtype);
    if (st != GCONV_OK || (st = check_strides(strides, 4)) != GCONV_OK) return st;
    const size_t need = gconv::causal_bwd_workspace(B, T, C, K), es = elem(dtype), ns = es * (size_t)(B * (K - 1) * C);
    if ((st = check_workspace(workspace, workspace_bytes, need)) != GCONV_OK) return st;
    if (!w || !dw) return fail(GCONV_ERR_INVALID_ARG, "NULL w or dw");
    if (B > 0 && T > 0 && (!x || !dy || !dx)) return fail(GCONV_ERR_INVALID_ARG, "NULL x, dy or dx");
    if (dinitial && !initial_state && ns > 0)
        return fail(GCONV_ERR_INVALID_ARG, "causal conv1d: dinitial goes with an initial state");
    const Range r[] = {
        {"dx", dx, es * (size_t)(B * T * C), true},
        {"dw", dw, es * (size_t)(C * K), true},
        {"db", db, es * (size_t)C, true},
        {"dinitial", dinitial, ns, true},
        {"workspace", workspace, need, true},
        {"x", x, extent(B, strides[0], T, strides[1], 1, 0, C, es), false},
        {"dy", dy, extent(B, strides[2], T, strides[3], 1, 0, C, es), false},
        {"w", w, es * (size_t)(C * K), false},
        {"bias", bias, es * (size_t)C, false},
        {"initial_state", initial_state, ns, false},
        {"dfinal", dfinal, ns, false},
        {"lengths", lengths, 4 * (size_t)B, false},
    };
    if ((st = check_ranges(r, sizeof(r) / sizeof(r[0]))) != GCONV_OK) return st;
    gconv::CausalArgs a = {};
    a.x = x; a.w = w; a.bias = bias; a.dy = dy; a.s0 = K > 1 ? initial_state : nullptr; a.dsf = K > 1 ? dfinal : nullptr;
    a.dx = dx; a.dw = dw; a.db = db; a.ds0 = K > 1 ? dinitial : nullptr; a.ws = (float *)workspace; a.lengths = lengths;
    a.B = B; a.T = T; a.C = C; a.K = K; a.xsb = strides[0]; a.xst = strides[1]; a.dysb = strides[2]; a.dyst = strides[3];
    a.silu = activation == GCONV_ACT_SILU;
    a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    if (!gconv::causal_bwd_fits(a)) return fail(GCONV_ERR_UNSUPPORTED, kTooManyThreads);
    const char *kname = "";
    const hipError_t err = gconv::launch_causal_bwd(a, &kname);
    return done(err, kname);
}

gconv_status_t gconv_dw1d_causal_step(const void *x, const void *w, const void *bias, void *state, void *y,
                                      const int32_t *slots, const int64_t *shape, int64_t x_stride,
                                      gconv_act_t activation, gconv_dtype_t dtype, void *hip_stream)
{
    gconv::set_last_error("");
    if (!shape) return fail(GCONV_ERR_INVALID_ARG, "NULL shape");
    const int64_t B = shape[0], C = shape[1], K = shape[2], n = shape[3];
    gconv_status_t st = causal_shape(B, 1, C, K, activation, dtype);
    if (st != GCONV_OK || (st = check_strides(&x_stride, 1)) != GCONV_OK) return st;
    if (n < 0) return fail(GCONV_ERR_INVALID_ARG, "causal conv1d step: n >= 0 states are needed");
    if (!slots && n < B)
        return fail(GCONV_ERR_SHAPE, "causal conv1d step: %lld states for %lld sequences without slots", (long long)n,
                    (long long)B);
    if ((double)n * K * C >= kCells)
        return fail(GCONV_ERR_UNSUPPORTED, "causal conv1d step: sizes exceed the library's index range");
    if (!w) return fail(GCONV_ERR_INVALID_ARG, "NULL w");
    if (B == 0) return done(hipSuccess, "");
    if (!x || !y || (!state && n > 0 && K > 1)) return fail(GCONV_ERR_INVALID_ARG, "NULL x, y or state");
    const size_t es = elem(dtype);
    const Range r[] = {
        {"y", y, es * (size_t)(B * C), true},
        {"state", state, es * (size_t)(n * (K - 1) * C), true},
        {"x", x, extent(B, x_stride, 1, 0, 1, 0, C, es), false},
        {"w", w, es * (size_t)(C * K), false},
        {"bias", bias, es * (size_t)C, false},
        {"slots", slots, 4 * (size_t)B, false},
    };
    if ((st = check_ranges(r, sizeof(r) / sizeof(r[0]))) != GCONV_OK) return st;
    gconv::CausalStepArgs a = {};
    a.x = x; a.w = w; a.bias = bias; a.y = y; a.state = state; a.slots = slots;
    a.B = B; a.C = C; a.K = K; a.n = n; a.xsb = x_stride; a.silu = activation == GCONV_ACT_SILU;
    a.dtype = (int)dtype; a.stream = (hipStream_t)hip_stream;
    if (!gconv::causal_step_fits(a)) return fail(GCONV_ERR_UNSUPPORTED, kTooManyThreads);
    const char *kname = "";
    const hipError_t err = gconv::launch_causal_step(a, &kname);
    return done(err, kname);
}

}  // extern "C"
