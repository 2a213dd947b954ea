"""Cases of the operators of a recurrent mixing block and of what stands behind the channels-last
convolutions: the gated linear recurrence (prompts, gradients, single tokens), group norm with an
activation over channels-last tensors (gradients too) and the product in 8-bit integers with a scale
for each token and each output channel.

Where `own` is false the operators run in their plain form: elementary torch operations in fp32
(quotients next to a border in fp64), rounded once at the end.  Where it is true the same inputs go
through the package's entry points.  `exact` computes the definitions in fp64, token by token where
the definition is a recurrence.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-5
_AMAX_FLOOR = 2.0 ** -100  # a token of zeros gets this over 127 as its scale


def _gc():
    import depthwise_convolution_gconv_amd as gc
    return gc


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # One user's long document through one recurrence of 4096 channels, x and both gates views of a
        # fused projection; a single sequence gives few independent channels.
        dict(name="rec_long_prompt", op="rec", dtype="bf16", B=1, T=32768, C=4096, state=False, ragged=False, fused=True),
        # A batch of prompts of unequal lengths that continue earlier ones, channels that fill no tile.
        dict(name="rec_ragged_f16", op="rec", dtype="f16", B=6, T=1021, C=1350, state=True, ragged=True, fused=False),
        # Training step of a layer: 4 sequences of 4096 tokens, 2560 channels.
        dict(name="rec_train", op="rec_bwd", dtype="bf16", B=4, T=4096, C=2560, state=False, ragged=False, fused=True),
        # The same at the framework's own sequence shape (8 x 1024 x 512) in fp32, segment after segment.
        dict(name="rec_train_f32", op="rec_bwd", dtype="f32", B=8, T=1024, C=512, state=True, ragged=False, fused=False),
        # A serving batch's next tokens, its states in a pool: the launch is all there is.
        dict(name="rec_tokens", op="rec_step", dtype="bf16", B=64, C=4096, slots=True),
        # Behind the channels-last ensemble layer: its output, 32 groups.
        dict(name="gn_ensemble_f16", op="gn", dtype="f16", N=64, P=784, C=2048, G=32, silu=True, ragged=False),
        # Padded utterances behind the Conformer's depthwise conv1d, statistics over the frames that exist.
        dict(name="gn_utterances_f32", op="gn", dtype="f32", N=8, P=1024, C=512, G=32, silu=True, ragged=True),
        # Training of the subsampling stage's channels-last frames (512 x 40 positions a sample).
        dict(name="gn_frames_train", op="gn_bwd", dtype="bf16", N=8, P=20480, C=256, G=32, silu=True, ragged=False),
        # A serving batch's next tokens, normed over each head of a mixer's output.
        dict(name="gn_heads_tokens", op="gn", dtype="bf16", N=64, P=1, C=4096, G=16, silu=True, ragged=False),
        # A prompt's projection.
        dict(name="int8_prompt", op="int8", dtype="bf16", M=8192, K=4096, N=6144, bias=False),
        # One token's projection: the weights are all there is to read.
        dict(name="int8_token", op="int8", dtype="bf16", M=1, K=4096, N=12288, bias=False),
        # A short prompt, sizes that fill no tile.
        dict(name="int8_ragged_f16", op="int8", dtype="f16", M=333, K=1350, N=4100, bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rec", "rec", "rec_bwd", "rec_bwd", "rec_step", "gn", "gn", "gn_bwd", "gn_bwd", "int8", "int8",
                     "int8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("rec"):
        c = dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256 if op == "rec_step" else 16),
                 C=rng.choice([_log_int(rng, 8, 8192), 64 * _log_int(rng, 1, 128)]))
        if op == "rec_step":
            c["slots"] = rng.random() < 0.5
            return c
        c["T"] = _log_int(rng, 1, 32768 if op == "rec" else 8192)
        c["state"], c["ragged"], c["fused"] = (rng.random() < 0.5 for _ in range(3))
        room = 32768 * 4096 if op == "rec" else 4 * 4096 * 2560      # no more than the largest listed case
        room //= _SIZE[dtype] // 2
        while c["B"] * c["T"] * c["C"] > room:
            c["B" if c["B"] > 1 and rng.random() < 0.5 else "T"] //= 2
        return c
    if op.startswith("gn"):
        G = rng.choice([1, 2, 4, 8, 16, 32, 32, rng.randint(1, 48)])
        P = rng.choice([1, _log_int(rng, 1, 32768)])
        c = dict(op=op, dtype=dtype, N=_log_int(rng, 1, 16384 if P == 1 else 128), P=P,
                 C=G * rng.choice([_log_int(rng, 1, 256), 4 * rng.randint(1, 64)]), G=G, silu=rng.random() < 0.7,
                 ragged=P > 1 and rng.random() < 0.4)
        room = 64 * 784 * 2048 if op == "gn" else 8 * 20480 * 256
        room //= _SIZE[dtype] // 2
        while c["N"] * c["P"] * c["C"] > room:
            c["N" if c["P"] == 1 or (c["N"] > 1 and rng.random() < 0.5) else "P"] //= 2
        return c
    K = rng.choice([_log_int(rng, 16, 16384), 128 * _log_int(rng, 1, 128)])
    N = rng.choice([_log_int(rng, 16, 16384), 128 * _log_int(rng, 1, 128)])
    M = rng.choice([_log_int(rng, 1, 64), _log_int(rng, 1, 16384)])
    while M * N * K > 8192 * 4096 * 6144 or M * max(N, K) > 8192 * 6144:
        M = max(1, M // 2)
    return dict(op=op, dtype=dtype, M=M, K=K, N=N, bias=rng.random() < 0.5)


def work(case):
    c, es = case, _SIZE[case["dtype"]]
    if c["op"] in ("rec", "rec_bwd"):
        n, st = c["B"] * c["T"] * c["C"], 4 * c["B"] * c["C"]
        live = 0.5 if c["ragged"] else 1.0        # of the tokens; all outputs are written
        if c["op"] == "rec":      # x and the gates read, h and the last state written
            return {"bytes": es * n * (3 * live + 1) + st * (2 if c["state"] else 1) + 4 * c["C"], "flops": 12 * n * live}
        # x, gates, h, dh read, three gradients written; with a state: it and its gradient read, its gradient written
        return {"bytes": es * n * (5 * live + 3) + (3 * st if c["state"] else 0) + 8 * c["C"], "flops": 30 * n * live}
    if c["op"] == "rec_step":
        n = c["B"] * c["C"]
        return {"bytes": n * (4 * es + 8) + 4 * c["C"], "flops": 12 * n}
    if c["op"] in ("gn", "gn_bwd"):
        n, st = c["N"] * c["P"] * c["C"], 8 * c["N"] * c["G"]
        live = 0.5 if c["ragged"] else 1.0
        if c["op"] == "gn":
            return {"bytes": es * n * (live + 1) + st + 2 * es * c["C"], "flops": 10 * n * live}
        return {"bytes": es * n * (2 * live + 1) + st + 4 * es * c["C"], "flops": 25 * n * live}
    M, K, N = c["M"], c["K"], c["N"]
    # x read, its 8-bit form and scales written, weights and their scales read, y written
    return {"bytes": M * K * (es + 1) + 4 * M + N * K + 4 * N + M * N * es + (N * es if c["bias"] else 0),
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def rand(*shape, sd=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * sd).to(dtype)

    def lengths(n, top):
        return torch.randint(0, top + 1, (n,), generator=g, device=dev, dtype=torch.int32) if c["ragged"] else None

    c = dict(case)
    s = {"case": c}
    if c["op"].startswith("rec"):
        B, C = c["B"], c["C"]
        # Memories from a few tokens to a few thousand over the channels, at a gate of one half.
        s["log_decay"] = 2.0 * torch.log1p(-(2.0 ** (-1.5 - 10.0 * torch.rand(C, generator=g, device=dev))))
        T = () if c["op"] == "rec_step" else (c["T"],)
        if c.get("fused"):
            s["x"], s["r"], s["i"] = rand(B, *T, 3 * C).split([C, C, C], dim=-1)
        else:
            s["x"], s["r"], s["i"] = rand(B, *T, C), rand(B, *T, C), rand(B, *T, C)
        if c["op"] == "rec_step":
            n = B + 7 if c["slots"] else B
            s["state"] = rand(n, C, dtype=torch.float32)
            s["slots"] = torch.randperm(n, generator=g, device=dev)[:B].to(torch.int32) if c["slots"] else None
            return s
        s["state"] = rand(B, C, dtype=torch.float32) if c["state"] else None
        s["lengths"] = lengths(B, c["T"])
        if c["op"] == "rec_bwd":
            s["h"] = _plain_rec(s)["h"]           # what the forward call returned
            s["dh"] = rand(B, c["T"], C)
            s["dstate"] = rand(B, C, dtype=torch.float32) if c["state"] else None
        return s
    if c["op"].startswith("gn"):
        N, P, C, G = c["N"], c["P"], c["C"], c["G"]
        # Channels of different sizes and offsets.
        size, at = torch.exp(0.5 * rand(C, dtype=torch.float32)), 1.5 * rand(C, dtype=torch.float32)
        s["x"] = (torch.randn(N, P, C, generator=g, device=dev) * size + at).to(dt)
        s["weight"], s["bias"] = (1.0 + 0.1 * rand(C, dtype=torch.float32)).to(dt), rand(C, sd=0.1)
        s["activation"] = "silu" if c["silu"] else None
        s["lengths"] = lengths(N, P)
        if c["op"] == "gn_bwd":
            s["dy"] = rand(N, P, C)
            s["stats"] = _statistics(s["x"].double(), _live(s["lengths"], N, P, dev), G).float()
        return s
    M, K, N = c["M"], c["K"], c["N"]
    # A token's row has a few channels far larger than the others.
    big = 1.0 + 20.0 * (torch.rand(K, generator=g, device=dev) < 0.01).float()
    s["x"] = (torch.randn(M, K, generator=g, device=dev) * big).to(dt)
    w = torch.randn(N, K, generator=g, device=dev) * K ** -0.5
    s["weight_scales"] = w.abs().amax(1) / 127.0
    s["weight"] = torch.round(w / s["weight_scales"][:, None]).clamp(-127, 127).to(torch.int8)
    s["bias"] = rand(N, sd=0.1) if c["bias"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"rec": _plain_rec, "rec_bwd": _plain_rec_bwd, "rec_step": _plain_rec_step, "gn": _plain_gn,
            "gn_bwd": _plain_gn_bwd, "int8": _plain_int8}[op](s)


def _run_own(s, op):
    gc = _gc()
    if op == "rec":
        h, st = gc.gated_recurrence(s["x"], s["r"], s["i"], s["log_decay"], initial_state=s["state"],
                                    lengths=s["lengths"], return_state=True)
        return {"h": h, "state": st}
    if op == "rec_bwd":
        dx, dr, di, dg, ds = gc.gated_recurrence_backward(s["x"], s["r"], s["i"], s["log_decay"], s["h"], s["dh"],
                                                          initial_state=s["state"], lengths=s["lengths"],
                                                          dstate=s["dstate"])
        return {"dx": dx, "dr": dr, "di": di, "dlog_decay": dg, "dstate": ds}
    if op == "rec_step":
        h = gc.gated_recurrence_step(s["x"], s["r"], s["i"], s["log_decay"], s["state"], slots=s["slots"])
        return {"h": h, "state": s["state"]}
    if op == "gn":
        y, stats = gc.group_norm(s["x"], s["case"]["G"], s["weight"], s["bias"], eps=_EPS, activation=s["activation"],
                                 lengths=s["lengths"], return_stats=True)
        return {"y": y, "stats": stats}
    if op == "gn_bwd":
        dx, dw, db = gc.group_norm_backward(s["dy"], s["x"], s["case"]["G"], s["weight"], s["bias"], s["stats"],
                                            activation=s["activation"], lengths=s["lengths"])
        return {"dx": dx, "dw": dw, "db": db}
    q, scales = gc.quantize_int8(s["x"])
    y = gc.matmul_int8(q, scales, s["weight"], s["weight_scales"], bias=s["bias"], dtype=s["x"].dtype)
    return {"q": q, "scales": scales, "y": y}


# ---------------------------------------------------------------- plain forms: gated recurrence

def _live(lengths, B, T, dev):
    """[B, T, 1] truth of the tokens that exist."""
    if lengths is None:
        return torch.ones(1, 1, 1, dtype=torch.bool, device=dev).expand(B, T, 1)
    return (torch.arange(T, device=dev)[None, :] < lengths[:, None])[..., None]


def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _scan(a, u, first):
    """h_t = a_t h_(t-1) + u_t over axis 1 from h_(-1) = first (or zero), all t at once: spans of
    1, 2, 4, ... tokens are joined with the span before them."""
    if first is not None:
        u = torch.cat([u[:, :1] + a[:, :1] * first[:, None], u[:, 1:]], 1)
    d, T = 1, a.shape[1]
    while d < T:
        u = torch.cat([u[:, :d], u[:, d:] + a[:, d:] * u[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return u


def _plain_rec(s):
    x, T = s["x"], s["x"].shape[1]
    live = _live(s["lengths"], x.shape[0], T, x.device)
    la = s["log_decay"] * _sigmoid(s["r"].float())
    a = torch.where(live, torch.exp(la), 1.0)
    u = torch.where(live, torch.sqrt(-torch.expm1(2.0 * la)) * _sigmoid(s["i"].float()) * x.float(), 0.0)
    h = _scan(a, u, s["state"])
    return {"h": torch.where(live, h, 0.0).to(x.dtype), "state": h[:, -1].contiguous()}


def _plain_rec_bwd(s):
    x, (B, T, C) = s["x"].float(), s["x"].shape
    live = _live(s["lengths"], B, T, x.device)
    sr, si = _sigmoid(s["r"].float()), _sigmoid(s["i"].float())
    la = s["log_decay"] * sr
    a, root = torch.exp(la), torch.sqrt(-torch.expm1(2.0 * la))
    before = s["state"] if s["state"] is not None else x.new_zeros(B, C)
    before = torch.cat([before[:, None], s["h"][:, :-1].float()], 1)
    keep = torch.where(live, a, 1.0)
    g = torch.where(live, s["dh"].float(), 0.0)
    # What reaches token t from the tokens behind it: c_t = a_t (g_t + c_(t+1)).
    c = _scan(keep.flip(1), (keep * g).flip(1), s["dstate"]).flip(1)
    last = s["dstate"] if s["dstate"] is not None else x.new_zeros(B, C)
    G = torch.where(live, g + torch.cat([c[:, 1:], last[:, None]], 1), 0.0)
    inner = G * (a * before - torch.where(root > 0, a * a / root, 0.0) * si * x)
    dt = s["x"].dtype
    return {"dx": (G * root * si).to(dt), "dr": (inner * la * (1.0 - sr)).to(dt),
            "di": (G * root * x * si * (1.0 - si)).to(dt), "dlog_decay": (inner * sr).sum(1).sum(0),
            "dstate": c[:, 0].contiguous() if s["state"] is not None else None}


def _plain_rec_step(s):
    la = s["log_decay"] * _sigmoid(s["r"].float())
    old = s["state"] if s["slots"] is None else s["state"][s["slots"].long()]
    new = torch.exp(la) * old + torch.sqrt(-torch.expm1(2.0 * la)) * _sigmoid(s["i"].float()) * s["x"].float()
    if s["slots"] is None:
        s["state"].copy_(new)
    else:
        s["state"][s["slots"].long()] = new
    return {"h": new.to(s["x"].dtype), "state": s["state"]}


# ---------------------------------------------------------------- plain forms: group norm

def _statistics(x, live, G):
    """Mean and 1 / root of the variance of each sample's groups over the positions that exist: [N, G, 2]."""
    N, P, C = x.shape
    n = (live.sum(1).to(x.dtype) * (C // G)).clamp(min=1.0).view(N, 1, 1, 1)
    v, live = x.view(N, P, G, C // G), live[..., None]
    mean = torch.where(live, v, 0.0).sum((1, 3), keepdim=True) / n
    var = torch.where(live, v - mean, 0.0).square().sum((1, 3), keepdim=True) / n
    return torch.stack([mean, torch.rsqrt(var + _EPS)], -1).view(N, G, 2)


def _plain_gn(s):
    x, c = s["x"].float(), s["case"]
    N, P, C = x.shape
    live = _live(s["lengths"], N, P, x.device)
    stats = _statistics(x, live, c["G"])
    mean, rstd = (t.repeat_interleave(C // c["G"], 1)[:, None] for t in stats.unbind(-1))
    z = (x - mean) * rstd * s["weight"].float() + s["bias"].float()
    if c["silu"]:
        z = z * _sigmoid(z)
    return {"y": torch.where(live, z, 0.0).to(s["x"].dtype), "stats": stats}


def _plain_gn_bwd(s):
    x, c = s["x"].float(), s["case"]
    N, P, C = x.shape
    G = c["G"]
    live = _live(s["lengths"], N, P, x.device)
    mean, rstd = (t.repeat_interleave(C // G, 1)[:, None] for t in s["stats"].unbind(-1))
    w, xhat, dz = s["weight"].float(), torch.where(live, (x - mean) * rstd, 0.0), s["dy"].float()
    if c["silu"]:
        z = xhat * w + s["bias"].float()
        sg = _sigmoid(z)
        dz = dz * (sg * (1.0 + z * (1.0 - sg)))
    dz = torch.where(live, dz, 0.0)
    n = (live.sum(1).float() * (C // G)).clamp(min=1.0).view(N, 1, 1)
    over = lambda t: (t.view(N, P, G, C // G).sum((1, 3)) / n[..., 0]).repeat_interleave(C // G, 1)[:, None]  # noqa: E731
    dx = rstd * (w * dz - over(w * dz) - xhat * over(w * dz * xhat))
    dt = s["x"].dtype
    return {"dx": torch.where(live, dx, 0.0).to(dt), "dw": (dz * xhat).sum(1).sum(0).to(dt),
            "db": dz.sum(1).sum(0).to(dt)}


# ---------------------------------------------------------------- plain forms: product in 8-bit integers

def _quantize(x):
    """Every row's largest magnitude becomes 127.  Quotients in fp64 and rounded to fp32, which gives fp32's own
    quotient: the definition rounds that one to a whole number, ties to even."""
    top = x.abs().float().amax(1, keepdim=True).clamp(min=_AMAX_FLOOR).double()
    scale = (top / torch.full_like(top, 127.0)).float()
    return torch.round((x.double() / scale.double()).float()).to(torch.int8), scale


def _plain_int8(s):
    q, scale = _quantize(s["x"])
    y = torch.matmul(q.float(), s["weight"].float().t().contiguous()) * scale * s["weight_scales"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"q": q, "scales": scale, "y": y.to(s["x"].dtype)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"].startswith("rec"):
        return _exact_rec(f, case)
    if case["op"].startswith("gn"):
        return _exact_gn(f, case)
    q, scale = _quantize(s["x"])      # whole numbers, by fp32's own quotient
    y = torch.matmul(q.double(), f["weight"].double().t()) * scale.double() * f["weight_scales"]
    return {"q": q, "scales": f["x"].abs().amax(1, keepdim=True).clamp(min=_AMAX_FLOOR) / 127,
            "y": y if f["bias"] is None else y + f["bias"]}


def _exact_rec(f, case):
    """Token by token; a token that does not exist multiplies by one and adds nothing."""
    x, r, i, g = f["x"], torch.sigmoid(f["r"]), torch.sigmoid(f["i"]), f["log_decay"]
    a = torch.exp(g * r)
    b = torch.sqrt(-torch.expm1(2 * g * r))
    if case["op"] == "rec_step":
        rows = f["slots"].long() if f["slots"] is not None else torch.arange(case["B"], device=x.device)
        new = a * f["state"][rows] + b * i * x
        f["state"][rows] = new
        return {"h": new, "state": f["state"]}
    B, T, C = x.shape
    n = f["lengths"].long() if f["lengths"] is not None else torch.full((B,), T, device=x.device)
    gone = (torch.arange(T, device=x.device)[None] >= n[:, None])[..., None]
    zero = torch.zeros(B, C, dtype=torch.float64, device=x.device)
    keep = a.masked_fill(gone, 1.0)
    if case["op"] == "rec":
        add = (b * i * x).masked_fill(gone, 0.0)
        h = f["state"].clone() if f["state"] is not None else zero
        for t in range(T):
            h = torch.addcmul(add[:, t], keep[:, t], h, out=add[:, t])
        return {"h": add.masked_fill(gone, 0.0), "state": add[:, T - 1].clone()}
    dh, prev = f["dh"].masked_fill(gone, 0.0), torch.empty_like(x)
    prev[:, 0] = f["state"] if f["state"] is not None else zero
    prev[:, 1:] = f["h"][:, :-1]
    c = f["dstate"].clone() if f["dstate"] is not None else zero
    for t in range(T - 1, -1, -1):
        dh[:, t] += c
        c = keep[:, t] * dh[:, t]
    dh.masked_fill_(gone, 0.0)        # the gradient of h_t itself, from its own output and all later ones
    # b^2 = 1 - a^2, so db/da = -a/b
    da = dh * (prev - a / b * i * x)
    dlog = da * a
    return {"dx": dh * b * i, "dr": dlog * g * r * (1 - r), "di": dh * b * x * i * (1 - i),
            "dlog_decay": (dlog * r).sum((0, 1)), "dstate": c if f["state"] is not None else None}


def _exact_gn(f, case):
    """The normed values of a group, their activation and, by the chain rule, their gradients."""
    x, G, (N, P, C) = f["x"], case["G"], f["x"].shape
    n = f["lengths"].double() if f["lengths"] is not None else torch.full((N,), float(P), dtype=torch.float64, device=x.device)
    live = (torch.arange(P, device=x.device)[None] < n[:, None]).double().view(N, P, 1, 1)
    m = (n * (C // G)).clamp(min=1).view(N, 1, 1, 1)
    v = x.reshape(N, P, G, C // G)
    mean = (v * live).sum((1, 3), keepdim=True) / m
    rstd = ((((v - mean) * live) ** 2).sum((1, 3), keepdim=True) / m + _EPS) ** -0.5
    hat = (v - mean) * rstd
    w, b = f["weight"].view(G, C // G), f["bias"].view(G, C // G)
    z = w * hat + b
    sg = torch.sigmoid(z)
    if case["op"] == "gn":
        y = (z * sg if case["silu"] else z) * live
        return {"y": y.reshape(N, P, C), "stats": torch.cat([mean, rstd], 3).reshape(N, G, 2)}
    dz = f["dy"].view_as(v) * live
    if case["silu"]:
        dz = dz * (sg + z * sg * (1 - sg))
    dhat = dz * w
    dx = rstd * (dhat - dhat.sum((1, 3), keepdim=True) / m - hat * (dhat * hat).sum((1, 3), keepdim=True) / m) * live
    return {"dx": dx.reshape(N, P, C), "dw": (dz * hat).sum((0, 1)).reshape(C), "db": dz.sum((0, 1)).reshape(C)}
