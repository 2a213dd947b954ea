"""Cases of the sequence-mixing operators: linear attention with a decay for each head
(prompts, gradients, single tokens), RMS norm with the residual's addition (16-bit and
8-bit outputs, gradients) and the causal depthwise conv1d that carries its state
(prompts, gradients, single tokens).

Where `own` is false the operators run in their plain form: elementary torch operations
in fp32 (powers of the decay in fp64), rounded once at the end.  Where it is true the
same inputs go through the package's entry points.  `exact` computes the definitions in
fp64, token by token where the definition is a recurrence.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-6
_E4M3_MAX = 448.0          # largest finite e4m3 value
_AMAX_FLOOR = 2.0 ** -100  # a block of zeros gets this over 448 as its scale


def _gc():
    import depthwise_convolution_gconv_amd as gc
    return gc


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # One user's long document (65536 tokens) through one layer: 16 heads of 128, the
        # views of a fused projection; a single sequence gives few independent heads.
        dict(name="attn_long_prompt", op="attn", dtype="bf16", B=1, T=65536, Hk=16, H=16, Dk=128, Dv=128,
             state=False, ragged=False, fused=True),
        # A batch of prompts of unequal lengths that continue earlier ones, 4 key heads for 12 value
        # heads, sizes that fill no tile.
        dict(name="attn_ragged_f16", op="attn", dtype="f16", B=5, T=1021, Hk=4, H=12, Dk=96, Dv=80,
             state=True, ragged=True, fused=False),
        # Training step of a layer: 4 sequences of 4096 tokens, 16 heads of 128.
        dict(name="attn_train", op="attn_bwd", dtype="bf16", B=4, T=4096, Hk=16, H=16, Dk=128, Dv=128,
             state=False, ragged=False, fused=True),
        # The same at the framework's own sequence shape (8 x 1024 x 512) in fp32.
        dict(name="attn_train_f32", op="attn_bwd", dtype="f32", B=8, T=1024, Hk=8, H=8, Dk=64, Dv=64,
             state=True, ragged=False, fused=False),
        # One user's next token: the launch is all there is.
        dict(name="attn_token", op="attn_step", dtype="bf16", B=1, Hk=8, H=8, Dk=64, Dv=64, slots=False),
        # A serving batch's next tokens, its states in a pool.
        dict(name="attn_tokens_batch", op="attn_step", dtype="bf16", B=256, Hk=16, H=16, Dk=128, Dv=128,
             slots=True),
        # A prompt's residual stream before an 8-bit product: one scale a token.
        dict(name="norm_fp8_prompt", op="norm", dtype="bf16", rows=8192, C=4096, residual=True, out="e4m3",
             block=0),
        # One token's residual stream.
        dict(name="norm_token", op="norm", dtype="bf16", rows=1, C=4096, residual=True, out="same", block=0),
        # Gradients of the norm over a training batch.
        dict(name="norm_train", op="norm_bwd", dtype="bf16", rows=16384, C=2048, residual=True),
        # The short conv over a fused q, k, v projection of two prompts.
        dict(name="conv_prompt", op="conv", dtype="bf16", B=2, T=8192, C=6144, K=4, silu=True, state=True,
             ragged=False),
        # Gradients of the Conformer's depthwise conv in its causal form.
        dict(name="conv_train_f32", op="conv_bwd", dtype="f32", B=8, T=1024, C=512, K=31, silu=True,
             state=False),
        # The short conv for a serving batch's next tokens.
        dict(name="conv_tokens_batch", op="conv_step", dtype="bf16", B=64, C=6144, K=4, silu=True, slots=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn_bwd", "attn_bwd", "attn_step", "norm", "norm", "norm_bwd", "conv",
                     "conv_bwd", "conv_step"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("attn"):
        Hk = rng.randint(1, 16)
        H = Hk * rng.choice([1, 1, 1, 2, 3])
        Dk = rng.choice([rng.randint(8, 256), rng.choice([32, 64, 96, 128, 256])])
        Dv = rng.choice([rng.randint(8, 256), rng.choice([32, 64, 96, 128, 256]), Dk])
        c = dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256 if op == "attn_step" else 16), Hk=Hk, H=H, Dk=Dk, Dv=Dv)
        if op == "attn_step":
            c["slots"] = rng.random() < 0.5
            c["B"] = max(1, min(c["B"], 2 ** 26 // (H * Dk * Dv)))
        else:
            c["T"] = _log_int(rng, 1, 65536 if op == "attn" else 8192)
            c["state"], c["ragged"], c["fused"] = (rng.random() < 0.5 for _ in range(3))
            # No more than the largest listed case of its kind.
            room = 2 ** 20 if op == "attn" else 2 ** 18
            while c["B"] * c["T"] * H * max(Dk, Dv, 64) > 128 * room or c["B"] * c["T"] * H * Dk * Dv > 2 ** 14 * room:
                c["B" if c["B"] > 1 and rng.random() < 0.5 else "T"] //= 2
        return c
    if op.startswith("norm"):
        C = rng.choice([_log_int(rng, 16, 16384), 128 * _log_int(rng, 1, 128)])
        c = dict(op=op, dtype=dtype, rows=min(_log_int(rng, 1, 16384), 2 ** 25 // C), C=C,
                 residual=rng.random() < 0.7)
        if op == "norm":
            c["out"] = rng.choice(["same", "e4m3"])
            c["block"] = rng.choice([0, 64, 128]) if c["out"] == "e4m3" else 0
        return c
    C = rng.choice([_log_int(rng, 8, 8192), 64 * _log_int(rng, 1, 128)])
    c = dict(op=op, dtype=dtype, B=_log_int(rng, 1, 256 if op == "conv_step" else 8), C=C,
             K=rng.choice([2, 3, 4, 4, rng.randint(5, 31)]), silu=rng.random() < 0.7)
    if op == "conv_step":
        c["slots"] = rng.random() < 0.5
    else:
        c["T"] = _log_int(rng, 1, 16384)
        c["state"] = rng.random() < 0.5
        if op == "conv":
            c["ragged"] = rng.random() < 0.5
        room = 2 * 8192 * 6144 if c["K"] <= 4 else 8 * 1024 * 512
        while c["B"] * c["T"] * C > room and c["T"] > 1:
            c["T"] //= 2
    return c


def work(case):
    c, es = case, _SIZE[case["dtype"]]
    if c["op"] in ("attn", "attn_bwd"):
        qk, vo = c["B"] * c["T"] * c["Hk"] * c["Dk"], c["B"] * c["T"] * c["H"] * c["Dv"]
        st, cell = 4 * c["B"] * c["H"] * c["Dk"] * c["Dv"], c["B"] * c["T"] * c["H"] * c["Dk"] * c["Dv"]
        if c["op"] == "attn":   # q, k, v read, o and the final state written
            return {"bytes": es * (2 * qk + 2 * vo) + st * (2 if c["state"] else 1), "flops": 4 * cell}
        # q, k, v, do read, dq, dk, dv written; with a state: it and its gradient read, its gradient written
        return {"bytes": es * (4 * qk + 3 * vo) + (3 * st if c["state"] else 0), "flops": 10 * cell}
    if c["op"] == "attn_step":
        n = c["B"] * c["H"] * c["Dk"] * c["Dv"]
        return {"bytes": 8 * n + es * c["B"] * (2 * c["Hk"] * c["Dk"] + 2 * c["H"] * c["Dv"]), "flops": 4 * n}
    if c["op"] == "norm":
        n = c["rows"] * c["C"]
        blocks = -(-c["C"] // c["block"]) if c["block"] else 1
        out = n * es if c["out"] == "same" else n + 4 * c["rows"] * blocks
        return {"bytes": n * es * (3 if c["residual"] else 1) + c["C"] * es + out, "flops": 5 * n}
    if c["op"] == "norm_bwd":
        n = c["rows"] * c["C"]
        return {"bytes": n * es * (4 if c["residual"] else 3) + 2 * c["C"] * es, "flops": 10 * n}
    if c["op"] == "conv_step":
        n = c["B"] * c["C"]
        return {"bytes": es * (n * (2 + 2 * (c["K"] - 1)) + c["C"] * (c["K"] + 1)), "flops": 2 * n * c["K"]}
    n, st = c["B"] * c["T"] * c["C"], c["B"] * (c["K"] - 1) * c["C"]
    w = c["C"] * (c["K"] + 1)
    if c["op"] == "conv":
        return {"bytes": es * (2 * n + w + st * (2 if c["state"] else 1)), "flops": 2 * n * c["K"]}
    return {"bytes": es * (3 * n + 2 * w + (3 * st if c["state"] else 0)), "flops": 6 * n * c["K"]}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    dt = _DT[case["dtype"]]

    def rand(*shape, sd=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev, dtype=torch.float32) * sd).to(dtype)

    c = dict(case)
    s = {"case": c}
    if c["op"].startswith("attn"):
        B, Hk, H, Dk, Dv = c["B"], c["Hk"], c["H"], c["Dk"], c["Dv"]
        # Memory lengths from a few tokens to a few thousand over the heads, as such layers are set up.
        h = torch.arange(H, device=dev, dtype=torch.float32)
        s["log_decay"] = torch.log1p(-(2.0 ** (-2.0 - 9.0 * (h + torch.rand(H, generator=g, device=dev)) / H)))
        s["scale"] = Dk ** -0.5
        T = () if c["op"] == "attn_step" else (c["T"],)
        if c.get("fused"):
            x = rand(B, *T, 2 * Hk * Dk + H * Dv)
            q, k, v = x.split([Hk * Dk, Hk * Dk, H * Dv], dim=-1)
            s["q"], s["k"], s["v"] = q.unflatten(-1, (Hk, Dk)), k.unflatten(-1, (Hk, Dk)), v.unflatten(-1, (H, Dv))
        else:
            s["q"], s["k"], s["v"] = rand(B, *T, Hk, Dk), rand(B, *T, Hk, Dk), rand(B, *T, H, Dv)
        if c["op"] == "attn_step":
            n = B + 7 if c["slots"] else B
            s["state"] = rand(n, H, Dk, Dv, sd=3.0, dtype=torch.float32)
            s["slots"] = torch.randperm(n, generator=g, device=dev)[:B].to(torch.int32) if c["slots"] else None
        else:
            s["state"] = rand(B, H, Dk, Dv, sd=3.0, dtype=torch.float32) if c["state"] else None
            s["lengths"] = (torch.randint(0, c["T"] + 1, (B,), generator=g, device=dev, dtype=torch.int32)
                            if c["ragged"] else None)
        if c["op"] == "attn_bwd":
            s["do"] = rand(B, c["T"], H, Dv)
            s["dstate"] = rand(B, H, Dk, Dv, dtype=torch.float32) if c["state"] else None
        return s
    if c["op"].startswith("norm"):
        R, C = c["rows"], c["C"]
        # A residual stream has a few channels far larger than the others.
        big = 1.0 + 20.0 * (torch.rand(C, generator=g, device=dev) < 0.01).float()
        s["weight"] = (1.0 + 0.1 * torch.randn(C, generator=g, device=dev)).to(dt)
        s["x"] = rand(R, C)
        if c["op"] == "norm_bwd":
            s["h"] = (torch.randn(R, C, generator=g, device=dev) * big).to(dt)
            s["dy"] = s.pop("x")
            s["dh"] = rand(R, C) if c["residual"] else None
        else:
            s["residual"] = (torch.randn(R, C, generator=g, device=dev) * big).to(dt) if c["residual"] else None
        return s
    B, C, K = c["B"], c["C"], c["K"]
    s["weight"], s["bias"] = rand(C, 1, K, sd=K ** -0.5), rand(C, sd=0.1)
    s["activation"] = "silu" if c["silu"] else None
    if c["op"] == "conv_step":
        n = B + 7 if c["slots"] else B
        s["x"], s["state"] = rand(B, C), rand(n, K - 1, C)
        s["slots"] = torch.randperm(n, generator=g, device=dev)[:B].to(torch.int32) if c["slots"] else None
        return s
    s["x"] = rand(B, c["T"], C)
    s["state"] = rand(B, K - 1, C) if c["state"] else None
    if c["op"] == "conv":
        s["lengths"] = (torch.randint(0, c["T"] + 1, (B,), generator=g, device=dev, dtype=torch.int32)
                        if c["ragged"] else None)
    else:
        s["dy"] = rand(B, c["T"], C)
        s["dstate"] = rand(B, K - 1, C) if c["state"] else None
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"attn": _plain_attn, "attn_bwd": _plain_attn_bwd, "attn_step": _plain_attn_step, "norm": _plain_norm,
            "norm_bwd": _plain_norm_bwd, "conv": _plain_conv, "conv_bwd": _plain_conv_bwd,
            "conv_step": _plain_conv_step}[op](s)


def _run_own(s, op):
    gc = _gc()
    if op == "attn":
        o, st = gc.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], scale=s["scale"],
                                    initial_state=s["state"], lengths=s["lengths"], return_state=True)
        return {"o": o, "state": st}
    if op == "attn_bwd":
        dq, dk, dv, ds = gc.linear_attention_backward(s["q"], s["k"], s["v"], s["log_decay"], s["do"],
                                                      scale=s["scale"], initial_state=s["state"],
                                                      lengths=s["lengths"], dstate=s["dstate"])
        return {"dq": dq, "dk": dk, "dv": dv, "dstate": ds}
    if op == "attn_step":
        o = gc.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], scale=s["scale"],
                                     slots=s["slots"])
        return {"o": o, "state": s["state"]}
    if op == "norm":
        if s["case"]["out"] == "e4m3":
            r = gc.rms_norm_e4m3(s["x"], s["weight"], residual=s["residual"], eps=_EPS, block=s["case"]["block"])
            return dict(zip(("q", "scales", "h"), r))
        r = gc.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=_EPS)
        return dict(zip(("y", "h"), r)) if s["residual"] is not None else {"y": r}
    if op == "norm_bwd":
        dx, dw = gc.rms_norm_backward(s["dy"], s["h"], s["weight"], eps=_EPS, dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "conv":
        y, st = gc.dwconv1d_causal(s["x"], s["weight"], s["bias"], activation=s["activation"],
                                   initial_state=s["state"], lengths=s["lengths"], return_state=True)
        return {"y": y, "state": st}
    if op == "conv_bwd":
        dx, dw, db, ds = gc.dwconv1d_causal_backward(s["x"], s["weight"], s["bias"], s["dy"],
                                                     activation=s["activation"], initial_state=s["state"],
                                                     dstate=s["dstate"])
        return {"dx": dx, "dw": dw, "db": db, "dstate": ds}
    y = gc.dwconv1d_causal_step(s["x"], s["weight"], s["bias"], s["state"], activation=s["activation"],
                                slots=s["slots"])
    return {"y": y, "state": s["state"]}


# ---------------------------------------------------------------- plain forms: linear attention

def _heads(t, H):
    """[B, T, Hk, D] -> fp32 [B, H, T, D], every key head repeated for its value heads."""
    return t.float().repeat_interleave(H // t.shape[2], dim=2).transpose(1, 2).contiguous()


def _back(t, Hk):
    """[B, H, T, D] -> [B, T, Hk, D], the value heads of a key head added."""
    B, H, T, D = t.shape
    return t.view(B, Hk, H // Hk, T, D).sum(2).transpose(1, 2)


def _power(log_decay, e):
    """exp(log_decay * e) in fp64, rounded to fp32: [H] x [...] -> [H, ...]."""
    g = log_decay.double().view(-1, *[1] * e.dim())
    return torch.exp(g * e.double()).float()


def _walk(a, b, c, log_decay):
    """sum over s <= t of lam^(t-s) (a_t . b_s) c_s for [B, H, T, D] operands: within chunks of L
    tokens through their scores, across chunks through the chunks' states."""
    B, H, T, Da = a.shape
    Dc = c.shape[-1]
    L = 256 if T > 4096 else 64
    n = -(-T // L)
    pad = n * L - T
    if pad:
        a, b, c = (torch.nn.functional.pad(t, (0, 0, 0, pad)) for t in (a, b, c))
    a, b, c = (t.reshape(B, H, n, L, -1) for t in (a, b, c))
    i = torch.arange(L, device=a.device)
    d = i[:, None] - i[None, :]
    mask = torch.where(d >= 0, _power(log_decay, d.clamp(min=0)), torch.zeros((), device=a.device))
    out = (torch.matmul(a, b.transpose(-1, -2).contiguous()) * mask[:, None]) @ c
    if n > 1:
        u = torch.matmul((b * _power(log_decay, L - 1 - i)[:, None, :, None]).transpose(-1, -2).contiguous(), c)
        j = torch.arange(n, device=a.device)
        e = j[:, None] - 1 - j[None, :]
        mix = torch.where(e >= 0, _power(log_decay, L * e.clamp(min=0)), torch.zeros((), device=a.device))
        z = torch.matmul(mix, u.reshape(B, H, n, Da * Dc)).view(B, H, n, Da, Dc)
        out = out + torch.matmul(a, z) * _power(log_decay, i + 1)[:, None, :, None]
    return out.reshape(B, H, n * L, Dc)[:, :, :T]


def _live(s, T):
    """[B, 1, T, 1] truth of the tokens that exist, and their number for each sequence."""
    t = torch.arange(T, device=s["q"].device)
    n = s["lengths"] if s["lengths"] is not None else torch.full((s["q"].shape[0],), T, device=t.device)
    return (t[None, :] < n[:, None])[:, None, :, None], n.long()


def _from_end(log_decay, n, T):
    """lam^(n-1-t) for t < n, 0 beyond: [B, H, T, 1]."""
    e = (n[:, None] - 1 - torch.arange(T, device=n.device)[None, :])
    return torch.where(e[:, None] >= 0, _power(log_decay, e.clamp(min=0)).transpose(0, 1),
                       torch.zeros((), device=n.device))[..., None]


def _plain_attn(s):
    T, H = s["q"].shape[1], s["v"].shape[2]
    live, n = _live(s, T)
    q, k, v = _heads(s["q"], H), _heads(s["k"], H), _heads(s["v"], H)
    k, v = torch.where(live, k, 0.0), torch.where(live, v, 0.0)
    o = _walk(q, k, v, s["log_decay"])
    state = torch.matmul((k * _from_end(s["log_decay"], n, T)).transpose(-1, -2).contiguous(), v)
    if s["state"] is not None:
        t = torch.arange(T, device=q.device)
        o = o + torch.matmul(q, s["state"]) * _power(s["log_decay"], t + 1)[None, :, :, None]
        state = state + s["state"] * _power(s["log_decay"], n).transpose(0, 1)[:, :, None, None]
    o = torch.where(live, o * s["scale"], 0.0)
    return {"o": o.transpose(1, 2).to(s["q"].dtype), "state": state}


def _plain_attn_bwd(s):
    T, Hk, H, scale = s["q"].shape[1], s["q"].shape[2], s["v"].shape[2], s["scale"]
    live, n = _live(s, T)
    g = s["log_decay"]
    q, k, v, do = (torch.where(live, _heads(s[x], H), 0.0) for x in ("q", "k", "v", "do"))
    rq, rk, rv, rdo = (t.flip(2) for t in (q, k, v, do))
    dq = _walk(do, v, k, g) * scale
    dk = _walk(rv, rdo, rq, g).flip(2) * scale
    dv = _walk(rk, rq, rdo, g).flip(2) * scale
    ds = None
    if s["state"] is not None:
        t = torch.arange(T, device=q.device)
        ahead = _power(g, t + 1)[None, :, :, None]
        end = _from_end(g, n, T)
        turned = s["dstate"].transpose(-1, -2).contiguous()
        dq = dq + torch.matmul(do, s["state"].transpose(-1, -2).contiguous()) * ahead * scale
        dk = dk + torch.matmul(v, turned) * end
        dv = dv + torch.matmul(k, s["dstate"]) * end
        ds = (torch.matmul((q * ahead).transpose(-1, -2).contiguous(), do) * scale
              + s["dstate"] * _power(g, n).transpose(0, 1)[:, :, None, None])
    dq, dk, dv = (torch.where(live, t, 0.0) for t in (dq, dk, dv))
    dt = s["q"].dtype
    return {"dq": _back(dq, Hk).to(dt), "dk": _back(dk, Hk).to(dt), "dv": dv.transpose(1, 2).to(dt), "dstate": ds}


def _plain_attn_step(s):
    H, r = s["v"].shape[1], s["v"].shape[1] // s["q"].shape[1]
    q, k, v = s["q"].float().repeat_interleave(r, 1), s["k"].float().repeat_interleave(r, 1), s["v"].float()
    lam = torch.exp(s["log_decay"].double()).float().view(1, H, 1, 1)
    old = s["state"] if s["slots"] is None else s["state"][s["slots"].long()]
    new = lam * old + k[..., :, None] * v[..., None, :]
    if s["slots"] is None:
        s["state"].copy_(new)
    else:
        s["state"][s["slots"].long()] = new
    o = torch.matmul(q[..., None, :], new)[..., 0, :] * s["scale"]
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


# ---------------------------------------------------------------- plain forms: RMS norm

def _plain_norm(s):
    c, x = s["case"], s["x"]
    h = x if s["residual"] is None else (x.float() + s["residual"].float()).to(x.dtype)
    hf = h.float()
    y = hf * torch.rsqrt((hf * hf).mean(-1, keepdim=True) + _EPS) * s["weight"].float()
    if c["out"] == "same":
        out = {"y": y.to(x.dtype)}
    else:
        R, C = y.shape
        blk = c["block"] or C
        nb = -(-C // blk)
        yb = torch.nn.functional.pad(y, (0, nb * blk - C)).view(R, nb, blk)
        scale = yb.abs().amax(-1).clamp(min=_AMAX_FLOOR) / _E4M3_MAX
        q = (yb / scale[..., None]).clamp(-_E4M3_MAX, _E4M3_MAX).view(R, nb * blk)[:, :C]
        out = {"q": q.to(torch.float8_e4m3fn), "scales": scale}
    if s["residual"] is not None:
        out["h"] = h
    return out


def _plain_norm_bwd(s):
    h, dy, w = s["h"].float(), s["dy"].float(), s["weight"].float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + _EPS)
    wdy = w * dy
    dx = rstd * (wdy - h * (rstd * rstd * (wdy * h).mean(-1, keepdim=True)))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    dt = s["h"].dtype
    return {"dx": dx.to(dt), "dw": (dy * h * rstd).sum(0).to(dt)}


# ---------------------------------------------------------------- plain forms: causal conv

def _before(s):
    """The inputs with the K-1 that stand before them, fp32 [B, K-1+T, C]."""
    x, K = s["x"].float(), s["weight"].shape[2]
    st = s["state"].float() if s["state"] is not None else x.new_zeros(x.shape[0], K - 1, x.shape[2])
    return torch.cat([st, x], 1)


def _silu(s, z):
    return z / (1.0 + torch.exp(-z)) if s["activation"] == "silu" else z


def _plain_conv(s):
    x, K, T = s["x"], s["weight"].shape[2], s["x"].shape[1]
    xs = _before(s)
    y = _silu(s, (xs.unfold(1, K, 1) * s["weight"][:, 0].float()).sum(-1) + s["bias"].float())
    t = torch.arange(T, device=x.device)
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((x.shape[0],), T, device=x.device)
    y = torch.where((t[None] < n[:, None])[..., None], y, 0.0)
    at = n[:, None] + torch.arange(K - 1, device=x.device)[None]
    state = torch.gather(xs, 1, at[..., None].expand(-1, -1, x.shape[2]))
    return {"y": y.to(x.dtype), "state": state.to(x.dtype)}


def _plain_conv_bwd(s):
    x, K, T, dy = s["x"], s["weight"].shape[2], s["x"].shape[1], s["dy"].float()
    xs, w = _before(s), s["weight"][:, 0].float()
    win = xs.unfold(1, K, 1)
    if s["activation"] == "silu":
        z = (win * w).sum(-1) + s["bias"].float()
        sg = 1.0 / (1.0 + torch.exp(-z))
        dy = dy * (sg * (1.0 + z * (1.0 - sg)))
    dxs = (torch.nn.functional.pad(dy, (0, 0, K - 1, K - 1)).unfold(1, K, 1) * w.flip(1)).sum(-1)
    if s["dstate"] is not None:
        dxs = dxs + torch.nn.functional.pad(s["dstate"].float(), (0, 0, T, 0))
    dt = x.dtype
    return {"dx": dxs[:, K - 1:].to(dt), "dw": (win * dy[..., None]).sum((0, 1)).unsqueeze(1).to(dt),
            "db": dy.sum((0, 1)).to(dt), "dstate": dxs[:, :K - 1].to(dt) if s["state"] is not None else None}


def _plain_conv_step(s):
    old = s["state"] if s["slots"] is None else s["state"][s["slots"].long()]
    xs = torch.cat([old, s["x"][:, None]], 1)
    y = _silu(s, (xs.float() * s["weight"][:, 0].float().t()).sum(1) + s["bias"].float())
    if s["slots"] is None:
        s["state"].copy_(xs[:, 1:])
    else:
        s["state"][s["slots"].long()] = xs[:, 1:]
    return {"y": y.to(s["x"].dtype), "state": s["state"]}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if op in ("attn", "attn_bwd"):
        return _exact_attn(f, op == "attn_bwd")
    if op == "attn_step":
        rows = f["slots"].long() if f["slots"] is not None else torch.arange(case["B"], device=f["q"].device)
        r = case["H"] // case["Hk"]
        k, q = f["k"].repeat_interleave(r, 1), f["q"].repeat_interleave(r, 1)
        new = torch.exp(f["log_decay"])[:, None, None] * f["state"][rows] + k.unsqueeze(3) * f["v"].unsqueeze(2)
        f["state"][rows] = new
        return {"o": case["Dk"] ** -0.5 * (q.unsqueeze(3) * new).sum(2), "state": f["state"]}
    if op == "norm":
        h = f["x"]
        if f["residual"] is not None:
            h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
        y = f["weight"] * h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["C"] + _EPS)
        if case["out"] == "same":
            out = {"y": y}
        else:
            blk = case["block"] or case["C"]
            col = torch.arange(case["C"], device=y.device) // blk
            top = torch.zeros(case["rows"], int(col[-1]) + 1, dtype=torch.float64, device=y.device)
            top = top.scatter_reduce(1, col.expand_as(y), y.abs(), "amax").clamp(min=_AMAX_FLOOR) / _E4M3_MAX
            out = {"q": y / top[:, col], "scales": top}
        return dict(out, h=h) if f["residual"] is not None else out
    if op == "norm_bwd":
        h, dy, w = f["h"], f["dy"], f["weight"]
        inv = 1.0 / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["C"] + _EPS)
        xhat = h * inv
        gx = dy * w
        dx = inv * (gx - xhat * (gx * xhat).sum(1, keepdim=True) / case["C"])
        return {"dx": dx if f["dh"] is None else dx + f["dh"], "dw": (dy * xhat).sum(0)}
    return _exact_conv(f, case)


def _exact_attn(f, backward):
    """Token by token: S <- lam S + k v^T; the sequence that has ended keeps its state."""
    B, T, Hk, Dk = f["q"].shape
    H, Dv, scale = f["v"].shape[2], f["v"].shape[3], Dk ** -0.5
    r, dev = H // Hk, f["q"].device
    lam = torch.exp(f["log_decay"]).view(1, H, 1, 1)
    n = f["lengths"].long() if f["lengths"] is not None else torch.full((B,), T, device=dev)
    live = (torch.arange(T, device=dev)[None] < n[:, None]).double().view(B, T, 1, 1)
    all_live = f["lengths"] is None
    # A token that does not exist multiplies the state by one and adds nothing.
    keep = torch.where(live[..., None] > 0, lam[:, None], torch.ones((), device=dev, dtype=torch.float64))
    q, k = f["q"].repeat_interleave(r, 2), f["k"].repeat_interleave(r, 2) * live
    v = f["v"]
    S = f["state"].clone() if f["state"] is not None else torch.zeros(B, H, Dk, Dv, dtype=torch.float64, device=dev)
    first = (f["do"] if backward else q).contiguous()
    out = torch.empty(B, T, H, Dk if backward else Dv, dtype=torch.float64, device=dev)
    for t in range(T):
        S.mul_(lam if all_live else keep[:, t])
        S.addcmul_(k[:, t].unsqueeze(3), v[:, t].unsqueeze(2))
        if backward:
            out[:, t].copy_(torch.matmul(S, first[:, t].unsqueeze(3)).squeeze(3))
        else:
            out[:, t].copy_(torch.matmul(first[:, t].unsqueeze(2), S).squeeze(2))
    out.mul_(scale).mul_(live)
    if not backward:
        return {"o": out, "state": S}
    do, q = f["do"] * live, q * live
    dk, dv = torch.empty_like(q), torch.empty_like(v)
    Z = f["dstate"].clone() if f["dstate"] is not None else torch.zeros_like(S)
    sq = q * scale
    for t in range(T - 1, -1, -1):
        Z.addcmul_(sq[:, t].unsqueeze(3), do[:, t].unsqueeze(2))
        dk[:, t].copy_(torch.matmul(Z, v[:, t].unsqueeze(3)).squeeze(3))
        dv[:, t].copy_(torch.matmul(k[:, t].unsqueeze(2), Z).squeeze(2))
        Z.mul_(lam if all_live else keep[:, t])
    group = lambda x: x.view(B, T, Hk, r, Dk).sum(3)  # noqa: E731
    return {"dq": group(out), "dk": group(dk * live), "dv": dv * live, "dstate": Z if f["state"] is not None else None}


def _exact_conv(f, case):
    """Tap by tap over the inputs with those before them."""
    w, b, K, x = f["weight"][:, 0], f["bias"], case["K"], f["x"]
    act = (lambda z: z * torch.sigmoid(z)) if case["silu"] else (lambda z: z)
    if case["op"] == "conv_step":
        rows = f["slots"].long() if f["slots"] is not None else torch.arange(case["B"], device=x.device)
        z = b + x * w[:, K - 1]
        for j in range(K - 1):
            z = z + f["state"][rows, j] * w[:, j]
        f["state"][rows] = torch.cat([f["state"][rows][:, 1:], x[:, None]], 1) if K > 1 else f["state"][rows]
        return {"y": act(z), "state": f["state"]}
    B, T, C = x.shape
    st = f["state"] if f["state"] is not None else x.new_zeros(B, K - 1, C)
    xs = torch.cat([st, x], 1)
    z = b.expand(B, T, C).clone()
    for j in range(K):
        z += xs[:, j:j + T] * w[:, j]
    if case["op"] == "conv":
        y = act(z)
        n = f["lengths"].tolist() if f["lengths"] is not None else [T] * B
        for i in range(B):
            y[i, n[i]:] = 0.0
        return {"y": y, "state": torch.stack([xs[i, n[i]:n[i] + K - 1] for i in range(B)])}
    dz = f["dy"]
    if case["silu"]:
        sg = torch.sigmoid(z)
        dz = dz * sg * (1.0 + z * (1.0 - sg))
    dxs, dw = torch.zeros_like(xs), torch.empty_like(w)
    for j in range(K):
        dxs[:, j:j + T] += dz * w[:, j]
        dw[:, j] = (dz * xs[:, j:j + T]).sum((0, 1))
    if f["dstate"] is not None:
        dxs[:, T:] += f["dstate"]
    return {"dx": dxs[:, K - 1:], "dw": dw.unsqueeze(1), "db": dz.sum((0, 1)),
            "dstate": dxs[:, :K - 1] if f["state"] is not None else None}
