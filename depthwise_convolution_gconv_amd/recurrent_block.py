"""One recurrent mixing block out of the package's operators, as a model would use them: RMS norm
with the residual's addition, a projection, the causal depthwise conv1d over the values, the gated
linear recurrence with its two gates, group norm with SiLU over the heads of each token, and the
projection back.

    python -m depthwise_convolution_gconv_amd.recurrent_block

runs prompts of unequal lengths, carries on from them token by token out of pools of states, takes
a training step, and serves the same tokens with the projections in 8-bit integers.
"""
from __future__ import annotations

import torch

from . import _block as ops
from . import _sequence as seq


class RecurrentBlock:
    """Weights of a block of `inner` channels in `heads` heads over a stream of `width` channels."""

    def __init__(self, width: int, inner: int, heads: int, taps: int = 4, dtype=torch.bfloat16, device="cuda", seed: int = 0):
        g = torch.Generator().manual_seed(seed)

        def param(*shape, sd):
            return (torch.randn(*shape, generator=g) * sd).to(device, dtype)

        self.inner, self.heads, self.taps = inner, heads, taps
        self.norm = (1.0 + 0.1 * torch.randn(width, generator=g)).to(device, dtype)
        self.w_in = param(3 * inner, width, sd=width ** -0.5)     # values, recurrence gates, input gates
        self.conv_w, self.conv_b = param(inner, 1, taps, sd=taps ** -0.5), param(inner, sd=0.1)
        # Memories from a few tokens to a few thousand over the channels, at a gate of one half.
        self.log_decay = 2.0 * torch.log1p(-(2.0 ** (-1.5 - 10.0 * torch.rand(inner, generator=g)))).float().to(device)
        self.gn_w = (1.0 + 0.1 * torch.randn(inner, generator=g)).to(device, dtype)
        self.gn_b = param(inner, sd=0.1)
        self.w_out = param(width, inner, sd=inner ** -0.5)
        self.int8 = None

    def quantize(self):
        """From here on prompt() and token() multiply by w_in and w_out in 8-bit integers, with a scale for
        each token and each output channel.  Returns the block."""
        self.int8 = {"w_in": ops.quantize_int8(self.w_in), "w_out": ops.quantize_int8(self.w_out)}
        return self

    def pools(self, n: int):
        """States of n sequences: the conv's last inputs and the recurrence's."""
        dev = self.norm.device
        return (torch.zeros(n, self.taps - 1, self.inner, dtype=self.norm.dtype, device=dev),
                torch.zeros(n, self.inner, dtype=torch.float32, device=dev))

    def _project(self, x, name):
        if self.int8 is None:
            return x @ getattr(self, name).t()
        q, scales = ops.quantize_int8(x)
        return ops.matmul_int8(q, scales, *self.int8[name], dtype=x.dtype)

    def _heads_norm(self, s, alive=None):
        """Group norm of each token over its heads; tokens that do not exist come out as zeros."""
        rows = s.reshape(-1, 1, self.inner)
        return ops.group_norm(rows, self.heads, self.gn_w, self.gn_b, activation="silu", lengths=alive).view(s.shape)

    def prompt(self, x, residual, lengths=None, states=None):
        """x, residual [B, T, width] -> (out, residual for the next block, states)."""
        y, h = seq.rms_norm(x, self.norm, residual=residual)
        v, r, i = self._project(y, "w_in").split(self.inner, dim=-1)
        conv, rec = states if states is not None else (None, None)
        u, conv = seq.dwconv1d_causal(v, self.conv_w, self.conv_b, activation="silu", initial_state=conv, lengths=lengths,
                                      return_state=True)
        s, rec = ops.gated_recurrence(u, r, i, self.log_decay, initial_state=rec, lengths=lengths, return_state=True)
        alive = None
        if lengths is not None:
            alive = (torch.arange(x.shape[1], device=x.device) < lengths[:, None]).to(torch.int32).view(-1)
        return self._project(self._heads_norm(s, alive), "w_out"), h, (conv, rec)

    def token(self, x, residual, pools, slots=None):
        """The next token of each sequence: x, residual [B, width] -> (out, residual); the rows `slots` of
        the pools are updated in place."""
        y, h = seq.rms_norm(x, self.norm, residual=residual)
        v, r, i = self._project(y, "w_in").split(self.inner, dim=-1)
        u = seq.dwconv1d_causal_step(v, self.conv_w, self.conv_b, pools[0], activation="silu", slots=slots)
        s = ops.gated_recurrence_step(u, r, i, self.log_decay, pools[1], slots=slots)
        return self._project(self._heads_norm(s), "w_out"), h

    def forward(self, x, residual):
        """prompt() that keeps what backward() needs: (out, residual, kept)."""
        y, h = seq.rms_norm(x, self.norm, residual=residual)
        p = y @ self.w_in.t()
        v, r, i = p.split(self.inner, dim=-1)
        u = seq.dwconv1d_causal(v, self.conv_w, self.conv_b, activation="silu")
        s = ops.gated_recurrence(u, r, i, self.log_decay)
        n, stats = ops.group_norm(s.view(-1, self.inner), self.heads, self.gn_w, self.gn_b, activation="silu", return_stats=True)
        return n.view(s.shape) @ self.w_out.t(), h, (h, y, p, u, s, n, stats)

    def backward(self, dout, dh, kept):
        """Gradients of x (and residual alike) and of the weights from those of forward()'s outputs."""
        h, y, p, u, s, n, stats = kept
        flat = lambda t: t.reshape(-1, t.shape[-1])  # noqa: E731
        v, r, i = p.split(self.inner, dim=-1)
        ds, dgn_w, dgn_b = ops.group_norm_backward(flat(dout) @ self.w_out, flat(s), self.heads, self.gn_w, self.gn_b, stats,
                                                   activation="silu")
        du, dr, di, dlog, _ = ops.gated_recurrence_backward(u, r, i, self.log_decay, s, ds.view(s.shape))
        dv, dconv_w, dconv_b, _ = seq.dwconv1d_causal_backward(v, self.conv_w, self.conv_b, du, activation="silu")
        dp = torch.cat([dv, dr, di], dim=-1)
        dx, dnorm = seq.rms_norm_backward(dp @ self.w_in, h, self.norm, dh=dh)
        return dx, {"norm": dnorm, "w_in": flat(dp).t() @ flat(y), "conv_w": dconv_w, "conv_b": dconv_b, "log_decay": dlog,
                    "gn_w": dgn_w, "gn_b": dgn_b, "w_out": flat(dout).t() @ n}


def main() -> None:
    block = RecurrentBlock(512, 640, 10)
    g = torch.Generator().manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=g).to("cuda", torch.bfloat16)  # noqa: E731

    B, T = 3, 200
    x, r = draw(B, T + 1, 512), draw(B, T + 1, 512)
    lengths = torch.tensor([200, 57, 0], dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")

    def serve():
        _, _, states = block.prompt(x[:, :T].contiguous(), r[:, :T].contiguous(), lengths)
        pools = block.pools(8)
        for pool, state in zip(pools, states):
            pool[slots.long()] = state
        out, _ = block.token(x[:, T], r[:, T], pools, slots)
        whole, _, _ = block.prompt(x[:1], r[:1])
        return out, whole[0, T]

    out, whole = serve()
    print("a token after a prompt of 200:", tuple(out.shape), "off the same token inside a prompt of 201 by",
          f"{float((out[0] - whole).abs().max()):.4f}")
    y, h, kept = block.forward(x, r)
    dx, grads = block.backward(y, h, kept)       # the loss (|out|^2 + |h|^2) / 2
    print("gradients:", "x", tuple(dx.shape), *(f"{n} {tuple(t.shape)}" for n, t in grads.items()))
    block.quantize()
    out8, _ = serve()
    print("in 8-bit integers: off by", f"{float((out8 - out).float().norm() / out.float().norm()):.4f}", "of the 2-norm")


if __name__ == "__main__":
    main()
