"""A layer of a sequence model from the library's layer norm, causal convolution and gated delta rule, and plain matrix
products:

    h = x + residual -> layer norm -> projection to (q, k), v and the gates -> causal convolutions -> q, k to unit length
      -> gated delta rule -> layer norm of each head -> projection back

run as it is used: prompts of uneven lengths packed one behind the other, then one token of each sequence at a time from
the carried windows and states, and a training step with every gradient.

    python examples/delta_layer.py [--type bf16] [--channels 512] [--tokens 700]

prints how far the token-by-token outputs are from those of the whole prompts, a gradient's directional derivative
beside a difference of two losses, and the times.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import implicit_gemm_amd as iga  # noqa: E402


class Layer:
    """C channels in and out, Hk key heads of Dk, H value heads of Dv that share them."""

    def __init__(self, C, Hk=2, H=4, Dk=64, Dv=64, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def matrix(rows, cols):
            return (torch.randn(rows, cols, generator=g, device=device) * rows ** -0.5).to(dtype)

        def vector(n, start=0.0):
            return start + 0.1 * torch.randn(n, generator=g, device=device)

        K, V = 2 * Hk * Dk, H * Dv
        self.sizes = C, Hk, H, Dk, Dv
        self.parts = [K, V, H, H]                        # of the projection: q and k, v, decay, beta
        self.norm_w, self.norm_b = vector(C, 1.0), vector(C)
        self.w_in, self.w_out = matrix(C, K + V + 2 * H), matrix(V, C)
        self.conv_qk = torch.randn(K, 4, generator=g, device=device) * 0.5
        self.conv_v = torch.randn(V, 4, generator=g, device=device) * 0.5
        self.unit = torch.full((Dk,), Dk ** -0.5, device=device)              # a norm to length 1
        self.A = 1 + 15 * torch.rand(H, generator=g, device=device)
        step = torch.exp(torch.rand(H, generator=g, device=device) * 4.6 - 6.9)        # 1e-3 .. 1e-1
        self.bias = step + torch.log(-torch.expm1(-step))
        self.head_w, self.head_b = vector(Dv, 1.0), vector(Dv)

    def new_cache(self, sequences):
        """Windows of the two convolutions and states of the delta rule, one per sequence, all zero."""
        C, Hk, H, Dk, Dv = self.sizes
        dtype, dev = self.w_in.dtype, self.A.device
        return (torch.zeros(sequences, 3, self.parts[0], dtype=dtype, device=dev),
                torch.zeros(sequences, 3, self.parts[1], dtype=dtype, device=dev),
                torch.zeros(sequences, H, Dk, Dv, device=dev))

    def _inputs(self, u, w, a, b):
        """(keys and queries, their norm's r, q, k, v, g, beta) from the convolutions' outputs and the gates."""
        C, Hk, H, Dk, Dv = self.sizes
        n, qk, r = iga.rms_norm(u.unflatten(-1, (2 * Hk, Dk)), self.unit, eps=1e-6)
        g = -self.A * torch.nn.functional.softplus(a.float() + self.bias)
        return qk, r, n[..., :Hk, :], n[..., Hk:, :], w.unflatten(-1, (H, Dv)), g, torch.sigmoid(b.float())

    def _out(self, o):
        """(output, the heads' norm and its statistics)"""
        z, _, m, r = iga.layer_norm(o, self.head_w, self.head_b)
        return z.flatten(-2) @ self.w_out, z, m, r

    def prompt(self, x, residual, offsets, cache):
        """Packed prompts [T, C]; the cache is read and brought to the prompts' ends.  Returns (output, h)."""
        y, h, _, _ = iga.layer_norm(x, self.norm_w, self.norm_b, residual=residual)
        pk, pv, a, b = (y @ self.w_in).split(self.parts, -1)
        u, _ = iga.causal_conv(pk, self.conv_qk, silu=True, offsets=offsets, state=cache[0], state_out=cache[0])
        w, _ = iga.causal_conv(pv, self.conv_v, silu=True, offsets=offsets, state=cache[1], state_out=cache[1])
        _, _, q, k, v, g, beta = self._inputs(u, w, a, b)
        o, _, _ = iga.gated_delta(q, k, v, g, beta, offsets=offsets, state=cache[2], state_out=cache[2])
        return self._out(o)[0], h

    def step(self, x, residual, cache, slots=None):
        """One token of each sequence [S, C], from the states at `slots` of the cache's pools."""
        y, h, _, _ = iga.layer_norm(x, self.norm_w, self.norm_b, residual=residual)
        pk, pv, a, b = (y @ self.w_in).split(self.parts, -1)
        u = iga.causal_conv_step(pk, cache[0], self.conv_qk, silu=True, slots=slots)
        w = iga.causal_conv_step(pv, cache[1], self.conv_v, silu=True, slots=slots)
        _, _, q, k, v, g, beta = self._inputs(u, w, a, b)
        return self._out(iga.gated_delta_step(q, k, v, g, beta, cache[2], slots=slots))[0], h

    def forward(self, x, residual):
        """Sequences of one length [S, L, C], keeping what the gradient needs: (output, h, kept)."""
        y, h, m, r = iga.layer_norm(x, self.norm_w, self.norm_b, residual=residual)
        p = (y @ self.w_in).split(self.parts, -1)
        u, _ = iga.causal_conv(p[0], self.conv_qk, silu=True)
        w, _ = iga.causal_conv(p[1], self.conv_v, silu=True)
        inputs = self._inputs(u, w, *p[2:])
        o, _, saved = iga.gated_delta(*inputs[2:], save=True)
        out, *head = self._out(o)
        return out, h, (y, m, r, p, inputs, o, saved, head)

    def backward(self, dout, dh, h, kept):
        """Gradients of x (and of the residual: the same) and of every parameter, from those of the output and of h."""
        C, Hk, H, Dk, Dv = self.sizes
        y, m, r, p, (qk, rq, q, k, v, g, beta), o, saved, (z, mo, ro) = kept

        def outer(a, b):      # the weight gradient a^T b over all tokens
            return a.reshape(-1, a.shape[-1]).T @ b.reshape(-1, b.shape[-1])

        dz = (dout @ self.w_out.T).unflatten(-1, (H, Dv))
        do, dhead_w, dhead_b = iga.layer_norm_grad(dz, o, self.head_w, mo, ro)
        d = iga.gated_delta_grad(do, q, k, v, g, beta, saved)
        dqk, _ = iga.rms_norm_grad(torch.cat([d.dq, d.dk], -2), qk, self.unit, rq)
        dpk, dconv_qk, _, _ = iga.causal_conv_grad(dqk.flatten(-2), p[0], self.conv_qk, silu=True)
        dpv, dconv_v, _, _ = iga.causal_conv_grad(d.dv.flatten(-2), p[1], self.conv_v, silu=True)
        da = -d.dg * self.A * torch.sigmoid(p[2].float() + self.bias)
        db = d.dbeta * beta * (1 - beta)
        dp = torch.cat([dpk, dpv, da.to(dpk.dtype), db.to(dpk.dtype)], -1)
        dx, dnorm_w, dnorm_b = iga.layer_norm_grad(dp @ self.w_in.T, h, self.norm_w, m, r, dh=dh)
        tokens = tuple(range(g.dim() - 1))
        return dx, dict(norm_w=dnorm_w, norm_b=dnorm_b, w_in=outer(y, dp), conv_qk=dconv_qk, conv_v=dconv_v,
                        A=(d.dg * g / self.A).sum(tokens), bias=da.sum(tokens), head_w=dhead_w, head_b=dhead_b,
                        w_out=outer(z.flatten(-2), dout))


def steps_against_prompt(layer, lengths, seed=1):
    """Largest difference, over the largest output, between whole prompts and the same prompts whose last four tokens
    come one at a time, the states at places of a pool that are not the sequences' own order."""
    C, dtype, dev = layer.sizes[0], layer.w_in.dtype, layer.A.device
    g = torch.Generator(device=dev).manual_seed(seed)
    tail, S = 4, len(lengths)
    x = [torch.randn(n, C, generator=g, device=dev).to(dtype) for n in lengths]
    res = [torch.randn(n, C, generator=g, device=dev).to(dtype) for n in lengths]

    def offsets(ns):
        return torch.tensor([sum(ns[:i]) for i in range(len(ns) + 1)], dtype=torch.int32, device=dev)

    whole, _ = layer.prompt(torch.cat(x), torch.cat(res), offsets(lengths), layer.new_cache(S))
    short = [n - tail for n in lengths]
    cache = layer.new_cache(S)
    layer.prompt(torch.cat([t[:n] for t, n in zip(x, short)]), torch.cat([t[:n] for t, n in zip(res, short)]),
                 offsets(short), cache)
    slots = torch.arange(S - 1, -1, -1, dtype=torch.int32, device=dev)
    cache = tuple(t.flip(0).contiguous() for t in cache)
    ends = torch.tensor([sum(lengths[:i + 1]) - tail for i in range(S)], device=dev)
    worst = 0.0
    for k in range(tail):
        out, _ = layer.step(torch.stack([t[n + k] for t, n in zip(x, short)]), torch.stack([t[n + k] for t, n in zip(res, short)]),
                            cache, slots)
        worst = max(worst, float((out.float() - whole[ends + k].float()).abs().max()))
    return worst / float(whole.float().abs().max())


def gradient_against_difference(C=64, S=2, L=90, seed=2):
    """(directional derivative from the gradients, central difference) of a loss of a float32 layer along a random
    direction of every parameter and of the input."""
    layer = Layer(C, dtype=torch.float32, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    x, res, dout, dh = (rand(S, L, C) for _ in range(4))
    out, h, kept = layer.forward(x, res)
    dx, grads = layer.backward(dout, dh, h, kept)
    names = sorted(grads)
    start = {n: getattr(layer, n) for n in names}
    along = {n: rand(*start[n].shape) * start[n].abs().mean().clamp(min=0.1) for n in names}
    along_x = rand(S, L, C)
    slope = float(sum((grads[n].double() * along[n].double()).sum() for n in names) + (dx.double() * along_x.double()).sum())

    def loss(e):
        for n in names:
            setattr(layer, n, start[n] + e * along[n])
        out, h, _ = layer.forward(x + e * along_x, res)
        return float((out.double() * dout.double()).sum() + (h.double() * dh.double()).sum())

    e = 1e-3
    return slope, (loss(e) - loss(-e)) / (2 * e)


def timed(f, n=20):
    for _ in range(3):
        f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n * 1e3


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--type", choices=("f32", "bf16", "f16"), default="bf16")
    ap.add_argument("--channels", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=700, help="of the longest prompt")
    a = ap.parse_args()
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[a.type]
    layer = Layer(a.channels, dtype=dtype)
    lengths = [a.tokens, max(5, a.tokens // 3), 5, max(5, a.tokens // 2)]
    print("tokens one at a time against whole prompts: %.2e of the largest output" % steps_against_prompt(layer, lengths))
    print("directional derivative %.4f, difference of losses %.4f" % gradient_against_difference())
    x = torch.randn(4, a.tokens, a.channels, device="cuda").to(dtype)
    res, dout = torch.randn_like(x), torch.randn_like(x)

    def train():
        out, h, kept = layer.forward(x, res)
        layer.backward(dout, dout, h, kept)

    cache, token = layer.new_cache(64), torch.randn(64, a.channels, device="cuda").to(dtype)
    print("training step of %d x %d tokens: %.0f us; one token of each of 64 sequences: %.0f us" % (
        4, a.tokens, timed(train), timed(lambda: layer.step(token, token, cache))))


if __name__ == "__main__":
    main()
