"""A layer of a sequence model from the library's sequence operators and plain matrix products:

    h = x + residual -> norm -> projection to (x', z) -> causal convolution -> u -> projections to (delta, B, C)
      -> selective scan over u, gated by z -> projection back

run as it is used: prompts of uneven lengths packed one behind the other, then one token of each sequence at a time from
the carried windows and states, and a training step with every gradient.

    python examples/selective_layer.py [--type bf16] [--channels 512] [--tokens 700]

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
    """C channels in and out, D = 2 C inside, N states, delta of rank R."""

    def __init__(self, C, N=16, R=None, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        D, R = 2 * C, R or max(1, C // 16)

        def matrix(rows, cols):
            return (torch.randn(rows, cols, generator=g, device=device) * rows ** -0.5).to(dtype)

        self.sizes = C, D, N, R
        self.norm_w = torch.ones(C, device=device)
        self.w_in, self.w_x = matrix(C, 2 * D), matrix(D, R + 2 * N)
        self.w_delta, self.w_out = matrix(R, D), matrix(D, C)
        self.conv_w = torch.randn(D, 4, generator=g, device=device) * 0.5
        self.conv_b = torch.zeros(D, device=device)
        self.A = -torch.arange(1, N + 1, device=device).float().repeat(D, 1)
        step = torch.exp(torch.rand(D, generator=g, device=device) * 4.6 - 6.9)       # 1e-3 .. 1e-1
        self.delta_bias = step + torch.log(-torch.expm1(-step))
        self.skip = torch.ones(D, device=device)

    def new_cache(self, sequences):
        """Windows of the convolution and states of the scan, one per sequence, all zero."""
        C, D, N, _ = self.sizes
        return (torch.zeros(sequences, 3, D, dtype=self.w_in.dtype, device=self.A.device),
                torch.zeros(sequences, D, N, device=self.A.device))

    def _scan_inputs(self, u):
        C, D, N, R = self.sizes
        p = u @ self.w_x
        B, Cs = p[..., R:R + N].unsqueeze(-2), p[..., R + N:].unsqueeze(-2)
        return p, p[..., :R] @ self.w_delta, B, Cs

    def _scan_params(self):
        return dict(skip=self.skip, delta_bias=self.delta_bias, softplus=True)

    def prompt(self, x, residual, offsets, cache, max_len=None):
        """Packed prompts [T, C]; the cache is read and brought to the prompts' ends.  Returns (output, h)."""
        D = self.sizes[1]
        y, h, _ = iga.rms_norm(x, self.norm_w, residual=residual)
        proj = y @ self.w_in
        u, _ = iga.causal_conv(proj[:, :D], self.conv_w, self.conv_b, silu=True, offsets=offsets, state=cache[0],
                               state_out=cache[0])
        _, delta, B, C = self._scan_inputs(u)
        s, _, _ = iga.selective_scan(u, delta, self.A, B, C, z=proj[:, D:], offsets=offsets, max_len=max_len,
                                     state=cache[1], state_out=cache[1], **self._scan_params())
        return s @ self.w_out, h

    def step(self, x, residual, cache, slots=None):
        """One token of each sequence [S, C], from the states at `slots` of the cache's pools."""
        D = self.sizes[1]
        y, h, _ = iga.rms_norm(x, self.norm_w, residual=residual)
        proj = y @ self.w_in
        u = iga.causal_conv_step(proj[:, :D], cache[0], self.conv_w, self.conv_b, silu=True, slots=slots)
        _, delta, B, C = self._scan_inputs(u)
        s = iga.selective_scan_step(u, delta, self.A, B, C, cache[1], z=proj[:, D:], slots=slots, **self._scan_params())
        return s @ self.w_out, h

    def forward(self, x, residual):
        """Sequences of one length [S, L, C], keeping what the gradient needs: (output, h, kept)."""
        D = self.sizes[1]
        y, h, r = iga.rms_norm(x, self.norm_w, residual=residual)
        proj = y @ self.w_in
        u, _ = iga.causal_conv(proj[..., :D], self.conv_w, self.conv_b, silu=True)
        p, delta, B, C = self._scan_inputs(u)
        s, _, saved = iga.selective_scan(u, delta, self.A, B, C, z=proj[..., D:], save=True, **self._scan_params())
        return s @ self.w_out, h, (y, r, proj, u, p, delta, B, C, s, saved)

    def backward(self, dout, dh, h, kept):
        """Gradients of x (and of the residual: the same) and of every parameter, from those of the output and of h."""
        C, D, N, R = self.sizes
        y, r, proj, u, p, delta, B, Cs, s, saved = kept

        def outer(a, b):      # the weight gradient a^T b over all tokens
            return a.reshape(-1, a.shape[-1]).T @ b.reshape(-1, b.shape[-1])

        g = iga.selective_scan_grad(dout @ self.w_out.T, u, delta, self.A, B, Cs, saved, z=proj[..., D:], **self._scan_params())
        dp = torch.cat([g.ddelta @ self.w_delta.T, g.dB.squeeze(-2), g.dC.squeeze(-2)], -1)
        dx_conv, dconv_w, dconv_b, _ = iga.causal_conv_grad(g.du + dp @ self.w_x.T, proj[..., :D], self.conv_w,
                                                            self.conv_b, silu=True)
        dproj = torch.cat([dx_conv, g.dz], -1)
        dx, dnorm_w = iga.rms_norm_grad(dproj @ self.w_in.T, h, self.norm_w, r, dh=dh)
        return dx, dict(norm_w=dnorm_w, w_in=outer(y, dproj), conv_w=dconv_w, conv_b=dconv_b, w_x=outer(u, dp),
                        w_delta=outer(p[..., :R], g.ddelta), A=g.dA, delta_bias=g.ddelta_bias, skip=g.dskip,
                        w_out=outer(s, dout))


def steps_against_prompt(layer, lengths, seed=1):
    """Largest difference, over the largest output, between whole prompts and the same prompts whose last four tokens
    come one at a time."""
    C, dtype, dev = layer.sizes[0], layer.w_in.dtype, layer.A.device
    g = torch.Generator(device=dev).manual_seed(seed)
    tail = 4
    x = [torch.randn(n, C, generator=g, device=dev).to(dtype) for n in lengths]
    res = [torch.randn(n, C, generator=g, device=dev).to(dtype) for n in lengths]

    def offsets(ns):
        return torch.tensor([sum(ns[:i]) for i in range(len(ns) + 1)], dtype=torch.int32, device=dev)

    whole, _ = layer.prompt(torch.cat(x), torch.cat(res), offsets(lengths), layer.new_cache(len(lengths)), max(lengths))
    short = [n - tail for n in lengths]
    cache = layer.new_cache(len(lengths))
    layer.prompt(torch.cat([t[:n] for t, n in zip(x, short)]), torch.cat([t[:n] for t, n in zip(res, short)]),
                 offsets(short), cache, max(short))
    ends = torch.tensor([sum(lengths[:i + 1]) - tail for i in range(len(lengths))], device=dev)
    worst = 0.0
    for k in range(tail):
        out, _ = layer.step(torch.stack([t[n + k] for t, n in zip(x, short)]), torch.stack([t[n + k] for t, n in zip(res, short)]),
                            cache)
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
