"""Measured cases of the sequence operators: the root-mean-square norm, the short causal convolution and the
selective state space scan, each for prompts, for training (forward and gradients) and for single tokens.

The operators' formulas (32-bit arithmetic whatever the element type, one rounding per output):

  norm   h = x + residual (rounded to the element type: the next layer reads it), r = 1 / sqrt(mean(h^2) + eps),
         y = h r w; in 8 bits per group of channels: scale = max|y| / 448, q = e4m3(y / scale).
         dh = r (dy w - h r^2 mean(dy w h)) + dh_next, dw = sum over rows of dy h r.
  conv   p[t, d] = bias[d] + sum_k w[d, k] x[t - (W - 1) + k, d] within a sequence (before its first token: the carried
         state), y = p sigmoid(p).
  scan   D[t, d] = softplus(delta + bias), h[t] = exp(D A) h[t - 1] + D u B[t], y = (sum_n h C[t] + skip u) z sigmoid(z).

`own` selects the framework's calls; the plain form is elementary torch arithmetic.
"""
import math

import torch

own = False
EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
WIDTH = 4            # taps of the convolution cases


def listed():
    return [
        # Serving: the norm in front of an 8-bit projection for one token of each of a few requests (latency only).
        {"name": "norm_token_e4m3", "op": "norm", "mode": "e4m3", "type": "bf16", "rows": 16, "C": 2048, "group": 128},
        # Serving: the same for a batch of prompts, one scale per row.
        {"name": "norm_prompt_e4m3", "op": "norm", "mode": "e4m3", "type": "f16", "rows": 6007, "C": 4096, "group": 0},
        # Training: residual addition, norm and gradients of a 16-bit model.
        {"name": "norm_train_bf16", "op": "norm", "mode": "train", "type": "bf16", "rows": 16384, "C": 2048, "group": 0},
        # Training at full precision with an odd number of channels (no aligned vectors).
        {"name": "norm_train_f32_odd", "op": "norm", "mode": "train", "type": "f32", "rows": 3136, "C": 1537, "group": 0},
        # Decoding: one token of each of 64 requests, windows in a pool.
        {"name": "conv_step_bf16", "op": "conv", "mode": "step", "type": "bf16", "S": 64, "T": 64, "D": 4096},
        # Prompts of uneven lengths packed one after the other, windows carried in and out.
        {"name": "conv_prompt_f16", "op": "conv", "mode": "prompt", "type": "f16", "S": 9, "T": 6007, "D": 2048},
        # Training: equal sequences, forward and all gradients.
        {"name": "conv_train_bf16", "op": "conv", "mode": "train", "type": "bf16", "S": 8, "T": 16384, "D": 4096},
        # Decoding: one token of each of 64 requests, states in a pool.
        {"name": "scan_step_bf16", "op": "scan", "mode": "step", "type": "bf16", "S": 64, "T": 64, "D": 4096, "N": 16, "G": 1},
        # One long prompt: the only parallelism is channels and the split over the sequence.
        {"name": "scan_prompt_bf16_long", "op": "scan", "mode": "prompt", "type": "bf16", "S": 1, "T": 8192, "D": 2048, "N": 16, "G": 1},
        # Packed prompts of uneven lengths with carried states and two groups of channels.
        {"name": "scan_prompt_f16_packed", "op": "scan", "mode": "prompt", "type": "f16", "S": 12, "T": 5003, "D": 1536, "N": 16, "G": 2},
        # Training: forward and all gradients of a 16-bit model.
        {"name": "scan_train_bf16", "op": "scan", "mode": "train", "type": "bf16", "S": 4, "T": 8192, "D": 2048, "N": 16, "G": 1},
        # Training at full precision, odd channels, lengths and state size.
        {"name": "scan_train_f32_odd", "op": "scan", "mode": "train", "type": "f32", "S": 3, "T": 1551, "D": 387, "N": 11, "G": 1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "conv", "scan", "scan"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        C = _log(rng, 64, 8192)
        C = C if rng.random() < 0.3 else max(64, C // 64 * 64)
        rows = _log(rng, 1, max(2, min(16384, (1 << 25) // C)))
        mode = rng.choice(["e4m3", "train"])
        return {"op": op, "mode": mode, "type": kind, "rows": rows, "C": C, "group": rng.choice([0, 128]) if mode == "e4m3" else 0}
    mode = rng.choice(["step", "prompt", "train"])
    if op == "conv":
        D = _log(rng, 48, 4096)
        D = D if rng.random() < 0.3 else max(64, D // 64 * 64)
        if mode == "step":
            S = _log(rng, 1, 256)
            return {"op": op, "mode": mode, "type": kind, "S": S, "T": S, "D": D}
        T = _log(rng, 1, min(16384, (1 << 25) // D))
        S = rng.randint(1, 12)
        return {"op": op, "mode": mode, "type": kind, "S": S, "T": T if mode == "prompt" else max(1, T // S) * S, "D": D}
    G = rng.choice([1, 1, 2])
    D = _log(rng, 32, 2048)
    D = G * (D // G if rng.random() < 0.3 else max(64, D // G // 64 * 64))
    N = rng.choice([16, 16, 8, 11, 24, 32])
    if mode == "step":
        S = _log(rng, 1, 256)
        return {"op": op, "mode": mode, "type": kind, "S": S, "T": S, "D": D, "N": N, "G": G}
    T = _log(rng, 1, min(8192, (1 << 27) // (D * N)))
    S = rng.randint(1, 12)
    return {"op": op, "mode": mode, "type": kind, "S": S, "T": T if mode == "prompt" else max(1, T // S) * S, "D": D, "N": N, "G": G}


def lengths(S, T):
    """Uneven lengths of S packed sequences with T tokens in all: one empty, one of a single token where there are enough."""
    if S == 1:
        return [T]
    share = [(5 * i + 3) % 11 + 1 for i in range(S)]
    if S > 3:
        share[1] = 0
    out = [T * s // sum(share) for s in share]
    if S > 4:
        out[2] = min(1, T)
    out[0] += T - sum(out)
    return out


def prepare(case, seed):
    dev, dt = "cuda", TYPES[case["type"]]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    s = dict(case)
    if case["op"] == "norm":
        M, C = case["rows"], case["C"]
        s.update(x=normal(M, C), residual=normal(M, C, std=2.0), w=uniform(C, lo=0.5, hi=1.5))
        if case["mode"] == "train":
            s.update(dy=normal(M, C, std=0.1), dh=normal(M, C, std=0.1))
        return s
    S, T, D, mode = case["S"], case["T"], case["D"], case["mode"]
    s["lens"] = [T // S] * S if mode == "train" else [1] * S if mode == "step" else lengths(S, T)
    s["max_len"] = max(s["lens"])
    starts = [0]
    for n in s["lens"]:
        starts.append(starts[-1] + n)
    s["offsets"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    if mode == "step":
        s["slots"] = torch.randperm(S, generator=gen, device=dev).to(torch.int32)
    if case["op"] == "conv":
        # x is the left half of an input projection's output; its right half is the gate of the scan.
        s["x"] = normal(T, 2 * D)[:, :D]
        s["w"] = uniform(D, WIDTH, lo=-0.5, hi=0.5)
        s["b"] = uniform(D, lo=-0.5, hi=0.5)
        if mode != "train":
            s["state"] = normal(S, WIDTH - 1, D)
            s["state_out"] = torch.empty_like(s["state"])
        else:
            s["dy"] = normal(T, D, std=0.1)
        return s
    N, G = case["N"], case["G"]
    s["u"] = normal(T, D)
    s["z"] = normal(T, 2 * D)[:, D:]
    s["delta"] = normal(T, D, std=0.5)
    bc = normal(T, G * 2 * N + 8)      # B and C are columns of one projection's output
    s["B"] = bc[:, 8:8 + G * N].unflatten(1, (G, N))
    s["C"] = bc[:, 8 + G * N:].unflatten(1, (G, N))
    s["A"] = -(torch.arange(1, N + 1, device=dev).float() * uniform(D, N, lo=0.8, hi=1.2)).contiguous()
    step = torch.exp(uniform(D, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["bias"] = step + torch.log(-torch.expm1(-step))        # softplus(bias) = step
    s["skip"] = uniform(D, lo=0.5, hi=1.5)
    if mode == "train":
        s["dy"] = normal(T, D, std=0.1)
    else:
        s["state"] = normal(S, D, N, std=0.5, dtype=torch.float32)
        s["state_out"] = torch.empty_like(s["state"])
    return s


def work(case):
    e = SIZE[case["type"]]
    if case["op"] == "norm":
        n = case["rows"] * case["C"]
        if case["mode"] == "e4m3":      # x, residual -> h, q, scales
            scales = case["rows"] * (-(-case["C"] // case["group"]) if case["group"] else 1)
            return {"bytes": n * (3 * e + 1) + 4 * (scales + case["C"]), "flops": 6 * n}
        # forward: x, residual -> h, y, r; gradients: dy, dh -> dx, dw (h is at hand)
        return {"bytes": n * 7 * e + 4 * (case["rows"] + 2 * case["C"]), "flops": 16 * n}
    T, D, S = case["T"], case["D"], case["S"]
    if case["op"] == "conv":
        state = 2 * S * (WIDTH - 1) * D * e
        param = 4 * D * (WIDTH + 1)
        if case["mode"] == "train":     # x, dy -> y, dx, dw, db
            return {"bytes": 4 * T * D * e + 2 * param, "flops": T * D * (8 * WIDTH + 20)}
        return {"bytes": 2 * T * D * e + state + param, "flops": T * D * (2 * WIDTH + 5)}
    N, G = case["N"], case["G"]
    bc, param = 2 * T * G * N * e, 4 * D * (N + 2)
    if case["mode"] == "train":         # u, delta, z, dy, B, C -> y, du, ddelta, dz, dB, dC, parameters' gradients
        return {"bytes": 8 * T * D * e + 2 * bc + 2 * param + 4 * S * D * N, "flops": T * D * (25 * N + 40)}
    return {"bytes": 4 * T * D * e + bc + param + 8 * S * D * N, "flops": T * D * (7 * N + 20)}


# ------------------------------------------------------------------------------------------------ plain form

def _round(t, like):
    return t.to(like.dtype)


def _plain_norm(s):
    x, w = s["x"], s["w"]
    h = _round(x.float() + s["residual"].float(), x)
    hf = h.float()
    r = torch.rsqrt((hf * hf).mean(1, keepdim=True) + EPS)
    y = hf * r * w
    if s["mode"] == "e4m3":
        M, C = y.shape
        g = s["group"] or C
        pad = -C % g
        blocks = torch.cat([y, y.new_zeros(M, pad)], 1).unflatten(1, (-1, g))
        top = blocks.abs().amax(2)
        scale = torch.where(top == 0, torch.ones_like(top), top / 448)
        q = (blocks / scale[..., None]).flatten(1)[:, :C].to(torch.float8_e4m3fn)
        return {"q": q, "scale": scale, "h": h}
    gw = s["dy"].float() * w
    mean = (gw * hf).mean(1, keepdim=True)
    dx = r * (gw - hf * r * r * mean) + s["dh"].float()
    dw = (s["dy"].float() * hf * r).sum(0)
    return {"y": _round(y, x), "h": h, "dx": _round(dx, x), "dw": dw}


def _window(s):
    """The inputs of every tap, [T, W, D], with what the carried windows hold before a sequence's first token."""
    x = s["x"].float()
    T, D = x.shape
    off = s["offsets"].long()
    row = torch.arange(T, device=x.device)
    seq = torch.bucketize(row, off[1:], right=True)
    at = row[:, None] + torch.arange(1 - WIDTH, 1, device=x.device)
    before = at - off[seq][:, None]                       # < 0: a carried input
    taps = x[at.clamp(min=0)]
    if s.get("state") is None:
        taps = torch.where((before < 0)[..., None], torch.zeros_like(taps), taps)
    else:
        carried = s["state"].float()[seq[:, None], (before + WIDTH - 1).clamp(0, WIDTH - 2)]
        taps = torch.where((before < 0)[..., None], carried, taps)
    return taps


def _last_window(s):
    """The last W - 1 inputs of every sequence, the carried ones among them."""
    x, state, off = s["x"], s["state"], s["offsets"].long()
    at = torch.arange(WIDTH - 1, device=x.device) - (WIDTH - 1)
    n = (off[1:] - off[:-1])[:, None]
    local = n + at                                        # < 0: still a carried input
    rows = (off[:-1][:, None] + local).clamp(0, max(0, x.shape[0] - 1))
    seq = torch.arange(len(n), device=x.device)[:, None]
    return torch.where((local < 0)[..., None], state[seq, (local + WIDTH - 1).clamp(max=WIDTH - 2)], x[rows])


def _plain_conv(s):
    x, w = s["x"], s["w"]
    if s["mode"] == "step":
        slots = s["slots"].long()
        taps = torch.cat([s["state"][slots].float(), x.float()[:, None]], 1)
        p = (taps * w.T).sum(1) + s["b"]
        s["state_out"][slots] = _round(taps[:, 1:], x)
        return {"y": _round(p / (1 + torch.exp(-p)), x), "state": s["state_out"]}
    taps = _window(s)
    p = (taps * w.T).sum(1) + s["b"]
    sig = 1 / (1 + torch.exp(-p))
    y = _round(p * sig, x)
    if s["mode"] == "prompt":
        return {"y": y, "state": _last_window(s)}
    T, D = x.shape
    g = s["dy"].float() * sig * (1 + p * (1 - sig))
    dw = (taps * g[:, None]).sum(0).T
    L = T // s["S"]
    ahead = torch.cat([g.view(-1, L, D), g.new_zeros(T // L, WIDTH - 1, D)], 1)
    dx = (ahead.unfold(1, WIDTH, 1).flip(-1) * w).sum(-1).view(T, D)
    return {"y": y, "dx": _round(dx, x), "dw": dw, "db": g.sum(0)}


def _linear_scan(a, b):
    """h[t] = a[t] h[t - 1] + b[t] along the first axis by doubling the distance that a value has travelled (both are overwritten)."""
    step = 1
    while step < a.shape[0]:
        b[step:] += a[step:] * b[:-step].clone()
        a[step:] *= a[:-step].clone()
        step *= 2
    return b


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(v.clamp(max=20))))


def _plain_scan(s):
    D, N, G, S = s["D"], s["N"], s["G"], s["S"]
    u, z = s["u"].float().unflatten(1, (G, -1)), s["z"].float().unflatten(1, (G, -1))
    raw = (s["delta"].float() + s["bias"]).unflatten(1, (G, -1))
    dl = _softplus(raw)
    A, skip = s["A"].view(G, D // G, N), s["skip"].view(G, D // G)
    B, C = s["B"].float()[:, :, None], s["C"].float()[:, :, None]      # [T, G, 1, N]
    gate = 1 / (1 + torch.exp(-z))
    if s["mode"] == "step":
        slots = s["slots"].long()
        h = torch.exp(dl[..., None] * A) * s["state"][slots].view(S, G, -1, N) + (dl * u)[..., None] * B
        y = ((h * C).sum(-1) + skip * u) * z * gate
        s["state_out"][slots] = h.view(S, D, N)
        return {"y": _round(y.flatten(1), s["u"]), "state": s["state_out"]}
    off = s["offsets"].long()
    n = off[1:] - off[:-1]
    full = n > 0
    first, last = off[:-1][full], off[1:][full] - 1
    a = torch.exp(dl[..., None] * A)
    b = (dl * u)[..., None] * B
    if s.get("state") is not None:
        b[first] += a[first] * s["state"][full].view(-1, G, D // G, N)
    cut = a.clone()
    cut[first] = 0
    h = _linear_scan(cut, b)
    o = (h * C).sum(-1) + skip * u
    y = _round((o * z * gate).flatten(1), s["u"])
    if s["mode"] == "prompt":
        state = s["state"].clone()
        state[full] = h[last].reshape(-1, D, N)
        return {"y": y, "state": state}
    state = h[last].reshape(-1, D, N)
    dy = s["dy"].float().unflatten(1, (G, -1))
    do = dy * z * gate
    dz = dy * o * gate * (1 + z * (1 - gate))
    back = torch.zeros_like(a)
    back[:-1] = a[1:]
    back[last] = 0
    g = _linear_scan(back.flip(0), (do[..., None] * C).flip(0)).flip(0)
    del back
    dC = (do[..., None] * h).sum(2)
    dB = (g * (dl * u)[..., None]).sum(2)
    gb = (g * B).sum(-1)
    du = skip * do + dl * gb
    h[1:] = h[:-1].clone()
    h[first] = 0
    q = g * a * h
    dA = (q * dl[..., None]).sum(0)
    ddl = ((q * A).sum(-1) + gb * u) / (1 + torch.exp(-raw))
    out = {"y": y, "state": state, "du": du, "ddelta": ddl, "dz": dz, "dB": dB, "dC": dC}
    out = {k: v if k in ("y", "state") else _round(v if k in ("dB", "dC") else v.flatten(1), s["u"]) for k, v in out.items()}
    return {**out, "dA": dA.view(D, N), "dskip": (do * u).sum(0).view(D), "dbias": ddl.sum(0).view(D)}


# ------------------------------------------------------------------------------------------------ the framework's calls

def _own_norm(s):
    import implicit_gemm_amd as iga
    if s["mode"] == "e4m3":
        q, scale, h = iga.rms_norm_e4m3(s["x"], s["w"], residual=s["residual"], eps=EPS, group=s["group"])
        return {"q": q, "scale": scale, "h": h}
    y, h, r = iga.rms_norm(s["x"], s["w"], residual=s["residual"], eps=EPS)
    dx, dw = iga.rms_norm_grad(s["dy"], h, s["w"], r, dh=s["dh"])
    return {"y": y, "h": h, "dx": dx, "dw": dw}


def _own_conv(s):
    import implicit_gemm_amd as iga
    if s["mode"] == "step":
        y = iga.causal_conv_step(s["x"], s["state"], s["w"], s["b"], silu=True, slots=s["slots"], state_out=s["state_out"])
        return {"y": y, "state": s["state_out"]}
    if s["mode"] == "prompt":
        y, state = iga.causal_conv(s["x"], s["w"], s["b"], silu=True, offsets=s["offsets"], state=s["state"],
                                   state_out=s["state_out"])
        return {"y": y, "state": state}
    x = s["x"].unflatten(0, (s["S"], -1))
    y, _ = iga.causal_conv(x, s["w"], s["b"], silu=True)
    dx, dw, db, _ = iga.causal_conv_grad(s["dy"].view(x.shape), x, s["w"], s["b"], silu=True)
    return {"y": y.flatten(0, 1), "dx": dx.flatten(0, 1), "dw": dw, "db": db}


def _own_scan(s):
    import implicit_gemm_amd as iga
    if s["mode"] == "step":
        y = iga.selective_scan_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], skip=s["skip"], z=s["z"],
                                    delta_bias=s["bias"], softplus=True, slots=s["slots"], state_out=s["state_out"])
        return {"y": y, "state": s["state_out"]}
    if s["mode"] == "prompt":
        y, state, _ = iga.selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], skip=s["skip"], z=s["z"],
                                         delta_bias=s["bias"], softplus=True, offsets=s["offsets"], max_len=s["max_len"],
                                         state=s["state"], state_out=s["state_out"])
        return {"y": y, "state": state}
    u, delta, z, B, C, dy = (s[k].unflatten(0, (s["S"], -1)) for k in ("u", "delta", "z", "B", "C", "dy"))
    y, state, saved = iga.selective_scan(u, delta, s["A"], B, C, skip=s["skip"], z=z, delta_bias=s["bias"], softplus=True,
                                         save=True)
    g = iga.selective_scan_grad(dy, u, delta, s["A"], B, C, saved, skip=s["skip"], z=z, delta_bias=s["bias"], softplus=True)
    return {"y": y.flatten(0, 1), "state": state, "du": g.du.flatten(0, 1), "ddelta": g.ddelta.flatten(0, 1),
            "dz": g.dz.flatten(0, 1), "dB": g.dB.flatten(0, 1), "dC": g.dC.flatten(0, 1), "dA": g.dA, "dskip": g.dskip,
            "dbias": g.ddelta_bias}


def run(state):
    if own:
        return {"norm": _own_norm, "conv": _own_conv, "scan": _own_scan}[state["op"]](state)
    return {"norm": _plain_norm, "conv": _plain_conv, "scan": _plain_scan}[state["op"]](state)


# ------------------------------------------------------------------------------------------------ the definition in 64 bits

def _exact_norm(s):
    h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype).double()
    C = h.shape[1]
    r = ((h ** 2).sum(1) / C + EPS) ** -0.5
    unit = h * r[:, None]
    y = unit * s["w"].double()
    if s["mode"] == "e4m3":
        g = s["group"] or C
        parts = y.split(g, dim=1)
        scale = torch.stack([p.abs().max(1).values / 448 for p in parts], 1)
        scale[scale == 0] = 1
        q = torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1)
        return {"q": q, "scale": scale, "h": h}
    dy = s["dy"].double()
    dunit = dy * s["w"].double()
    dx = r[:, None] * (dunit - unit * ((dunit * unit).sum(1) / C)[:, None]) + s["dh"].double()
    return {"y": y, "h": h, "dx": dx, "dw": (dy * unit).sum(0)}


def _sequences(s):
    out, at = [], 0
    for n in s["lens"]:
        out.append((at, at + n))
        at += n
    return out


def _exact_conv(s):
    x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
    step = s["mode"] == "step"
    y, dx = torch.empty_like(x), torch.zeros_like(x)
    dw, db = torch.zeros_like(w), torch.zeros_like(b)
    state = torch.empty_like(s["state"], dtype=torch.float64) if s.get("state") is not None else None
    slots = s["slots"].tolist() if step else list(range(s["S"]))
    for i, (lo, hi) in enumerate(_sequences(s)):
        head = s["state"][slots[i]].double() if state is not None else x.new_zeros(WIDTH - 1, x.shape[1])
        line = torch.cat([head, x[lo:hi]])
        n = hi - lo
        p = b + sum(line[k:k + n] * w[:, k] for k in range(WIDTH))
        sg = torch.sigmoid(p)
        y[lo:hi] = p * sg
        if state is not None:
            state[slots[i]] = line[n:]
        else:
            g = s["dy"][lo:hi].double() * (sg + p * sg * (1 - sg))
            dline = torch.zeros_like(line)
            for k in range(WIDTH):
                dline[k:k + n] += g * w[:, k]
                dw[:, k] += (g * line[k:k + n]).sum(0)
            db += g.sum(0)
            dx[lo:hi] = dline[WIDTH - 1:]
    return {"y": y, "dx": dx, "dw": dw, "db": db} if state is None else {"y": y, "state": state}


def _exact_scan(s):
    S, D, N, G = s["S"], s["D"], s["N"], s["G"]
    u, z, A, skip = s["u"].double(), s["z"].double(), s["A"].double(), s["skip"].double()
    raw = s["delta"].double() + s["bias"].double()
    dl = torch.logaddexp(raw, torch.zeros_like(raw))
    chan = torch.arange(D, device=u.device) // (D // G)
    B, C = s["B"].double(), s["C"].double()
    lens = torch.tensor(s["lens"], device=u.device)
    starts = torch.cumsum(lens, 0) - lens
    step, train = s["mode"] == "step", s["mode"] == "train"
    place = s["slots"].long() if step else torch.arange(S, device=u.device)
    h = s["state"].double()[place] if s.get("state") is not None else u.new_zeros(S, D, N)
    o = torch.empty_like(u)
    kept = []
    for t in range(max(s["lens"])):
        on = None if min(s["lens"]) > t else torch.nonzero(lens > t)[:, 0]
        r = (starts if on is None else starts[on]) + t
        prev = h if on is None else h[on]
        if train:
            kept.append(prev.float() if S * D * N * len(s["lens"]) * max(s["lens"]) > 1 << 31 else prev)
        new = torch.exp(dl[r][..., None] * A) * prev + (dl[r] * u[r])[..., None] * B[r][:, chan]
        o[r] = (new * C[r][:, chan]).sum(-1) + skip * u[r]
        if on is None:
            h = new
        else:
            h = h.clone()
            h[on] = new
    sz = torch.sigmoid(z)
    state = torch.empty_like(h)
    state[place] = h
    out = {"y": o * z * sz, "state": state}
    if not train:
        return out
    dy = s["dy"].double()
    do = dy * z * sz
    du, ddl = skip * do, torch.zeros_like(u)
    dB, dC, dA = torch.zeros_like(B), torch.zeros_like(C), torch.zeros_like(A)
    carry = torch.zeros_like(h)
    for t in range(max(s["lens"]) - 1, -1, -1):          # equal lengths in training
        r = starts + t
        prev = kept.pop().double()
        a = torch.exp(dl[r][..., None] * A)
        Br, Cr = B[r][:, chan], C[r][:, chan]
        now = a * prev + (dl[r] * u[r])[..., None] * Br
        dC.view(-1, G, N)[r] = (do[r][..., None] * now).view(S, G, D // G, N).sum(2)
        g = carry + do[r][..., None] * Cr
        dB.view(-1, G, N)[r] = (g * (dl[r] * u[r])[..., None]).view(S, G, D // G, N).sum(2)
        gb = (g * Br).sum(-1)
        du[r] += dl[r] * gb
        carry = g * a
        q = carry * prev
        ddl[r] = (q * A).sum(-1) + u[r] * gb
        dA += (q * dl[r][..., None]).sum(0)
    ddl = ddl * torch.sigmoid(raw)
    return {**out, "du": du, "ddelta": ddl, "dz": dy * o * (sz + z * sz * (1 - sz)), "dB": dB, "dC": dC, "dA": dA,
            "dskip": (do * u).sum(0), "dbias": ddl.sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan}[s["op"]](s)
