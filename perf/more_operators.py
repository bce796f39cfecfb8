"""Measured cases of the layer norm (with its gradient) and of the gated delta rule (prompts, training, single tokens).

The operators' formulas (32-bit arithmetic whatever the element type, one rounding per output):

  norm   h = x + residual (rounded to the element type: the next layer reads it), m = mean(h), r = 1 / sqrt(mean((h - m)^2)
         + eps), y = (h - m) r w + b.  With n = (h - m) r: dh = r (dy w - mean(dy w) - n mean(dy w n)) + dh_next,
         dw = sum over rows of dy n, db = sum over rows of dy.
  delta  per head, with a state S [Dk, Dv] that maps keys to values and a decay a = e^g:
         S[t] = a S[t-1] + beta k (v - (a S[t-1])^T k)^T,  o[t] = scale S[t]^T q.
         Heads of v share the heads of q and k in order (H / Hk of them each).

`own` selects the framework's calls; the plain form is elementary torch arithmetic.  It takes the delta rule 64 tokens at a
time: inside of such a chunk the tokens' mutual corrections are a unit triangular system, between chunks the state carries.
"""
import math

import torch

own = False
EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 64


def listed():
    return [
        # Serving: the norm in front of a projection for one token of each of a few requests (latency only).
        {"name": "ln_token_bf16", "op": "norm", "mode": "infer", "type": "bf16", "rows": 16, "C": 2048, "residual": True},
        # Serving: the same for a batch of prompts.
        {"name": "ln_prompt_f16", "op": "norm", "mode": "infer", "type": "f16", "rows": 6007, "C": 4096, "residual": True},
        # Training: residual addition, norm and gradients of a 16-bit model.
        {"name": "ln_train_bf16", "op": "norm", "mode": "train", "type": "bf16", "rows": 16384, "C": 2048, "residual": True},
        # Training: the channels of a feature map behind a depthwise 7x7 convolution (64 images of 56 x 56).
        {"name": "ln_map_bf16", "op": "norm", "mode": "train", "type": "bf16", "rows": 200704, "C": 384, "residual": False},
        # Training at full precision with an odd number of channels (no aligned vectors).
        {"name": "ln_train_f32_odd", "op": "norm", "mode": "train", "type": "f32", "rows": 3136, "C": 1537, "residual": True},
        # Decoding: one token of each of 64 requests, states in a pool, two value heads to a key head.
        {"name": "delta_step_bf16", "op": "delta", "mode": "step", "type": "bf16", "S": 64, "T": 64, "Hk": 16, "H": 32, "Dk": 128, "Dv": 128},
        # Decoding a few requests of a small model in full precision, odd head sizes (latency only).
        {"name": "delta_step_f32_odd", "op": "delta", "mode": "step", "type": "f32", "S": 5, "T": 5, "Hk": 3, "H": 6, "Dk": 72, "Dv": 41},
        # One long prompt: chunks follow one another, the only parallelism is heads and columns of the state.
        {"name": "delta_prompt_bf16_long", "op": "delta", "mode": "prompt", "type": "bf16", "S": 1, "T": 8192, "Hk": 16, "H": 32, "Dk": 128, "Dv": 128},
        # Packed prompts of uneven lengths with carried states.
        {"name": "delta_prompt_f16_packed", "op": "delta", "mode": "prompt", "type": "f16", "S": 12, "T": 5003, "Hk": 8, "H": 8, "Dk": 128, "Dv": 128},
        # Packed prompts with wide heads (keys of 256).
        {"name": "delta_prompt_bf16_wide", "op": "delta", "mode": "prompt", "type": "bf16", "S": 3, "T": 4099, "Hk": 4, "H": 4, "Dk": 256, "Dv": 256},
        # Training: forward and all gradients of a 16-bit model.
        {"name": "delta_train_bf16", "op": "delta", "mode": "train", "type": "bf16", "S": 4, "T": 8192, "Hk": 16, "H": 16, "Dk": 128, "Dv": 128},
        # Training at full precision, odd sizes and lengths, value heads that share keys.
        {"name": "delta_train_f32_odd", "op": "delta", "mode": "train", "type": "f32", "S": 3, "T": 1551, "Hk": 3, "H": 6, "Dk": 72, "Dv": 41},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "delta", "delta"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op == "norm":
        C = _log(rng, 64, 8192)
        C = C if rng.random() < 0.3 else max(64, C // 64 * 64)
        rows = _log(rng, 1, max(2, min(200704, (1 << 25) // C)))
        return {"op": op, "mode": rng.choice(["infer", "train"]), "type": kind, "rows": rows, "C": C, "residual": rng.random() < 0.6}
    mode = rng.choice(["step", "prompt", "train"])
    share = rng.choice([1, 1, 2, 4])
    Hk = _log(rng, 1, 16)
    H = min(32, Hk * share) // Hk * Hk
    Dk, Dv = (rng.choice([64, 128, 128, 256, rng.randint(16, 128)]) for _ in range(2))
    base = {"op": op, "mode": mode, "type": kind}
    if mode == "step":
        S = _log(rng, 1, max(2, min(256, (1 << 26) // (H * Dk * Dv))))
        return {**base, "S": S, "T": S, "Hk": Hk, "H": H, "Dk": Dk, "Dv": Dv}
    T = _log(rng, 1, max(2, min(8192, (1 << 31) // (H * Dk * Dv))))
    S = rng.randint(1, 12)
    return {**base, "S": S, "T": T if mode == "prompt" else max(1, T // S) * S, "Hk": Hk, "H": H, "Dk": Dk, "Dv": Dv}


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
    gen.manual_seed(int(seed) * 7919 + 23)

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=dev) * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=gen, device=dev) * (hi - lo) + lo

    s = dict(case)
    if case["op"] == "norm":
        M, C = case["rows"], case["C"]
        s.update(x=normal(M, C), w=uniform(C, lo=0.5, hi=1.5), b=normal(C, std=0.2, dtype=torch.float32))
        s["res"] = normal(M, C, std=2.0) + 0.5 if case["residual"] else None
        if case["mode"] == "train":
            s.update(dy=normal(M, C, std=0.1), dh=normal(M, C, std=0.1) if case["residual"] else None)
        return s
    S, T, Hk, H, Dk, Dv, mode = (case[k] for k in ("S", "T", "Hk", "H", "Dk", "Dv", "mode"))
    s["lens"] = [T // S] * S if mode == "train" else [1] * S if mode == "step" else lengths(S, T)
    starts = [0]
    for n in s["lens"]:
        starts.append(starts[-1] + n)
    s["offsets"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    # q, k and v are columns of one projection's output; keys and queries have unit length, as a model makes them.
    x = torch.randn(T, (2 * Hk * Dk + H * Dv), generator=gen, device=dev)
    qk = x[:, :2 * Hk * Dk].unflatten(1, (2 * Hk, Dk))
    qk.mul_(torch.rsqrt((qk * qk).sum(-1, keepdim=True) + 1e-6))
    x = x.to(dt)
    s["q"] = x[:, :Hk * Dk].unflatten(1, (Hk, Dk))
    s["k"] = x[:, Hk * Dk:2 * Hk * Dk].unflatten(1, (Hk, Dk))
    s["v"] = x[:, 2 * Hk * Dk:].unflatten(1, (H, Dv))
    # g = -A softplus(a + bias): decays from nearly none to a few tokens' memory, as the heads of a model have them.
    step = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(1e-1)))
    bias = step + torch.log(-torch.expm1(-step))
    a = normal(T, H, std=0.5, dtype=torch.float32) + bias
    s["g"] = -uniform(H, lo=1.0, hi=16.0) * torch.log1p(torch.exp(a))
    s["beta"] = torch.sigmoid(normal(T, H, dtype=torch.float32))
    if mode == "train":
        s["do"] = normal(T, H, Dv, std=0.1)
    else:
        s["state"] = normal(S, H, Dk, Dv, std=0.2, dtype=torch.float32)
        s["state_out"] = torch.empty_like(s["state"])
    if mode == "step":
        s["slots"] = torch.randperm(S, generator=gen, device=dev).to(torch.int32)
    return s


def work(case):
    e = SIZE[case["type"]]
    if case["op"] == "norm":
        n, res = case["rows"] * case["C"], case["residual"]
        forward = n * e * (4 if res else 2) + 8 * case["C"]     # x, residual -> h, y
        if case["mode"] == "infer":
            return {"bytes": forward, "flops": 8 * n}
        # gradients: dy, dh -> dx, dw, db (h is at hand)
        return {"bytes": forward + n * e * (3 if res else 2) + 8 * (case["rows"] + case["C"]), "flops": 20 * n}
    S, T, Hk, H, Dk, Dv = (case[k] for k in ("S", "T", "Hk", "H", "Dk", "Dv"))
    qk, vo, gb, state = 2 * T * Hk * Dk * e, 2 * T * H * Dv * e, 8 * T * H, 4 * S * H * Dk * Dv
    if case["mode"] == "train":         # q, k, v, g, beta, do -> o, state and the five gradients
        return {"bytes": 2 * qk + 2 * vo + 2 * gb + state, "flops": 23 * T * H * Dk * Dv}
    return {"bytes": qk + vo + gb + 2 * state, "flops": 7 * T * H * Dk * Dv}


# ------------------------------------------------------------------------------------------------ plain form

def _plain_norm(s):
    x, w, dt = s["x"], s["w"], s["x"].dtype
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(dt)
    hf = h.float()
    m = hf.mean(1, keepdim=True)
    c = hf - m
    r = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
    n = c * r
    out = {"y": (n * w + s["b"]).to(dt), "h": h}
    if s["mode"] == "infer":
        return out
    dy = s["dy"].float()
    gw = dy * w
    dx = r * (gw - gw.mean(1, keepdim=True) - n * (gw * n).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {**out, "dx": dx.to(dt), "dw": (dy * n).sum(0), "db": dy.sum(0)}


def _heads(t, s):
    """[T, Hk, Dk] -> [T, H, Dk] in 32 bits."""
    return t.float().repeat_interleave(s["H"] // s["Hk"], 1)


def _plain_step(s):
    slots = s["slots"].long()
    q, k, v = _heads(s["q"], s), _heads(s["k"], s), s["v"].float()
    S = s["state"][slots] * torch.exp(s["g"])[..., None, None]
    z = (v - (S * k[..., None]).sum(-2)) * s["beta"][..., None]
    S = S + k[..., None] * z[..., None, :]
    o = (S * q[..., None]).sum(-2) * s["Dk"] ** -0.5
    s["state_out"][slots] = S
    return {"o": o.to(s["v"].dtype), "state": s["state_out"]}


def _cut(t, s, at):
    """[T, H, ...] -> [S, H, chunks, CHUNK, ...] with zeros behind each sequence's end."""
    out = t.new_zeros((at[1],) + t.shape[1:])
    out[at[0]] = t
    return out.unflatten(0, (s["S"], -1, CHUNK)).movedim(3, 1)


def _join(t, at):
    """The inverse of _cut."""
    return t.movedim(1, 3).flatten(0, 2)[at[0]]


def _plain_delta(s):
    if s["mode"] == "step":
        return _plain_step(s)
    T, H, Hk, Dk, Dv, dt = s["T"], s["H"], s["Hk"], s["Dk"], s["Dv"], s["v"].dtype
    chunks = max(1, -(-max(s["lens"]) // CHUNK))
    off, row = s["offsets"].long(), torch.arange(T, device=s["v"].device)
    seq = torch.bucketize(row, off[1:], right=True)
    at = (seq * chunks * CHUNK + row - off[seq], s["S"] * chunks * CHUNK)
    q, k, v, g, b = (_cut(t, s, at) for t in (_heads(s["q"], s), _heads(s["k"], s), s["v"].float(), s["g"], s["beta"]))
    scale = Dk ** -0.5
    G = g.double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=g.device).tril()
    e = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf))      # from token j to token i >= j
    first, last = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    kk = (k.double() @ k.double().transpose(-1, -2)) * e
    M = kk.tril(-1) * b.double()[..., None, :]
    inv = torch.eye(CHUNK, device=g.device, dtype=torch.float64) - M
    for _ in range(5):                                    # (1 + M)^-1 = (1 - M)(1 + M^2)(1 + M^4) ..., M^64 = 0
        M = M @ M
        inv = inv + inv @ M
    inv, e = inv.float(), e.float()
    P = (q @ k.transpose(-1, -2)) * e * b[..., None, :]
    S = s["state"] if s.get("state") is not None else v.new_zeros(s["S"], H, Dk, Dv)
    states, o, z = [S], torch.empty_like(v), torch.empty_like(v)
    for n in range(chunks):
        x = v[:, :, n] - first[:, :, n] * (k[:, :, n] @ S)
        z[:, :, n] = inv[:, :, n] @ x
        o[:, :, n] = (first[:, :, n] * (q[:, :, n] @ S) + P[:, :, n] @ z[:, :, n]) * scale
        S = first[:, :, n, -1:] * S + (k[:, :, n] * last[:, :, n] * b[:, :, n, :, None]).transpose(-1, -2) @ z[:, :, n]
        states.append(S)
    out = {"o": _join(o, at).to(dt), "state": S}
    if s["mode"] == "prompt":
        return out
    do = _cut(s["do"].float() * scale, s, at)
    bc = b[..., None]
    dS = torch.zeros_like(S)
    dS_of, dx, tail = [], torch.empty_like(v), g.new_empty(g.shape[:3])
    for n in reversed(range(chunks)):
        dS_of.insert(0, dS)
        tail[:, :, n] = (dS * states[n + 1]).sum((-1, -2))
        dz = bc[:, :, n] * last[:, :, n] * (k[:, :, n] @ dS) + P[:, :, n].transpose(-1, -2) @ do[:, :, n]
        dx[:, :, n] = inv[:, :, n].transpose(-1, -2) @ dz
        dS = (first[:, :, n, -1:] * dS + (first[:, :, n] * q[:, :, n]).transpose(-1, -2) @ do[:, :, n]
              - (first[:, :, n] * k[:, :, n]).transpose(-1, -2) @ dx[:, :, n])
    S_in, dS_out = torch.stack(states[:-1], 2).transpose(-1, -2), torch.stack(dS_of, 2).transpose(-1, -2)
    E = (do @ z.transpose(-1, -2)) * e
    R = (dx @ z.transpose(-1, -2)) * e.tril(-1)
    dq = first * (do @ S_in) + (E * b[..., None, :]) @ k
    reads = -first * (dx @ S_in) - (R * b[..., None, :]) @ k
    writes = last * (z @ dS_out) + E.transpose(-1, -2) @ q - R.transpose(-1, -2) @ k
    db = (k * writes).sum(-1)
    dG = (q * dq + k * reads).sum(-1) - b * db
    dg = dG.flip(-1).cumsum(-1).flip(-1) + tail[..., None]

    def group(t):
        return _join(t, at).unflatten(1, (Hk, -1)).sum(2).to(dt)

    return {**out, "dq": group(dq), "dk": group(reads + bc * writes), "dv": _join(dx, at).to(dt), "dg": _join(dg, at),
            "dbeta": _join(db, at)}


# ------------------------------------------------------------------------------------------------ the framework's calls

def _own_norm(s):
    import implicit_gemm_amd as iga
    y, h, m, r = iga.layer_norm(s["x"], s["w"], s["b"], residual=s["res"], eps=EPS)
    if s["mode"] == "infer":
        return {"y": y, "h": h}
    dx, dw, db = iga.layer_norm_grad(s["dy"], h, s["w"], m, r, dh=s["dh"])
    return {"y": y, "h": h, "dx": dx, "dw": dw, "db": db}


def _own_delta(s):
    import implicit_gemm_amd as iga
    if s["mode"] == "step":
        o = iga.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], slots=s["slots"], state_out=s["state_out"])
        return {"o": o, "state": s["state_out"]}
    if s["mode"] == "prompt":
        o, state, _ = iga.gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], offsets=s["offsets"], state=s["state"],
                                      state_out=s["state_out"])
        return {"o": o, "state": state}
    q, k, v, g, beta, do = (s[n].unflatten(0, (s["S"], -1)) for n in ("q", "k", "v", "g", "beta", "do"))
    o, state, saved = iga.gated_delta(q, k, v, g, beta, save=True)
    d = iga.gated_delta_grad(do, q, k, v, g, beta, saved)
    return {"o": o.flatten(0, 1), "state": state, "dq": d.dq.flatten(0, 1), "dk": d.dk.flatten(0, 1), "dv": d.dv.flatten(0, 1),
            "dg": d.dg.flatten(0, 1), "dbeta": d.dbeta.flatten(0, 1)}


def run(state):
    if own:
        return (_own_norm if state["op"] == "norm" else _own_delta)(state)
    return (_plain_norm if state["op"] == "norm" else _plain_delta)(state)


# ------------------------------------------------------------------------------------------------ the definition in 64 bits

def _exact_norm(s):
    h = s["x"].double()
    if s["res"] is not None:
        h = (h + s["res"].double()).to(s["x"].dtype).double()
    C, w = h.shape[1], s["w"].double()
    mean = h.sum(1) / C
    var = ((h - mean[:, None]) ** 2).sum(1) / C
    unit = (h - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
    out = {"y": unit * w + s["b"].double(), "h": h}
    if s["mode"] == "infer":
        return out
    dy = s["dy"].double()
    dunit = dy * w
    # through the variance and through the mean, one after the other
    dc = dunit / torch.sqrt(var + EPS)[:, None]
    dvar = -(dunit * unit).sum(1) / (2 * (var + EPS))
    dc = dc + (2 * dvar / C)[:, None] * (h - mean[:, None])
    dx = dc - (dc.sum(1) / C)[:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].double()
    return {**out, "dx": dx, "dw": (dy * unit).sum(0), "db": dy.sum(0)}


def _exact_delta(s):
    """Token by token, all sequences and heads at once; the gradient walks back over the kept states."""
    S, H, Hk, Dk, Dv = (s[n] for n in ("S", "H", "Hk", "Dk", "Dv"))
    dev = s["v"].device
    head = torch.arange(H, device=dev) // (H // Hk)
    q, k, v, b = s["q"].double(), s["k"].double(), s["v"].double(), s["beta"].double()
    a = torch.exp(s["g"].double())
    lens = torch.tensor(s["lens"], device=dev)
    starts = torch.cumsum(lens, 0) - lens
    train, longest, shortest = s["mode"] == "train", max(s["lens"]), min(s["lens"])
    place = s["slots"].long() if s["mode"] == "step" else torch.arange(S, device=dev)
    state = s["state"].double()[place] if s.get("state") is not None else v.new_zeros(S, H, Dk, Dv)
    o, scale, kept = torch.empty_like(v), Dk ** -0.5, []
    for t in range(longest):
        on = None if shortest > t else torch.nonzero(lens > t)[:, 0]
        r = (starts if on is None else starts[on]) + t
        prev = state if on is None else state[on]
        if train:
            kept.append(prev)
        kt = k[r][:, head]
        new = prev * a[r][..., None, None]
        err = v[r] - (kt[:, :, None] @ new)[:, :, 0]
        new = new + kt[..., None] * (b[r][..., None] * err)[:, :, None]
        o[r] = (q[r][:, head][:, :, None] @ new)[:, :, 0] * scale
        if on is None:
            state = new
        else:
            state = state.index_copy(0, on, new)
    final = torch.empty_like(state)
    final[place] = state
    out = {"o": o, "state": final}
    if not train:
        return out
    do = s["do"].double() * scale
    dq, dk = v.new_zeros(v.shape[0], H, Dk), v.new_zeros(v.shape[0], H, Dk)
    dv, dg, db = torch.zeros_like(v), torch.zeros_like(a), torch.zeros_like(b)
    D = torch.zeros_like(state)
    for t in range(longest - 1, -1, -1):                  # equal lengths in training
        r = starts + t
        prev = kept.pop()
        kt, qt, bt, dot = k[r][:, head], q[r][:, head], b[r][..., None], do[r]
        dec = prev * a[r][..., None, None]
        err = v[r] - (kt[:, :, None] @ dec)[:, :, 0]
        after = dec + kt[..., None] * (bt * err)[:, :, None]
        dq[r] = (after @ dot[..., None])[..., 0]
        D = D + qt[..., None] * dot[:, :, None]
        kD = (kt[:, :, None] @ D)[:, :, 0]                # of beta err
        db[r] = (kD * err).sum(-1)
        derr = bt * kD
        dv[r] = derr
        dk[r] = (D @ (bt * err)[..., None])[..., 0] - (dec @ derr[..., None])[..., 0]
        D = D - kt[..., None] * derr[:, :, None]
        dg[r] = (D * dec).sum((-1, -2))
        D = D * a[r][..., None, None]
    return {**out, "dq": dq.unflatten(1, (Hk, -1)).sum(2), "dk": dk.unflatten(1, (Hk, -1)).sum(2), "dv": dv, "dg": dg, "dbeta": db}


def exact(case, seed):
    s = prepare(case, seed)
    return (_exact_norm if s["op"] == "norm" else _exact_delta)(s)
