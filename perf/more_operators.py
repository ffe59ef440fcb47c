"""Cases of the layer norm, the short causal convolution and the selective scan.

``run`` computes a case in plain torch operations, or, where ``own`` is set,
with the library's entry points; ``exact`` gives the same values in float64
from the definitions.

Layer norm, per row of D values, s = x (+ residual, the sum rounded to the
type, as it is stored):
    y = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias
Short causal convolution, per channel of [B, T, D], K taps, x_t = 0 (or the
state) before the first token:
    c_t = bias + sum_k w_k x_{t-K+1+k},  y = c or c / (1 + exp(-c))
Selective scan, per channel d and state n (h in float32):
    delta = log(1 + exp(dt + dt_bias)),  h_t = exp(delta A) h_{t-1} + delta u B_t
    y_t = (sum_n C_t h_t + D u) z / (1 + exp(-z))
"""
import math

import torch

own = False

EPS = 1e-5
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
LARGEST = {"norm": 32768 * 1536, "conv": 8 * 4096 * 1536, "scan": 8 * 4096 * 1536 * 16}


def listed():
    return [
        # one token's norm in a decode: the row of one sequence
        dict(name="norm_token", op="norm", train=False, dtype="f32", rows=1, D=768, residual=True),
        # a layer's norm with the residual stream at the model's batch (4 x 2048 tokens)
        dict(name="norm_layer", op="norm", train=False, dtype="bf16", rows=8192, D=768,
             residual=True),
        # the norm of a training step, 8 x 4096 tokens, the residual's gradient coming in
        dict(name="norm_train", op="norm", train=True, dtype="bf16", rows=32768, D=768,
             residual=True),
        # a final norm at an odd width, in float32
        dict(name="norm_odd", op="norm", train=True, dtype="f32", rows=5005, D=771,
             residual=False),
        # one token of a batch of 64 sequences
        dict(name="conv_token", op="conv_step", dtype="bf16", B=64, D=1536, K=4, act=True),
        # prompts of unequal lengths that go on from states, odd sizes, one half of a projection
        dict(name="conv_ragged", op="conv", train=False, dtype="f32", B=5, T=1001, D=771, K=4,
             act=True, state=True, ragged=True, joined=True),
        # the convolution of a training step, on one half of the layer's input projection
        dict(name="conv_train", op="conv", train=True, dtype="bf16", B=8, T=4096, D=1536, K=4,
             act=True, state=False, ragged=False, joined=True),
        # one token of one sequence
        dict(name="scan_token", op="scan_step", dtype="f32", B=1, D=1536, N=16, gated=True),
        # one token of a batch of 512 sequences, all its states
        dict(name="scan_tokens", op="scan_step", dtype="bf16", B=512, D=1536, N=16, gated=True),
        # a long prompt: 1 x 32768 tokens, its last state kept
        dict(name="scan_long", op="scan", train=False, dtype="bf16", B=1, T=32768, D=1536, N=16,
             gated=True, state=False, ragged=False, joined=True),
        # a stretch of a longer text in training: states come in, their gradients go out; odd sizes
        dict(name="scan_stretch", op="scan", train=True, dtype="f32", B=3, T=1001, D=771, N=13,
             gated=True, state=True, ragged=True, joined=False),
        # a training step's forward and backward
        dict(name="scan_train", op="scan", train=True, dtype="bf16", B=8, T=4096, D=1536, N=16,
             gated=True, state=False, ragged=False, joined=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "conv", "conv", "conv_step", "scan", "scan", "scan", "scan_step"])
    dtype, train = rng.choice(["f32", "bf16"]), rng.random() < 0.5
    if op == "norm":
        D = _log(rng, 5, 9000)
        rows = min(_log(rng, 1, 40000), LARGEST["norm"] // (2 * D))
        return dict(op=op, train=train, dtype=dtype, rows=rows, D=D, residual=rng.random() < 0.5)
    D = _log(rng, 1, 2500)
    K, act, N = rng.choice([4, 4, 4, 3, 2, 7]), rng.random() < 0.8, _log(rng, 1, 64)
    N = rng.choice([16, 16, N, N])
    gated = rng.random() < 0.6
    if op == "conv_step":
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 2000), D=D, K=K, act=act)
    if op == "scan_step":
        return dict(op=op, dtype=dtype, B=_log(rng, 1, 600), D=D, N=N, gated=gated)
    B = _log(rng, 1, 24)
    each = D * N if op == "scan" else D
    T = min(_log(rng, 1, 32768), max(1, LARGEST[op] // 2 // (B * each)))
    case = dict(op=op, train=train, dtype=dtype, B=B, T=T, D=D, state=rng.random() < 0.5,
                ragged=rng.random() < 0.4, joined=rng.random() < 0.5)
    return dict(case, K=K, act=act) if op == "conv" else dict(case, N=N, gated=gated)


def _lengths(B, T):
    """Lengths of a padded batch: from the whole row down, the last one short."""
    return [max(0, T - (b * T) // B - (b % 3)) for b in range(B)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    op, D, dt = case["op"], case["D"], DTYPE[case["dtype"]]
    s = dict(case=case)
    if op == "norm":
        shape = (case["rows"], D)
        s["x"] = (1.5 * normal(*shape) + 0.3 * normal(D)).to(dt)
        s["residual"] = (2 * normal(*shape) + 0.5).to(dt) if case["residual"] else None
        s["weight"], s["bias"] = 1 + 0.2 * normal(D), 0.1 * normal(D)
        if case["train"]:
            s["dy"] = normal(*shape).to(dt)
            s["ds"] = normal(*shape).to(dt) if case["residual"] else None
        return s
    B = case["B"]
    step = op.endswith("step")
    lead = (B,) if step else (B, case["T"])
    lens = not step and case["ragged"]
    s["lens"] = torch.tensor(_lengths(B, case["T"]), device="cuda") if lens else None
    state = step or case["state"]
    joined = not step and case["joined"]
    # the two halves of the layer's input projection: the convolution's and the gate's
    both = normal(*lead, 2 * D).to(dt) if joined else None
    if op.startswith("conv"):
        K = case["K"]
        s["x"] = both[..., :D] if joined else normal(*lead, D).to(dt)
        s["w"], s["bias"] = normal(D, K) / math.sqrt(K), 0.2 * normal(D)
        s["s"] = normal(B, K - 1, D).to(dt).float() if state else None
        if not step and case["train"]:
            s["dy"] = normal(*lead, D).to(dt)
            s["ds"] = normal(B, K - 1, D) if state else None
        return s
    N = case["N"]
    c = normal(*lead, D)
    s["u"] = (c / (1 + torch.exp(-c)) * 1.5).to(dt)
    # steps from 0.001 to 0.1, each channel its own, moved by the token
    size = torch.exp(uniform(D) * math.log(100) + math.log(0.001))
    s["dt_bias"] = size + torch.log(-torch.expm1(-size))
    s["dt"] = (0.6 * normal(*lead, D)).to(dt)
    s["A"] = -(torch.arange(N, device="cuda") + 1.0) * torch.exp(0.1 * normal(D, N))
    if joined:      # rows of the projection that also gives dt, of rank D / 16
        rank = -(-D // 16)
        rows = normal(*lead, rank + 2 * N).to(dt)
        s["B"], s["C"] = rows[..., rank:rank + N], rows[..., rank + N:]
    else:
        s["B"], s["C"] = normal(*lead, N).to(dt), normal(*lead, N).to(dt)
    s["D"] = 1 + 0.1 * normal(D)
    s["z"] = (both[..., D:] if joined else normal(*lead, D).to(dt)) if case["gated"] else None
    s["h"] = 0.1 * normal(B, D, N) if state else None
    if not step and case["train"]:
        s["dy"] = normal(*lead, D).to(dt)
        s["dh"] = normal(B, D, N) if state else None
    return s


# The plain form.

def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _norm_plain(s):
    x, dt = s["x"].float(), s["x"].dtype
    if s["residual"] is not None:
        total = (x + s["residual"].float()).to(dt)
        x = total.float()
    far = x - x.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((far * far).mean(-1, keepdim=True) + EPS)
    hat = far * rstd
    out = [(hat * s["weight"] + s["bias"]).to(dt)]
    if s["residual"] is not None:
        out.append(total)
    if not s["case"]["train"]:
        return out
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - hat * (g * hat).mean(-1, keepdim=True))
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return out + [dx.to(dt), (dy * hat).sum(0), dy.sum(0)]


def _there(s):
    """[B, T, 1] truth values: the tokens that are there; None where all are."""
    if s["lens"] is None:
        return None
    return (torch.arange(s["case"]["T"], device="cuda") < s["lens"][:, None]).unsqueeze(-1)


def _only(there, x):
    return x if there is None else torch.where(there, x, 0.0)


def _conv_plain(s):
    case, dt = s["case"], s["x"].dtype
    B, T, D, K = (case[n] for n in ("B", "T", "D", "K"))
    there = _there(s)
    x = _only(there, s["x"].float())
    first = torch.zeros(B, K - 1, D, device="cuda") if s["s"] is None else s["s"]
    x = torch.cat([first, x], 1)
    windows = x.unfold(1, K, 1)                               # [B, T, D, K]
    c = (windows * s["w"]).sum(-1) + s["bias"]
    sig = _sigmoid(c)
    y = _only(there, c * sig if case["act"] else c).to(dt)
    ends = s["lens"] if there is not None else torch.full((B,), T, device="cuda")
    last = (ends[:, None] + torch.arange(K - 1, device="cuda"))[..., None].expand(-1, -1, D)
    out = [y, torch.gather(x, 1, last)]
    if not case["train"]:
        return out
    dc = _only(there, s["dy"].float())
    if case["act"]:
        dc = dc * (sig + c * sig * (1 - sig))
    later = torch.cat([dc, torch.zeros(B, K - 1, D, device="cuda")], 1)
    full = torch.cat([torch.zeros(B, K - 1, D, device="cuda"), later], 1)
    dx = (full.unfold(1, K, 1) * s["w"].flip(-1)).sum(-1)     # of the state, then of the tokens
    if s["ds"] is not None:
        dx = dx.scatter_add(1, last, s["ds"])
    dw, db = (windows * dc.unsqueeze(-1)).sum((0, 1)), dc.sum((0, 1))
    out += [_only(there, dx[:, K - 1:]).to(dt), dw, db]
    return out + [dx[:, :K - 1]] if case["state"] else out


def _conv_step_plain(s):
    x = torch.cat([s["s"], s["x"].float().unsqueeze(1)], 1)
    c = (x * s["w"].t()).sum(1) + s["bias"]
    s["s"].copy_(x[:, 1:])
    return [(c * _sigmoid(c) if s["case"]["act"] else c).to(s["x"].dtype), s["s"]]


def _scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dim 1, by doubling."""
    step = 1
    while step < a.shape[1]:
        u = torch.cat([u[:, :step], u[:, step:] + a[:, step:] * u[:, :-step]], 1)
        a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
        step *= 2
    return u


def _delta(s):
    raw = s["dt"].float() + s["dt_bias"]
    return torch.clamp(raw, min=0) + torch.log1p(torch.exp(-raw.abs())), raw


def _scan_plain(s):
    case, dt = s["case"], s["u"].dtype
    there = _there(s)
    delta, raw = _delta(s)
    delta = _only(there, delta)
    u, Bm, Cm = (_only(there, s[n].float()) for n in ("u", "B", "C"))
    dB, dC = Bm.unsqueeze(2), Cm.unsqueeze(2)                  # [B, T, 1, N]
    a = torch.exp(delta.unsqueeze(-1) * s["A"])                # [B, T, D, N]
    b = (delta * u).unsqueeze(-1) * dB
    if s["h"] is not None:
        b = torch.cat([(b[:, 0] + a[:, 0] * s["h"]).unsqueeze(1), b[:, 1:]], 1)
    h = _scan(a, b)
    y = (h * dC).sum(-1) + u * s["D"]
    gate = None
    if s["z"] is not None:
        z = _only(there, s["z"].float())
        sig = _sigmoid(z)
        gate = z * sig
    out = [_only(there, y if gate is None else y * gate).to(dt), h[:, -1]]
    if not case["train"]:
        return out
    dy = _only(there, s["dy"].float())
    dz = None
    if gate is not None:
        dz = (dy * y * (sig + gate * (1 - sig))).to(dt)
        dy = dy * gate
    dh = dy.unsqueeze(-1) * dC
    if s["dh"] is not None:
        dh = torch.cat([dh[:, :-1], dh[:, -1:] + s["dh"].unsqueeze(1)], 1)
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    dh = _scan(later.flip(1), dh.flip(1)).flip(1)
    first = torch.zeros_like(h[:, 0]) if s["h"] is None else s["h"]
    w = dh * a * torch.cat([first.unsqueeze(1), h[:, :-1]], 1)
    sums = (dh * dB).sum(-1)
    du = delta * sums + dy * s["D"]
    ddelta = (w * s["A"]).sum(-1) + u * sums
    ddt = _only(there, ddelta * _sigmoid(raw))
    out += [_only(there, du).to(dt), ddt.to(dt), (w * delta.unsqueeze(-1)).sum((0, 1)),
            (dh * (delta * u).unsqueeze(-1)).sum(2).to(dt), (dy.unsqueeze(-1) * h).sum(2).to(dt),
            (dy * u).sum((0, 1)), ddt.sum((0, 1))]
    if dz is not None:
        out.append(dz)
    return out + [a[:, 0] * dh[:, 0]] if case["state"] else out


def _scan_step_plain(s):
    delta, _ = _delta(s)
    u = s["u"].float()
    a = torch.exp(delta.unsqueeze(-1) * s["A"])
    s["h"].copy_(a * s["h"] + (delta * u).unsqueeze(-1) * s["B"].float().unsqueeze(1))
    y = (s["h"] * s["C"].float().unsqueeze(1)).sum(-1) + u * s["D"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return [y.to(s["u"].dtype), s["h"]]


PLAIN = {"norm": _norm_plain, "conv": _conv_plain, "conv_step": _conv_step_plain,
         "scan": _scan_plain, "scan_step": _scan_step_plain}


def run(state):
    if own:
        return _run_own(state, state["case"])
    return PLAIN[state["case"]["op"]](state)


def _run_own(s, case):
    from constant_state_recurrence_gb300 import sanatan as S
    op = case["op"]
    if op == "norm":
        y, total, stats = S.sanatan_layer_norm_fwd(s["x"], s["weight"], s["bias"], s["residual"],
                                                   eps=EPS, want_stats=case["train"])
        out = [y] if s["residual"] is None else [y, total]
        if not case["train"]:
            return out
        d = S.sanatan_layer_norm_bwd(s["x"] if total is None else total, s["weight"], s["dy"],
                                     stats, ds=s["ds"])
        return out + [d["dx"], d["dweight"], d["dbias"]]
    act = ("silu" if case["act"] else None) if op.startswith("conv") else None
    if op == "conv_step":
        return [S.sanatan_causal_conv_step(s["s"], s["x"], s["w"], s["bias"], act), s["s"]]
    if op == "conv":
        y, last = S.sanatan_causal_conv_fwd(s["x"], s["w"], s["bias"], act, s0=s["s"],
                                            lens=s["lens"], want_state=True)
        if not case["train"]:
            return [y, last]
        d = S.sanatan_causal_conv_bwd(s["x"], s["w"], s["dy"], s["bias"], act, s0=s["s"],
                                      lens=s["lens"], ds_last=s["ds"], want_ds0=case["state"])
        out = [y, last, d["dx"], d["dw"], d["dbias"]]
        return out + [d["ds0"]] if case["state"] else out
    if op == "scan_step":
        y = S.sanatan_selective_scan_step(s["h"], s["u"], s["dt"], s["A"], s["B"], s["C"],
                                          D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
        return [y, s["h"]]
    train = case["train"]
    y, h, marks = S.sanatan_selective_scan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], D=s["D"],
                                               z=s["z"], dt_bias=s["dt_bias"], h0=s["h"],
                                               lens=s["lens"], want_state=True, want_marks=train)
    if not train:
        return [y, h]
    d = S.sanatan_selective_scan_bwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["dy"], marks,
                                     D=s["D"], z=s["z"], dt_bias=s["dt_bias"], lens=s["lens"],
                                     dh_last=s["dh"], want_dh0=case["state"])
    out = [y, h] + [d[n] for n in ("du", "ddt", "dA", "dB", "dC", "dD", "ddt_bias")]
    if s["z"] is not None:
        out.append(d["dz"])
    return out + [d["dh0"]] if case["state"] else out


def work(case):
    op, D = case["op"], case["D"]
    e = 4 if case["dtype"] == "f32" else 2
    if op == "norm":
        n, r = case["rows"] * D, 2 if case["residual"] else 0
        if not case["train"]:
            return dict(bytes=n * e * (2 + r) + 8 * D, flops=8 * n)
        return dict(bytes=n * e * (4 + r + r // 2) + 16 * D, flops=20 * n)
    B = case["B"]
    if op == "conv_step":
        K = case["K"]
        return dict(bytes=B * D * (2 * e + 8 * (K - 1)) + 4 * D * (K + 1),
                    flops=B * D * (2 * K + 5))
    if op == "scan_step":
        N = case["N"]
        return dict(bytes=B * D * (e * (4 if case["gated"] else 3) + 8 * N) + 4 * D * (N + 2)
                    + 2 * B * N * e, flops=B * D * (8 * N + 12))
    T, train = case["T"], case["train"]
    n = (sum(_lengths(B, T)) if case["ragged"] else B * T)    # tokens that are there
    if op == "conv":
        K = case["K"]
        state = 4 * B * (K - 1) * D * (2 if case["state"] else 1)
        params = 4 * D * (K + 1)
        if not train:
            return dict(bytes=n * D * e + B * T * D * e + state + params, flops=n * D * (2 * K + 5))
        return dict(bytes=2 * n * D * e + 2 * B * T * D * e + 2 * state + 2 * params,
                    flops=n * D * (8 * K + 16))
    N, z = case["N"], 1 if case["gated"] else 0
    state, params = 4 * B * D * N * (2 if case["state"] else 1), 4 * D * (N + 2)
    if not train:
        return dict(bytes=n * D * e * (2 + z) + B * T * D * e + 2 * n * N * e + state + params,
                    flops=n * D * (8 * N + 12))
    return dict(bytes=n * D * e * (3 + z) + B * T * D * e * (3 + z)
                + (2 * n + 2 * B * T) * N * e + 2 * state + 2 * params,
                flops=n * D * (28 * N + 40))


# The definitions in 64 bits: rows, windows tap by tap, and the scan token by token.

def _exact_norm(s):
    x = s["x"].double()
    if s["residual"] is not None:
        x = (x + s["residual"].double()).to(s["x"].dtype).double()
    weight = s["weight"].double()
    mean = x.sum(-1, keepdim=True) / x.shape[-1]
    var = ((x - mean) ** 2).sum(-1, keepdim=True) / x.shape[-1]
    hat = (x - mean) / (var + EPS) ** 0.5
    out = [hat * weight + s["bias"].double()]
    if s["residual"] is not None:
        out.append(x)
    if not s["case"]["train"]:
        return out
    dy = s["dy"].double()
    g = dy * weight
    dx = (g - g.mean(-1, keepdim=True) - hat * (g * hat).mean(-1, keepdim=True)) \
        / (var + EPS) ** 0.5
    if s["ds"] is not None:
        dx = dx + s["ds"].double()
    return out + [dx, (hat * dy).sum(0), dy.sum(0)]


def _exact_conv(s):
    case = s["case"]
    step = case["op"] == "conv_step"
    B, D, K, T = case["B"], case["D"], case["K"], 1 if step else case["T"]
    x = s["x"].double().view(B, T, D) if step else s["x"].double()
    lens = [T] * B if step or s["lens"] is None else s["lens"].tolist()
    w, bias = s["w"].double(), s["bias"].double()
    y, last = torch.zeros(B, T, D, dtype=torch.float64, device="cuda"), []
    train = not step and case["train"]
    if train:
        dx, dw = torch.zeros_like(y), torch.zeros_like(w)
        db, ds0 = torch.zeros_like(bias), []
    for b, n in enumerate(lens):
        first = x.new_zeros(K - 1, D) if s["s"] is None else s["s"][b].double()
        row = torch.cat([first, x[b, :n]])
        c = bias + sum(w[:, k] * row[k:k + n] for k in range(K))
        sig = torch.sigmoid(c)
        y[b, :n] = c * sig if case["act"] else c
        last.append(row[n:])
        if train:
            dc = s["dy"][b, :n].double()
            if case["act"]:
                dc = dc * sig * (1 + c * (1 - sig))
            d = torch.zeros_like(row)
            for k in range(K):
                d[k:k + n] += w[:, k] * dc
                dw[:, k] += (row[k:k + n] * dc).sum(0)
            db += dc.sum(0)
            if s["ds"] is not None:
                d[n:] += s["ds"][b].double()
            dx[b, :n] = d[K - 1:]
            ds0.append(d[:K - 1])
    out = [y[:, 0] if step else y, torch.stack(last)]
    if not train:
        return out
    out += [dx, dw, db]
    return out + [torch.stack(ds0)] if case["state"] else out


def _exact_scan(s):
    case = s["case"]
    step = case["op"] == "scan_step"
    T, train = 1 if step else case["T"], not step and case["train"]
    u, raw, Bm, Cm = (s[n].double() for n in ("u", "dt", "B", "C"))
    if step:
        u, raw, Bm, Cm = (t.unsqueeze(1) for t in (u, raw, Bm, Cm))
    A, skip = s["A"].double(), s["D"].double()
    raw = raw + s["dt_bias"].double()
    delta = torch.nn.functional.softplus(raw, threshold=60)
    z = None if s["z"] is None else s["z"].double().view(u.shape)
    gone = None
    if not step and s["lens"] is not None:
        gone = (torch.arange(T, device="cuda")[None, :] >= s["lens"][:, None]).unsqueeze(-1)
        delta, u, Bm, Cm = (t.masked_fill(gone, 0) for t in (delta, u, Bm, Cm))
    B, N = case["B"], case["N"]
    h = u.new_zeros(B, case["D"], N) if s["h"] is None else s["h"].double()
    every = u.new_empty(B, T + 1, case["D"], N) if train else None
    y = torch.empty_like(u)
    for t in range(T):
        if train:
            every[:, t] = h
        a = torch.exp(delta[:, t, :, None] * A)
        h = a * h + (delta[:, t] * u[:, t])[..., None] * Bm[:, t, None]
        y[:, t] = (h @ Cm[:, t, :, None])[..., 0]
    y = y + skip * u
    gate = None if z is None else z * torch.sigmoid(z)
    o = y if gate is None else y * gate
    if gone is not None:
        o = o.masked_fill(gone, 0)
    if step:
        return [o[:, 0], h]
    if not train:
        return [o, h]
    last = h
    every[:, T] = h
    dy = s["dy"].double()
    if gone is not None:
        dy = dy.masked_fill(gone, 0)
    dz = None
    if gate is not None:
        sig = torch.sigmoid(z)
        dz = dy * y * sig * (1 + z * (1 - sig))
        if gone is not None:
            dz = dz.masked_fill(gone, 0)
        dy = dy * gate
    g = torch.zeros_like(h) if s["dh"] is None else s["dh"].double()
    du, ddelta = torch.empty_like(u), torch.empty_like(u)
    dB, dC, dA = torch.empty_like(Bm), torch.empty_like(Cm), torch.zeros_like(A)
    for t in range(T - 1, -1, -1):
        g = g + dy[:, t, :, None] * Cm[:, t, None]
        dC[:, t] = (dy[:, t, None] @ every[:, t + 1])[:, 0]
        dB[:, t] = ((delta[:, t] * u[:, t])[:, None] @ g)[:, 0]
        sums = (g @ Bm[:, t, :, None])[..., 0]
        du[:, t] = delta[:, t] * sums
        g = g * torch.exp(delta[:, t, :, None] * A)
        w = g * every[:, t]
        ddelta[:, t] = u[:, t] * sums + (w * A).sum(-1)
        dA += (w * delta[:, t, :, None]).sum(0)
    du = du + dy * skip
    ddt = ddelta * torch.sigmoid(raw)
    if gone is not None:
        du, ddt = du.masked_fill(gone, 0), ddt.masked_fill(gone, 0)
    out = [o, last, du, ddt, dA, dB, dC, (dy * u).sum((0, 1)), ddt.sum((0, 1))]
    if dz is not None:
        out.append(dz)
    return out + [g] if case["state"] else out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    return _exact_conv(s) if op.startswith("conv") else _exact_scan(s)
