"""The operators around the selective scan, as cases to measure: normalisation
over the channels, the causal depthwise convolution, and the gated linear
recurrence, each in the library's (batch, dim, L) layout, forward, backward
and (convolution, recurrence) as one decoding step.

A case is a dict of sizes and flags.  ``prepare`` makes its inputs on the GPU
from a seed, ``run`` takes one pass through the operator (plain torch
operations in 32 bits, or the library's calls where ``own`` is true), ``exact``
gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-5


def case(name, op, batch, dim, len, dtype, **flags):
    c = {"name": name, "op": op, "batch": batch, "dim": dim, "len": len, "dtype": dtype}
    c.update(flags)
    return c


def listed():
    return [
        # Decoding, 8 sequences: the norm before a layer of width 768. Latency.
        case("norm_rows_decode", "norm_fwd", 8, 768, 1, "bf16", rms=False),
        # Training, 8 x 2048 tokens of the residual stream (one row each).
        case("norm_rows_bwd", "norm_bwd", 16384, 768, 1, "bf16", rms=False),
        # The scan's output (batch, dim, L) normalised before out_proj.
        case("norm_steps_fwd", "norm_fwd", 8, 1536, 2048, "bf16", rms=False),
        # The same in training: fp32, RMS form, sizes that nothing divides.
        case("norm_steps_bwd_odd", "norm_bwd", 3, 1000, 4099, "fp32", rms=True),
        # Prefill or training forward: the conv1d between in_proj and the scan.
        case("conv_fwd", "conv_fwd", 8, 1536, 2048, "bf16", width=4, silu=True, packed=0, state=False),
        case("conv_bwd", "conv_bwd", 8, 1536, 2048, "bf16", width=4, silu=True, packed=0, state=False),
        # Packed sequences of about 500 steps, continued from a state, odd length.
        case("conv_packed", "conv_fwd", 2, 1024, 20011, "bf16", width=5, silu=True, packed=500, state=True),
        # One decoding step of 8 sequences. Latency.
        case("conv_step", "conv_step", 8, 1536, 1, "bf16", width=4, silu=True),
        # A long input read once, its last state kept (the genomic shape).
        case("recurrence_long", "glr_fwd", 4, 1024, 100000, "bf16", sigmoid=True, couple=True, gated=False, packed=0,
             state=False),
        # A training step's forward and backward with the output gate.
        case("recurrence_train", "glr_train", 8, 1536, 2048, "bf16", sigmoid=True, couple=True, gated=True, packed=0,
             state=False),
        # Packed sequences from a state, decays given, fp32, odd sizes.
        case("recurrence_packed", "glr_fwd", 3, 1000, 4099, "fp32", sigmoid=False, couple=False, gated=False,
             packed=300, state=True),
        # One decoding step of 8 sequences. Latency.
        case("recurrence_step", "glr_step", 8, 1536, 1, "bf16", sigmoid=True, couple=True, gated=True),
    ]


def draw(rng):
    """Batches 1..32, widths 48..4096, lengths 1..65536 (rows: up to 32768 of
    them), at most 24 M elements, half of the sizes left odd."""
    def log_int(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        n = min(max(n, lo), hi)
        return n if rng.random() < 0.5 or n < 16 else n // 8 * 8

    op = rng.choice(["norm_rows_fwd", "norm_rows_bwd", "norm_fwd", "norm_bwd", "conv_fwd", "conv_bwd", "conv_step",
                     "glr_fwd", "glr_train", "glr_step"])
    dim = log_int(48, 4096)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    most = 24_000_000
    c = {"dim": dim, "dtype": dtype}
    if op in ("norm_rows_fwd", "norm_rows_bwd"):
        c.update(op=op.replace("_rows", ""), batch=log_int(1, min(32768, most // dim)), len=1, rms=rng.random() < 0.5)
    elif op in ("conv_step", "glr_step"):
        c.update(op=op, batch=log_int(1, 256), len=1)
    else:
        batch = log_int(1, 32)
        c.update(op=op, batch=batch, len=log_int(1, min(65536, max(2, most // (dim * batch)))))
    if op in ("norm_fwd", "norm_bwd"):
        c["rms"] = rng.random() < 0.5
    if op.startswith("conv"):
        c.update(width=rng.choice([2, 3, 4, 4, 4, 5, 6, 7, 8]), silu=rng.random() < 0.8)
    if op.startswith("glr"):
        c.update(sigmoid=rng.random() < 0.7, couple=rng.random() < 0.6, gated=rng.random() < 0.5)
    if op in ("conv_fwd", "conv_bwd", "glr_fwd", "glr_train"):
        c.update(packed=rng.choice([0, 0, 7, 150, 2000]), state=rng.random() < 0.5)
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    B, D, L, dt = case["batch"], case["dim"], case["len"], DTYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, dtype=dt, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale + shift).to(dtype)

    f32 = torch.float32
    s = {"case": case, "op": op}
    full = (B, D) if op.endswith("_step") else (B, D, L)
    s["x"] = normal(*full)
    if op.startswith("norm"):
        s["x"] = s["x"] * 2 + 0.5  # activations with an offset of their own
        s["weight"] = normal(D, dtype=f32, scale=0.1, shift=1.0)
        s["bias"] = None if case["rms"] else normal(D, dtype=f32, scale=0.1)
        if op == "norm_bwd":  # what a forward pass kept
            x = s["x"].double()
            m = torch.zeros((B, L), dtype=torch.float64, device="cuda") if case["rms"] else x.mean(1)
            s["rstd"] = ((x - m[:, None]).square().mean(1) + EPS).rsqrt().float()
            s["mean"] = None if case["rms"] else m.float()
            s["dy"] = normal(B, D, L)
    elif op.startswith("conv"):
        W = case["width"]
        s["weight"] = normal(D, W, dtype=f32, scale=W ** -0.5)
        s["bias"] = normal(D, dtype=f32, scale=0.1)
        if op == "conv_step":
            s["state"] = normal(B, D, W - 1)
        else:
            s["h0"] = normal(B, D, W - 1) if case["state"] else None
        if op == "conv_bwd":
            s["dy"] = normal(B, D, L)
    else:
        # Forget gates open most of the time: decays between about 0.5 and 0.999.
        g = torch.randn(full, generator=gen, device="cuda") * 1.5 + 3.0
        s["g"] = (g if case["sigmoid"] else torch.sigmoid(g)).to(dt)
        s["z"] = normal(*full) if case["gated"] else None
        if op == "glr_step":
            s["state"] = normal(B, D, dtype=f32)
        else:
            s["h0"] = normal(B, D, dtype=f32) if case["state"] else None
        if op == "glr_train":
            s["dy"] = normal(B, D, L)
    if case.get("packed"):
        # One starts wherever a sequence of that mean length ends.
        s["reset"] = (torch.rand((B, L), generator=gen, device="cuda") < 1.0 / case["packed"]).to(torch.uint8)
    else:
        s["reset"] = None
    return s


# ------------------------------------------------------------------ the calls


def run(s):
    if own:
        return _run_own(s)
    return PLAIN[s["op"]](s)


def _run_own(s):
    import selective_state_space_41_b200 as ss
    c, op = s["case"], s["op"]
    if op == "norm_fwd":
        return ss.layer_norm_fwd(s["x"], s["weight"], s["bias"], eps=EPS, rms=c["rms"])
    if op == "norm_bwd":
        g = ss.layer_norm_bwd(s["x"], s["dy"], s["rstd"], mean=s["mean"], weight=s["weight"], bias=s["bias"],
                              rms=c["rms"])
        return {k: g[k] for k in ("dx", "dweight", "dbias")}
    if op == "conv_fwd":
        return ss.causal_conv_fwd(s["x"], s["weight"], s["bias"], silu=c["silu"], initial_state=s["h0"],
                                  reset=s["reset"], return_last_state=True)
    if op == "conv_bwd":
        g = ss.causal_conv_bwd(s["x"], s["weight"], s["dy"], bias=s["bias"], silu=c["silu"], initial_state=s["h0"],
                               reset=s["reset"])
        return {k: g[k] for k in ("dx", "dweight", "dbias", "dinitial_state")}
    if op == "conv_step":
        y = ss.causal_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], silu=c["silu"])
        return y, s["state"]
    flags = {"gate_sigmoid": c["sigmoid"], "couple": c["couple"]}
    if op == "glr_fwd":
        return ss.gated_recurrence_fwd(s["x"], s["g"], z=s["z"], initial_state=s["h0"], reset=s["reset"],
                                       return_last_state=True, **flags)
    if op == "glr_train":
        y, ckpt = ss.gated_recurrence_fwd(s["x"], s["g"], z=s["z"], initial_state=s["h0"], reset=s["reset"],
                                          return_ckpt=True, **flags)
        g = ss.gated_recurrence_bwd(s["x"], s["g"], s["dy"], ckpt, z=s["z"], reset=s["reset"],
                                    return_dinitial_state=s["h0"] is not None, **flags)
        return {"y": y, **{k: g[k] for k in ("dx", "dg", "dz", "dinitial_state")}}
    y = ss.gated_recurrence_step(s["x"], s["g"], s["state"], z=s["z"], **flags)
    return y, s["state"]


# ------------------------------------------------------------ the plain forms


def _norm_fwd(s):
    x = s["x"].float()
    if not s["case"]["rms"]:
        x = x - x.mean(1, keepdim=True)
    y = x * (x.square().mean(1, keepdim=True) + EPS).rsqrt() * s["weight"][:, None]
    if s["bias"] is not None:
        y = y + s["bias"][:, None]
    return y.to(s["x"].dtype)


def _norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = (x if s["mean"] is None else x - s["mean"][:, None]) * rstd
    wdy = dy * s["weight"][:, None]
    dx = wdy - xh * (wdy * xh).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - wdy.mean(1, keepdim=True)
    dx = dx * rstd
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum((0, 2)),
            "dbias": None if s["bias"] is None else dy.sum((0, 2))}


def _steps_since_start(s):
    """(B, L): how many steps of its own sequence lie before each step; the
    steps before the row count where no sequence has started in it yet."""
    B, L = s["case"]["batch"], s["case"]["len"]
    t = torch.arange(L, device="cuda").expand(B, L)
    if s["reset"] is None:
        return t + 64
    last = torch.where(s["reset"] != 0, t, -64).cummax(1).values
    return t - last


def _taps(s):
    """x behind its state, (B, D, L + W - 1) in 32 bits, and how far back each
    step may look, (B, 1, L)."""
    x, W = s["x"], s["case"]["width"]
    head = s["h0"] if s["h0"] is not None else x.new_zeros((*x.shape[:2], W - 1))
    return torch.cat([head, x], 2).float(), _steps_since_start(s)[:, None]


def _conv_pre(s):
    xs, since = _taps(s)
    W, L = s["case"]["width"], s["case"]["len"]
    seen = torch.arange(W - 1, -1, -1, device="cuda") <= since[..., None]  # (B, 1, L, W)
    return ((xs.unfold(2, W, 1) * seen) * s["weight"][:, None]).sum(3) + s["bias"][:, None], xs, seen


def _conv_fwd(s):
    p, xs, _ = _conv_pre(s)
    y = p * torch.sigmoid(p) if s["case"]["silu"] else p
    W, L = s["case"]["width"], s["case"]["len"]
    # the last W - 1 inputs; those before the last start are zero
    back = torch.arange(W - 2, -1, -1, device="cuda")
    kept = back <= _steps_since_start(s)[:, None, -1:]
    return y.to(s["x"].dtype), (xs[..., L:] * kept).to(s["x"].dtype)


def _conv_bwd(s):
    p, xs, seen = _conv_pre(s)
    dp = s["dy"].float()
    if s["case"]["silu"]:
        sg = torch.sigmoid(p)
        dp = dp * sg * (1 + p * (1 - sg))
    W, L = s["case"]["width"], s["case"]["len"]
    per_tap = dp[..., None] * seen  # (B, D, L, W)
    dw = (per_tap * xs.unfold(2, W, 1)).sum((0, 2))
    dxs = torch.zeros_like(xs)
    for j in range(W):
        dxs[..., j:j + L] += per_tap[..., j] * s["weight"][:, j, None]
    dt = s["x"].dtype
    return {"dx": dxs[..., W - 1:].to(dt), "dweight": dw, "dbias": dp.sum((0, 2)),
            "dinitial_state": dxs[..., :W - 1].to(dt) if s["h0"] is not None else None}


def _conv_step(s):
    x, state = s["x"], s["state"]
    xs = torch.cat([state, x[..., None]], 2)
    p = (xs.float() * s["weight"]).sum(2) + s["bias"]
    y = p * torch.sigmoid(p) if s["case"]["silu"] else p
    state.copy_(xs[..., 1:])
    return y.to(x.dtype), state


def _scan(a, b):
    """h_t = a_t h_(t-1) + b_t along the last axis by doubling: after the pass
    of distance d, (a_t, b_t) stand for the last 2 d steps up to t."""
    d = 1
    while d < a.shape[-1]:
        b = torch.cat([b[..., :d], a[..., d:] * b[..., :-d] + b[..., d:]], -1)
        a = torch.cat([a[..., :d], a[..., d:] * a[..., :-d]], -1)
        d *= 2
    return a, b


def _gates(s):
    a = s["g"].float()
    keep = 1 - a
    if s["case"]["sigmoid"]:
        a, keep = torch.sigmoid(a), torch.sigmoid(-a)
    x = s["x"].float()
    return a, keep, (keep * x if s["case"]["couple"] else x)


def _glr_states(s):
    a, keep, b = _gates(s)
    carried = a if s["reset"] is None else a * (s["reset"] == 0)[:, None]
    prod, h = _scan(carried, b)
    if s["h0"] is not None:
        h = h + prod * s["h0"][..., None]
    return a, keep, carried, h


def _glr_fwd(s):
    h = _glr_states(s)[3]
    y = h if s["z"] is None else h * (s["z"].float() * torch.sigmoid(s["z"].float()))
    return y.to(s["x"].dtype), h[..., -1].contiguous()


def _glr_train(s):
    a, keep, carried, h = _glr_states(s)
    dt, dy, dz = s["x"].dtype, s["dy"].float(), None
    y, dh = h, dy
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        y, dh, dz = h * (z * sg), dy * (z * sg), (dy * h * sg * (1 + z * (1 - sg))).to(dt)
    # the adjoint runs from the last step back, through the next step's decay
    nxt = torch.cat([carried[..., 1:], torch.zeros_like(carried[..., :1])], -1)
    lam = _scan(nxt.flip(-1), dh.flip(-1))[1].flip(-1)
    h0 = torch.zeros_like(h[..., 0]) if s["h0"] is None else s["h0"]
    before = torch.cat([h0[..., None], h[..., :-1]], -1)
    if s["reset"] is not None:
        before = before * (s["reset"] == 0)[:, None]
    x = s["x"].float()
    da = lam * (before - x) if s["case"]["couple"] else lam * before
    dg = da * a * keep if s["case"]["sigmoid"] else da
    dx = lam * keep if s["case"]["couple"] else lam
    return {"y": y.to(dt), "dx": dx.to(dt), "dg": dg.to(dt), "dz": dz,
            "dinitial_state": carried[..., 0] * lam[..., 0] if s["h0"] is not None else None}


def _glr_step(s):
    a, _, b = _gates(s)
    s["state"].copy_(a * s["state"] + b)
    y = s["state"]
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    return y.to(s["x"].dtype), s["state"]


PLAIN = {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "conv_fwd": _conv_fwd, "conv_bwd": _conv_bwd,
         "conv_step": _conv_step, "glr_fwd": _glr_fwd, "glr_train": _glr_train, "glr_step": _glr_step}


# --------------------------------------------------------------- the figures


def work(case):
    """Every input read once and every output written once."""
    B, D, L, e, op = case["batch"], case["dim"], case["len"], SIZE[case["dtype"]], case["op"]
    n, mask = B * D * L, B * L if case.get("packed") else 0
    if op == "norm_fwd":
        return {"bytes": 2 * n * e + (1 if case["rms"] else 2) * D * 4, "flops": 7 * n}
    if op == "norm_bwd":
        return {"bytes": 3 * n * e + (2 if case["rms"] else 4) * D * 4 + (1 if case["rms"] else 2) * B * L * 4,
                "flops": 12 * n}
    if op.startswith("conv"):
        W = case["width"]
        act = 5 if case["silu"] else 0
        small = D * (W + 1) * 4 + B * D * (W - 1) * e * (1 if op == "conv_fwd" else 0)
        if op == "conv_step":
            return {"bytes": 2 * n * e + 2 * B * D * (W - 1) * e + D * (W + 1) * 4, "flops": n * (2 * W + act)}
        given = B * D * (W - 1) * e if case["state"] else 0
        if op == "conv_fwd":
            return {"bytes": 2 * n * e + small + given + mask, "flops": n * (2 * W + act)}
        return {"bytes": 3 * n * e + 2 * small + 2 * given + mask, "flops": n * (6 * W + 2 * act)}
    z = 1 if case["gated"] else 0
    gate = (5 if case["sigmoid"] else 0) + (2 if case["couple"] else 0) + 6 * z
    if op == "glr_step":
        return {"bytes": (3 + z) * n * e + 8 * B * D, "flops": n * (2 + gate)}
    given = 4 * B * D if case["state"] else 0
    if op == "glr_fwd":
        return {"bytes": (3 + z) * n * e + 4 * B * D + given + mask, "flops": n * (2 + gate)}
    return {"bytes": (6 + 2 * z) * n * e + 2 * given + mask, "flops": n * (10 + 3 * gate)}


# ------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v) for k, v in s.items()}
    op = case["op"]
    if op.startswith("norm"):
        return _exact_norm(case, d)
    if op.startswith("conv"):
        return _exact_conv(case, d)
    return _exact_glr(case, d)


def _exact_norm(case, d):
    x, w = d["x"], d["weight"].view(1, -1, 1)
    B, D, L = x.shape
    if case["op"] == "norm_fwd":
        c = x if case["rms"] else x - x.sum(1, keepdim=True) / D
        y = c / torch.sqrt((c * c).sum(1, keepdim=True) / D + EPS) * w
        return y if d["bias"] is None else y + d["bias"].view(1, -1, 1)
    # Vector-Jacobian product of x -> (x - m) r w with m, r the saved values.
    r = d["rstd"].view(B, 1, L)
    xh = x * r if case["rms"] else (x - d["mean"].view(B, 1, L)) * r
    v = d["dy"] * w
    along = torch.einsum("bdl,bdl->bl", v, xh).view(B, 1, L) / D
    dx = v - xh * along
    if not case["rms"]:
        dx = dx - v.sum(1, keepdim=True) / D
    return {"dx": dx * r, "dweight": torch.einsum("bdl,bdl->d", d["dy"], xh),
            "dbias": None if d["bias"] is None else torch.einsum("bdl->d", d["dy"])}


def _exact_conv(case, d):
    W, L, op = case["width"], case["len"], case["op"]
    if op == "conv_step":
        x = torch.cat([d["state"], d["x"][..., None]], 2)
        p = torch.einsum("bdw,dw->bd", x, d["weight"]) + d["bias"]
        return (p / (1 + torch.exp(-p)) if case["silu"] else p), x[..., 1:]
    B, D, _ = d["x"].shape
    back = op == "conv_bwd"
    x, w, b = d["x"].requires_grad_(back), d["weight"].requires_grad_(back), d["bias"].requires_grad_(back)
    h0 = d["h0"]
    if h0 is not None:
        h0.requires_grad_(back)
    # The sequence that each step belongs to; the state belongs to the row's first.
    if d["reset"] is None:
        seq = torch.zeros((B, L + W - 1), dtype=torch.int64, device="cuda")
    else:
        seq = torch.cat([torch.zeros((B, W - 1), dtype=torch.int64, device="cuda"),
                         (d["reset"] != 0).long().cumsum(1)], 1)
    xs = torch.cat([h0 if h0 is not None else torch.zeros((B, D, W - 1), dtype=torch.float64, device="cuda"), x], 2)
    p = b.view(1, -1, 1).expand(B, D, L)
    for j in range(W):
        same = (seq[:, j:j + L] == seq[:, W - 1:]).double()[:, None]
        p = p + w[:, j].view(1, -1, 1) * xs[:, :, j:j + L] * same
    y = p / (1 + torch.exp(-p)) if case["silu"] else p
    if not back:
        return y, xs[:, :, L:] * (seq[:, L:] == seq[:, -1:]).double()[:, None]
    leaves = [x, w, b] + ([h0] if h0 is not None else [])
    g = torch.autograd.grad(y, leaves, d["dy"])
    return {"dx": g[0], "dweight": g[1], "dbias": g[2], "dinitial_state": g[3] if h0 is not None else None}


def _exact_recur(a, b, h0):
    """h_t = a_t h_(t-1) + b_t step by step: blocks of the row side by side
    from a zero state, then the state carried from block to block."""
    B, D, L = a.shape
    T = max(1, int(math.sqrt(L)))
    n = -(-L // T)
    pad = n * T - L
    a = torch.nn.functional.pad(a, (0, pad)).view(B, D, n, T)
    h = torch.nn.functional.pad(b, (0, pad)).view(B, D, n, T).clone()
    decay = a.clone()
    for t in range(1, T):
        h[..., t] += a[..., t] * h[..., t - 1]
        decay[..., t] *= decay[..., t - 1]
    carry = torch.zeros_like(a[:, :, 0, 0]) if h0 is None else h0.clone()
    for k in range(n):
        h[:, :, k] += decay[:, :, k] * carry[..., None]
        carry = h[:, :, k, -1]
    return h.reshape(B, D, n * T)[..., :L]


def _exact_glr(case, d):
    x, g = d["x"], d["g"]
    a = 1 / (1 + torch.exp(-g)) if case["sigmoid"] else g
    keep = 1 / (1 + torch.exp(g)) if case["sigmoid"] else 1 - g
    b = keep * x if case["couple"] else x
    sz, z = 1.0, d["z"]
    if z is not None:
        sz = z / (1 + torch.exp(-z))
    if case["op"] == "glr_step":
        h = a * d["state"] + b
        return h * sz, h
    carried = a if d["reset"] is None else torch.where(d["reset"][:, None] != 0, torch.zeros_like(a), a)
    h = _exact_recur(carried, b, d["h0"])
    if case["op"] == "glr_fwd":
        return h * sz, h[..., -1]
    dy = d["dy"]
    shifted = torch.zeros_like(carried)
    shifted[..., :-1] = carried[..., 1:]
    lam = _exact_recur(shifted.flip(2), (dy * sz).flip(2), None).flip(2)
    before = torch.zeros_like(h)
    before[..., 1:] = h[..., :-1]
    if d["h0"] is not None:
        before[..., 0] = d["h0"]
    # d h_t / d a_t: the carried state where one is carried, less the input where it is coupled
    slope = before if d["reset"] is None else torch.where(d["reset"][:, None] != 0, torch.zeros_like(before), before)
    if case["couple"]:
        slope = slope - x
    dz = None
    if z is not None:
        e = torch.exp(-z)
        dz = dy * h * ((1 + e + z * e) / (1 + e) ** 2)
    return {"y": h * sz, "dx": lam * keep if case["couple"] else lam,
            "dg": lam * slope * (a * keep if case["sigmoid"] else 1.0), "dz": dz,
            "dinitial_state": carried[..., 0] * lam[..., 0] if d["h0"] is not None else None}
