"""The operators around the scan in 64 bits, from their definitions, and how
far a float32 computation of them may be off.

Each function returns (values, bounds): dicts of float64 CPU tensors with the
same keys.  A bound counts the roundings of a 32-bit evaluation in units of
U = 2^-24 and carries them through the formula beside the values (an error e
of h leaves an error |a| e of a h, and so on); the rounding of an output to
its own type is added by ``check``.

What the counts stand for: an elementary float32 operation is off by U
relative.  The logistic function and its complement, computed with the SFU's
exponential (2 ulp) and reciprocal (1 ulp): at most GATE U, plus |v| U from
rounding the exponent's argument.  Sums are counted by their depth.
"""
import torch

U = 2.0 ** -24
GATE = 12


def sig(v):
    return 1 / (1 + torch.exp(-v))


def check(got, want, bound, what):
    """|got - want| <= bound + half a step of got's type, element by element
    (non-finite values have to be the same)."""
    assert got.shape == want.shape, f"{what}: {tuple(got.shape)}, not {tuple(want.shape)}"
    dt = got.dtype
    g = got.detach().cpu().double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(g), fine), f"{what}: finite in other places"
    tiny = 2.0 ** -126  # results below the smallest normal number may be flushed
    lim = bound * (1 + 2.0 ** -7) + torch.finfo(dt).eps / 2 * want.abs() + tiny
    over = torch.where(fine, (g - want).abs() - lim, torch.zeros_like(g))
    if over.numel() and float(over.max()) > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: element {i} is {g.flatten()[i]:.9g}, not {want.flatten()[i]:.9g} "
                             f"(bound {lim.flatten()[i]:.3g}); {int((over > 0).sum())} of {over.numel()} are off")


# ------------------------------------------------------------------- the norm


def norm_depth(dim):
    """Additions on the longest way to a sum over dim channels."""
    return 128 + dim / 16


def norm_fwd(x, weight, bias, eps, rms):
    """x (B, D, L) float64."""
    D = x.shape[1]
    K = norm_depth(D) * U
    m = torch.zeros_like(x[:, :1]) if rms else x.mean(1, keepdim=True)
    em = torch.zeros_like(m) if rms else K * x.abs().mean(1, keepdim=True)
    c = x - m
    var = c.square().mean(1, keepdim=True)
    r = (var + eps).rsqrt()
    # variance: its own sum, and the mean's error (squares are stationary there: second order)
    evar = K * var + em.square() + 4 * U * (c.abs() * (x.abs() + m.abs())).mean(1, keepdim=True)
    er = r * (0.5 * evar / (var + eps) + 6 * U)
    w = torch.ones(D, dtype=x.dtype) if weight is None else weight
    b = torch.zeros(D, dtype=x.dtype) if bias is None else bias
    w, b = w[:, None], b[:, None]
    y = c * r * w + b
    ec = em + U * (x.abs() + m.abs())
    ey = (ec * r + c.abs() * er) * w.abs() + 4 * U * ((c * r * w).abs() + b.abs())
    return ({"y": y, "mean": m[:, 0], "rstd": r[:, 0]}, {"y": ey, "mean": em[:, 0] + U * m[:, 0].abs(), "rstd": er[:, 0]})


def norm_bwd(x, dy, mean, rstd, weight):
    """Gradients from saved mean (None: RMS form) and rstd, (B, L)."""
    B, D, L = x.shape
    K = norm_depth(D) * U
    r = rstd[:, None]
    m = torch.zeros_like(r) if mean is None else mean[:, None]
    w = (torch.ones(D, dtype=x.dtype) if weight is None else weight)[:, None]
    xh = (x - m) * r
    exh = U * (x.abs() + m.abs()) * r + U * xh.abs()
    v = dy * w
    ev = U * v.abs()
    c2 = (v * xh).mean(1, keepdim=True)
    ec2 = K * (v * xh).abs().mean(1, keepdim=True) + (v.abs() * exh + ev * xh.abs()).mean(1, keepdim=True)
    c1 = torch.zeros_like(c2) if mean is None else v.mean(1, keepdim=True)
    ec1 = torch.zeros_like(c2) if mean is None else K * v.abs().mean(1, keepdim=True)
    dx = (v - c1 - xh * c2) * r
    edx = r * (ev + ec1 + exh * c2.abs() + xh.abs() * ec2) + 6 * U * r * (v.abs() + c1.abs() + (xh * c2).abs())
    # the sums over steps: at most 592 .. 1184 partial sums of B L terms
    Ks = (2 * (B * L) ** 0.5 + 256) * U
    t = dy * xh
    return ({"dx": dx, "dweight": t.sum((0, 2)), "dbias": dy.sum((0, 2))},
            {"dx": edx, "dweight": Ks * t.abs().sum((0, 2)) + (dy.abs() * exh + U * t.abs()).sum((0, 2)),
             "dbias": Ks * dy.abs().sum((0, 2))})


# -------------------------------------------------------- the causal convolution


def _since_start(reset, B, L):
    """(B, L): steps of the same sequence before each step; the state counts
    while no sequence has started in the row."""
    far = 64
    out = torch.empty((B, L), dtype=torch.long)
    for b in range(B):
        n = far
        for t in range(L):
            n = 0 if reset is not None and reset[b, t] else n
            out[b, t] = n
            n += 1
    return out


def _windows(x, W, initial_state, reset):
    """(B, D, L, W) of taps, zero where none is taken, and (B, 1, L, W) truth values."""
    B, D, L = x.shape
    h0 = torch.zeros((B, D, W - 1), dtype=x.dtype) if initial_state is None else initial_state
    xs = torch.cat([h0, x], 2)
    since = _since_start(reset, B, L)
    seen = (torch.arange(W - 1, -1, -1) <= since[..., None])[:, None]
    return torch.where(seen, xs.unfold(2, W, 1), torch.zeros((), dtype=x.dtype)), seen, xs


def conv_fwd(x, weight, bias, silu, initial_state=None, reset=None):
    B, D, L = x.shape
    W = weight.shape[1]
    win, seen, xs = _windows(x, W, initial_state, reset)
    w = weight[:, None]
    b = torch.zeros(D, dtype=x.dtype) if bias is None else bias
    p = (win * w).sum(3) + b[:, None]
    ep = (W + 1) * U * ((win * w).abs().sum(3) + b.abs()[:, None])
    y, ey = p, ep
    if silu:
        y = p * sig(p)
        ey = 1.1 * ep + (GATE + 2 + p.abs()) * U * y.abs()
    last = xs[..., L:]
    if L:
        far = _since_start(reset, B, L)[:, None, -1:]
        last = torch.where(torch.arange(W - 2, -1, -1) <= far, last, torch.zeros((), dtype=x.dtype))
    return {"y": y, "last": last, "p": p}, {"y": ey, "last": torch.zeros_like(last), "p": ep}


def conv_bwd(x, weight, bias, silu, dy, initial_state=None, reset=None, d_last=None):
    B, D, L = x.shape
    W = weight.shape[1]
    win, seen, xs = _windows(x, W, initial_state, reset)
    v, e = conv_fwd(x, weight, bias, silu, initial_state, reset)
    p, ep = v["p"], e["p"]
    q, eq = dy, torch.zeros_like(dy)
    if silu:
        s = sig(p)
        q = dy * s * (1 + p * (1 - s))
        # |silu''| <= 1/2; silu' is a product of the logistic function and 1 + p (1 - s)
        eq = dy.abs() * (0.5 * ep + (2 * GATE + 4 + 2 * p.abs()) * U * s * (1 + (p * (1 - s)).abs()))
    qt = torch.where(seen, q[..., None], torch.zeros((), dtype=x.dtype))
    eqt = torch.where(seen, eq[..., None], torch.zeros((), dtype=x.dtype))
    dxs, mag, err = torch.zeros_like(xs), torch.zeros_like(xs), torch.zeros_like(xs)
    for j in range(W):
        dxs[..., j:j + L] += qt[..., j] * weight[:, j, None]
        mag[..., j:j + L] += (qt[..., j] * weight[:, j, None]).abs()
        err[..., j:j + L] += eqt[..., j] * weight[:, j, None].abs()
    if d_last is not None:  # the last state's elements are inputs
        _, sn, _ = _windows(x, W, initial_state, reset)
        kept = torch.ones((B, 1, W - 1), dtype=torch.bool)
        if L:
            kept = torch.arange(W - 2, -1, -1) <= _since_start(reset, B, L)[:, None, -1:]
        g = torch.where(kept, d_last, torch.zeros((), dtype=x.dtype))
        dxs[..., L:] += g
        mag[..., L:] += g.abs()
    err = err + (W + 2) * U * mag
    # sums over the steps: 128 threads or more for a channel, each with its
    # share of the terms, whole vectors of 8 or 16, then the threads' sums
    Ks = (B * (L + 14) / 128 + 64) * U
    t = q[..., None] * win
    return ({"dx": dxs[..., W - 1:], "dinitial_state": dxs[..., :W - 1], "dweight": t.sum((0, 2)), "dbias": q.sum((0, 2))},
            {"dx": err[..., W - 1:], "dinitial_state": err[..., :W - 1],
             "dweight": Ks * t.abs().sum((0, 2)) + (eq[..., None] * win.abs()).sum((0, 2)),
             "dbias": Ks * q.abs().sum((0, 2)) + eq.sum((0, 2))})


# ------------------------------------------------------- the gated recurrence


def _gate(g, sigmoid):
    """a, 1 - a and their relative errors in units of U."""
    if not sigmoid:
        return g, 1 - g, torch.zeros_like(g), torch.ones_like(g)
    e = GATE + g.abs()
    return sig(g), sig(-g), e, e


def glr_fwd(x, g, z=None, sigmoid=True, couple=False, initial_state=None, reset=None):
    B, D, L = x.shape
    a, keep, ea, ek = _gate(g, sigmoid)
    b = keep * x if couple else x
    eb = (ek + 2) * U * b.abs() if couple else torch.zeros_like(b)
    h = torch.zeros((B, D), dtype=x.dtype) if initial_state is None else initial_state.clone()
    e, mag = torch.zeros_like(h), h.abs()
    out, err, before, ebefore, mags = [], [], [], [], []
    for t in range(L):
        if reset is not None:
            cut = reset[:, t:t + 1] != 0
            h, e, mag = (torch.where(cut, torch.zeros((), dtype=x.dtype), v) for v in (h, e, mag))
        before.append(h), ebefore.append(e)
        # the step's product is rounded once more, and again each time its factor is
        # folded into a product over lanes or warps: two more units a step cover them
        # (a step belongs to at most one such product per level, and the levels' own
        # roundings, some 12 in all, are paid once: the 12 U of the sum below)
        e = a[..., t].abs() * e + (ea[..., t] + 4) * U * a[..., t].abs() * mag + eb[..., t] + 12 * U * b[..., t].abs()
        mag = a[..., t].abs() * mag + b[..., t].abs()
        h = a[..., t] * h + b[..., t]
        out.append(h), err.append(e + 2 * U * mag)
    st = lambda v: torch.stack(v, 2) if v else torch.zeros_like(x)  # noqa: E731
    H, E = st(out), st(err)
    y, ey = H, E
    if z is not None:
        sz = z * sig(z)
        y, ey = H * sz, E * sz.abs() + (GATE + 3 + z.abs()) * U * (H * sz).abs()
    return ({"y": y, "last": h, "h": H, "before": st(before)},
            {"y": ey, "last": e + 2 * U * mag, "h": E, "before": st(ebefore)})


def glr_bwd(x, g, dy, z=None, sigmoid=True, couple=False, initial_state=None, reset=None, d_last=None):
    B, D, L = x.shape
    v, e = glr_fwd(x, g, z, sigmoid, couple, initial_state, reset)
    a, keep, ea, ek = _gate(g, sigmoid)
    dh, edh, dz, edz = dy, torch.zeros_like(dy), None, None
    if z is not None:
        s = sig(z)
        dh = dy * z * s
        edh = (GATE + 2 + z.abs()) * U * dh.abs()
        sl = s * (1 + z * (1 - s))
        esl = (2 * GATE + 6 + 2 * z.abs()) * U * s * (1 + (z * (1 - s)).abs())
        dz = dy * v["h"] * sl
        edz = (dy * sl).abs() * e["h"] + (dy * v["h"]).abs() * esl + 4 * U * dz.abs()
    m = torch.zeros((B, D), dtype=x.dtype) if d_last is None else d_last.clone()
    em, mag = torch.zeros_like(m), m.abs()
    lam, elam = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(L - 1, -1, -1):
        lam[..., t] = dh[..., t] + m
        el = edh[..., t] + em + 2 * U * (dh[..., t].abs() + mag)
        elam[..., t] = el
        ma = dh[..., t].abs() + mag
        m = a[..., t] * lam[..., t]
        em = a[..., t].abs() * (edh[..., t] + em) + (ea[..., t] + 16) * U * a[..., t].abs() * ma
        mag = a[..., t].abs() * ma
        if reset is not None:
            cut = reset[:, t:t + 1] != 0
            m, em, mag = (torch.where(cut, torch.zeros((), dtype=x.dtype), q) for q in (m, em, mag))
    slope = v["before"] - x if couple else v["before"]
    eslope = e["before"] + 3 * U * (v["before"].abs() + (x.abs() if couple else 0))
    da = lam * slope
    eda = elam * slope.abs() + lam.abs() * eslope + 2 * U * da.abs()
    dg, edg = da, eda
    if sigmoid:
        dg = da * a * keep
        edg = (a * keep).abs() * eda + (ea + ek + 4) * U * dg.abs()
    dx, edx = (lam * keep, elam * keep.abs() + (ek + 2) * U * (lam * keep).abs()) if couple else (lam, elam)
    return ({"dx": dx, "dg": dg, "dz": dz, "dinitial_state": m},
            {"dx": edx, "dg": edg, "dz": edz, "dinitial_state": em + 2 * U * mag})
