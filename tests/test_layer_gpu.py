"""The operators around the scan as a layer uses them: together with the scan
and with each other, trained through autograd, decoded step by step, captured
into graphs, on other streams and from several threads."""
import threading

import pytest
import torch

import layer_ref as R
import selective_state_space_41_b200 as ss
from test_norm_gpu import BF, F32, d64, rand

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


# ------------------------------------------------------- layers, in both forms


def plain_norm(x, w, b, rms):
    c = x if rms else x - x.mean(1, keepdim=True)
    y = c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w[:, None]
    return y if b is None else y + b[:, None]


def plain_conv(x, w, b, reset):
    W, L = w.shape[1], x.shape[2]
    since = R._since_start(reset, x.shape[0], L)
    seen = (torch.arange(W - 1, -1, -1) <= since[..., None])[:, None]
    win = torch.nn.functional.pad(x, (W - 1, 0)).unfold(2, W, 1)
    p = (win * seen * w[:, None]).sum(3) + b[:, None]
    return p * torch.sigmoid(p)


def plain_recurrence(x, g, z, reset):
    h, out = torch.zeros_like(x[..., 0]), []
    for t in range(x.shape[2]):
        keep = (1 - reset[:, t:t + 1].to(x.dtype))
        a = torch.sigmoid(g[..., t])
        h = a * keep * h + (1 - a) * x[..., t]
        out.append(h)
    h = torch.stack(out, 2)
    return h * z * torch.sigmoid(z)


def plain_scan(u, delta, A, Bm, C, D, z, reset):
    h, out = u.new_zeros(*u.shape[:2], A.shape[1]), []
    dl = torch.nn.functional.softplus(delta)
    for t in range(u.shape[2]):
        keep = (1 - reset[:, t:t + 1].to(u.dtype))[..., None]
        d = dl[..., t, None]
        h = torch.exp(d * A) * keep * h + d * Bm[:, None, :, t] * u[..., t, None]
        out.append((h * C[:, None, :, t]).sum(2))
    return (torch.stack(out, 2) + D[:, None] * u) * z * torch.sigmoid(z)


OPS = {
    "plain": (plain_norm, plain_conv, plain_recurrence, plain_scan),
    "library": (lambda x, w, b, rms: ss.layer_norm_fn(x, w, b, rms=rms),
                lambda x, w, b, reset: ss.causal_conv_fn(x, w, b, silu=True, reset=reset),
                lambda x, g, z, reset: ss.gated_recurrence_fn(x, g, z, couple=True, reset=reset),
                lambda u, d, A, B, C, D, z, reset: ss.selective_scan_fn(u, d, A, B, C, D=D, z=z, delta_softplus=True,
                                                                        reset=reset)),
}


def recurrent_layer(ops, p, x, reset):
    """x + W_out norm(recurrence(conv(W_in norm(x)))), gates and output gate from the normalised input."""
    norm, conv, recurrence, _ = ops
    y = norm(x, p["nw"], None, True)
    u = conv(p["W_in"] @ y, p["cw"], p["cb"], reset)
    h = recurrence(u, p["W_g"] @ y + 2, p["W_z"] @ y, reset)
    return x + p["W_out"] @ norm(h, p["ow"], p["ob"], False)


def mamba_layer(ops, p, x, reset):
    """x + W_out scan(conv(W_in norm(x))), the scan's delta, B and C from the convolved input."""
    norm, conv, _, scan = ops
    y = norm(x, p["nw"], p["nb"], False)
    u = conv(p["W_in"] @ y, p["cw"], p["cb"], reset)
    s = scan(u, p["W_dt"] @ u - 1, -torch.exp(p["A_log"]), p["W_B"] @ u, p["W_C"] @ u, p["D"], p["W_z"] @ y, reset)
    return x + p["W_out"] @ s


def parameters(d, e, n, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, k=1.0, m=0.0: torch.randn(s, generator=g, dtype=torch.float64) * k + m  # noqa: E731
    return {"nw": r(d, k=.2, m=1), "nb": r(d, k=.2), "ow": r(e, k=.2, m=1), "ob": r(e, k=.2), "cw": r(e, 4, k=.5),
            "cb": r(e, k=.2), "W_in": r(e, d, k=d ** -.5), "W_g": r(e, d, k=d ** -.5), "W_z": r(e, d, k=d ** -.5),
            "W_out": r(d, e, k=e ** -.5), "W_dt": r(e, e, k=.5 * e ** -.5), "W_B": r(n, e, k=e ** -.5),
            "W_C": r(n, e, k=e ** -.5), "A_log": torch.log(torch.arange(1, n + 1, dtype=torch.float64)).repeat(e, 1),
            "D": r(e)}


@pytest.mark.parametrize("layer", [recurrent_layer, mamba_layer])
@pytest.mark.parametrize("L", [48, 301])
def test_training_pass_of_a_layer(layer, L):
    """A layer's output and the gradients of all its parameters and its input
    agree with the 64-bit composition.

    Tolerance: every operator returns its result within about 2^-18 of its
    largest value here (the bounds of layer_ref.py, and 1e-5 for the scan), a
    gradient passes at most six of them and three products with rows of norm
    about one, whose own fp32 sums are smaller still; each may double an error
    that comes in.  2^-18 (1 + 2 + .. + 64) is 2^-11; held to 2^-11 of each
    tensor's largest value."""
    B, d, e, n = 2, 24, 40, 8
    x0 = rand(B, d, L, seed=L).double()
    reset = torch.zeros((B, L), dtype=torch.uint8)
    reset[0, L // 3] = reset[1, L - 2] = 1
    dy = rand(B, d, L, seed=L + 1).double()

    def run(kind, to):
        p = {k: to(v).requires_grad_() for k, v in parameters(d, e, n, 7).items()}
        x = to(x0).requires_grad_()
        prev = torch.backends.cuda.matmul.allow_tf32
        torch.backends.cuda.matmul.allow_tf32 = False
        try:
            y = layer(OPS[kind], p, x, reset if kind == "plain" else reset.cuda())
            y.backward(to(dy))
        finally:
            torch.backends.cuda.matmul.allow_tf32 = prev
        return {"y": y.detach(), "x": x.grad, **{k: v.grad for k, v in p.items()}}

    want = run("plain", lambda t: t.clone())
    got = run("library", lambda t: t.float().cuda())
    for k, w in want.items():
        assert (w is None) == (got[k] is None), k
        if w is not None:
            err = float((got[k].cpu().double() - w).abs().max()) / max(float(w.abs().max()), 1e-30)
            assert err <= 2.0 ** -11, f"{k}: {err:.2e}"


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_then_decode(dtype):
    """norm, convolution and recurrence over a prompt, their states then
    carried on one token at a time, against the 64-bit values of each operator
    on the inputs it was given."""
    B, D, L, W, start = 3, 72, 37, 4, 29
    x = rand(B, D, L, seed=1, dtype=dtype).cuda()
    w, b, cw, cb = (t.cuda() for t in (rand(D, seed=2, shift=1.0), rand(D, seed=3), rand(D, W, seed=4), rand(D, seed=5)))
    g, z = rand(B, D, L, seed=6, dtype=dtype, shift=2.0).cuda(), rand(B, D, L, seed=7, dtype=dtype).cuda()

    def check(got, ref, what):
        v, e = ref
        R.check(got, v, e, what)

    c = lambda t: t.cpu().double()  # noqa: E731
    y = ss.layer_norm_fwd(x[..., :start], w, b)
    u, conv_state = ss.causal_conv_fwd(y, cw, cb, silu=True, return_last_state=True)
    h, state = ss.gated_recurrence_fwd(u, g[..., :start], z[..., :start], couple=True, return_last_state=True)
    ys, us, hs = [y], [u], [h]
    for t in range(start, L):
        y = ss.layer_norm_fwd(x[..., t].contiguous(), w, b)  # (batch, dim): rows
        u = ss.causal_conv_step(y, cw, conv_state, bias=cb, silu=True)
        h = ss.gated_recurrence_step(u, g[..., t], state, z[..., t], couple=True)
        ys.append(y[..., None]), us.append(u[..., None]), hs.append(h[..., None])
    ys, us, hs = (torch.cat(v, 2) for v in (ys, us, hs))
    v, e = R.norm_fwd(c(x), c(w), c(b), 1e-5, False)
    check(ys, (v["y"], e["y"]), "norm")
    v, e = R.conv_fwd(c(ys), c(cw), c(cb), True)
    check(us, (v["y"], e["y"]), "convolution")
    assert torch.equal(c(conv_state), v["last"])
    v, e = R.glr_fwd(c(us), c(g), c(z), True, True)
    check(hs, (v["y"], e["y"]), "recurrence"), check(state, (v["last"], e["last"]), "state")


# ----------------------------------------------------- one training step, raw


def step_inputs(seed, B=2, D=200, L=333, dtype=BF):
    r = lambda *s, k: rand(*s, seed=10 * seed + k, dtype=dtype).cuda()  # noqa: E731
    f = lambda *s, k: rand(*s, seed=10 * seed + k).cuda()  # noqa: E731
    reset = torch.zeros((B, L), dtype=torch.uint8)
    reset[0, 100] = 1
    return {"x": r(B, D, L, k=1), "g": r(B, D, L, k=2), "z": r(B, D, L, k=3), "dy": r(B, D, L, k=4), "w": f(D, k=5),
            "b": f(D, k=6), "cw": f(D, 4, k=7), "cb": f(D, k=8), "reset": reset.cuda()}


def step(s, **kw):
    """Forward and backward of norm, convolution and recurrence by the raw calls."""
    y, mean, rstd = ss.layer_norm_fwd(s["x"], s["w"], s["b"], return_stats=True, **kw)
    u, _ = ss.causal_conv_fwd(y, s["cw"], s["cb"], silu=True, reset=s["reset"], return_last_state=True, **kw)
    h, ck = ss.gated_recurrence_fwd(u, s["g"], s["z"], couple=True, reset=s["reset"], return_ckpt=True, **kw)
    dr = ss.gated_recurrence_bwd(u, s["g"], s["dy"], ck, s["z"], couple=True, reset=s["reset"], **kw)
    dc = ss.causal_conv_bwd(y, s["cw"], dr["dx"], bias=s["cb"], silu=True, reset=s["reset"], **kw)
    dn = ss.layer_norm_bwd(s["x"], dc["dx"], rstd, mean, s["w"], s["b"], **kw)
    return [h, dr["dg"], dr["dz"], dc["dweight"], dc["dbias"], dn["dx"], dn["dweight"], dn["dbias"]]


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b, strict=True))


def test_captured_and_replayed():
    """Two graphs of the same step, each with workspaces of its own, replayed
    in turn, at once on two streams, and after their inputs changed."""
    s1, s2, s3 = step_inputs(1), step_inputs(2), step_inputs(3)
    want1, want2, want3 = step(s1), step(s2), step(s3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(s1)
    torch.cuda.synchronize()
    graphs = []
    for s in (s1, s2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(s)
        graphs.append((g, out))
    for _ in range(2):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert same(graphs[0][1], want1) and same(graphs[1][1], want2)
    for k in s1:
        s1[k].copy_(s3[k])
    torch.cuda.synchronize()
    graphs[0][0].replay()
    with torch.cuda.stream(side):
        graphs[1][0].replay()
    torch.cuda.synchronize()
    assert same(graphs[0][1], want3) and same(graphs[1][1], want2)


def test_on_a_stream_of_ones_own():
    """``stream=`` queues everything there, copies of strided inputs among it."""
    s = step_inputs(4)
    want = step(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(s, stream=side)
    side.synchronize()
    assert same(got, want)
    wide = torch.stack([s["x"], s["x"]], 3)  # (B, D, L, 2): every second element
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        wide.mul_(2)
    y = ss.layer_norm_fwd(wide[..., 0], s["w"], s["b"], stream=side)
    side.synchronize()
    assert torch.equal(y, ss.layer_norm_fwd((s["x"] * 2).contiguous(), s["w"], s["b"]))


def test_two_threads_at_once():
    ins = [step_inputs(k) for k in (5, 6)]
    want = [step(s) for s in ins]
    torch.cuda.synchronize()
    got = [None, None]

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(20):
                got[i] = step(ins[i])
        st.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert same(got[0], want[0]) and same(got[1], want[1])


# ------------------------------------------------------------ the buffers' ends


@pytest.mark.parametrize("L", [1, 5, 37, 40, 263])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_nothing_is_written_outside_the_outputs(L, off, dtype):
    """Outputs inside larger buffers, on the 16-byte grid and off it: what lies
    around them stays."""
    B, D, W, guard = 3, 5, 4, 64
    n = B * D * L
    made = []

    def out(*shape, dtype=dtype):
        size = 1
        for k in shape:
            size *= k
        flat = torch.full((size + 2 * guard + off,), 7.0, dtype=dtype, device="cuda")
        made.append((flat, guard + off, size))
        return flat[guard + off:guard + off + size].view(shape)

    x, g, z, dy = (rand(B, D, L, seed=k, dtype=dtype).cuda() for k in range(4))
    w, cw = rand(D, seed=5).cuda(), rand(D, W, seed=6).cuda()
    mean, rstd = out(B, L, dtype=F32), out(B, L, dtype=F32)
    ss.ss_norm_fwd(x, out(B, D, L), w, w, mean=mean, rstd=rstd)
    ss.ss_norm_bwd(x, dy, rstd, out(B, D, L), mean, w, out(D, dtype=F32), out(D, dtype=F32))
    ss.ss_conv_fwd(x, cw, out(B, D, L), w, True, last_state=out(B, D, W - 1))
    h0 = rand(B, D, W - 1, seed=7, dtype=dtype).cuda()
    ss.ss_conv_bwd(x, cw, dy, out(B, D, L), w, True, initial_state=h0, dweight=out(D, W, dtype=F32),
                   dbias=out(D, dtype=F32), dinitial_state=out(B, D, W - 1))
    ck = out(ss.ss_glr_ckpt_elems(B, D, L, dtype), dtype=F32)
    ss.ss_glr_fwd(x, g, out(B, D, L), z, last_state=out(B, D, dtype=F32), ckpt=ck)
    ss.ss_glr_bwd(x, g, dy, ck, out(B, D, L), out(B, D, L), z, out(B, D, L), dinitial_state=out(B, D, dtype=F32))
    torch.cuda.synchronize()
    assert n == x.numel()
    for k, (flat, a, size) in enumerate(made):
        assert bool((flat[:a] == 7).all()) and bool((flat[a + size:] == 7).all()), k
        assert bool(torch.isfinite(flat).all()), k


def test_more_than_2_31_elements():
    """The last rows of tensors past 2^31 elements are those of a small call."""
    D, L = 1100, 2_000_003
    x = torch.empty(1, D, L, dtype=BF, device="cuda")
    part = rand(1, 8, L, seed=1, dtype=BF).cuda()
    for d in range(0, D, 4):
        x[:, d:d + 4] = part[:, (d // 4 % 2) * 4:(d // 4 % 2) * 4 + 4]
    assert x.numel() > 2 ** 31
    tail = x[:, -6:].contiguous()
    w, b = rand(D, 4, seed=2).cuda(), rand(D, seed=3).cuda()
    y, last = ss.causal_conv_fwd(x, w, b, silu=True, return_last_state=True)
    yt, lt = ss.causal_conv_fwd(tail, w[-6:].contiguous(), b[-6:].contiguous(), silu=True, return_last_state=True)
    assert torch.equal(y[:, -6:], yt) and torch.equal(last[:, -6:], lt)
    g = ss.causal_conv_bwd(x, w, y, bias=b, silu=True)
    gt = ss.causal_conv_bwd(tail, w[-6:].contiguous(), yt, bias=b[-6:].contiguous(), silu=True)
    assert torch.equal(g["dx"][:, -6:], gt["dx"])
    del g, y
    y, ck = ss.gated_recurrence_fwd(x, x, couple=True, return_ckpt=True)
    yt, ckt = ss.gated_recurrence_fwd(tail, tail, couple=True, return_ckpt=True)
    # (rows start on another place of the 8-element grid: other groupings of the same products)
    assert float((y[:, -6:].float() - yt.float()).abs().max()) <= 2.0 ** -7 * float(yt.float().abs().max())
    d = ss.gated_recurrence_bwd(x, x, y, ck, couple=True)
    dt = ss.gated_recurrence_bwd(tail, tail, yt, ckt, couple=True)
    assert float((d["dx"][:, -6:].float() - dt["dx"].float()).abs().max()) <= 2.0 ** -6 * float(dt["dx"].float().abs().max())
    del d, y
    y, mean, rstd = ss.layer_norm_fwd(x, b, return_stats=True)
    yt = ss.layer_norm_fwd(x[..., -40:].contiguous(), b)
    assert float((y[..., -40:].float() - yt.float()).abs().max()) <= 2.0 ** -7 * float(yt.float().abs().max())
    g = ss.layer_norm_bwd(x, y, rstd, mean, b)["dx"]
    gt = ss.layer_norm_bwd(x[..., -40:].contiguous(), y[..., -40:].contiguous(), rstd[:, -40:].contiguous(),
                           mean[:, -40:].contiguous(), b)["dx"]
    assert float((g[..., -40:].float() - gt.float()).abs().max()) <= 2.0 ** -7 * float(gt.float().abs().max())


@pytest.mark.parametrize("lo,hi", [(-1, 1), (-5, 5), (-20, -5), (5, 20), (-80, -20)])
def test_logistic_function_of_fp32(lo, hi):
    """silu of the convolution, the recurrence's decay, its complement and its
    output gate keep their relative precision however large the argument.

    Tolerances, in units of U = 2^-24: the exponential 4 (2 ulp), the sum 1, the
    reciprocal 2 (1 ulp), a product 1: 8 for silu and the complement (in which
    the exponential's error counts once, as the sum's share of it falls out);
    with the gate's product and a state of one 9.  silu' = s (1 + v (1 - s)) for
    v <= -5: s 7, the bracket 3 (its part v (1 - s) is at most 5/4 of it), two
    products."""
    n = 250_000
    v = torch.linspace(lo, hi, n, dtype=torch.float64).float().cuda()
    d = v.double()
    s, k = 1 / (1 + torch.exp(-d)), 1 / (1 + torch.exp(d))

    def near(got, want, units, what):
        off = float(((got.flatten().double() - want).abs() / want.abs()).nan_to_num(0.0).max()) / R.U
        assert off <= units, f"{what}: {off:.1f} units"

    row, w = v.view(1, 1, n), torch.tensor([[0.0, 1.0]], device="cuda")
    one, state = torch.ones(n // 500, 500, 1, device="cuda"), torch.ones(n // 500, 500, device="cuda")
    g = v.view(one.shape)
    near(ss.causal_conv_fwd(row, w, silu=True), d * s, 8, "silu")
    near(ss.gated_recurrence_fwd(0 * one, g, initial_state=state), s, 8, "decay")
    near(ss.gated_recurrence_fwd(one, g, couple=True), k, 8, "complement")
    near(ss.gated_recurrence_fwd(one, 0 * one, g, gate_sigmoid=False), d * s, 9, "output gate")
    near(ss.gated_recurrence_step(0 * state, g[..., 0], state), s, 8, "decay of a step")
    y = ss.causal_conv_step(g[..., 0], w.expand(500, 2), 0 * one, silu=True)
    near(y, d * s, 8, "silu of a step")
    if hi <= -5:
        dx = ss.causal_conv_bwd(row, w, torch.ones_like(row), silu=True)["dx"]
        near(dx, s * (1 + d * k), 12, "silu'")
        ck = ss.gated_recurrence_fwd(one, 0 * one, g, gate_sigmoid=False, return_ckpt=True)[1]
        dz = ss.gated_recurrence_bwd(one, 0 * one, one, ck, g, gate_sigmoid=False)["dz"]
        near(dz, s * (1 + d * k), 12, "gradient of the output gate")
