"""The gated linear recurrence on the GPU against the 64-bit reference."""
import pytest
import torch

import layer_ref as R
import selective_state_space_41_b200 as ss
from test_conv_gpu import starts
from test_norm_gpu import BF, F32, TYPES, cuda, d64, rand

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

FLAGS = [(True, True), (True, False), (False, True), (False, False)]


def gates(B, D, L, sigmoid, dtype, seed):
    g = rand(B, D, L, seed=seed, scale=1.5, shift=2.0)
    return (g if sigmoid else R.sig(g)).to(dtype)


def run(B, D, L, dtype=F32, out_dtype=None, sigmoid=True, couple=True, gated=True, every=0, state=True, seed=1,
        reset=None, g=None):
    out_dtype = out_dtype or dtype
    x, g = rand(B, D, L, seed=seed, dtype=dtype), gates(B, D, L, sigmoid, dtype, seed + 1) if g is None else g
    z = rand(B, D, L, seed=seed + 2, dtype=dtype) if gated else None
    h0, dl = (rand(B, D, seed=seed + 3), rand(B, D, seed=seed + 4)) if state else (None, None)
    dy = rand(B, D, L, seed=seed + 5, dtype=out_dtype)
    reset = starts(B, L, every) if reset is None else reset
    flags = dict(gate_sigmoid=sigmoid, couple=couple)
    what = f"{B}x{D}x{L} {dtype} sigmoid {sigmoid} couple {couple}"
    y, last, ckpt = ss.gated_recurrence_fwd(cuda(x), cuda(g), cuda(z), initial_state=cuda(h0), reset=cuda(reset),
                                            return_last_state=True, return_ckpt=True, out_dtype=out_dtype, **flags)
    v, e = R.glr_fwd(d64(x), d64(g), d64(z), sigmoid, couple, d64(h0), reset)
    R.check(y, v["y"], e["y"], what + " y")
    R.check(last, v["last"], e["last"], what + " last state")
    d = ss.gated_recurrence_bwd(cuda(x), cuda(g), cuda(dy), ckpt, cuda(z), reset=cuda(reset), d_last_state=cuda(dl),
                                return_dinitial_state=True, **flags)
    v, e = R.glr_bwd(d64(x), d64(g), d64(dy), d64(z), sigmoid, couple, d64(h0), reset, d64(dl))
    for k in ("dx", "dg", "dz", "dinitial_state"):
        if v[k] is None:
            assert d[k] is None
        else:
            R.check(d[k], v[k], e[k], f"{what} {k}")


@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("every", [0, 20])
def test_forms(flags, types, every):
    run(2, 5, 300, *types, *flags, every=every)
    run(2, 5, 301, *types, *flags, gated=False, state=False, every=every)


# one step, a vector, a warp's 256 steps and what lies around them, several warps
@pytest.mark.parametrize("L", [1, 2, 7, 8, 9, 31, 255, 256, 257, 263, 511, 513, 1000, 4097, 9000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(L, dtype):
    run(2, 3, L, dtype, every=40 if L % 2 else 0, seed=L)


@pytest.mark.parametrize("B,D,L", [(40, 130, 20), (40, 130, 300), (1, 6000, 33), (3, 800, 700), (7, 301, 1030)])
@pytest.mark.parametrize("every", [0, 15])
def test_rows(B, D, L, every):
    """Many rows: a warp each, or a few warps each."""
    run(B, D, L, BF, every=every, seed=D)


def test_every_step_starts():
    run(2, 3, 600, F32, reset=torch.ones((2, 600), dtype=torch.uint8))


def test_slow_and_closed_gates():
    """Decays that hold for the whole row, and gates shut for good."""
    g = torch.full((1, 2, 3000), 12.0)
    g[:, 1] = -60.0
    run(1, 2, 3000, F32, g=g)
    run(1, 2, 3000, F32, sigmoid=False, couple=False, g=torch.ones(1, 2, 3000))
    run(1, 2, 700, F32, sigmoid=False, couple=False, g=-torch.ones(1, 2, 700))
    run(1, 2, 700, F32, sigmoid=False, couple=False, g=torch.zeros(1, 2, 700))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("at", [200, 255, 256, 300])
def test_nonfinite_stays_behind_a_start(dtype, at):
    """A NaN or an infinity in one sequence, state or gate reaches nothing of
    the next, forward and backward."""
    B, D, L = 1, 4, 1100
    x, g, dy = rand(B, D, L, seed=1, dtype=dtype), gates(B, D, L, True, dtype, 2), rand(B, D, L, seed=3, dtype=dtype)
    reset = torch.zeros((B, L), dtype=torch.uint8)
    reset[0, at + 1] = 1
    flags = dict(couple=True, reset=reset.cuda())
    y0, ck0 = ss.gated_recurrence_fwd(x.cuda(), g.cuda(), return_ckpt=True, **flags)
    d0 = ss.gated_recurrence_bwd(x.cuda(), g.cuda(), dy.cuda(), ck0, **flags)
    x[0, 0, at], g[0, 1, at], x[0, 2, at] = float("nan"), float("nan"), float("inf")
    h0 = torch.full((B, D), float("inf")).cuda()
    y, ck = ss.gated_recurrence_fwd(x.cuda(), g.cuda(), initial_state=h0, return_ckpt=True, **flags)
    assert torch.equal(y[..., at + 1:], y0[..., at + 1:])
    d = ss.gated_recurrence_bwd(x.cuda(), g.cuda(), dy.cuda(), ck, **flags)
    for k in ("dx", "dg"):
        assert torch.equal(d[k][..., at + 1:], d0[k][..., at + 1:]), k
    # and the other way: a NaN in a later gradient stays off the earlier sequence
    dy[0, :, at + 5] = float("nan")
    d = ss.gated_recurrence_bwd(x.cuda(), g.cuda(), dy.cuda(), ck0, **flags)
    assert torch.isfinite(d["dx"][:, 3, :at + 1]).all() and torch.isnan(d["dx"][:, 3, at + 1:at + 6]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("flags", FLAGS)
def test_steps_equal_whole(dtype, flags):
    """Decoding one step at a time agrees with the whole row."""
    B, D, L = 3, 70, 40
    x, g, z = (t.cuda() for t in (rand(B, D, L, seed=1, dtype=dtype), gates(B, D, L, flags[0], dtype, 2),
                                  rand(B, D, L, seed=3, dtype=dtype)))
    h0 = rand(B, D, seed=4)
    v, e = R.glr_fwd(*(t.cpu().double() for t in (x, g, z)), *flags, h0.double())
    state = h0.cuda()
    for t in range(L):
        y = ss.gated_recurrence_step(x[..., t], g[..., t], state, z[..., t], *flags)
        R.check(y, v["y"][..., t], e["y"][..., t], f"step {t}")
    R.check(state, v["last"], e["last"], "state")


def test_pieces_equal_whole():
    """A row in pieces, the state updated in place, forward and backward."""
    B, D, L, cuts = 2, 9, 1500, (0, 1, 300, 301, 1100, 1500)
    x, g, dy = (t.cuda() for t in (rand(B, D, L, seed=1), gates(B, D, L, True, F32, 2), rand(B, D, L, seed=3)))
    h0 = rand(B, D, seed=4)
    v, e = R.glr_fwd(d64(x.cpu()), d64(g.cpu()), None, True, True, d64(h0))
    gv, ge = R.glr_bwd(d64(x.cpu()), d64(g.cpu()), d64(dy.cpu()), None, True, True, d64(h0))
    state, outs, cks = h0.cuda(), [], []
    for a, b in zip(cuts, cuts[1:]):
        piece = [t[..., a:b].contiguous() for t in (x, g)]
        y = torch.empty_like(piece[0])
        ck = torch.empty(ss.ss_glr_ckpt_elems(B, D, b - a, F32), device="cuda")
        ss.ss_glr_fwd(*piece, y, couple=True, initial_state=state, last_state=state, ckpt=ck)
        outs.append(y), cks.append(ck)
    R.check(torch.cat(outs, 2), v["y"], e["y"], "y"), R.check(state, v["last"], e["last"], "state")
    m, grads = None, []
    for (a, b), ck in reversed(list(zip(zip(cuts, cuts[1:]), cks))):
        d = ss.gated_recurrence_bwd(x[..., a:b], g[..., a:b], dy[..., a:b], ck, couple=True, d_last_state=m,
                                    return_dinitial_state=True)
        m = d["dinitial_state"]
        grads.insert(0, d)
    R.check(torch.cat([d["dx"] for d in grads], 2), gv["dx"], ge["dx"], "dx")
    R.check(torch.cat([d["dg"] for d in grads], 2), gv["dg"], ge["dg"], "dg")
    R.check(m, gv["dinitial_state"], ge["dinitial_state"], "dinitial_state")


def test_state_alone_and_no_outputs_touched():
    """y may be left out; the last state is then the same."""
    x, g = rand(2, 5, 700, seed=1).cuda(), gates(2, 5, 700, True, F32, 2).cuda()
    _, want = ss.gated_recurrence_fwd(x, g, return_last_state=True)
    last = torch.empty_like(want)
    ss.ss_glr_fwd(x, g, None, last_state=last)
    assert torch.equal(last, want)


def test_misaligned_inputs():
    B, D, L = 2, 5, 520
    flat = rand(B * D * L + 1, seed=4, dtype=BF).cuda()
    x, g, dy = flat[1:].view(B, D, L), gates(B, D, L, True, BF, 5).cuda(), rand(B, D, L, seed=6, dtype=BF).cuda()
    (y0, c0), (y1, c1) = (ss.gated_recurrence_fwd(x_, g, return_ckpt=True) for x_ in (x, x.clone()))
    assert torch.equal(y0, y1) and torch.equal(c0, c1)
    a, b = (ss.gated_recurrence_bwd(x_, g, dy, c0) for x_ in (x, x.clone()))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dg"], b["dg"])


def test_empty():
    h0 = torch.randn(2, 3, device="cuda")
    x = torch.empty(2, 3, 0, device="cuda")
    y, last, ckpt = ss.gated_recurrence_fwd(x, x, initial_state=h0, return_last_state=True, return_ckpt=True)
    assert torch.equal(last, h0) and ckpt.numel() == 0
    d = ss.gated_recurrence_bwd(x, x, x, ckpt, d_last_state=h0, return_dinitial_state=True)
    assert torch.equal(d["dinitial_state"], h0)
    _, last = ss.gated_recurrence_fwd(x, x, return_last_state=True)
    assert last.abs().sum() == 0
    x = torch.empty(0, 3, 5, device="cuda")
    assert ss.gated_recurrence_fwd(x, x).shape == x.shape


def test_same_bits_for_every_number_of_rows():
    """How many warps share a row depends on the rows; the result does not."""
    x, g, dy = rand(1, 3, 5000, seed=1).cuda(), gates(1, 3, 5000, True, F32, 2).cuda(), rand(1, 3, 5000, seed=3).cuda()
    few, ck = ss.gated_recurrence_fwd(x, g, return_ckpt=True)
    dfew = ss.gated_recurrence_bwd(x, g, dy, ck)
    many = [t.repeat(1, 2000, 1) for t in (x, g, dy)]
    y, ck = ss.gated_recurrence_fwd(*many[:2], return_ckpt=True)
    d = ss.gated_recurrence_bwd(*many, ck)
    assert torch.equal(y[:, :3], few) and torch.equal(y[:, -3:], few)
    assert torch.equal(d["dx"][:, 3:6], dfew["dx"]) and torch.equal(d["dg"][:, -3:], dfew["dg"])


@pytest.mark.parametrize("flags", FLAGS)
def test_autograd(flags):
    B, D, L = 2, 5, 300
    sig = flags[0]
    x, g, z, h0 = (t.cuda().requires_grad_() for t in (rand(B, D, L, seed=1), gates(B, D, L, sig, F32, 2),
                                                       rand(B, D, L, seed=3), rand(B, D, seed=4)))
    reset = starts(B, L, 60).cuda()
    y, last = ss.gated_recurrence_fn(x, g, z, *flags, initial_state=h0, reset=reset, return_last_state=True)
    dy, dl = rand(B, D, L, seed=5).cuda(), rand(B, D, seed=6).cuda()
    torch.autograd.backward([y, last], [dy, dl])
    c = lambda t: t.detach().cpu().double()  # noqa: E731
    v, e = R.glr_bwd(c(x), c(g), c(dy), c(z), *flags, c(h0), reset.cpu(), c(dl))
    for t, k in ((x, "dx"), (g, "dg"), (z, "dz"), (h0, "dinitial_state")):
        R.check(t.grad, v[k], e[k], k)
    with torch.no_grad():
        y2 = ss.gated_recurrence_fn(x, g, z, *flags, initial_state=h0, reset=reset)
    assert torch.equal(y2, y) and not y2.requires_grad
    ss.gated_recurrence_fn(x, g, None, *flags).sum().backward()  # a broadcast gradient


@pytest.mark.parametrize("B,D,L,every,dtype", [(1, 1, 50003, 0, BF), (1, 1, 25001, 3000, F32), (1, 3, 24600, 900, BF),
                                               (2, 5, 12301, 0, F32), (1, 40, 12300, 0, F32), (1, 74, 12289, 2000, F32)])
def test_rows_over_several_blocks(B, D, L, every, dtype):
    """Few long rows: the blocks of a cluster share one."""
    run(B, D, L, dtype, every=every, seed=D, gated=D != 40)


def test_same_bits_over_several_blocks():
    """The same rows among few (clusters) and among many (a block each)."""
    x, g = rand(1, 160, 100003, seed=3, dtype=BF).cuda(), rand(1, 160, 100003, seed=4, dtype=BF).cuda()
    few = [t[:, :16].contiguous() for t in (x, g)]
    y, last, ck = ss.gated_recurrence_fwd(x, g, return_last_state=True, return_ckpt=True)
    yf, lf, ckf = ss.gated_recurrence_fwd(*few, return_last_state=True, return_ckpt=True)
    assert torch.equal(y[:, :16], yf) and torch.equal(last[:, :16], lf)
    d = ss.gated_recurrence_bwd(x, g, x, ck)
    df = ss.gated_recurrence_bwd(*few, few[0], ckf)
    assert torch.equal(d["dx"][:, :16], df["dx"]) and torch.equal(d["dg"][:, :16], df["dg"])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("couple", [True, False])
@pytest.mark.parametrize("B,D,L", [(1, 3, 700), (2, 40, 45), (1, 2, 25001)])
def test_decays_over_their_whole_range(B, D, L, couple, dtype):
    """Decays of either sign up to one in size, runs of zeros, of ones and of
    decays whose products vanish, beside inputs and states of zero."""
    g = rand(B, D, L, seed=L).clamp(-1, 1)
    g[..., L // 5:L // 4] = 0
    g[..., L // 4:L // 3] = 1e-6
    g[..., L // 3:L // 2] = -1
    g[..., L // 2:2 * L // 3] = 1
    x = rand(B, D, L, seed=L + 1)
    x[..., L // 4:2 * L // 3] = 0
    x, g = x.to(dtype), g.to(dtype)
    what = f"{B}x{D}x{L} {dtype}"
    dy = rand(B, D, L, seed=L + 2, dtype=dtype)
    for h0 in (None, rand(B, D, seed=L + 3)):
        y, last, ck = ss.gated_recurrence_fwd(x.cuda(), g.cuda(), gate_sigmoid=False, couple=couple, initial_state=cuda(h0),
                                              return_last_state=True, return_ckpt=True)
        v, e = R.glr_fwd(d64(x), d64(g), None, False, couple, d64(h0))
        R.check(y, v["y"], e["y"], what + " y"), R.check(last, v["last"], e["last"], what + " last state")
        d = ss.gated_recurrence_bwd(x.cuda(), g.cuda(), dy.cuda(), ck, gate_sigmoid=False, couple=couple,
                                    return_dinitial_state=True)
        v, e = R.glr_bwd(d64(x), d64(g), d64(dy), None, False, couple, d64(h0))
        for k in ("dx", "dg", "dinitial_state"):
            R.check(d[k], v[k], e[k], f"{what} {k}")
