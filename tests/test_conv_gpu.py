"""The causal depthwise convolution on the GPU against the 64-bit reference."""
import pytest
import torch

import layer_ref as R
import selective_state_space_41_b200 as ss
from test_norm_gpu import BF, F32, TYPES, cuda, d64, rand

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]


def starts(B, L, every, seed=0):
    if not every:
        return None
    g = torch.Generator().manual_seed(seed + B + L)
    return (torch.rand((B, L), generator=g) < 1.0 / every).to(torch.uint8)


def run(B, D, L, W, dtype=F32, out_dtype=None, silu=True, every=0, state=True, bias=True, seed=1, reset=None):
    out_dtype = out_dtype or dtype
    x, w = rand(B, D, L, seed=seed, dtype=dtype), rand(D, W, seed=seed + 1, scale=W ** -0.5)
    b = rand(D, seed=seed + 2, scale=0.3) if bias else None
    h0 = rand(B, D, W - 1, seed=seed + 3, dtype=dtype) if state else None
    dy, dl = rand(B, D, L, seed=seed + 4, dtype=out_dtype), rand(B, D, W - 1, seed=seed + 5, dtype=dtype) if state else None
    reset = starts(B, L, every) if reset is None else reset
    what = f"{B}x{D}x{L} width {W} {dtype}"
    y, last = ss.causal_conv_fwd(cuda(x), cuda(w), cuda(b), silu=silu, initial_state=cuda(h0), reset=cuda(reset),
                                 return_last_state=True, out_dtype=out_dtype)
    v, e = R.conv_fwd(d64(x), d64(w), d64(b), silu, d64(h0), reset)
    R.check(y, v["y"], e["y"], what + " y")
    assert torch.equal(last.cpu().double(), v["last"]), what + " last state"
    g = ss.causal_conv_bwd(cuda(x), cuda(w), cuda(dy), bias=cuda(b), silu=silu, initial_state=cuda(h0),
                           reset=cuda(reset), d_last_state=cuda(dl))
    v, e = R.conv_bwd(d64(x), d64(w), d64(b), silu, d64(dy), d64(h0), reset, d64(dl))
    for k in ("dx", "dweight", "dbias", "dinitial_state"):
        if g[k] is not None:
            R.check(g[k], v[k], e[k], f"{what} {k}")
    assert (g["dbias"] is None) == (not bias) and (g["dinitial_state"] is None) == (not state)


@pytest.mark.parametrize("W", range(2, 9))
@pytest.mark.parametrize("types", TYPES)
def test_widths(W, types):
    run(2, 5, 67, W, *types, seed=W)
    run(2, 5, 64, W, *types, seed=W + 20, every=6)


# one step to a few vectors, lengths that no vector divides, rows shorter than the taps
@pytest.mark.parametrize("L", [1, 2, 3, 5, 7, 8, 9, 15, 16, 17, 23, 24, 31, 40, 63, 129, 300])
@pytest.mark.parametrize("every", [0, 3])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(L, every, dtype):
    run(3, 6, L, 4, dtype, every=every, seed=L)
    run(2, 3, L, 8, dtype, every=every, state=False, silu=False, seed=L + 1)


@pytest.mark.parametrize("silu,state,bias", [(True, False, False), (False, True, True), (False, False, True)])
def test_options(silu, state, bias):
    run(2, 7, 50, 4, F32, silu=silu, state=state, bias=bias)


@pytest.mark.parametrize("B,D,L", [(1, 2, 20000), (1, 1, 5001), (37, 3, 130), (2, 1400, 33), (300, 40, 5)])
def test_sizes(B, D, L):
    """Channels shared by a cluster of blocks, many rows, many batch entries."""
    run(B, D, L, 4, BF, every=50)


def test_every_step_starts():
    """Sequences of one step: only the newest tap counts, everywhere."""
    run(2, 4, 70, 5, F32, reset=torch.ones((2, 70), dtype=torch.uint8))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nonfinite_stays_behind_a_start(dtype):
    """A NaN and an infinity before a start reach nothing after it, and reach
    W - 1 steps on where there is none."""
    x, w = rand(1, 3, 64, seed=2, dtype=dtype), rand(3, 4, seed=3)
    reset = torch.zeros((1, 64), dtype=torch.uint8)
    reset[0, 21] = 1
    clean = ss.causal_conv_fwd(x.cuda(), w.cuda(), reset=reset.cuda()).cpu()
    x[0, :, 20], x[0, :, 40] = float("nan"), float("inf")
    y = ss.causal_conv_fwd(x.cuda(), w.cuda(), reset=reset.cuda()).cpu()
    hit = torch.zeros(64, dtype=torch.bool)
    hit[20], hit[40:44] = True, True
    assert not torch.isfinite(y[..., hit]).any()
    assert torch.equal(y[..., ~hit], clean[..., ~hit])
    dy = rand(1, 3, 64, seed=4, dtype=dtype).cuda()
    dy[0, :, 25] = float("nan")
    g = ss.causal_conv_bwd(x.cuda(), w.cuda(), dy, reset=reset.cuda())["dx"].cpu()
    assert torch.isnan(g[..., 22:26]).all() and torch.isfinite(g[..., 26:]).all() and torch.isfinite(g[..., :22]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 4, 8])
def test_pieces_and_steps_equal_whole(dtype, W):
    """A row in one call, in pieces and one step at a time: the same bits."""
    B, D, L = 2, 6, 45
    x, w, b = rand(B, D, L, seed=1, dtype=dtype).cuda(), rand(D, W, seed=2).cuda(), rand(D, seed=3).cuda()
    h0 = rand(B, D, W - 1, seed=4, dtype=dtype).cuda()
    y, last = ss.causal_conv_fwd(x, w, b, silu=True, initial_state=h0, return_last_state=True)
    outs, state = [], h0
    for a, c in ((0, 1), (1, 3), (3, 30), (30, 45)):
        o, state = ss.causal_conv_fwd(x[..., a:c], w, b, silu=True, initial_state=state, return_last_state=True)
        outs.append(o)
    assert torch.equal(torch.cat(outs, 2), y) and torch.equal(state, last)
    state = h0.clone()
    for t in range(L):
        o = ss.causal_conv_step(x[..., t], w, state, bias=b, silu=True)
        assert torch.equal(o, y[..., t]), t
    assert torch.equal(state, last)


def test_misaligned_inputs():
    B, D, L = 2, 5, 64
    flat = rand(B * D * L + 1, seed=4, dtype=BF).cuda()
    x, w, dy = flat[1:].view(B, D, L), rand(D, 4, seed=5).cuda(), rand(B, D, L, seed=6, dtype=BF).cuda()
    assert torch.equal(ss.causal_conv_fwd(x, w, silu=True), ss.causal_conv_fwd(x.clone(), w, silu=True))
    a, b = (ss.causal_conv_bwd(x_, w, dy, silu=True) for x_ in (x, x.clone()))
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    t = rand(2, 64, 5, seed=7).cuda().transpose(1, 2)
    assert torch.equal(ss.causal_conv_fwd(t, w), ss.causal_conv_fwd(t.contiguous(), w))


def test_empty():
    w, b = torch.ones(3, 4, device="cuda"), torch.ones(3, device="cuda")
    for shape in ((0, 3, 5), (2, 3, 0)):
        x = torch.empty(shape, device="cuda")
        h0 = torch.randn(shape[0], 3, 3, device="cuda")
        y, last = ss.causal_conv_fwd(x, w, b, initial_state=h0, return_last_state=True)
        assert y.shape == x.shape and torch.equal(last, h0)
        g = ss.causal_conv_bwd(x, w, x, bias=b, initial_state=h0, d_last_state=2 * h0)
        assert torch.equal(g["dinitial_state"], 2 * h0)
        assert g["dweight"].abs().sum() == 0 and g["dbias"].abs().sum() == 0
    _, last = ss.causal_conv_fwd(torch.empty(2, 3, 0, device="cuda"), w, return_last_state=True)
    assert last.abs().sum() == 0


def test_same_bits_twice():
    x, w, dy = rand(4, 60, 999, dtype=BF).cuda(), rand(60, 4, seed=1).cuda(), rand(4, 60, 999, seed=2, dtype=BF).cuda()
    first = ss.causal_conv_bwd(x, w, dy, bias=w[:, 0], silu=True)
    for _ in range(3):
        g = ss.causal_conv_bwd(x, w, dy, bias=w[:, 0], silu=True)
        assert all(torch.equal(g[k], first[k]) for k in ("dx", "dweight", "dbias"))


def test_autograd():
    B, D, L, W = 2, 5, 40, 4
    x, w, b, h0 = (t.cuda().requires_grad_() for t in (rand(B, D, L, seed=1), rand(D, W, seed=2), rand(D, seed=3),
                                                       rand(B, D, W - 1, seed=4)))
    reset = starts(B, L, 9).cuda()
    y, last = ss.causal_conv_fn(x, w, b, silu=True, initial_state=h0, reset=reset, return_last_state=True)
    dy, dl = rand(B, D, L, seed=5).cuda(), rand(B, D, W - 1, seed=6).cuda()
    torch.autograd.backward([y, last], [dy, dl])
    c = lambda t: t.detach().cpu().double()  # noqa: E731
    v, e = R.conv_bwd(c(x), c(w), c(b), True, c(dy), c(h0), reset.cpu(), c(dl))
    for t, k in ((x, "dx"), (w, "dweight"), (b, "dbias"), (h0, "dinitial_state")):
        R.check(t.grad, v[k], e[k], k)
    # a broadcast gradient, and a loss on the last state alone
    for t in (x, w, b, h0):
        t.grad = None
    y, last = ss.causal_conv_fn(x, w, b, silu=True, initial_state=h0, return_last_state=True)
    last.sum().backward()
    want = torch.zeros_like(x)
    want[..., -(W - 1):] = 1
    assert torch.equal(x.grad, want) and w.grad.abs().sum() == 0 and h0.grad.abs().sum() == 0


@pytest.mark.parametrize("W,silu,every,dtype", [(2, True, 0, F32), (4, False, 40, BF), (8, True, 40, F32), (8, False, 0, BF)])
@pytest.mark.parametrize("B,D,L", [(1, 2, 20000), (1, 3, 4133), (5, 2, 1001)])
def test_blocks_of_a_channel(B, D, L, W, silu, every, dtype):
    """Few channels: several blocks to each, whose parts of a row meet."""
    run(B, D, L, W, dtype, silu=silu, every=every, seed=W)


def leave_nan_behind(W, silu, every, dtype):
    """A backward over NaN gradients in every block that the GPU holds at once:
    what it kept in shared memory, later kernels find there."""
    B, D, L = 1, 1200, 5000
    x, w, dy = rand(B, D, L, dtype=dtype).cuda(), rand(D, W).cuda(), torch.full((B, D, L), float("nan"), dtype=dtype).cuda()
    ss.causal_conv_bwd(x, w, dy, silu=silu, reset=cuda(starts(B, L, every)))


@pytest.mark.parametrize("silu,every,dtype", [(True, 0, BF), (False, 0, F32), (True, 300, F32)])
@pytest.mark.parametrize("B,D,L,W", [(1, 8, 2049, 4), (1, 8, 2050, 4), (1, 8, 2051, 4), (1, 8, 4097, 4), (1, 8, 4099, 4),
                                     (1, 8, 2049, 8), (1, 8, 2052, 8), (1, 8, 2055, 8), (1, 8, 4101, 8), (1, 3, 8193, 3),
                                     (4, 160, 674, 7), (3, 56, 2051, 7), (2, 8, 2049, 5)])
def test_row_that_ends_just_behind_a_block(B, D, L, W, silu, every, dtype):
    """A channel's blocks meet fewer than W - 1 steps before a row's end: the
    steps behind the end give the block before nothing."""
    leave_nan_behind(W, silu, every, dtype)
    run(B, D, L, W, dtype, silu=silu, every=every, seed=L + W)


def against_reference(x, w, b, silu, dy, h0, reset, dl, what):
    """Forward and backward against the 64-bit values, non-finite ones included."""
    y, last = ss.causal_conv_fwd(cuda(x), cuda(w), cuda(b), silu=silu, initial_state=cuda(h0), reset=cuda(reset),
                                 return_last_state=True)
    v, e = R.conv_fwd(d64(x), d64(w), d64(b), silu, d64(h0), reset)
    R.check(y, v["y"], e["y"], what + " y"), R.check(last, v["last"], e["last"], what + " last state")
    g = ss.causal_conv_bwd(cuda(x), cuda(w), cuda(dy), bias=cuda(b), silu=silu, initial_state=cuda(h0),
                           reset=cuda(reset), d_last_state=cuda(dl))
    v, e = R.conv_bwd(d64(x), d64(w), d64(b), silu, d64(dy), d64(h0), reset, d64(dl))
    for k in ("dx", "dweight", "dbias", "dinitial_state"):
        if g[k] is not None:
            R.check(g[k], v[k], e[k], f"{what} {k}")
    return g


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("W,silu,dtype", [(2, True, F32), (4, True, BF), (4, False, F32), (8, True, F32), (8, False, BF)])
@pytest.mark.parametrize("L", [1, 5, 37, 64, 301, 2049])
def test_nonfinite_state_behind_a_start(L, W, silu, dtype, value):
    """A row whose first step is a start uses no state: whatever the state
    holds, no gradient of a weight, the bias or another row knows of it, on
    the 8-element grid or off it."""
    B, D = 3, 5
    x, w, b = rand(B, D, L, seed=1, dtype=dtype), rand(D, W, seed=2), rand(D, seed=3)
    dy, h0, dl = rand(B, D, L, seed=4, dtype=dtype), rand(B, D, W - 1, seed=5, dtype=dtype), rand(B, D, W - 1, seed=6, dtype=dtype)
    reset = starts(B, L, 40, seed=7)
    reset[0, 0], reset[1, 0], reset[2, 0] = 1, 0, 1
    h0[0], h0[2] = value, value
    g = against_reference(x, w, b, silu, dy, h0, reset, dl, f"{B}x{D}x{L} width {W} {dtype}")
    assert all(bool(torch.isfinite(v).all()) for v in g.values())


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("W,silu,dtype", [(2, False, F32), (4, False, BF), (4, True, F32), (8, False, F32), (8, True, BF)])
@pytest.mark.parametrize("L,every", [(3, 0), (37, 0), (40, 0), (40, 9), (301, 50), (2049, 0)])
def test_nonfinite_at_a_row_end(L, every, W, silu, dtype, value):
    """An infinity or a NaN among the last inputs, or in the state of a row that
    goes on from it, reaches those weights' gradients that have a part in it."""
    B, D = 3, 5
    x, w, b = rand(B, D, L, seed=1, dtype=dtype), rand(D, W, seed=2), rand(D, seed=3)
    dy, h0 = rand(B, D, L, seed=4, dtype=dtype), rand(B, D, W - 1, seed=5, dtype=dtype)
    x[1, 0, L - 1], x[2, 1, max(L - 2, 0)], x[0, 2, max(L - W, 0)], h0[1, 3, W - 2] = (value,) * 4
    against_reference(x, w, b, silu, dy, h0, starts(B, L, every), None, f"{B}x{D}x{L} width {W} {dtype}")
