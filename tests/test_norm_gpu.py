"""Normalisation over the channels on the GPU against the 64-bit reference
(layer_ref.py gives the values and the bounds)."""
import threading

import pytest
import torch

import layer_ref as R
import selective_state_space_41_b200 as ss

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")]

BF, F32 = torch.bfloat16, torch.float32


def rand(*shape, seed=0, dtype=F32, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(1000 * seed + sum(shape))
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale + shift).to(dtype)


def d64(t):
    return None if t is None else t.double()


def cuda(t):
    return None if t is None else t.cuda()


def run(B, D, L, dtype, out_dtype=None, rms=False, affine=True, seed=1, x=None, rows=False):
    out_dtype = out_dtype or dtype
    if x is None:
        x = rand(B, D, L, seed=seed, dtype=dtype, scale=2.0, shift=0.7)
    w = rand(D, seed=seed + 1, scale=0.3, shift=1.0) if affine else None
    b = rand(D, seed=seed + 2, scale=0.5) if affine and not rms else None
    dy = rand(B, D, L, seed=seed + 3, dtype=out_dtype)
    view = (lambda t: t[..., 0] if rows else t)
    y, mean, rstd = ss.layer_norm_fwd(cuda(view(x)), cuda(w), cuda(b), eps=1e-5, rms=rms, return_stats=True,
                                      out_dtype=out_dtype)
    v, e = R.norm_fwd(d64(x), d64(w), d64(b), 1e-5, rms)
    what = f"{B}x{D}x{L} {dtype}"
    R.check(y, view(v["y"]), view(e["y"]), what + " y")
    R.check(rstd, view(v["rstd"]), view(e["rstd"]), what + " rstd")
    if rms:
        assert mean is None
    else:
        R.check(mean, view(v["mean"]), view(e["mean"]), what + " mean")
    # the backward from the statistics that the forward gave
    g = ss.layer_norm_bwd(cuda(view(x)), cuda(view(dy)), rstd, mean=mean, weight=cuda(w), bias=cuda(b), rms=rms)
    full = (lambda t: None if t is None else t.cpu().double().view(B, L))
    v, e = R.norm_bwd(d64(x), d64(dy), full(mean), full(rstd), d64(w))
    assert g["dx"].dtype == dtype
    R.check(g["dx"], view(v["dx"]), view(e["dx"]), what + " dx")
    assert (g["dweight"] is None) == (w is None) and (g["dbias"] is None) == (b is None)
    if w is not None:
        R.check(g["dweight"], v["dweight"], e["dweight"], what + " dweight")
    if b is not None:
        R.check(g["dbias"], v["dbias"], e["dbias"], what + " dbias")


TYPES = [(BF, BF), (BF, F32), (F32, F32)]

# rows: one warp, several warps, whole and broken vectors, every count of
# vectors per thread, the widest row a block holds and one more
ROW_DIMS = [1, 7, 8, 48, 250, 256, 520, 768, 1000, 1001, 1024, 1032, 1536, 2050, 4096, 5000, 16384, 16392]


@pytest.mark.parametrize("dim", ROW_DIMS)
@pytest.mark.parametrize("types", TYPES)
def test_rows(dim, types):
    run(5, dim, 1, *types, rms=dim % 3 == 0, seed=dim, rows=dim % 2 == 0)


@pytest.mark.parametrize("rows", [1, 3, 4, 130, 5000])
@pytest.mark.parametrize("rms", [False, True])
def test_row_counts(rows, rms):
    run(rows, 200, 1, BF, rms=rms, seed=rows)


# steps: lengths around a warp's 32, batches whose steps share a warp, one
# block, clusters of several sizes, more channels than a cluster holds
@pytest.mark.parametrize("B,D,L", [(1, 1, 2), (2, 31, 3), (3, 33, 31), (1, 64, 32), (2, 255, 33), (2, 256, 100),
                                   (3, 257, 65), (1, 700, 70), (2, 1000, 37), (1, 1536, 64), (1, 2048, 40),
                                   (1, 2100, 33), (2, 4096, 5), (1, 4097, 34), (1, 5000, 9)])
@pytest.mark.parametrize("types", TYPES)
def test_steps(B, D, L, types):
    run(B, D, L, *types, rms=(B + L) % 2 == 0, seed=D + L)


def test_many_steps():
    run(3, 96, 2777, BF, seed=5)


@pytest.mark.parametrize("shape", [(4, 64, 1), (2, 64, 40)])
def test_no_weight(shape):
    run(*shape, F32, affine=False)


@pytest.mark.parametrize("shape", [(6, 512, 1), (2, 512, 40)])
def test_large_offset(shape):
    """Channels far from zero: the variance comes from differences to the
    mean, not from a difference of squares."""
    run(*shape, F32, x=rand(*shape, seed=3, shift=300.0))


@pytest.mark.parametrize("shape", [(3, 40, 1), (1, 40, 33)])
def test_constant_channels(shape):
    """No variance at all: y is the bias, and eps keeps everything finite."""
    x = torch.full(shape, 1.5, dtype=BF)
    w, b = rand(40, seed=1), rand(40, seed=2)
    y = ss.layer_norm_fwd(x.cuda(), w.cuda(), b.cuda())
    assert torch.equal(y.cpu(), b.to(BF).view(1, 40, 1).expand(shape))


@pytest.mark.parametrize("shape", [(4, 96, 1), (2, 96, 40)])
def test_nonfinite_stays_in_its_step(shape):
    x = rand(*shape, seed=9)
    y0 = ss.layer_norm_fwd(x.cuda())
    x[1, 5, 0], x[0, 3, -1] = float("nan"), float("inf")
    y = ss.layer_norm_fwd(x.cuda())
    bad = torch.zeros(shape[0], shape[2], dtype=torch.bool)
    bad[1, 0] = bad[0, -1] = True
    assert torch.isnan(y.cpu()[bad[:, None].expand(shape)]).all()
    keep = ~bad[:, None].expand(shape)
    assert torch.equal(y.cpu()[keep], y0.cpu()[keep])


def test_misaligned_and_strided_inputs():
    """Bases off the 16-byte grid, and views that have to be made dense."""
    B, D = 6, 256
    flat = rand(B * D + 1, seed=4, dtype=BF).cuda()
    x, w = flat[1:].view(B, D, 1), rand(D, seed=5).cuda()
    dy, rstd = rand(B * D + 1, seed=6, dtype=BF).cuda()[1:].view(B, D, 1), torch.rand(B, 1, device="cuda")
    v, e = R.norm_fwd(d64(x.cpu()), d64(w.cpu()), None, 1e-5, False)
    R.check(ss.layer_norm_fwd(x, w), v["y"], e["y"], "y")
    v, e = R.norm_bwd(d64(x.cpu()), d64(dy.cpu()), None, d64(rstd.cpu()), d64(w.cpu()))
    g = ss.layer_norm_bwd(x, dy, rstd, weight=w, rms=True)
    R.check(g["dx"], v["dx"], e["dx"], "dx"), R.check(g["dweight"], v["dweight"], e["dweight"], "dweight")
    t = rand(2, 40, 64, seed=7).cuda().transpose(1, 2)  # (2, 64, 40)
    assert torch.equal(ss.layer_norm_fwd(t), ss.layer_norm_fwd(t.contiguous()))


@pytest.mark.parametrize("shape", [(0, 8, 1), (3, 8, 0), (0, 8, 4)])
def test_empty(shape):
    x = torch.empty(shape, device="cuda")
    w, b = torch.ones(8, device="cuda"), torch.zeros(8, device="cuda")
    y, mean, rstd = ss.layer_norm_fwd(x, w, b, return_stats=True)
    assert y.shape == x.shape
    g = ss.layer_norm_bwd(x, x, rstd, mean, w, b)
    assert g["dweight"].abs().sum() == 0 and g["dbias"].abs().sum() == 0


@pytest.mark.parametrize("shape", [(300, 768, 1), (2, 768, 200)])
def test_same_bits_twice(shape):
    x, dy, w = rand(*shape, dtype=BF).cuda(), rand(*shape, seed=1, dtype=BF).cuda(), rand(shape[1], seed=2).cuda()
    y, mean, rstd = ss.layer_norm_fwd(x, w, w, return_stats=True)
    first = ss.layer_norm_bwd(x, dy, rstd, mean, w, w)
    for _ in range(3):
        g = ss.layer_norm_bwd(x, dy, rstd, mean, w, w)
        assert all(torch.equal(g[k], first[k]) for k in g)


@pytest.mark.parametrize("shape", [(40, 96), (2, 96, 30)])
@pytest.mark.parametrize("rms", [False, True])
def test_autograd(shape, rms):
    x, w, b = (t.cuda().requires_grad_() for t in (rand(*shape, seed=1), rand(96, seed=2), rand(96, seed=3)))
    y = ss.layer_norm_fn(x, w, b, rms=rms)
    dy = rand(*shape, seed=4).cuda()
    y.backward(dy)
    x3 = x.detach().cpu().double().view(shape[0], 96, -1)
    v, _ = R.norm_fwd(x3, d64(w.detach().cpu()), d64(b.detach().cpu()), 1e-5, rms)
    gv, ge = R.norm_bwd(x3, dy.cpu().double().view(x3.shape), None if rms else v["mean"], v["rstd"], d64(w.detach().cpu()))
    # the saved statistics are rounded to float32 and carry the forward's bound: some 200 U relative
    R.check(x.grad.view(x3.shape), gv["dx"], ge["dx"] + 512 * R.U * gv["dx"].abs().amax(1, keepdim=True), "dx")
    R.check(w.grad, gv["dweight"], ge["dweight"] + 512 * R.U * gv["dweight"].abs().max(), "dweight")
    R.check(b.grad, gv["dbias"], ge["dbias"], "dbias")
    # a gradient of a broadcast
    x.grad = None
    ss.layer_norm_fn(x, w, b, rms=rms).sum().backward()
    assert torch.isfinite(x.grad).all()


# rows, wide rows, tiles of whole vectors, clusters, wide steps
KINDS = [(4, 96, 1), (2, 17000, 1), (2, 96, 40), (2, 1536, 40), (2, 96, 37), (2, 1536, 37), (1, 33000, 24)]


@pytest.mark.parametrize("shape", KINDS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rms", [False, True])
def test_nonfinite_reaches_its_whole_step(shape, dtype, rms):
    """One channel's NaN or infinity, as the formula has it: NaN in every
    channel of the step (rms: zero beside an infinity)."""
    x = rand(*shape, seed=31, dtype=dtype)
    last = x.shape[2] - 1
    x[0, 5, 0], x[1 % x.shape[0], 90, last] = float("nan"), float("inf")
    y, mean, rstd = ss.layer_norm_fwd(x.cuda(), rms=rms, return_stats=True)
    c = x.double() if rms else x.double() - x.double().mean(1, keepdim=True)
    want_r = (c.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    want = c * want_r
    assert torch.equal(y.isnan().cpu(), want.isnan())
    assert torch.equal(rstd.isnan().cpu(), want_r[:, 0].isnan())
    assert torch.equal(rstd.cpu() == 0, want_r[:, 0] == 0)
    assert torch.equal(y.isfinite().cpu(), want.isfinite())


def test_sizes_of_two_threads_do_not_meet():
    """Calls of different widths from two threads at once: neither changes what
    the other's launch may use."""
    xs = [rand(1, d, 64, seed=d, dtype=BF).cuda() for d in (768, 1536)]
    want = [ss.layer_norm_fwd(x) for x in xs]
    torch.cuda.synchronize()
    failed = []

    def work(x, y):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(3000):
                    got = ss.layer_norm_fwd(x)
                torch.cuda.current_stream().synchronize()
                assert torch.equal(got, y)
        except Exception as e:  # noqa: BLE001 (handed to the test)
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(xs, want)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not failed, failed


def test_workspace_elsewhere_is_refused():
    """A workspace that the kernels cannot write, or that is not one block."""
    x = rand(4, 64, 1, seed=1).cuda()
    dw, dx, rstd = torch.empty(64, device="cuda"), torch.empty_like(x), torch.ones(4, 1, device="cuda")
    n = ss.ss_norm_bwd_workspace_bytes(4, 64, 1, F32)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8, device="cuda").expand(n)):
        with pytest.raises(ValueError, match="workspace"):
            ss.ss_norm_bwd(x, x, rstd, dx, dweight=dw, workspace=ws)
    with pytest.raises(ss.SelscanError):
        ss.ss_norm_bwd(x, x, rstd, dx, dweight=dw, workspace=torch.empty(n - 4, dtype=torch.uint8, device="cuda"))
    ss.ss_norm_bwd(x, x, rstd, dx, dweight=dw, workspace=torch.empty(n, dtype=torch.uint8, device="cuda"))


# Rows that are not whole vectors, in words of two steps: rows that start in
# the middle of a word or not, tiles of 63 steps and their ends, a tensor that
# ends with half a word, channels that fill no warp or several blocks.
@pytest.mark.parametrize("B,D,L", [(300, 1, 63), (301, 3, 61), (150, 31, 126), (101, 33, 127), (150, 17, 125), (100, 64, 189),
                                   (61, 255, 315), (25, 257, 317), (25, 1000, 133), (1, 1001, 4723), (41, 2047, 61), (100, 768, 62),
                                   (10, 1024, 442), (1, 2, 18901)])
@pytest.mark.parametrize("types", TYPES)
def test_words_of_two_steps(B, D, L, types):
    run(B, D, L, *types, rms=D % 3 == 0, seed=D + L)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_nonfinite_in_words(dtype):
    """A NaN in one half of a word stays out of the other step, of the next
    tile and of the gradients of other batch entries."""
    B, D, L = 101, 40, 127
    x = rand(B, D, L, seed=41, dtype=dtype)
    y0, m0, r0 = ss.layer_norm_fwd(x.cuda(), return_stats=True)
    bad = torch.zeros(B, L, dtype=torch.bool)
    for b, d, t in ((0, 3, 0), (0, 4, 62), (0, 5, 63), (1, 6, 126), (1, 7, 40)):
        x[b, d, t], bad[b, t] = float("nan"), True
    y, m, r = ss.layer_norm_fwd(x.cuda(), return_stats=True)
    bad3 = bad[:, None].expand(B, D, L)
    assert y.cpu()[bad3].isnan().all() and torch.equal(y.cpu()[~bad3], y0.cpu()[~bad3])
    assert torch.equal(r.isnan().cpu(), bad)
    dy = rand(B, D, L, seed=42, dtype=dtype)
    g0 = ss.layer_norm_bwd(rand(B, D, L, seed=41, dtype=dtype).cuda(), dy.cuda(), r0, mean=m0)
    g = ss.layer_norm_bwd(x.cuda(), dy.cuda(), r, mean=m)
    assert torch.equal(g["dx"].cpu()[~bad3], g0["dx"].cpu()[~bad3]) and g["dx"].cpu()[bad3].isnan().all()
