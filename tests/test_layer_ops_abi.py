"""The operators around the scan refuse bad calls on the host, before any
CUDA call (no GPU needed: no pointer given here is ever dereferenced)."""
import ctypes

import pytest
import torch

import selective_state_space_41_b200 as ss
from selective_state_space_41_b200 import build, selscan

P = ctypes.c_void_p(0x10000)
Q = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def lib():
    build.build_selscan()
    return selscan.lib()


def desc(**kw):
    d = dict(batch=2, dim=3, seqlen=16, dstate=0, in_dtype=0, out_dtype=0)
    d.update(kw)
    return ctypes.byref(selscan.Desc(**d))


BAD_DESCS = [(dict(seqlen=-1), 2), (dict(batch=1 << 40, dim=1 << 40), 2), (dict(in_dtype=2), 3),
             (dict(in_dtype=0, out_dtype=1), 3)]


def norm(lib, d, x=P, w=None, b=None, y=Q, mean=None, rstd=None):
    return lib.ss_norm_fwd(d, x, w, b, 1e-5, 0, y, mean, rstd, None)


def norm_bwd(lib, d, x=P, w=None, mean=P, rstd=P, dy=P, dx=Q, dw=None, db=None, ws=None, n=0):
    return lib.ss_norm_bwd(d, x, w, mean, rstd, dy, dx, dw, db, ws, n, None)


def conv(lib, d, W=4, x=P, w=P, b=None, h0=None, reset=None, y=Q, last=None):
    return lib.ss_conv_fwd(d, W, x, w, b, 1, h0, reset, y, last, None)


def conv_bwd(lib, d, W=4, x=P, w=P, b=None, h0=None, reset=None, dy=P, dl=None, dx=Q, dw=None, db=None, dh0=None):
    return lib.ss_conv_bwd(d, W, x, w, b, 1, h0, reset, dy, dl, dx, dw, db, dh0, None)


def conv_step(lib, d, W=4, x=P, w=P, b=None, state=P, y=Q):
    return lib.ss_conv_step(d, W, x, w, b, 1, state, y, None)


def glr(lib, d, x=P, g=P, z=None, h0=None, reset=None, y=Q, last=None, ckpt=None):
    return lib.ss_glr_fwd(d, x, g, z, 1, 1, h0, reset, y, last, ckpt, None)


def glr_bwd(lib, d, x=P, g=P, z=None, reset=None, ckpt=P, dy=P, dl=None, dx=Q, dg=Q, dz=None, dh0=None):
    return lib.ss_glr_bwd(d, x, g, z, 1, 1, reset, ckpt, dy, dl, dx, dg, dz, dh0, None)


def glr_step(lib, d, x=P, g=P, z=None, state=P, y=Q):
    return lib.ss_glr_step(d, x, g, z, 1, 1, state, y, None)


ALL = [norm, norm_bwd, conv, conv_bwd, conv_step, glr, glr_bwd, glr_step]


@pytest.mark.parametrize("call", ALL)
def test_descriptors(lib, call):
    assert call(lib, None) == 1
    for kw, status in BAD_DESCS:
        kw = dict({"seqlen": 1} if call in (conv_step, glr_step) else {}, **kw)
        assert call(lib, desc(**kw)) == status, kw


@pytest.mark.parametrize("call,names", [(norm, "x y"), (norm_bwd, "x rstd dy dx"), (conv, "x w y"),
                                        (conv_bwd, "x w dy dx"), (conv_step, "x w state y"), (glr, "x g"),
                                        (glr_bwd, "x g ckpt dy dx dg"), (glr_step, "x g state y")])
def test_required_and_misaligned_pointers(lib, call, names):
    d = desc(seqlen=1) if call in (conv_step, glr_step) else desc()
    for n in names.split():
        assert call(lib, d, **{n: None}) == 1, n
        assert call(lib, d, **{n: ODD}) == 5, n


@pytest.mark.parametrize("call,names", [(norm, "w b mean rstd"), (norm_bwd, "w mean dw db"), (conv, "b h0 last"),
                                        (conv_bwd, "b h0 dl dw db dh0"), (conv_step, "b"), (glr, "z h0 last ckpt y"),
                                        (glr_bwd, "dl dh0"), (glr_step, "z")])
def test_optional_pointers_alignment(lib, call, names):
    d = desc(seqlen=1) if call in (conv_step, glr_step) else desc()
    for n in names.split():
        assert call(lib, d, **{n: ODD}) == 5, n


def test_own_rules(lib):
    assert conv(lib, desc(), W=1) == 2 and conv(lib, desc(), W=9) == 2
    assert conv_bwd(lib, desc(), W=9) == 2 and conv_step(lib, desc(seqlen=1), W=0) == 2
    assert conv_step(lib, desc(seqlen=2)) == 2 and glr_step(lib, desc(seqlen=0)) == 2
    assert conv(lib, desc(), y=P) == 10 and conv(lib, desc(), h0=P, last=P) == 10
    assert conv_bwd(lib, desc(), dx=P) == 10 and conv_bwd(lib, desc(), dl=P, dh0=P) == 10
    assert glr_bwd(lib, desc(), z=P) == 1 and glr_bwd(lib, desc(), dz=Q) == 1     # dz exactly with z
    assert glr(lib, desc(), y=None) == 1                                        # nothing asked for
    assert norm_bwd(lib, desc(), dw=P) == 8 and norm_bwd(lib, desc(), dw=P, ws=Q, n=16) == 8
    n = lib.ss_norm_bwd_workspace_bytes(desc())
    assert n > 0 and norm_bwd(lib, desc(), dw=P, ws=ODD, n=n) == 5
    assert glr(lib, desc(batch=1 << 20, dim=1 << 20)) == 2
    assert "distinct" in ss.ss_status_string(10)


def test_empty_calls_need_no_pointers(lib):
    for kw in (dict(batch=0), dict(dim=0)):
        e = desc(**kw)
        none = dict(x=None)
        assert norm(lib, e, y=None, **none) == 0 and conv(lib, e, w=None, y=None, **none) == 0
        assert glr(lib, e, g=None, y=None, **none) == 0
        assert glr_bwd(lib, e, g=None, ckpt=None, dy=None, dx=None, dg=None, **none) == 0
        assert conv_bwd(lib, e, w=None, dy=None, dx=None, **none) == 0
        assert norm_bwd(lib, e, mean=None, rstd=None, dy=None, dx=None, **none) == 0
    assert glr(lib, desc(seqlen=0), x=None, g=None, y=None) == 0
    assert conv(lib, desc(seqlen=0), x=None, w=None, y=None) == 0


def test_sizes(lib):
    """One state per 256 steps of a row, the row's start on an 8-step grid;
    the norm's partial sums: two rows of dim floats per block or cluster."""
    assert ss.ss_glr_ckpt_elems(2, 3, 256) == 2 * 3 * 2 and ss.ss_glr_ckpt_elems(2, 3, 249) == 2 * 3
    assert ss.ss_glr_ckpt_elems(2, 0, 256) == 0 and lib.ss_glr_ckpt_elems(None) == 0
    assert ss.ss_norm_bwd_workspace_bytes(4, 64, 1) == 2 * 64 * 4
    assert ss.ss_norm_bwd_workspace_bytes(1 << 20, 64, 1) < 4 << 20
    assert ss.ss_norm_bwd_workspace_bytes(0, 64, 1) == 0 and lib.ss_norm_bwd_workspace_bytes(None) == 0


X = torch.zeros(2, 6, 16)
W4 = torch.zeros(6, 4)


@pytest.mark.parametrize("call", [
    lambda: ss.layer_norm_fwd(torch.zeros(3)),                                       # dimensions
    lambda: ss.layer_norm_fwd(X.half()),                                             # type
    lambda: ss.layer_norm_fwd(X, torch.zeros(5)),                                    # weight's size
    lambda: ss.layer_norm_fwd(X, torch.zeros(6, dtype=torch.bfloat16)),              # weight's type
    lambda: ss.layer_norm_fwd(X, out_dtype=torch.bfloat16),                          # float32 to bf16
    lambda: ss.ss_norm_fwd(X, torch.zeros(6, 2, 16).transpose(0, 1)),                # output not dense
    lambda: ss.layer_norm_bwd(X, X, torch.zeros(2, 15), rms=True),                   # statistics' size
    lambda: ss.layer_norm_bwd(X, X, torch.zeros(2, 16), mean=torch.zeros(2, 16), rms=True),
    lambda: ss.layer_norm_bwd(X, X, torch.zeros(2, 16)),                             # no mean
    lambda: ss.causal_conv_fwd(X[0], W4),
    lambda: ss.causal_conv_fwd(X, torch.zeros(5, 4)),
    lambda: ss.causal_conv_fwd(X, torch.zeros(6)),
    lambda: ss.causal_conv_fwd(X, W4, initial_state=torch.zeros(2, 6, 4)),
    lambda: ss.causal_conv_fwd(X, W4, initial_state=torch.zeros(2, 6, 3, dtype=torch.bfloat16)),
    lambda: ss.causal_conv_fwd(X, W4, reset=torch.zeros(2, 15, dtype=torch.uint8)),
    lambda: ss.causal_conv_fwd(X, W4, reset=torch.zeros(2, 16, dtype=torch.int32)),
    lambda: ss.causal_conv_bwd(X, W4, X[..., :8]),
    lambda: ss.causal_conv_step(X[..., 0], W4, torch.zeros(2, 3, 6).transpose(1, 2)),  # state not dense
    lambda: ss.causal_conv_step(X, W4, torch.zeros(2, 6, 3)),
    lambda: ss.gated_recurrence_fwd(X, X[:1]),
    lambda: ss.gated_recurrence_fwd(X, X.bfloat16()),
    lambda: ss.gated_recurrence_fwd(X, X, initial_state=torch.zeros(2, 6, 1)),
    lambda: ss.gated_recurrence_bwd(X, X, X, torch.zeros(3)),                        # checkpoints' size
    lambda: ss.gated_recurrence_step(X[..., 0], X[..., 0], torch.zeros(2, 6, dtype=torch.bfloat16)),
    # good calls, but for the device
    lambda: ss.layer_norm_fwd(X), lambda: ss.causal_conv_fwd(X, W4), lambda: ss.gated_recurrence_fwd(X, X),
    lambda: ss.gated_recurrence_step(X[..., 0], X[..., 0], torch.zeros(2, 6)),
])
def test_binding_refuses(lib, call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call,sizes", [(norm, (1, 1 << 31, 1)), (norm, (1 << 31, 1, 1)), (norm, (1 << 16, 1, 1 << 16)),
                                        (norm_bwd, (1 << 16, 1, 1 << 16)), (conv, (1 << 14, 1 << 14, 5)),
                                        (conv_bwd, (1 << 14, 1 << 14, 5)), (conv_step, (1 << 14, 1 << 14, 1)),
                                        (glr, (1 << 16, 1 << 15, 5)), (glr_bwd, (1 << 16, 1 << 15, 5)),
                                        (glr_step, (1 << 16, 1 << 15, 1))])
def test_sizes_that_launches_cannot_count(lib, call, sizes):
    assert call(lib, desc(batch=sizes[0], dim=sizes[1], seqlen=sizes[2])) == 2
