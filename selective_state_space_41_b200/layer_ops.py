"""Python binding of the operators around the scan: normalisation over the
channels, the causal depthwise convolution and the gated linear recurrence
(argument marshalling only, as ``selscan.py``; the computation runs in the
kernels of ``libselscan.so``, whose ``include/selscan.h`` states formulas,
shapes and errors).

``ss_norm_*``, ``ss_conv_*`` and ``ss_glr_*`` are the C entry points on tensors
that the caller provides; ``layer_norm_*``, ``causal_conv_*`` and
``gated_recurrence_*`` allocate their results, and the ``_fn`` forms are torch
autograd Functions.  Sequences are (batch, dim, L) as everywhere in this
library; the norm also takes (rows, dim).

All tensors of a call lie on one CUDA device, which need not be the current
one.  Work is queued on that device's current stream, or on the ``stream`` that
every call but the ``_fn`` forms takes by keyword; copies of non-contiguous
inputs are made on the same stream.  Outputs must be
contiguous.  A wrong shape, dtype or device raises ValueError, a call that the
library rejects SelscanError.

The forward and backward calls and the decoding steps may be captured into
CUDA graphs.  Captured calls that may overlap need workspaces of their own
(the allocating forms make one per call).  Through autograd, capture as torch
requires it: warm up on a side stream, and keep no eager graph of the same
leaves alive while a backward pass is captured (torch ends the process when a
captured backward meets a leaf's accumulation on another stream).
"""
import ctypes
import functools

import torch

from .selscan import _DTYPE_CODE, Desc, _check, lib

__all__ = ["ss_norm_fwd", "ss_norm_bwd", "ss_norm_bwd_workspace_bytes", "layer_norm_fwd", "layer_norm_bwd",
           "layer_norm_fn", "LayerNormFn", "ss_conv_fwd", "ss_conv_bwd", "ss_conv_step", "causal_conv_fwd",
           "causal_conv_bwd", "causal_conv_step", "causal_conv_fn", "CausalConvFn", "ss_glr_fwd", "ss_glr_bwd",
           "ss_glr_step", "ss_glr_ckpt_elems", "gated_recurrence_fwd", "gated_recurrence_bwd",
           "gated_recurrence_step", "gated_recurrence_fn", "GatedRecurrenceFn"]

_F32 = torch.float32


def _on_device(fn):
    """Runs ``fn(x, ...)`` on ``stream`` when given, and otherwise on the
    current stream of x's device, whichever device is current."""
    @functools.wraps(fn)
    def call(x, *args, stream=None, **kw):
        if stream is None:
            if not x.is_cuda or x.get_device() == torch._C._cuda_getDevice():
                return fn(x, *args, **kw)
            with torch.cuda.device(x.device):
                return fn(x, *args, **kw)
        if stream.device != x.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {x.device}")
        with torch.cuda.stream(stream):  # also sets the device
            return fn(x, *args, **kw)
    return call


def _stream(x):
    if not x.is_cuda:
        raise ValueError(f"the library runs on CUDA tensors only, got one on {x.device}")
    return torch._C._cuda_getCurrentRawStream(x.get_device())


def _refuse(t, name, shape, dtype, x):
    raise ValueError(f"{name} must be a {tuple(shape)} {dtype} tensor on {x.device}, got {tuple(t.shape)} {t.dtype} "
                     f"on {t.device}")


def _input(t, name, shape, dtype, x):
    """``t`` (or None) as a dense tensor of that shape and dtype on x's device."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != x.get_device():
        _refuse(t, name, shape, dtype, x)
    return t if t.is_contiguous() else t.contiguous()


def _output(t, name, shape, dtype, x):
    """``t`` (or None) checked as an output, which is never copied."""
    if t is not None:
        if t.shape != shape or t.dtype is not dtype or t.get_device() != x.get_device():
            _refuse(t, name, shape, dtype, x)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return t


def _starts(reset, batch, L, x):
    if reset is None:
        return None
    if reset.dtype is torch.bool:
        reset = reset.view(torch.uint8)
    return _input(reset, "reset", (batch, L), torch.uint8, x)


def _main(x, dims, what):
    """The leading tensor of a call: dense, of a type the library has."""
    if x.dim() not in dims:
        raise ValueError(f"{what} must have {' or '.join(map(str, dims))} dimensions, got {tuple(x.shape)}")
    if x.dtype not in _DTYPE_CODE:
        raise ValueError(f"{what} must be float32 or bfloat16, got {x.dtype}")
    return x if x.is_contiguous() else x.contiguous()


def _out_type(dtype, x, name):
    """The type of an output (or its gradient): x's own, or float32."""
    if dtype is not x.dtype and dtype is not _F32:
        raise ValueError(f"{name} must be {x.dtype} or float32, got {dtype}")
    return dtype


def _new(x, dtype=None):
    """A dense tensor of x's shape on its device."""
    if (dtype is None or dtype is x.dtype) and x.is_contiguous():
        return torch.empty_like(x)
    return x.new_empty(x.shape, dtype=dtype or x.dtype)


@functools.lru_cache(maxsize=1024)
def _sizes(batch, dim, L, in_dtype, out_dtype):
    """The descriptor of these sizes, by reference (made once for each)."""
    return ctypes.byref(Desc(batch, dim, L, 0, _DTYPE_CODE[in_dtype], _DTYPE_CODE[out_dtype]))


def _desc(batch, dim, L, x, out_dtype):
    return _sizes(batch, dim, L, x.dtype, out_dtype)


def _p(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------- the norm


def _norm_sizes(x):
    return (x.shape[0], x.shape[1], 1 if x.dim() == 2 else x.shape[2])


def _norm_fwd(x, y, weight, bias, eps, rms, mean, rstd):
    batch, dim, L = _norm_sizes(x)
    weight, bias = _input(weight, "weight", (dim,), _F32, x), _input(bias, "bias", (dim,), _F32, x)
    _check(lib().ss_norm_fwd(_desc(batch, dim, L, x, y.dtype), x.data_ptr(), _p(weight), _p(bias), eps,
                             1 if rms else 0, y.data_ptr(), _p(mean), _p(rstd), _stream(x)), "ss_norm_fwd")


@_on_device
def ss_norm_fwd(x, y, weight=None, bias=None, eps=1e-5, rms=False, mean=None, rstd=None):
    """Queue the normalisation of x ((batch, dim, L), or (rows, dim)) over its
    channels into y.  weight, bias: (dim,) float32; mean, rstd: float32
    outputs of x's shape without its channels (mean only without ``rms``)."""
    x = _main(x, (2, 3), "x")
    kept = x.shape[:1] + x.shape[2:]
    _output(y, "y", x.shape, _out_type(y.dtype, x, "y"), x)
    _output(mean, "mean", kept, _F32, x), _output(rstd, "rstd", kept, _F32, x)
    _norm_fwd(x, y, weight, bias, eps, rms, mean, rstd)


@_on_device
def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, rms=False, return_stats=False, out_dtype=None):
    """y, or (y, mean, rstd) with ``return_stats`` (mean is None with ``rms``)."""
    x = _main(x, (2, 3), "x")
    y = _new(x, out_dtype and _out_type(out_dtype, x, "out_dtype"))
    mean = rstd = None
    if return_stats:
        kept = x.shape[:1] + x.shape[2:]
        rstd = x.new_empty(kept, dtype=_F32)
        mean = None if rms else x.new_empty(kept, dtype=_F32)
    _norm_fwd(x, y, weight, bias, eps, rms, mean, rstd)
    return (y, mean, rstd) if return_stats else y


def ss_norm_bwd_workspace_bytes(batch, dim, seqlen, in_dtype=torch.bfloat16, out_dtype=None) -> int:
    desc = Desc(batch, dim, seqlen, 0, _DTYPE_CODE[in_dtype], _DTYPE_CODE[out_dtype or in_dtype])
    return int(lib().ss_norm_bwd_workspace_bytes(ctypes.byref(desc)))


def _norm_bwd(x, dy, rstd, dx, mean, weight, dweight, dbias, workspace):
    batch, dim, L = _norm_sizes(x)
    kept = x.shape[:1] + x.shape[2:]
    dy = _input(dy, "dy", x.shape, _out_type(dy.dtype, x, "dy"), x)
    mean, rstd = _input(mean, "mean", kept, _F32, x), _input(rstd, "rstd", kept, _F32, x)
    weight = _input(weight, "weight", (dim,), _F32, x)
    desc, size = _desc(batch, dim, L, x, dy.dtype), 0
    if workspace is not None:
        if workspace.get_device() != x.get_device() or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on {x.device}, got one on {workspace.device}")
        size = workspace.numel() * workspace.element_size()
    elif dweight is not None or dbias is not None:
        size = lib().ss_norm_bwd_workspace_bytes(desc)
        workspace = x.new_empty(size, dtype=torch.uint8)
    _check(lib().ss_norm_bwd(desc, x.data_ptr(), _p(weight), _p(mean), rstd.data_ptr(), dy.data_ptr(),
                             dx.data_ptr(), _p(dweight), _p(dbias), _p(workspace), size, _stream(x)),
           "ss_norm_bwd")


@_on_device
def ss_norm_bwd(x, dy, rstd, dx, mean=None, weight=None, dweight=None, dbias=None, workspace=None):
    """Queue the norm's backward from the forward's mean and rstd (mean None:
    the RMS form) into dx and, where given, dweight and dbias ((dim,) float32).
    ``workspace``: a CUDA tensor of ss_norm_bwd_workspace_bytes() bytes, made
    here when None and needed."""
    x = _main(x, (2, 3), "x")
    _output(dx, "dx", x.shape, x.dtype, x)
    _output(dweight, "dweight", x.shape[1:2], _F32, x), _output(dbias, "dbias", x.shape[1:2], _F32, x)
    _norm_bwd(x, dy, rstd, dx, mean, weight, dweight, dbias, workspace)


@_on_device
def layer_norm_bwd(x, dy, rstd, mean=None, weight=None, bias=None, rms=False):
    """Gradients of sum(dy * y) as a dict: dx, dweight (None without weight),
    dbias (None without bias).  mean and rstd are layer_norm_fwd's
    (``return_stats``); ``rms`` as there."""
    if (mean is None) != bool(rms):
        raise ValueError("mean goes with the layer norm, none with rms")
    x = _main(x, (2, 3), "x")
    bias = _input(bias, "bias", x.shape[1:2], _F32, x)
    weight = _input(weight, "weight", x.shape[1:2], _F32, x)
    g = {"dx": torch.empty_like(x), "dweight": torch.empty_like(weight) if weight is not None else None,
         "dbias": torch.empty_like(bias) if bias is not None else None}
    _norm_bwd(x, dy, rstd, g["dx"], mean, weight, g["dweight"], g["dbias"], None)
    return g


class LayerNormFn(torch.autograd.Function):
    """The norm as a torch autograd Function (gradients of x, weight, bias)."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms):
        if not any(ctx.needs_input_grad):
            return layer_norm_fwd(x, weight, bias, eps, rms)
        y, mean, rstd = layer_norm_fwd(x, weight, bias, eps, rms, return_stats=True)
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        ctx.rms = bool(rms)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, bias, mean, rstd = ctx.saved_tensors
        g = layer_norm_bwd(x, dy, rstd, mean, weight, bias, ctx.rms)
        return g["dx"], g["dweight"], g["dbias"], None, None


def layer_norm_fn(x, weight=None, bias=None, eps=1e-5, rms=False):
    """Layer norm (RMS norm with ``rms``) over the channels of x, (batch, dim,
    L) or (rows, dim), differentiable; y has x's dtype."""
    return LayerNormFn.apply(x, weight, bias, eps, rms)


# -------------------------------------------------------- the causal convolution


def _width(weight):
    if weight.dim() != 2 or not 2 <= weight.shape[1] <= 8:
        raise ValueError(f"weight must be (dim, width) with a width from 2 to 8, got {tuple(weight.shape)}")
    return weight.shape[1]


def _conv_fwd(x, weight, y, bias, silu, initial_state, reset, last_state):
    (batch, dim, L), W = x.shape, _width(weight)
    weight, bias = _input(weight, "weight", (dim, W), _F32, x), _input(bias, "bias", (dim,), _F32, x)
    initial_state = _input(initial_state, "initial_state", (batch, dim, W - 1), x.dtype, x)
    reset = _starts(reset, batch, L, x)
    _check(lib().ss_conv_fwd(_desc(batch, dim, L, x, y.dtype), W, x.data_ptr(), weight.data_ptr(), _p(bias),
                             1 if silu else 0, _p(initial_state), _p(reset), y.data_ptr(), _p(last_state),
                             _stream(x)), "ss_conv_fwd")


@_on_device
def ss_conv_fwd(x, weight, y, bias=None, silu=False, initial_state=None, reset=None, last_state=None):
    """Queue the causal depthwise convolution of x (batch, dim, L) into y.
    weight: (dim, width) float32, width 2..8; bias: (dim,) float32;
    initial_state, last_state: (batch, dim, width - 1) in x's dtype, two
    buffers; reset: (batch, L) uint8 or bool, nonzero where a sequence starts."""
    x = _main(x, (3,), "x")
    _output(y, "y", x.shape, _out_type(y.dtype, x, "y"), x)
    _output(last_state, "last_state", (*x.shape[:2], _width(weight) - 1), x.dtype, x)
    _conv_fwd(x, weight, y, bias, silu, initial_state, reset, last_state)


@_on_device
def causal_conv_fwd(x, weight, bias=None, silu=False, initial_state=None, reset=None, return_last_state=False,
                    out_dtype=None):
    """y (and the last state) of the causal depthwise convolution."""
    x = _main(x, (3,), "x")
    y = _new(x, out_dtype and _out_type(out_dtype, x, "out_dtype"))
    last = None
    if return_last_state:
        last = x.new_empty((*x.shape[:2], _width(weight) - 1))
    _conv_fwd(x, weight, y, bias, silu, initial_state, reset, last)
    return (y, last) if return_last_state else y


def _conv_bwd(x, weight, dy, dx, bias, silu, initial_state, reset, d_last_state, dweight, dbias, dinitial_state):
    (batch, dim, L), W = x.shape, _width(weight)
    state = (batch, dim, W - 1)
    weight, bias = _input(weight, "weight", (dim, W), _F32, x), _input(bias, "bias", (dim,), _F32, x)
    initial_state, reset = _input(initial_state, "initial_state", state, x.dtype, x), _starts(reset, batch, L, x)
    dy = _input(dy, "dy", x.shape, _out_type(dy.dtype, x, "dy"), x)
    d_last_state = _input(d_last_state, "d_last_state", state, x.dtype, x)
    _check(lib().ss_conv_bwd(_desc(batch, dim, L, x, dy.dtype), W, x.data_ptr(), weight.data_ptr(), _p(bias),
                             1 if silu else 0, _p(initial_state), _p(reset), dy.data_ptr(), _p(d_last_state),
                             dx.data_ptr(), _p(dweight), _p(dbias), _p(dinitial_state), _stream(x)),
           "ss_conv_bwd")


@_on_device
def ss_conv_bwd(x, weight, dy, dx, bias=None, silu=False, initial_state=None, reset=None, d_last_state=None,
                dweight=None, dbias=None, dinitial_state=None):
    """Queue the convolution's backward into dx and, where given, dweight
    ((dim, width) float32), dbias ((dim,) float32) and dinitial_state."""
    x = _main(x, (3,), "x")
    (batch, dim, L), W = x.shape, _width(weight)
    _output(dx, "dx", x.shape, x.dtype, x), _output(dinitial_state, "dinitial_state", (batch, dim, W - 1), x.dtype, x)
    _output(dweight, "dweight", (dim, W), _F32, x), _output(dbias, "dbias", (dim,), _F32, x)
    _conv_bwd(x, weight, dy, dx, bias, silu, initial_state, reset, d_last_state, dweight, dbias, dinitial_state)


@_on_device
def causal_conv_bwd(x, weight, dy, bias=None, silu=False, initial_state=None, reset=None, d_last_state=None):
    """Gradients of sum(dy * y) (+ sum(d_last_state * last state)) as a dict:
    dx, dweight, dbias (None without bias), dinitial_state (None without an
    initial state)."""
    x = _main(x, (3,), "x")
    dim, W = x.shape[1], _width(weight)
    weight, bias = _input(weight, "weight", (dim, W), _F32, x), _input(bias, "bias", (dim,), _F32, x)
    initial_state = _input(initial_state, "initial_state", (x.shape[0], dim, W - 1), x.dtype, x)
    g = {"dx": torch.empty_like(x), "dweight": torch.empty_like(weight),
         "dbias": torch.empty_like(bias) if bias is not None else None,
         "dinitial_state": torch.empty_like(initial_state) if initial_state is not None else None}
    _conv_bwd(x, weight, dy, g["dx"], bias, silu, initial_state, reset, d_last_state, g["dweight"], g["dbias"],
              g["dinitial_state"])
    return g


def _conv_step(x, weight, state, y, bias, silu):
    (batch, dim), W = x.shape, _width(weight)
    weight, bias = _input(weight, "weight", (dim, W), _F32, x), _input(bias, "bias", (dim,), _F32, x)
    _output(state, "state", (batch, dim, W - 1), x.dtype, x)
    _check(lib().ss_conv_step(_desc(batch, dim, 1, x, y.dtype), W, x.data_ptr(), weight.data_ptr(), _p(bias),
                              1 if silu else 0, state.data_ptr(), y.data_ptr(), _stream(x)), "ss_conv_step")


@_on_device
def ss_conv_step(x, weight, state, y, bias=None, silu=False):
    """Queue one decoding step: x, y (batch, dim); state (batch, dim, width -
    1) in x's dtype, updated in place."""
    x = _main(x, (2,), "x")
    _output(y, "y", x.shape, _out_type(y.dtype, x, "y"), x)
    _conv_step(x, weight, state, y, bias, silu)


@_on_device
def causal_conv_step(x, weight, state, bias=None, silu=False, out_dtype=None):
    """y (batch, dim) of one decoding step; the state is updated in place."""
    x = _main(x, (2,), "x")
    y = _new(x, out_dtype and _out_type(out_dtype, x, "out_dtype"))
    _conv_step(x, weight, state, y, bias, silu)
    return y


class CausalConvFn(torch.autograd.Function):
    """The convolution as a torch autograd Function (gradients of x, weight,
    bias, the initial state; through y and the last state)."""

    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, reset, silu, return_last_state):
        out = causal_conv_fwd(x, weight, bias, silu, initial_state, reset, return_last_state)
        ctx.save_for_backward(x, weight, bias, initial_state, reset)
        ctx.silu = bool(silu)
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dlast=None):
        x, weight, bias, initial_state, reset = ctx.saved_tensors
        g = causal_conv_bwd(x, weight, dy, bias, ctx.silu, initial_state, reset, dlast)
        return g["dx"], g["dweight"], g["dbias"], g["dinitial_state"], None, None, None


def causal_conv_fn(x, weight, bias=None, silu=False, initial_state=None, reset=None, return_last_state=False):
    """y (and the last state) of the causal depthwise convolution,
    differentiable; see CausalConvFn."""
    return CausalConvFn.apply(x, weight, bias, initial_state, reset, silu, return_last_state)


# ------------------------------------------------------- the gated recurrence


def ss_glr_ckpt_elems(batch, dim, seqlen, in_dtype=torch.bfloat16, out_dtype=None) -> int:
    """Floats in the checkpoints that a forward of these sizes keeps."""
    desc = Desc(batch, dim, seqlen, 0, _DTYPE_CODE[in_dtype], _DTYPE_CODE[out_dtype or in_dtype])
    return int(lib().ss_glr_ckpt_elems(ctypes.byref(desc)))


def _glr_fwd(x, g, y, z, gate_sigmoid, couple, initial_state, reset, last_state, ckpt, desc):
    batch, dim, L = x.shape
    g, z = _input(g, "g", x.shape, x.dtype, x), _input(z, "z", x.shape, x.dtype, x)
    initial_state = _input(initial_state, "initial_state", (batch, dim), _F32, x)
    reset = _starts(reset, batch, L, x)
    _check(lib().ss_glr_fwd(desc, x.data_ptr(), g.data_ptr(), _p(z), 1 if gate_sigmoid else 0, 1 if couple else 0,
                            _p(initial_state), _p(reset), _p(y), _p(last_state), _p(ckpt), _stream(x)), "ss_glr_fwd")


@_on_device
def ss_glr_fwd(x, g, y, z=None, gate_sigmoid=True, couple=False, initial_state=None, reset=None, last_state=None,
               ckpt=None):
    """Queue the gated linear recurrence of x, g (batch, dim, L) into y (None:
    only the states are wanted).  z: output gate; initial_state, last_state:
    (batch, dim) float32, one buffer or two; reset: (batch, L) uint8 or bool,
    nonzero where a sequence starts; ckpt: ss_glr_ckpt_elems() float32, for
    the backward.  g is a decay's logit, or with ``gate_sigmoid`` false the
    decay, in [-1, 1] (products of larger ones may overflow, to NaN)."""
    x = _main(x, (3,), "x")
    out = x.dtype if y is None else _out_type(y.dtype, x, "y")
    _output(y, "y", x.shape, out, x), _output(last_state, "last_state", x.shape[:2], _F32, x)
    desc = _desc(*x.shape, x, out)
    if ckpt is not None:
        _output(ckpt, "ckpt", (int(lib().ss_glr_ckpt_elems(desc)),), _F32, x)
    _glr_fwd(x, g, y, z, gate_sigmoid, couple, initial_state, reset, last_state, ckpt, desc)


@_on_device
def gated_recurrence_fwd(x, g, z=None, gate_sigmoid=True, couple=False, initial_state=None, reset=None,
                         return_last_state=False, return_ckpt=False, out_dtype=None):
    """y of the gated linear recurrence, then the last state
    (``return_last_state``) and the backward's checkpoints (``return_ckpt``).
    g: the decays' logits, or with ``gate_sigmoid`` false decays in [-1, 1]."""
    x = _main(x, (3,), "x")
    out = _out_type(out_dtype or x.dtype, x, "out_dtype")
    y, desc = _new(x, out), _desc(*x.shape, x, out)
    last = x.new_empty(x.shape[:2], dtype=_F32) if return_last_state else None
    ckpt = x.new_empty(lib().ss_glr_ckpt_elems(desc), dtype=_F32) if return_ckpt else None
    _glr_fwd(x, g, y, z, gate_sigmoid, couple, initial_state, reset, last, ckpt, desc)
    more = ((last,) if return_last_state else ()) + ((ckpt,) if return_ckpt else ())
    return (y, *more) if more else y


def _glr_bwd(x, g, dy, ckpt, dx, dg, z, dz, gate_sigmoid, couple, reset, d_last_state, dinitial_state):
    batch, dim, L = x.shape
    g, z = _input(g, "g", x.shape, x.dtype, x), _input(z, "z", x.shape, x.dtype, x)
    dy = _input(dy, "dy", x.shape, _out_type(dy.dtype, x, "dy"), x)
    desc, reset = _desc(batch, dim, L, x, dy.dtype), _starts(reset, batch, L, x)
    ckpt = _input(ckpt, "ckpt", (lib().ss_glr_ckpt_elems(desc),), _F32, x)
    d_last_state = _input(d_last_state, "d_last_state", (batch, dim), _F32, x)
    _check(lib().ss_glr_bwd(desc, x.data_ptr(), g.data_ptr(), _p(z), 1 if gate_sigmoid else 0, 1 if couple else 0,
                            _p(reset), ckpt.data_ptr(), dy.data_ptr(), _p(d_last_state), dx.data_ptr(),
                            dg.data_ptr(), _p(dz), _p(dinitial_state), _stream(x)), "ss_glr_bwd")


@_on_device
def ss_glr_bwd(x, g, dy, ckpt, dx, dg, z=None, dz=None, gate_sigmoid=True, couple=False, reset=None,
               d_last_state=None, dinitial_state=None):
    """Queue the recurrence's backward, from the forward's checkpoints, into
    dx, dg, dz (with z) and, where given, dinitial_state."""
    x = _main(x, (3,), "x")
    _output(dx, "dx", x.shape, x.dtype, x), _output(dg, "dg", x.shape, x.dtype, x)
    _output(dz, "dz", x.shape, x.dtype, x), _output(dinitial_state, "dinitial_state", x.shape[:2], _F32, x)
    _glr_bwd(x, g, dy, ckpt, dx, dg, z, dz, gate_sigmoid, couple, reset, d_last_state, dinitial_state)


@_on_device
def gated_recurrence_bwd(x, g, dy, ckpt, z=None, gate_sigmoid=True, couple=False, reset=None, d_last_state=None,
                         return_dinitial_state=False):
    """Gradients of sum(dy * y) (+ sum(d_last_state * last state)) as a dict:
    dx, dg, dz (None without z), dinitial_state (None unless asked for).
    ckpt: gated_recurrence_fwd's, of the same inputs, initial state and starts."""
    x = _main(x, (3,), "x")
    d = {"dx": torch.empty_like(x), "dg": torch.empty_like(x), "dz": torch.empty_like(x) if z is not None else None,
         "dinitial_state": x.new_empty(x.shape[:2], dtype=_F32) if return_dinitial_state else None}
    _glr_bwd(x, g, dy, ckpt, d["dx"], d["dg"], z, d["dz"], gate_sigmoid, couple, reset, d_last_state,
             d["dinitial_state"])
    return d


def _glr_step(x, g, state, y, z, gate_sigmoid, couple):
    batch, dim = x.shape
    g, z = _input(g, "g", x.shape, x.dtype, x), _input(z, "z", x.shape, x.dtype, x)
    _output(state, "state", x.shape, _F32, x)
    _check(lib().ss_glr_step(_desc(batch, dim, 1, x, y.dtype), x.data_ptr(), g.data_ptr(), _p(z),
                             1 if gate_sigmoid else 0, 1 if couple else 0, state.data_ptr(), y.data_ptr(),
                             _stream(x)), "ss_glr_step")


@_on_device
def ss_glr_step(x, g, state, y, z=None, gate_sigmoid=True, couple=False):
    """Queue one decoding step: x, g, z, y (batch, dim); state (batch, dim)
    float32, updated in place."""
    x = _main(x, (2,), "x")
    _output(y, "y", x.shape, _out_type(y.dtype, x, "y"), x)
    _glr_step(x, g, state, y, z, gate_sigmoid, couple)


@_on_device
def gated_recurrence_step(x, g, state, z=None, gate_sigmoid=True, couple=False, out_dtype=None):
    """y (batch, dim) of one decoding step; the state is updated in place."""
    x = _main(x, (2,), "x")
    y = _new(x, out_dtype and _out_type(out_dtype, x, "out_dtype"))
    _glr_step(x, g, state, y, z, gate_sigmoid, couple)
    return y


class GatedRecurrenceFn(torch.autograd.Function):
    """The recurrence as a torch autograd Function (gradients of x, g, z and
    the initial state; through y and the last state).  The forward keeps the
    inputs and one state per 256 steps."""

    @staticmethod
    def forward(ctx, x, g, z, initial_state, reset, gate_sigmoid, couple, return_last_state):
        kw = dict(gate_sigmoid=gate_sigmoid, couple=couple, initial_state=initial_state, reset=reset,
                  return_last_state=return_last_state)
        if not any(ctx.needs_input_grad):
            return gated_recurrence_fwd(x, g, z, **kw)
        *out, ckpt = gated_recurrence_fwd(x, g, z, return_ckpt=True, **kw)
        ctx.save_for_backward(x, g, z, reset, ckpt)
        ctx.flags = (bool(gate_sigmoid), bool(couple))
        return tuple(out) if return_last_state else out[0]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dlast=None):
        x, g, z, reset, ckpt = ctx.saved_tensors
        d = gated_recurrence_bwd(x, g, dy, ckpt, z, *ctx.flags, reset=reset, d_last_state=dlast,
                                 return_dinitial_state=ctx.needs_input_grad[3])
        return d["dx"], d["dg"], d["dz"], d["dinitial_state"], None, None, None, None


def gated_recurrence_fn(x, g, z=None, gate_sigmoid=True, couple=False, initial_state=None, reset=None,
                        return_last_state=False):
    """y (and the float32 last state) of the gated linear recurrence,
    differentiable; see GatedRecurrenceFn.  g: the decays' logits, or with
    ``gate_sigmoid`` false decays in [-1, 1]."""
    return GatedRecurrenceFn.apply(x, g, z, initial_state, reset, gate_sigmoid, couple, return_last_state)
