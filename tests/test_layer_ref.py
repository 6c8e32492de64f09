"""The 64-bit references of the operators around the scan: their backward
formulas against differences of their forward, and the forward against
hand-worked values."""
import pytest
import torch

import layer_ref as R

H = 1e-6


def differences(f, args, names, outs):
    """d/dt sum_k <outs_k, f_k> by central differences in every element of
    args[n], n in names."""
    def loss():
        v = f(**args)
        return sum(float((outs[k] * v[k]).sum()) for k in outs)

    g = {}
    for n in names:
        flat, d = args[n].view(-1), torch.zeros(args[n].numel(), dtype=torch.float64)
        for i in range(flat.numel()):
            keep = float(flat[i])
            flat[i] = keep + H
            up = loss()
            flat[i] = keep - H
            d[i] = (up - loss()) / (2 * H)
            flat[i] = keep
        g[n] = d.view(args[n].shape)
    return g


def near(a, b, what):
    # central differences: H^2 of a third derivative of order one, and 2^-52 / H of rounding
    assert torch.allclose(a, b, rtol=1e-7, atol=2e-8), f"{what}: {float((a - b).abs().max()):.2e}"


def rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed + sum(shape)), dtype=torch.float64)


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients(rms):
    x, w, b, dy = rand(2, 5, 3), rand(5, seed=1), rand(5, seed=2), rand(2, 5, 3, seed=3)
    v, _ = R.norm_fwd(x, w, b, 1e-5, rms)
    g, _ = R.norm_bwd(x, dy, None if rms else v["mean"], v["rstd"], w)
    d = differences(lambda x, weight, bias: R.norm_fwd(x, weight, bias, 1e-5, rms)[0],
                    {"x": x, "weight": w, "bias": b}, ("x", "weight", "bias"), {"y": dy})
    near(g["dx"], d["x"], "dx"), near(g["dweight"], d["weight"], "dweight"), near(g["dbias"], d["bias"], "dbias")


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("L", [1, 2, 6])
def test_conv_gradients(silu, L):
    W = 4
    x, w, b, h0, dy = rand(2, 3, L), rand(3, W, seed=1), rand(3, seed=2), rand(2, 3, W - 1, seed=3), rand(2, 3, L, seed=4)
    dl, reset = rand(2, 3, W - 1, seed=5), torch.zeros((2, L), dtype=torch.uint8)
    reset[1, L // 2] = 1
    g, _ = R.conv_bwd(x, w, b, silu, dy, h0, reset, dl)
    d = differences(lambda x, weight, bias, h0: R.conv_fwd(x, weight, bias, silu, h0, reset)[0],
                    {"x": x, "weight": w, "bias": b, "h0": h0}, ("x", "weight", "bias", "h0"), {"y": dy, "last": dl})
    for k, n in (("dx", "x"), ("dweight", "weight"), ("dbias", "bias"), ("dinitial_state", "h0")):
        near(g[k], d[n], k)


@pytest.mark.parametrize("sigmoid,couple", [(True, True), (True, False), (False, True), (False, False)])
def test_recurrence_gradients(sigmoid, couple):
    x, g, z, h0, dy = (rand(2, 3, 5, seed=s) for s in (0, 1, 2, 3, 4))
    h0, dl = h0[..., 0].contiguous(), rand(2, 3, seed=5)
    reset = torch.zeros((2, 5), dtype=torch.uint8)
    reset[0, 0] = reset[1, 3] = 1
    v, _ = R.glr_bwd(x, g, dy, z, sigmoid, couple, h0, reset, dl)
    d = differences(lambda x, g, z, h0: R.glr_fwd(x, g, z, sigmoid, couple, h0, reset)[0],
                    {"x": x, "g": g, "z": z, "h0": h0}, ("x", "g", "z", "h0"), {"y": dy, "last": dl})
    for k, n in (("dx", "x"), ("dg", "g"), ("dz", "z"), ("dinitial_state", "h0")):
        near(v[k], d[n], k)


def test_hand_worked_values():
    one = lambda *v: torch.tensor(v, dtype=torch.float64).view(1, 1, -1)  # noqa: E731
    # h = 1/2 h + x from 4: 2 + 1, 1.5 + 2, then a start: 3, 1.5 + 1
    v, _ = R.glr_fwd(one(1, 2, 3, 1), one(.5, .5, .5, .5), sigmoid=False, initial_state=torch.full((1, 1), 4.0, dtype=torch.float64),
                     reset=torch.tensor([[0, 0, 1, 0]]))
    assert v["h"].flatten().tolist() == [3, 3.5, 3, 2.5]
    # taps 1, 10, 100 from a state of 7, 8; a start at step 2
    v, _ = R.conv_fwd(one(1, 2, 3, 4), torch.tensor([[1., 10., 100.]], dtype=torch.float64), None, False, one(7, 8),
                      torch.tensor([[0, 0, 1, 0]]))
    assert v["y"].flatten().tolist() == [187, 218, 300, 430] and v["last"].flatten().tolist() == [3, 4]
    v, _ = R.norm_fwd(torch.tensor([1., 3.], dtype=torch.float64).view(1, 2, 1), None, None, 0.0, False)
    assert v["y"].flatten().tolist() == [-1, 1]
