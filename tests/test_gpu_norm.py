"""GPU parity of layer norm with the residual sum against its formulas in 64 bits.

Tolerances.  An output is rounded once to its type: half a step, eps / 2 of
the value.  Before that the row's values are computed in fp32 from sums of n
terms: mean and variance are off by at most about log2(n) + n / 64 roundings of
the terms (lane sums of n / 64, then a tree), far fewer in the root mean square;
64 fp32 steps of the largest term of the row cover it.  Weight gradients are
fp32 sums of T terms in T / (waves) + partials steps: 2^-24 sqrt(T) of the
root-sum-square of the terms would be the random walk, and 16 of these are
allowed.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
EPS32 = 2.0 ** -24


def _ttc():
    import tensor_train_compressed_tt_amd as ttc
    return ttc


def _reference(h, gamma, beta, dy, dh, eps):
    h, gamma, beta, dy = (t.double() for t in (h, gamma, beta, dy))
    n = h.shape[1]
    mean = h.sum(1, keepdim=True) / n
    c = h - mean
    rstd = 1.0 / ((c * c).sum(1, keepdim=True) / n + eps).sqrt()
    xhat = c * rstd
    u = dy * gamma
    dx = (u - u.sum(1, keepdim=True) / n - xhat * (u * xhat).sum(1, keepdim=True) / n) * rstd
    if dh is not None:
        dx = dx + dh.double()
    return {"y": xhat * gamma + beta, "dx": dx, "dgamma": (dy * xhat).sum(0), "dbeta": dy.sum(0), "xhat": xhat, "rstd": rstd,
            "c": c, "mean": mean}


def _close(got, ref, half, slack, what):
    """|got - ref| <= half |ref| + slack, element by element."""
    off = (got.double() - ref).abs() - (half * ref.abs() + slack)
    assert bool((off <= 0).all()), f"{what}: {float(off.max()):.3g} over its bound"


def _half(t):
    return torch.finfo(t).eps / 2


def _tiny(t):  # half the smallest subnormal step: what a value next to zero may lose
    f = torch.finfo(t)
    return f.smallest_normal * f.eps / 2


def _case(T, n, tx, ty, res, seed=0, eps=1e-5, dh=True, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(T, n) + shift + r(T, 1)).to(tx)
    d = {"x": x, "res": (2 * r(T, n)).to(tx) if res else None, "gamma": 1 + 0.3 * r(n), "beta": 0.2 * r(n),
         "dy": r(T, n).to(ty), "dh": r(T, n).to(tx) if dh else None}
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _check(T, n, tx, ty, res, dh=True, eps=1e-5, shift=0.0, seed=0):
    ttc = _ttc()
    d = _case(T, n, tx, ty, res, seed, eps, dh, shift)
    layer = ttc.LayerNorm(n, tx, ty, eps=eps)
    y, h, saved = layer.forward(d["x"], d["gamma"], d["beta"], res=d["res"])
    dx, dgamma, dbeta = layer.backward(d["dy"], h, d["gamma"], saved, dh=d["dh"])
    torch.cuda.synchronize()
    if res:  # one rounded sum
        assert torch.equal(h, (d["x"].float() + d["res"].float()).to(tx))
    else:
        assert h is d["x"]
    ref = _reference(h, d["gamma"], d["beta"], d["dy"], d["dh"], eps)
    # the centred value loses what the mean's size loses
    scale = (ref["c"].abs().amax(1, keepdim=True) + ref["mean"].abs()) * ref["rstd"]
    _close(y, ref["y"], _half(ty), 64 * EPS32 * (scale * d["gamma"].abs().max() + d["beta"].abs().max()) + _tiny(ty), "y")
    u = (d["dy"].double() * d["gamma"].double()).abs().amax(1, keepdim=True)
    _close(dx, ref["dx"], _half(tx), 64 * EPS32 * (u * (1 + scale) * ref["rstd"] * (1 + scale) + (0 if d["dh"] is None else d["dh"].double().abs())), "dx")
    for name, got, terms in (("dgamma", dgamma, d["dy"].double() * ref["xhat"]), ("dbeta", dbeta, d["dy"].double())):
        slack = 16 * EPS32 * (T ** 0.5) * (terms.square().sum(0).sqrt() + (scale.max() * d["dy"].double().abs().max() if name == "dgamma" else 0))
        _close(got, ref[name], EPS32, slack + 1e-30, name)


@pytest.mark.parametrize("tx", [F32, BF16])
@pytest.mark.parametrize("ty", [F32, BF16, FP8])
@pytest.mark.parametrize("res", [False, True])
def test_types(tx, ty, res):
    _check(70, 768, tx, ty, res, dh=res)


# one element, around a wave, each register form and its ends, the looped form
@pytest.mark.parametrize("n", [1, 2, 3, 4, 63, 64, 65, 252, 256, 257, 260, 511, 512, 516, 768, 1001, 1020, 1023, 1024, 1025, 1028, 2048,
                               2052, 3001, 4092, 4095, 4096, 4097, 5000, 9001])
@pytest.mark.parametrize("tx,ty", [(BF16, BF16), (F32, FP8)])
def test_widths(n, tx, ty):
    _check(37, n, tx, ty, True, seed=n)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 255, 1024, 4095, 4096, 4097, 20001])
def test_token_counts(T):
    _check(T, 96, BF16, BF16, True, seed=T)
    _check(T, 97, F32, F32, False, seed=T)


@pytest.mark.parametrize("T", [1, 15, 16, 33, 1025])
def test_long_rows_token_counts(T):
    _check(T, 4100, F32, BF16, True, seed=T)


def test_large_mean():
    """A mean far over the deviation: the variance must come from centred values."""
    _check(64, 768, F32, F32, False, shift=1000.0)


def test_constant_rows_and_zero_eps():
    ttc = _ttc()
    layer = ttc.LayerNorm(256, F32, F32, eps=1e-5)
    x = torch.full((3, 256), 2.5, device="cuda")
    gamma, beta = torch.ones(256, device="cuda"), torch.arange(256, device="cuda", dtype=F32)
    y, h, saved = layer.forward(x, gamma, beta)
    assert torch.equal(y, beta.expand(3, 256))
    dx, dgamma, dbeta = layer.backward(torch.ones_like(x), h, gamma, saved)
    assert torch.equal(dgamma, torch.zeros_like(gamma)) and torch.equal(dbeta, torch.full_like(beta, 3.0))
    assert torch.equal(dx, torch.zeros_like(dx))
    # eps = 0 on a constant row: 0 / 0 by the formula
    y, _, _ = ttc.LayerNorm(256, F32, F32, eps=0.0).forward(x, gamma, beta)
    assert bool(torch.isnan(y).all())


def test_nan_and_infinity_stay_in_their_rows():
    ttc = _ttc()
    for ty in (F32, BF16, FP8):
        d = _case(8, 768, F32, ty, False)
        layer = ttc.LayerNorm(768, F32, ty)
        clean = layer.forward(d["x"], d["gamma"], d["beta"])[0].float()
        d["x"][2, 5], d["x"][6, 700] = float("nan"), float("inf")
        y = layer.forward(d["x"], d["gamma"], d["beta"])[0].float()
        bad = torch.tensor([2, 6], device="cuda")
        keep = torch.tensor([0, 1, 3, 4, 5, 7], device="cuda")
        assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[keep], clean[keep])


def test_e4m3_saturates():
    ttc = _ttc()
    x = torch.randn(4, 64, generator=torch.Generator().manual_seed(1)).cuda()
    gamma, beta = torch.full((64,), 1000.0, device="cuda"), torch.zeros(64, device="cuda")
    y = ttc.LayerNorm(64, F32, FP8).forward(x, gamma, beta)[0].float()
    full = ttc.LayerNorm(64, F32, F32).forward(x, gamma, beta)[0]
    assert torch.equal(y[full.abs() >= 464], torch.sign(full[full.abs() >= 464]) * 448)
    assert float(y.abs().max()) == 448.0


def test_no_tokens():
    ttc = _ttc()
    layer = ttc.LayerNorm(100, BF16, BF16)
    x, gamma = torch.empty((0, 100), dtype=BF16, device="cuda"), torch.ones(100, device="cuda")
    y, h, saved = layer.forward(x, gamma, gamma)
    assert y.shape == (0, 100)
    dgamma, dbeta = (torch.full((100,), 7.0, device="cuda") for _ in range(2))
    layer.backward(x, h, gamma, saved, dgamma=dgamma, dbeta=dbeta)
    assert not bool(dgamma.any()) and not bool(dbeta.any())


def test_gradient_is_the_difference_quotient():
    """d(sum dy y)/dx, /dgamma, /dbeta against central differences of the kernel's
    own forward, in fp32 rows scaled so that a step of 2^-6 moves y by far more
    than its rounding: the quotient's own error is step^2 times the third
    derivative (below 1e-3 here) plus two roundings of a sum of 2 * 24 values."""
    ttc = _ttc()
    d = _case(2, 24, F32, F32, False, seed=5, dh=False)
    layer = ttc.LayerNorm(24, F32, F32)
    f = lambda: float((layer.forward(d["x"], d["gamma"], d["beta"])[0].double() * d["dy"].double()).sum())  # noqa: E731
    _, h, saved = layer.forward(d["x"], d["gamma"], d["beta"])
    dx, dgamma, dbeta = layer.backward(d["dy"], h.clone(), d["gamma"], saved)
    step = 2.0 ** -6
    for t, grad in ((d["x"], dx), (d["gamma"], dgamma), (d["beta"], dbeta)):
        flat, got = t.view(-1), grad.view(-1)
        for i in range(0, flat.numel(), 5):
            was = float(flat[i])
            flat[i] = was + step
            hi, up = f(), float(flat[i])
            flat[i] = was - step
            lo, down = f(), float(flat[i])
            flat[i] = was
            assert abs((hi - lo) / (up - down) - float(got[i])) < 5e-3


def test_repeatable_and_captured():
    """Bitwise the same on every call, and in a graph replayed between eager work."""
    ttc = _ttc()
    d = _case(1000, 768, BF16, BF16, True)
    layer = ttc.LayerNorm(768, BF16, BF16)

    def step():
        y, h, saved = layer.forward(d["x"], d["gamma"], d["beta"], res=d["res"])
        return (y, h) + layer.backward(d["dy"], h, d["gamma"], saved, dh=d["dh"])

    first = [t.clone() for t in step()]
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    x0 = d["x"].clone()
    for k in range(4):
        d["x"].copy_(x0 * (1 + k))
        g.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), k


def test_other_stream():
    ttc = _ttc()
    d = _case(500, 768, BF16, F32, True)
    layer = ttc.LayerNorm(768, BF16, F32)
    want = layer.forward(d["x"], d["gamma"], d["beta"], res=d["res"])[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = layer.forward(d["x"], d["gamma"], d["beta"], res=d["res"])[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    ttc = _ttc()
    layer = ttc.LayerNorm(64, BF16, BF16)
    ok = lambda *s, t=BF16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    gamma = ok(64, t=F32)
    with pytest.raises(ValueError):
        layer.forward(ok(4, 65), gamma, gamma)
    with pytest.raises(ValueError):
        layer.forward(ok(4, 64, t=F32), gamma, gamma)
    with pytest.raises(ValueError):
        layer.forward(ok(64, 4).t(), gamma, gamma)
    with pytest.raises(ValueError):
        layer.forward(ok(4, 64), gamma, gamma, h=ok(4, 64))
    with pytest.raises(ttc.TTCError) as e:  # rows from the middle of a buffer, 2 bytes off
        layer.forward(ok(300)[1:257].view(4, 64), gamma, gamma)
    assert e.value.code == 5
    with pytest.raises(ttc.TTCError) as e:
        layer.forward(ok(4, 64), gamma, gamma, saved=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 6
