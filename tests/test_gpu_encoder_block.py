"""The example block: its gradients against the formulas in 64 bits, its training, and its single-token pass.

Tolerances.  fp32: a gradient passes through at most a dozen operators, each off by
at most 64 fp32 half steps of its terms' size in the root mean square, and none of
them enlarges a relative error by more than a few times: 1e-4 in the relative L2
norm is twelve times 64 2^-24 (4.6e-5) doubled.  Decoding against the training pass
is the same sums in another order: the same bound in fp32; in bf16 the two round
every activation (2^-8 each) differently where they differ at all: 2^-6.
"""

import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _rel(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


def _dense(cores, n_out):
    t = cores[0]
    for c in cores[1:]:
        t = torch.tensordot(t, c, dims=1)
    return t.reshape(n_out, -1)


def _reference(block, x, lens, window, sinks, heads):
    """The block on the CPU in 64 bits, with autograd on the cores."""
    cores = {n: [c.detach().double().cpu().requires_grad_(True) for c in block.cores[n]] for n in block.LAYERS}
    gamma, beta = ([p.detach().double().cpu().requires_grad_(True) for p in ps] for ps in (block.gamma, block.beta))
    w = {n: _dense(cores[n], block.tt[n].n_out) for n in block.LAYERS}
    x = x.detach().double().cpu().requires_grad_(True)
    norm = lambda h, k: torch.nn.functional.layer_norm(h, (block.width,), gamma[k], beta[k], 1e-5)  # noqa: E731
    y1 = norm(x, 0)
    q, k, v = (y1 @ w[n].t() for n in "qkv")
    parts, at, d = [], 0, block.width // heads
    for n in lens:
        cut = lambda t: t[at:at + n].view(n, heads, d).transpose(0, 1)  # noqa: E731
        i, j = torch.arange(n)[:, None], torch.arange(n)[None, :]
        seen = (j <= i) & ((j >= i - window) | (j < sinks))
        s = (cut(q) @ cut(k).transpose(1, 2) * d ** -0.5).masked_fill(~seen, float("-inf"))
        parts.append((s.softmax(-1) @ cut(v)).transpose(0, 1).reshape(n, -1))
        at += n
    h = x + torch.cat(parts) @ w["o"].t()
    return x, cores, gamma, beta, h + torch.relu(norm(h, 1) @ w["ffn1"].t()) @ w["ffn2"].t()


def _setup(dtype, lens, **kw):
    from encoder_block import Block
    block = Block(dtype=dtype, **kw)
    g = torch.Generator().manual_seed(7)
    x, dout = (torch.randn(sum(lens), block.width, generator=g).to(dtype).cuda() for _ in range(2))
    return block, x, dout, torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()


@pytest.mark.parametrize("lens", [[50, 1, 128, 33], [200, 7]])
def test_gradients(lens):
    block, x, dout, offsets = _setup(torch.float32, lens)
    out, saved = block.forward(x, offsets, max(lens))
    dx, grads, dgamma, dbeta = block.backward(dout, saved)
    rx, cores, gamma, beta, ref = _reference(block, x, lens, 24, 1, 4)
    ref.backward(dout.double().cpu())
    assert _rel(out, ref.detach()) < 1e-4 and _rel(dx, rx.grad) < 1e-4
    for k in range(2):
        assert _rel(dgamma[k], gamma[k].grad) < 1e-4 and _rel(dbeta[k], beta[k].grad) < 1e-4
    for n in block.LAYERS:
        for got, want in zip(grads[n], cores[n]):
            assert _rel(got, want.grad) < 1e-4, n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_lowers_the_loss(dtype):
    from encoder_block import Block, train
    lens = [100, 37, 128, 1, 64]
    block, x, _, offsets = _setup(dtype, lens)
    target, _ = Block(dtype=dtype, seed=1).forward(x, offsets, max(lens))
    losses = train(block, x, target, offsets, max(lens), 40)
    assert losses[-1] < 0.7 * losses[0] and all(l == l for l in losses)


@pytest.mark.parametrize("dtype,bound", [(torch.float32, 1e-4), (torch.bfloat16, 2.0 ** -6)])
def test_decoding_gives_the_training_pass(dtype, bound):
    lens = [70]
    block, x, _, offsets = _setup(dtype, lens)
    out, _ = block.forward(x, offsets, 70)
    cache = [torch.full((1, 75, block.width), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = torch.cat([block.decode(x[i:i + 1], *cache, n) for i in range(70)])
    assert int(n) == 70 and _rel(got, out.double().cpu()) < bound
