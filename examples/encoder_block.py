"""A transformer block of tensor-train layers, trained and then served one token at a time.

    python examples/encoder_block.py [--steps 60] [--dtype bf16|f32]

The block, with every link diagonal at one:

    y1 = norm1(x);  a = attention(Q y1, K y1, V y1);  h = x + O a
    y2 = norm2(h);  out = h + FFN2 relu(FFN1 y2)

Q, K, V, O and the FFN are TTLinear layers, the norms LayerNorm (the second one adds O a to x by itself),
the attention WindowAttention (causal, a sliding window, the first token kept visible), and the cores are
updated by OrthogonalUpdate.  Training fits the outputs of another block of the same shape, on sequences of
unequal length packed without padding; serving then decodes one of them token by token over a cache and
compares with the training pass.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tensor_train_compressed_tt_amd as ttc  # noqa: E402


class Block:
    """Parameters, the two passes and the single-token pass of the block."""

    LAYERS = ("q", "k", "v", "o", "ffn1", "ffn2")

    def __init__(self, d_modes=(8, 4, 4), f_modes=(8, 8, 4), rank=8, heads=4, window=24, sinks=1, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        ranks = [1] + [rank] * 5 + [1]
        self.dtype, self.tt, self.cores, self.links = dtype, {}, {}, {}
        for name in self.LAYERS:
            out, into = (f_modes, d_modes) if name == "ffn1" else (d_modes, f_modes) if name == "ffn2" else (d_modes, d_modes)
            layer = self.tt[name] = ttc.TTLinear(out, into, ranks, dtype)
            # a chain of six cores whose product has elements of variance 1 / n_in
            std = (layer.n_in * rank ** 5) ** (-1 / 12)
            self.cores[name] = [(torch.randn(s, generator=g) * std).cuda() for s in layer.core_shapes]
            self.links[name] = [torch.ones(s[2], device="cuda") for s in layer.core_shapes[:-1]]
        self.width = self.tt["q"].n_out
        self.norm = [ttc.LayerNorm(self.width, dtype) for _ in range(2)]
        self.gamma = [torch.ones(self.width, device="cuda") for _ in range(2)]
        self.beta = [torch.zeros(self.width, device="cuda") for _ in range(2)]
        self.attention = ttc.WindowAttention(heads, self.width // heads, window=(window, 0), sinks=sinks, dtype=dtype)

    def _linear(self, name, x):
        return self.tt[name].forward(x, self.cores[name], self.links[name])

    def _linear_back(self, name, x, dy, saved, grads):
        dx, grads[name] = self.tt[name].backward(x, dy, self.cores[name], self.links[name], saved)
        return dx

    def forward(self, x, offsets, longest):
        """(out, what the backward needs); x: all sequences' tokens, offsets: where they begin, and the end."""
        s = {"x": x, "seqs": dict(batch=offsets.numel() - 1, q_offsets=offsets, k_offsets=offsets, max_q=longest)}
        s["y1"], _, s["n1"] = self.norm[0].forward(x, self.gamma[0], self.beta[0])
        for name in "qkv":
            s[name], s["s" + name] = self._linear(name, s["y1"])
        s["a"], s["sa"] = self.attention.forward(s["q"], s["k"], s["v"], **s["seqs"])
        o, s["so"] = self._linear("o", s["a"])
        s["y2"], s["h"], s["n2"] = self.norm[1].forward(x, self.gamma[1], self.beta[1], res=o)
        f, s["sf1"] = self._linear("ffn1", s["y2"])
        s["r"] = torch.relu(f)
        f2, s["sf2"] = self._linear("ffn2", s["r"])
        return s["h"] + f2, s

    def backward(self, dout, s):
        """(dx, gradients of the cores by layer, of gamma, of beta)."""
        grads = {}
        df = self._linear_back("ffn2", s["r"], dout, s["sf2"], grads) * (s["r"] > 0)
        dy2 = self._linear_back("ffn1", s["y2"], df, s["sf1"], grads)
        dh, dg2, db2 = self.norm[1].backward(dy2, s["h"], self.gamma[1], s["n2"], dh=dout)  # of x and of O a alike
        da = self._linear_back("o", s["a"], dh, s["so"], grads)
        dqkv = self.attention.backward(s["q"], s["k"], s["v"], s["a"], da, s["sa"], **s["seqs"])
        dy1 = sum(self._linear_back(name, s["y1"], d, s["s" + name], grads).float() for name, d in zip("qkv", dqkv))
        dx, dg1, db1 = self.norm[0].backward(dy1.to(self.dtype), s["x"], self.gamma[0], s["n1"], dh=dh)
        return dx, grads, [dg1, dg2], [db1, db2]

    def decode(self, x, cache_k, cache_v, lens):
        """The block for one new token of each sequence; the caches (batch, capacity, width) get its k and v at lens, which then counts it."""
        rows = torch.arange(x.shape[0], device=x.device)
        y1, _, _ = self.norm[0].forward(x, self.gamma[0], self.beta[0])
        q, k, v = (self._linear(name, y1)[0] for name in "qkv")
        cache_k[rows, lens.long()], cache_v[rows, lens.long()] = k, v
        lens += 1
        a = self.attention.decode(q, cache_k, cache_v, lens)
        y2, h, _ = self.norm[1].forward(x, self.gamma[1], self.beta[1], res=self._linear("o", a)[0])
        return h + self._linear("ffn2", torch.relu(self._linear("ffn1", y2)[0]))[0]


def train(block, x, target, offsets, longest, steps, lr=0.01):
    """Losses of `steps` steps: the cores by OrthogonalUpdate, the norms' weights by plain descent."""
    grads = {n: [torch.zeros_like(c) for c in block.cores[n]] for n in block.LAYERS}
    flat = lambda by: [t for n in block.LAYERS for t in by[n]]  # noqa: E731
    update = ttc.OrthogonalUpdate(flat(block.cores), flat(grads), [torch.zeros_like(c) for c in flat(block.cores)])
    losses = []
    for k in range(steps):
        out, saved = block.forward(x, offsets, longest)
        off = out.float() - target.float()
        losses.append(off.square().mean())
        _, got, dgamma, dbeta = block.backward((off * (2 / off.numel())).to(block.dtype), saved)
        for to, of in zip(flat(grads), flat(got)):
            to.copy_(of)
        update.step(lr * (1 - k / steps))
        for p, d in zip(block.gamma + block.beta, dgamma + dbeta):
            p -= lr * d
    return [float(t) for t in losses]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", default="bf16", choices=["bf16", "f32"])
    args = ap.parse_args()
    dtype = torch.bfloat16 if args.dtype == "bf16" else torch.float32
    lens = [100, 37, 128, 1, 64, 90]
    offsets = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    block, teacher = Block(dtype=dtype), Block(dtype=dtype, seed=1)
    x = torch.randn(sum(lens), block.width, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    target, _ = teacher.forward(x, offsets, max(lens))
    losses = train(block, x, target, offsets, max(lens), args.steps)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {args.steps} steps")
    out, _ = block.forward(x, offsets, max(lens))
    first = out[:lens[0]]
    cache = [torch.zeros(1, lens[0], block.width, dtype=dtype, device="cuda") for _ in range(2)]
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = torch.cat([block.decode(x[i:i + 1], *cache, n) for i in range(lens[0])])
    print(f"decoded {lens[0]} tokens: {float((got.float() - first.float()).norm() / first.float().norm()):.2e} from the training pass")


if __name__ == "__main__":
    main()
