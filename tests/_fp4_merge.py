"""Long contexts over a 4-bit cache cut into many partitions: inputs on which a
lost, doubled or misplaced partition shows, the 64-bit result, and the bound that
a kernel is held to.  Every partition's values have a mean of their own (+1 or -1
per dimension) and the scores are nearly level, so that each partition carries its
share of the output."""
import math

import numpy as np
import torch

from tests import _ref64 as R

KS, VS = 1 / 256, 1 / 128
U = R.U


class Case:
    def __init__(self, lens, Hq, Hkv, D, dt, part, seed):
        rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.dt, self.part = lens, Hq, Hkv, D, dt, part
        self.scale = 1 / math.sqrt(D)
        used = [(n + 15) // 16 for n in lens]
        NB = sum(used) + 2
        perm = rng.permutation(NB)
        self.tables = np.full((len(lens), max(used)), -1, np.int32)
        key = rng.standard_normal((NB, 16, Hkv, D)).astype(np.float32)
        val = (0.3 * rng.standard_normal((NB, 16, Hkv, D))).astype(np.float32)
        at = 0
        for b, (n, u) in enumerate(zip(lens, used)):
            ids = perm[at:at + u]
            self.tables[b, :u] = ids
            at += u
            mean = rng.choice([-1.0, 1.0], (self.parts(b), Hkv, D)).astype(np.float32)
            val[ids] += mean[(np.arange(16 * u) // part).clip(max=self.parts(b) - 1)].reshape(u, 16, Hkv, D)
        self.pools, self.kv = [], []
        for x, isv, s in ((key, False, KS), (val, True, VS)):
            codes, sc = R.quantise_fp4(x, s)
            self.pools.append(R.pack_tiles(codes, sc, isv))
            self.kv.append(R.E2M1[codes] * np.repeat(R.E4M3[sc], 16, -1) * s)
        self.q = (0.25 * torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(seed))).to(dt)

    def parts(self, b):
        return (self.lens[b] + self.part - 1) // self.part

    def row(self, b):
        """Softmax weights [Hkv, G, n], values [n, Hkv, D], log2 distance of the scores from the row's maximum,
        and the largest sum of |q_d k_d| scale per head."""
        j = np.arange(self.lens[b])
        k, v = (x[self.tables[b, j // 16], j % 16] for x in self.kv)
        q = self.q[b].double().numpy().reshape(self.Hkv, -1, self.D)
        s = np.einsum("hgd,nhd->hgn", q, k) * self.scale
        mag = (np.einsum("hgd,nhd->hgn", np.abs(q), np.abs(k)) * self.scale).max(-1)
        far = (s - s.max(-1, keepdims=True)) / math.log(2.0)
        p = np.exp2(far)
        return p / p.sum(-1, keepdims=True), v, far, mag

    def result(self, b, without=()):
        """The output row [Hq, D]; `without`: partitions left out of sum and normalisation."""
        p, v, _, _ = self.row(b)
        keep = ~np.isin(np.arange(self.lens[b]) // self.part, list(without))
        p = p * keep
        return np.einsum("hgn,nhd->hgd", p / p.sum(-1, keepdims=True), v).reshape(self.Hq, self.D)

    def bound(self, b):
        """How far a kernel's row may be from result(b), per element:
          * the output's rounding, U |out| and half a subnormal step;
          * a weight w = 2^(s - r), r the running reference, enters the product with V in fp16: 2^-11 of it, or 2^-25
            where w < 2^-14.  r is never above the row's maximum M, so only weights with s < M - 14 can be that small,
            and 2^r over the softmax sum is at most the largest weight of the row;
          * a score: fp32 sums of D products and a few steps more (2^-24 of the sum of magnitudes each; 140 of them
            at D <= 128), and 2^x: 2^-20; an error d of a score moves numerator and sum by d each;
          * fp32 accumulation: a product step per 16 tokens of a partition, one addition per partition in the merge,
            and 32 more, each at most 2^-22 of the sum of p |v|."""
        p, v, far, mag = self.row(b)
        out = np.abs(self.result(b))
        A = np.einsum("hgn,nhd->hgd", p, np.abs(v)).reshape(self.Hq, self.D)
        d = 140 * 2.0 ** -24 * mag.reshape(-1, 1) + 2.0 ** -20
        small = ((far < -14).sum(-1) * p.max(-1)).reshape(-1, 1) * 2.0 ** -25 * np.abs(v).max()
        steps = (self.part / 16 + self.parts(b) + 32) * 2.0 ** -22
        return U[self.dt] * out + R.SUB[self.dt] + (2.0 ** -11 + 2 * d + steps) * A * (1 + U[self.dt]) + 2 * small


F16, BF16 = torch.float16, torch.bfloat16
SHORT = [3, 40, 17, 64, 33] * 103
CASES = {
    # few rows: a CTA merges each (row, head)
    "few_rows": dict(lens=[9000, 33000], Hq=2, Hkv=1, D=64, dt=F16, part=512, seed=1),
    "few_rows_bf16_8_columns": dict(lens=[9000, 33000], Hq=16, Hkv=2, D=128, dt=BF16, part=1024, seed=2),
    # more partitions than a pass of either merge holds (1024, 256)
    "few_rows_two_passes": dict(lens=[17000, 16500], Hq=2, Hkv=1, D=64, dt=F16, part=16, seed=3),
    # many rows: a warp merges each
    "many_rows": dict(lens=[9000, 33000] + SHORT, Hq=2, Hkv=1, D=64, dt=F16, part=512, seed=4),
    "many_rows_two_passes": dict(lens=[9000, 7777] + SHORT, Hq=2, Hkv=2, D=128, dt=F16, part=16, seed=5),
}


def drops(case, b):
    """Sets of partitions whose loss has to show: single ones, or runs of about 1 % where there are hundreds."""
    n = case.parts(b)
    run = max(1, n // 100)
    return [range(i, min(n, i + run)) for i in range(0, n, run)] if n > 1 else []
