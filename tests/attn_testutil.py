"""Inputs and comparisons of the attention and rotary tests.

Tolerances (u16 = 2^-8: a bf16 value is off by at most half a step, eps / 2 of its size), per element, with
e the exact output and A = sum_j w_j |v_j| its weighted mean of magnitudes:
  - out is rounded to bf16 once: u16 |e|;
  - a score is a sum of 128 products in fp32, off by at most 128 * 2^-23 of the sum of their magnitudes (an
    accumulation that truncates); with q and k of standard deviations up to 2 and 1 that sum times the scale is
    under 32 for all but astronomically few rows: an error of 2^-11, which changes weights by 2^-11 of themselves and a
    quotient of sums of them by at most twice that: 2^-10 A.  exp2 adds 2^-22, the fp32 sums 2^-16;
  - weights go into the product as bf16: u16 A; as bf16 pairs: 2^-16 A.
Rotated values: u16 |e| and 2^-20 of the pair's size (angles off by 1e-7 and three fp32 roundings).
"""
import numpy as np
import torch

from oracle import attn

D = 128
U16 = 2.0 ** -8
SCALE = D ** -0.5
TOL_PAIR = 2.0 ** -10 + 2.0 ** -16
TOL_BF16 = 2.0 ** -10 + U16


def f64(t):
    return t.detach().to("cpu").double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


class Cache:
    """A paged cache with `lens[b]` positions of each request in scattered pages; what belongs to no position holds
    NaN.  alternate: keys and values in turn in one array."""

    def __init__(self, lens, Hkv, P, seed=0, spare=3, alternate=False, width=None):
        gen = torch.Generator().manual_seed(seed + 17)
        need = [-(-n // P) for n in lens]
        E = sum(need) + spare
        order = torch.randperm(E, generator=gen).int()
        self.width = width or max([1] + need)
        self.table = torch.full((len(lens), self.width), 1 << 30, dtype=torch.int32)  # past a request's pages: never read
        both = torch.full((E, 2, Hkv, P, D), float("nan")).bfloat16()
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            for j in range(need[b]):
                m = min(P, n - j * P)
                both[int(self.table[b, j]), :, :, :m] = torch.randn(2, Hkv, m, D, generator=gen).bfloat16()
        self.lens, self.P, self.Hkv, self.alternate = list(lens), P, Hkv, alternate
        self.both = both
        self.kv = i32(list(lens))

    def to(self, dev):
        """(k_pages, v_pages, page_table, kv_lens) on the device."""
        if self.alternate:
            both = self.both.to(dev)
            return both[:, 0], both[:, 1], self.table.to(dev), self.kv.to(dev)
        return (self.both[:, 0].contiguous().to(dev), self.both[:, 1].contiguous().to(dev), self.table.to(dev),
                self.kv.to(dev))

    def rows(self, b):
        table = self.table[b].numpy()
        return [attn.rows(f64(self.both[:, i]), table, self.lens[b]) for i in range(2)]


def queries(T, H, seed=0, spread=2.0):
    gen = torch.Generator().manual_seed(seed + 5)
    return (torch.randn(T, H * D, generator=gen) * spread).bfloat16()


def check(actual, expected, size, tol, what):
    a = np.asarray(actual, np.float64).reshape(expected.shape)
    assert np.isfinite(a).all(), f"{what}: {int((~np.isfinite(a)).sum())} values that are not finite"
    off = np.abs(a - expected)
    bad = off > U16 * np.abs(expected) + tol * size
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {float(off.max()):.3g}"
