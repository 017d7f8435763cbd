"""Paged caches with shuffled blocks for the bounded-cache tests, and the
operators' definitions in 64 bits (plain torch, one head at a time)."""
import math
from fractions import Fraction

import numpy as np
import torch

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


class Cache:
    """Pools and tables of sequences of the given lengths; NaN wherever no token lives."""

    def __init__(self, lens, Hkv, D, dtype, block=16, seed=0, spare=2, device="cuda:0", layers=1):
        self.lens_host = [int(n) for n in lens]
        self.block, self.dtype, self.device = block, dtype, device
        nb = [-(-n // block) for n in self.lens_host]
        total = sum(nb) + spare
        ids = np.random.default_rng(seed).permutation(total).astype(np.int32)
        self.tables_host = np.full((len(nb), max(max(nb), 1)), -1, np.int32)
        pos = 0
        for s, n in enumerate(nb):
            self.tables_host[s, :n] = ids[pos:pos + n]
            pos += n
        self.spare = ids[pos:]
        g = torch.Generator(device=device).manual_seed(seed)
        shape = (layers, total, Hkv, block, D)
        k = torch.randn(shape, generator=g, device=device).to(dtype)
        v = torch.randn(shape, generator=g, device=device).to(dtype)
        live = torch.zeros(total, block, dtype=torch.bool, device=device)
        for s, n in enumerate(self.lens_host):
            for i in range(nb[s]):
                live[self.tables_host[s, i], :min(block, n - i * block)] = True
        k.masked_fill_(~live[None, :, None, :, None], math.nan)
        v.masked_fill_(~live[None, :, None, :, None], math.nan)
        self.k, self.v = list(k), list(v)
        self.tables = torch.as_tensor(self.tables_host, device=device)
        self.lens = torch.as_tensor(np.asarray(self.lens_host, np.int32), device=device)

    @property
    def max_len(self):
        return max(self.lens_host)

    def rows(self, pool, s, h, n=None):
        """Rows 0..n-1 of sequence s and head h, as stored."""
        n = self.lens_host[s] if n is None else n
        t = np.arange(n)
        blk = torch.as_tensor(self.tables_host[s, t // self.block].astype(np.int64), device=self.device)
        return pool[blk, h, torch.as_tensor(t % self.block, device=self.device)]


def logits64(q, k, scale):
    """(scores, bound on their fp32 error): the error of a sum of D products in 32 bits, in
    any order, is below D 2^-24 sum |q k|, and q may be scaled before the product (2^-23 more
    of every term)."""
    q, k = q.double(), k.double()
    x = q @ k.T * scale
    err = (q.shape[-1] + 2) * 2.0 ** -24 * scale * (q.abs() @ k.abs().T)
    return x, err


def weights64(x, err):
    """Softmax weights and a bound on their error: a relative 2 max err from the exponent, 2^-21
    from two exponentials, and n 2^-24 from the sum of n terms (at most 2^-12)."""
    p = torch.softmax(x, -1)
    rel = 2 * err.amax(-1, keepdim=True) + 2.0 ** -21 + min(x.shape[-1] * 2.0 ** -24, 2.0 ** -12)
    return p, p * rel


def turn_fraction(w):
    """The fraction of a turn of `w` radians (a double), times 2^64, to 2^-100."""
    def arctan_inverse(x, one):
        term = total = one // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total

    one = 1 << 1600
    two_pi = 8 * (4 * arctan_inverse(5, one) - arctan_inverse(239, one))  # Machin
    num, den = float(w).as_integer_ratio()
    return (num * one * one // (den * two_pi) % one) / Fraction(one) * 2 ** 64
