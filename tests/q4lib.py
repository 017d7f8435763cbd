"""The 4-bit cache's format and attention in 64 bits (plain torch), for its tests."""
import numpy as np
import torch

import paged_kv_cache_pa_gb300 as pa
from cachelib import Cache

GROUP = 64


def held(x):
    """(codes, scales, least values) of x [..., D], a 16-bit type, in 64 bits: the definition,
    the range and its fifteenth in 32 bits as it says."""
    g = x.unflatten(-1, (-1, GROUP))
    z, top = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    width = top.float() - z.float()
    s = (width / 15.0).to(x.dtype)
    n = torch.clamp(torch.round((g.double() - z.double()) / s.double().masked_fill(s == 0, 1.0)), 0, 15)
    bad = ~torch.isfinite(width)
    nan = torch.full_like(s, float("nan"))
    s, z = torch.where(bad, nan, s), torch.where(bad, nan, z)
    n = torch.where(bad | (s == 0), torch.zeros_like(n), n)
    return n, s.double(), z.double()


def values(x):
    """What x reads as once it went through the cache, in 64 bits, and the bound on the terms
    of its sum, s n + |z|."""
    n, s, z = held(x)
    return (n * s + z).flatten(-2), (n * s + z.abs()).flatten(-2)


def decode_bytes(pool, D, dtype):
    """The 4-bit pool's (codes, scales, least values) from its bytes, by the layout that the
    kernels' header states: tiles of 16 tokens, cells of 64 channels, 32 bytes a token whose
    halves are exchanged in tokens 4-7 and 12-15, then scale and least value a token."""
    nb, hkv, B, row = pool.shape
    C = D // GROUP
    raw = pool.cpu().numpy().reshape(nb, hkv, B // 16, C, 576)
    nib = raw[..., :512].reshape(nb, hkv, B // 16, C, 16, 2, 16)
    swap = (np.arange(16) >> 2) & 1 == 1
    nib[..., swap, :, :] = nib[..., swap, ::-1, :].copy()
    nib = nib.reshape(nb, hkv, B // 16, C, 16, 32)
    codes = np.stack([nib & 15, nib >> 4], -1).reshape(nb, hkv, B // 16, C, 16, 64)
    par = torch.from_numpy(raw[..., 512:].copy().view(np.int16).reshape(nb, hkv, B // 16, C, 16, 2)).view(dtype)
    to = lambda t: torch.as_tensor(t).movedim(3, 4).reshape(nb, hkv, B, C, *t.shape[5:])  # noqa: E731
    return to(torch.from_numpy(codes)).double(), to(par[..., 0]).double(), to(par[..., 1]).double()


class Q4Cache(Cache):
    """A Cache (tables, lengths, 16-bit pools with NaN where no token lives) and its 4-bit
    pools, whose other bytes are all ones: scales and least values of NaN."""

    def __init__(self, lens, Hkv, D, dtype, block=16, seed=0, **kw):
        super().__init__(lens, Hkv, D, dtype, block, seed, **kw)
        dev = self.device
        slots = [torch.as_tensor(self.tables_host[s, np.arange(n) // block].astype(np.int64) * block +
                                 np.arange(n) % block, device=dev) for s, n in enumerate(self.lens_host)]
        self.slots = torch.cat(slots) if slots else torch.zeros(0, dtype=torch.int64, device=dev)
        self.k4, self.v4 = [], []
        for k, v in zip(self.k, self.v):
            shape = pa.q4_pool_shape(k.shape[0], Hkv, block, D)
            k4, v4 = (torch.full(shape, 255, dtype=torch.uint8, device=dev) for _ in range(2))
            at = (self.slots // block, slice(None), self.slots % block)
            pa.cache_write_q4(k[at].contiguous(), v[at].contiguous(), k4, v4, self.slots)
            self.k4.append(k4)
            self.v4.append(v4)


def attention(c, q, starts, scale, layer=0):
    """(out, bound on the kernel's fp32 error) in 64 bits for query rows q [T][H][D]; starts
    [S+1].

    The bound.  A logit is a sum of D products in 32 bits of q with s n, and z times a sum of
    q: off by at most (D + 8) 2^-23 of the sum of |q| (s n + |z|) in any order of addition.  A
    weight takes twice that from its exponent and the maximum's, 2^-21 from two
    exponentials, 2^-22 from its two parts in fp16.  Sums of L terms in 32 bits: L 2^-23, in
    parts that are added up (at most 2^-11).  Weights below 2^-25 of the scaled largest are
    flushed: 2^-25 15 s each, of weights that reach 2^7 s; within 2^-24 a token."""
    T, H, D = q.shape
    Hkv = c.k[layer].shape[1]
    G = H // Hkv
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for s, L in enumerate(c.lens_host):
        r0, r1 = int(starts[s]), int(starts[s + 1])
        n = r1 - r0
        if n == 0 or L == 0:
            continue
        for h in range(Hkv):
            k, kb = values(c.rows(c.k[layer], s, h))
            v, vb = values(c.rows(c.v[layer], s, h))
            x_q = q[r0:r1, h * G:(h + 1) * G].double()                       # [n][G][D]
            x = x_q @ k.T * scale
            err = (D + 8) * 2.0 ** -23 * abs(scale) * (x_q.abs() @ kb.T)
            mask = torch.ones(n, L, dtype=torch.bool, device=q.device).triu(L - n + 1)[:, None]
            x = x.masked_fill(mask, float("-inf"))
            err = err.masked_fill(mask, 0.0)
            p = torch.softmax(x, -1)
            rel = 2 * err.amax(-1, keepdim=True) + 2.0 ** -20 + min(L * 2.0 ** -23, 2.0 ** -11)
            out[r0:r1, h * G:(h + 1) * G] = p @ v
            tol[r0:r1, h * G:(h + 1) * G] = 2 * rel * (p @ vb) + L * 2.0 ** -24 * 2.0 ** -7 * vb.max()
    return out, tol


def rounded(tol, want, dtype):
    """The bound with one rounding to dtype added."""
    if dtype == torch.float32:
        return tol
    eps = torch.finfo(dtype).eps / 2
    return tol * (1 + eps) + eps * want.abs() + torch.finfo(dtype).smallest_normal * eps
