"""A bound on decode_attention_q4's error that a lost or doubled part of a context, sums that
drift, or lost bits of small values do not meet: an error model by squares, against values as
they are weighted, where q4lib.attention adds up worst cases of all tokens.

With p_j the weights, v = s n + z a group's values, b = s n + |z|, the error of a row's 64
channels of a group, as a length, is below the sum of

* 4 sqrt(sum_j p_j^2 d_j^2 |b_j|^2): errors of the weights, independent from token to token (a
  row's weights do not know its values), four deviations.  d_j = 2^-18 + 2^-20 |scale| sum |q| b:
  two parts of a weight 2^-19, exponential and maximum 2^-22 each; a logit's sums are cut off
  up to eight times a group of channels, by 2^-23 of what they reach.
* 8 (the length of 64 channels) times 2^-18 sum_j p_j s_j: the values' products are cut off
  towards zero up to twice in a sum, which reaches 7.5 sum p s in two equal steps:
  2^-23 (3.75 + 7.5) < 2^-19, for each of the two parts of a weight.
* 8 times 2^-18 sum_j p_j (|z_j| + 7.5 s_j): a warp adds up at most 2^13 tokens, an eighth in each
  lane: 2^10 roundings by 2^-24 of the sum, 2^-19 as a random walk, of the least values and of
  the products' sums; the lanes' parts are an eighth each and independent, so that this is five
  deviations.

and one rounding of the output.
"""
import torch

from q4lib import GROUP, held


def attention(c, q, starts, scale, layer=0, seqs=None):
    """(out, bound): out [T][H][D] in 64 bits, bound [T][H][D / 64] on the length of the error
    of a group of channels.  seqs: the sequences to work out (the other rows are NaN)."""
    T, H, D = q.shape
    Hkv = c.k[layer].shape[1]
    G = H // Hkv
    out = torch.full((T, H, D), float("nan"), dtype=torch.float64, device=q.device)
    tol = torch.full((T, H, D // GROUP), float("nan"), dtype=torch.float64, device=q.device)
    for s, L in enumerate(c.lens_host):
        r0, r1 = int(starts[s]), int(starts[s + 1])
        n = r1 - r0
        if n == 0 or (seqs is not None and s not in seqs):
            continue
        if L == 0:
            out[r0:r1], tol[r0:r1] = 0.0, 0.0
            continue
        for h in range(Hkv):
            o, t = rows_attention(c.rows(c.k[layer], s, h), c.rows(c.v[layer], s, h),
                                  q[r0:r1, h * G:(h + 1) * G], scale)
            out[r0:r1, h * G:(h + 1) * G], tol[r0:r1, h * G:(h + 1) * G] = o, t
    return out, tol


def rows_attention(k, v, q, scale):
    """The same for one sequence and KV head: k, v [L][D] in 16 bits, q [n][G][D]."""
    (n, G, D), L = q.shape, k.shape[0]
    kn, ks, kz = held(k)
    vn, vs, vz = held(v)
    keys, key_terms = (kn * ks + kz).flatten(-2), (kn * ks + kz.abs()).flatten(-2)
    vals, val_terms = (vn * vs + vz).flatten(-2), vn * vs + vz.abs()          # [L][D], [L][C][64]
    x = q.double().reshape(n * G, D)
    d = 2.0 ** -18 + 2.0 ** -20 * abs(scale) * (x.abs() @ key_terms.T)
    mask = torch.ones(n, L, dtype=torch.bool, device=q.device).triu(L - n + 1)
    mask = mask[:, None].expand(n, G, L).reshape(n * G, L)
    p = torch.softmax((x @ keys.T * scale).masked_fill(mask, float("-inf")), -1)
    squares = val_terms.square().sum(-1)                                     # [L][C]
    tol = 4 * ((p * d).square() @ squares).sqrt()
    tol += 8 * 2.0 ** -18 * (p @ vs[..., 0])
    tol += 8 * 2.0 ** -18 * (p @ (vz.abs() + 7.5 * vs)[..., 0])
    return (p @ vals).view(n, G, D), tol.view(n, G, D // GROUP)


def off(out, want, tol):
    """(largest error as a share of the bound, largest bound as a share of the output's length)
    over rows and groups; the output's own rounding is allowed for.  NaN counts as off."""
    a, b = (t.double().unflatten(-1, (-1, GROUP)) for t in (out, want))
    size = b.norm(dim=-1)
    room = tol + torch.finfo(out.dtype).eps / 2 * size + torch.finfo(out.dtype).smallest_normal
    share = torch.nan_to_num((a - b).norm(dim=-1) / room, nan=float("inf"), posinf=float("inf"))
    return float(share.max()), float((tol / size.clamp(min=1e-300)).max())
