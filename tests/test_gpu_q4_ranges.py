"""decode_attention_q4 against 64 bits with q4tight's bound: values and queries next to the ends
of their type, scales far apart."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
import q4tight
from q4lib import Q4Cache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _query(T, H, D, dtype, seed=0, factor=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed + 177)
    return (torch.randn(T, H, D, generator=g, device=DEV) * factor).to(dtype)


def _decode(c, q, starts=None, most=1, scale=None, **kw):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qsl = None if starts is None else torch.as_tensor(np.asarray(starts, np.int32), device=DEV)
    out = pa.decode_attention_q4(q, c.k4[0], c.v4[0], c.tables, c.lens, c.max_len, scale, query_start_loc=qsl,
                                 max_query_len=most, error_word=err, **kw)
    assert int(err.item()) == 0
    return out


def _check(c, q, starts=None, most=1, scale=None, seqs=None, sharp=50, **kw):
    """sharp: the bound is that much smaller than the output, or the test would show nothing."""
    out = _decode(c, q, starts, most, scale, **kw)
    s = q.shape[-1] ** -0.5 if scale is None else scale
    at = list(range(len(c.lens_host) + 1)) if starts is None else starts
    want, tol = q4tight.attention(c, q, at, s, seqs=seqs)
    rows = ~torch.isnan(tol[:, 0, 0])
    share, size = q4tight.off(out[rows], want[rows], tol[rows])
    assert share <= 1.0, (share, size)
    assert sharp is None or size * sharp <= 1.0, size


def _rewrite(c):
    """The 4-bit pools from c.k and c.v as they are now."""
    at = (c.slots // c.block, slice(None), c.slots % c.block)
    pa.cache_write_q4(c.k[0][at].contiguous(), c.v[0][at].contiguous(), c.k4[0], c.v4[0], c.slots)


ROWS = [(1, 1, 64), (4, 2, 64), (8, 2, 64), (6, 1, 64), (16, 1, 64), (2, 2, 128), (4, 2, 128), (8, 2, 128), (12, 2, 128),
        (12, 1, 128), (2, 2, 256), (4, 1, 256), (6, 1, 256)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", ROWS)
def test_values_near_the_largest(H, Hkv, D, dtype):
    """Groups whose range is just held, and others of ordinary size beside them: finite values
    give finite outputs."""
    top = torch.finfo(DT[dtype]).max
    c = Q4Cache([300, 40, 2000, 16], Hkv, D, DT[dtype], seed=D)
    g = torch.Generator(device=DEV).manual_seed(1)
    live = ~torch.isnan(c.v[0])
    c.v[0].copy_(torch.where(live, (torch.rand(c.v[0].shape, generator=g, device=DEV) * 0.98 - 0.49) * top, c.v[0]))
    if D > 64:
        c.v[0][..., 64:128] = torch.where(live[..., 64:128], c.v[0][..., 64:128] / top, c.v[0][..., 64:128])
    _rewrite(c)
    _check(c, _query(4, H, D, DT[dtype]), sharp=None)
    # one sign: the sums of all tokens stay below the largest value only as they are weighted
    c.v[0].copy_(torch.where(live, (c.v[0].abs() + 0.4 * top).to(DT[dtype]), c.v[0]))
    _rewrite(c)
    _check(c, _query(4, H, D, DT[dtype], seed=1), sharp=None)


@pytest.mark.parametrize("H,Hkv,D", ROWS)
def test_queries_and_keys_next_to_the_ends(H, Hkv, D):
    """Powers of two on the query or the keys, taken back by the scale, change nothing."""
    c = Q4Cache([300, 20, 1000], Hkv, D, torch.bfloat16, seed=8)
    q = _query(3, H, D, torch.bfloat16)
    scale = 2.0 ** -3
    want = _decode(c, q, scale=scale)
    _check(c, q, scale=scale, sharp=None)
    for e in (-100, -60, 60, 110, 120):
        assert torch.equal(_decode(c, q * 2.0 ** e, scale=scale * 2.0 ** -e), want), e
    k = c.k[0].clone()
    for e in (-60, 60, 100):
        c.k[0].copy_(k * 2.0 ** e)
        _rewrite(c)
        assert torch.equal(_decode(c, q, scale=scale * 2.0 ** -e), want), e
    # (the scale times the query's sums is subnormal here: off by 2^-149 of keys of 2^117, far
    # less than a logit's bound)
    c.k[0].copy_(k * 2.0 ** 115)
    _rewrite(c)
    _check(c, q, scale=scale * 2.0 ** -115, sharp=None)
    c.k[0].copy_(k * 2.0 ** 60)
    _rewrite(c)
    assert torch.equal(_decode(c, q * 2.0 ** -60, scale=scale), want)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", ROWS)
def test_a_token_without_weight_does_not_coarsen_the_others(H, Hkv, D, dtype):
    """A few tokens of huge values, far below every other token's logit: the others keep their
    bits, wherever in the context those tokens are."""
    dt = DT[dtype]
    lens = [900, 50, 4000]
    c = Q4Cache(lens, Hkv, D, dt, seed=11)
    small, big = (2.0 ** -7, 2.0 ** 14) if dtype == "f16" else (2.0 ** -20, 2.0 ** 40)
    c.v[0] *= small
    c.k[0][..., 0] = torch.where(torch.isnan(c.k[0][..., 0]), c.k[0][..., 0], torch.zeros_like(c.k[0][..., 0]))
    far = torch.cat([c.slots[torch.tensor([3, 400, 895, 900 + 20, 950, 3000, 4940])]])
    at = (far // 16, slice(None), far % 16)
    c.v[0][at] = (torch.sign(c.v[0][at].float()) * big).to(dt)
    k = c.k[0][at]
    k[..., 0] = -200.0
    c.k[0][at] = k
    _rewrite(c)
    q = _query(3, H, D, dt)
    q[..., 0] = 16.0
    _check(c, q, sharp=None, scale=1.0 if dtype == "bf16" else D ** -0.5)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", [r for r in ROWS if r[2] > 64])
def test_groups_of_channels_keep_their_own_precision(H, Hkv, D, dtype):
    """Groups of 64 channels whose values are far apart, in all tokens."""
    dt = DT[dtype]
    c = Q4Cache([700, 33, 1800], Hkv, D, dt, seed=12)
    step = 2.0 ** -5 if dtype == "f16" else 2.0 ** -20
    for i in range(D // 64):
        c.v[0][..., i * 64:(i + 1) * 64] *= step ** i
    _rewrite(c)
    _check(c, _query(3, H, D, dt), sharp=None)


@pytest.mark.parametrize("H,Hkv,D", ROWS)
@pytest.mark.parametrize("up", [True, False])
def test_values_that_grow_or_shrink_along_the_context(H, Hkv, D, up):
    """Scales that move by a factor of two every 40 tokens, with logits that move the other way:
    what counts at last is not what counted at first."""
    c = Q4Cache([1200, 90], Hkv, D, torch.bfloat16, seed=13)
    for s, n in enumerate(c.lens_host):
        i = torch.arange(n, device=DEV) // 40
        i = i if up else i.flip(0)
        at = torch.as_tensor(c.tables_host[s, np.arange(n) // 16].astype(np.int64), device=DEV)
        o = torch.arange(n, device=DEV) % 16
        c.v[0][at, :, o] *= torch.exp2(i.float()).bfloat16()[:, None, None]
        k = c.k[0][at, :, o]
        k[..., 0] = -(i.float() * 0.7).bfloat16()[:, None]
        c.k[0][at, :, o] = k
    _rewrite(c)
    q = _query(2, H, D, torch.bfloat16, factor=0.5)
    q[..., 0] = 1.0
    _check(c, q, scale=1.0 if D == 64 else 0.7, sharp=None)


@pytest.mark.parametrize("H,Hkv,D", ROWS)
@pytest.mark.parametrize("logit", [-2.3e38, -2.2e38, 2.3e38])
def test_equal_logits_next_to_the_end_of_fp32(H, Hkv, D, logit):
    """Keys that are all alike: every logit the same, next to the largest of either sign (in
    units of log2 3.3e38), and every weight 1 / L."""
    lens = [40, 600]
    c = Q4Cache(lens, Hkv, D, torch.bfloat16, seed=21)
    c.k[0][...] = torch.where(torch.isnan(c.k[0]), c.k[0], torch.ones_like(c.k[0]))
    _rewrite(c)
    q = torch.ones(2, H, D, dtype=torch.bfloat16, device=DEV)
    out = _decode(c, q, scale=logit / D).double()
    want, tol = q4tight.attention(c, torch.zeros_like(q), range(3), 1.0)
    assert q4tight.off(out.float(), want, tol)[0] <= 1.0
