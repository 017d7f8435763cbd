"""decode_attention_q4 against 64 bits with q4tight's bound: long contexts, cut into the parts
of many warps."""
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


ROWS = [(1, 1, 64), (4, 2, 64), (8, 2, 64), (6, 1, 64), (16, 1, 64), (2, 2, 128), (4, 2, 128), (8, 2, 128), (12, 2, 128),
        (12, 1, 128), (2, 2, 256), (4, 1, 256), (6, 1, 256)]


@pytest.mark.parametrize("H,Hkv,D", ROWS)
def test_long_contexts(H, Hkv, D):
    c = Q4Cache([50001, 700, 20000], Hkv, D, torch.bfloat16, 64, seed=H)
    _check(c, _query(3, H, D, torch.bfloat16))


@pytest.mark.parametrize("H,Hkv,D,most", [(8, 2, 128, 4), (12, 2, 128, 5), (4, 1, 256, 7), (16, 2, 64, 16), (2, 2, 128, 3)])
def test_long_drafts(H, Hkv, D, most):
    c = Q4Cache([9000, 333, 17001], Hkv, D, torch.float16, 16, seed=most)
    starts = [0, most, most + 1, 2 * most + 1]
    _check(c, _query(starts[-1], H, D, torch.float16), starts, most)


@pytest.mark.parametrize("H,Hkv,D", ROWS)
def test_sums_do_not_drift(H, Hkv, D):
    """Warps with hundreds of chunks of one context (32 sequences that share the blocks of a long
    one): sums of one sign that were cut off towards zero would be off by a percent of the output."""
    S, L = 32, 40000
    c = Q4Cache([L], Hkv, D, torch.float16, 64, seed=3)
    c.lens_host, c.tables = c.lens_host * S, c.tables.expand(S, -1).contiguous()
    c.tables_host, c.lens = np.repeat(c.tables_host, S, 0), torch.full((S,), L, dtype=torch.int32, device=DEV)
    _check(c, _query(S, H, D, torch.float16), seqs=(0, 17, 31))


@pytest.mark.parametrize("H,Hkv,D", ROWS)
@pytest.mark.parametrize("lens", [[131072], [70001, 5, 40000], [4096, 300] * 20])
def test_every_chunk_counts(H, Hkv, D, lens):
    """All weights alike, and values of +1 and -1 that spell the number of their chunk of 16 tokens:
    a chunk that is lost or taken twice moves some channel by 1 / chunks."""
    c = Q4Cache([16], Hkv, D, torch.float16, 16)
    most = -(-max(lens) // 16)
    # block i holds chunk i: channels d mod 64 its bits, the first of a group +1 and the last -1
    bit = (torch.arange(most, device=DEV)[:, None] >> (torch.arange(D, device=DEV) % 16)[None]) & 1
    v = (2.0 * bit - 1.0)
    v[:, ::64], v[:, 63::64] = 1.0, -1.0
    v = (v[:, None, None] * torch.arange(1, Hkv + 1, device=DEV)[None, :, None, None]).expand(most, Hkv, 16, D).half()
    k4, v4 = (torch.zeros(pa.q4_pool_shape(most, Hkv, 16, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    rows = v.transpose(1, 2).reshape(-1, Hkv, D).contiguous()
    pa.cache_write_q4(rows, rows, k4, v4, torch.arange(most * 16, device=DEV))
    S = len(lens)
    tables = torch.arange(most, dtype=torch.int32, device=DEV).expand(S, -1).contiguous()
    out = pa.decode_attention_q4(torch.zeros(S, H, D, dtype=torch.float16, device=DEV), k4, v4, tables,
                                 torch.tensor(lens, dtype=torch.int32, device=DEV), max(lens), 0.1).double()
    s = float(torch.tensor(2.0 / 15).half())
    for i, n in enumerate(lens):
        tokens = torch.full((most,), 0.0, dtype=torch.float64, device=DEV)
        tokens[:-(-n // 16)] = 16
        tokens[-(-n // 16) - 1] = n - 16 * (-(-n // 16) - 1)
        # +1 is held as 15 s - 1
        up = tokens @ torch.cat([bit, bit], 1)[:, :D].double() / n
        up[::64], up[63::64] = 1.0, 0.0
        want = up * 15 * s - 1
        for h in range(H):
            x = h // (H // Hkv) + 1
            sx = float(torch.tensor(2.0 * x / 15).half())
            # 2^-16 s + 2^-19 (1 + 7.5 s) of q4tight, per channel
            tol = 2.0 ** -16 * sx + 2.0 ** -19 * 2 * x
            assert float((out[i, h] - (up * 15 * sx - x)).abs().max()) <= tol
        assert want.shape == (D,)
        assert n < 16 or 8 * (2.0 ** -16 * s + 2.0 ** -18) < 16 / n      # a chunk is well above that
