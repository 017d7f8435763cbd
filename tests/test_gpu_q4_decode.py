"""pa_decode_attention_q4 on the GPU against the definition in 64 bits over what the
cache's codes stand for (q4lib.attention states the tolerance's terms)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from q4lib import Q4Cache, attention, rounded, values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 129, 255, 256, 257, 300, 511, 513, 1025]


def _query(T, H, D, dtype, seed=0, factor=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed + 77)
    return (torch.randn(T, H, D, generator=g, device=DEV) * factor).to(dtype)


def _run(c, q, starts=None, max_query=1, out_dtype=torch.float32, scale=None, layer=0, **kw):
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    qsl = None if starts is None else torch.as_tensor(np.asarray(starts, np.int32), device=DEV)
    out = pa.decode_attention_q4(q, c.k4[layer], c.v4[layer], c.tables, c.lens, kw.pop("max_len", c.max_len), scale,
                                 query_start_loc=qsl, max_query_len=max_query, out_dtype=out_dtype,
                                 error_word=err, **kw)
    torch.cuda.synchronize()
    return out, int(err.item())


def _check(c, q, starts=None, max_query=1, out_dtype=torch.float32, scale=None, **kw):
    out, err = _run(c, q, starts, max_query, out_dtype, scale, **kw)
    assert err == 0
    s = q.shape[-1] ** -0.5 if scale is None else scale
    want, tol = attention(c, q, list(range(len(c.lens_host) + 1)) if starts is None else starts, s)
    d = (out.double() - want).abs()
    tol = rounded(tol, want, out.dtype)
    assert bool((d <= tol).all()), (float(d.max()), float((d / tol.clamp(min=1e-300)).max()))
    return out


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,B", [
    (1, 1, 64, 16), (8, 8, 64, 16), (4, 2, 128, 16), (12, 2, 128, 32), (5, 5, 128, 64), (8, 1, 64, 16), (16, 2, 128, 16),
    (32, 2, 64, 256), (10, 2, 256, 16), (3, 3, 256, 128), (7, 1, 256, 16), (36, 2, 128, 16)])
def test_edge_lengths(H, Hkv, D, B, dtype):
    c = Q4Cache(EDGES, Hkv, D, DT[dtype], B, seed=H)
    _check(c, _query(len(EDGES), H, D, DT[dtype]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D", [(8, 8, 64), (12, 2, 128), (40, 40, 128), (16, 2, 64), (6, 2, 256)])
def test_short_contexts_are_not_cut(H, Hkv, D, dtype):
    lens = [n for n in EDGES if n <= 256] * 3
    c = Q4Cache(lens, Hkv, D, DT[dtype], seed=D)
    a = _check(c, _query(len(lens), H, D, DT[dtype]), out_dtype=DT[dtype])
    # the same lengths under a larger bound go the other way
    b, _ = _run(c, _query(len(lens), H, D, DT[dtype]), out_dtype=torch.float32, max_len=16 * c.tables.shape[1])
    assert torch.allclose(a.float(), b, atol=2e-2, rtol=2e-2)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,most", [(8, 8, 64, 2), (32, 8, 128, 5), (12, 2, 128, 16), (4, 4, 128, 4), (8, 8, 128, 16),
                                          (6, 2, 256, 3), (16, 1, 64, 7), (40, 40, 128, 3)])
def test_several_query_tokens(H, Hkv, D, most, dtype):
    """Ragged drafts, some sequences without any, one as long as its context; each token sees
    those up to its own."""
    lens = [most, 40, 16 + most, 300, 0, 257, 700, most + 1, 33, 1000]
    r = np.random.default_rng(most)
    new = [most, 1, min(most, 3), most, 0, 0, int(r.integers(1, most + 1)), most, most, 1]
    starts = np.concatenate([[0], np.cumsum(new)])
    c = Q4Cache(lens, Hkv, D, DT[dtype], seed=most)
    _check(c, _query(int(starts[-1]), H, D, DT[dtype], seed=most), starts, most)
    short = [min(n, 250) for n in lens]
    c = Q4Cache(short, Hkv, D, DT[dtype], seed=most + 1)
    _check(c, _query(int(starts[-1]), H, D, DT[dtype], seed=most), starts, most, out_dtype=DT[dtype])


@pytest.mark.parametrize("S,lo,hi,H,Hkv,D", [(700, 1, 90, 8, 8, 64), (1300, 0, 40, 4, 2, 128), (300, 1, 700, 2, 1, 128)])
def test_many_sequences(S, lo, hi, H, Hkv, D):
    lens = [int(n) for n in np.random.default_rng(S).integers(lo, hi + 1, S)]
    c = Q4Cache(lens, Hkv, D, torch.bfloat16, seed=S)
    _check(c, _query(S, H, D, torch.bfloat16))
    _check(c, _query(S, H, D, torch.bfloat16), max_len=16 * c.tables.shape[1] if hi <= 256 else c.max_len)


@pytest.mark.parametrize("L,H,Hkv,D,B", [(70001, 8, 1, 128, 64), (33333, 4, 2, 64, 16), (40000, 2, 2, 256, 256)])
def test_one_long_sequence(L, H, Hkv, D, B):
    """A sequence that every worker has a part of."""
    c = Q4Cache([L, 5], Hkv, D, torch.float16, B, seed=L)
    _check(c, _query(2, H, D, torch.float16))


def test_seeded_shapes():
    r = np.random.default_rng(11)
    for i in range(40):
        Hkv = int(r.integers(1, 6))
        H, D = Hkv * int(r.integers(1, 10)), int(r.choice([64, 128, 256]))
        dtype, B = DT[str(r.choice(["f16", "bf16"]))], int(r.choice([16, 32, 64, 128, 256]))
        S, most = int(r.integers(1, 12)), int(r.choice([1, 1, 2, 5, 16]))
        hi = int(r.choice([30, 256, 600, 3000]))
        lens = [int(n) for n in r.integers(0, hi + 1, S)]
        new = [min(int(r.integers(0, most + 1)), n) for n in lens]
        starts = np.concatenate([[0], np.cumsum(new)])
        if starts[-1] == 0:
            continue
        c = Q4Cache(lens, Hkv, D, dtype, B, seed=100 + i)
        _check(c, _query(int(starts[-1]), H, D, dtype, seed=i), starts, most, max_len=max(max(lens), 1))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 6, 12])
def test_uneven_scales_and_queries(rows, dtype):
    """Values and scales over several orders of magnitude, weights on one far token, rows of
    zeros, query elements far apart."""
    dt = DT[dtype]
    lens = [400, 90, 1200]
    c = Q4Cache(lens, 2, 128, dt, seed=5)
    g = torch.Generator(device=DEV).manual_seed(6)
    c.k[0] *= torch.exp2(torch.randint(-3, 2, c.k[0].shape[:3], generator=g, device=DEV)).to(dt)[..., None]
    c.v[0] *= torch.exp2(torch.randint(-10, 11, c.v[0].shape[:3], generator=g, device=DEV)).to(dt)[..., None]
    c.v[0][:, :, 3] = 0.0
    c.k[0][:, :, 5] = 0.5
    at = (c.slots // 16, slice(None), c.slots % 16)
    pa.cache_write_q4(c.k[0][at].contiguous(), c.v[0][at].contiguous(), c.k4[0], c.v4[0], c.slots)
    q = _query(3, 2 * rows, 128, dt, factor=3.0)
    q[0, 1] = 0.0
    q[1, :, ::7] *= 2.0 ** -12
    q[2, 0] *= 2.0 ** -10
    _check(c, q)
    _check(c, q, scale=2.0)
    _check(c, q, scale=-0.3)
    _check(c, q, scale=0.0)


def test_large_bf16_queries():
    c = Q4Cache([300, 20], 2, 64, torch.bfloat16, seed=8)
    q = _query(2, 4, 64, torch.bfloat16)
    want = _check(c, q)
    got, _ = _run(c, q * 2.0 ** 60, scale=64 ** -0.5 * 2.0 ** -60)
    assert torch.equal(got, want)
    got, _ = _run(c, q * 2.0 ** -60, scale=64 ** -0.5 * 2.0 ** 60)
    assert torch.equal(got, want)


def test_a_nan_reaches_only_who_sees_it():
    """A NaN in the last token's value: earlier query tokens of the draft do not see it.  In a
    key: every row that sees it is NaN.  In a query: its row alone."""
    lens, starts = [300, 50, 270], [0, 3, 6, 9]
    c = Q4Cache(lens, 2, 128, torch.float16, seed=9)
    q = _query(9, 8, 128, torch.float16)
    clean, _ = _run(c, q, starts, 3)
    last = c.slots[torch.tensor([299, 349, 619])]
    bad = c.v[0][last // 16, :, last % 16].clone()
    bad[:, 1, 70] = float("nan")
    keep = [t.clone() for t in (c.k4[0], c.v4[0])]
    pa.cache_write_q4(bad, bad, keep[0], c.v4[0], last)
    out, _ = _run(c, q, starts, 3)
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[2::3, 4:, 64:] = True                   # the group's channels, KV head 1
    assert torch.equal(nan, want) and torch.equal(out[~nan], clean[~nan])
    c.v4[0].copy_(_fresh_v(c))
    first = c.slots[:1] + 0
    bad = c.k[0][first // 16, :, first % 16].clone()
    bad[:, 0, 3] = float("inf")
    spare = c.v4[0].clone()
    pa.cache_write_q4(bad, bad, c.k4[0], spare, first)
    out, _ = _run(c, q, starts, 3)
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[:3, :4] = True
    assert torch.equal(nan, want) and torch.equal(out[~nan], clean[~nan])
    c = Q4Cache(lens, 2, 128, torch.float16, seed=9)
    q[4, 2, 9] = float("nan")
    out, _ = _run(c, q, starts, 3)
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[4, 2] = True
    assert torch.equal(nan, want) and torch.equal(out[~nan], clean[~nan])


def _fresh_v(c):
    return Q4Cache(c.lens_host, 2, 128, torch.float16, seed=9).v4[0]


def test_bad_lengths_and_blocks():
    lens = [100, 300, 40, 600, 33]
    c = Q4Cache(lens, 2, 128, torch.bfloat16, seed=12)
    q = _query(5, 4, 128, torch.bfloat16)
    want, _ = _run(c, q)
    good = c.lens.clone()
    c.lens[1], c.lens[2] = 601, -1
    out = torch.full_like(want, 9.0)
    got, err = _run(c, q, max_len=600, out=out)
    assert err == pa.ERRBIT_CONTEXT_LEN and not got[1:3].any()
    # (the others' contexts are cut elsewhere now: other sums, each within the bound)
    ref, tol = attention(c, q, range(6), 128 ** -0.5)
    assert bool(((got.double() - ref).abs() <= tol)[[0, 3, 4]].all())
    c.lens.copy_(good)
    # a block outside the pool: its tokens are left out of sequences 0 and 3
    c.tables[0, 2], c.tables[3, 10] = c.k4[0].shape[0], -7
    got, err = _run(c, q)
    assert err == pa.ERRBIT_BLOCK_OOB and torch.equal(got[[1, 2, 4]], want[[1, 2, 4]])
    for s, b in ((0, 2), (3, 10)):
        keep = [i for i in range(lens[s]) if i // 16 != b]
        d = Q4Cache([len(keep)], 2, 128, torch.bfloat16)
        idx = torch.tensor(keep, device=DEV)
        t = torch.as_tensor(c.tables_host[s].astype(np.int64), device=DEV)
        for mine, theirs in ((d.k, c.k), (d.v, c.v)):
            rows = theirs[0][t[idx // 16], :, idx % 16]
            mine[0][d.slots // 16, :, d.slots % 16] = rows
        ref, tol = attention(d, q[s:s + 1], [0, 1], 128 ** -0.5)
        assert bool(((got[s:s + 1].double() - ref).abs() <= tol).all())
    # every block of a sequence outside: nothing to see
    c.tables[4] = -1
    got, err = _run(c, q)
    assert err == pa.ERRBIT_BLOCK_OOB and not got[4].any()


def test_lengths_shorter_than_the_draft_and_bad_starts():
    lens = [100, 3, 300, 50]
    c = Q4Cache(lens, 2, 64, torch.float16, seed=13)
    q = _query(12, 4, 64, torch.float16)
    got, err = _run(c, q, [0, 2, 7, 10, 12], 5)           # five tokens on a context of three
    assert err == pa.ERRBIT_CONTEXT_LEN and not got[2:7].any() and got[7:].any(-1).all() and got[:2].any(-1).all()
    got, err = _run(c, q, [0, 2, 4, 10, 12], 5)           # six where five are announced
    assert err == pa.ERRBIT_CONTEXT_LEN and not got[4:10].any() and got[10:].any(-1).all()
    got, err = _run(c, q, [0, 2, 4, 7, 40], 5)            # past the rows there are
    assert err == pa.ERRBIT_CONTEXT_LEN and not got[7:].any() and got[4:7].any(-1).all()
    got, err = _run(c, q, [0, 2, 4, 7, -9], 5)
    assert err == pa.ERRBIT_CONTEXT_LEN and got[4:7].any(-1).all()


def test_no_sequences_no_tokens():
    c = Q4Cache([5, 9], 2, 64, torch.float16)
    assert pa.decode_attention_q4(_query(0, 4, 64, torch.float16), c.k4[0], c.v4[0], c.tables[:0], c.lens[:0], 16,
                                  0.1).shape == (0, 4, 64)
    out, err = _run(c, _query(0, 4, 64, torch.float16), [0, 0, 0], 3)
    assert out.shape == (0, 4, 64) and err == 0


def test_results_do_not_depend_on_block_size_or_run():
    outs = []
    for B in (16, 64, 256):
        c = Q4Cache([777, 2000, 130], 2, 128, torch.bfloat16, 16, seed=14)
        d = Q4Cache([777, 2000, 130], 2, 128, torch.bfloat16, B, seed=15)
        at = (c.slots // 16, slice(None), c.slots % 16)
        pa.cache_write_q4(c.k[0][at].contiguous(), c.v[0][at].contiguous(), d.k4[0], d.v4[0], d.slots)
        for _ in range(3):
            outs.append(_run(d, _query(3, 12, 128, torch.bfloat16))[0])
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_calls_of_other_sizes_share_a_workspace():
    a = Q4Cache([3000, 100, 1700], 2, 128, torch.float16, seed=16)
    b = Q4Cache([900] * 7, 4, 64, torch.bfloat16, seed=17)
    qa, qb = _query(3, 12, 128, torch.float16), _query(7, 4, 64, torch.bfloat16)
    wa, wb = _run(a, qa)[0], _run(b, qb)[0]
    n = max(pa.decode_q4_workspace_size(3, 12, 2, 128, 1, 3000), pa.decode_q4_workspace_size(7, 4, 4, 64, 1, 900),
            pa.decode_workspace_size(3, 12, 2, 128, 3000))
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    got = []
    for _ in range(10):
        got.append((wa, pa.decode_attention_q4(qa, a.k4[0], a.v4[0], a.tables, a.lens, 3000, 128 ** -0.5, workspace=ws)))
        # (a 16-bit call of the library between them)
        pa.decode_attention(qa, a.k[0], a.v[0], a.tables, a.lens, 3000, 128 ** -0.5, workspace=ws)
        got.append((wb, pa.decode_attention_q4(qb, b.k4[0], b.v4[0], b.tables, b.lens, 900, 64 ** -0.5, workspace=ws)))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in got)


def test_pools_past_four_gigabytes():
    Hkv, D, B, L = 8, 256, 256, 700
    nb = (1 << 32) // (Hkv * B * 144) + 40
    c = Q4Cache([L], Hkv, D, torch.bfloat16, B, seed=18)
    k4, v4 = (torch.full(pa.q4_pool_shape(nb, Hkv, B, D), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    n = c.tables.shape[1]
    far = torch.arange(nb - n, nb, dtype=torch.int32, device=DEV)[None]
    k4[far[0].long()], v4[far[0].long()] = c.k4[0][c.tables[0].long()], c.v4[0][c.tables[0].long()]
    q = _query(1, 16, D, torch.bfloat16)
    want, _ = _run(c, q)
    got = pa.decode_attention_q4(q, k4, v4, far, c.lens, L, D ** -0.5)
    assert torch.equal(got, want)


@pytest.mark.parametrize("H", [2, 12, 24])
@pytest.mark.parametrize("scale", [1e30, -1e32, 3e34])
def test_logits_of_any_size(H, scale):
    """All weight on the largest logit, however far from zero the logits are: the output is that
    token's value, s n + z in fp32."""
    c = Q4Cache([300, 40], 2, 128, torch.bfloat16, seed=30)
    q = _query(2, H, 128, torch.bfloat16)
    out, err = _run(c, q, scale=scale)
    assert err == 0
    checked = 0
    for s in range(2):
        for h in range(H):
            k, v = values(c.rows(c.k[0], s, h // (H // 2)))[0], values(c.rows(c.v[0], s, h // (H // 2)))
            x = (q[s, h].double() @ k.T) * (1 if scale > 0 else -1)
            top = x.topk(2)
            if top.values[0] - top.values[1] < 1e-2:    # (fp32's rounding of a logit is far less)
                continue
            j = top.indices[0]
            # two parts of the weight, 2^-22, and a few roundings in 32 bits
            assert bool(((out[s, h].double() - v[0][j]).abs() <= 2.0 ** -20 * v[1][j]).all())
            checked += 1
    assert checked >= H
