"""pa_prefill_attention_lse and pa_prefill_scores on the GPU against the
definition in 64 bits.

Tolerances.  lse: the largest score error of the row, 2^-21 from exponentials
and sums, n 2^-24 from the sum of n terms, and one rounding of the result.
Scores: a weight exp(x - lse) is off by the error of x (cachelib.logits64) and
two roundings of lse log2 e (2^-23 |lse|) relative to itself, plus 2^-21 from
the exponential; a sum of N weights adds N 2^-24, at most 2^-12."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from cachelib import DT, Cache, logits64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _batch(c, new, H, D, seed=3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.randn(int(starts[-1]), H, D, generator=g, device=DEV).to(c.dtype)
    return q, torch.as_tensor(starts, device=DEV), starts


def _attend(c, q, qsl, new, scale, max_len=None, err=None):
    T, H, _ = q.shape
    lse = torch.full((T, H), 7.0, device=DEV)
    out = pa.prefill_attention(q, c.k[0], c.v[0], c.tables, qsl, c.lens, max(max(new), 1), max_len or c.max_len,
                               scale, lse=lse, error_word=err)
    return out, lse


def _want(c, q, starts, new, lse, scale, s, h, G, block_ok=None):
    """Scores of (s, h) and their tolerance."""
    n, m = c.lens_host[s], new[s]
    k = c.rows(c.k[0], s, h)
    k = torch.nan_to_num(k) if block_ok is not None else k
    want = torch.zeros(n, dtype=torch.float64, device=DEV)
    tol = torch.zeros_like(want)
    hide = torch.ones(m, n, dtype=torch.bool, device=DEV).triu(n - m + 1)
    if block_ok is not None:
        hide |= ~block_ok[s][None]
    for qh in range(h * G, (h + 1) * G):
        rows = slice(int(starts[s]), int(starts[s]) + m)
        x, e = logits64(q[rows, qh], k, scale)
        e = e.masked_fill(hide, 0.0)
        ls = lse[rows, qh].double()[:, None]
        p = torch.exp(x.masked_fill(hide, -math.inf) - ls)
        p = torch.where(ls == -math.inf, torch.zeros_like(p), p)
        rel = e + 2.0 ** -23 * ls.abs().nan_to_num(posinf=0) + 2.0 ** -21
        want += p.sum(0)
        tol += (p * rel).sum(0)
    return want, tol + want * min(m * G * 2.0 ** -24, 2.0 ** -12)


def _check_scores(c, q, starts, qsl, new, lse, scale, stride=None, max_len=None, block_ok=None, expect_err=0):
    Hkv, H = c.k[0].shape[1], q.shape[1]
    G, max_len = H // Hkv, max_len or c.max_len
    S, stride = len(c.lens_host), stride or max_len
    base = torch.rand(S, Hkv, stride, device=DEV)
    scores = base.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, max(max(new), 1), max_len, scale, scores,
                            error_word=err)
    assert got is scores
    torch.cuda.synchronize()
    assert int(err.item()) == expect_err
    for s in range(S):
        for h in range(Hkv):
            n = c.lens_host[s]
            w, tol = _want(c, q, starts, new, lse, scale, s, h, G, block_ok)
            d = (scores[s, h, :n].double() - base[s, h, :n].double() - w).abs()
            lim = tol + 2 * 2.0 ** -24 * (w + 1) + 1e-30
            assert bool((d <= lim).all()), (s, h, float((d - lim).max()), float(d.max()))
            assert torch.equal(scores[s, h, n:], base[s, h, n:])
    return scores


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,B", [(1, 1, 64, 16), (4, 2, 128, 8), (12, 2, 128, 16), (5, 1, 64, 32),
                                       (8, 8, 128, 64), (16, 1, 64, 128), (3, 1, 128, 256), (24, 2, 64, 16)])
def test_prompts_chunks_and_windows(H, Hkv, D, B, dtype):
    lens = [1, 17, 130, 300, 257, 600, 128, 40]
    new = [1, 17, 130, 33, 1, 200, 127, 0]
    c = Cache(lens, Hkv, D, DT[dtype], B, seed=H)
    q, qsl, starts = _batch(c, new, H, D)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = _attend(c, q, qsl, new, D ** -0.5, err=err)
    assert int(err.item()) == 0
    plain = pa.prefill_attention(q, c.k[0], c.v[0], c.tables, qsl, c.lens, 200, 600, D ** -0.5)
    assert torch.equal(out, plain)  # the same kernel, one more output
    for s, (n, m) in enumerate(zip(lens, new)):
        hide = torch.ones(m, n, dtype=torch.bool, device=DEV).triu(n - m + 1)
        for qh in range(H):
            rows = slice(int(starts[s]), int(starts[s]) + m)
            x, e = logits64(q[rows, qh], c.rows(c.k[0], s, qh // (H // Hkv)), D ** -0.5)
            want = torch.logsumexp(x.masked_fill(hide, -math.inf), -1)
            lim = e.masked_fill(hide, 0).amax(-1) + 2.0 ** -20 + n * 2.0 ** -24 + 2.0 ** -22 * want.abs() if n else 0
            assert bool(((lse[rows, qh].double() - want).abs() <= lim).all())
    _check_scores(c, q, starts, qsl, new, lse, D ** -0.5)


@pytest.mark.parametrize("H,Hkv,D,new,lens", [
    (32, 8, 128, [1024], [1024]), (6, 2, 128, [700, 3], [2000, 4097]), (2, 2, 64, [2049], [2049]),
    (4, 1, 128, [32], [9000]), (8, 1, 64, [1] * 9, [1, 255, 256, 257, 511, 512, 513, 128, 129]),
    (2, 1, 128, [65], [65])])
def test_longer_ones(H, Hkv, D, new, lens):
    c = Cache(lens, Hkv, D, torch.bfloat16, 16, seed=5)
    q, qsl, starts = _batch(c, new, H, D)
    _, lse = _attend(c, q, qsl, new, D ** -0.5)
    _check_scores(c, q, starts, qsl, new, lse, D ** -0.5, stride=c.max_len + 5)


@pytest.mark.parametrize("S", [100, 512, 513])
def test_many_ragged_sequences(S):
    """Past 512 sequences the items are numbered without the table."""
    rng = np.random.default_rng(S)
    lens = rng.integers(1, 700, S)
    lens[S // 2] = 1500
    new = [int(rng.integers(0, min(n, 40) + 1)) for n in lens]
    c = Cache(lens, 1, 64, torch.float16, 32, seed=S)
    q, qsl, starts = _batch(c, new, 2, 64)
    _, lse = _attend(c, q, qsl, new, 0.125)
    _check_scores(c, q, starts, qsl, new, lse, 0.125)


def test_split_items_give_the_lse_too():
    """One long prompt on few heads: its heaviest items are split and merged."""
    c = Cache([6000], 1, 64, torch.float16, 16, seed=5)
    q, qsl, starts = _batch(c, [6000], 2, 64)
    _, lse = _attend(c, q, qsl, [6000], 0.125)
    x, e = logits64(q[:, 1], c.rows(c.k[0], 0, 0), 0.125)
    x.masked_fill_(torch.ones(6000, 6000, dtype=torch.bool, device=DEV).triu(1), -math.inf)
    want = torch.logsumexp(x, -1)
    lim = e.amax(-1) + 2.0 ** -20 + 6000 * 2.0 ** -24 + 2.0 ** -22 * want.abs()
    assert bool(((lse[:, 1].double() - want).abs() <= lim).all())
    _check_scores(c, q, starts, qsl, [6000], lse, 0.125)


def test_chunks_add_up_to_the_whole_prompt():
    H, Hkv, D, n = 4, 2, 64, 500
    c = Cache([n], Hkv, D, torch.float16, 16, seed=6)
    q, qsl, _ = _batch(c, [n], H, D)
    _, lse = _attend(c, q, qsl, [n], 0.1)
    whole = pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, n, n, 0.1, torch.zeros(1, Hkv, n, device=DEV))
    parts = torch.zeros_like(whole)
    for a, b in ((0, 64), (64, 65), (65, 333), (333, 500)):
        pa.prefill_scores(q[a:b], lse[a:b], c.k[0], c.tables, torch.tensor([0, b - a], dtype=torch.int32, device=DEV),
                          torch.tensor([b], dtype=torch.int32, device=DEV), b - a, n, 0.1, parts)
    assert torch.allclose(whole, parts, rtol=1e-5, atol=1e-6)
    # every row's weights sum to one
    assert abs(float(whole.double().sum()) - n * H) < 1e-4 * n * H


def test_decode_rows_agree_with_the_scored_decode():
    lens = [300, 1, 77, 512]
    c = Cache(lens, 2, 128, torch.bfloat16, 16, seed=7)
    q, qsl, starts = _batch(c, [1] * 4, 12, 128)
    _, lse = _attend(c, q, qsl, [1] * 4, 0.09)
    a = pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 1, 512, 0.09, torch.zeros(4, 2, 512, device=DEV))
    b = torch.zeros_like(a)
    pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 512, 0.09, b)
    assert torch.allclose(a, b, rtol=1e-4, atol=1e-8)


@pytest.mark.parametrize("B", [8, 16, 64])
def test_bad_lengths_and_skipped_blocks(B):
    lens, new = [300, 140, 100, 70], [40, 140, 5, 70]
    c = Cache(lens, 2, 64, torch.float16, B, seed=8)
    q, qsl, starts = _batch(c, new, 4, 64)
    ok = [torch.ones(n, dtype=torch.bool, device=DEV) for n in lens]
    for s, i, bad in ((0, 1, -1), (1, 0, 10 ** 7)):
        c.tables[s, i] = bad
        ok[s][i * B:(i + 1) * B] = False
    c.tables[3] = -1  # nothing to read: every row's lse is -inf
    ok[3][:] = False
    _, lse = _attend(c, q, qsl, new, 0.125)
    assert bool((lse[int(starts[3]):] == -math.inf).all())
    # the first rows of sequence 1 see only the skipped block
    assert bool((lse[int(starts[1]):int(starts[1]) + B] == -math.inf).all())
    _check_scores(c, q, starts, qsl, new, lse, 0.125, block_ok=ok, expect_err=pa.ERRBIT_BLOCK_OOB)
    c.lens[2] = 4  # fewer tokens than rows
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sc = torch.full((4, 2, 300), 0.5, device=DEV)
    pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 140, 300, 0.125, sc, error_word=err)
    assert int(err.item()) & pa.ERRBIT_CONTEXT_LEN and bool((sc[2] == 0.5).all())
    _, lse = _attend(c, q, qsl, new, 0.125)
    assert bool((lse[int(starts[2]):int(starts[3])] == -math.inf).all())


def test_infinite_and_nan_rows_stay_where_they_belong():
    c = Cache([200, 150], 1, 64, torch.bfloat16, 16, seed=9)
    new = [30, 150]
    q, qsl, starts = _batch(c, new, 2, 64)
    _, lse = _attend(c, q, qsl, new, 0.125)
    clean = pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 150, 200, 0.125, torch.zeros(2, 1, 200, device=DEV))
    q2, lse2 = q.clone(), lse.clone()
    q2[int(starts[1]) + 100] = math.nan  # row 100 of the second sequence sees keys 0..100
    got = pa.prefill_scores(q2, lse2, c.k[0], c.tables, qsl, c.lens, 150, 200, 0.125, torch.zeros(2, 1, 200, device=DEV))
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1, 0, 101:], clean[1, 0, 101:])
    assert bool(torch.isnan(got[1, 0, :101]).all())
    lse2 = lse.clone()
    lse2[5] = -math.inf  # a row that saw nothing
    q2 = q.clone()
    q2[5] = math.inf
    got = pa.prefill_scores(q2, lse2, c.k[0], c.tables, qsl, c.lens, 150, 200, 0.125, torch.zeros(2, 1, 200, device=DEV))
    assert bool(torch.isfinite(got).all()) and torch.equal(got[1], clean[1])


def test_repeatable_captured_and_replayed():
    c = Cache([700, 300], 2, 128, torch.bfloat16, 16, seed=10)
    new = [400, 64]
    q, qsl, _ = _batch(c, new, 12, 128)
    _, lse = _attend(c, q, qsl, new, 0.1)
    want = pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 400, 700, 0.1, torch.zeros(2, 2, 700, device=DEV))
    ws = torch.empty(max(256, pa.prefill_scores_workspace_size(2, 12, 2, 128, 400, 700)), dtype=torch.uint8, device=DEV)
    aws = torch.empty(pa.prefill_workspace_size(2, 12, 2, 128, 400), dtype=torch.uint8, device=DEV)
    sc, out, l2 = torch.zeros_like(want), torch.empty_like(q), torch.empty_like(lse)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pa.prefill_attention(q, c.k[0], c.v[0], c.tables, qsl, c.lens, 400, 700, 0.1, out=out, workspace=aws, lse=l2)
        pa.prefill_scores(q, l2, c.k[0], c.tables, qsl, c.lens, 400, 700, 0.1, sc, workspace=ws)
    ws.fill_(255)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(l2, lse) and torch.equal(sc, want + want)


@pytest.mark.parametrize("H,Hkv,D,new,lens", [
    (8, 1, 128, [1024], [1024]), (1, 1, 64, [2000], [2001]), (6, 2, 64, [700, 3, 64], [700, 2000, 300]),
    (32, 8, 128, [500], [1024]), (4, 4, 128, [257, 0, 1, 640], [257, 100, 700, 641]), (24, 8, 64, [300], [333]),
    (8, 8, 64, [4000], [4100]), (4, 4, 64, [3000, 200], [4096, 1500]), (16, 2, 128, [1500], [1500])])
def test_few_items_shared_by_several_blocks_of_threads(H, Hkv, D, new, lens):
    """Few items of many queries: clusters share them, some with parts that are
    empty, and the sums do not depend on timing."""
    c = Cache(lens, Hkv, D, torch.bfloat16, 16, seed=D + H)
    q, qsl, starts = _batch(c, new, H, D)
    _, lse = _attend(c, q, qsl, new, D ** -0.5)
    _check_scores(c, q, starts, qsl, new, lse, D ** -0.5, stride=c.max_len + 5)
    runs = [pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, max(new), c.max_len, D ** -0.5,
                              torch.zeros(len(lens), Hkv, c.max_len, device=DEV)) for _ in range(3)]
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_shared_items_with_bad_lengths_and_blocks():
    lens, new = [900, 500, 700], [900, 400, 600]
    c = Cache(lens, 1, 64, torch.float16, 16, seed=9)
    q, qsl, starts = _batch(c, new, 4, 64)
    _, lse = _attend(c, q, qsl, new, 0.125)
    tables = c.tables.clone()
    tables[2, 3] = -1  # tokens 48 .. 63 of the last sequence
    lens_bad = c.lens.clone()
    lens_bad[1] = 399  # fewer than its new tokens
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    good = pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 900, 900, 0.125, torch.zeros(3, 1, 900, device=DEV))
    got = pa.prefill_scores(q, lse, c.k[0], tables, qsl, lens_bad, 900, 900, 0.125, torch.zeros(3, 1, 900, device=DEV),
                            error_word=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.ERRBIT_CONTEXT_LEN | pa.ERRBIT_BLOCK_OOB
    assert torch.equal(got[0], good[0]) and not got[1].any()
    assert not got[2, 0, 48:64].any()
    assert torch.equal(got[2, 0, :48], good[2, 0, :48]) and torch.equal(got[2, 0, 64:], good[2, 0, 64:])


@pytest.mark.parametrize("S", [40, 600])
def test_many_items_for_each_block_of_threads(S):
    """More items than a CTA lists ahead (with and without the numbering table)."""
    lens, new = [9000] + [700] * (S - 1), [3] + [2] * (S - 1)
    if S == 40:  # 40 sequences of up to 9000 tokens, 64 heads: more than 200 items a CTA
        lens = [9000 - 64 * s for s in range(S)]
    c = Cache(lens, 64, 64, torch.float16, 64, seed=S)
    q, qsl, starts = _batch(c, new, 64, 64)
    _, lse = _attend(c, q, qsl, new, 0.125)
    scores = pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 3, c.max_len, 0.125,
                               torch.zeros(S, 64, c.max_len, device=DEV))
    for s in {0, 1, S // 2, S - 1}:
        for h in (0, 17, 63):
            w, tol = _want(c, q, starts, new, lse, 0.125, s, h, 1)
            d = (scores[s, h, :lens[s]].double() - w).abs()
            assert bool((d <= tol + 2 * 2.0 ** -24 * (w + 1) + 1e-30).all()), (s, h, float(d.max()))
    assert not scores[1, :, lens[1]:].any()
    per_row = scores.sum((1, 2), dtype=torch.float64).cpu()
    want = torch.tensor(new, dtype=torch.float64) * 64  # every row's weights sum to one
    assert float((per_row - want).abs().max()) < 1e-3


def _mixed():
    lens = [2500] + [40 + 97 * (i % 11) for i in range(40)]
    return [500] + [min(n, 1 + 13 * (i % 9)) for i, n in enumerate(lens[1:])], lens


@pytest.mark.parametrize("B", [8, 16, 128])
@pytest.mark.parametrize("H,Hkv,D,new,lens", [
    (32, 8, 128, [17] * 8, [1500 + 211 * i for i in range(8)]), (32, 8, 128, [32] * 8, [3000 + 130 * i for i in range(8)]),
    (32, 8, 128, [64] * 8, [2900 - 129 * i for i in range(8)]), (32, 8, 128, [96] * 6, [2900 - 129 * i for i in range(6)]),
    (16, 2, 128, [16] * 24, [900 + 257 * i for i in range(24)]), (8, 8, 128, [128] * 8, [2000 + 129 * i for i in range(8)]),
    (32, 8, 64, [32] * 8, [3000 + 130 * i for i in range(8)]), (12, 2, 128, [32] * 16, [3000 + 300 * i for i in range(16)]),
    (32, 8, 128, *_mixed()), (12, 2, 64, *_mixed())])
def test_many_items_of_few_query_tiles(H, Hkv, D, new, lens, B):
    """Several items a CTA with one to a few query tiles each: the two key tiles of an item,
    and the items after it, share rings of a few slots, whose copies land in any order (part
    of the keys in L2, part not)."""
    c = Cache(lens, Hkv, D, torch.bfloat16, B, seed=B + H)
    q, qsl, starts = _batch(c, new, H, D)
    _, lse = _attend(c, q, qsl, new, D ** -0.5)
    _check_scores(c, q, starts, qsl, new, lse, D ** -0.5)
    want, flush = None, torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    for i in range(12):
        if i % 3 == 0:
            flush.fill_(i)
        if i % 3 == 1:
            torch.nan_to_num(c.k[0][::2]).sum()  # every other block into L2
        got = pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, max(new), c.max_len, D ** -0.5,
                                torch.zeros(len(lens), Hkv, c.max_len, device=DEV))
        want = got if want is None else want
        assert torch.equal(got, want)
