"""pa_evict_tokens on the GPU against the definition (numpy): everything it
moves is compared bit by bit, and so is everything it must leave alone."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from cachelib import DT, Cache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _kept(sc, L, keep, sink, recent):
    n = min(L, keep)
    r = min(recent, n)
    a = min(sink, n - r)
    if n == L:
        return np.arange(L)
    mid = np.arange(a, L - r)
    x = sc[mid].astype(np.float64)
    rank = np.where(np.isnan(x), 1, 0)  # NaN after everything
    order = np.lexsort((mid, -np.where(np.isnan(x), 0.0, x), rank))
    return np.sort(np.concatenate([np.arange(a), mid[order[:n - r - a]], np.arange(L - r, L)])).astype(np.int64)


def _bits(t):
    return t.view(torch.int16).clone()


def _check(c, scores, keep, sink, recent, out_of_place=False, split_scores=False, max_len=None,
           max_keep=None, want_err=0, skip=(), kw=None):
    layers, S, Hkv, stride = scores.shape
    B = c.block
    keep = list(keep)
    max_len = max_len or max(c.max_len, 1)
    n_host = [min(L, k) for L, k in zip(c.lens_host, keep)]
    max_keep = max(n_host) if max_keep is None else max_keep
    k0, v0 = [_bits(x) for x in c.k], [_bits(x) for x in c.v]
    s0 = scores.cpu().numpy().copy()
    dst = dst_host = None
    if out_of_place:
        nb = [-(-n // B) for n in n_host]
        assert sum(nb) <= len(c.spare)
        dst_host = np.full((S, max(max(nb), 1) + 1), -1, np.int32)
        pos = 0
        for s, m in enumerate(nb):
            dst_host[s, :m] = c.spare[pos:pos + m]
            pos += m
        dst = torch.as_tensor(dst_host, device=DEV)
    out = torch.full((layers, S, Hkv, stride + 3), 9.0, device=DEV) if split_scores else None
    kept = torch.full((layers, S, Hkv, max_keep + 1), -5, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    new = pa.evict_tokens(c.k, c.v, list(scores), c.tables, c.lens, torch.tensor(keep, dtype=torch.int32, device=DEV),
                          max_len, max_keep, num_sink=sink, num_recent=recent, dst_block_tables=dst,
                          scores_out=None if out is None else list(out), kept=list(kept), error_word=err, **(kw or {}))
    torch.cuda.synchronize()
    assert int(err.item()) == want_err
    want_k, want_v = [x.clone() for x in k0], [x.clone() for x in v0]
    want_sc = s0.copy() if out is None else np.full(out.shape, 9.0, np.float32)
    want_kept = np.full(kept.shape, -5, np.int32)
    for s, L in enumerate(c.lens_host):
        if s in skip:
            assert int(new[s]) == int(c.lens[s])
            continue
        n = n_host[s]
        assert int(new[s]) == n
        to = np.arange(n)
        table = dst_host if out_of_place else c.tables_host
        for l in range(layers):
            for h in range(Hkv):
                idx = _kept(s0[l, s, h], L, keep[s], sink, recent)
                assert len(idx) == n
                want_kept[l, s, h, :n] = idx
                want_sc[l, s, h, :L] = 0
                want_sc[l, s, h, :n] = s0[l, s, h, idx]
                src = [torch.as_tensor(x, device=DEV) for x in (c.tables_host[s, idx // B].astype(np.int64), idx % B)]
                d = [torch.as_tensor(x, device=DEV) for x in (table[s, to // B].astype(np.int64), to % B)]
                want_k[l][d[0], h, d[1]] = k0[l][src[0], h, src[1]]
                want_v[l][d[0], h, d[1]] = v0[l][src[0], h, src[1]]
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    got_sc = (scores if out is None else out).cpu().numpy()
    assert np.array_equal(got_sc, want_sc, equal_nan=True)
    if out is not None:
        assert np.array_equal(scores.cpu().numpy(), s0, equal_nan=True)
    for l in range(layers):
        assert torch.equal(_bits(c.k[l]), want_k[l]) and torch.equal(_bits(c.v[l]), want_v[l])
    return new


def _scores(layers, S, Hkv, stride, seed=0, levels=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.rand(layers, S, Hkv, stride, generator=g, device=DEV)
    return x if levels is None else (x * levels).floor() / levels


@pytest.mark.parametrize("out_of_place", [False, True])
@pytest.mark.parametrize("Hkv,D,dtype,B,layers", [(1, 64, "f16", 16, 1), (2, 128, "bf16", 8, 3), (3, 256, "f16", 32, 2),
                                                  (5, 64, "bf16", 256, 1), (2, 128, "f16", 64, 2)])
def test_lengths_and_budgets(Hkv, D, dtype, B, layers, out_of_place):
    lens = [0, 1, 1, 15, 16, 17, 100, 300, 257, 64, 512, 40]
    keep = [0, 0, 1, 15, 9, 16, 1, 299, 128, 1000, 33, 20]
    c = Cache(lens, Hkv, D, DT[dtype], B, seed=D, spare=80 if B == 8 else 60, layers=layers)
    _check(c, _scores(layers, len(lens), Hkv, 512), keep, 4, 8, out_of_place, split_scores=out_of_place)


@pytest.mark.parametrize("sink,recent", [(0, 0), (1000, 0), (0, 1000), (7, 9), (30, 30), (50, 50), (40, 21)])
def test_first_and_last_tokens(sink, recent):
    c = Cache([200, 61, 60, 5], 2, 64, torch.float16, 16, seed=1)
    _check(c, _scores(1, 4, 2, 203, seed=2), [60] * 4, sink, recent)


@pytest.mark.parametrize("levels", [1, 2, 7])
def test_equal_scores_go_to_the_lowest_index(levels):
    c = Cache([5000, 777, 4096, 4097], 2, 64, torch.bfloat16, 16, seed=3)
    _check(c, _scores(1, 4, 2, 5000, seed=4, levels=levels), [1234, 500, 4095, 1], 3, 17)


def test_odd_scores():
    """NaN, infinities, negative scores, both zeros and denormals."""
    c = Cache([400, 400, 400], 2, 64, torch.float16, 16, seed=5)
    sc = torch.randn(1, 3, 2, 400, generator=torch.Generator(device=DEV).manual_seed(6), device=DEV)
    sc[0, 0, :, ::3] = float("nan")
    sc[0, 1, :, ::2] = -float("inf")
    sc[0, 1, :, 5::50] = float("inf")
    sc[0, 2, 0, ::2] = 0.0
    sc[0, 2, 0, 1::2] = -0.0
    sc[0, 2, 1] = 1e-40 * torch.arange(400, device=DEV)
    sc[0, 2, 1, 7] = -1e-40
    _check(c, sc, [300, 150, 133], 2, 5)
    c = Cache([400, 400], 1, 64, torch.float16, 16, seed=5)
    _check(c, torch.full((1, 2, 1, 400), float("nan"), device=DEV), [100, 399], 0, 0)


@pytest.mark.parametrize("out_of_place", [False, True])
def test_long_sequences(out_of_place):
    lens = [70001, 8192, 12289]
    c = Cache(lens, 1, 64, torch.float16, 16, seed=7, spare=5000)
    _check(c, _scores(1, 3, 1, 70001, seed=8), [40000, 8191, 200], 16, 128, out_of_place)
    c = Cache(lens, 1, 64, torch.float16, 64, seed=7, spare=2000)
    _check(c, _scores(1, 3, 1, 70001, seed=9, levels=100), [69999, 5, 12288], 0, 0, out_of_place)


@pytest.mark.parametrize("L,n,levels", [(393216, 200000, None), (196609, 1, 3), (100000, 99999, 1), (9000, 4000, 50)])
def test_long_sequences_split_over_a_cluster(L, n, levels):
    c = Cache([L, 7], 1, 64, torch.float16, 256, seed=17)
    _check(c, _scores(1, 2, 1, L, seed=18, levels=levels), [n, 5], 100, 300)


@pytest.mark.parametrize("n", [3000, 4095])
def test_in_place_moves_by_one_and_by_many(n):
    """One early token leaves (every later row moves by one), or a quarter does."""
    c = Cache([4096] * 3, 2, 128, torch.bfloat16, 16, seed=19)
    sc = _scores(1, 3, 2, 4096, seed=20)
    sc[..., 5] = -1.0
    _check(c, sc, [n] * 3, 0, 0)


def test_many_layers_and_sequences():
    lens = list(np.random.default_rng(9).integers(0, 200, 30))
    c = Cache(lens, 4, 64, torch.bfloat16, 16, seed=9, layers=5)
    _check(c, _scores(5, 30, 4, 256, seed=10), [64] * 30, 4, 16)


def test_nothing_to_evict_leaves_everything():
    c = Cache([10, 200], 2, 64, torch.float16, 16, seed=11)
    _check(c, _scores(1, 2, 2, 200), [10, 1 << 30], 4, 4)


def test_bad_lengths_and_blocks():
    c = Cache([100, 100, 100, 100, 100], 2, 64, torch.float16, 16, seed=12)
    c.lens = torch.tensor([-1, 201, 100, 100, 100], dtype=torch.int32, device=DEV)
    # tables wide enough for the bound of 200 tokens
    c.tables = torch.nn.functional.pad(c.tables, (0, 6), value=-1)
    # a negative length, one past the bound, a negative budget, a budget past its bound
    _check(c, _scores(1, 5, 2, 200), [50, 50, -1, 61, 60], 2, 2, max_len=200, max_keep=60,
           want_err=pa.ERRBIT_CONTEXT_LEN, skip=(0, 1, 2, 3))
    c = Cache([100, 100], 2, 64, torch.float16, 16, seed=12)
    before = [_bits(x) for x in c.k + c.v]
    c.tables[0] = -1
    c.tables[1] = 1 << 20
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.evict_tokens(c.k, c.v, [torch.rand(2, 2, 100, device=DEV)], c.tables, c.lens,
                    torch.tensor([50, 50], dtype=torch.int32, device=DEV), 100, 50, error_word=err)
    assert int(err.item()) == pa.ERRBIT_BLOCK_OOB
    assert all(torch.equal(_bits(a), b) for a, b in zip(c.k + c.v, before))


def test_sources_behind_the_budget_may_be_shared():
    """Two sequences share their last blocks, which eviction only reads."""
    c = Cache([128, 64], 2, 64, torch.float16, 16, seed=13)
    c.tables_host = np.concatenate([c.tables_host, np.full((2, 0), -1, np.int32)], 1)
    c.tables_host[1, 4:8] = c.tables_host[0, 4:8]
    c.tables = torch.as_tensor(c.tables_host, device=DEV)
    c.lens_host = [128, 128]
    c.lens = torch.tensor([128, 128], dtype=torch.int32, device=DEV)
    _check(c, _scores(1, 2, 2, 128, seed=14), [64, 50], 0, 10)


def test_captured_and_replayed():
    c = Cache([300, 200], 2, 128, torch.bfloat16, 16, seed=15, spare=30)
    sc = _scores(1, 2, 2, 300, seed=16)
    keep = torch.tensor([100, 150], dtype=torch.int32, device=DEV)
    nb = -(-150 // 16)
    dst = torch.as_tensor(c.spare[:2 * nb].reshape(2, nb).copy(), device=DEV)
    args = lambda k, v, o, n: dict(  # noqa: E731
        k_caches=[k], v_caches=[v], scores=[sc[0]], block_tables=c.tables, context_lens=c.lens, keep_lens=keep,
        max_context_len=300, max_keep_len=150, num_sink=4, num_recent=20, dst_block_tables=dst, scores_out=[o],
        new_lens=n)
    k1, v1, o1 = c.k[0].clone(), c.v[0].clone(), torch.zeros_like(sc[0])
    n1 = torch.zeros(2, dtype=torch.int32, device=DEV)
    pa.evict_tokens(**args(k1, v1, o1, n1))
    k2, v2, o2, n2 = c.k[0].clone(), c.v[0].clone(), torch.zeros_like(sc[0]), torch.zeros_like(n1)
    ws = torch.empty(pa.evict_workspace_size(1, 2, 2, 300, 150), dtype=torch.uint8, device=DEV)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pa.evict_tokens(**args(k2, v2, o2, n2), workspace=ws)
    for fill in (255, 0, 7):
        ws.fill_(fill)
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(_bits(k1), _bits(k2)) and torch.equal(_bits(v1), _bits(v2))
    assert torch.equal(o1, o2) and n1.tolist() == n2.tolist() == [100, 150]


@pytest.mark.parametrize("D,run,gap", [(64, 100, 1), (128, 1, 100), (128, 500, 130), (256, 33, 31)])
def test_in_place_runs_of_kept_tokens(D, run, gap):
    """Runs of kept tokens between gaps: new rows reach the old rows of chunks
    right before and far before their own."""
    L = [20000, 4097, 130]
    c = Cache(L, 2, D, torch.bfloat16, 16, seed=run, layers=2)
    sc = _scores(2, len(L), 2, 20000, seed=gap)
    t = torch.arange(20000, device=DEV) % (run + gap)
    sc += (t < run).float()
    keep = [int((t[:n] < run).sum()) for n in L]
    _check(c, sc, keep, 0, 0)
