"""pa_decode_attention_scored on the GPU: output and scores against the
definition in 64 bits (tolerances: see cachelib)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from cachelib import DT, Cache, logits64, weights64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _check(c, q, scale, max_len=None, stride=None, block_ok=None, out_dtype=torch.float32, steps=1):
    S, H, D = q.shape
    Hkv = c.k[0].shape[1]
    G = H // Hkv
    max_len = max_len or c.max_len
    stride = stride or max_len
    base = torch.rand(S, Hkv, stride, device=DEV)
    scores = base.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(steps):
        out = pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, max_len, scale, scores,
                                         out_dtype=out_dtype, error_word=err)
    torch.cuda.synchronize()
    for s, n in enumerate(c.lens_host):
        if n <= 0 or n > max_len:
            assert not out[s].any() and torch.equal(scores[s], base[s])
            continue
        for h in range(Hkv):
            x, e = logits64(q[s, h * G:(h + 1) * G], c.rows(c.k[0], s, h), scale)
            v = c.rows(c.v[0], s, h).double()
            if block_ok is not None:
                x[:, ~block_ok[s]] = -np.inf
                e[:, ~block_ok[s]] = 0
                v[~block_ok[s]] = 0
            p, tol = weights64(x, e)
            want = base[s, h, :n].double() + steps * p.sum(0)
            lim = steps * tol.sum(0) + (steps + 1) * 2.0 ** -24 * want + 1e-30
            d = (scores[s, h, :n].double() - want).abs()
            assert bool((d <= lim).all()), (s, h, float((d - lim).max()))
            assert torch.equal(scores[s, h, n:], base[s, h, n:])
            o = p @ v
            # P is rounded to 16 bits in two parts (2^-15 of the weights at most) before P V
            lo = tol @ v.abs() + 2.0 ** -15 * (p @ v.abs()) + n * 2.0 ** -24 * (p @ v.abs())
            lo = lo + torch.finfo(out_dtype).eps / 2 * o.abs() * 1.001 + 2.0 ** -25
            got = out[s, h * G:(h + 1) * G].double()
            assert bool(((got - o).abs() <= lo).all()), (s, h)
    return out, scores, int(err.item())


def _q(S, H, D, dtype, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(S, H, D, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,B", [
    (1, 1, 64, 16), (4, 4, 128, 8), (2, 2, 256, 16), (4, 2, 64, 8), (12, 2, 128, 16), (8, 1, 128, 32),
    (15, 5, 64, 256), (7, 1, 128, 64), (4, 2, 256, 16), (3, 1, 256, 128), (6, 1, 256, 8), (16, 2, 256, 16)])
def test_lengths_at_the_edges(H, Hkv, D, B, dtype):
    lens = [1, 15, 16, 17, 0, 255, 256, 257, 33, 511, 512, 513, 700]
    c = Cache(lens, Hkv, D, DT[dtype], B, seed=H)
    _, _, err = _check(c, _q(len(lens), H, D, DT[dtype]), D ** -0.5)
    assert err == 0


@pytest.mark.parametrize("H,Hkv", [(4, 4), (12, 2)])
@pytest.mark.parametrize("lens", [[1], [5, 9, 200], [256] * 4, [1024, 1, 1023], [0, 0], [20000]])
def test_small_and_long_batches(lens, H, Hkv):
    c = Cache(lens, Hkv, 128, torch.bfloat16, seed=len(lens))
    _check(c, _q(len(lens), H, 128, torch.bfloat16), 0.1, max_len=max(max(lens), 1))


def test_many_sequences_use_the_plan():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 700, 90)
    c = Cache(lens, 4, 64, torch.float16, seed=2)
    _check(c, _q(90, 4, 64, torch.float16), 0.125)


def test_odd_strides_a_loose_bound_and_several_steps():
    c = Cache([40, 300, 77], 2, 128, torch.float16, seed=4)
    _check(c, _q(3, 6, 128, torch.float16), 0.2, max_len=304, stride=1001, out_dtype=torch.float16, steps=3)


def test_negative_and_zero_scale():
    c = Cache([40, 300, 77], 2, 128, torch.float16, seed=4)
    _check(c, _q(3, 2, 128, torch.float16), 0.0)
    q = _q(3, 2, 128, torch.float16)
    a, b = torch.zeros(2, 3, 2, 300, device=DEV)
    pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 300, -0.1, a)
    pa.decode_attention_scored(-q, c.k[0], c.v[0], c.tables, c.lens, 300, 0.1, b)
    assert torch.allclose(a, b, rtol=1e-6, atol=0)


@pytest.mark.parametrize("H,Hkv,B", [(2, 2, 16), (12, 2, 16), (2, 2, 64), (8, 2, 32)])
def test_bad_lengths_and_skipped_blocks(H, Hkv, B):
    lens = [300, 40, 100, 600, 64]
    c = Cache(lens, Hkv, 64, torch.bfloat16, B, seed=6)
    ok = [torch.ones(n, dtype=torch.bool, device=DEV) for n in lens]
    for s, i, bad in ((0, 1, -1), (3, 0, 10 ** 6), (3, 4, -7)):
        c.tables[s, i] = bad
        ok[s][i * B:(i + 1) * B] = False
    for i in range(-(-lens[4] // B)):  # no readable block at all
        c.tables[4, i] = -1
    lens_in = c.lens.clone()
    c.lens = torch.tensor([300, -3, 100, 600, 64], dtype=torch.int32, device=DEV)
    c.lens_host = [300, -3, 100, 600, 0]  # the oracle's zero row and untouched scores
    _, _, err = _check(c, _q(5, H, 64, torch.bfloat16), 0.125, max_len=600, block_ok=ok)
    assert err == pa.ERRBIT_BLOCK_OOB | pa.ERRBIT_CONTEXT_LEN
    c.lens = lens_in
    c.lens[2] = 601
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    sc = torch.zeros(5, Hkv, 600, device=DEV)
    pa.decode_attention_scored(_q(5, H, 64, torch.bfloat16), c.k[0], c.v[0], c.tables, c.lens, 600, 0.1,
                               sc, error_word=err)
    assert int(err.item()) & pa.ERRBIT_CONTEXT_LEN and not sc[2].any()


def test_shared_blocks_and_repeatability():
    """Sequences that name the same blocks keep their own scores; two runs are bit-identical."""
    c = Cache([512], 4, 128, torch.float16, seed=7)
    S = 40
    c.tables_host = np.repeat(c.tables_host, S, 0)
    c.tables = torch.as_tensor(c.tables_host, device=DEV)
    c.lens_host = [512 - 3 * s for s in range(S)]
    c.lens = torch.tensor(c.lens_host, dtype=torch.int32, device=DEV)
    q = _q(S, 4, 128, torch.float16)
    a, sa, _ = _check(c, q, 0.1)
    sb, sc = torch.zeros_like(sa), torch.zeros_like(sa)
    b = pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 512, 0.1, sb)
    pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 512, 0.1, sc)
    assert torch.equal(a, b) and torch.equal(sb, sc)


def test_weights_sum_to_the_group_and_match_the_unscored_output():
    lens = [700, 33, 5000, 256]
    c = Cache(lens, 2, 128, torch.bfloat16, seed=8)
    q = _q(4, 12, 128, torch.bfloat16)
    sc = torch.zeros(4, 2, 5000, device=DEV)
    out = pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 5000, 0.0884, sc)
    # n terms of at most 6 in total: below 5000 * 2^-24 * 6
    assert torch.allclose(sc.double().sum(-1), torch.full((4, 2), 6.0, dtype=torch.float64, device=DEV),
                          rtol=5000 * 2.0 ** -24, atol=0)
    plain = pa.decode_attention(q, c.k[0], c.v[0], c.tables, c.lens, 5000, 0.0884)
    assert torch.allclose(out, plain, rtol=1e-4, atol=1e-5)


def test_captured_into_a_graph_and_replayed():
    c = Cache([300, 90, 0, 511], 2, 64, torch.float16, seed=9)
    q = _q(4, 8, 64, torch.float16)
    want = torch.zeros(4, 2, 511, device=DEV)
    ws = torch.empty(pa.decode_scored_workspace_size(4, 8, 2, 64, 511), dtype=torch.uint8, device=DEV)
    ref = pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 511, 0.125, want)
    sc, out = torch.zeros_like(want), torch.empty_like(ref)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 511, 0.125, sc, out=out, workspace=ws)
    ws.fill_(255)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(sc, want + want)


@pytest.mark.parametrize("H,Hkv", [(2, 2), (12, 2)])
def test_nan_stays_with_its_sequence_and_head(H, Hkv):
    c = Cache([600, 90], Hkv, 64, torch.bfloat16, seed=11)
    q = _q(2, H, 64, torch.bfloat16)
    clean = torch.zeros(2, Hkv, 600, device=DEV)
    pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 600, 0.125, clean)
    c.k[0][int(c.tables_host[0, 3]), 1, 5] = float("nan")  # token 53 of sequence 0, head 1
    got = torch.zeros_like(clean)
    pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 600, 0.125, got)
    assert bool(torch.isnan(got[0, 1, :600]).all())
    assert torch.equal(got[0, 0], clean[0, 0]) and torch.equal(got[1], clean[1])


@pytest.mark.parametrize("B", [8, 16, 64])
@pytest.mark.parametrize("H,Hkv,D", [(2, 2, 64), (12, 2, 64), (6, 2, 256)])
def test_a_nan_row_leaves_the_skipped_blocks_alone(H, Hkv, D, B):
    c = Cache([600, 90], Hkv, D, torch.bfloat16, B, seed=11)
    q = _q(2, H, D, torch.bfloat16)
    c.k[0][int(c.tables_host[0, 53 // B]), 1, 53 % B] = float("nan")  # token 53 of sequence 0, head 1
    first, last = (128 // B, 143 // B) if B < 64 else (2, 2)
    c.tables[0, first] = 10 ** 7
    c.tables[0, 599 // B] = -1  # the last, short block
    skipped = torch.zeros(600, dtype=torch.bool, device=DEV)
    skipped[first * B:(last + 1) * B] = True
    skipped[599 // B * B // 16 * 16:] = True
    base = torch.rand(2, Hkv, 603, device=DEV)
    for sc in (base.clone(), base.clone()[:, :, :600].contiguous()):  # any row stride
        pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 600, 0.1, sc)
        assert torch.equal(sc[:, :, :600][0][:, skipped], base[:, :, :600][0][:, skipped])
        assert bool(torch.isnan(sc[0, 1, :600][~skipped]).all())
        assert bool(torch.isfinite(sc[0, 0]).all()) and bool(torch.isfinite(sc[1]).all())
        assert bool((sc[0, 0, :600][~skipped] > base[0, 0, :600][~skipped]).any())
