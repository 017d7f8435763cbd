"""Calls on a stream of their own, which allocate what they need, while the
current stream allocates and fills memory: the results are those of calls on
the current stream."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from cachelib import Cache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LENS = [700, 1500, 33, 900]


def _decode(c, q, kw):
    return [pa.decode_attention(q, c.k[0], c.v[0], c.tables, c.lens, 1500, 0.1, **kw)]


def _contiguous(c, q, kw):
    k = torch.nan_to_num(c.k[0])[:4 * 32].reshape(4, 2, 16 * 32, 128)
    torch.cuda.synchronize()
    return [pa.decode_attention_contiguous(q, k, k, c.lens.clamp(max=512), 512, 0.1, **kw), k]


def _scored(c, q, kw):
    sc = torch.zeros(4, 2, 1500, device=DEV)
    torch.cuda.synchronize()
    return [pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 1500, 0.1, sc, **kw), sc]


def _prompt(c, q, kw):
    qsl = torch.arange(5, dtype=torch.int32, device=DEV)
    sc, lse = torch.zeros(4, 2, 1500, device=DEV), torch.empty(4, 12, device=DEV)
    torch.cuda.synchronize()
    out = pa.prefill_attention(q, c.k[0], c.v[0], c.tables, qsl, c.lens, 1, 1500, 0.1, lse=lse, **kw)
    return [out, lse, pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 1, 1500, 0.1, sc, **kw), qsl]


def _rotary(c, q, kw):
    slots = torch.as_tensor(np.arange(4, dtype=np.int64) * 16, device=DEV)
    key, pos, rot = q[:, :2].contiguous(), torch.arange(4, device=DEV), pa.Rotary([0.1] * 64)
    torch.cuda.synchronize()
    return [pa.rotary_cache_write(q, key, key, pos, rot, c.k[0], c.v[0], slots, **kw), c.k[0], c.v[0], slots, key, pos]


def _evict(c, q, kw):
    g = torch.Generator(device=DEV).manual_seed(5)
    sc = torch.rand(4, 2, 1500, generator=g, device=DEV)
    kept = torch.zeros(4, 2, 600, dtype=torch.int32, device=DEV)
    keep = torch.full((4,), 600, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    new = pa.evict_tokens(c.k, c.v, [sc], c.tables, c.lens, keep, 1500, 600, 4, 16, kept=[kept], **kw)
    return [new, sc, kept, c.k[0], c.v[0], keep]


@pytest.mark.parametrize("call", [_decode, _contiguous, _scored, _prompt, _rotary, _evict])
def test_a_call_on_a_stream_of_its_own(call):
    def inputs():
        c = Cache(LENS, 2, 128, torch.bfloat16, 16, seed=3)
        return c, torch.randn(4, 12, 128, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).bfloat16()

    want = [t.clone() for t in call(*inputs(), {})]
    c, q = inputs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # the call's kernels start some 20 ms later
    got = call(c, q, {"stream": side})
    filled = []
    for nbytes in [1 << i for i in range(8, 25)] * 3:  # whatever the call has given back
        filled.append(torch.empty(nbytes, dtype=torch.uint8, device=DEV).fill_(0x7f))
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    same = [torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float())) for a, b in zip(got, want)]
    assert all(same), same
    assert all(bool((t == 0x7f).all()) for t in filled)  # and the call's kernels left the others' memory alone
