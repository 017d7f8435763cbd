"""The give-up path of the bounded-cache kernels' waits, in the way of
test_gpu_wait_expiry: a test copy of the library whose ordinary waits give up
after a few polls reports PA_ERRBIT_TIMEOUT, the GPU keeps answering, and the
next call through the product library is right."""
import json
import os
import subprocess
import sys

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
for p in (ROOT, HERE):
    if p not in sys.path:
        sys.path.insert(0, p)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CASES = ["decode_scored_g1", "decode_scored_g6", "prefill_scores_64", "prefill_scores_128", "prefill_scores_many_128",
         "evict_in_place"]


def _run(case, err):
    import paged_kv_cache_pa_gb300 as pa
    from cachelib import Cache
    g = torch.Generator(device=DEV).manual_seed(2)
    if case.startswith("decode"):
        H, Hkv = (4, 4) if case.endswith("g1") else (12, 2)
        c = Cache([700, 1500, 33, 4000, 2], Hkv, 128, torch.bfloat16, seed=1)
        q = torch.randn(5, H, 128, generator=g, device=DEV).to(torch.bfloat16)
        sc = torch.zeros(5, Hkv, 4000, device=DEV)
        pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 4000, 0.09, sc, error_word=err)
        return c, sc, H
    if case.startswith("prefill"):
        D = int(case.rsplit("_", 1)[1])
        times = 20 if "many" in case else 1  # more items than are shared by clusters
        c = Cache([900, 600, 300] * times, 2, D, torch.float16, seed=1)
        new = [900, 200, 64] * times
        q = torch.randn(sum(new), 6, D, generator=g, device=DEV).to(torch.float16)
        lse = torch.full((sum(new), 6), 7.0, device=DEV)
        qsl = torch.tensor([0] + new, device=DEV).cumsum(0).int()
        sc = torch.zeros(len(new), 2, 900, device=DEV)
        pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 900, 900, D ** -0.5, sc, error_word=err)
        return c, sc, (q, new)
    c = Cache([40000], 4, 128, torch.float16, seed=1)
    before = c.k[0].clone()
    sc = torch.rand(1, 4, 40000, generator=g, device=DEV)
    kept = torch.zeros(1, 4, 30000, dtype=torch.int32, device=DEV)
    pa.evict_tokens(c.k, c.v, [sc], c.tables, c.lens, torch.tensor([30000], dtype=torch.int32, device=DEV), 40000,
                    30000, kept=[kept], error_word=err)
    return c, kept, before


def _child(case, lib_path):
    import paged_kv_cache_pa_gb300 as pa
    pa._LIB_PATH = lib_path                 # this process loads only the test copy
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    _run(case, err)
    torch.cuda.synchronize()
    a = torch.randn(256, 256, device=DEV)
    ok = bool(torch.allclose(a @ torch.eye(256, device=DEV), a))
    print(json.dumps({"err": int(err.item()), "gpu_answers": ok}), flush=True)


@pytest.mark.parametrize("case", CASES)
def test_waits_give_up_then_the_next_call_is_right(case):
    if not torch.cuda.is_available():  # pragma: no cover
        pytest.skip("needs a CUDA device")
    from paged_kv_cache_pa_gb300.build import build
    lib = build(variant="shortwait")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), case, lib], capture_output=True, text=True,
                       timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["err"] & 8, res              # PA_ERRBIT_TIMEOUT
    assert res["gpu_answers"]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    c, got, more = _run(case, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    if case.startswith("decode"):           # the group's weights sum to its heads
        G = more // got.shape[1]
        assert torch.allclose(got.double().sum(-1), torch.full(got.shape[:2], float(G), dtype=torch.float64, device=DEV),
                              rtol=4000 * 2.0 ** -24, atol=0)
    elif case.startswith("prefill"):
        q, new = more
        i = 0
        for s, (n, m) in enumerate(zip(c.lens_host, new)):
            k = c.rows(c.k[0], s, 1).double()
            x = q[i:i + m, 3:6].double().transpose(0, 1) @ k.T * q.shape[-1] ** -0.5
            x.masked_fill_(torch.ones(m, n, dtype=torch.bool, device=DEV).triu(n - m + 1), float("-inf"))
            want = torch.exp(x - 7.0).sum((0, 1))
            assert torch.allclose(got[s, 1, :n].double(), want, rtol=1e-3, atol=1e-9)
            i += m
    else:
        idx = got[0, 2].long().cpu().numpy()
        t = c.tables_host[0]
        src = more[torch.as_tensor(t[idx // 16].astype("int64"), device=DEV), 2, torch.as_tensor(idx % 16, device=DEV)]
        assert torch.equal(c.rows(c.k[0], 0, 2, 30000), src)


if __name__ == "__main__":
    _child(sys.argv[1], sys.argv[2])
