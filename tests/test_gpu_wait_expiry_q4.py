"""The give-up path of the 4-bit decode kernel's waits, in the way of
test_gpu_wait_expiry: a test copy of the library whose waits give up after a few
polls reports PA_ERRBIT_TIMEOUT, the GPU keeps answering, and the next call
through the product library is right."""
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
# heads, KV heads, head_dim, query tokens a sequence
CASES = {"rows1_64": (4, 4, 64, 1), "rows4_128": (8, 2, 128, 1), "rows6_128": (12, 2, 128, 1), "rows12_128": (12, 2, 128, 2),
         "rows2_256": (4, 2, 256, 1), "short_128": (4, 4, 128, 1)}


def _run(case, err):
    import paged_kv_cache_pa_gb300 as pa
    from q4lib import Q4Cache
    H, Hkv, D, n = CASES[case]
    lens = [200, 33, 2, 250] if case.startswith("short") else [700, 1500, 33, 4000, 2]
    c = Q4Cache(lens, Hkv, D, torch.bfloat16, seed=1)
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn(n * len(lens), H, D, generator=g, device=DEV).to(torch.bfloat16)
    starts = torch.arange(0, n * len(lens) + 1, n, dtype=torch.int32, device=DEV)
    out = pa.decode_attention_q4(q, c.k4[0], c.v4[0], c.tables, c.lens, c.max_len, 0.09, query_start_loc=starts,
                                 max_query_len=n, error_word=err)
    return c, q, starts, out


def _child(case, lib_path):
    import paged_kv_cache_pa_gb300 as pa
    pa._LIB_PATH = lib_path                 # this process loads only the test copy
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    _run(case, err)
    torch.cuda.synchronize()
    a = torch.randn(256, 256, device=DEV)
    ok = bool(torch.allclose(a @ torch.eye(256, device=DEV), a))
    print(json.dumps({"err": int(err.item()), "gpu_answers": ok}), flush=True)


@pytest.mark.parametrize("case", sorted(CASES))
def test_waits_give_up_then_the_next_call_is_right(case):
    if not torch.cuda.is_available():  # pragma: no cover
        pytest.skip("needs a CUDA device")
    from paged_kv_cache_pa_gb300.build import build
    from q4lib import attention
    lib = build(variant="shortwait")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), case, lib], capture_output=True, text=True,
                       timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["err"] == 8, res             # PA_ERRBIT_TIMEOUT
    assert res["gpu_answers"]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    c, q, starts, out = _run(case, err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want, tol = attention(c, q, starts.tolist(), 0.09)
    assert bool(((out.double() - want).abs() <= tol).all())


if __name__ == "__main__":
    _child(sys.argv[1], sys.argv[2])
