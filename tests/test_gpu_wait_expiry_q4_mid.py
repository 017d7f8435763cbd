"""Waits of the 4-bit decode kernel that give up in the middle of a call, when some of a
warp's copies have come and others are in flight: a call that reports nothing is right, one
that reports PA_ERRBIT_TIMEOUT leaves the GPU answering."""
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
# heads, KV heads, head_dim, query tokens a sequence, lengths
CASES = {"rows1_128": (8, 8, 128, 1, [4000, 900, 33, 2500]), "rows6_128": (12, 2, 128, 1, [4000, 900, 33, 2500]),
         "rows12_64": (12, 2, 64, 2, [1500] * 40), "rows2_256": (4, 2, 256, 1, [700, 1500, 33, 9000, 2]),
         "short_64": (4, 4, 64, 1, [200, 33, 2, 250] * 20)}


def _child(case, lib_path):
    import paged_kv_cache_pa_gb300 as pa
    if lib_path:
        pa._LIB_PATH = lib_path             # this process loads only the test copy
    from q4lib import Q4Cache, attention
    H, Hkv, D, n, lens = CASES[case]
    c = Q4Cache(lens, Hkv, D, torch.bfloat16, seed=1)
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn(n * len(lens), H, D, generator=g, device=DEV).to(torch.bfloat16)
    starts = torch.arange(0, n * len(lens) + 1, n, dtype=torch.int32, device=DEV)
    want, tol = attention(c, q, starts.tolist(), 0.09)
    runs = []
    for _ in range(20):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = pa.decode_attention_q4(q, c.k4[0], c.v4[0], c.tables, c.lens, c.max_len, 0.09, query_start_loc=starts,
                                     max_query_len=n, error_word=err)
        runs.append((int(err.item()), bool(((out.double() - want).abs() <= tol).all())))
    a = torch.randn(256, 256, device=DEV)
    ok = bool(torch.allclose(a @ torch.eye(256, device=DEV), a))
    print(json.dumps({"runs": runs, "gpu_answers": ok}), flush=True)


@pytest.mark.parametrize("case", sorted(CASES))
def test_a_call_is_right_or_says_that_it_gave_up(case):
    from paged_kv_cache_pa_gb300.build import build
    lib = build(variant="midwait")
    r = subprocess.run([sys.executable, os.path.abspath(__file__), case, lib], capture_output=True, text=True,
                       timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res["gpu_answers"]
    for err, right in res["runs"]:
        assert err in (0, 8) and (right or err == 8), res


if __name__ == "__main__":
    _child(sys.argv[1], sys.argv[2])
