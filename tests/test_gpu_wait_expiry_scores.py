"""Scores after a wait that gave up: a call that reports PA_ERRBIT_TIMEOUT has
added a token's whole weight or nothing.  The child process runs the test copy
of the library whose waits give up after a few polls (test_gpu_wait_expiry).

Tolerance of a whole weight, relative: 130 2^-24 sum |q k| scale = 7e-5 from x
(128 products of standard normal numbers, scaled, sum to 9 at most), 2^-20 from
lse and its product, 2^-21 from the exponential, and 2^-12 from a sum of 3600
terms in any order: together below 4e-4.  The score itself, below 2^5, adds
2^-18.  A sum that lacks a product lacks one of at most 38, some hundredths of
it."""
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


def _prompts(pa, D, times, calls, err):
    """(scores left, whole, neither) of `calls` calls."""
    from cachelib import Cache
    lens, new = [900, 600, 1500] * times, [900, 500, 1200] * times
    c = Cache(lens, 2, D, torch.float16, seed=1)
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn(sum(new), 6, D, generator=g, device=DEV).to(torch.float16)
    lse = torch.full((sum(new), 6), 7.0, device=DEV)
    qsl = torch.tensor([0] + new, device=DEV).cumsum(0).int()
    base = torch.rand(len(new), 2, 1500, generator=g, device=DEV)
    want = torch.zeros(len(new), 2, 1500, dtype=torch.float64, device=DEV)
    i = 0
    for s, (n, m) in enumerate(zip(lens, new)):
        for h in range(2):
            x = q[i:i + m, 3 * h:3 * h + 3].double().transpose(0, 1) @ c.rows(c.k[0], s, h).double().T * D ** -0.5
            x.masked_fill_(torch.ones(m, n, dtype=torch.bool, device=DEV).triu(n - m + 1), float("-inf"))
            want[s, h, :n] = torch.exp(x - 7.0).sum((0, 1))
        i += m
    count, flush = [0, 0, 0], torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    for i in range(calls):
        sc = base.clone()
        if i % 2 == 0:
            flush.fill_(i)  # copies from memory now, from L2 then
        pa.prefill_scores(q, lse, c.k[0], c.tables, qsl, c.lens, 1200, 1500, D ** -0.5, sc, error_word=err)
        torch.cuda.synchronize()
        left = sc == base
        whole = ~left & ((sc.double() - base.double() - want).abs() <= 4e-4 * want + 2.0 ** -18)
        for k, x in enumerate((left, whole, ~left & ~whole)):
            count[k] += int(x.sum())
    return count, int((want > 0).sum())


def _decode(pa, H, Hkv, S, err):
    """(scores left, others) of 20 steps, each with the error word zeroed before and set after."""
    from cachelib import Cache
    lens = ([700, 1500, 33, 4000, 2] * S)[:S] if S > 2 else [200, 33]
    c = Cache(lens, Hkv, 128, torch.bfloat16, seed=1)
    g = torch.Generator(device=DEV).manual_seed(2)
    q = torch.randn(S, H, 128, generator=g, device=DEV).to(torch.bfloat16)
    base = torch.rand(S, Hkv, c.max_len, generator=g, device=DEV)
    live = torch.arange(c.max_len, device=DEV)[None, None] < c.lens[:, None, None]
    live = live.expand_as(base)
    left = other = 0
    for i in range(20):
        err.zero_()
        sc = base.clone()
        # a workspace with something in it that could pass for logits and states
        ws = torch.full((pa.decode_scored_workspace_size(S, H, Hkv, 128, c.max_len) // 4,), 0.5, device=DEV)
        pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, c.max_len, 0.09, sc, workspace=ws, error_word=err)
        torch.cuda.synchronize()
        if not int(err.item()) & 8:
            continue  # every wait was short enough this time
        left += int((sc == base)[live].sum())
        other += int((sc != base)[live].sum())
    return left, other


def _child(case, lib_path):
    import paged_kv_cache_pa_gb300 as pa
    pa._LIB_PATH = lib_path                 # this process loads only the test copy
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if case.startswith("decode"):
        left, other = _decode(pa, *(int(x) for x in case.split("_")[1:]), err)
        print(json.dumps({"left": left, "other": other}), flush=True)
        return
    _, D, times = case.split("_")
    (left, whole, other), _ = _prompts(pa, int(D), int(times), 40 if times == "1" else 4, err)
    print(json.dumps({"err": int(err.item()), "left": left, "whole": whole, "other": other}), flush=True)


def _run(case, variant):
    from paged_kv_cache_pa_gb300.build import build
    r = subprocess.run([sys.executable, os.path.abspath(__file__), case, build(variant=variant)],
                       capture_output=True, text=True, timeout=600, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


# With 4 polls every first wait gives up; with more, some items are done before one does.
@pytest.mark.parametrize("variant", ["shortwait", "midwait"])
@pytest.mark.parametrize("case", ["prompts_64_1", "prompts_128_1", "prompts_128_12"])
def test_prompt_scores_are_left_or_whole(case, variant):
    """One prompt of each length: clusters share the items; many: they do not."""
    import paged_kv_cache_pa_gb300 as pa
    res = _run(case, variant)
    assert res["err"] & 8 and res["left"] and res["other"] == 0, res
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    (_, whole, other), tokens = _prompts(pa, int(case.split("_")[1]), int(case.split("_")[2]), 1, err)
    assert int(err.item()) == 0 and other == 0 and whole == tokens


@pytest.mark.parametrize("variant", ["shortwait", "midwait"])
@pytest.mark.parametrize("case", ["decode_4_4_5", "decode_12_2_5", "decode_12_2_2"])
def test_decode_scores_are_left(case, variant):
    """(H, Hkv, sequences): both attention kernels, with and without partitions and plan."""
    res = _run(case, variant)
    assert res["other"] == 0 and (res["left"] or variant == "midwait"), res


def test_scores_are_added_again_once_the_error_word_is_zeroed():
    import paged_kv_cache_pa_gb300 as pa
    from cachelib import Cache
    c = Cache([300, 40], 2, 64, torch.float16, seed=1)
    q = torch.randn(2, 4, 64, device=DEV).to(torch.float16)
    sc = torch.zeros(2, 2, 300, device=DEV)
    err = torch.full((1,), pa.ERRBIT_TIMEOUT, dtype=torch.int32, device=DEV)
    pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 300, 0.1, sc, error_word=err)
    assert not sc.any()
    for word in (0, pa.ERRBIT_BLOCK_OOB):  # another bit does not hold the scores back
        err.fill_(word)
        sc.zero_()
        pa.decode_attention_scored(q, c.k[0], c.v[0], c.tables, c.lens, 300, 0.1, sc, error_word=err)
        assert torch.allclose(sc.sum(-1), torch.full((2, 2), 2.0, device=DEV), rtol=1e-4)


if __name__ == "__main__":
    _child(sys.argv[1], sys.argv[2])
