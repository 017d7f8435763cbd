"""A 16-bit decode call whose workspace is memory that the call ahead of it on the stream
still uses: inputs that the caller dropped, or a workspace of its own.  Kernels overlap
their launches, so the decode's first kernel runs while the call ahead does, and must not
write before that has ended."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from cachelib import Cache
from q4lib import Q4Cache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = torch.bfloat16


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


class Step16:
    """A decode step whose plan has many items (64 sequences of up to 40 pages, 8 heads), in a
    workspace at the start of `mem`."""

    def __init__(self, seqs=64):
        g = torch.Generator(device=DEV).manual_seed(3)
        self.kv = [torch.randn(seqs * 40, 8, 16, 128, generator=g, device=DEV).to(DT) for _ in range(2)]
        self.q = torch.randn(seqs, 8, 128, generator=g, device=DEV).to(DT)
        self.tables = _i32(np.arange(seqs * 40).reshape(seqs, 40))
        self.lens = _i32(np.arange(seqs) * 9 % 640 + 1)
        self.out = torch.empty(seqs, 8, 128, device=DEV)
        self.nbytes = pa.decode_workspace_size(seqs, 8, 8, 128, 640)
        self.mem = torch.empty(max(self.nbytes, 1 << 28), dtype=torch.uint8, device=DEV)
        self.want = pa.decode_attention(self.q, *self.kv, self.tables, self.lens, 640, 0.1).clone()

    def run(self):
        pa.decode_attention(self.q, *self.kv, self.tables, self.lens, 640, 0.1, out=self.out, workspace=self.mem)

    def view(self, x):
        """A tensor like x at the start of the workspace, where the plan's lists go."""
        return self.mem[:x.nbytes].view(x.dtype).view(x.shape)


def _check(step, data, run, results, rounds=20):
    """run(x) with the input at the workspace's start and the decode step right behind it:
    results and step as with memory of their own."""
    want = [t.clone() for t in run(data)]
    there = step.view(data)
    for _ in range(rounds):
        there.copy_(data)
        for t in results:
            t.zero_()
        got = run(there)
        step.run()
        # (bytes: slots that were never written may read as NaN)
        assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
                   for a, b in zip(got, want))
        assert torch.equal(step.out, step.want)


@pytest.mark.parametrize("which", ["query", "key", "positions", "slots"])
@pytest.mark.parametrize("T,H,Hkv,q4", [(64, 12, 2, True), (4000, 12, 2, True), (3000, 40, 40, True), (64, 12, 2, False),
                                        (4000, 12, 2, False), (3000, 40, 40, False)])
def test_rotary_write(T, H, Hkv, q4, which):
    g = torch.Generator(device=DEV).manual_seed(T)
    step = Step16()
    args = {"query": torch.randn(T, H, 128, generator=g, device=DEV).to(DT),
            "key": torch.randn(T, Hkv, 128, generator=g, device=DEV).to(DT),
            "positions": torch.randint(0, 9000, (T,), generator=g, device=DEV),
            "slots": torch.randperm(T, generator=g, device=DEV)}
    nb = -(-T // 16)
    shape, dt = (pa.q4_pool_shape(nb, Hkv, 16, 128), torch.uint8) if q4 else ((nb, Hkv, 16, 128), DT)
    pools = [torch.zeros(shape, dtype=dt, device=DEV) for _ in range(2)]
    out, value = torch.empty(T, H, 128, dtype=DT, device=DEV), args["key"].clone()
    rot = pa.Rotary([0.5 ** (i / 8) for i in range(64)])
    call = pa.rotary_cache_write_q4 if q4 else pa.rotary_cache_write

    def run(x):
        a = {**args, which: x}
        call(a["query"], a["key"], value, a["positions"], rot, *pools, a["slots"], query_out=out)
        return [out, *pools]

    _check(step, args[which], run, [out, *pools])


@pytest.mark.parametrize("which", ["key", "slots"])
@pytest.mark.parametrize("q4", [True, False])
def test_plain_write(q4, which):
    T, Hkv = 5000, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    step = Step16()
    args = {"key": torch.randn(T, Hkv, 128, generator=g, device=DEV).to(DT),
            "slots": torch.randperm(T, generator=g, device=DEV)}
    nb = -(-T // 16)
    shape, dt = (pa.q4_pool_shape(nb, Hkv, 16, 128), torch.uint8) if q4 else ((nb, Hkv, 16, 128), DT)
    pools = [torch.zeros(shape, dtype=dt, device=DEV) for _ in range(2)]
    value = args["key"].clone()
    call = pa.cache_write_q4 if q4 else pa.cache_write

    def run(x):
        a = {**args, which: x}
        call(a["key"], value, *pools, a["slots"])
        return pools

    _check(step, args[which], run, pools)


@pytest.mark.parametrize("which", ["query", "workspace"])
@pytest.mark.parametrize("call", ["prefill", "decode_q4", "decode_q4_cut", "decode", "scored"])
def test_attention_ahead(call, which):
    """The query of the call ahead, or its whole workspace, in the decode step's workspace."""
    g = torch.Generator(device=DEV).manual_seed(5)
    step = Step16()
    H, Hkv = 16, 4
    if call == "prefill":
        lens, new = [900, 700, 512, 1500], [800, 600, 512, 700]
        c = Cache(lens, Hkv, 128, DT, 16, seed=2)
        starts = _i32(np.concatenate([[0], np.cumsum(new)]))
        q = torch.randn(sum(new), H, 128, generator=g, device=DEV).to(DT)
        out = torch.empty(q.shape, device=DEV)
        nbytes = pa.prefill_workspace_size(4, H, Hkv, 128, max(new))

        def attend(x, ws):
            pa.prefill_attention(x, c.k[0], c.v[0], c.tables, starts, c.lens, max(new), c.max_len, 0.1, out=out,
                                 workspace=ws)
    else:
        lens = [200 if call == "decode_q4" else 900 + 10 * i for i in range(64)]
        c = Q4Cache(lens, Hkv, 128, DT, 16, seed=2) if "q4" in call else Cache(lens, Hkv, 128, DT, 16, seed=2)
        q = torch.randn(64, H, 128, generator=g, device=DEV).to(DT)
        out = torch.empty(q.shape, device=DEV)
        scores = torch.zeros(64, Hkv, c.max_len, device=DEV)
        sizes = {"decode": pa.decode_workspace_size, "scored": pa.decode_scored_workspace_size}
        nbytes = (pa.decode_q4_workspace_size(64, H, Hkv, 128, 1, c.max_len) if "q4" in call
                  else sizes[call](64, H, Hkv, 128, c.max_len))

        def attend(x, ws):
            if "q4" in call:
                pa.decode_attention_q4(x, c.k4[0], c.v4[0], c.tables, c.lens, c.max_len, 0.1, out=out, workspace=ws)
            elif call == "scored":
                pa.decode_attention_scored(x, c.k[0], c.v[0], c.tables, c.lens, c.max_len, 0.1, scores, out=out,
                                           workspace=ws)
            else:
                pa.decode_attention(x, c.k[0], c.v[0], c.tables, c.lens, c.max_len, 0.1, out=out, workspace=ws)

    own = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=DEV)
    assert own.nbytes <= step.mem.nbytes
    if which == "query":
        def run(x):
            attend(x, own)
            return [out]
        _check(step, q, run, [out])
    else:
        def run(ws):
            attend(q, ws)
            return [out]
        _check(step, own, run, [out])
