"""The 4-bit cache as a server uses it: prompts in chunks over unpacked blocks, decode
steps with rotation, drafts, forks with copy-on-write, swapping, captured steps, other
streams."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from paged_kv_cache_pa_gb300.manager import BlockManager
from q4lib import Q4Cache, attention, rounded, values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


def _i64(x):
    return torch.as_tensor(np.asarray(x, np.int64), device=DEV)


class Server:
    """One layer of a server: a block manager, 4-bit pools, and what every sequence's
    tokens were (the turned 16-bit keys and values)."""

    def __init__(self, H, Hkv, D, dtype, block=16, blocks=60, seed=0):
        self.H, self.Hkv, self.D, self.dtype, self.block = H, Hkv, D, dtype, block
        self.bm = BlockManager(blocks, blocks, block)
        shape = pa.q4_pool_shape(blocks, Hkv, block, D)
        self.k, self.v = (torch.full(shape, 255, dtype=torch.uint8, device=DEV) for _ in range(2))
        self.rot = pa.Rotary([10000.0 ** (-i / (D // 2)) for i in range(D // 2)])
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.tokens = {}
        self.scale = D ** -0.5

    def append(self, news):
        """news: (sequence, count); returns the turned queries, in order."""
        slots, pos, n = [], [], sum(m for _, m in news)
        qkv = torch.randn(n, (self.H + 2 * self.Hkv) * self.D, generator=self.g, device=DEV).to(self.dtype)
        q, k, v = qkv.split([self.H * self.D, self.Hkv * self.D, self.Hkv * self.D], 1)
        q, k, v = (t.view(n, -1, self.D) for t in (q, k, v))
        for s, m in news:
            at = self.bm.seq_len(s)
            slots += list(self.bm.append(s, m))
            pos += list(range(at, at + m))
        copies = self.bm.take_copies()
        if len(copies):
            pa.copy_blocks([self.k], [self.v], _i64(copies).view(-1, 2))
        # what a 16-bit cache would hold
        k16 = torch.zeros(-(-n // 16), self.Hkv, 16, self.D, dtype=self.dtype, device=DEV)
        pa.rotary_cache_write(q, k, v, _i64(pos), self.rot, k16, torch.zeros_like(k16), torch.arange(n, device=DEV))
        turned = k16.transpose(1, 2).reshape(-1, self.Hkv, self.D)[:n]
        out = pa.rotary_cache_write_q4(q, k, v, _i64(pos), self.rot, self.k, self.v, _i64(slots))
        i = 0
        for s, m in news:
            old = self.tokens.get(s)
            new = (turned[i:i + m].clone(), v[i:i + m].clone())
            self.tokens[s] = new if old is None else tuple(torch.cat(p) for p in zip(old, new))
            i += m
        return out

    def batch(self, seqs):
        tables = [self.bm.table(s) for s in seqs]
        w = max(len(t) for t in tables)
        return _i32([list(t) + [-1] * (w - len(t)) for t in tables]), _i32([self.bm.seq_len(s) for s in seqs])

    def want(self, seqs, q, starts):
        """(out, tolerance) in 64 bits from the tokens, and not from any pool."""
        lens = [self.bm.seq_len(s) for s in seqs]
        c = Q4Cache(lens, self.Hkv, self.D, self.dtype, 16)
        k = torch.cat([self.tokens[s][0] for s in seqs])
        v = torch.cat([self.tokens[s][1] for s in seqs])
        c.k[0][c.slots // 16, :, c.slots % 16] = k
        c.v[0][c.slots // 16, :, c.slots % 16] = v
        return attention(c, q, starts, self.scale)

    def decode(self, seqs, q, new=None):
        tables, lens = self.batch(seqs)
        starts = np.concatenate([[0], np.cumsum(new or [1] * len(seqs))])
        L = int(lens.max())
        out = pa.decode_attention_q4(q, self.k, self.v, tables, lens, L, self.scale,
                                     query_start_loc=None if new is None else _i32(starts),
                                     max_query_len=1 if new is None else max(new))
        want, tol = self.want(seqs, q, starts)
        assert bool(((out.double() - want).abs() <= tol).all()), float(((out.double() - want).abs() / tol).max())
        return out


@pytest.mark.parametrize("H,Hkv,D,dtype,block", [(12, 2, 128, torch.bfloat16, 16), (8, 8, 64, torch.float16, 32)])
def test_a_server(H, Hkv, D, dtype, block):
    """Prompts, decode steps, a fork that both branches go on from, a draft of which the
    tail is taken back, a swap out and in: attention is that of the sequences' tokens at
    every step."""
    srv = Server(H, Hkv, D, dtype, block)
    a, b = srv.bm.new_sequence(), srv.bm.new_sequence()
    srv.append([(a, 37), (b, 150)])
    for _ in range(3):
        srv.decode([a, b], srv.append([(a, 1), (b, 1)]))
    c = srv.bm.fork(a)
    srv.tokens[c] = tuple(t.clone() for t in srv.tokens[a])
    for _ in range(2):
        srv.decode([b, c, a], srv.append([(b, 1), (c, 1), (a, 1)]))
    # drafts: five tokens of b, three of c; two of b's are refused
    srv.decode([b, c], srv.append([(b, 5), (c, 3)]), [5, 3])
    srv.bm.shrink(b, srv.bm.seq_len(b) - 2)
    srv.tokens[b] = tuple(t[:-2] for t in srv.tokens[b])
    srv.decode([c, b], srv.append([(c, 1), (b, 4)]), [1, 4])


def test_chunked_prefill_over_unpacked_blocks():
    """A prompt in chunks: each chunk is written in 4 bits, the sequence's blocks are unpacked,
    and prefill_attention over them is the attention over what the cache holds, rounded to the
    type; a decode step over the 4-bit pool follows."""
    H, Hkv, D, B, dt = 12, 2, 128, 16, torch.bfloat16
    n, chunks = 700, [300, 256, 144]
    c = Q4Cache([n], Hkv, D, dt, B, seed=3)
    g = torch.Generator(device=DEV).manual_seed(4)
    q = torch.randn(n, H, D, generator=g, device=DEV).to(dt)
    t = c.tables[0].long()
    nb = t.numel()
    k4, v4 = (torch.full_like(x, 255) for x in (c.k4[0], c.v4[0]))
    k16, v16 = (torch.zeros(nb, Hkv, B, D, dtype=dt, device=DEV) for _ in range(2))
    tables = torch.arange(nb, dtype=torch.int32, device=DEV)[None]
    rows = [x[0][c.slots // B, :, c.slots % B] for x in (c.k, c.v)]
    done, outs = 0, []
    for m in chunks:
        pa.cache_write_q4(rows[0][done:done + m], rows[1][done:done + m], k4, v4, c.slots[done:done + m])
        done += m
        used = -(-done // B)
        pairs = torch.stack([t[:used], torch.arange(used, device=DEV)], 1).contiguous()
        pa.unpack_blocks_q4([k16], [v16], [k4], [v4], pairs)
        outs.append(pa.prefill_attention(q[done - m:done], k16, v16, tables, _i32([0, m]), _i32([done]), m, done, D ** -0.5))
    assert torch.equal(k4[t], c.k4[0][t]) or bool((k4 == c.k4[0]).all())
    out = torch.cat(outs).double()
    for h in range(H):
        k, v = (values(x[:, h // 6])[0].to(dt).double() for x in rows)
        x = q[:, h].double() @ k.T * D ** -0.5
        x.masked_fill_(torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1), float("-inf"))
        want = torch.softmax(x, -1) @ v
        # the weights go to bf16 in two parts: 2^-16 of |v| <= 8, and sums of 700 in 32 bits
        assert float((out[:, h] - want).abs().max()) <= 8 * (2.0 ** -15 + 700 * 2.0 ** -23)
    got = pa.decode_attention_q4(q[-1:], k4, v4, c.tables, c.lens, n, D ** -0.5, out_dtype=dt)
    want, tol = attention(c, q[-1:], [0, 1], D ** -0.5)
    assert bool(((got.double() - want).abs() <= rounded(tol, want, dt)).all())


@pytest.mark.parametrize("B", [16, 64])
def test_copies_and_swaps_of_4_bit_blocks(B):
    c = Q4Cache([10 * B], 3, 128, torch.float16, B, seed=5, layers=2, spare=6)
    before = [x.clone() for x in c.k4 + c.v4]
    free = [int(i) for i in c.spare]
    src = [int(i) for i in c.tables_host[0][:3]]
    pairs = _i64([[s, d] for s, d in zip(src, free)])
    pa.copy_blocks(c.k4, c.v4, pairs)
    for x, y in zip(c.k4 + c.v4, before):
        for s, d in zip(src, free):
            assert torch.equal(x[d], y[s])
        rest = [i for i in range(y.shape[0]) if i not in free[:3]]
        assert torch.equal(x[rest], y[rest])
    host = [torch.zeros_like(x, device="cpu").pin_memory() for x in before]
    out = _i64([[int(b), i] for i, b in enumerate(c.tables_host[0])])
    pa.swap_blocks(host[:2], host[2:], c.k4, c.v4, out)
    torch.cuda.synchronize()
    for h, y in zip(host, before):
        assert torch.equal(h[:10], y[c.tables[0].long()].cpu())
    back = [torch.zeros_like(x) for x in before]
    pa.swap_blocks(back[:2], back[2:], host[:2], host[2:], out.flip(1).contiguous())
    q = torch.randn(1, 6, 128, device=DEV).half()
    want = pa.decode_attention_q4(q, before[1], before[3], c.tables, c.lens, 10 * B, 0.1)
    got = pa.decode_attention_q4(q, back[1], back[3], c.tables, c.lens, 10 * B, 0.1)
    assert torch.equal(got, want)


def test_a_captured_step_replayed():
    """Write and attention captured, replayed with other inputs and lengths in place."""
    lens = [500, 20, 300, 90]
    c = Q4Cache([n + 8 for n in lens], 2, 128, torch.bfloat16, seed=6)
    g = torch.Generator(device=DEV).manual_seed(7)
    rnd = lambda h: torch.randn(4, h, 128, generator=g, device=DEV).bfloat16()  # noqa: E731
    q, k, v, pos = rnd(12), rnd(2), rnd(2), torch.zeros(4, dtype=torch.int64, device=DEV)
    slots, cur = torch.zeros(4, dtype=torch.int64, device=DEV), c.lens.clone()
    rot = pa.Rotary([1.0 / 2 ** (i / 4) for i in range(64)])
    k4, v4 = c.k4[0].clone(), c.v4[0].clone()
    ws = torch.empty(pa.decode_q4_workspace_size(4, 12, 2, 128, 1, 508), dtype=torch.uint8, device=DEV)

    def step():
        qq = pa.rotary_cache_write_q4(q, k, v, pos, rot, k4, v4, slots)
        return pa.decode_attention_q4(qq, k4, v4, c.tables, cur, 508, 0.09, workspace=ws)

    def inputs(i):
        r = torch.Generator(device=DEV).manual_seed(i)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=r, device=DEV))
        n = [m + i for m in lens]
        pos.copy_(_i64([m for m in n]))
        slots.copy_(_i64([int(c.tables_host[s, m // 16]) * 16 + m % 16 for s, m in enumerate(n)]))
        cur.copy_(_i32([m + 1 for m in n]))

    want = []
    for i in range(5):
        inputs(i)
        want.append(step().clone())
    k4.copy_(c.k4[0])
    v4.copy_(c.v4[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = step()
        for i in range(5):
            inputs(i)
            graph.replay()
            st.synchronize()
            assert torch.equal(out, want[i]), i
    torch.cuda.synchronize()


def _write(c, q, kw):
    k4, v4 = c.k4[0].clone(), c.v4[0].clone()
    slots = torch.arange(4, device=DEV)
    key, pos, rot = q[:, :2].contiguous(), torch.arange(4, device=DEV), pa.Rotary([0.1] * 64)
    torch.cuda.synchronize()
    out = pa.rotary_cache_write_q4(q, key, key, pos, rot, k4, v4, slots, **kw)
    pa.cache_write_q4(key, key, k4, v4, slots + 20 if not kw else _AT20, **kw)
    return [out, k4, v4, slots, key, pos]


def _attend(c, q, kw):
    qsl = _QSL
    return [pa.decode_attention_q4(q, c.k4[0], c.v4[0], c.tables, c.lens, 1500, 0.1, **kw),
            pa.decode_attention_q4(q, c.k4[0], c.v4[0], c.tables, c.lens, 1500, 0.1, query_start_loc=qsl,
                                   max_query_len=2, **kw)]


def _unpack(c, q, kw):
    d, e = (torch.zeros(20, 2, 16, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pairs = torch.stack([c.tables[1, :20].long(), torch.arange(20, device=DEV)], 1).contiguous()
    torch.cuda.synchronize()
    pa.unpack_blocks_q4([d], [e], [c.k4[0]], [c.v4[0]], pairs, **kw)
    return [d, e, pairs]


_AT20 = _QSL = None


@pytest.mark.parametrize("call", [_write, _attend, _unpack])
def test_a_call_on_a_stream_of_its_own(call):
    """Calls on another stream, which allocate what they need, while the current stream
    allocates and fills memory: the results are those of calls on the current stream."""
    global _AT20, _QSL
    _AT20, _QSL = torch.arange(20, 24, device=DEV), _i32([0, 2, 3, 3, 4])

    def inputs():
        c = Q4Cache([700, 1500, 33, 900], 2, 128, torch.bfloat16, 16, seed=3)
        return c, torch.randn(4, 12, 128, generator=torch.Generator(device=DEV).manual_seed(4), device=DEV).bfloat16()

    want = [t.clone() for t in call(*inputs(), {})]
    c, q = inputs()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # the call's kernels start some 20 ms later
    got = call(c, q, {"stream": side})
    filled = []
    for nbytes in [1 << i for i in range(8, 25)] * 3:
        filled.append(torch.empty(nbytes, dtype=torch.uint8, device=DEV).fill_(0x7f))
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(bool((t == 0x7f).all()) for t in filled)


def test_two_streams_at_once():
    """Batches of two streams, each with a workspace of its own, in flight together."""
    cs = [Q4Cache([2000 + 500 * i, 300, 77], 2, 128, torch.float16, seed=20 + i) for i in range(2)]
    g = torch.Generator(device=DEV).manual_seed(1)
    q = [torch.randn(3, 8, 128, generator=g, device=DEV).half() for _ in range(2)]
    args = [(q[i], cs[i].k4[0], cs[i].v4[0], cs[i].tables, cs[i].lens, cs[i].max_len, 0.1) for i in range(2)]
    want = [pa.decode_attention_q4(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(pa.decode_attention_q4(*args[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


@pytest.mark.parametrize("H,Hkv,D", [(8, 8, 128), (12, 2, 128), (16, 1, 64), (4, 2, 256)])
def test_a_query_written_by_the_kernel_ahead(H, Hkv, D):
    """The attention starts while the write ahead of it, a long one whose last tokens are the
    queries, still runs: it must see what that writes."""
    S, T, dt = 32, 6000, torch.bfloat16
    g = torch.Generator(device=DEV).manual_seed(9)
    c = Q4Cache([int(n) for n in torch.randint(20, 900, (S,), generator=torch.Generator().manual_seed(3))], Hkv, D, dt,
                seed=2)
    qkv = torch.randn(T, (H + 2 * Hkv) * D, generator=g, device=DEV).to(dt)
    q, k, v = (t.view(T, -1, D) for t in qkv.split([H * D, Hkv * D, Hkv * D], 1))
    spare = [torch.zeros(pa.q4_pool_shape(T // 16 + 1, Hkv, 16, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
    pos, slots = torch.arange(T, device=DEV), torch.arange(T, device=DEV)
    rot = pa.Rotary([0.01 * (i + 1) for i in range(D // 2)])
    out = torch.empty(T, H, D, dtype=dt, device=DEV)
    ws = torch.empty(pa.decode_q4_workspace_size(S, H, Hkv, D, 1, c.max_len), dtype=torch.uint8, device=DEV)

    def attend():
        return pa.decode_attention_q4(out[-S:], c.k4[0], c.v4[0], c.tables, c.lens, c.max_len, 0.1, workspace=ws)

    pa.rotary_cache_write_q4(q, k, v, pos, rot, *spare, slots, query_out=out)
    torch.cuda.synchronize()
    want = attend()
    for _ in range(20):
        out.fill_(float("nan"))
        attend()                                      # (lines of the old query in the caches)
        torch.cuda.synchronize()
        pa.rotary_cache_write_q4(q, k, v, pos, rot, *spare, slots, query_out=out)
        got = attend()
        assert torch.equal(got, want)


@pytest.mark.parametrize("call", ["attend", "attend_cut", "write", "unpack"])
def test_a_16_bit_decode_in_memory_that_the_inputs_had(call):
    """A 16-bit decode step right behind a 4-bit call, whose workspace lies where that call's
    inputs did: its plan writes there as soon as it starts, and the 4-bit call must have read
    them by then."""
    g = torch.Generator(device=DEV).manual_seed(3)
    S, H, Hkv, D, dt = 256, 32, 8, 128, torch.bfloat16
    c = Q4Cache([250 if call != "attend_cut" else 700] * S, Hkv, D, dt, 16, seed=8)
    # the 16-bit step: 64 sequences of 40 pages
    k16, v16 = (torch.randn(64 * 40, 8, 16, 128, generator=g, device=DEV).to(dt) for _ in range(2))
    q16 = torch.randn(64, 8, 128, generator=g, device=DEV).to(dt)
    t16, l16 = _i32(np.arange(64 * 40).reshape(64, 40)), _i32(np.arange(64) * 9 + 1)
    out16 = torch.empty(64, 8, 128, device=DEV)
    nbytes = pa.decode_workspace_size(64, 8, 8, 128, 640)
    mem = torch.empty(max(nbytes, 1 << 24), dtype=torch.uint8, device=DEV)
    want16 = pa.decode_attention(q16, k16, v16, t16, l16, 640, 0.1)

    def step16():
        pa.decode_attention(q16, k16, v16, t16, l16, 640, 0.1, out=out16, workspace=mem)

    if call in ("attend", "attend_cut"):
        data = torch.randn(S, H, D, generator=g, device=DEV).to(dt)
        there = mem[:data.nbytes].view(dt).view(S, H, D)
        out = torch.empty(S, H, D, device=DEV)
        ws = torch.empty(pa.decode_q4_workspace_size(S, H, Hkv, D, 1, c.max_len), dtype=torch.uint8, device=DEV)

        def run(x):
            pa.decode_attention_q4(x, c.k4[0], c.v4[0], c.tables, c.lens, c.max_len, 0.1, out=out, workspace=ws)
            return [out]
    elif call == "write":
        T = 4000
        data = torch.randn(T, Hkv, D, generator=g, device=DEV).to(dt)
        there = mem[:data.nbytes].view(dt).view(T, Hkv, D)
        pools = [torch.zeros(pa.q4_pool_shape(T // 16, Hkv, 16, D), dtype=torch.uint8, device=DEV) for _ in range(2)]
        slots = torch.randperm(T, device=DEV)

        def run(x):
            pa.cache_write_q4(x, x, *pools, slots)
            return pools
    else:
        n = c.tables.numel()
        data = torch.stack([c.tables.flatten().long(), torch.arange(n, device=DEV)], 1).contiguous()
        there = mem[:data.nbytes].view(torch.int64).view(n, 2)
        pools = [torch.zeros(n, Hkv, 16, D, dtype=dt, device=DEV) for _ in range(2)]

        def run(x):
            pa.unpack_blocks_q4(pools[:1], pools[1:], c.k4[:1], c.v4[:1], x)
            return pools
    want = [t.clone() for t in run(data)]
    for _ in range(20):
        there.copy_(data)
        for t in run(data):
            t.zero_()
        got = run(there)
        step16()
        # (bytes: slots that were never written unpack to NaN)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
        assert torch.equal(out16, want16)
