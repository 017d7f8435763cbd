"""Workloads of a KV cache held in 4 bits, with the operators' plain forms.

Three operators that a server with such a cache runs around the paged kernels:

* ``rotary_cache_write_q4`` / ``cache_write_q4``: new keys (rotated on the way, or
  not) and values into the cache, quantised to 4 bits;
* ``decode_attention_q4``: attention of each sequence's newest token, or of its
  newest few (a draft under verification), over the 4-bit cache;
* ``unpack_blocks_q4``: blocks of the 4-bit cache as 16-bit blocks, which
  ``prefill_attention`` and the other 16-bit kernels read.

The format: a token's 64 channels of a head form a group with, in the type of the
keys and values, its least value z and a scale s = (greatest - z) / 15 (computed in
32 bits and rounded to the type); an element x is held as the whole number
n = (x - z) / s, rounded to nearest (ties to even) and cut to 0 .. 15, and is read
as s n + z.

``own = False`` computes each from elementary torch operations in 32 bits (angles
and quantisation in 64); ``own = True`` calls the library.
"""
from __future__ import annotations

import math
import random
from types import SimpleNamespace

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
GROUP = 64  # channels that share a scale and a least value


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _append(name, seqs, new, heads, kv_heads, dim, dtype, block, axes, rot, interleaved, far):
    """axes 0: no rotation."""
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "block": block, "axes": axes,
            "rot": rot, "interleaved": interleaved, "far": far}


def _decode(name, seqs, lo, hi, lens_seed, query, heads, kv_heads, dim, dtype, block):
    """query: the most query tokens of a sequence; with more than one, ragged."""
    return {"name": name, "op": "decode", "seqs": seqs, "lo": lo, "hi": hi,
            "lens_seed": lens_seed, "query": query, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "block": block}


def _unpack(name, layers, pairs, kv_heads, dim, dtype, block):
    return {"name": name, "op": "unpack", "layers": layers, "pairs": pairs,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "block": block}


def listed():
    return [
        # a decode step of the small configuration: four new tokens, and their blocks
        # read back in 16 bits
        _append("append_step_4", 4, 1, 8, 8, 64, "f16", 16, 1, 64, False, 4096),
        # learned or additive positions (no rotation): chunks of eight prompts
        _append("append_plain_8x509", 8, 509, 32, 8, 128, "bf16", 32, 0, 0, False, 1),
        # a prompt with images, three position axes, grouped queries, an odd length
        _append("append_images_4099", 1, 4099, 12, 2, 128, "bf16", 16, 3, 128, False, 32768),
        # a large prefill step at the 40-head shape: sixteen prompts, half of each head
        # rotated, neighbouring pairs, positions far out
        _append("append_prompts_16x1024", 16, 1024, 40, 40, 128, "f16", 32, 1, 64, True, 1 << 20),
        # the small configuration's decode step
        _decode("decode_tiny_4", 4, 1, 128, 1, 1, 8, 8, 64, "f16", 16),
        # the grouped-query serving batch, ragged
        _decode("decode_gqa_64", 64, 512, 4096, 2, 1, 12, 2, 128, "bf16", 16),
        # the 40-head serving batch
        _decode("decode_mha_256", 256, 64, 1024, 3, 1, 40, 40, 128, "f16", 16),
        # drafts under verification: up to five tokens a sequence, 32 heads on 8
        _decode("decode_drafts_32", 32, 1000, 8000, 4, 5, 32, 8, 128, "bf16", 16),
        # two long documents, large blocks
        _decode("decode_long_2", 2, 100000, 131072, 5, 1, 32, 8, 128, "bf16", 64),
        # one layer's blocks of four prompts, ahead of their next chunk
        _unpack("unpack_chunk_500", 1, 500, 8, 64, "f16", 16),
        # every layer of a few preempted sequences
        _unpack("unpack_layers_16x1021", 16, 1021, 8, 128, "bf16", 16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "unpack"])
    dtype = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 128, 256])
    block = rng.choice([16, 32, 64, 128, 256])
    heads, kv = rng.choice([(8, 8), (12, 2), (32, 8), (40, 40), (6, 2), (16, 2), (5, 1)])
    if op == "append":
        seqs = _log_int(rng, 1, 256)
        most = max(1, int(16384 * 120 * 128 / ((heads + 2 * kv) * dim * seqs)))
        new = 1 if rng.random() < 0.3 else _log_int(rng, 1, min(most, 20000))
        axes = rng.choice([0, 1, 1, 2, 3])
        rot = rng.choice([dim, dim // 2, dim // 4]) if axes else 0
        c = _append("", seqs, new, heads, kv, dim, dtype, block, axes, rot,
                    bool(axes) and rng.random() < 0.5, _log_int(rng, 64, 1 << 20))
        while work(c)["bytes"] > 1.1e9:  # (many short prompts in large blocks)
            c["seqs"], c["new"] = -(-c["seqs"] // 2), -(-c["new"] // 2)
    elif op == "decode":
        seqs = _log_int(rng, 1, 256)
        query = rng.choice([1, 1, 1, 2, 4, 6, 9])
        most = int(256 * 1024 * 40 * 128 / (2 * seqs * max(heads, 2 * kv) * dim))
        hi = _log_int(rng, max(2, query), max(12, min(65536, most // (1 if query == 1 else 2))))
        c = _decode("", seqs, rng.randint(max(1, min(hi, query)), hi), hi,
                    rng.randrange(1 << 20), query, heads, kv, dim, dtype, block)
    else:
        layers = _log_int(rng, 1, 32)
        most = max(1, int(16 * 1021 * 8 * 16 * 128 / (layers * kv * block * dim)))
        c = _unpack("", layers, _log_int(rng, 1, most), kv, dim, dtype, block)
    del c["name"]
    return c


def _lens(case):
    """The sequences' lengths: the case's own, whatever the seed."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    lens[r.randrange(len(lens))] = case["hi"]
    return lens


def _queries(case):
    """Query tokens of each sequence."""
    if case["query"] == 1:
        return [1] * case["seqs"]
    r = random.Random(case["lens_seed"] + 1)
    n = [r.randint(1, case["query"]) for _ in range(case["seqs"])]
    n[r.randrange(len(n))] = case["query"]
    return [min(a, b) for a, b in zip(n, _lens(case))]


def _row_bytes(dim):
    """Bytes of a token's key or value of one head: half a byte an element, a scale and a
    least value of 16 bits a group."""
    return dim // 2 + 4 * (dim // GROUP)


def work(case):
    dim, kv, block = case["dim"], case["kv_heads"], case["block"]
    if case["op"] == "append":
        t = case["seqs"] * case["new"]
        rot_rows = t * (case["heads"] + kv) if case["axes"] else 0
        q_rows = t * case["heads"] if case["axes"] else 0
        touched = case["seqs"] * _blocks_each(case) * block
        return {"bytes": 2 * q_rows * dim * 2 + t * 2 * kv * (dim * 2 + _row_bytes(dim))
                + touched * 2 * kv * dim * 2 + t * 8 * (case["axes"] + 1),
                "flops": 3.0 * rot_rows * case["rot"] + 6.0 * t * 2 * kv * dim}
    if case["op"] == "decode":
        lens, new, h = _lens(case), _queries(case), case["heads"]
        n = sum(lens)
        return {"bytes": n * kv * 2 * _row_bytes(dim) + sum(new) * h * dim * 4
                + sum(-(-m // block) for m in lens) * 4,
                "flops": 4.0 * h * dim * sum(a * b for a, b in zip(lens, new))}
    rows = case["layers"] * case["pairs"] * 2 * kv * block
    return {"bytes": rows * (_row_bytes(dim) + 2 * dim), "flops": 2.0 * rows * dim}


def _blocks_each(case):
    """Blocks that a sequence's new tokens touch: they begin in the middle of one."""
    return -(-(_start_in_block(case) + case["new"]) // case["block"])


def _start_in_block(case):
    return (case["new"] * 7 + 3) % case["block"]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, dtype, *shape):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV, dtype=torch.float32).to(dtype)
    return out


def _even(g, dtype, *shape):
    """Evenly spread values of variance 1: bounded, as keys behind a norm are."""
    x = torch.rand(shape, generator=g, device=DEV, dtype=torch.float32)
    return x.sub_(0.5).mul_(math.sqrt(12.0)).to(dtype)


def _tables(seed, lens, block):
    """Block tables [S][max blocks] of a shuffled pool that just holds the sequences; entries
    past a sequence's blocks are -1."""
    nb = [-(-n // block) for n in lens]
    total = sum(nb)
    ids = np.random.default_rng(seed).permutation(total).astype(np.int32)
    tables = np.full((len(lens), max(nb)), -1, np.int32)
    pos = 0
    for s, n in enumerate(nb):
        tables[s, :n] = ids[pos:pos + n]
        pos += n
    return tables, total


def _int32(x):
    return torch.as_tensor(np.ascontiguousarray(x, np.int32)).to(DEV)


def _quantise(x):
    """Codes (uint8), scales and least values of x [..., dim]."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    low, high = g.amin(-1), g.amax(-1)
    scale = ((high.float() - low.float()) / 15.0).to(x.dtype)
    s = scale.double()[..., None]
    n = ((g.double() - low.double()[..., None]) / s.masked_fill(s == 0, 1.0)).round_().clamp_(0, 15)
    return n.to(torch.uint8).view(x.shape), scale, low


def _values(codes, scale, low):
    """What a cache's codes stand for, in 32 bits."""
    g = codes.view(*codes.shape[:-1], scale.shape[-1], GROUP).float()
    return (g * scale.float()[..., None] + low.float()[..., None]).view(codes.shape)


def _cache(x):
    """A 4-bit pool with the values of x [blocks][Hkv][B][dim]: the library's, or its codes,
    scales and least values."""
    if not own:
        codes = torch.empty(x.shape, dtype=torch.uint8, device=DEV)
        scale = torch.empty(*x.shape[:-1], x.shape[-1] // GROUP, dtype=x.dtype, device=DEV)
        low = torch.empty_like(scale)
        step = max(1, (1 << 26) // max(1, x[0].numel()))
        for i in range(0, x.shape[0], step):
            codes[i:i + step], scale[i:i + step], low[i:i + step] = _quantise(x[i:i + step])
        return codes, scale, low
    import paged_kv_cache_pa_gb300 as pa
    blocks, kv, block, dim = x.shape
    pool = torch.zeros(pa.q4_pool_shape(blocks, kv, block, dim), dtype=torch.uint8, device=DEV)
    spare = torch.zeros_like(pool)  # the other side of the call, unused
    rows = x.permute(0, 2, 1, 3).reshape(blocks * block, kv, dim)
    slots = torch.arange(blocks * block, device=DEV)
    pa.cache_write_q4(rows, rows, pool, spare, slots)
    return pool


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dtype, dim, kv, block = DTYPES[case["dtype"]], case["dim"], case["kv_heads"], case["block"]
    st = SimpleNamespace(case=case, op=case["op"], scale=1.0 / math.sqrt(dim))
    if case["op"] == "append":
        h, t = case["heads"], case["seqs"] * case["new"]
        # one projection's output: query, key and value are views of its rows
        if case["axes"]:
            qkv = _even(g, dtype, t, (h + 2 * kv) * dim)
            st.q = qkv[:, :h * dim].view(t, h, dim)
            st.k = qkv[:, h * dim:(h + kv) * dim].view(t, kv, dim)
            st.v = qkv[:, (h + kv) * dim:].view(t, kv, dim)
            st.q_out = torch.empty(t, h, dim, dtype=dtype, device=DEV)
            st.positions = torch.randint(0, case["far"], (case["axes"], t), generator=g,
                                         device=DEV, dtype=torch.int64)
            pairs = case["rot"] // 2
            st.inv_freq = [10000.0 ** (-i / pairs) for i in range(pairs)]
            # the frequencies in order, an equal share to each axis
            st.pair_axis = [min(case["axes"] - 1, i * case["axes"] // pairs) for i in range(pairs)]
            st.inv_freq_t = torch.tensor(st.inv_freq, dtype=torch.float64, device=DEV)
            st.pair_axis_t = torch.tensor(st.pair_axis, dtype=torch.int64, device=DEV)
        else:
            st.k, st.v = _randn(g, dtype, t, kv, dim), _randn(g, dtype, t, kv, dim)
        # the pool holds earlier tokens everywhere; the new ones go to their sequences' blocks
        each = _blocks_each(case)
        blocks = case["seqs"] * each
        ids = np.random.default_rng(seed).permutation(blocks + 4)[:blocks].reshape(case["seqs"], each)
        at = _start_in_block(case) + np.arange(case["new"])
        slots = ids[:, at // block] * block + at % block
        st.slots = torch.as_tensor(slots.reshape(-1).astype(np.int64)).to(DEV)
        st.k_cache = _cache(_even(g, dtype, blocks + 4, kv, block, dim))
        st.v_cache = _cache(_even(g, dtype, blocks + 4, kv, block, dim))
        # the touched blocks, in the sequences' order, to a 16-bit pool of their own
        st.blocks = torch.as_tensor(ids.reshape(-1).astype(np.int64)).to(DEV)
        st.pairs = torch.stack([st.blocks, torch.arange(blocks, device=DEV)], 1).contiguous()
        st.k16 = torch.zeros(blocks, kv, block, dim, dtype=dtype, device=DEV)
        st.v16 = torch.zeros_like(st.k16)
        if own and case["axes"]:
            import paged_kv_cache_pa_gb300 as pa
            st.rotary = pa.Rotary(st.inv_freq, axes=st.pair_axis, interleaved=case["interleaved"])
        return st

    if case["op"] == "unpack":
        layers, pairs = case["layers"], case["pairs"]
        blocks = pairs + pairs // 4 + 1
        st.k_cache = [_cache(_randn(g, dtype, blocks, kv, block, dim)) for _ in range(layers)]
        st.v_cache = [_cache(_randn(g, dtype, blocks, kv, block, dim)) for _ in range(layers)]
        r = np.random.default_rng(seed)
        pairs = np.stack([r.permutation(blocks)[:pairs], r.permutation(pairs)], 1)
        st.pairs = torch.as_tensor(pairs.astype(np.int64)).to(DEV)
        st.k16 = torch.zeros(layers, case["pairs"], kv, block, dim, dtype=dtype, device=DEV)
        st.v16 = torch.zeros_like(st.k16)
        st.k16_list, st.v16_list = list(st.k16), list(st.v16)
        if not own:
            st.k_cache = [torch.stack(x) for x in zip(*st.k_cache)]
            st.v_cache = [torch.stack(x) for x in zip(*st.v_cache)]
        return st

    lens, new, h = _lens(case), _queries(case), case["heads"]
    st.max_len, st.max_new = max(lens), max(new)
    tables, total = _tables(seed, lens, block)
    st.tables, st.lens = _int32(tables), _int32(lens)
    st.k_cache = _cache(_randn(g, dtype, total, kv, block, dim))
    st.v_cache = _cache(_randn(g, dtype, total, kv, block, dim))
    starts = np.concatenate([[0], np.cumsum(new)])
    st.starts = _int32(starts) if case["query"] > 1 else None
    st.q = _randn(g, dtype, int(starts[-1]), h, dim)
    st.out = torch.empty_like(st.q)
    # padded views of the ragged batch, for the plain form
    at = np.minimum(starts[:-1, None] + np.arange(st.max_new)[None], starts[-1] - 1)
    st.rows = torch.as_tensor(at.astype(np.int64)).to(DEV)
    st.row_ok = torch.as_tensor(np.arange(st.max_new)[None] < np.asarray(new)[:, None]).to(DEV)
    st.flat_rows = torch.nonzero(st.row_ok.reshape(-1)).reshape(-1)
    if own:
        import paged_kv_cache_pa_gb300 as pa
        st.workspace = torch.empty(
            max(256, pa.decode_q4_workspace_size(len(lens), h, kv, dim, st.max_new, st.max_len)),
            dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_append(st):
    c = st.case
    got, k = {}, st.k
    if c["axes"]:
        angle = st.positions.double()[st.pair_axis_t] * st.inv_freq_t[:, None]  # [pairs][T]
        cos, sin = angle.cos().float().t()[:, None], angle.sin().float().t()[:, None]

        def turn(x):
            x = x.float()
            r, rest = x[..., :c["rot"]], x[..., c["rot"]:]
            if c["interleaved"]:
                a, b = r[..., 0::2], r[..., 1::2]
                r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
            else:
                a, b = r.chunk(2, -1)
                r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
            return torch.cat([r, rest], -1)

        st.q_out.copy_(turn(st.q))
        got, k = {"query": st.q_out}, turn(st.k).to(st.k.dtype)
    heads = torch.arange(c["kv_heads"], device=DEV)
    at = ((st.slots // c["block"])[:, None], heads[None], (st.slots % c["block"])[:, None])
    for pool, x in ((st.k_cache, k), (st.v_cache, st.v)):
        for part, new in zip(pool, _quantise(x)):
            part[at] = new
    st.k16.copy_(_values(*(part[st.blocks] for part in st.k_cache)))
    st.v16.copy_(_values(*(part[st.blocks] for part in st.v_cache)))
    return {**got, "k": st.k16, "v": st.v16}


def _gather(cache, tables, n):
    """[S][Hkv][n][D] in 32 bits: the first n tokens of every sequence (what is past a
    sequence's own blocks reads block 0 and is masked by the caller)."""
    at = tables.clamp(min=0).long()
    x = _values(*(part[at] for part in cache))                  # [S][blocks][Hkv][B][D]
    s, nb, kv, b, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(s, kv, nb * b, d)[:, :, :n]


def _plain_decode(st):
    c = st.case
    kv, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    s = st.lens.numel()
    # query rows [S][Hkv][new * G][D]
    q = st.q.float()[st.rows].view(s, st.max_new, kv, g, d).transpose(1, 2)
    q = q.reshape(s, kv, st.max_new * g, d)
    k = _gather(st.k_cache, st.tables, st.max_len)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(st.scale).view(s, kv, st.max_new, g, st.max_len)
    del k
    new = st.row_ok.sum(1)
    at = (st.lens - new)[:, None] + torch.arange(st.max_new, device=DEV)      # [S][n]
    j = torch.arange(st.max_len, device=DEV)
    seen = (j <= at[:, :, None]) & st.row_ok[:, :, None]                      # [S][n][L]
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    p = p.div_(p.sum(-1, keepdim=True).clamp(min=1e-30)).view(s, kv, st.max_new * g, st.max_len)
    o = torch.matmul(p, _gather(st.v_cache, st.tables, st.max_len))
    o = o.view(s, kv, st.max_new, g, d).transpose(1, 2).reshape(-1, kv * g, d)
    st.out.copy_(o[st.flat_rows])
    return {"out": st.out}


def _plain_unpack(st):
    src, dst = st.pairs[:, 0], st.pairs[:, 1]
    st.k16[:, dst] = _values(*(part[:, src] for part in st.k_cache)).to(st.k16.dtype)
    st.v16[:, dst] = _values(*(part[:, src] for part in st.v_cache)).to(st.v16.dtype)
    return {"k": st.k16, "v": st.v16}


def run(st):
    if not own:
        return {"append": _plain_append, "decode": _plain_decode, "unpack": _plain_unpack}[st.op](st)
    import paged_kv_cache_pa_gb300 as pa
    c = st.case
    if st.op == "append":
        got = {}
        if c["axes"]:
            pa.rotary_cache_write_q4(st.q, st.k, st.v, st.positions, st.rotary, st.k_cache,
                                     st.v_cache, st.slots, query_out=st.q_out)
            got = {"query": st.q_out}
        else:
            pa.cache_write_q4(st.k, st.v, st.k_cache, st.v_cache, st.slots)
        pa.unpack_blocks_q4([st.k16], [st.v16], [st.k_cache], [st.v_cache], st.pairs)
        return {**got, "k": st.k16, "v": st.v16}
    if st.op == "decode":
        pa.decode_attention_q4(st.q, st.k_cache, st.v_cache, st.tables, st.lens, st.max_len,
                               st.scale, query_start_loc=st.starts, max_query_len=st.max_new,
                               out=st.out, workspace=st.workspace)
        return {"out": st.out}
    pa.unpack_blocks_q4(st.k16_list, st.v16_list, st.k_cache, st.v_cache, st.pairs)
    return {"k": st.k16, "v": st.v16}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _held(x):
    """What x [..., dim] (values of a 16-bit type) is read as after it went through the cache."""
    g = x.double().unflatten(-1, (-1, GROUP))
    z = g.min(-1, keepdim=True).values
    s = ((g.max(-1, keepdim=True).values - z) / 15.0).to(x.dtype).double()
    return torch.where(s > 0, torch.clamp(torch.round((g - z) / s), 0, 15) * s + z, z).flatten(-2)


def _16bit_inputs(case, seed):
    """The values that prepare(case, seed) fills its caches with, drawn again in its order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    dtype, dim, kv, block = DTYPES[case["dtype"]], case["dim"], case["kv_heads"], case["block"]
    if case["op"] == "append":
        t, n = case["seqs"] * case["new"], case["seqs"] * _blocks_each(case) + 4
        if case["axes"]:
            _even(g, dtype, t, (case["heads"] + 2 * kv) * dim)
            torch.randint(0, case["far"], (case["axes"], t), generator=g, device=DEV)
        else:
            _randn(g, dtype, t, kv, dim), _randn(g, dtype, t, kv, dim)
        return _even(g, dtype, n, kv, block, dim), _even(g, dtype, n, kv, block, dim)
    if case["op"] == "unpack":
        n = case["pairs"] + case["pairs"] // 4 + 1
        k = [_randn(g, dtype, n, kv, block, dim) for _ in range(case["layers"])]
        return k, [_randn(g, dtype, n, kv, block, dim) for _ in range(case["layers"])]
    n = sum(-(-m // block) for m in _lens(case))
    return _randn(g, dtype, n, kv, block, dim), _randn(g, dtype, n, kv, block, dim)


def exact(case, seed):
    st = prepare(case, seed)
    op, dim, kv, block = case["op"], case["dim"], case["kv_heads"], case["block"]
    k, v = _16bit_inputs(case, seed)
    if op == "unpack":
        src, dst = st.pairs[:, 0], st.pairs[:, 1]
        back = torch.argsort(dst)
        return {"k": torch.stack([_held(x[src[back]]) for x in k]),
                "v": torch.stack([_held(x[src[back]]) for x in v])}
    if op == "append":
        got, key = {}, st.k
        if case["axes"]:
            half = case["rot"] // 2
            axis = st.positions.double()
            angle = torch.stack([axis[a] * f for a, f in zip(st.pair_axis, st.inv_freq)], 1)
            z = torch.polar(torch.ones_like(angle), angle)[:, None]               # [T][1][pairs]

            def turn(x):
                x = x.double().clone()
                r = x[..., :case["rot"]]
                a, b = (r[..., ::2], r[..., 1::2]) if case["interleaved"] else (r[..., :half], r[..., half:])
                w = torch.complex(a.contiguous(), b.contiguous()) * z
                if case["interleaved"]:
                    x[..., 0:case["rot"]:2], x[..., 1:case["rot"]:2] = w.real, w.imag
                else:
                    x[..., :half], x[..., half:case["rot"]] = w.real, w.imag
                return x

            got, key = {"query": turn(st.q)}, turn(st.k).to(st.k.dtype)
        for name, pool, new in (("k", k, key), ("v", v, st.v)):
            x = pool.transpose(1, 2).reshape(-1, kv, dim)
            x[st.slots] = new
            x = x.view(-1, block, kv, dim)[st.blocks].transpose(1, 2)
            got[name] = _held(x)
        return got
    g, out = case["heads"] // kv, torch.zeros(st.q.shape, dtype=torch.float64, device=DEV)
    row = 0
    for s, (n, m) in enumerate(zip(_lens(case), _queries(case))):
        ids = st.tables[s, :-(-n // block)].long()
        ks, vs = (_held(x[ids]).transpose(0, 1).reshape(kv, -1, dim)[:, :n] for x in (k, v))
        q = st.q[row:row + m].double().view(m, kv, g, dim).permute(1, 2, 0, 3)    # [Hkv][G][m][D]
        x = q @ ks[:, None].transpose(2, 3) * st.scale
        x.masked_fill_(torch.ones(m, n, dtype=torch.bool, device=DEV).triu(n - m + 1), -math.inf)
        o = torch.softmax(x, -1) @ vs[:, None]
        out[row:row + m] = o.permute(2, 0, 1, 3).reshape(m, kv * g, dim)
        row += m
    return {"out": out}
