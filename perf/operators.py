"""Workloads of the bounded-cache operators, with their plain forms.

Four operators that a server with a bounded KV cache runs around the paged
attention kernels:

* ``rotary_cache_write``: rotary positions with one to three axes on the query
  and the key, and the write of key and value into the paged cache;
* ``decode_attention_scored``: one decode step of attention that also adds the
  attention weight every cached token received to its score;
* ``prefill_scores`` (with the log-sum-exp that ``prefill_attention`` gives):
  the same scores for the new tokens of a prompt, a chunk or a window;
* ``evict_tokens``: keeps the first, the last and the highest-scored tokens of
  every sequence, layer and KV head, and compacts the cache.

``own = False`` computes each from elementary torch operations in 32 bits
(angles in 64); ``own = True`` calls the library.
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


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rotary(name, tokens, heads, kv_heads, dim, dtype, axes, rot, interleaved, far, block):
    return {"name": name, "op": "rotary", "tokens": tokens, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "axes": axes, "rot": rot, "interleaved": interleaved,
            "far": far, "block": block}


def _decode(name, seqs, lo, hi, lens_seed, heads, kv_heads, dim, dtype, block):
    return {"name": name, "op": "decode", "seqs": seqs, "lo": lo, "hi": hi,
            "lens_seed": lens_seed, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "block": block}


def _prompt(name, seqs, new, lo, hi, lens_seed, heads, kv_heads, dim, dtype, block, attend):
    return {"name": name, "op": "prompt", "seqs": seqs, "new": new, "lo": lo, "hi": hi,
            "lens_seed": lens_seed, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "block": block, "attend": attend}


def _evict(name, layers, seqs, lo, hi, lens_seed, keep, sink, recent, kv_heads, dim, dtype, block):
    return {"name": name, "op": "evict", "layers": layers, "seqs": seqs, "lo": lo, "hi": hi,
            "lens_seed": lens_seed, "keep": keep, "sink": sink, "recent": recent,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "block": block}


def listed():
    return [
        # a decode step of the small configuration: four new tokens, text positions
        _rotary("rotary_decode_4", 4, 8, 8, 64, "f16", 1, 64, False, 4096, 16),
        # the prompts of a step, images among them: time, height and width axes,
        # the grouped-query head shape, an odd token count
        _rotary("rotary_images_4099", 4099, 12, 2, 128, "bf16", 3, 128, False, 32768, 16),
        # a large prefill step at the 40-head shape, half of each head rotated,
        # neighbouring pairs, positions far out
        _rotary("rotary_prefill_16384", 16384, 40, 40, 128, "f16", 1, 64, True, 1 << 20, 32),
        # the small configuration's decode step
        _decode("decode_tiny_4", 4, 1, 128, 1, 8, 8, 64, "f16", 16),
        # the grouped-query serving batch, ragged
        _decode("decode_gqa_64", 64, 512, 4096, 2, 12, 2, 128, "bf16", 16),
        # the 40-head serving batch
        _decode("decode_mha_256", 256, 64, 1024, 3, 40, 40, 128, "f16", 16),
        # the scores of a prompt from its last 32 queries, long contexts
        _prompt("prompt_window_32", 8, 32, 3000, 16384, 4, 12, 2, 128, "bf16", 16, False),
        # one chunk of a chunked prefill: attention over the cache and the scores
        _prompt("prompt_chunk_509", 4, 509, 509, 2500, 5, 8, 8, 64, "f16", 32, True),
        # whole prompts, every query's weights, 32 query heads on 8 KV heads
        _prompt("prompt_whole_4096", 2, 4096, 4096, 4096, 6, 32, 8, 128, "bf16", 16, False),
        # one layer of a small decode batch that ran over its budget
        _evict("evict_step_8", 1, 8, 900, 1088, 7, 1024, 4, 128, 2, 128, "bf16", 16),
        # all layers of a few prompts, to a quarter or so of their length
        _evict("evict_prompts_16x4", 16, 4, 1500, 8000, 8, 1200, 16, 64, 8, 128, "bf16", 16),
        # one long document, one layer, half of it kept
        _evict("evict_long_1", 1, 1, 131072, 131072, 9, 65000, 4, 512, 8, 64, "f16", 64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "decode", "prompt", "evict"])
    dtype = rng.choice(["f16", "bf16"])
    dim = rng.choice([64, 128])
    block = rng.choice([8, 16, 32, 64, 128])
    heads, kv = rng.choice([(8, 8), (12, 2), (32, 8), (40, 40), (6, 2), (16, 2), (5, 1)])
    lens_seed = rng.randrange(1 << 20)
    if op == "rotary":
        dim = rng.choice([64, 128, 256])
        most = int(16384 * 120 * 128 / ((heads + 2 * kv) * dim))
        rot = rng.choice([dim, dim // 2, dim // 4])
        c = _rotary("", _log_int(rng, 1, min(most, 40000)), heads, kv, dim, dtype,
                    rng.choice([1, 2, 3]), rot, rng.random() < 0.5,
                    _log_int(rng, 64, 1 << 20), block)
    elif op == "decode":
        seqs = _log_int(rng, 1, 192)
        hi = _log_int(rng, 2, max(3, min(32768, int(256 * 1024 * 40 * 128 / (2 * seqs * heads * dim)))))
        c = _decode("", seqs, rng.randint(1, hi), hi, lens_seed, heads, kv, dim, dtype, block)
    elif op == "prompt":
        seqs = _log_int(rng, 1, 12)
        hi = _log_int(rng, 16, 20000)
        most = max(1, int(2 * 4096 * 4096 * 32 * 128 / (2.0 * seqs * hi * heads * dim)))
        new = _log_int(rng, 1, max(1, min(hi, most)))
        c = _prompt("", seqs, new, rng.randint(new, hi), hi, lens_seed, heads, kv, dim, dtype,
                    block, rng.random() < 0.3)
    else:
        layers, seqs = _log_int(rng, 1, 24), _log_int(rng, 1, 24)
        most = max(64, int(16 * 4 * 4500 * 8 * 128 / (layers * seqs * kv * dim)))
        hi = _log_int(rng, 32, min(most, 100000))
        keep = max(1, int(hi * rng.uniform(0.05, 0.95)))
        c = _evict("", layers, seqs, rng.randint(max(1, hi // 4), hi), hi, lens_seed, keep,
                   rng.choice([0, 4, 16]), rng.choice([0, 32, 128]), kv, dim, dtype, block)
    del c["name"]
    return c


def _lens(case):
    """The sequences' lengths: the case's own, whatever the seed."""
    r = random.Random(case["lens_seed"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])]
    lens[r.randrange(len(lens))] = case["hi"]
    return lens


def _new(case):
    """New tokens of each sequence (a prompt shorter than the window is all of it)."""
    return [min(case["new"], n) for n in _lens(case)]


def _kept(case):
    return [min(n, case["keep"]) for n in _lens(case)]


def work(case):
    op, dim = case["op"], case["dim"]
    if op == "rotary":
        t, h, kv = case["tokens"], case["heads"], case["kv_heads"]
        rows = t * (h + 2 * kv) * dim * 2
        return {"bytes": 2 * rows + t * 8 * (case["axes"] + 1),
                "flops": 6.0 * t * (h + kv) * case["rot"] / 2}
    lens = _lens(case)
    kv = case["kv_heads"]
    if op == "decode":
        n, s, h = sum(lens), len(lens), case["heads"]
        return {"bytes": n * kv * dim * 4 + s * h * dim * 4 + n * kv * 8 + n // case["block"] * 4,
                "flops": 4.0 * n * h * dim}
    if op == "prompt":
        h, new = case["heads"], _new(case)
        pairs = sum(m * (n - m) + m * (m + 1) // 2 for n, m in zip(lens, new))
        rows = sum(new) * h
        n = sum(lens)
        if case["attend"]:  # query in, out and lse out; K and V; the scores
            return {"bytes": rows * (dim * 4 + 4) + n * kv * (dim * 4 + 8),
                    "flops": 6.0 * pairs * h * dim}
        return {"bytes": rows * (dim * 2 + 4) + n * kv * (dim * 2 + 8),
                "flops": 2.0 * pairs * h * dim}
    units = case["layers"] * kv
    kept = sum(_kept(case))
    return {"bytes": units * (sum(lens) * 8 + kept * (dim * 2 * 2 * 2 + 4)),
            "flops": float(units * sum(lens))}


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


def _tables(seed, lens, block, spare=0):
    """Block tables [S][max blocks] of a shuffled pool that just holds the sequences, and
    `spare` more blocks; entries past a sequence's blocks are -1."""
    nb = [-(-n // block) for n in lens]
    total = sum(nb) + spare
    ids = np.random.default_rng(seed).permutation(total).astype(np.int32)
    tables = np.full((len(lens), max(nb)), -1, np.int32)
    pos = 0
    for s, n in enumerate(nb):
        tables[s, :n] = ids[pos:pos + n]
        pos += n
    return tables, total, ids[pos:]


def _int32(x):
    return torch.as_tensor(np.ascontiguousarray(x, np.int32)).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dtype, dim, kv, block = DTYPES[case["dtype"]], case["dim"], case["kv_heads"], case["block"]
    st = SimpleNamespace(case=case, op=case["op"], scale=1.0 / math.sqrt(dim))
    if case["op"] == "rotary":
        t, h = case["tokens"], case["heads"]
        # one projection's output: query, key and value are views of its rows
        qkv = _randn(g, dtype, t, (h + 2 * kv) * dim)
        st.q = qkv[:, :h * dim].view(t, h, dim)
        st.k = qkv[:, h * dim:(h + kv) * dim].view(t, kv, dim)
        st.v = qkv[:, (h + kv) * dim:].view(t, kv, dim)
        st.positions = torch.randint(0, case["far"], (case["axes"], t), generator=g, device=DEV,
                                     dtype=torch.int64)
        pairs = case["rot"] // 2
        st.inv_freq = [10000.0 ** (-i / pairs) for i in range(pairs)]
        # the frequencies in order, an equal share to each axis
        st.pair_axis = [min(case["axes"] - 1, i * case["axes"] // pairs) for i in range(pairs)]
        blocks = -(-t // block) + 8
        st.k_cache = _randn(g, dtype, blocks, kv, block, dim)
        st.v_cache = _randn(g, dtype, blocks, kv, block, dim)
        slots = np.random.default_rng(seed).permutation(blocks)[:-(-t // block)]
        slots = (slots[:, None] * block + np.arange(block)[None]).reshape(-1)[:t]
        st.slots = torch.as_tensor(slots.astype(np.int64)).to(DEV)
        st.q_out = torch.empty(t, h, dim, dtype=dtype, device=DEV)
        st.inv_freq_t = torch.tensor(st.inv_freq, dtype=torch.float64, device=DEV)
        st.pair_axis_t = torch.tensor(st.pair_axis, dtype=torch.int64, device=DEV)
        if own:
            import paged_kv_cache_pa_gb300 as pa
            st.rotary = pa.Rotary(st.inv_freq, axes=st.pair_axis,
                                  interleaved=case["interleaved"])
        return st

    lens = _lens(case)
    st.max_len = max(lens)
    if case["op"] == "evict":
        kept = _kept(case)
        n_dst = sum(-(-n // block) for n in kept)
        tables, total, rest = _tables(seed, lens, block, spare=n_dst)
        dst = np.full((len(lens), max(-(-n // block) for n in kept)), -1, np.int32)
        pos = 0
        for s, n in enumerate(kept):
            m = -(-n // block)
            dst[s, :m] = rest[pos:pos + m]
            pos += m
        layers = case["layers"]
        st.k = _randn(g, dtype, layers, total, kv, block, dim)
        st.v = _randn(g, dtype, layers, total, kv, block, dim)
        # accumulated weights: positive, spread over some orders of magnitude
        st.scores = torch.randn(layers, len(lens), kv, st.max_len, generator=g, device=DEV).mul_(2).exp_()
        st.scores_out = torch.zeros_like(st.scores)
        st.tables, st.dst = _int32(tables), _int32(dst)
        st.lens, st.keep = _int32(lens), _int32([case["keep"]] * len(lens))
        st.max_keep = max(kept)
        st.kept = torch.full((layers, len(lens), kv, st.max_keep), -1, dtype=torch.int32, device=DEV)
        st.new_lens = torch.empty(len(lens), dtype=torch.int32, device=DEV)
        st.k_list, st.v_list = list(st.k), list(st.v)
        st.scores_list, st.out_list, st.kept_list = list(st.scores), list(st.scores_out), list(st.kept)
        if own:
            import paged_kv_cache_pa_gb300 as pa
            st.workspace = torch.empty(
                pa.evict_workspace_size(layers, len(lens), kv, st.max_len, st.max_keep),
                dtype=torch.uint8, device=DEV)
        return st

    h = case["heads"]
    tables, total, _ = _tables(seed, lens, block)
    st.tables, st.lens = _int32(tables), _int32(lens)
    st.k_cache = _randn(g, dtype, total, kv, block, dim)
    st.v_cache = _randn(g, dtype, total, kv, block, dim)
    # scores of earlier steps
    st.scores = torch.rand(len(lens), kv, st.max_len, generator=g, device=DEV)
    if case["op"] == "decode":
        st.q = _randn(g, dtype, len(lens), h, dim)
        st.out = torch.empty_like(st.q)
        if own:
            import paged_kv_cache_pa_gb300 as pa
            st.workspace = torch.empty(
                pa.decode_scored_workspace_size(len(lens), h, kv, dim, st.max_len),
                dtype=torch.uint8, device=DEV)
        return st

    new = _new(case)
    st.max_new = max(new)
    st.new_host, st.lens_host = new, lens
    starts = np.concatenate([[0], np.cumsum(new)])
    st.starts = _int32(starts)
    st.q = _randn(g, dtype, int(starts[-1]), h, dim)
    st.out = torch.empty_like(st.q)
    st.lse = torch.empty(int(starts[-1]), h, dtype=torch.float32, device=DEV)
    # padded views of the ragged batch, for the plain form
    at = np.minimum(starts[:-1, None] + np.arange(st.max_new)[None], starts[-1] - 1)
    st.rows = torch.as_tensor(at.astype(np.int64)).to(DEV)
    st.row_ok = torch.as_tensor(np.arange(st.max_new)[None] < np.asarray(new)[:, None]).to(DEV)
    st.flat_rows = torch.nonzero(st.row_ok.reshape(-1)).reshape(-1)
    if not case["attend"]:  # the attention before gave it
        st.lse.copy_(_lse(st)[1])
    if own:
        import paged_kv_cache_pa_gb300 as pa
        st.attend_ws = torch.empty(
            max(256, pa.prefill_workspace_size(len(lens), h, kv, dim, st.max_new)),
            dtype=torch.uint8, device=DEV)
        st.workspace = torch.empty(
            pa.prefill_scores_workspace_size(len(lens), h, kv, dim, st.max_new, st.max_len),
            dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _gather(cache, tables, n):
    """[S][Hkv][n][D] in 32 bits: the first n tokens of every sequence (what is past a
    sequence's own blocks reads block 0 and is masked by the caller)."""
    x = cache[tables.clamp(min=0).long()]                       # [S][blocks][Hkv][B][D]
    s, nb, kv, b, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(s, kv, nb * b, d)[:, :, :n].float()


def _causal_logits(st):
    """Scaled scores [S][Hkv][G][n][L] of a ragged batch of new tokens, -inf where masked."""
    c = st.case
    kv, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    s = st.lens.numel()
    k = _gather(st.k_cache, st.tables, st.max_len)
    q = st.q.float()[st.rows].view(s, st.max_new, kv, g, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(s, kv, g * st.max_new, d), k.transpose(2, 3)).mul_(st.scale)
    x = x.view(s, kv, g, st.max_new, st.max_len)
    new = st.row_ok.sum(1)
    at = (st.lens - new)[:, None] + torch.arange(st.max_new, device=DEV)      # [S][n]
    j = torch.arange(st.max_len, device=DEV)
    seen = (j <= at[:, :, None]) & st.row_ok[:, :, None]                      # [S][n][L]
    return x.masked_fill_(~seen[:, None, None], -math.inf)


def _lse(st):
    """The causal scores and their log-sum-exp, [T][H] in the batch's row order."""
    x = _causal_logits(st)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    lse = m.squeeze(-1) + (x - m).exp_().sum(-1).log_()                       # [S][Hkv][G][n]
    h = st.case["heads"]
    flat = lse.permute(0, 3, 1, 2).reshape(-1, h)
    return x, flat[st.flat_rows]


def _plain_rotary(st):
    c = st.case
    pos = st.positions.double()[st.pair_axis_t]                               # [pairs][T]
    angle = pos * st.inv_freq_t[:, None]
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

    blk, off = st.slots // c["block"], st.slots % c["block"]
    heads = torch.arange(c["kv_heads"], device=DEV)
    at = (blk[:, None], heads[None], off[:, None])
    st.k_cache[at] = turn(st.k).to(st.k_cache.dtype)
    st.v_cache[at] = st.v
    return {"query": turn(st.q).to(st.q.dtype), "k_cache": st.k_cache, "v_cache": st.v_cache}


def _plain_decode(st):
    c = st.case
    kv, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    s = st.lens.numel()
    live = torch.arange(st.max_len, device=DEV) < st.lens[:, None]            # [S][L]
    q = st.q.float().view(s, kv, g, d)
    x = torch.matmul(q, _gather(st.k_cache, st.tables, st.max_len).transpose(2, 3)).mul_(st.scale)
    x.masked_fill_(~live[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp_()
    p = p / p.sum(-1, keepdim=True)
    v = _gather(st.v_cache, st.tables, st.max_len).masked_fill_(~live[:, None, :, None], 0.0)
    st.out.copy_(torch.matmul(p, v).view(s, kv * g, d))
    st.scores += p.sum(2)
    return {"out": st.out, "scores": st.scores}


def _plain_prompt(st):
    c = st.case
    kv, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    s = st.lens.numel()
    got = {}
    if c["attend"]:
        x, lse = _lse(st)
        st.lse.copy_(lse)
    else:
        x = _causal_logits(st)
    lse = st.lse[st.rows].view(s, st.max_new, kv, g).permute(0, 2, 3, 1)      # [S][Hkv][G][n]
    p = x.sub_(lse[..., None]).exp_()
    if c["attend"]:
        v = _gather(st.v_cache, st.tables, st.max_len)
        o = torch.matmul(p.view(s, kv, g * st.max_new, st.max_len), v)
        o = o.view(s, kv, g, st.max_new, d).permute(0, 3, 1, 2, 4).reshape(-1, kv * g, d)
        st.out.copy_(o[st.flat_rows])
        got = {"out": st.out, "lse": st.lse}
    st.scores += p.sum((2, 3))
    return {**got, "scores": st.scores}


def _plain_evict(st):
    c = st.case
    block, n_max = c["block"], st.max_len
    j = torch.arange(n_max, device=DEV)
    lens = st.lens.long()[:, None]                                            # [S][1]
    new = torch.minimum(lens, st.keep.long()[:, None])
    recent = torch.clamp(new, max=c["recent"])
    sink = torch.minimum(new - recent, torch.full_like(new, c["sink"]))
    fixed = (j < sink) | ((j >= lens - recent) & (j < lens))                  # [S][L]
    middle = (j < lens) & ~fixed
    # the highest scores of the middle first, equal ones by index
    ranked = st.scores.masked_fill(~middle[None, :, None], -math.inf)
    order = ranked.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order))
    keep = fixed[None, :, None] | (middle[None, :, None] & (rank < (new - recent - sink)[None, :, None]))
    idx = torch.sort((~keep).to(torch.uint8), dim=-1, stable=True).indices[..., :st.max_keep]
    i = torch.arange(st.max_keep, device=DEV)
    live = (i < new)[None, :, None]                                           # [1][S][1][K]
    torch.where(live, idx.int(), st.kept, out=st.kept)
    moved = st.scores.gather(-1, idx) * live
    past = (j[st.max_keep:] < lens)[None, :, None]
    st.scores_out[..., :st.max_keep] = torch.where(
        live | (i < lens)[None, :, None], moved, st.scores_out[..., :st.max_keep])
    st.scores_out[..., st.max_keep:].masked_fill_(past, 0.0)
    st.new_lens.copy_(new[:, 0])
    # rows past a sequence's end repeat its first row
    idx = torch.where(live, idx, idx[..., :1])
    to = torch.where(i < new, i, 0)                                           # [S][K]
    s = torch.arange(lens.numel(), device=DEV)[:, None]
    head = torch.arange(c["kv_heads"], device=DEV)[None, :, None]
    layer = torch.arange(c["layers"], device=DEV)[:, None, None, None]
    src_blk = st.tables.long()[s[:, :, None], idx // block]                   # [layers][S][Hkv][K]
    dst_blk = st.dst.long()[s, to // block][:, None]                          # [S][1][K]
    dst = (layer, dst_blk[None], head[None], (to % block)[None, :, None])
    src = (layer, src_blk, head[None], idx % block)
    st.k[dst] = st.k[src]
    st.v[dst] = st.v[src]
    return {"k": st.k, "v": st.v, "scores": st.scores_out, "kept": st.kept, "lens": st.new_lens}


def run(st):
    if not own:
        return {"rotary": _plain_rotary, "decode": _plain_decode, "prompt": _plain_prompt,
                "evict": _plain_evict}[st.op](st)
    import paged_kv_cache_pa_gb300 as pa
    c = st.case
    if st.op == "rotary":
        pa.rotary_cache_write(st.q, st.k, st.v, st.positions, st.rotary, st.k_cache, st.v_cache,
                              st.slots, query_out=st.q_out)
        return {"query": st.q_out, "k_cache": st.k_cache, "v_cache": st.v_cache}
    if st.op == "decode":
        pa.decode_attention_scored(st.q, st.k_cache, st.v_cache, st.tables, st.lens, st.max_len,
                                   st.scale, st.scores, out=st.out, workspace=st.workspace)
        return {"out": st.out, "scores": st.scores}
    if st.op == "prompt":
        got = {}
        if c["attend"]:
            pa.prefill_attention(st.q, st.k_cache, st.v_cache, st.tables, st.starts, st.lens,
                                 st.max_new, st.max_len, st.scale, out=st.out,
                                 workspace=st.attend_ws, lse=st.lse)
            got = {"out": st.out, "lse": st.lse}
        pa.prefill_scores(st.q, st.lse, st.k_cache, st.tables, st.starts, st.lens, st.max_new,
                          st.max_len, st.scale, st.scores, workspace=st.workspace)
        return {**got, "scores": st.scores}
    pa.evict_tokens(st.k_list, st.v_list, st.scores_list, st.tables, st.lens, st.keep, st.max_len,
                    st.max_keep, num_sink=c["sink"], num_recent=c["recent"],
                    dst_block_tables=st.dst, scores_out=st.out_list, kept=st.kept_list,
                    new_lens=st.new_lens, workspace=st.workspace)
    return {"k": st.k, "v": st.v, "scores": st.scores_out, "kept": st.kept, "lens": st.new_lens}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, one sequence at a time
# ---------------------------------------------------------------------------
def _sequence(cache, table, n, head):
    block = cache.shape[2]
    t = torch.arange(n, device=DEV)
    return cache[table.long()[t // block], head, t % block].double()


def exact(case, seed):
    st = prepare(case, seed)
    op, dim, kv = case["op"], case["dim"], case["kv_heads"]
    if op == "rotary":
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

        kc = st.k_cache.double().permute(0, 2, 1, 3).reshape(-1, kv, dim)
        vc = st.v_cache.double().permute(0, 2, 1, 3).reshape(-1, kv, dim)
        kc[st.slots], vc[st.slots] = turn(st.k), st.v.double()
        back = lambda x: x.view(-1, case["block"], kv, dim).permute(0, 2, 1, 3).contiguous()  # noqa: E731
        return {"query": turn(st.q), "k_cache": back(kc), "v_cache": back(vc)}
    lens = _lens(case)
    if op == "evict":
        return _exact_evict(case, st, lens)
    g = case["heads"] // kv
    scores = st.scores.double()
    if op == "decode":
        out = torch.zeros(st.q.shape, dtype=torch.float64, device=DEV)
        for s, n in enumerate(lens):
            for h in range(kv):
                q = st.q[s, h * g:(h + 1) * g].double()
                p = torch.softmax(q @ _sequence(st.k_cache, st.tables[s], n, h).T * st.scale, -1)
                out[s, h * g:(h + 1) * g] = p @ _sequence(st.v_cache, st.tables[s], n, h)
                scores[s, h, :n] += p.sum(0)
        return {"out": out, "scores": scores}
    out = torch.zeros(st.q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(st.lse.shape, dtype=torch.float64, device=DEV)
    row = 0
    for s, (n, m) in enumerate(zip(lens, _new(case))):
        mask = torch.ones(m, n, dtype=torch.bool, device=DEV).triu(n - m + 1)
        for h in range(kv):
            k = _sequence(st.k_cache, st.tables[s], n, h)
            for qh in range(h * g, (h + 1) * g):
                x = (st.q[row:row + m, qh].double() @ k.T * st.scale).masked_fill_(mask, -math.inf)
                if case["attend"]:
                    p = torch.softmax(x, -1)
                    lse[row:row + m, qh] = torch.logsumexp(x, -1)
                    out[row:row + m, qh] = p @ _sequence(st.v_cache, st.tables[s], n, h)
                else:
                    p = torch.exp(x - st.lse[row:row + m, qh].double()[:, None])
                scores[s, h, :n] += p.sum(0)
        row += m
    return {"out": out, "lse": lse, "scores": scores} if case["attend"] else {"scores": scores}


def _exact_evict(case, st, lens):
    block = case["block"]
    tables, dst = st.tables.cpu().numpy(), st.dst.cpu().numpy()
    scores, out = st.scores.cpu().numpy(), st.scores_out.double().cpu().numpy()
    kept = st.kept.cpu().numpy()
    k, v = st.k.double(), st.v.double()
    for layer in range(case["layers"]):
        for s, n in enumerate(lens):
            new = min(n, case["keep"])
            recent = min(case["recent"], new)
            sink = min(case["sink"], new - recent)
            for h in range(case["kv_heads"]):
                sc = scores[layer, s, h, :n]
                mid = np.arange(sink, n - recent)
                best = mid[np.lexsort((mid, -sc[mid].astype(np.float64)))][:new - recent - sink]
                idx = np.sort(np.concatenate([np.arange(sink), best, np.arange(n - recent, n)]))
                out[layer, s, h, :n] = 0.0
                out[layer, s, h, :new] = sc[idx]
                kept[layer, s, h, :new] = idx
                to = np.arange(new)
                a = (torch.as_tensor(tables[s, idx // block]).long().to(DEV),
                     torch.as_tensor(idx % block).to(DEV))
                b = (torch.as_tensor(dst[s, to // block]).long().to(DEV),
                     torch.as_tensor(to % block).to(DEV))
                k[layer, b[0], h, b[1]] = k[layer, a[0], h, a[1]]
                v[layer, b[0], h, b[1]] = v[layer, a[0], h, a[1]]
    new = [min(n, case["keep"]) for n in lens]
    return {"k": k, "v": v, "scores": torch.as_tensor(out), "kept": torch.as_tensor(kept),
            "lens": torch.as_tensor(np.asarray(new, np.int32))}
