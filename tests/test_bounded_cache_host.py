"""Refusals of the bounded-cache entry points, all decided on the host before
anything is enqueued (no GPU needed)."""
import ctypes
import math

import pytest

import paged_kv_cache_pa_gb300 as pa

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = 0, 1, 2, 3, 4
P = 1 << 20  # a 256-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_pa_gb300.build import build
    build()
    return pa.load_library()


def _init(lib, n, freqs=None, axes=None, inter=0, scale=1.0):
    r = pa._RotaryStruct()
    f = (ctypes.c_double * max(n, 1))(*(freqs or [1.0] * n))
    a = None if axes is None else ctypes.cast((ctypes.c_int32 * n)(*axes), ctypes.c_void_p)
    st = lib.pa_rotary_init(ctypes.addressof(r), ctypes.cast(f, ctypes.c_void_p), a, n, inter, scale)
    return st, r


def test_rotary_init(lib):
    st, r = _init(lib, 8, freqs=[2 * math.pi * t for t in (0.5, 0.25, -0.25, 1.0, 3.75, 0.0, 2 ** -20, -0.5)],
                  axes=[0, 1, 2, 0, 1, 2, 3, 0])
    assert st == OK and r.rotary_dim == 16 and r.num_axes == 4
    for got, want in zip(r.turns, (0.5, 0.25, 0.75, 0.0, 0.75, 0.0, 2 ** -20, 0.5)):
        # modulo one turn, to the 53 bits of the frequency
        d = (got - int(want * 2 ** 64)) % 2 ** 64
        assert min(d, 2 ** 64 - d) <= 2 ** 15
    assert list(r.axis[:8]) == [0, 1, 2, 0, 1, 2, 3, 0]


@pytest.mark.parametrize("n,kw,want", [
    (0, {}, UNSUPPORTED), (7, {}, UNSUPPORTED), (12, {}, UNSUPPORTED), (136, {}, UNSUPPORTED),
    (8, {"freqs": [math.nan] * 8}, INVALID), (8, {"freqs": [math.inf] * 8}, INVALID),
    (8, {"axes": [0] * 7 + [8]}, INVALID), (8, {"axes": [-1] + [0] * 7}, INVALID),
    (8, {"scale": math.nan}, INVALID), (128, {}, OK)])
def test_rotary_init_refusals(lib, n, kw, want):
    assert _init(lib, n, **kw)[0] == want


def test_rotary_class_refuses():
    with pytest.raises(ValueError):
        pa.Rotary([1.0] * 8, axes=[0] * 7)
    with pytest.raises(pa.PaError):
        pa.Rotary([1.0] * 9)
    r = pa.Rotary([1.0] * 32, axes=[0] * 16 + [2] * 16)
    assert r.rotary_dim == 64 and r.num_axes == 3


def _rot_call(lib, **kw):
    _, r = _init(lib, kw.pop("pairs", 32))
    for name, v in kw.pop("rot", {}).items():
        setattr(r, name, v)
    a = dict(qo=P, qos=512, q=P, qs=512, k=P, ks=128, v=P, vs=128, pos=P, kc=P, vc=P, slots=P, T=4,
             nb=4, bs=16, H=8, Hkv=2, D=64, dt=0)
    a.update(kw)
    return lib.pa_rotary_cache_write(a["qo"], a["qos"], a["q"], a["qs"], a["k"], a["ks"], a["v"],
                                     a["vs"], a["pos"], a.get("r", ctypes.addressof(r)), a["kc"],
                                     a["vc"], a["slots"], a["T"], a["nb"], a["bs"], a["H"], a["Hkv"],
                                     a["D"], a["dt"], None, None)


@pytest.mark.parametrize("kw,want", [
    ({"T": 0}, OK), ({"T": 0, "q": None}, OK), ({"T": -1}, INVALID), ({"nb": 0}, INVALID),
    ({"H": 0}, INVALID), ({"Hkv": 0}, INVALID), ({"dt": 2}, INVALID), ({"dt": 9}, INVALID),
    ({"bs": 12}, UNSUPPORTED), ({"bs": 512}, UNSUPPORTED), ({"bs": 4}, UNSUPPORTED),
    ({"D": 96}, UNSUPPORTED), ({"D": 64, "pairs": 64}, INVALID), ({"r": None}, INVALID),
    ({"rot": {"num_axes": 0}}, INVALID), ({"rot": {"num_axes": 9}}, INVALID),
    ({"rot": {"rotary_dim": 24}}, INVALID), ({"qs": 504}, INVALID), ({"qs": 513}, INVALID),
    ({"qos": 508}, INVALID), ({"ks": 120}, INVALID), ({"vs": 129}, INVALID), ({"q": None}, INVALID),
    ({"qo": None}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID), ({"pos": None}, INVALID),
    ({"kc": None}, INVALID), ({"vc": None}, INVALID), ({"slots": None}, INVALID),
    ({"q": P + 8}, INVALID), ({"k": P + 2}, INVALID), ({"vc": P + 4}, INVALID)])
def test_rotary_cache_write_refusals(lib, kw, want):
    assert _rot_call(lib, **kw) == want


def test_rotary_axis_past_the_rows_is_refused(lib):
    _, r = _init(lib, 32)
    r.axis[5] = 1
    assert lib.pa_rotary_cache_write(P, 512, P, 512, P, 128, P, 128, P, ctypes.addressof(r), P, P, P,
                                     4, 4, 16, 8, 2, 64, 0, None, None) == INVALID


def _scored(lib, **kw):
    a = dict(out=P, odt=2, q=P, k=P, v=P, tab=P, mb=8, lens=P, L=100, S=2, H=8, Hkv=2, D=64, nb=16,
             bs=16, dt=0, sc=P, stride=100, ws=P, wb=1 << 30)
    a.update(kw)
    return lib.pa_decode_attention_scored(a["out"], a["odt"], a["q"], a["k"], a["v"], a["tab"], a["mb"],
                                          a["lens"], a["L"], a["S"], a["H"], a["Hkv"], a["D"], a["nb"],
                                          a["bs"], 0.1, a["dt"], a["sc"], a["stride"], a["ws"], a["wb"],
                                          None, None)


@pytest.mark.parametrize("kw,want", [
    ({"S": 0}, OK), ({"S": 0, "sc": None}, OK), ({"S": -1}, INVALID), ({"stride": 99}, INVALID),
    ({"sc": None}, INVALID), ({"sc": P + 2}, INVALID), ({"H": 9}, INVALID), ({"H": 18}, UNSUPPORTED),
    ({"D": 80}, UNSUPPORTED), ({"bs": 24}, UNSUPPORTED), ({"dt": 2}, INVALID), ({"odt": 1}, INVALID),
    ({"L": 129, "stride": 129}, INVALID), ({"ws": None}, INVALID), ({"ws": P + 16}, WORKSPACE),
    ({"wb": 100}, WORKSPACE), ({"q": P + 8}, INVALID), ({"out": None}, INVALID), ({"tab": None}, INVALID),
    ({"lens": None}, INVALID), ({"nb": 0}, INVALID), ({"mb": 0}, INVALID)])
def test_decode_scored_refusals(lib, kw, want):
    assert _scored(lib, **kw) == want


def test_decode_scored_workspace_size(lib):
    a = pa.decode_scored_workspace_size(64, 12, 2, 128, 4096)
    assert a >= 64 * 12 * 4096 * 4
    assert pa.decode_scored_workspace_size(64, 12, 2, 128, 8192) > a
    assert pa.decode_scored_workspace_size(-1, 12, 2, 128, 10) == 0
    assert _scored(lib, wb=pa.decode_scored_workspace_size(2, 8, 2, 64, 100) - 1) == WORKSPACE


def _pscores(lib, **kw):
    a = dict(q=P, lse=P, k=P, tab=P, mb=8, qsl=P, lens=P, mq=50, L=100, S=2, T=60, H=8, Hkv=2, D=64, nb=16,
             bs=16, dt=0, sc=P, stride=100, ws=P, wb=1 << 30)
    a.update(kw)
    return lib.pa_prefill_scores(a["q"], a["lse"], a["k"], a["tab"], a["mb"], a["qsl"], a["lens"], a["mq"],
                                 a["L"], a["S"], a["T"], a["H"], a["Hkv"], a["D"], a["nb"], a["bs"], 0.1,
                                 a["dt"], a["sc"], a["stride"], a["ws"], a["wb"], None, None)


@pytest.mark.parametrize("kw,want", [
    ({"S": 0}, OK), ({"T": 0}, OK), ({"mq": 0}, OK), ({"S": -1}, INVALID), ({"T": -1}, INVALID),
    ({"mq": -1}, INVALID), ({"L": -1}, INVALID), ({"nb": 0}, INVALID), ({"mb": 0}, INVALID),
    ({"H": 9}, INVALID), ({"D": 256}, UNSUPPORTED), ({"D": 32}, UNSUPPORTED), ({"bs": 4}, UNSUPPORTED),
    ({"dt": 2}, INVALID), ({"L": 129, "stride": 129}, INVALID), ({"stride": 99}, INVALID), ({"q": None}, INVALID),
    ({"lse": None}, INVALID), ({"k": None}, INVALID), ({"tab": None}, INVALID), ({"qsl": None}, INVALID),
    ({"lens": None}, INVALID), ({"sc": None}, INVALID), ({"ws": None}, INVALID), ({"q": P + 8}, INVALID),
    ({"lse": P + 1}, INVALID), ({"sc": P + 2}, INVALID), ({"k": P + 4}, INVALID), ({"ws": P + 64}, WORKSPACE),
    ({"wb": 0}, WORKSPACE), ({"S": 70000}, UNSUPPORTED)])
def test_prefill_scores_refusals(lib, kw, want):
    assert _pscores(lib, **kw) == want


def test_prefill_lse_refuses_a_misaligned_pointer(lib):
    st = lib.pa_prefill_attention_lse(P, 2, P, P, P, P, 8, P, P, 50, 100, 2, 60, 8, 2, 64, 16, 16, 0.1, 0,
                                      P + 2, P, 1 << 30, None, None)
    assert st == INVALID
    assert pa.prefill_scores_workspace_size(2, 8, 2, 96, 50, 100) == 0
    assert pa.prefill_scores_workspace_size(2, 8, 3, 64, 50, 100) == 0


def _ptrs(*ps):
    return ctypes.cast((ctypes.c_void_p * len(ps))(*ps), ctypes.c_void_p)


def _evict(lib, **kw):
    a = dict(k=_ptrs(P, P), v=_ptrs(P, P), layers=2, sc=_ptrs(P, P), ss=100, so=None, sos=0, kept=None, ks=0, tab=P,
             mb=8, dst=None, dmb=0, lens=P, keep=P, new=2 * P, L=100, K=50, sink=4, recent=4, S=2, nb=16, bs=16,
             Hkv=2, D=64, dt=0, ws=P, wb=1 << 30)
    a.update(kw)
    return lib.pa_evict_tokens(a["k"], a["v"], a["layers"], a["sc"], a["ss"], a["so"], a["sos"], a["kept"], a["ks"],
                               a["tab"], a["mb"], a["dst"], a["dmb"], a["lens"], a["keep"], a["new"], a["L"], a["K"],
                               a["sink"], a["recent"], a["S"], a["nb"], a["bs"], a["Hkv"], a["D"], a["dt"], a["ws"],
                               a["wb"], None, None)


@pytest.mark.parametrize("kw,want", [
    ({"S": 0}, OK), ({"S": -1}, INVALID), ({"layers": 0}, INVALID), ({"layers": 129}, UNSUPPORTED),
    ({"L": -1}, INVALID), ({"K": -1}, INVALID), ({"K": 101}, INVALID), ({"sink": -1}, INVALID),
    ({"recent": -1}, INVALID), ({"nb": 0}, INVALID), ({"mb": 0}, INVALID), ({"Hkv": 0}, INVALID),
    ({"bs": 48}, UNSUPPORTED), ({"D": 32}, UNSUPPORTED), ({"dt": 2}, INVALID), ({"L": 129, "ss": 129}, INVALID),
    ({"ss": 99}, INVALID), ({"so": _ptrs(P, P), "sos": 99}, INVALID), ({"kept": _ptrs(P, P), "ks": 49}, INVALID),
    ({"dst": P, "dmb": 3}, INVALID), ({"dst": P, "dmb": 0}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID),
    ({"sc": None}, INVALID), ({"tab": None}, INVALID), ({"lens": None}, INVALID), ({"keep": None}, INVALID),
    ({"new": None}, INVALID), ({"new": P}, INVALID), ({"k": _ptrs(P, None)}, INVALID), ({"v": _ptrs(P, P + 8)}, INVALID),
    ({"sc": _ptrs(P, P + 2)}, INVALID), ({"so": _ptrs(P, None), "sos": 100}, INVALID),
    ({"kept": _ptrs(P, P + 1), "ks": 50}, INVALID), ({"ws": P + 128}, WORKSPACE), ({"ws": None}, INVALID),
    ({"wb": 100}, WORKSPACE), ({"S": 65536}, UNSUPPORTED), ({"Hkv": 65536}, UNSUPPORTED),
    ({"L": 393217, "ss": 393217, "mb": 1 << 20}, UNSUPPORTED),
    ({"S": 65535, "Hkv": 65535, "L": 100, "K": 50}, UNSUPPORTED)])
def test_evict_refusals(lib, kw, want):
    assert _evict(lib, **kw) == want


def test_evict_workspace_size(lib):
    a = pa.evict_workspace_size(4, 8, 2, 1000, 500)
    assert a >= 4 * 8 * 2 * 500 * 4
    assert pa.evict_workspace_size(0, 8, 2, 1000, 500) == 0
    assert pa.evict_workspace_size(129, 8, 2, 1000, 500) == 0
    assert pa.evict_workspace_size(4, 8, 2, 1000, -1) == 0


def test_manager_make_private_and_shrink():
    from paged_kv_cache_pa_gb300.manager import BlockManager, NoFreeBlocks
    bm = BlockManager(10, 0, 16)
    a = bm.new_sequence()
    bm.append(a, 70)                       # 5 blocks, the last with 6 tokens
    b = bm.fork(a)
    bm.make_private(b, 33)                 # its first three blocks
    assert bm.table(a) == [0, 1, 2, 3, 4] and bm.table(b) == [5, 6, 7, 3, 4]
    assert bm.take_copies().tolist() == [[0, 5], [1, 6], [2, 7]]
    bm.make_private(a, 33)                 # already its own
    assert bm.take_copies().tolist() == [] and bm.table(a) == [0, 1, 2, 3, 4]
    bm.shrink(b, 33)
    assert bm.table(b) == [5, 6, 7] and bm.seq_len(b) == 33 and bm.num_free_gpu == 2
    assert bm.refcount(3) == 1 and bm.refcount(4) == 1
    assert bm.append(b, 2).tolist() == [7 * 16 + 1, 7 * 16 + 2]   # goes on behind the kept tokens
    bm.shrink(a, 70)
    assert bm.seq_len(a) == 70
    bm.shrink(a, 0)
    assert bm.table(a) == [] and bm.num_free_gpu == 7
    c = bm.fork(b)
    assert bm.append(a, 7 * 16).size == 112 and bm.num_free_gpu == 0
    with pytest.raises(NoFreeBlocks):
        bm.make_private(c, 1)
    assert bm.table(c) == bm.table(b) and bm.take_copies().tolist() == []
    for bad in (-1, 36):
        with pytest.raises(pa.PaError):
            bm.shrink(b, bad)
        with pytest.raises(pa.PaError):
            bm.make_private(b, bad)
    with pytest.raises(pa.PaError):
        bm.shrink(99, 0)
    bm.close()


def test_manager_swapped_out_sequences_are_refused():
    from paged_kv_cache_pa_gb300.manager import BlockManager
    bm = BlockManager(4, 4, 16)
    a = bm.new_sequence()
    bm.append(a, 20)
    bm.swap_out([a])
    for f in (bm.shrink, bm.make_private):
        with pytest.raises(pa.PaError):
            f(a, 1)
    bm.close()


def test_rotary_frequencies_are_right_to_64_bits(lib):
    """A position far out multiplies what the frequency is off by: rounded once, to 2^-65 turns."""
    import random
    from cachelib import turn_fraction
    rng = random.Random(3)
    freqs = [10000.0 ** (-i / 64) for i in range(64)] + [1e6 ** (-i / 32) for i in range(32)]
    freqs += [math.ldexp(rng.uniform(0.5, 1), e) for e in range(64, -80, -7)]
    freqs += [math.pi, 2 * math.pi, 0.0, -0.0, 5e-324, 1e-300, 2.0 ** 64 * (1 - 2.0 ** -53), -1.0, -10000.0]
    freqs += [1.0] * (-len(freqs) % 8)
    for i in range(0, len(freqs), 8):
        st, r = _init(lib, 8, freqs=freqs[i:i + 8])
        assert st == OK
        for w, got in zip(freqs[i:i + 8], r.turns):
            d = abs(got - turn_fraction(w))
            assert min(d, 2 ** 64 - d) <= 0.5 + 2.0 ** -40, (w, float(d))
    for w in (2.0 ** 64, -2.0 ** 64, 1e300):
        assert _init(lib, 8, freqs=[w] * 8)[0] == INVALID


def test_make_private_queues_no_chains():
    """The pairs of one copy call are independent: no destination is another's source or destination."""
    from paged_kv_cache_pa_gb300.manager import BlockManager

    def independent(pairs):
        src, dst = set(pairs[:, 0].tolist()), pairs[:, 1].tolist()
        return len(set(dst)) == len(dst) and not src & set(dst)

    bm = BlockManager(8, 0, 16)
    a = bm.new_sequence()
    bm.append(a, 20)
    b = bm.fork(a)
    bm.append(b, 1)                        # queues a copy of block 1 to a block of b's
    c = bm.fork(b)
    with pytest.raises(pa.PaError):
        bm.make_private(c, 21)             # would copy from that block
    assert bm.table(c) == bm.table(b) and bm.num_free_gpu == 5
    pairs = bm.take_copies()
    assert pairs.tolist() == [[1, 2]]
    bm.make_private(c, 21)
    pairs = bm.take_copies()
    assert len(pairs) == 2 and independent(pairs)
    bm.close()

    bm = BlockManager(8, 0, 16)
    a, d = bm.new_sequence(), bm.new_sequence()
    bm.append(a, 20)
    bm.append(d, 30)
    b, e = bm.fork(a), bm.fork(d)
    bm.append(b, 1)                        # copies block 1
    bm.free(a)                             # and block 1 is free again
    with pytest.raises(pa.PaError):
        bm.make_private(e, 30)             # would copy to block 1
    assert bm.table(e) == bm.table(d) and bm.num_free_gpu == 4
    bm.take_copies()
    bm.make_private(e, 30)
    assert bm.table(e) == [1, 5]
    # two copies of one block are independent
    f = bm.fork(d)
    bm.make_private(f, 16)
    pairs = bm.take_copies()
    assert len(pairs) == 3 and independent(pairs)
    bm.close()


def test_prefill_scores_without_a_workspace(lib):
    """Without one: what is refused is what else is wrong."""
    for kw, want in (({"S": 0}, OK), ({"L": 128, "stride": 99}, INVALID), ({"sc": P + 2}, INVALID),
                     ({"D": 256}, UNSUPPORTED), ({"wb": 256}, INVALID)):
        assert _pscores(lib, **{"ws": None, "wb": 0, **kw}) == want
