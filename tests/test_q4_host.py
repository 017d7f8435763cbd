"""Refusals of the 4-bit cache's entry points, decided on the host before anything is
enqueued (no GPU needed), and their sizes."""
import ctypes

import pytest

import paged_kv_cache_pa_gb300 as pa

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = 0, 1, 2, 3, 4
P = 1 << 20  # a 256-byte aligned address that is never read


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_pa_gb300.build import build
    build()
    return pa.load_library()


def _write(lib, **kw):
    a = dict(k=P, ks=128, v=P, vs=128, kc=P, vc=P, slots=P, T=4, nb=4, bs=16, Hkv=2, D=64, dt=0)
    a.update(kw)
    return lib.pa_cache_write_q4(a["k"], a["ks"], a["v"], a["vs"], a["kc"], a["vc"], a["slots"], a["T"], a["nb"],
                                 a["bs"], a["Hkv"], a["D"], a["dt"], None, None)


@pytest.mark.parametrize("kw,want", [
    ({"T": 0}, OK), ({"T": 0, "k": None}, OK), ({"T": -1}, INVALID), ({"nb": 0}, INVALID), ({"Hkv": 0}, INVALID),
    ({"dt": 2}, INVALID), ({"dt": 3}, INVALID), ({"bs": 8}, UNSUPPORTED), ({"bs": 24}, UNSUPPORTED),
    ({"bs": 512}, UNSUPPORTED), ({"D": 96}, UNSUPPORTED), ({"D": 32}, UNSUPPORTED), ({"ks": 120}, INVALID),
    ({"vs": 129}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID), ({"kc": None}, INVALID),
    ({"vc": None}, INVALID), ({"slots": None}, INVALID), ({"k": P + 8}, INVALID), ({"vc": P + 4}, INVALID),
    ({"Hkv": 1 << 20, "ks": 1 << 26, "vs": 1 << 26}, UNSUPPORTED)])
def test_cache_write_refusals(lib, kw, want):
    assert _write(lib, **kw) == want


def _rot_call(lib, pairs=32, **kw):
    r = pa._RotaryStruct()
    lib.pa_rotary_init(ctypes.addressof(r), ctypes.cast((ctypes.c_double * pairs)(*[1.0] * pairs), ctypes.c_void_p),
                       None, pairs, 0, 1.0)
    a = dict(qo=P, qos=512, q=P, qs=512, k=P, ks=128, v=P, vs=128, pos=P, kc=P, vc=P, slots=P, T=4, nb=4, bs=16, H=8,
             Hkv=2, D=64, dt=0, r=ctypes.addressof(r))
    a.update(kw)
    return lib.pa_rotary_cache_write_q4(a["qo"], a["qos"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"],
                                        a["r"], a["kc"], a["vc"], a["slots"], a["T"], a["nb"], a["bs"], a["H"],
                                        a["Hkv"], a["D"], a["dt"], None, None)


@pytest.mark.parametrize("kw,want", [
    ({"T": 0}, OK), ({"T": -1}, INVALID), ({"r": None}, INVALID), ({"H": 0}, INVALID), ({"Hkv": 0}, INVALID),
    ({"bs": 8}, UNSUPPORTED), ({"D": 96}, UNSUPPORTED), ({"pairs": 64}, INVALID), ({"q": None}, INVALID),
    ({"qo": None}, INVALID), ({"pos": None}, INVALID), ({"qs": 504}, INVALID), ({"qos": 508}, INVALID),
    ({"dt": 3}, INVALID), ({"kc": P + 8}, INVALID)])
def test_rotary_write_refusals(lib, kw, want):
    assert _rot_call(lib, **kw) == want


def _decode(lib, **kw):
    a = dict(out=P, odt=2, q=P, k=P, v=P, tab=P, mb=8, qsl=P, lens=P, mq=4, L=100, S=2, T=6, H=8, Hkv=2, D=64, nb=16,
             bs=16, dt=0, ws=P, wb=1 << 30)
    a.update(kw)
    return lib.pa_decode_attention_q4(a["out"], a["odt"], a["q"], a["k"], a["v"], a["tab"], a["mb"], a["qsl"], a["lens"],
                                      a["mq"], a["L"], a["S"], a["T"], a["H"], a["Hkv"], a["D"], a["nb"], a["bs"], 0.1,
                                      a["dt"], a["ws"], a["wb"], None, None)


@pytest.mark.parametrize("kw,want", [
    ({"S": 0}, OK), ({"T": 0}, OK), ({"S": -1}, INVALID), ({"T": -1}, INVALID), ({"mq": 0}, INVALID),
    ({"mq": 17}, UNSUPPORTED), ({"mq": 16, "S": 0}, OK), ({"L": -1}, INVALID), ({"L": 129}, INVALID), ({"nb": 0}, INVALID),
    ({"mb": 0}, INVALID), ({"H": 9}, INVALID), ({"H": 0}, INVALID), ({"Hkv": 0}, INVALID), ({"D": 80}, UNSUPPORTED),
    ({"bs": 8}, UNSUPPORTED), ({"bs": 48}, UNSUPPORTED), ({"dt": 2}, INVALID), ({"dt": 3}, INVALID), ({"odt": 1}, INVALID),
    ({"odt": 3}, INVALID), ({"qsl": None}, INVALID), ({"qsl": None, "T": 2}, INVALID), ({"qsl": None, "mq": 1}, INVALID),
    ({"q": None}, INVALID), ({"out": None}, INVALID), ({"k": None}, INVALID), ({"v": None}, INVALID),
    ({"tab": None}, INVALID), ({"lens": None}, INVALID), ({"ws": None}, INVALID), ({"q": P + 8}, INVALID),
    ({"out": P + 4}, INVALID), ({"k": P + 8}, INVALID), ({"v": P + 2}, INVALID), ({"ws": P + 128}, WORKSPACE),
    ({"wb": 100}, WORKSPACE), ({"L": 1 << 30, "mb": 1 << 27, "Hkv": 64, "H": 64}, UNSUPPORTED)])
def test_decode_refusals(lib, kw, want):
    assert _decode(lib, **kw) == want


def test_decode_workspace_size(lib):
    a = pa.decode_q4_workspace_size(64, 12, 2, 128, 1, 4096)
    assert a > 0 and a == pa.decode_q4_workspace_size(64, 12, 2, 128, 1, 4096)
    assert pa.decode_q4_workspace_size(64, 12, 2, 128, 1, 8192) >= a
    assert pa.decode_q4_workspace_size(1 << 16, 40, 40, 256, 16, 1 << 20) < 1 << 27  # bounded by the GPU, not the batch
    assert 0 < pa.decode_q4_workspace_size(4, 8, 8, 64, 1, 128) <= 256
    for bad in ((-1, 8, 8, 64, 1, 10), (4, 9, 8, 64, 1, 10), (4, 8, 8, 96, 1, 10), (4, 8, 8, 64, 0, 10),
                (4, 8, 8, 64, 17, 10), (4, 8, 8, 64, 1, -1), (4, 0, 8, 64, 1, 10)):
        assert pa.decode_q4_workspace_size(*bad) == 0
    need = pa.decode_q4_workspace_size(2, 8, 2, 64, 4, 2000)
    assert _decode(lib, L=2000, mb=125, wb=need - 1) == WORKSPACE


def _ptrs(*ps):
    return ctypes.cast((ctypes.c_void_p * len(ps))(*ps), ctypes.c_void_p)


def _unpack(lib, **kw):
    a = dict(dk=_ptrs(P, P), dv=_ptrs(P, P), sk=_ptrs(P, P), sv=_ptrs(P, P), layers=2, pairs=P, n=3, nd=9, ns=9, bs=16,
             Hkv=2, D=64, dt=0)
    a.update(kw)
    return lib.pa_unpack_blocks_q4(a["dk"], a["dv"], a["sk"], a["sv"], a["layers"], a["pairs"], a["n"], a["nd"], a["ns"],
                                   a["bs"], a["Hkv"], a["D"], a["dt"], None, None)


@pytest.mark.parametrize("kw,want", [
    ({"n": 0}, OK), ({"n": -1}, INVALID), ({"layers": 0}, INVALID), ({"layers": 129}, UNSUPPORTED), ({"nd": 0}, INVALID),
    ({"ns": 0}, INVALID), ({"Hkv": 0}, INVALID), ({"bs": 8}, UNSUPPORTED), ({"D": 48}, UNSUPPORTED), ({"dt": 2}, INVALID),
    ({"dt": 3}, INVALID), ({"dk": None}, INVALID), ({"dv": None}, INVALID), ({"sk": None}, INVALID),
    ({"sv": None}, INVALID), ({"pairs": None}, INVALID), ({"sk": _ptrs(P, None)}, INVALID),
    ({"dv": _ptrs(P, P + 8)}, INVALID), ({"sv": _ptrs(P + 4, P)}, INVALID),
    ({"Hkv": 1 << 16, "bs": 256, "D": 256}, UNSUPPORTED)])
def test_unpack_refusals(lib, kw, want):
    assert _unpack(lib, **kw) == want


@pytest.mark.parametrize("bs,dt,want", [(16, 3, OK), (256, 3, OK), (8, 3, UNSUPPORTED), (8, 0, OK), (16, 2, INVALID),
                                        (16, 4, INVALID), (24, 3, UNSUPPORTED)])
def test_block_moves_know_4_bit_pools(lib, bs, dt, want):
    assert lib.pa_copy_blocks_ex(_ptrs(P), _ptrs(P), 1, P, 0, 4, bs, 2, 64, dt, None, None) == want
    assert lib.pa_swap_blocks(_ptrs(P), _ptrs(P), _ptrs(P), _ptrs(P), 1, P, 0, 4, 4, bs, 2, 64, dt, None, None) == want


def test_pool_shape():
    assert pa.q4_pool_shape(10, 2, 16, 64) == (10, 2, 16, 36)
    assert pa.q4_pool_shape(1, 8, 256, 256) == (1, 8, 256, 144)
    with pytest.raises(ValueError):
        pa.q4_pool_shape(1, 8, 16, 96)


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    pool = torch.zeros(pa.q4_pool_shape(4, 2, 16, 64), dtype=torch.uint8)
    half = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    x, slots = torch.zeros(3, 2, 64, dtype=torch.float16), torch.zeros(3, dtype=torch.int64)
    i32 = torch.zeros(3, dtype=torch.int32)
    tab = torch.zeros(3, 4, dtype=torch.int32)
    rot = pa.Rotary([1.0] * 32)
    for call, exc in [
            (lambda: pa.cache_write_q4(x, x, half, half, slots), TypeError),
            (lambda: pa.cache_write_q4(x, x[:2], pool, pool, slots), ValueError),
            (lambda: pa.cache_write_q4(x, x.bfloat16(), pool, pool, slots), ValueError),
            (lambda: pa.cache_write_q4(x[:, :1], x[:, :1], pool, pool, slots), ValueError),
            (lambda: pa.cache_write_q4(torch.cat([x, x], -1), torch.cat([x, x], -1), pool, pool, slots), ValueError),
            (lambda: pa.cache_write_q4(x, x, pool, pool, i32), TypeError),
            (lambda: pa.cache_write_q4(x, x, pool, pool, slots[:2]), ValueError),
            (lambda: pa.cache_write_q4(x, x, pool, pool, slots), ValueError),                # not on a GPU
            (lambda: pa.rotary_cache_write_q4(x, x, x, slots, rot, half, half, slots), TypeError),
            (lambda: pa.rotary_cache_write_q4(x, x, x.bfloat16(), slots, rot, pool, pool, slots), ValueError),
            (lambda: pa.rotary_cache_write_q4(x, x, x, slots[:2], rot, pool, pool, slots), ValueError),
            (lambda: pa.rotary_cache_write_q4(x, x, x, i32, rot, pool, pool, slots), TypeError),
            (lambda: pa.rotary_cache_write_q4(x, x, x, slots, rot, pool, pool, slots, query_out=x.float()), ValueError),
            (lambda: pa.decode_attention_q4(x, half, half, tab, i32, 10, 0.1), TypeError),
            (lambda: pa.decode_attention_q4(x, pool, pool, tab, slots, 10, 0.1), TypeError),
            (lambda: pa.decode_attention_q4(x, pool, pool, tab[:2], i32, 10, 0.1), ValueError),
            (lambda: pa.decode_attention_q4(x, pool, pool, tab[:2], i32[:2], 10, 0.1), ValueError),
            (lambda: pa.decode_attention_q4(x, pool, pool, tab, i32, 10, 0.1, max_query_len=2), ValueError),
            (lambda: pa.decode_attention_q4(x, pool, pool, tab, i32, 10, 0.1, query_start_loc=i32), ValueError),
            (lambda: pa.decode_attention_q4(x, pool, pool, tab, i32, 10, 0.1, out=x[:2]), ValueError),
            (lambda: pa.unpack_blocks_q4([half], [half], [pool], [half], slots.view(1, 3)), TypeError),
            (lambda: pa.unpack_blocks_q4([half], [half], [pool], [], slots), ValueError),
            (lambda: pa.unpack_blocks_q4([half[:, :, :8]], [half[:, :, :8]], [pool], [pool], slots), ValueError),
            (lambda: pa.copy_blocks([pool[..., :35]], [pool[..., :35]], slots), ValueError)]:
        with pytest.raises(exc):
            call()


def test_error_values_match_the_header():
    import os
    import re
    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "pa.h")).read()
    assert re.search(r"#define PA_MAX_Q4_QUERY (\d+)", text).group(1) == str(pa.MAX_Q4_QUERY)
    assert re.search(r"PA_Q4 = (\d+)", text).group(1) == str(pa.PA_Q4)


@pytest.mark.parametrize("shape", [(2,), (6,), (2, 3), (1, 2, 2)])
def test_unpack_wants_pairs(shape):
    """Rows of two: anything else would be read past its end."""
    torch = pytest.importorskip("torch")
    pool = torch.zeros(pa.q4_pool_shape(4, 2, 16, 64), dtype=torch.uint8)
    half = torch.zeros(4, 2, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="block_pairs must be"):
        pa.unpack_blocks_q4([half], [half], [pool], [pool], torch.zeros(shape, dtype=torch.int64))
