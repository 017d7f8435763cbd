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
