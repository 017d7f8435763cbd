"""pa_rotary_cache_write on the GPU against the rotation's formula in 64 bits.

Tolerance: a fraction of a turn below one half is rounded to 32 bits (2^-25
turns, 1.9e-7 rad), sine and cosine carry two steps (2.4e-7 at most), and two
products and a sum in fp32 add 2^-23 of |x| + |y|; together below 1e-6 (|x| +
|y|).  The one rounding to the 16-bit type adds eps / 2 of the value (and half
the smallest fp16 step near zero)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from cachelib import turn_fraction

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _freqs(pairs, base=10000.0):
    return [base ** (-i / pairs) for i in range(pairs)]


def _turn(x, pos, freqs, axes, interleaved, scale):
    """x [T][H][D] in 64 bits, pos [A][T] Python-exact; returns (turned, |x| + |y|)."""
    x = x.double().cpu().numpy()
    pairs = len(freqs)
    pos = pos.cpu().numpy()
    # the angle modulo a turn, in exact integer steps of the position
    ang = np.empty((x.shape[0], pairs))
    for i, f in enumerate(freqs):
        p = pos[axes[i]].astype(np.longdouble)
        ang[:, i] = np.fmod(p * np.longdouble(f), np.longdouble(2) * np.pi).astype(np.float64)
    c, s = np.cos(ang)[:, None] * scale, np.sin(ang)[:, None] * scale
    out, mag = x.copy(), np.zeros_like(x)
    if interleaved:
        a, b = slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)
    else:
        a, b = slice(0, pairs), slice(pairs, 2 * pairs)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(scale)
    return out, mag


def _close(got, want, mag, dtype):
    got = got.double().cpu().numpy()
    tol = torch.finfo(dtype).eps / 2 * np.abs(want) * (1 + 1e-3) + 1e-6 * mag
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))


def _case(T, H, Hkv, D, dtype, B=16, seed=0, axes=1, far=5000, pad=8):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn(T, (H + 2 * Hkv) * D + pad, generator=g, device=DEV).to(dtype)
    q = qkv[:, :H * D].view(T, H, D)
    k = qkv[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (H + Hkv) * D:(H + 2 * Hkv) * D].view(T, Hkv, D)
    nb = -(-max(T, 1) // B) + 3
    kc = torch.randn(nb, Hkv, B, D, generator=g, device=DEV).to(dtype)
    vc = torch.randn(nb, Hkv, B, D, generator=g, device=DEV).to(dtype)
    slots = torch.as_tensor(np.random.default_rng(seed).permutation(nb * B)[:T].astype(np.int64))
    pos = torch.randint(0, far, (axes, T), generator=g, device=DEV)
    return q, k, v, kc, vc, slots.to(DEV), pos


def _check(q, k, v, kc, vc, slots, pos, freqs, axes, interleaved, scale, **kw):
    dtype, B, T = q.dtype, kc.shape[2], q.shape[0]
    k0, v0 = kc.clone(), vc.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    rot = pa.Rotary(freqs, axes=axes, interleaved=interleaved, scale=scale)
    wq, mq = _turn(q, pos, freqs, axes, interleaved, scale)
    wk, mk = _turn(k, pos, freqs, axes, interleaved, scale)
    vw = v.clone()
    out = pa.rotary_cache_write(q, k, v, pos, rot, kc, vc, slots, error_word=err, **kw)
    torch.cuda.synchronize()
    _close(out, wq, mq, dtype)
    live = (slots >= 0) & (slots < kc.shape[0] * B)
    s = slots[live]
    _close(kc[s // B, :, s % B], wk[live.cpu().numpy()], mk[live.cpu().numpy()], dtype)
    assert torch.equal(vc[s // B, :, s % B], vw[live])
    untouched = torch.ones(kc.shape[0], B, dtype=torch.bool, device=DEV)
    untouched[s // B, s % B] = False
    keep = untouched[:, None, :].expand(-1, kc.shape[1], -1)
    assert torch.equal(kc[keep], k0[keep]) and torch.equal(vc[keep], v0[keep])
    return out, int(err.item())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,Hkv,D,rot,B", [
    (1, 1, 1, 64, 64, 16), (1, 40, 40, 128, 128, 16), (3, 8, 8, 64, 16, 8), (7, 12, 2, 128, 128, 16),
    (33, 5, 1, 128, 96, 32), (130, 6, 2, 256, 256, 64), (65, 3, 3, 256, 48, 256), (257, 64, 8, 128, 64, 16),
    (2, 100, 50, 256, 128, 16)])
def test_rotation_and_write(T, H, Hkv, D, rot, B, interleaved, dtype):
    q, k, v, kc, vc, slots, pos = _case(T, H, Hkv, D, DT[dtype], B, seed=T)
    _, err = _check(q, k, v, kc, vc, slots, pos, _freqs(rot // 2), [0] * (rot // 2), interleaved, 1.0)
    assert err == 0


@pytest.mark.parametrize("axes", [[0] * 16 + [1] * 24 + [2] * 24, [i % 3 for i in range(64)],
                                  [7] * 64])
def test_several_axes_and_scale(axes):
    n = max(axes) + 1
    q, k, v, kc, vc, slots, pos = _case(70, 12, 2, 128, torch.bfloat16, axes=n, seed=3)
    _check(q, k, v, kc, vc, slots, pos, _freqs(64, 1e6), axes, False, 1.25)


@pytest.mark.parametrize("far", [1 << 20, 1 << 31, 1 << 40])
def test_far_and_negative_positions(far):
    """The angle is exact modulo a turn; frequencies that are short binary fractions of a
    turn keep the oracle's own angle exact."""
    q, k, v, kc, vc, slots, pos = _case(40, 4, 2, 64, torch.float16, seed=5, far=far)
    pos[0, ::2] *= -1
    turns = [(2 * i + 1) / 2.0 ** 12 for i in range(32)]
    rot = pa.Rotary([2 * math.pi * t for t in turns])
    out = pa.rotary_cache_write(q, k, v, pos, rot, kc, vc, slots)
    p = pos[0].cpu().numpy().astype(object)
    ang = np.array([[float((int(x) * (2 * i + 1)) % 4096) / 4096 for i in range(32)] for x in p])
    z = np.exp(2j * np.pi * ang)[:, None]
    x = q.double().cpu().numpy()
    w = (x[..., :32] + 1j * x[..., 32:]) * z
    mag = np.abs(x[..., :32]) + np.abs(x[..., 32:])
    # 2 pi t is rounded to 53 bits before it becomes a fraction: far * 2^-53 turns
    slack = far * 2.0 ** -50 * mag
    _close_far(out, np.concatenate([w.real, w.imag], -1), np.concatenate([mag, mag], -1),
               np.concatenate([slack, slack], -1))


def _close_far(got, want, mag, slack):
    got = got.double().cpu().numpy()
    tol = 2.0 ** -11 * np.abs(want) * (1 + 1e-3) + 1e-6 * mag + 2.0 ** -25 + slack
    assert np.all(np.abs(got - want) <= tol)


def test_in_place_and_other_output_stride():
    q, k, v, kc, vc, slots, pos = _case(21, 12, 2, 128, torch.bfloat16, seed=8)
    want, _ = _check(q.clone(), k, v, kc.clone(), vc.clone(), slots, pos, _freqs(64), [0] * 64, False, 1.0)
    wide = torch.zeros(21, 12 * 128 + 64, dtype=torch.bfloat16, device=DEV)
    got = pa.rotary_cache_write(q, k, v, pos, pa.Rotary(_freqs(64)), kc, vc, slots,
                                query_out=wide[:, :12 * 128].view(21, 12, 128))
    assert torch.equal(got, want) and not wide[:, 12 * 128:].any()
    same = pa.rotary_cache_write(q, k, v, pos, pa.Rotary(_freqs(64)), kc, vc, slots, query_out=q)
    assert same is q and torch.equal(q, want)


def test_padding_and_slots_past_the_pool():
    q, k, v, kc, vc, slots, pos = _case(50, 8, 4, 64, torch.float16, seed=9)
    slots[::3] = -1
    _, err = _check(q, k, v, kc, vc, slots, pos, _freqs(32), [0] * 32, False, 1.0)
    assert err == 0
    slots[1] = kc.shape[0] * 16
    slots[4] = 1 << 40
    _, err = _check(q, k, v, kc, vc, slots, pos, _freqs(32), [0] * 32, False, 1.0)
    assert err == pa.ERRBIT_SLOT_OOB


def test_no_tokens_and_nan_stays_in_its_pair():
    q, k, v, kc, vc, slots, pos = _case(0, 8, 4, 64, torch.float16)
    assert pa.rotary_cache_write(q, k, v, pos, pa.Rotary(_freqs(32)), kc, vc, slots).shape == (0, 8, 64)
    q, k, v, kc, vc, slots, pos = _case(4, 8, 4, 64, torch.float16, seed=2)
    clean = pa.rotary_cache_write(q, k, v, pos, pa.Rotary(_freqs(32)), kc, vc, slots)
    q[2, 3, 5] = float("nan")
    out = pa.rotary_cache_write(q, k, v, pos, pa.Rotary(_freqs(32)), kc, vc, slots)
    bad = torch.isnan(out)
    assert bad.sum() == 2 and bad[2, 3, 5] and bad[2, 3, 37]
    assert torch.equal(out[~bad], clean[~bad])


def test_captured_and_replayed_on_another_stream():
    q, k, v, kc, vc, slots, pos = _case(30, 12, 2, 128, torch.bfloat16, seed=4)
    rot = pa.Rotary(_freqs(64))
    want = pa.rotary_cache_write(q, k, v, pos, rot, kc, vc, slots)
    out = torch.empty_like(want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            pa.rotary_cache_write(q, k, v, pos, rot, kc, vc, slots, query_out=out)
        del rot  # the frequencies are part of the captured call
        kc.zero_()
        g.replay()
    st.synchronize()
    assert torch.equal(out, want) and kc[slots // 16, :, slots % 16].any()


@pytest.mark.parametrize("far", [1 << 20, 1 << 31, 1 << 40])
def test_far_positions_of_ordinary_frequencies(far):
    """Slack: the frequency is right to 2^-65 turns, 2 pi far 2^-65 of an angle."""
    q, k, v, kc, vc, slots, pos = _case(40, 4, 2, 64, torch.float16, seed=6, far=far)
    pos = far - 1 - pos % 1000
    pos[0, ::2] *= -1
    freqs = _freqs(32)
    out = pa.rotary_cache_write(q, k, v, pos, pa.Rotary(freqs), kc, vc, slots)
    turns = [turn_fraction(f) for f in freqs]
    ang = np.array([[float(int(p) * t % 2 ** 64) / 2 ** 64 for t in turns] for p in pos[0].cpu().numpy()])
    z = np.exp(2j * np.pi * ang)[:, None]
    x = q.double().cpu().numpy()
    w = (x[..., :32] + 1j * x[..., 32:]) * z
    mag = np.abs(x[..., :32]) + np.abs(x[..., 32:])
    slack = 2 * math.pi * far * 2.0 ** -65 * mag
    _close_far(out, np.concatenate([w.real, w.imag], -1), np.concatenate([mag, mag], -1),
               np.concatenate([slack, slack], -1))
