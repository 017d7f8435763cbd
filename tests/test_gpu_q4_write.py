"""pa_cache_write_q4, pa_rotary_cache_write_q4 and pa_unpack_blocks_q4 on the GPU against
the format's definition in 64 bits and an independent reading of the pools' bytes.

Codes, scales and least values are compared bit for bit: the definition rounds the quotient
once, from an exact difference (the inputs' difference fits 32 bits but for elements far
below the least value, which random inputs do not bring next to a tie)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from q4lib import decode_bytes, held, values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _pools(nb, Hkv, B, D, fill=255):
    shape = pa.q4_pool_shape(nb, Hkv, B, D)
    return [torch.full(shape, fill, dtype=torch.uint8, device=DEV) for _ in range(2)]


def _case(T, Hkv, D, dtype, B=16, seed=0, pad=8):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kv = torch.randn(T, 2 * Hkv * D + pad, generator=g, device=DEV).to(dtype)
    k, v = kv[:, :Hkv * D].view(T, Hkv, D), kv[:, Hkv * D:2 * Hkv * D].view(T, Hkv, D)
    nb = -(-max(T, 1) // B) + 3
    slots = np.random.default_rng(seed).permutation(nb * B)[:T].astype(np.int64)
    return k, v, nb, torch.as_tensor(slots, device=DEV)


def _same(got, want):
    return torch.equal(torch.nan_to_num(got, nan=1e9), torch.nan_to_num(want, nan=1e9))


def _check_pool(pool, x, slots, dtype):
    """The written rows hold x; every other byte is as it was (all ones)."""
    nb, hkv, B, _ = pool.shape
    D = x.shape[-1]
    n, s, z = (t.to(DEV) for t in decode_bytes(pool, D, dtype))
    live = (slots >= 0) & (slots < nb * B)
    at = slots[live]
    wn, ws, wz = held(x[live])
    at = (at // B, slice(None), at % B)
    assert _same(n[at], wn.to(n.dtype))
    assert _same(s[at], ws[..., 0]) and _same(z[at], wz[..., 0])
    other = torch.ones(nb, B, dtype=torch.bool, device=DEV)
    other[at[0], at[2]] = False
    keep = other[:, None, :].expand(-1, hkv, -1)
    assert bool((n[keep] == 15).all()) and bool(torch.isnan(s[keep]).all()) and bool(torch.isnan(z[keep]).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hkv,D,B", [
    (1, 1, 64, 16), (1, 40, 128, 16), (3, 8, 64, 32), (16, 2, 128, 16), (33, 1, 256, 64), (130, 3, 256, 256),
    (257, 8, 128, 128), (1031, 2, 64, 16), (2, 50, 256, 16), (4099, 2, 128, 16), (700, 1, 64, 16)])
def test_write_holds_the_definition(T, Hkv, D, B, dtype):
    k, v, nb, slots = _case(T, Hkv, D, DT[dtype], B, seed=T)
    k4, v4 = _pools(nb, Hkv, B, D)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.cache_write_q4(k, v, k4, v4, slots, error_word=err)
    _check_pool(k4, k, slots, DT[dtype])
    _check_pool(v4, v, slots, DT[dtype])
    assert int(err.item()) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_special_groups(dtype):
    """Constant, zero, subnormal, huge, non-finite groups, and exact ties."""
    dt = DT[dtype]
    fi = torch.finfo(dt)
    rows = []
    rows.append(torch.zeros(64))
    rows.append(torch.full((64,), -0.0))
    rows.append(torch.full((64,), 3.25))
    rows.append(torch.linspace(-1, 1, 64) * fi.smallest_normal)             # subnormal scales
    rows.append(torch.linspace(0, 1, 64) * fi.smallest_normal * 2.0 ** -4)
    rows.append(torch.linspace(-0.7, 1, 64) * fi.max * 0.5)
    rows.append(torch.cat([torch.tensor([-fi.max, fi.max]), torch.zeros(62)]))
    rows.append(torch.cat([torch.tensor([float("nan")]), torch.ones(63)]))
    rows.append(torch.cat([torch.ones(63), torch.tensor([float("inf")])]))
    rows.append(torch.cat([torch.tensor([float("-inf")]), torch.ones(63)]))
    rows.append(torch.cat([torch.tensor([0.0, 15.0]), torch.arange(15) + 0.5, torch.zeros(47)]))     # s = 1
    rows.append(torch.cat([torch.tensor([-8.0, -0.5]), torch.arange(15) * 0.5 - 7.75, torch.full((47,), -4.0)]))
    rows.append(torch.cat([torch.full((63,), 100.0), torch.tensor([101.0])]))
    x = torch.stack(rows).to(dt).to(DEV).view(-1, 1, 64)
    T = x.shape[0]
    k4, v4 = _pools(2, 1, 16, 64)
    slots = torch.arange(T, device=DEV)
    pa.cache_write_q4(x, -x, k4, v4, slots)
    _check_pool(k4, x, slots, dt)
    _check_pool(v4, -x, slots, dt)


def test_scales_next_to_the_smallest_of_bf16():
    """Scales whose reciprocal leaves fp32: 2^-126 .. 2^-100 and below."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.rand(64, 2, 128, generator=g, device=DEV)
    x = (x * torch.logspace(-132, -95, 64, base=2.0, device=DEV)[:, None, None]).bfloat16()
    k4, v4 = _pools(4, 2, 16, 128)
    slots = torch.arange(64, device=DEV)
    pa.cache_write_q4(x, x, k4, v4, slots)
    _check_pool(k4, x, slots, torch.bfloat16)


def test_a_nan_stays_in_its_group():
    k, v, nb, slots = _case(20, 2, 128, torch.bfloat16, seed=3)
    k4, v4 = _pools(nb, 2, 16, 128)
    pa.cache_write_q4(k, v, k4, v4, slots)
    clean = k4.clone()
    k2 = k.clone()
    k2[7, 1, 70] = float("nan")
    pa.cache_write_q4(k2, v, k4, v4, slots)
    n0, s0, z0 = decode_bytes(clean, 128, torch.bfloat16)
    n1, s1, z1 = decode_bytes(k4, 128, torch.bfloat16)
    b, o = int(slots[7]) // 16, int(slots[7]) % 16
    same = torch.ones(s0.shape, dtype=torch.bool)
    same[b, 1, o, 1] = False
    assert torch.isnan(s1[b, 1, o, 1]) and torch.isnan(z1[b, 1, o, 1]) and not n1[b, 1, o, 1].any()
    for a, c in ((n0, n1), (s0, s1), (z0, z1)):
        assert _same(a[same], c[same])


def test_padding_and_slots_past_the_pool():
    k, v, nb, slots = _case(50, 4, 64, torch.float16, seed=9)
    slots[::3] = -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    k4, v4 = _pools(nb, 4, 16, 64)
    pa.cache_write_q4(k, v, k4, v4, slots, error_word=err)
    _check_pool(k4, k, slots, torch.float16)
    assert int(err.item()) == 0
    slots[1], slots[4] = nb * 16, 1 << 40
    k4, v4 = _pools(nb, 4, 16, 64)
    pa.cache_write_q4(k, v, k4, v4, slots, error_word=err)
    _check_pool(k4, k, slots, torch.float16)
    _check_pool(v4, v, slots, torch.float16)
    assert int(err.item()) == pa.ERRBIT_SLOT_OOB
    pa.cache_write_q4(k[:0], v[:0], k4, v4, slots[:0])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,Hkv,D,rot,B,inter,axes", [
    (1, 8, 8, 64, 64, 16, False, 1), (7, 12, 2, 128, 128, 16, False, 3), (33, 5, 1, 128, 96, 32, False, 1),
    (130, 6, 2, 256, 256, 64, True, 1), (65, 3, 3, 256, 48, 256, False, 2), (257, 64, 8, 128, 64, 16, True, 1),
    (2, 100, 50, 256, 128, 16, False, 1), (1500, 12, 2, 128, 128, 16, False, 1), (40, 4, 2, 64, 16, 16, False, 1)])
def test_rotation_and_write(T, H, Hkv, D, rot, B, inter, axes, dtype):
    """The 16-bit call on the same inputs gives the turned query and key, bit for bit; the key
    is quantised from there."""
    dt = DT[dtype]
    g = torch.Generator(device=DEV).manual_seed(T)
    qkv = torch.randn(T, (H + 2 * Hkv) * D + 8, generator=g, device=DEV).to(dt)
    q = qkv[:, :H * D].view(T, H, D)
    k = qkv[:, H * D:(H + Hkv) * D].view(T, Hkv, D)
    v = qkv[:, (H + Hkv) * D:(H + 2 * Hkv) * D].view(T, Hkv, D)
    pos = torch.randint(0, 50000, (axes, T), generator=g, device=DEV)
    r = pa.Rotary([10000.0 ** (-i / (rot // 2)) for i in range(rot // 2)],
                  axes=[i % axes for i in range(rot // 2)], interleaved=inter, scale=1.0)
    nb = -(-T // B) + 3
    slots = torch.as_tensor(np.random.default_rng(T).permutation(nb * B)[:T].astype(np.int64), device=DEV)
    slots[T // 2] = -1
    k16, v16 = (torch.zeros(nb, Hkv, B, D, dtype=dt, device=DEV) for _ in range(2))
    want_q = pa.rotary_cache_write(q, k, v, pos, r, k16, v16, slots)
    k4, v4 = _pools(nb, Hkv, B, D)
    got_q = pa.rotary_cache_write_q4(q, k, v, pos, r, k4, v4, slots)
    assert torch.equal(got_q, want_q)
    turned = torch.zeros(T, Hkv, D, dtype=dt, device=DEV)
    live = slots >= 0
    turned[live] = k16[slots[live] // B, :, slots[live] % B]
    _check_pool(k4, turned, slots, dt)
    _check_pool(v4, v, slots, dt)
    q2 = q.clone()
    assert pa.rotary_cache_write_q4(q2, k, v, pos, r, k4, v4, slots, query_out=q2) is q2
    assert torch.equal(q2, want_q)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("Hkv,D,B,layers", [(1, 64, 16, 1), (3, 128, 32, 2), (8, 256, 256, 1), (2, 128, 16, 5)])
def test_unpack(Hkv, D, B, layers, dtype):
    dt = DT[dtype]
    T, nb = 5 * B, 7
    src, dst, want = [], [], []
    for i in range(2 * layers):
        k, v, _, _ = _case(T, Hkv, D, dt, B, seed=i)
        k4, spare = _pools(nb, Hkv, B, D, fill=0)
        pa.cache_write_q4(k, v, k4, spare, torch.arange(T, device=DEV))
        src.append(k4)
        full = torch.zeros(nb * B, Hkv, D, dtype=torch.float64, device=DEV)
        full[:T] = values(k)[0]
        want.append(full.view(nb, B, Hkv, D).transpose(1, 2))
        dst.append(torch.full((9, Hkv, B, D), 7.0, dtype=dt, device=DEV))
    pairs = torch.tensor([[3, 0], [0, 8], [6, 4], [1, 1], [3, 5], [7, 2], [2, 9], [-1, 3]], device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    pa.unpack_blocks_q4(dst[:layers], dst[layers:], src[:layers], src[layers:], pairs, error_word=err)
    assert int(err.item()) == pa.ERRBIT_BLOCK_OOB
    for d, w in zip(dst, want):
        for a, b in ((3, 0), (0, 8), (6, 4), (1, 1), (3, 5)):
            # s n + z: one rounding to fp32, one to the type
            exact = w[a]
            assert torch.equal(d[b], exact.float().to(dt))
        for b in (2, 3, 6, 7):
            assert bool((d[b] == 7.0).all())
    pa.unpack_blocks_q4(dst[:layers], dst[layers:], src[:layers], src[layers:], pairs[:0])


def test_unpack_across_sixty_four_bits_of_offset():
    """Blocks behind the first 4 GiB of a pool."""
    Hkv, D, B = 8, 256, 256
    nb = (1 << 32) // (Hkv * B * 144) + 40
    k4 = torch.zeros(pa.q4_pool_shape(nb, Hkv, B, D), dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    k = torch.randn(B, Hkv, D, generator=g, device=DEV).half()
    pa.cache_write_q4(k, k, k4, k4, (nb - 1) * B + torch.arange(B, device=DEV))
    d = torch.zeros(1, Hkv, B, D, dtype=torch.float16, device=DEV)
    pa.unpack_blocks_q4([d], [d], [k4], [k4], torch.tensor([[nb - 1, 0]], device=DEV))
    assert torch.equal(d[0].transpose(0, 1), values(k)[0].float().half())
