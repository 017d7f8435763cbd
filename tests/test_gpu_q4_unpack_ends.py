"""Groups next to the ends of their type, unpacked: finite values stay finite."""
import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa
from q4lib import held

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_finite_groups_unpack_to_finite_values(D, dtype):
    """Ranges up to the type's largest number (and, in fp16, from its least), whose scale is
    rounded up or down: s n + z where that is finite, the largest number past it.  Groups with a
    NaN or an infinity stay NaN."""
    top = torch.finfo(dtype).max
    g = torch.Generator(device=DEV).manual_seed(D)
    x = torch.rand(128, 1, D, generator=g, device=DEV)
    least = -1 if dtype == torch.float16 else -0.003
    # (the second half: ranges whose scale has its coarsest step, 15 / 2 of which is past the end)
    low = torch.cat([torch.linspace(least, 0.99, 64), torch.linspace(least, 0.05, 64)]).to(DEV)[:, None, None]
    x = ((low + (1 - low) * x) * top).to(dtype).clamp(-top, top)
    x[..., 5::64], x[..., 9::64] = top, (low[:, :, :1] * top).to(dtype)
    x[7, 0, 3], x[8, 0, 3], x[9, 0, 3] = float("nan"), float("inf"), float("-inf")
    k4, v4 = (torch.zeros(pa.q4_pool_shape(8, 1, 16, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    pa.cache_write_q4(x, -x, k4, v4, torch.arange(128, device=DEV))
    k, v = (torch.zeros(8, 1, 16, D, dtype=dtype, device=DEV) for _ in range(2))
    pa.unpack_blocks_q4([k], [v], [k4], [v4], torch.arange(8, device=DEV)[:, None].expand(8, 2).contiguous())
    over = 0
    for got, y in ((k, x), (v, -x)):
        n, s, z = held(y)
        want = (n * s + z).flatten(-2)[:, 0]
        got = got.view(128, D)
        bad = torch.isnan(want)
        assert torch.equal(torch.isnan(got), bad) and bad.any()
        over += int((want.float().to(dtype).isinf() & ~bad).sum())
        assert torch.equal(got[~bad], want.float().to(dtype).clamp(-top, top)[~bad])
    assert over > 0


def test_a_continued_prompt_at_the_ends():
    """Prefill over unpacked blocks whose values reach the largest of fp16: as the decode call
    over the 4-bit blocks, finite."""
    D, L = 128, 48
    g = torch.Generator(device=DEV).manual_seed(2)
    k = torch.randn(L, 1, D, generator=g, device=DEV).half()
    v = torch.rand(L, 1, D, generator=g, device=DEV).half()
    v[:, :, ::16], v[:, :, 1::16] = 65504.0, 0.0
    q = torch.randn(1, 2, D, generator=g, device=DEV).half()
    k4, v4 = (torch.zeros(pa.q4_pool_shape(3, 1, 16, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    pa.cache_write_q4(k, v, k4, v4, torch.arange(L, device=DEV))
    k16, v16 = (torch.zeros(3, 1, 16, D, dtype=torch.float16, device=DEV) for _ in range(2))
    pa.unpack_blocks_q4([k16], [v16], [k4], [v4], torch.arange(3, device=DEV)[:, None].expand(3, 2).contiguous())
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    tables = i32([[0, 1, 2]])
    a = pa.prefill_attention(q, k16, v16, tables, i32([0, 1]), i32([L]), 1, L, 0.1)
    b = pa.decode_attention_q4(q, k4, v4, tables, i32([L]), L, 0.1)
    assert torch.isfinite(a).all() and torch.isfinite(b).all()
    # 65520 and 65504 are 2^-12 apart, the unpacked values and prefill's weights are rounded to 2^-11 each
    assert float((a - b).abs().max()) <= 65520 * (2.0 ** -12 + 2 * 2.0 ** -11)
