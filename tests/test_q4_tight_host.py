"""q4tight's bound, on the CPU: below what it is to see, above what 32 bits give."""
import pytest

torch = pytest.importorskip("torch")

import q4tight
from q4lib import held


def _rows(L, D, n=1, G=2, seed=1):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(L, D, generator=g).bfloat16() for _ in range(2))
    return k, v, torch.randn(n, G, D, generator=g).bfloat16()


@pytest.mark.parametrize("L,D", [(20000, 128), (60000, 64), (40000, 256), (700, 128)])
def test_planted_mistakes_are_seen(L, D):
    """A context of which ten chunks are missing, one with eight chunks twice, outputs of zero
    and outputs off by 2^-6 of themselves."""
    k, v, q = _rows(L, D)
    want, tol = q4tight.rows_attention(k, v, q, D ** -0.5)
    assert q4tight.off(want.float(), want, tol)[0] <= 1.0
    assert q4tight.off(want, want, tol)[1] * 50 <= 1.0
    a = L // 3
    for keep in (torch.cat([torch.arange(a), torch.arange(a + 160, L)]), torch.cat([torch.arange(L), torch.arange(a, a + 128)])):
        wrong, _ = q4tight.rows_attention(k[keep], v[keep], q, D ** -0.5)
        assert q4tight.off(wrong, want, tol)[0] > 1.0
    assert q4tight.off(torch.zeros_like(want), want, tol)[0] > 50
    assert q4tight.off(want * (1 - 2.0 ** -6), want, tol)[0] > 1.0


def _cut(x):
    """x in 24 bits, cut off towards zero."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.trunc(m * 2.0 ** 24), e - 24)


@pytest.mark.parametrize("apart", [True, False])
def test_sums_that_drift_are_seen(apart):
    """Sums of p s n, n >= 0, a chunk at a time and cut off to 24 bits each time: within the bound
    where they are of two chunks, added up with ordinary rounding, beyond it where they go on."""
    L, D = 40960, 64
    k, v, q = _rows(L, D, G=1, seed=2)
    want, tol = q4tight.rows_attention(k, v, q, D ** -0.5)
    n, s, z = held(v)
    keys = torch.cat([(a * b + c).flatten(-2) for a, b, c in [held(k)]])
    p = torch.softmax(q.double().view(1, D) @ keys.T * D ** -0.5, -1)[0]
    w = p * s[:, 0, 0]
    acc, total = torch.zeros(64, dtype=torch.float64), torch.zeros(64)
    for i in range(0, L, 16):
        acc = _cut(acc + w[i:i + 16] @ n[i:i + 16, 0])
        if apart and (i // 16) % 2 == 1:
            total, acc = total + acc.float(), torch.zeros_like(acc)
    out = total.double() + acc + p @ z[:, 0, 0]
    share = q4tight.off(out.view(1, 1, D), want, tol)[0]
    assert share <= 1.0 if apart else share > 1.0, share


def test_small_values_are_not_covered_by_large_ones_without_weight():
    """A huge token of no weight leaves the bound as it is."""
    k, v, q = _rows(500, 64)
    v, k[:, 0], q[..., 0] = v * 2.0 ** -10, 0.0, 8.0
    want, tol = q4tight.rows_attention(k, v, q, 1.0)
    v[100] *= 2.0 ** 30
    k[100, 0] = -200.0
    want2, tol2 = q4tight.rows_attention(k, v, q, 1.0)
    assert torch.allclose(tol2, tol, rtol=0.2) and torch.allclose(want2, want, rtol=0.2, atol=2.0 ** -12)
