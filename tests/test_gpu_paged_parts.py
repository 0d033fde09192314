"""A unit that is cut among all CTAs: that each of its many parts is there, once and with its
weight.  Each feature of the values is there for a few stretches of keys alone, shorter than a
part, so a part too many or too few changes some outputs by a large share of themselves."""
import pytest
import torch

from paged import DT, U, Cache, int32, near
from test_gpu_paged_attention import gdn  # noqa: F401  (a fixture)


def definition(q, k, v, first, left_out=None):
    """Outputs and logs in 64 bits of one key head, causal; without the keys of a range."""
    n, t, d = k.shape[0], q.shape[0], q.shape[2]
    x = torch.einsum("thd,nd->thn", q.double(), k[:, 0].double()) * d ** -0.5
    hidden = torch.arange(n, device=q.device) > torch.arange(first, first + t, device=q.device)[:, None]
    if left_out is not None:
        hidden[:, left_out[0]:left_out[1]] = True
    x = x.masked_fill(hidden[:, None], -torch.inf)
    lse = torch.logsumexp(x, -1)
    return torch.einsum("thn,nd->thd", torch.exp(x - lse[..., None]), v[:, 0].double()), lse


def bounds(q, k, v, o, lse, depth):
    """As in paged.attend, but a sum is as deep as a part's keys and the parts, not as the row:
    depth additions of fp32, each off by 2^-24 of the magnitudes so far."""
    d = q.shape[2]
    size = q.double().abs().amax() * k.double().abs().sum(-1).amax() * d ** -0.5
    weights = 2 * (d + 4) * 2.0 ** -24 * size + (depth + 16) * 2.0 ** -23
    u = U[q.dtype]
    # (values are not negative: outputs are their own sums of magnitudes)
    return ((u if q.dtype != torch.float32 else 0) + weights + u * (1 + 2 * u)) * o.abs() + 2.0 ** -25, weights + 2.0 ** -22 * lse.abs()


def values(n, d, parts, dt, dev):
    """[n, 1, d]: of the key's stretch (a third of a part) one feature 1 or a little more."""
    j = torch.arange(n, device=dev)
    stretch = j * (3 * parts) // n
    v = torch.zeros(n, 1, d, dtype=dt, device=dev)
    v[j, 0, stretch % d] = (1 + j % 7 / 8).to(dt)
    return v


CASES = [("bf16", 64, 152), ("bf16", 128, 152), ("f16", 128, 152), ("f16", 32, 152), ("f32", 32, 304), ("f32", 128, 304)]


@pytest.mark.parametrize("dtype,d,parts", CASES)
def test_the_bound_tells_a_part_left_out(dtype, d, parts):
    """On the CPU: the definition without any of some parts is beyond the bound."""
    n, dt = 20003, DT[dtype]
    g = torch.Generator().manual_seed(1)
    k = torch.randn(n, 1, d, generator=g).to(dt)
    v = values(n, d, parts, dt, "cpu")
    q = torch.randn(1, 2, d, generator=g).to(dt)
    o, lse = definition(q, k, v, n - 1)
    bound, lse_bound = bounds(q, k, v, o, lse, n // parts + parts)
    for x in (0, 1, parts // 2, parts - 2, parts - 1):
        o2, lse2 = definition(q, k, v, n - 1, (x * n // parts, (x + 1) * n // parts))
        assert bool(((o2 - o).abs() > bound).any(-1).all()) and bool(((lse2 - lse).abs() > lse_bound).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,parts", CASES)
@pytest.mark.parametrize("T,Hq", [(1, 1), (1, 8), (5, 2), (40, 8)])
def test_every_part_counts(gdn, T, Hq, dtype, d, parts):  # noqa: F811
    dt, n = DT[dtype], 100003
    cache = Cache([n], 1, d, 64, dt)
    k = cache.rows[0][0]
    v = values(n, d, parts, dt, "cuda")
    cache.put(0, 0, k, v)
    q = torch.randn(T, Hq, d, device="cuda").to(dt)
    out, lse = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n]), B=1, want_lse=True)
    o, l = definition(q, k, v, n - T)
    bound, lse_bound = bounds(q, k, v, o, l, n // parts + parts)
    near(out, o, bound)
    near(lse, l, lse_bound, "lse")
