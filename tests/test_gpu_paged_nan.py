"""gdn_paged_attention: a score that is NaN makes the queries that see it NaN, in every kernel,
wherever the key lies; no other query."""
import math

import pytest
import torch

from paged import Cache, DT, attend, int32, near
from test_gpu_paged_attention import gdn  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu

KINDS = [  # dtype, elements that queries begin behind a boundary of 16 bytes
    ("f32", 0), ("f32", 3), ("bf16", 0), ("f16", 0), ("bf16", 4), ("f16", 3)]


def run(gdn, cache, q, slack, **kw):  # noqa: F811
    T, Hq, d = q.shape
    wide = torch.zeros(T, Hq * d + slack, dtype=q.dtype, device="cuda")
    wide[:, slack:] = q.flatten(1)
    out, lse = gdn.gdn_paged_attention(wide[:, slack:].unflatten(1, (Hq, d)), cache.k, cache.v, cache.table,
                                       int32(cache.lens), B=1, want_lse=True, **kw)
    assert gdn.gdn_device_errors() == 0
    return out, lse


def compare(out, lse, q, k, v, bad):
    """All of `bad` [T, Hq] NaN; the rest as defined; without keys 0 and a log of -inf."""
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    n, T, d = k.shape[0], q.shape[0], q.shape[2]
    none = torch.zeros_like(bad)
    none[:max(0, T - n)] = True
    assert bool((out[none] == 0).all()) and bool((lse[none] == -math.inf).all())
    # (a NaN that a query sees or holds is in none of the others' sums)
    o, l, bound, lse_bound = attend(q.nan_to_num(0), k.nan_to_num(0), v, n - T, d ** -0.5)
    rest = ~bad & ~none
    if rest.any():
        near(out[rest], o[rest], bound[rest])
        near(lse[rest], l[rest], lse_bound[rest], "lse")


@pytest.mark.parametrize("dtype,slack", KINDS)
@pytest.mark.parametrize("T,Hq,Hk,d,n", [(1, 1, 1, 128, 5), (1, 4, 1, 64, 300), (1, 8, 1, 32, 700), (3, 2, 1, 128, 90),
                                         (40, 4, 2, 64, 200), (1300, 8, 2, 64, 1400)])
def test_a_query(gdn, dtype, slack, T, Hq, Hk, d, n):  # noqa: F811
    """One element of one head of one token."""
    cache = Cache([n], Hk, d, 16, DT[dtype])
    q = torch.randn(T, Hq, d, device="cuda").to(DT[dtype])
    q[T // 2, Hq - 1, 3] = math.nan
    bad = torch.zeros(T, Hq, dtype=torch.bool, device="cuda")
    bad[T // 2, Hq - 1] = True
    compare(*run(gdn, cache, q, slack), q, *cache.rows[0], bad)


@pytest.mark.parametrize("dtype,slack", KINDS)
@pytest.mark.parametrize("T,Hq,Hk,d,n,at", [(1, 1, 1, 64, 1, 0), (1, 1, 1, 128, 5, 4), (1, 4, 1, 128, 5, 4),
                                            (1, 8, 1, 64, 40, 33), (2, 4, 1, 32, 70, 69), (4, 1, 1, 64, 3, 1),
                                            (1, 4, 1, 128, 3000, 2999), (40, 4, 2, 64, 200, 180),
                                            (1300, 8, 2, 64, 1400, 900)])
def test_a_key(gdn, dtype, slack, T, Hq, Hk, d, n, at):  # noqa: F811
    """Alone, or one that a group of lanes has alone, or among many: the queries from there on."""
    cache = Cache([n], Hk, d, 16, DT[dtype])
    k, v = cache.rows[0]
    k[at, 0, 5] = math.nan
    cache.put(0, 0, k, v)
    q = torch.randn(T, Hq, d, device="cuda").to(DT[dtype])
    at_or_behind = torch.arange(n - T, n, device="cuda")[:, None] >= at
    of_head_0 = torch.arange(Hq, device="cuda") < Hq // Hk
    compare(*run(gdn, cache, q, slack), q, k, v, at_or_behind & of_head_0)
