"""gdn_paged_append: a negative number of keys counts as none, for the positions too."""
import pytest
import torch

from paged import Cache, DT, int32
from test_gpu_paged_append import bits, gdn  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_negative_lengths_count_as_none(gdn, dtype, packed):  # noqa: F811
    """Queries of rows of -5 and of the least number of keys, turned as those of a row without
    keys; nothing is kept of their tokens, and the rows next to them have theirs."""
    dt = DT[dtype]
    Hq, Hk, d, page, T = 4, 2, 64, 16, 3
    lens = [20, -5, 0, -2**31, 7]
    B = len(lens)
    f = (1e2 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    q, k, v = (torch.randn(B * T, h, d, device="cuda").to(dt) for h in (Hq, Hk, Hk))
    results = []
    for these in (lens, [max(0, n) for n in lens]):
        cache = Cache(these, Hk, d, page, dt, fill=False)
        rows = dict(cu_seqlens=int32([T * b for b in range(B + 1)])) if packed else dict(T=T)
        qr = gdn.gdn_paged_append(k, v, cache.k, cache.v, cache.table, int32(these), B=B, q=q, inv_freq=f, **rows)
        results.append((qr, cache.k, cache.v))
        assert gdn.gdn_device_errors() == 0
    for a, b in zip(*results):
        assert torch.equal(bits(a), bits(b))
    # and those are what a turn by the positions -3, -2, -1 gives
    pos = int32([-T + t for t in range(T)])
    assert torch.equal(bits(results[0][0][T:2 * T]), bits(gdn.gdn_rotary(q[T:2 * T].contiguous(), pos, f)))
