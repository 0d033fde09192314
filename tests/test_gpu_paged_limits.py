"""The paged cache at the ends of its range: offsets beyond 32 bits, a cache without pages, rows
that are very long or very many, waits that run out, another current stream."""
import pytest
import torch

from paged import Cache, DT, attend, int32, near, turn, turn_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_recurrence_02_gb300 import build, gdn as g
    build.build()
    g.lib()
    return g


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("bf16", 20), ("f32", 16)])
def test_offsets_beyond_32_bits(gdn, dtype, page):
    """Pages 2^30 elements apart: the last one starts 2^33 (bf16: 2^32) bytes into the buffer."""
    dt = DT[dtype]
    Hq, Hk, d = 4, 2, 64
    step = 1 << 30
    if torch.cuda.mem_get_info()[0] < 5 * step * dt.itemsize:
        pytest.skip("not enough memory")
    buf = torch.empty(2 * step + (1 << 20), dtype=dt, device="cuda")
    shape, strides = (3, page, Hk, d), (step, Hk * d, d, 1)
    kp = buf.as_strided(shape, strides)
    vp = buf.as_strided(shape, strides, 1 << 18)
    n = 2 * page + 5
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(n, h, d, generator=g).to(dt).cuda() for h in (Hq, Hk, Hk))
    table, lens = int32([[2, 0, 1]]), int32([n])
    f = (1e4 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    for p in range(3):  # (rows that hold no token hold NaN)
        kp[p], vp[p] = float("nan"), float("nan")
    qr = gdn.gdn_paged_append(k, v, kp, vp, table, lens, B=1, q=q, inv_freq=f)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    kr = gdn.gdn_rotary(k, pos, f)
    assert torch.equal(qr, gdn.gdn_rotary(q, pos, f))
    assert torch.equal(kp[2], kr[:page]) and torch.equal(kp[1, :5], kr[2 * page:]) and torch.equal(vp[0], v[page:2 * page])
    for rows in (n, 1):
        out, _ = gdn.gdn_paged_attention(qr[n - rows:], kp, vp, table, lens, B=1)
        o, _, bound, _ = attend(qr[n - rows:], kr, v, n - rows, d ** -0.5)
        near(out, o, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_cache_without_pages(gdn, dtype):
    dt = DT[dtype]
    kp = torch.empty(0, 16, 2, 64, dtype=dt, device="cuda")
    table = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    q = torch.randn(6, 4, 64, device="cuda").to(dt)
    out, lse = gdn.gdn_paged_attention(q, kp, torch.empty_like(kp), table, int32([0, 7]), B=2, T=3, want_lse=True)
    assert bool((out == 0).all()) and bool(torch.isinf(lse).all()) and gdn.gdn_device_errors() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f16", 128), ("f32", 32)])
def test_one_very_long_row(gdn, dtype, d):
    """A row cut among all CTAs, many parts to a unit; outputs near the mean of the values."""
    dt = DT[dtype]
    n = 100003
    cache = Cache([n], 1, d, 64, dt)
    for T, Hq in ((1, 1), (1, 8), (40, 8)):
        q = torch.randn(T, Hq, d, device="cuda").to(dt)
        out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n]), B=1)
        o, _, bound, _ = attend(q, *cache.rows[0], n - T, d ** -0.5)
        near(out, o, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_very_many_short_rows(gdn, dtype):
    """More rows than the search looks through at once, some without tokens or keys."""
    dt = DT[dtype]
    B, Hq, Hk, d, page = 20000, 2, 1, 32, 8
    g = torch.Generator().manual_seed(2)
    lens = torch.randint(0, 4, (B,), generator=g, dtype=torch.int32)
    new = torch.randint(0, 3, (B,), generator=g, dtype=torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), new.cumsum(0).to(torch.int32)])
    tok = int(cu[-1])
    kp, vp = (torch.randn(B, page, Hk, d, generator=g).to(dt).cuda() for _ in range(2))
    table = torch.randperm(B, generator=g).to(torch.int32)[:, None]
    q = torch.randn(tok, Hq, d, generator=g).to(dt).cuda()
    out, _ = gdn.gdn_paged_attention(q, kp, vp, table.cuda(), lens.cuda(), B=B, cu_seqlens=cu.cuda())
    # all rows at once: up to three keys each
    row = torch.repeat_interleave(torch.arange(B), new.long())
    at = (lens[row] - new[row]).long() + torch.arange(tok) - cu[row].long()
    k, v = (x[table[row, 0].long().cuda(), :3, 0].double() for x in (kp, vp))
    x = torch.einsum("thd,tkd->thk", q.double(), k) * d ** -0.5
    see = (torch.arange(3) <= at[:, None]).cuda()[:, None]
    p = torch.softmax(x.masked_fill(~see, -1e300), -1) * see
    ref = torch.einsum("thk,tkd->thd", p, v)
    mass = torch.einsum("thk,tkd->thd", p, v.abs())
    u = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -20}[dt]
    near(out, ref, 2.5 * u * mass + u * ref.abs() + 2.0 ** -24)


@pytest.mark.parametrize("T", [1, 200])
def test_a_wait_that_runs_out_is_reported(gdn, T):
    """With a limit of a nanosecond the warps give up; the call says so, and the next one is right."""
    from gated_deltanet_recurrence_02_gb300.gdn import GdnError
    Hq, Hk, d, n = 4, 2, 128, 600
    cache = Cache([n], Hk, d, 16, torch.bfloat16)
    q = torch.randn(T, Hq, d, device="cuda").to(torch.bfloat16)
    args = (q, cache.k, cache.v, cache.table, int32([n]))
    gdn.gdn_paged_attention(*args, B=1)
    assert gdn.gdn_device_errors() == 0
    gdn.gdn_set_wait_limit_ns(1)
    try:
        gdn.gdn_paged_attention(*args, B=1)
        with pytest.raises(GdnError) as e:
            gdn.gdn_device_errors()
        assert e.value.status == 6
    finally:
        gdn.gdn_set_wait_limit_ns(0)
    out, _ = gdn.gdn_paged_attention(*args, B=1)
    o, _, bound, _ = attend(q, *cache.rows[0], n - T, d ** -0.5)
    near(out, o, bound)
    assert gdn.gdn_device_errors() == 0


def test_memory_of_a_call_on_another_stream(gdn):
    """Outputs and workspace of a call on another stream, dropped and allocated again at once on
    the current one, are not written over."""
    Hq, Hk, d, n = 8, 2, 128, 3000
    cache = Cache([n] * 4, Hk, d, 16, torch.bfloat16)
    q = torch.randn(4, Hq, d, device="cuda").to(torch.bfloat16)
    args = (q, cache.k, cache.v, cache.table, int32([n] * 4))
    want, _ = gdn.gdn_paged_attention(*args, B=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        out, _ = gdn.gdn_paged_attention(*args, B=4, stream=s)
        junk = [torch.full((1 << 20,), 7.0, device="cuda") for _ in range(3)]
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(out, want)
        del junk
