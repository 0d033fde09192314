"""gdn_paged_append: what lands in which slot, rotated or not, and what stays as it was."""
import pytest
import torch

from paged import Cache, DT, int32, near, starts, turn, turn_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_recurrence_02_gb300 import build, gdn as g
    build.build()
    g.lib()
    return g


def freq(half):
    return (1e6 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda()


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


def check(gdn, new, lens, Hq, Hk, d, page, dtype, R, A=0, pairs=False, layout="psh", packed=True, tail=0, seed=0):
    """Appends the last new[b] tokens of rows of lens[b] keys and compares pages and queries."""
    dt = DT[dtype]
    B, tok = len(new), sum(new)
    cache = Cache(lens, Hk, d, page, dt, seed, layout, fill=False)
    g = torch.Generator().manual_seed(seed + 1)
    wide = torch.randn(tok + tail, (Hq + 2 * Hk) * d, generator=g).to(dt).cuda()
    q, k, v = (x.unflatten(1, (-1, d)) for x in wide.split([Hq * d, Hk * d, Hk * d], 1))
    at = torch.cat([torch.arange(m - n, m) for n, m in zip(new, lens)] + [torch.zeros(tail, dtype=torch.long)])
    f = freq(R // 2) if R else None
    pos = axes = None
    if A:
        pos = torch.randint(0, 4000, (A, tok + tail), generator=g, dtype=torch.int32).cuda()
        axes = int32([i * A // (R // 2) for i in range(R // 2)])
    kp0, vp0 = cache.k.clone(), cache.v.clone()
    q_out = torch.full((tok + tail, Hq, d), 7.0, dtype=dt, device="cuda")
    rows = dict(cu_seqlens=int32(starts(new))) if packed else dict(T=new[0])
    got = gdn.gdn_paged_append(k, v, cache.k, cache.v, cache.table, int32(lens), B=B, q=q, q_out=q_out, inv_freq=f,
                               positions=pos, axes=axes, pairs=pairs, **rows)
    assert got is q_out and gdn.gdn_device_errors() == 0
    p64 = at[None].cuda() if pos is None else pos
    kr = turn(k, p64, f, axes, pairs) if R else k.double()
    qr = turn(q, p64, f, axes, pairs) if R else q.double()
    near(q_out[:tok], qr[:tok], turn_bound(q, qr, R // 2, pairs)[:tok], "q")
    assert bool((q_out[tok:] == 7.0).all())
    kept = torch.ones(kp0.shape[:2], dtype=torch.bool)
    for b, (n, m) in enumerate(zip(new, lens)):
        lo = max(0, m - n)
        if m <= lo:
            continue
        gk, gv = cache.get(b, lo, m)
        r = slice(starts(new)[b] + n - (m - lo), starts(new)[b] + n)
        near(gk, kr[r], turn_bound(k, kr, R // 2, pairs)[r], f"k of row {b}")
        assert torch.equal(gv, v[r])
        pg, sl = cache.places(b, lo, m)
        kept[pg.cpu(), sl.cpu()] = False
    # nothing else was written
    assert torch.equal(bits(cache.k)[kept.cuda()], bits(kp0)[kept.cuda()])
    assert torch.equal(bits(cache.v)[kept.cuda()], bits(vp0)[kept.cuda()])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", [
    dict(new=[1], lens=[1], Hq=2, Hk=1, d=64, page=16, R=64),
    dict(new=[1, 1, 1], lens=[17, 16, 33], Hq=8, Hk=2, d=128, page=16, R=128, packed=False),
    dict(new=[4, 0, 9, 1], lens=[4, 5, 40, 1000], Hq=6, Hk=2, d=64, page=20, R=32, pairs=True),
    dict(new=[100, 37], lens=[100, 90], Hq=4, Hk=4, d=128, page=64, R=96, A=3, layout="phs"),
    dict(new=[5, 5], lens=[3, 0], Hq=3, Hk=1, d=32, page=8, R=32, packed=False),   # more tokens than keys
    dict(new=[70], lens=[200], Hq=2, Hk=2, d=128, page=1, R=0, layout="kv"),
    dict(new=[33, 2], lens=[40, 2], Hq=5, Hk=5, d=80, page=7, R=46, A=2, layout="hps", tail=6),
    dict(new=[0, 0, 3, 0], lens=[9, 0, 3, 2], Hq=2, Hk=1, d=5, page=3, R=4, tail=2),
    dict(new=[1500, 1], lens=[1500, 3], Hq=2, Hk=1, d=64, page=128, R=64),
])
def test_matches_definition(gdn, dtype, case):
    check(gdn, dtype=dtype, **case)


def test_many_rows(gdn):
    g = torch.Generator().manual_seed(3)
    new = torch.randint(0, 4, (700,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 50, (700,), generator=g))]
    check(gdn, new, lens, 2, 1, 32, 16, "bf16", 32, tail=5)


def test_without_queries_and_in_a_fused_buffer(gdn):
    Hq, Hk, d, page = 4, 2, 64, 16
    new, lens = [5, 3], [20, 3]
    wide = torch.randn(8, (Hq + 2 * Hk) * d, device="cuda").to(torch.bfloat16)
    before = wide.clone()
    q, k, v = (x.unflatten(1, (-1, d)) for x in wide.split([Hq * d, Hk * d, Hk * d], 1))
    a, b = (Cache(lens, Hk, d, page, torch.bfloat16, fill=False) for _ in range(2))
    cu, ln, f = int32(starts(new)), int32(lens), freq(32)
    assert gdn.gdn_paged_append(k, v, a.k, a.v, a.table, ln, B=2, cu_seqlens=cu, inv_freq=f) is None
    want = gdn.gdn_rotary(q, torch.cat([torch.arange(15, 20), torch.arange(3)]).int().cuda(), f)
    got = gdn.gdn_paged_append(k, v, b.k, b.v, b.table, ln, B=2, cu_seqlens=cu, q=q, q_out=q, inv_freq=f)
    assert got is q and torch.equal(q, want)
    assert torch.equal(bits(a.k), bits(b.k)) and torch.equal(bits(a.v), bits(b.v))
    assert torch.equal(wide[:, Hq * d:], before[:, Hq * d:])


def test_missing_pages_are_reported_and_left_out(gdn):
    Hk, d, page = 2, 64, 16
    cache = Cache([40, 40], Hk, d, page, torch.float16, fill=False)
    cache.table[0, 1] = -1
    cache.table[1, 2] = cache.k.shape[0]
    k, v = (torch.randn(80, Hk, d, device="cuda").half() for _ in range(2))
    gdn.gdn_paged_append(k, v, cache.k, cache.v, cache.table, int32([40, 40]), B=2, T=40)
    assert gdn.gdn_device_errors() == 1
    for b, there in ((0, [0, 2]), (1, [0, 1])):
        for i in there:
            n = min(page, 40 - i * page)
            page_id = int(cache.host_table[b, i])
            r = slice(b * 40 + i * page, b * 40 + i * page + n)
            assert torch.equal(cache.k[page_id, :n], k[r]) and torch.equal(cache.v[page_id, :n], v[r])
    # a length that the table has no room for: the tokens behind it are left out
    cache = Cache([16], Hk, d, page, torch.float16, fill=False, extra=0)
    table = cache.table[:, :1].contiguous()
    gdn.gdn_paged_append(k[:4], v[:4], cache.k, cache.v, table, int32([18]), B=1, T=4)
    assert gdn.gdn_device_errors() == 1
    assert torch.equal(cache.k[int(table[0, 0]), 14:16], k[:2])


def test_graph(gdn):
    """A captured append follows lengths and tables that change on the device."""
    Hk, d, page, B = 2, 64, 16, 3
    lens = [20, 5, 33]
    cache = Cache([64] * B, Hk, d, page, torch.bfloat16, fill=False)
    k, v, q = (torch.randn(B, h, d, device="cuda").to(torch.bfloat16) for h in (Hk, Hk, 4))
    ln, f = int32(lens), freq(32)
    q_out = torch.empty_like(q)
    args = dict(B=B, T=1, q=q, q_out=q_out, inv_freq=f)
    gdn.gdn_paged_append(k, v, cache.k, cache.v, cache.table, ln, **args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_paged_append(k, v, cache.k, cache.v, cache.table, ln, **args)
    for step in range(3):
        ln += 1
        k.normal_()
        graph.replay()
        for b in range(B):
            p = lens[b] + step
            gk, _ = cache.get(b, p, p + 1)
            ref = turn(k[b:b + 1], int32([[p]]), f)
            near(gk, ref, turn_bound(k[b:b + 1], ref, 32))


def test_no_tokens(gdn):
    cache = Cache([4], 1, 32, 8, torch.float32, fill=False)
    k = torch.empty(0, 1, 32, device="cuda")
    assert gdn.gdn_paged_append(k, k, cache.k, cache.v, cache.table, int32([4]), B=1, T=0, q=k).shape == (0, 1, 32)
