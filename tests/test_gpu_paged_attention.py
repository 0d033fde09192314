"""gdn_paged_attention against its definition in 64 bits, within bounds derived in paged.py."""
import math

import pytest
import torch

from paged import Cache, DT, attend, int32, near, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_recurrence_02_gb300 import build, gdn as g
    build.build()
    g.lib()
    return g


def check(gdn, new, lens, Hq, Hk, d, page, dtype, causal=True, window=0, layout="psh", packed=True, tail=0, slack=0,
          scale=None, gain=1.0, seed=0):
    dt = DT[dtype]
    B, tok = len(new), sum(new)
    cache = Cache(lens, Hk, d, page, dt, seed, layout)
    g = torch.Generator().manual_seed(seed + 1)
    wide = (gain * torch.randn(tok + tail, Hq * d + slack, generator=g)).to(dt).cuda()
    q = wide[:, slack:].unflatten(1, (Hq, d))
    out = torch.full((tok + tail, Hq, d), 7.0, dtype=dt, device="cuda")
    lse = torch.full((tok + tail, Hq), 7.0, device="cuda")
    rows = dict(cu_seqlens=int32(starts(new))) if packed else dict(T=new[0])
    got, got_lse = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32(lens), B=B, causal=causal,
                                           window=window, scale=scale, out=out, lse=lse, **rows)
    assert got is out and got_lse is lse and gdn.gdn_device_errors() == 0
    assert bool((out[tok:] == 7.0).all()) and bool((lse[tok:] == 7.0).all())
    for b, (n, m) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        r = slice(starts(new)[b], starts(new)[b] + n)
        k, v = cache.rows[b]
        o, l, bound, lse_bound = attend(q[r], k, v, max(m, 0) - n, d ** -0.5 if scale is None else scale, causal, window)
        near(out[r], o, bound, f"row {b}")
        none = torch.isinf(l)
        assert torch.equal(torch.isinf(lse[r]), none) and bool((out[r][none] == 0).all())
        near(lse[r].nan_to_num(0, 0, 0), l.nan_to_num(0, 0, 0), lse_bound, f"lse of row {b}")


CASES = [
    dict(new=[1], lens=[1], Hq=1, Hk=1, d=64, page=16),
    dict(new=[1], lens=[0], Hq=2, Hk=1, d=64, page=16),                       # no keys at all
    dict(new=[1, 1, 1], lens=[17, 128, 129], Hq=8, Hk=2, d=128, page=16, packed=False),
    dict(new=[1] * 5, lens=[1000, 64, 63, 0, 257], Hq=4, Hk=4, d=64, page=32, packed=False),
    dict(new=[1], lens=[3001], Hq=8, Hk=1, d=128, page=64, packed=False),     # one row, cut among CTAs
    dict(new=[5, 5], lens=[700, 5], Hq=12, Hk=2, d=128, page=64, packed=False),
    dict(new=[5], lens=[2], Hq=3, Hk=1, d=32, page=16, packed=False),         # more tokens than keys
    dict(new=[300], lens=[300], Hq=4, Hk=2, d=64, page=16),
    dict(new=[200, 0, 3, 130], lens=[900, 70, 3, 131], Hq=6, Hk=2, d=128, page=32, tail=9),
    dict(new=[129, 64], lens=[129, 640], Hq=5, Hk=1, d=32, page=128),
    dict(new=[77], lens=[500], Hq=14, Hk=2, d=64, page=16, slack=64),         # 7 query heads a key head
    dict(new=[40, 500], lens=[40, 555], Hq=2, Hk=2, d=128, page=48, layout="phs"),
    dict(new=[257], lens=[258], Hq=3, Hk=3, d=64, page=8, layout="kv"),
    dict(new=[33], lens=[100], Hq=4, Hk=2, d=64, page=7),                     # pages of odd sizes
    dict(new=[9], lens=[70], Hq=4, Hk=2, d=128, page=1, layout="hps"),
    dict(new=[50], lens=[90], Hq=4, Hk=2, d=64, page=16, slack=3),            # rows on no boundary
    dict(new=[2], lens=[400], Hq=200, Hk=1, d=64, page=16),                   # very wide groups
    dict(new=[3], lens=[300], Hq=64, Hk=2, d=128, page=16),
    dict(new=[1, 1], lens=[700, 333], Hq=5, Hk=1, d=128, page=20, packed=False),  # 5 rows of 8
    dict(new=[3], lens=[500], Hq=3, Hk=1, d=32, page=24, packed=False),       # 9 rows of 16
    dict(new=[2], lens=[500], Hq=4, Hk=2, d=32, page=12, packed=False),       # 4 rows
    dict(new=[1] * 9, lens=[100] * 9, Hq=8, Hk=1, d=64, page=20, packed=False, window=30),
    dict(new=[2, 2], lens=[1, 9], Hq=4, Hk=1, d=128, page=16, packed=False, causal=False),
    dict(new=[100, 20], lens=[400, 20], Hq=4, Hk=2, d=64, page=16, window=1),
    dict(new=[100, 20], lens=[400, 20], Hq=4, Hk=2, d=128, page=16, window=37),
    dict(new=[300], lens=[900], Hq=8, Hk=2, d=64, page=64, window=256),
    dict(new=[1, 1], lens=[900, 10], Hq=8, Hk=2, d=128, page=16, window=100, packed=False),
    dict(new=[30], lens=[900], Hq=4, Hk=2, d=64, page=16, window=5000),
    dict(new=[60, 7], lens=[300, 0], Hq=4, Hk=2, d=64, page=16, causal=False),
    dict(new=[200], lens=[150], Hq=4, Hk=4, d=128, page=32, causal=False),
    dict(new=[64], lens=[320], Hq=4, Hk=2, d=64, page=16, scale=-0.5),
    dict(new=[64], lens=[320], Hq=4, Hk=2, d=64, page=16, scale=0.0),
    dict(new=[64, 1], lens=[320, 200], Hq=4, Hk=2, d=64, page=16, gain=20.0),  # one key takes nearly all
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("case", CASES)
def test_matches_definition(gdn, dtype, case):
    check(gdn, dtype=dtype, **case)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_ragged_rows(gdn, dtype):
    g = torch.Generator().manual_seed(5)
    new = torch.randint(0, 6, (400,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(new, torch.randint(0, 300, (400,), generator=g))]
    check(gdn, new, lens, 4, 2, 64, 16, dtype, tail=3)


@pytest.mark.parametrize("new,longest,d,Hq", [(1, 1500, 128, 8), (1, 1500, 64, 8), (3, 700, 128, 12), (90, 400, 128, 8), (90, 400, 64, 8)])
def test_many_rows_a_CTA(gdn, new, longest, d, Hq):
    """Rows of up to a dozen tiles, several of them and parts of others for each CTA."""
    g = torch.Generator().manual_seed(6)
    lens = [int(x) for x in torch.randint(1, longest, (300 if new < 10 else 60,), generator=g)]
    check(gdn, [new] * len(lens), lens, Hq, 2, d, 16, "bf16", packed=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_keys_of_growing_size(gdn, dtype):
    """The maximum grows tile after tile, so everything summed before is scaled down."""
    dt = DT[dtype]
    Hq, Hk, d, n = 4, 2, 64, 1200
    cache = Cache([n], Hk, d, 16, dt)
    k, v = cache.rows[0]
    q = torch.randn(40, Hq, d, device="cuda").to(dt)
    k.copy_((q[0].unflatten(0, (Hk, 2)).float().mean(1) * torch.linspace(0, 12, n, device="cuda")[:, None, None]).to(dt))
    cache.put(0, 0, k, v)
    out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n]), B=1)
    o, _, bound, _ = attend(q, k, v, n - 40, d ** -0.5)
    near(out, o, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new,Hq", [(1, 4), (150, 4)])
def test_what_is_not_finite_stays_with_its_row(gdn, dtype, new, Hq):
    """NaN and infinities in one row's keys and values do not reach other rows, and what no
    query of the row sees (behind the window's first tile) does not reach the row."""
    dt = DT[dtype]
    Hk, d, n = 2, 64, 600
    cache = Cache([n, n], Hk, d, 16, dt)
    clean = [x.clone() for x in cache.rows[1]]
    k, v = cache.rows[0]
    k[10] = math.nan
    v[11] = math.inf
    cache.put(0, 0, k, v)
    q = torch.randn(2 * new, Hq, d, device="cuda").to(dt)
    kw = dict(B=2, T=new)
    out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n, n]), **kw)
    o, _, bound, _ = attend(q[new:], *clean, n - new, d ** -0.5)
    near(out[new:], o, bound)
    assert not bool(torch.isfinite(out[:new]).any())
    out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n, n]), window=200, **kw)
    k[:128], v[:128] = 0, 0
    o, _, bound, _ = attend(q[:new], k, v, n - new, d ** -0.5, window=200)
    near(out[:new], o, bound)


def test_masked_by_the_lowest_value(gdn):
    """Keys that score the type's lowest value weigh nothing next to others; where there are no
    others, equal scores of -2^19 weigh the same."""
    d, n = 64, 200
    for dt in (torch.bfloat16, torch.float32):
        cache = Cache([n], 1, d, 16, dt)
        k, v = cache.rows[0]
        q = torch.ones(1, 1, d, device="cuda", dtype=dt)
        k[:] = 0
        k[:150, :, 0] = torch.finfo(dt).min
        cache.put(0, 0, k, v)
        out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n]), B=1, scale=1.0)
        ref = v[150:, 0].double().mean(0)
        u = 2.0 ** -8 if dt == torch.bfloat16 else 2.0 ** -20
        near(out[0, 0], ref, 2 * u * v[150:, 0].double().abs().mean(0) + u * ref.abs())
        out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([150]), B=1,
                                         scale=2.0 ** 19 / -torch.finfo(dt).min)
        ref = v[:150, 0].double().mean(0)
        near(out[0, 0], ref, 2 * u * v[:150, 0].double().abs().mean(0) + u * ref.abs())


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("f32", 16), ("f16", 7)])
def test_missing_pages_count_as_zeros(gdn, dtype, page):
    dt = DT[dtype]
    d, n = 64, 100
    cache = Cache([n], 1, d, page, dt)
    k, v = cache.rows[0]
    q = torch.randn(3, 2, d, device="cuda").to(dt)
    cache.table[0, 1] = -1
    cache.table[0, 3] = cache.k.shape[0]
    for i in (1, 3):
        k[i * page:(i + 1) * page] = 0
        v[i * page:(i + 1) * page] = 0
    out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n]), B=1)
    assert gdn.gdn_device_errors() == 1
    o, _, bound, _ = attend(q, k, v, n - 3, d ** -0.5)
    near(out, o, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_past_the_table(gdn, dtype):
    """Keys past the table's room do not exist; queries keep their positions."""
    dt = DT[dtype]
    d = 64
    cache = Cache([64], 1, d, 16, dt, extra=0)
    table = cache.table[:, :4].contiguous()
    k, v = cache.rows[0]
    q = torch.randn(20, 2, d, device="cuda").to(dt)
    out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, table, int32([70]), B=1)
    o, _, bound, _ = attend(q, k, v, 50, d ** -0.5)
    near(out, o, bound)
    out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, table, int32([-3]), B=1)
    assert bool((out == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_result_every_time_and_pages_shared(gdn, dtype):
    """Rows that share a prefix's pages, and the same bits call after call."""
    dt = DT[dtype]
    Hq, Hk, d, n = 8, 2, 128, 700
    cache = Cache([n] * 3, Hk, d, 16, dt)
    shared = 20
    cache.table[1, :shared] = cache.table[0, :shared]
    cache.table[2] = cache.table[0]
    q = torch.randn(6, Hq, d, device="cuda").to(dt)
    runs = [gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n] * 3), B=3, T=2)[0] for _ in range(4)]
    assert all(torch.equal(runs[0], x) for x in runs)
    for b in range(3):
        k, v = (x.clone() for x in cache.rows[b if b < 2 else 0])
        if b == 1:
            k[:shared * 16], v[:shared * 16] = (x[:shared * 16] for x in cache.rows[0])
        o, _, bound, _ = attend(q[2 * b:2 * b + 2], k, v, n - 2, d ** -0.5)
        near(runs[0][2 * b:2 * b + 2], o, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_streams_and_graph(gdn, dtype):
    """Two calls at once on two streams, and a captured call that follows lengths that change."""
    dt = DT[dtype]
    Hq, Hk, d, B = 8, 2, 64, 4
    cache = Cache([900, 500, 30, 777], Hk, d, 16, dt)
    ln = int32(cache.lens)
    q = torch.randn(B, Hq, d, device="cuda").to(dt)
    want, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, ln, B=B)
    s = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for x in s:
        x.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for x in s:
            got.append(gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, ln, B=B, stream=x)[0])
    for x in s:
        torch.cuda.current_stream().wait_stream(x)
    assert all(torch.equal(want, x) for x in got)
    out = torch.empty_like(q)
    ws = torch.empty(gdn.gdn_paged_attention_workspace_size(B, 1, Hq, Hk, d, dt), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, ln, B=B, out=out, workspace=ws)
    for lens in ([900, 500, 30, 777], [1, 499, 16, 300]):
        ln.copy_(int32(lens))
        graph.replay()
        for b, n in enumerate(lens):
            k, v = cache.rows[b]
            o, _, bound, _ = attend(q[b:b + 1], k[:n], v[:n], n - 1, d ** -0.5)
            near(out[b:b + 1], o, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_layer_from_prompt_to_drafts(gdn, dtype):
    """Append and attention as a program calls them: a ragged prompt, single tokens, a pass over
    drafts of which some are taken back, against the whole rows at once."""
    dt = DT[dtype]
    Hq, Hk, d, page, B = 8, 2, 64, 16, 3
    f = (1e4 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    cache = Cache([160] * B, Hk, d, page, dt, fill=False)
    have = [0] * B
    rows = [[torch.empty(0, Hk, d, device="cuda", dtype=dt) for _ in range(2)] for _ in range(B)]
    g = torch.Generator().manual_seed(8)

    def step(new, keep=None):
        tok = sum(new)
        q, k, v = (torch.randn(tok, h, d, generator=g).to(dt).cuda() for h in (Hq, Hk, Hk))
        lens = int32([h + n for h, n in zip(have, new)])
        kw = dict(B=B, T=new[0]) if len(set(new)) == 1 else dict(B=B, cu_seqlens=int32(starts(new)))
        qr = gdn.gdn_paged_append(k, v, cache.k, cache.v, cache.table, lens, q=q, inv_freq=f, **kw)
        out, _ = gdn.gdn_paged_attention(qr, cache.k, cache.v, cache.table, lens, **kw)
        for b, n in enumerate(new):
            r = slice(starts(new)[b], starts(new)[b] + n)
            pos = torch.arange(have[b], have[b] + n, dtype=torch.int32, device="cuda")
            ks = torch.cat([rows[b][0], gdn.gdn_rotary(k[r], pos, f)])
            vs = torch.cat([rows[b][1], v[r]])
            assert torch.equal(qr[r], gdn.gdn_rotary(q[r], pos, f))
            if n:
                o, _, bound, _ = attend(qr[r], ks, vs, have[b], d ** -0.5)
                near(out[r], o, bound)
            took = n if keep is None else keep[b]
            rows[b] = [ks[:have[b] + took], vs[:have[b] + took]]
            have[b] += took

    step([90, 17, 1])
    for _ in range(3):
        step([1, 1, 1])
    step([5, 5, 5], keep=[1, 5, 3])
    step([5, 5, 5], keep=[2, 2, 2])
    step([20, 0, 40])
    assert gdn.gdn_device_errors() == 0
