"""gdn_paged_attention's paths one by one, each with cases that are known to reach it: units of
one and of two blocks of query rows, pages that are copied 16 bytes a lane, and 16-bit rows
on no 16-byte boundary."""
import math

import pytest
import torch

from paged import DT, Cache, attend, int32, near
from test_gpu_paged_attention import check, gdn  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def blocks_of(new, Hq, Hk):
    """Blocks of up to 128 query rows that a batch has by its mean number of tokens, and whether
    units have two each: where there are as many as multiprocessors."""
    G = Hq // Hk
    per_key = -(-G // 128)
    tokens = 128 // -(-G // per_key)
    blocks = -(-(-(-sum(new) // len(new))) // tokens)
    n = blocks * len(new) * Hk * per_key
    return n, blocks > 1 and n >= torch.cuda.get_device_properties(0).multi_processor_count


def tiles_a_cta(new, lens, Hq, Hk):
    """Tiles of 128 keys that a CTA has on average, causal, no window, at the least."""
    n, two = blocks_of(new, Hq, Hk)
    units = n / (len(new) * (2 if two else 1))  # of a row
    return sum(units * m / 256 for m in lens) / torch.cuda.get_device_properties(0).multi_processor_count


ROWS = {  # tokens and keys of the rows, and whether units have two blocks
    "single": ([1] * 150, [400 + 13 * b for b in range(150)], False),
    "chunks": ([300] * 26, [300 + 60 * b for b in range(26)], True),
}


@pytest.mark.parametrize("dtype,d,page", [("bf16", 64, 20), ("f16", 128, 7), ("bf16", 128, 12), ("f16", 32, 1)])
@pytest.mark.parametrize("rows", ROWS)
def test_pages_of_odd_sizes_over_many_tiles(gdn, rows, dtype, d, page):  # noqa: F811
    """More tiles a CTA than stages in flight, so that copies wait for stages to come free."""
    new, lens, two = ROWS[rows]
    assert blocks_of(new, 8, 2)[1] == two and tiles_a_cta(new, lens, 8, 2) > 6
    check(gdn, new, lens, 8, 2, d, page, dtype, packed=False)


# tokens and keys of ragged rows: none, one, blocks of 32 tokens that are full and that are not,
# units whose second block has no tokens, rows with more tokens than keys and without keys
NEW = [330, 0, 61, 500, 33, 129, 280, 1, 700, 97, 210, 64]
LENS = [900, 70, 61, 777, 10, 640, 281, 300, 702, 1300, 0, 64]

TWO_BLOCKS = [
    dict(Hq=8, Hk=2, d=64, page=16, tail=9),
    dict(Hq=8, Hk=2, d=128, page=64, layout="phs"),
    dict(Hq=8, Hk=2, d=32, page=8, layout="kv"),
    dict(Hq=6, Hk=2, d=64, page=32, slack=64, tail=1, new=NEW * 2, lens=LENS * 2),  # 42 tokens a block
    dict(Hq=8, Hk=2, d=128, page=16, window=37),
    dict(Hq=8, Hk=2, d=64, page=16, window=1),
    dict(Hq=8, Hk=2, d=64, page=128, window=256),
    dict(Hq=8, Hk=2, d=32, page=20, window=130),
    dict(Hq=8, Hk=2, d=64, page=16, causal=False),
    dict(Hq=8, Hk=2, d=128, page=20, causal=False, tail=5),
    dict(Hq=8, Hk=2, d=64, page=16, scale=-0.5),
    dict(Hq=8, Hk=2, d=128, page=16, scale=0.0),
    dict(Hq=8, Hk=2, d=64, page=16, gain=20.0),
    dict(Hq=8, Hk=2, d=128, page=7, window=300),
    dict(Hq=200, Hk=1, d=64, page=16, new=[4, 5, 3, 4] * 5, lens=[300, 5, 129, 2] * 5),  # a token a block
    dict(Hq=3, Hk=3, d=64, page=16, new=[257] * 18, lens=[258 + 40 * b for b in range(18)], packed=False),
    dict(Hq=8, Hk=2, d=128, page=16, new=[280] * 9, lens=[100 + 90 * b for b in range(9)], packed=False, window=64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", TWO_BLOCKS)
def test_units_of_two_blocks(gdn, case, dtype):  # noqa: F811
    case = {**dict(new=NEW, lens=LENS), **case}
    assert blocks_of(case["new"], case["Hq"], case["Hk"])[1]
    check(gdn, dtype=dtype, **case)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
def test_what_is_not_finite_and_two_blocks(gdn, dtype, d):  # noqa: F811
    """NaN and infinities in one row's keys and values do not reach the other row, and what no
    query of the row sees does not reach the row."""
    dt, Hq, Hk, new, n = DT[dtype], 8, 2, 1300, 1900
    assert blocks_of([new] * 2, Hq, Hk)[1]
    cache = Cache([n, n], Hk, d, 16, dt)
    clean = [x.clone() for x in cache.rows[1]]
    k, v = cache.rows[0]
    k[10], v[11] = math.nan, math.inf
    cache.put(0, 0, k, v)
    q = torch.randn(2 * new, Hq, d, device="cuda").to(dt)
    args = (q, cache.k, cache.v, cache.table, int32([n, n]))
    out, _ = gdn.gdn_paged_attention(*args, B=2, T=new)
    o, _, bound, _ = attend(q[new:], *clean, n - new, d ** -0.5)
    near(out[new:], o, bound)
    assert not bool(torch.isfinite(out[:new]).any())
    out, _ = gdn.gdn_paged_attention(*args, B=2, T=new, window=200)
    k[:128], v[:128] = 0, 0
    o, _, bound, _ = attend(q[:new], k, v, n - new, d ** -0.5, window=200)
    near(out[:new], o, bound)


@pytest.mark.parametrize("dtype,page", [("bf16", 16), ("f16", 20)])
def test_missing_pages_and_two_blocks(gdn, dtype, page):  # noqa: F811
    """Pages that are not there count as zeros, and keys past the table's room do not exist."""
    dt, Hq, Hk, d, new, n = DT[dtype], 16, 4, 64, 1300, 1400
    assert blocks_of([new], Hq, Hk)[1]
    cache = Cache([n], Hk, d, page, dt)
    k, v = cache.rows[0]
    q = torch.randn(new, Hq, d, device="cuda").to(dt)
    cache.table[0, 1], cache.table[0, 60] = -1, cache.k.shape[0]
    for i in (1, 60):
        k[i * page:(i + 1) * page], v[i * page:(i + 1) * page] = 0, 0
    out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table, int32([n]), B=1)
    assert gdn.gdn_device_errors() == 1
    o, _, bound, _ = attend(q, k, v, n - new, d ** -0.5)
    near(out, o, bound)
    cache.table[0, 1] = cache.table[0, 60] = cache.table[0, 0]
    for i in (1, 60):
        k[i * page:(i + 1) * page], v[i * page:(i + 1) * page] = k[:page], v[:page]
    width = 50
    out, _ = gdn.gdn_paged_attention(q, cache.k, cache.v, cache.table[:, :width].contiguous(), int32([n]), B=1)
    o, _, bound, _ = attend(q, k[:width * page], v[:width * page], n - new, d ** -0.5)
    near(out, o, bound)
    assert gdn.gdn_device_errors() == 0


@pytest.mark.parametrize("T,page", [(1, 20), (200, 20), (2500, 16), (2500, 20)])
def test_waits_that_run_out(gdn, T, page):  # noqa: F811
    """With a limit of a nanosecond the warps give up; the call says so, and the next one is right."""
    Hq, Hk, d, n = 8, 2, 128, 2600
    assert blocks_of([T], Hq, Hk)[1] == (T == 2500)
    cache = Cache([n], Hk, d, page, torch.bfloat16)
    q = torch.randn(T, Hq, d, device="cuda").to(torch.bfloat16)
    args = (q, cache.k, cache.v, cache.table, int32([n]))
    o, _, bound, _ = attend(q, *cache.rows[0], n - T, d ** -0.5)
    near(gdn.gdn_paged_attention(*args, B=1)[0], o, bound)
    assert gdn.gdn_device_errors() == 0
    gdn.gdn_set_wait_limit_ns(1)
    try:
        gdn.gdn_paged_attention(*args, B=1)
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_device_errors()
        assert e.value.status == 6
    finally:
        gdn.gdn_set_wait_limit_ns(0)
    near(gdn.gdn_paged_attention(*args, B=1)[0], o, bound)
    assert gdn.gdn_device_errors() == 0


CUDA_CORES = [  # of up to 4, 8 and 64 query rows a unit
    dict(new=[1] * 3, lens=[700, 1, 64], Hq=4, Hk=1, page=16, packed=False),
    dict(new=[2, 2], lens=[400, 0], Hq=4, Hk=2, page=12, packed=False, window=70),
    dict(new=[4], lens=[500], Hq=1, Hk=1, page=1, causal=False),
    dict(new=[1] * 20, lens=[100 + 37 * b for b in range(20)], Hq=8, Hk=1, page=20, packed=False),
    dict(new=[5, 0, 2], lens=[900, 30, 1], Hq=5, Hk=1, page=16, tail=2, window=33),
    dict(new=[30, 9, 8], lens=[300, 9, 80], Hq=1, Hk=1, page=7, scale=-0.4),
    dict(new=[100, 20, 3], lens=[400, 20, 900], Hq=6, Hk=2, page=16, tail=4),
    dict(new=[150], lens=[100], Hq=4, Hk=2, page=20, window=37),
    dict(new=[70, 30], lens=[200, 10], Hq=3, Hk=3, page=48, layout="phs", causal=False),
]


@pytest.mark.parametrize("dtype,slack", [("bf16", 4), ("bf16", 3), ("f16", 4), ("f16", 1), ("f32", 4), ("f32", 3)])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("case", CUDA_CORES)
def test_the_cuda_cores(gdn, case, d, dtype, slack):  # noqa: F811
    """Rows of queries that begin on a boundary of 8 (fp32: 16) bytes and no wider, and on none."""
    check(gdn, d=d, dtype=dtype, slack=slack, **case)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("page", [1000, 1001, 1024])
@pytest.mark.parametrize("B,Hk,T", [(1, 1, 1), (1, 2, 40), (3, 2, 5), (3, 1, 300)])
def test_rows_that_are_one_page_each(gdn, B, Hk, T, page, dtype):  # noqa: F811
    """A cache without paging, [B, length, Hk, d]: as many pages as rows, one of them alone too."""
    dt, d, Hq = DT[dtype], 64, 4 * Hk
    k, v = (torch.randn(B, page, Hk, d, device="cuda").to(dt) for _ in range(2))
    q = torch.randn(B * T, Hq, d, device="cuda").to(dt)
    lens = [page, 700, 333][:B]
    table = int32([[b] for b in range(B)])
    out, _ = gdn.gdn_paged_attention(q, k, v, table, int32(lens), B=B)
    for b, n in enumerate(lens):
        r = slice(b * T, b * T + T)
        o, _, bound, _ = attend(q[r], k[b, :n], v[b, :n], n - T, d ** -0.5)
        near(out[r], o, bound)
    # and appended to in place: a row's last T positions
    new = [torch.randn(B * T, Hk, d, device="cuda").to(dt) for _ in range(2)]
    want = [x.clone() for x in (k, v)]
    for x, y in zip(want, new):
        for b, n in enumerate(lens):
            x[b, n - T:n] = y[b * T:b * T + T]
    gdn.gdn_paged_append(*new, k, v, table, int32(lens), B=B)
    assert torch.equal(k, want[0]) and torch.equal(v, want[1]) and gdn.gdn_device_errors() == 0


def test_two_graphs_replayed_at_once(gdn):  # noqa: F811
    """Each captured with a workspace of its own, replayed on two streams at the same time."""
    Hq, Hk, d = 8, 2, 128
    calls, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i, (n, T) in enumerate(((3000, 1), (1500, 200))):
        cache = Cache([n], Hk, d, 16, torch.bfloat16, seed=i)
        q = torch.randn(T, Hq, d, device="cuda").to(torch.bfloat16)
        args = (q, cache.k, cache.v, cache.table, int32([n]))
        calls.append((args, gdn.gdn_paged_attention(*args, B=1)[0]))
    for args, _ in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = [gdn.gdn_paged_attention(*args, B=1)[0] for _ in range(10)]
        graphs.append((graph, outs))
    for _ in range(10):
        for s, (graph, _) in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, want), (_, outs) in zip(calls, graphs):
            assert all(torch.equal(x, want) for x in outs)
