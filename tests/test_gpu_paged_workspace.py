"""Workspaces of gdn_paged_attention that the binding provides: calls of growing and shrinking
sizes one after the other, two threads at once, a captured call next to eager ones."""
import threading

import pytest
import torch

from paged import Cache, attend, int32, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_recurrence_02_gb300 import build, gdn as g
    build.build()
    g.lib()
    return g


def case(Hq, Hk, d, n, T, dt, seed):
    cache = Cache([n], Hk, d, 16, dt, seed)
    q = torch.randn(T, Hq, d, generator=torch.Generator().manual_seed(seed)).to(dt).cuda()
    o, _, bound, _ = attend(q, *cache.rows[0], n - T, d ** -0.5)
    return (q, cache.k, cache.v, cache.table, int32([n])), o, bound


SIZES = [(8, 2, 64, 700, 1, torch.bfloat16), (8, 2, 128, 900, 130, torch.float16), (2, 2, 32, 400, 50, torch.float32),
         (8, 1, 128, 2000, 5, torch.bfloat16)]


def test_sizes_in_turn(gdn):
    cases = [case(*x, seed=i) for i, x in enumerate(SIZES)]
    got = [gdn.gdn_paged_attention(*args, B=1)[0] for _ in range(3) for args, _, _ in cases]
    for y, (_, o, bound) in zip(got, cases * 3):
        near(y, o, bound)
    assert gdn.gdn_device_errors() == 0


def test_two_threads_at_once(gdn):
    """Both on the default stream, their launches in between each other's."""
    cases = [case(*SIZES[i], seed=i) for i in (1, 3)]
    want = [gdn.gdn_paged_attention(*args, B=1)[0] for args, _, _ in cases]
    got = [[], []]
    start = threading.Barrier(2)

    def calls(i):
        torch.cuda.set_device(0)
        start.wait()
        for _ in range(100):
            got[i].append(gdn.gdn_paged_attention(*cases[i][0], B=1)[0])

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 100 and all(torch.equal(y, want[i]) for y in got[i])


def test_a_captured_call_next_to_eager_ones(gdn):
    """Replays on another stream while calls run on the default one: workspaces of their own."""
    cases = [case(*SIZES[i], seed=i) for i in (1, 3)]
    want = [gdn.gdn_paged_attention(*args, B=1)[0] for args, _, _ in cases]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [gdn.gdn_paged_attention(*cases[0][0], B=1)[0] for _ in range(20)]
    side = torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(side):
            graph.replay()
        eager = [gdn.gdn_paged_attention(*cases[1][0], B=1)[0] for _ in range(20)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[0]) for y in captured) and all(torch.equal(y, want[1]) for y in eager)


def test_the_default_stream_named_from_another(gdn):
    """stream=0 with another one current: the kept workspace, none yet, and one that is too small."""
    small, large = case(*SIZES[2], seed=2), case(*SIZES[1], seed=1)
    torch.cuda.synchronize()

    def calls():
        torch.cuda.set_device(0)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            results.append((gdn.gdn_paged_attention(*small[0], B=1, stream=0)[0], small))
        results.append((gdn.gdn_paged_attention(*small[0], B=1)[0], small))
        with torch.cuda.stream(side):
            results.append((gdn.gdn_paged_attention(*large[0], B=1, stream=0)[0], large))
        torch.cuda.synchronize()

    results = []
    t = threading.Thread(target=calls)  # (with no workspace kept)
    t.start()
    t.join()
    assert len(results) == 3
    for y, (_, o, bound) in results:
        near(y, o, bound)
