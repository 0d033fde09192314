"""gdn_rotary against its definition in 64 bits: types, widths, strides, axes, far positions,
the turn back as the gradient, in-place calls, streams and graphs."""
import pytest
import torch

from paged import DT, int32, near, turn, turn_bound

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_recurrence_02_gb300 import build, gdn as g
    build.build()
    g.lib()
    return g


def freq(half, theta=10000.0):
    return (theta ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float().cuda()


def make(N, H, d, dtype, slack=0, off=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(N, H * d + slack + off, generator=g).to(dtype).cuda()
    return wide[:, off:off + H * d].unflatten(1, (H, d))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,H,d,R,A,pairs,slack,off", [
    (1, 1, 2, 2, 1, False, 0, 0),       # one pair
    (1, 1, 1, 0, 1, False, 0, 0),       # nothing turns
    (5, 3, 64, 64, 1, False, 0, 0),
    (5, 3, 64, 32, 1, True, 0, 0),
    (33, 2, 80, 46, 3, False, 0, 0),    # halves of 23
    (33, 2, 80, 46, 3, True, 5, 3),     # odd strides, an odd start
    (7, 1, 5, 4, 2, True, 0, 0),        # a head of five
    (300, 8, 128, 128, 3, False, 1024, 8),
    (2000, 4, 128, 96, 2, True, 0, 0),  # several turns of a CTA
    (40, 16, 256, 256, 1, False, 4, 4),
    (3, 2, 1024, 1024, 1, False, 0, 0),
    (9000, 1, 32, 16, 3, False, 0, 0),  # many tokens, one narrow head
])
def test_matches_definition(gdn, dtype, N, H, d, R, A, pairs, slack, off):
    x = make(N, H, d, DT[dtype], slack, off)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(0, 5000, (A, N), generator=g, dtype=torch.int32).cuda()
    axes = int32([i % A for i in range(R // 2)]) if A > 1 else None
    f = freq(R // 2)
    for inverse in (False, True):
        out = gdn.gdn_rotary(x, pos if A > 1 else pos[0], f, axes=axes, pairs=pairs, inverse=inverse)
        ref = turn(x, pos, f, axes, pairs, inverse)
        near(out, ref, turn_bound(x, ref, R // 2, pairs))
        assert torch.equal(out[..., R:], x[..., R:])
    assert gdn.gdn_device_errors() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_and_negative_positions(gdn, dtype):
    pos = int32([[0, -1, 1000000, 16777217, 1 << 30, (1 << 31) - 1, -(1 << 31), 123456789]])
    x = make(8, 2, 64, DT[dtype])
    f = freq(32)
    f[3] = 7.25   # more than a turn a position
    f[5] = -0.3
    f[7] = 0.0
    out = gdn.gdn_rotary(x, pos, f)
    ref = turn(x, pos, f)
    # the angle's own 2^-50, and that of the definition in 64 bits, at 2^31 x 7.25 rad
    far = (2.0 ** -50 + 2.0 ** -52) * pos[0].double().abs()[:, None, None] * 7.25
    near(out, ref, turn_bound(x, ref, 32) + far * x.double().abs().amax(-1, keepdim=True) * 2)


def test_turn_back_is_the_gradient(gdn):
    """The turn is linear, y = M x: differences of the outputs along a direction v are M v, and
    the gradient of w.y is the turn back of w; <w, M v> = <M^T w, v> in 64-bit sums."""
    N, H, d, half = 50, 4, 64, 24
    x, v, w = (make(N, H, d, torch.float32, seed=s) for s in (1, 2, 3))
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(0, 3000, (2, N), generator=g, dtype=torch.int32).cuda()
    axes = int32([i * 2 // half for i in range(half)])
    f = freq(half)
    for pairs in (False, True):
        def run(t, inverse=False):
            return gdn.gdn_rotary(t, pos, f, axes=axes, pairs=pairs, inverse=inverse).double()
        back = run(w, True)
        step = (run(x + 0.5 * v) - run(x - 0.5 * v))
        left, right = (w.double() * step).sum(), (back * v.double()).sum()
        # fp32 roundings of N H d terms of size |w| (|x| + |v|) each, 2^-21 of them at most
        size = (w.double().abs() * (x.double().abs() + v.double().abs())).sum() * 2
        assert abs(float(left - right)) <= 2.0 ** -20 * float(size)
        near(run(run(x).float(), True), x.double(), 2.0 ** -19 * x.double().abs().amax(-1, keepdim=True))


def test_in_place_on_slices_and_rows_behind(gdn):
    N, H, d = 20, 4, 64
    wide = make(N, 12, d, torch.bfloat16)
    before = wide.clone()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    x = wide[:, 2:2 + H]
    out = gdn.gdn_rotary(x[:15], pos[:15], freq(32), out=x[:15])
    assert out.data_ptr() == x.data_ptr()
    ref = turn(before[:15, 2:2 + H], pos[None, :15], freq(32))
    near(x[:15], ref, turn_bound(before[:15, 2:2 + H], ref, 32))
    rest = torch.ones_like(wide, dtype=torch.bool)
    rest[:15, 2:2 + H] = False
    assert torch.equal(wide[rest], before[rest])


def test_special_values(gdn):
    """What is not finite stays in its own pair; elements that do not turn keep their bits."""
    x = make(4, 2, 64, torch.float32)
    x[1, 1, 3] = float("nan")
    x[2, 0, 60] = float("inf")
    pos = int32([0, 1, 2, 3])
    out = gdn.gdn_rotary(x, pos, freq(16))
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[1, 1, 3], [1, 1, 19], [2, 0, 60]]
    assert torch.equal(gdn.gdn_rotary(x, pos, freq(0)).nan_to_num(), x.nan_to_num())


def test_bad_axis_is_reported(gdn):
    x = make(3, 1, 8, torch.float32)
    pos = int32([[5, 6, 7], [1, 2, 3]])
    out = gdn.gdn_rotary(x, pos, freq(4), axes=int32([0, 1, 2, -1]))
    assert gdn.gdn_device_errors() == 1
    f = freq(4)
    f[2:] = 0
    ref = turn(x, pos, f, [0, 1, 0, 0])
    near(out, ref, turn_bound(x, ref, 4))


def test_stream_and_graph(gdn):
    N, H, d = 130, 8, 128
    x = make(N, H, d, torch.bfloat16)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")
    f = freq(64)
    want = gdn.gdn_rotary(x, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gdn.gdn_rotary(x, pos, f, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_rotary(x, pos, f, out=out)
    x2 = make(N, H, d, torch.bfloat16, seed=9)
    want2 = gdn.gdn_rotary(x2, pos, f)
    x.copy_(x2)
    graph.replay()
    assert torch.equal(out, want2)


def test_no_tokens(gdn):
    x = torch.empty(0, 4, 64, device="cuda")
    assert gdn.gdn_rotary(x, torch.empty(0, dtype=torch.int32, device="cuda"), freq(32)).shape == (0, 4, 64)
