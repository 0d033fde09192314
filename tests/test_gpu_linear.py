"""Linear attention with a decay for each head: the chunked prefill and the
recurrent form against the recurrence evaluated token by token in 64 bits.

Tolerances (relative Frobenius error, per row and value head).  State: fp32
arithmetic on exact inputs, each step within a few 2^-24 and contracted by the
decay; sums of T terms of random sign stay below 1e-5 by a wide margin.
Outputs in 16 bits: one rounding of the result and one of each term of it (the
scores, or the state, where the tensor cores take them), each at most u = 2^-8
(bf16) or 2^-11 (fp16), so 2u in norm where the terms do not cancel, as they do
not in these inputs; fp32 outputs 1e-5."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from gated_deltanet_recurrence_02_gb300.inputs import DTYPES, make_inputs
from helpers import Guarded, rel_per_unit

pytestmark = pytest.mark.gpu

TOL_OUT = {"f32": 1e-5, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}
TOL_STATE = 1e-5


def definition(x, alpha, *, state=None, index=None, scale=1.0):
    """S <- alpha S + v k^T, o = S (scale q), in 64 bits on the device."""
    dev = "cuda"
    q, k, v, a = (t.to(dev).double() for t in (x.q, x.k, x.v, alpha))
    G = x.Hv // x.Hk
    q, k = q.repeat_interleave(G, 1), k.repeat_interleave(G, 1)
    a = a.expand(x.total_T, x.Hv) if a.dim() == 1 else a
    out = torch.zeros(x.total_T, x.Hv, x.dv, dtype=torch.float64, device=dev)
    last = torch.zeros(x.B, x.Hv, x.dv, x.dk, dtype=torch.float64, device=dev)
    t0 = 0
    for b, n in enumerate(x.lengths):
        S = last[b]
        src = b if index is None else index[b]
        if state is not None and 0 <= src < state.shape[0]:
            S += state[src].to(dev).double()
        for t in range(t0, t0 + n):
            S.mul_(a[t, :, None, None]).add_(v[t, :, :, None] * k[t, :, None, :])
            out[t] = (S @ (scale * q[t])[..., None]).squeeze(-1)
        t0 += n
    return out.cpu().numpy(), last.cpu().numpy()


def call(x, alpha, fn, *, conventions=0, state=None, index=None, packed=False, scale=1.0, **more):
    out = Guarded((x.total_T, x.Hv, x.dv), x.v.dtype)
    final = Guarded((x.B, x.Hv, x.dv, x.dk), torch.float32)
    r = fn(x.q.cuda(), x.k.cuda(), x.v.cuda(), alpha.cuda(), B=x.B,
           T=None if packed else x.uniform_T, cu_seqlens=x.cu_seqlens.cuda() if packed else None,
           initial_state=None if state is None else state.cuda(),
           initial_state_indices=None if index is None else torch.tensor(index, dtype=torch.int32).cuda(),
           final_state=final.t, out=out.t, scale=scale, conventions=conventions, **more)
    torch.cuda.synchronize()
    assert out.guards_intact() and final.guards_intact()
    return out.t, final.t, r


def check(x, alpha, out, last, dtype, **how):
    ro, rs = definition(x, alpha.double(), **how)
    bounds = x.cu_seqlens.numpy()
    e, where = rel_per_unit(out, ro, bounds)
    assert e < TOL_OUT[dtype], ("out", e, where)
    e, where = rel_per_unit(last, rs, np.arange(x.B + 1))
    assert e < TOL_STATE, ("state", e, where)


SHAPES = [  # lengths, Hk, Hv, dk, dv
    ([1], 1, 1, 32, 32),
    ([63], 1, 2, 64, 128),
    ([64, 64], 2, 4, 128, 128),
    ([65], 2, 2, 128, 64),
    ([1, 0, 129, 64, 2, 300], 1, 3, 128, 128),
    ([0, 0], 1, 1, 64, 64),
    ([257, 5], 2, 2, 32, 128),
    ([200, 131], 2, 6, 64, 32),
    ([1111], 1, 2, 128, 128),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[0] + list(s[1:]))))
@pytest.mark.parametrize("per_head", [False, True])
def test_prefill(shape, dtype, per_head):
    lens, Hk, Hv, dk, dv = shape
    x = make_inputs(7, lengths=lens, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype_qkv=dtype, dtype_gate="f32")
    alpha = torch.linspace(0.85, 0.9999, Hv) if per_head else x.alpha
    out, last, _ = call(x, alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True,
                        scale=0.7, conventions=gdn.GDN_ALPHA_PER_HEAD if per_head else 0)
    check(x, alpha, out, last, dtype, state=x.initial_state, scale=0.7)


@pytest.mark.parametrize("gate", ["f32", "f16", "bf16"])
def test_prefill_uniform_rows_log_decay_and_no_state(gate):
    x = make_inputs(8, lengths=[190] * 3, Hk=2, Hv=4, dk=128, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    g = torch.log(x.alpha).to(DTYPES[gate])
    out, last, _ = call(x, g, gdn.gdn_linear_prefill, conventions=gdn.GDN_ALPHA_LOG)
    check(x, torch.exp(g.double()), out, last, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_row_slow_decay(dtype):
    """One row long enough to be split, decays that keep all of it alive."""
    x = make_inputs(9, lengths=[4500], Hk=1, Hv=2, dk=128, dv=128, dtype_qkv=dtype, dtype_gate="f32")
    alpha = torch.tensor([0.9995, 0.99])
    out, last, _ = call(x, alpha, gdn.gdn_linear_prefill, state=x.initial_state,
                        conventions=gdn.GDN_ALPHA_PER_HEAD)
    check(x, alpha, out, last, dtype, state=x.initial_state)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_strong_and_zero_decays(dtype):
    """Decays of 0 drop the state; products that underflow inside a chunk."""
    x = make_inputs(10, lengths=[150, 70], Hk=1, Hv=2, dk=64, dv=128, dtype_qkv=dtype, dtype_gate="f32")
    alpha = x.alpha.clone()
    alpha[::7] = 0.0
    alpha[3::11] = 1e-30
    alpha[40:60] = 1.0
    out, last, _ = call(x, alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    check(x, alpha, out, last, dtype, state=x.initial_state)
    alpha[:] = 0.0  # o_t = v_t (k_t . q_t)
    out, last, _ = call(x, alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    check(x, alpha, out, last, dtype, state=x.initial_state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_snapshot_index_in_place_and_bad_index(dtype):
    x = make_inputs(11, lengths=[70, 3, 140], Hk=1, Hv=2, dk=128, dv=64, dtype_qkv=dtype,
                    dtype_gate="bf16", n_states=2)
    out, last, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, index=[1, 0, 1], packed=True)
    check(x, x.alpha, out, last, dtype, state=x.initial_state, index=[1, 0, 1])
    assert gdn.gdn_device_errors() == 0
    out, last, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, index=[1, 2, -1], packed=True)
    check(x, x.alpha, out, last, dtype, state=x.initial_state, index=[1, 2, -1])
    assert gdn.gdn_device_errors() == gdn.GDN_DEVERR_BAD_INDEX
    y = make_inputs(12, lengths=[130] * 2, Hk=1, Hv=2, dk=128, dv=64, dtype_qkv=dtype, dtype_gate="f32")
    g = [t.cuda() for t in (y.q, y.k, y.v, y.alpha)]
    S = y.initial_state.cuda()
    _, apart = gdn.gdn_linear_prefill(*g, B=2, T=130, initial_state=S)
    _, same = gdn.gdn_linear_prefill(*g, B=2, T=130, initial_state=S, final_state=S)
    assert same.data_ptr() == S.data_ptr() and torch.equal(apart, same)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_magnitudes(dtype, size):
    """States and values far from 1: nothing may overflow or vanish on the way."""
    x = make_inputs(13, lengths=[300], Hk=1, Hv=1, dk=128, dv=128, dtype_qkv=dtype, dtype_gate="f32")
    x.v = (x.v.float() * size).to(x.v.dtype)
    x.k = (x.k.float() * size).to(x.k.dtype)
    x.q = (x.q.float() / size).to(x.q.dtype)
    x.initial_state *= size * size
    alpha = torch.full((1,), 0.999)
    out, last, _ = call(x, alpha, gdn.gdn_linear_prefill, state=x.initial_state, conventions=gdn.GDN_ALPHA_PER_HEAD)
    check(x, alpha, out, last, dtype, state=x.initial_state)


def test_not_finite_stays_in_its_row_and_head():
    x = make_inputs(14, lengths=[140, 90], Hk=2, Hv=2, dk=128, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    clean, cl, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    clean, cl = clean.clone(), cl.clone()
    x.v[100, 1, 5] = float("nan")
    x.v[160, 0, 7] = float("inf")
    out, last, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    assert torch.equal(out[:140, 0], clean[:140, 0]) and torch.equal(out[140:, 1], clean[140:, 1])
    assert torch.equal(last[0, 0], cl[0, 0]) and torch.equal(last[1, 1], cl[1, 1])
    assert torch.isnan(out[100:140, 1, 5]).all() and torch.isnan(last[0, 1, 5]).all()
    assert not torch.isfinite(last[1, 0, 7]).any()
    assert torch.equal(out[:100, 1, :5], clean[:100, 1, :5])


def test_same_bits_twice_and_on_another_stream():
    x = make_inputs(15, lengths=[2200], Hk=1, Hv=2, dk=128, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    a, s, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        b, t, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state)
    stream.synchronize()
    assert torch.equal(a, b) and torch.equal(s, t)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [([1] * 5, 1, 2, 128, 128), ([4] * 3, 2, 6, 64, 32),
                                   ([3, 0, 9, 1], 1, 1, 32, 64)], ids=["T1", "T4", "ragged"])
@pytest.mark.parametrize("per_head", [False, True])
def test_recurrent_and_capture_replays(shape, dtype, per_head):
    lens, Hk, Hv, dk, dv = shape
    x = make_inputs(16, lengths=lens, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype_qkv=dtype, dtype_gate="f32")
    alpha = torch.linspace(0.9, 0.99, Hv) if per_head else x.alpha
    cap = 4
    counts = [(3 * b + 1) % (cap + 2) for b in range(x.B)]
    out, last, (_, _, su) = call(
        x, alpha, gdn.gdn_linear_recurrent, state=x.initial_state, packed=len(set(lens)) > 1,
        conventions=gdn.GDN_ALPHA_PER_HEAD if per_head else 0, state_update_capacity=cap,
        capture_count=torch.tensor(counts, dtype=torch.int32).cuda())
    check(x, alpha, out, last, dtype, state=x.initial_state)
    # replaying a prefix of the capture gives the state after as many tokens
    n = [min(c, cap, L) for c, L in zip(counts, lens)]
    S = gdn.gdn_replay_state_updates(x.initial_state.cuda(), su, torch.tensor(n, dtype=torch.int32).cuda(),
                                     state_update_capacity=cap, Hk=Hk)
    cut = make_inputs(16, lengths=lens, Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype_qkv=dtype, dtype_gate="f32")
    pick = torch.cat([torch.arange(int(c), int(c) + m) for c, m in zip(x.cu_seqlens, n)]).long()
    cut.q, cut.k, cut.v = x.q[pick], x.k[pick], x.v[pick]
    cut.lengths = n
    cut.cu_seqlens = torch.tensor([sum(n[:b]) for b in range(x.B + 1)], dtype=torch.int32)
    _, rs = definition(cut, alpha if per_head else alpha[pick], state=x.initial_state)
    e, where = rel_per_unit(S, rs, np.arange(x.B + 1))
    assert e < TOL_STATE, (e, where)


def test_recurrent_inactive_capture_clears():
    x = make_inputs(17, lengths=[2, 2], Hk=1, Hv=2, dk=64, dv=64, dtype_qkv="bf16", dtype_gate="f32")
    su = torch.full((2, 3, gdn.slot_width(1, 2, 64, 64)), 7.0, device="cuda")
    out, last, _ = call(x, x.alpha, gdn.gdn_linear_recurrent, state=x.initial_state, state_update_capacity=3,
                        capture_count=torch.tensor([2, 2], dtype=torch.int32).cuda(), state_update=su,
                        state_update_active=torch.zeros(1, dtype=torch.int32).cuda())
    check(x, x.alpha, out, last, "bf16", state=x.initial_state)
    assert not su.any()


def test_prefill_equals_recurrent_continued():
    """A prompt in two calls, the second from the first one's state, and token by token."""
    x = make_inputs(18, lengths=[333], Hk=2, Hv=2, dk=128, dv=128, dtype_qkv="f32", dtype_gate="f32")
    g = [t.cuda() for t in (x.q, x.k, x.v, x.alpha)]
    whole, S = gdn.gdn_linear_prefill(*g, B=1, T=333)
    a, Sa = gdn.gdn_linear_prefill(*[t[:200].contiguous() for t in g], B=1, T=200)
    b, Sb = gdn.gdn_linear_prefill(*[t[200:].contiguous() for t in g], B=1, T=133, initial_state=Sa)
    c, Sc, _ = gdn.gdn_linear_recurrent(*g, B=1, T=333)
    for o, s in ((torch.cat([a, b]), Sb), (c, Sc)):
        assert float((o - whole).norm() / whole.norm()) < 1e-5
        assert float((s - S).norm() / S.norm()) < 1e-5


def test_segmented_prefill_in_a_graph_and_in_place():
    """A row long enough for both passes, captured; the last state in the place of the initial one."""
    x = make_inputs(19, lengths=[1500], Hk=1, Hv=2, dk=128, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    g = [t.cuda() for t in (x.q, x.k, x.v, x.alpha)]
    S0 = x.initial_state.cuda()
    assert gdn.gdn_linear_prefill_workspace_size(1, 1500, 1, 2, 128, 128, torch.bfloat16) > 0
    out, last = gdn.gdn_linear_prefill(*g, B=1, T=1500, initial_state=S0)
    S = S0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, _ = gdn.gdn_linear_prefill(*g, B=1, T=1500, initial_state=S, final_state=S)
    for _ in range(2):
        S.copy_(S0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(S, last)


@pytest.mark.parametrize("offset", [4, 8])
def test_states_on_16_byte_boundaries(offset):
    """States that start on 16 but not on 32 bytes."""
    x = make_inputs(20, lengths=[130], Hk=1, Hv=2, dk=64, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    g = [t.cuda() for t in (x.q, x.k, x.v, x.alpha)]
    S0 = x.initial_state.cuda()
    buf = torch.zeros(2, S0.numel() + 16, device="cuda")
    a, b = (t[offset:offset + S0.numel()].view(S0.shape) for t in (buf[0], buf[1]))
    a.copy_(S0)
    o1, s1 = gdn.gdn_linear_prefill(*g, B=1, T=130, initial_state=S0)
    o2, s2 = gdn.gdn_linear_prefill(*g, B=1, T=130, initial_state=a, final_state=b)
    assert torch.equal(o1, o2) and torch.equal(s1, s2)


@pytest.mark.parametrize("rows", [[90] * 3, [900]])
def test_wait_that_runs_out_is_reported(rows):
    """With a limit that gives up at the first incomplete check the call ends with the
    timeout bit, and the next call, with the limit restored, is right."""
    x = make_inputs(21, lengths=rows, Hk=1, Hv=2, dk=128, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    gdn.gdn_set_wait_limit_ns(1)
    try:
        call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state)
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_device_errors()
        assert e.value.status == 6
    finally:
        gdn.gdn_set_wait_limit_ns(0)
    out, last, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state)
    check(x, x.alpha, out, last, "bf16", state=x.initial_state)
    assert gdn.gdn_device_errors() == 0
