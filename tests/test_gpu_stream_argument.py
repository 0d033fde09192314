"""Calls on a stream that is not the current one: the memory that the binding takes for
them (scratch, and outputs that the caller drops at once) is not handed to the current
stream's next tensor while the call still has to run."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from gated_deltanet_recurrence_02_gb300.inputs import make_inputs

pytestmark = pytest.mark.gpu


def held_back(calls, stream, handle):
    """Runs calls(stream argument) behind a wait on `stream`, takes as much memory as they
    did on the current stream, and returns whether that memory kept its values."""
    calls(stream.cuda_stream if handle else stream)  # (first calls load and configure their kernels)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = torch.cuda.memory_reserved()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(100_000_000)  # some 50 ms
    calls(stream.cuda_stream if handle else stream)
    assert not stream.query(), "the calls have run already"
    more = torch.cuda.memory_reserved() - before
    assert more > 0
    junk = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in [1 << 16] * 64 + [1 << 20] * 16 + [more // 2]]
    torch.cuda.current_stream().synchronize()
    stream.synchronize()
    return all(bool((j == 7).all()) for j in junk)


def linear(dtype):
    x = make_inputs(71, lengths=[2000], Hk=1, Hv=2, dk=128, dv=128, dtype_qkv=dtype, dtype_gate="f32")
    g = [t.cuda() for t in (x.q, x.k, x.v, x.alpha)]
    assert gdn.gdn_linear_prefill_workspace_size(1, 2000, 1, 2, 128, 128, x.q.dtype) > 0
    return lambda s: (gdn.gdn_linear_prefill(*g, B=1, stream=s), gdn.gdn_linear_recurrent(*g, B=1, stream=s))


def delta(dtype):
    x = make_inputs(72, lengths=[500], Hk=1, Hv=2, dk=128, dv=128, dtype_qkv=dtype, dtype_gate="f32")
    g = [t.cuda() for t in (x.q, x.k, x.v, x.alpha, x.beta)]
    n = torch.tensor([2], dtype=torch.int32, device="cuda")
    S = x.initial_state.cuda()
    su = torch.zeros(1, 3, gdn.slot_width(1, 2, 128, 128), device="cuda")

    def run(s):
        gdn.gdn_prefill_chunked(*g, B=1, stream=s)
        gdn.gdn_prefill_chunked_checkpoints(*g, B=1, checkpoint_capacity=8, stream=s)
        gdn.gdn_prefill_chunked_capture(*g, B=1, state_update_capacity=3, capture_count=n, stream=s)
        gdn.gdn_recurrent_capture(*g, B=1, state_update_capacity=3, capture_count=n, stream=s)
        gdn.gdn_replay_state_updates(S, su, n, state_update_capacity=3, Hk=1, stream=s)
        gdn.gdn_replay_verify(*g, B=1, state_in=S, prev_state_update=su, prev_capacity=3, accepted_count=n,
                              want_draft_final_state=True, stream=s)
    return run


def around(dtype):
    y = torch.randn(600, 16, 128, device="cuda").bfloat16()
    p = torch.softmax(torch.randn(64, 3, 1000, device="cuda"), -1)
    x, u = torch.zeros(64, 2, dtype=torch.int32, device="cuda"), torch.rand(64, 3, device="cuda")
    return lambda s: (gdn.gdn_gated_norm(y, y, stream=s), gdn.gdn_residual_norm(y[:, 0].contiguous(), stream=s),
                      gdn.gdn_accept_drafts(p, None, x, u, stream=s))


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
@pytest.mark.parametrize("calls,dtype", [(linear, "bf16"), (linear, "f32"), (delta, "bf16"), (around, "bf16")],
                         ids=["linear", "linear-f32", "delta", "norms"])
def test_memory_of_a_call_on_another_stream(calls, dtype, handle):
    run, stream = calls(dtype), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        assert held_back(run, stream, handle)


@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_results_on_another_stream(handle):
    """The results are those of the current stream, and stay the caller's to use there."""
    x = make_inputs(73, lengths=[1500], Hk=1, Hv=2, dk=128, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    g = [t.cuda() for t in (x.q, x.k, x.v, x.alpha)]
    out, last = gdn.gdn_linear_prefill(*g, B=1)
    stream = torch.cuda.Stream()
    for _ in range(5):
        stream.wait_stream(torch.cuda.current_stream())
        a, S = gdn.gdn_linear_prefill(*g, B=1, stream=stream.cuda_stream if handle else stream)
        torch.cuda.current_stream().wait_stream(stream)
        a, S = a + 0, S + 0  # read here, dropped here
        assert torch.equal(a, out) and torch.equal(S, last)
