"""Linear-attention prefill at the lengths where it takes another way: rows long
enough for segments (each joined to the one before it), packed with rows too short
for any, and rows of a few tokens.  Against the recurrence in 64 bits, with the
tolerances derived in test_gpu_linear."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from gated_deltanet_recurrence_02_gb300.inputs import make_inputs
from test_gpu_linear import call, check, definition, TOL_OUT
from helpers import rel_per_unit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Hk,Hv,dk,dv", [(1, 2, 128, 128), (1, 1, 64, 32), (1, 3, 32, 128)])
@pytest.mark.parametrize("per_head", [False, True])
def test_segments_of_ragged_rows(dtype, Hk, Hv, dk, dv, per_head):
    x = make_inputs(31, lengths=[2100, 1, 1700, 1999], Hk=Hk, Hv=Hv, dk=dk, dv=dv, dtype_qkv=dtype,
                    dtype_gate="f32", n_states=3)
    need = gdn.gdn_linear_prefill_workspace_size(x.B, x.total_T, Hk, Hv, dk, dv, x.q.dtype, varlen=True)
    assert need > 0  # the rows are cut
    alpha = torch.linspace(0.97, 0.9999, Hv) if per_head else x.alpha
    how = dict(state=x.initial_state, index=[2, 0, 2, 1], scale=0.5)
    out, last, _ = call(x, alpha, gdn.gdn_linear_prefill, packed=True,
                        conventions=gdn.GDN_ALPHA_PER_HEAD if per_head else 0, **how)
    check(x, alpha, out, last, dtype, **how)
    # without a final state the last segments' end states are not formed
    got, none = gdn.gdn_linear_prefill(x.q.cuda(), x.k.cuda(), x.v.cuda(), alpha.cuda(), B=x.B,
                                       cu_seqlens=x.cu_seqlens.cuda(), initial_state=x.initial_state.cuda(),
                                       initial_state_indices=torch.tensor([2, 0, 2, 1], dtype=torch.int32).cuda(),
                                       scale=0.5, want_final_state=False,
                                       conventions=gdn.GDN_ALPHA_PER_HEAD if per_head else 0)
    assert none is None and torch.equal(got, out)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("B", [1, 7])
def test_rows_of_a_few_tokens(dtype, T, B):
    x = make_inputs(32, lengths=[T] * B, Hk=2, Hv=4, dk=128, dv=64, dtype_qkv=dtype, dtype_gate="bf16", n_states=2)
    how = dict(state=x.initial_state, index=[b % 2 for b in range(B)])
    out, last, _ = call(x, x.alpha, gdn.gdn_linear_prefill, **how)
    check(x, x.alpha, out, last, dtype, **how)


@pytest.mark.parametrize("lengths", [[1, 0, 2], [0, 4], [3, 1], [5, 0]])
def test_a_few_packed_tokens(lengths):
    x = make_inputs(33, lengths=lengths, Hk=1, Hv=2, dk=64, dv=128, dtype_qkv="bf16", dtype_gate="f32")
    out, last, _ = call(x, x.alpha, gdn.gdn_linear_prefill, state=x.initial_state, packed=True)
    ref, state = definition(x, x.alpha.double(), state=x.initial_state)
    e, where = rel_per_unit(out, ref, x.cu_seqlens.numpy())
    assert e < TOL_OUT["bf16"], (e, where)
    # (a row of no tokens keeps its state to the last bit)
    for b, n in enumerate(lengths):
        if n == 0:
            assert torch.equal(last[b].cpu(), x.initial_state[b])
    check(x, x.alpha, out, last, "bf16", state=x.initial_state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_states_of_few_tokens_in_place(dtype):
    x = make_inputs(34, lengths=[3] * 4, Hk=1, Hv=2, dk=128, dv=128, dtype_qkv=dtype, dtype_gate="f32")
    g = [t.cuda() for t in (x.q, x.k, x.v, x.alpha)]
    S = x.initial_state.cuda()
    out, apart = gdn.gdn_linear_prefill(*g, B=4, T=3, initial_state=S)
    here, same = gdn.gdn_linear_prefill(*g, B=4, T=3, initial_state=S, final_state=S)
    assert same is S and torch.equal(S, apart) and torch.equal(out, here)
