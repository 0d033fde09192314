"""The operators together: speculative decoding of a small linear-attention model."""
import os
import sys

import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def test_states_are_those_of_the_emitted_text():
    """After any steps the committed states equal a prefill over prompt and emitted
    tokens (all but each row's last, which no pass has seen yet)."""
    from speculative_linear_layer import Model, generate
    model = Model(layers=2)
    prompt = torch.randint(0, model.vocab, (3, 70), device="cuda")
    emitted, states = generate(model, prompt, steps=6, K=3)
    n = (emitted >= 0).sum(-1)
    assert int(n.min()) >= 1 and int(n.max()) <= 4
    for b in range(3):
        text = torch.cat([prompt[b], torch.tensor([t for t in emitted[b].flatten().tolist() if t >= 0], device="cuda")])
        want = model.states(1)
        model.run(text[:-1].long(), 1, want)
        for s, w in zip(states, want):
            # bf16 activations through another split of the tokens: a layer's inputs
            # differ by roundings of 2^-8, averaged over the sums of the state
            assert float((s[b] - w[0]).norm() / w[0].norm()) < 2.0 ** -5
    assert gdn.gdn_device_errors() == 0


def test_step_is_captured_in_a_graph():
    """Recurrent pass, verification and commit in a CUDA graph, replayed with new
    inputs, bit for bit as eager calls."""
    B, K, H, d, V = 3, 2, 2, 64, 500
    g = torch.Generator("cuda").manual_seed(0)
    T = K + 1

    def inputs():
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        p = torch.softmax(3 * r(B, T, V), -1)
        return [r(B * T, H, d).bfloat16(), r(B * T, H, d).bfloat16(), r(B * T, H, d).bfloat16(),
                torch.rand(B * T, H, device="cuda", generator=g), p, torch.rand(B, T, device="cuda", generator=g),
                torch.randint(0, V, (B, K), device="cuda", generator=g, dtype=torch.int32)]

    cc = torch.full((B,), T, dtype=torch.int32, device="cuda")

    def step(x, S):
        o, _, su = gdn.gdn_linear_recurrent(x[0], x[1], x[2], x[3], B=B, T=T, initial_state=S, want_final_state=False,
                                            state_update_capacity=T, capture_count=cc)
        tok, n = gdn.gdn_accept_drafts(x[4], None, x[6], x[5])
        gdn.gdn_replay_state_updates(S, su, n, state_update_capacity=T, Hk=H, state_out=S)
        y = gdn.gdn_gated_norm(o, x[2], None)
        res, h = gdn.gdn_residual_norm(y.flatten(1), o.flatten(1))
        po, pS = gdn.gdn_linear_prefill(x[0], x[1], x[2], x[3], B=B, T=T, initial_state=S)
        return [o, tok, n, S, y, res, h, po, pS]

    static, S = inputs(), torch.randn(B, H, d, d, device="cuda", generator=g)
    step([t.clone() for t in static], S.clone())  # attributes are set outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(static, S)
    for _ in range(3):
        new, start = inputs(), torch.randn(B, H, d, d, device="cuda", generator=g)
        for a, b in zip(static, new):
            a.copy_(b)
        S.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        want = step(new, start.clone())
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
