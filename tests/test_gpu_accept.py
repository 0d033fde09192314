"""Draft verification against its definition, evaluated with Python's whole
numbers: the outputs are tokens and counts and have to be equal."""
import numpy as np
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn

pytestmark = pytest.mark.gpu


def units(x):
    x = np.where(np.isnan(x), 0, np.clip(np.nan_to_num(x, nan=0.0, posinf=2.0, neginf=-2.0), 0, 1))
    return np.floor(x.astype(np.float64) * 2.0 ** 40).astype(np.int64)


def definition(p, q, x, u, count):
    p = p.float().cpu().numpy()
    q = None if q is None else q.float().cpu().numpy()
    x, u = x.cpu().numpy(), u.cpu().numpy()
    B, K1, V = p.shape
    K = K1 - 1
    toks, n_out = np.full((B, K1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        c = K if count is None else min(max(int(count[b]), 0), K)
        n = 0
        while n < c:
            t = int(x[b, n])
            if not 0 <= t < V:
                break
            qx = np.float32(1) if q is None else q[b, n, t]
            if not np.float32(u[b, n] * qx) < p[b, n, t]:
                break
            n += 1
        w = units(p[b, n])
        if n < c:
            if q is not None:
                with np.errstate(invalid="ignore"):
                    w = units(p[b, n] - q[b, n])
            elif 0 <= x[b, n] < V:
                w[x[b, n]] = 0
        if w.sum() == 0:
            w = units(p[b, n])
        total = int(w.sum())
        toks[b, :n] = x[b, :n]
        n_out[b] = n + 1
        if total > 0:
            goal = min(int(float(u[b, K]) * float(total)), total - 1)
            toks[b, n] = int(np.searchsorted(np.cumsum(w), goal, side="right"))
    return toks, n_out


def check(p, q, x, u, count=None):
    tokens, emitted = gdn.gdn_accept_drafts(p, q, x, u, draft_count=count)
    want, n = definition(p, q, x, u, None if count is None else count.cpu().numpy())
    assert np.array_equal(emitted.cpu().numpy(), n)
    assert np.array_equal(tokens.cpu().numpy(), want)
    return tokens, emitted


def inputs(B, K, V, dtype=torch.float32, seed=0, sharp=3.0):
    g = torch.Generator("cuda").manual_seed(seed)
    l = sharp * torch.randn(B, K + 1, V, device="cuda", generator=g)
    p = torch.softmax(l, -1)
    q = torch.softmax(l[:, :K] + 0.7 * torch.randn(B, K, V, device="cuda", generator=g), -1)
    x = (torch.multinomial(q.flatten(0, 1), 1, generator=g).view(B, K) if B * K else torch.zeros(B, K, device="cuda"))
    u = torch.rand(B, K + 1, device="cuda", generator=g)
    return p.to(dtype), q.to(dtype), x.to(torch.int32), u


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (1, 4, 5), (3, 0, 33), (5, 3, 1000), (2, 40, 257), (17, 4, 32000),
                                   (200, 2, 4099), (1, 7, 131072), (700, 1, 100)])
def test_against_definition(B, K, V, dtype):
    p, q, x, u = inputs(B, K, V, dtype, seed=B + V)
    check(p, q, x, u)
    check(p, None, x, u)
    count = torch.randint(-1, K + 2, (B,), device="cuda", dtype=torch.int32)
    check(p, q, x, u, count)


def test_ends_of_the_random_numbers_and_ties():
    p, q, x, u = inputs(8, 2, 777, seed=3)
    u[:4] = 0.0
    u[4:] = 1 - 2.0 ** -24
    check(p, q, x, u)
    flat = torch.full((4, 3, 777), 1 / 777, device="cuda")
    u = torch.tensor([0.0, 0.25, 0.5, 1 - 2.0 ** -24], device="cuda")[:, None].expand(4, 3).contiguous()
    t, n = check(flat, flat[:, :2].contiguous(), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), u)
    assert (n == 3).all() and int(t[0, 2]) == 0 and int(t[3, 2]) == 776
    # a draft that equals its own probability times u is rejected: the test is strict
    one = torch.zeros(1, 2, 8, device="cuda")
    one[0, :, 3] = 0.5
    check(one, None, torch.tensor([[3]], dtype=torch.int32, device="cuda"), torch.tensor([[0.5, 0.5]], device="cuda"))


def test_empty_rows_and_not_finite():
    V = 300
    p, q, x, u = inputs(6, 1, V, seed=5)
    p[0] = 0                                    # nothing to sample at all
    q[1] = 1.0                                  # no weight left after the draft: the target itself
    u[1, 0] = 0.999
    p[2, :, 10:20] = float("nan")
    p[3, :, 7] = float("inf")
    p[4, 0] = 0
    p[4, 0, 5] = 1.0                            # a certain target whose token the draft missed
    x[4] = 6
    q[5, 0, :50] = float("nan")
    t, n = check(p, q, x, u)
    assert int(t[0, 0]) == -1 and int(n[0]) == 1 and int(t[4, 0]) == 5
    certain = torch.zeros(1, 2, V, device="cuda")
    certain[0, 0, 9] = 0.25                     # the only token is the one rejected: it is sampled after all
    t, _ = check(certain, None, torch.tensor([[9]], dtype=torch.int32, device="cuda"),
                 torch.tensor([[0.5, 0.5]], device="cuda"))
    assert int(t[0, 0]) == 9


def test_token_out_of_range_is_rejected_and_reported():
    p, q, x, u = inputs(4, 3, 500, seed=6)
    u[:] = 1e-6
    x[1, 1], x[2, 0] = 500, -1
    assert gdn.gdn_device_errors() == 0
    _, n = check(p, q, x, u)
    assert int(n[1]) == 2 and int(n[2]) == 1
    assert gdn.gdn_device_errors() == gdn.GDN_DEVERR_BAD_INDEX


def test_frequencies_are_the_targets():
    """Over many requests the emitted first token follows the target's distribution."""
    B, V = 60000, 6
    g = torch.Generator("cuda").manual_seed(1)
    p1 = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1], device="cuda")
    q1 = torch.tensor([0.4, 0.05, 0.05, 0.3, 0.1, 0.1], device="cuda")
    x = torch.multinomial(q1, B, replacement=True, generator=g).view(B, 1).to(torch.int32)
    u = torch.rand(B, 2, device="cuda", generator=g)
    t, _ = gdn.gdn_accept_drafts(p1.expand(B, 2, V).contiguous(), q1.expand(B, 1, V).contiguous(), x, u)
    f = torch.bincount(t[:, 0].long(), minlength=V).double() / B
    # five standard deviations of a frequency
    assert bool(((f - p1.double()).abs() < 5 * torch.sqrt(p1.double() * (1 - p1.double()) / B)).all()), f


def test_padded_vocabulary_and_offsets_past_32_bits():
    """Rows of a wider buffer; and probabilities of more than 2^31 elements."""
    p, q, x, u = inputs(5, 3, 900, seed=8)
    wide_p, wide_q = torch.full((5, 4, 1024), 9.0, device="cuda"), torch.full((5, 3, 1024), 9.0, device="cuda")
    wide_p[..., :900], wide_q[..., :900] = p, q
    t, n = gdn.gdn_accept_drafts(p, q, x, u)
    t2, n2 = gdn.gdn_accept_drafts(wide_p[..., :900], wide_q[..., :900], x, u)
    assert torch.equal(t, t2) and torch.equal(n, n2)
    B, V = 600, 1 << 20
    big = torch.zeros(B, 4, V, device="cuda")          # 2.5e9 elements
    at = torch.randint(0, V, (B, 4), device="cuda")
    big.scatter_(2, at[..., None], 1.0)
    drafts = at[:, :3].to(torch.int32)
    t, n = gdn.gdn_accept_drafts(big, None, drafts.contiguous(), torch.full((B, 4), 0.5, device="cuda"))
    assert (n == 4).all() and torch.equal(t.long(), at)
