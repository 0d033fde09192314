"""Norms of more rows than the grid takes in one turn: rings of rows that wrap, for every
kernel that rows are given to, in place and apart.  Formulas in 64 bits and tolerances
as in test_gpu_norms."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from test_gpu_norms import near, rms

pytestmark = pytest.mark.gpu

DTYPES = pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["f32", "f16", "bf16"])


def normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


@DTYPES
@pytest.mark.parametrize("H,d", [(7, 32), (4, 128), (1, 256), (3, 129), (1, 1024)])
@pytest.mark.parametrize("first", [False, True])
def test_gated_in_place(dtype, H, d, first):
    """Values of the call in place, over several turns of the grid."""
    N = 40_000_000 // (H * d) // (4 if dtype == torch.float32 else 2) + 3
    g = torch.Generator("cuda").manual_seed(d)
    x, z = normal(g, N, H, d).to(dtype), normal(g, N, H, d).to(dtype)
    w = 1 + 0.1 * normal(g, d)
    how = gdn.GDN_GATE_SILU | (gdn.GDN_GATE_FIRST if first else 0)
    apart = gdn.gdn_gated_norm(x, z, w, gate=how)
    zd = z.double() * torch.sigmoid(z.double())
    near(apart, rms(x.double() * zd, 1e-6) * w.double() if first else rms(x.double(), 1e-6) * w.double() * zd)
    gdn.gdn_gated_norm(x, z, w, gate=how, out=x)
    assert torch.equal(x, apart)


@DTYPES
@pytest.mark.parametrize("D", [64, 512, 1000, 1024, 1784, 1792, 2000, 2048, 2047, 4096])
@pytest.mark.parametrize("wide,post,gate", [(True, True, True), (False, True, False), (False, False, True)],
                         ids=["wide", "post", "gate"])
def test_residual_in_place(dtype, D, wide, post, gate):
    N = 16_000_000 // D + 5
    res = torch.float32 if wide else dtype
    g = torch.Generator("cuda").manual_seed(D)
    y, z, x = normal(g, N, D).to(dtype), normal(g, N, D).to(dtype), normal(g, N, D).to(res)
    w1, w2 = (1 + 0.1 * normal(g, D) for _ in range(2))
    how = dict(post_weight=w1 if post else None, gate=z if gate else None, pre_weight=w2, res_scale=0.5)
    a, h = gdn.gdn_residual_norm(y, x, **how)
    u = rms(y.double(), 1e-6) * w1.double() if post else y.double()
    u = 0.5 * u * (torch.sigmoid(z.double()) if gate else 1)
    want = x.double() + u
    near(a, want, terms=x.double().abs() + u.abs())
    # the norm of x' is relative to its terms too
    size = (x.double().abs() + u.abs()) * w2.double() / torch.sqrt(want.pow(2).mean(-1, keepdim=True) + 1e-6)
    near(h, rms(want, 1e-6) * w2.double(), terms=size)
    b, k = gdn.gdn_residual_norm(y, x, residual_out=x, **how)
    assert b is x and torch.equal(x, a) and torch.equal(k, h)
