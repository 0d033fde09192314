"""Gated norms whose one token has more than 2^32 elements (heads or rows flattened into
it).  Tolerances as in test_gpu_norms; the heads around 2^32 and the last ones are
compared, which read and write wrong ones wherever an offset is held in 32 bits."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from test_gpu_norms import near, rms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 4096, 127], ids=["d128", "d4096", "odd"])
def test_one_token_past_32_bits(d):
    H = (1 << 32) // d + 40
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.empty(1, H, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    z = torch.empty(1, H, d, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
    out = torch.zeros_like(x)
    gdn.gdn_gated_norm(x, z, w, gate=gdn.GDN_GATE_SIGMOID, out=out)
    for lo in (0, H // 2, H - 80):
        s = slice(lo, lo + 80)
        near(out[0, s], rms(x[0, s].double(), 1e-6) * w.double() * torch.sigmoid(z[0, s].double()))
