"""Probabilities of one position for each request, cut out of tensors of more."""
import pytest
import torch

from gated_deltanet_recurrence_02_gb300 import gdn
from test_gpu_accept import check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [1000, 1003])
@pytest.mark.parametrize("certain", [False, True])
def test_one_draft_of_several(V, certain):
    """The draft's probabilities are the first position of K."""
    p, q, x, u = inputs(9, 4, V, seed=4)
    p, x, u = p[:, :2].contiguous(), x[:, :1].contiguous(), u[:, :2].contiguous()
    assert not q[:, :1].is_contiguous()
    check(p, None if certain else q[:, :1], x, u)


def test_no_draft():
    """K = 0: a token is sampled from the last position's distribution."""
    p, _, x, u = inputs(9, 4, 1000, seed=5)
    tokens, emitted = check(p[:, 4:], None, x[:, :0].contiguous(), u[:, 4:].contiguous())
    assert bool((emitted == 1).all()) and tokens.shape == (9, 1)


def test_rows_that_are_not_even():
    p, q, x, u = inputs(4, 2, 1000, seed=6)
    wide = torch.empty(4, 5, 1000, device="cuda")[:, :3]
    with pytest.raises(ValueError, match="evenly spaced"):
        gdn.gdn_accept_drafts(wide, q, x, u)
