"""gdn_paged_attention's paths one by one, each with a case that is known to reach it: units of
one and of two blocks of query rows, pages that are copied 16 bytes a lane."""
import pytest
import torch

from test_gpu_paged_attention import check, gdn  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def blocks_of(new, Hq, Hk):
    """Blocks of up to 128 query rows that a batch has by its mean number of tokens, and whether
    units have two each: where there are as many as multiprocessors."""
    G = Hq // Hk
    per_key = -(-G // 128)
    tokens = 128 // -(-G // per_key)
    blocks = -(-(-(-sum(new) // len(new))) // tokens)
    n = blocks * len(new) * Hk * per_key
    return n, blocks > 1 and n >= torch.cuda.get_device_properties(0).multi_processor_count


def tiles_a_cta(new, lens, Hq, Hk):
    """Tiles of 128 keys that a CTA has on average, causal, no window, at the least."""
    n, two = blocks_of(new, Hq, Hk)
    units = n / (len(new) * (2 if two else 1))  # of a row
    return sum(units * m / 256 for m in lens) / torch.cuda.get_device_properties(0).multi_processor_count


ROWS = {  # tokens and keys of the rows, and whether units have two blocks
    "single": ([1] * 150, [400 + 13 * b for b in range(150)], False),
    "chunks": ([300] * 26, [300 + 60 * b for b in range(26)], True),
}


@pytest.mark.parametrize("dtype,d,page", [("bf16", 64, 20), ("f16", 128, 7), ("bf16", 128, 12), ("f16", 32, 1)])
@pytest.mark.parametrize("rows", ROWS)
def test_pages_of_odd_sizes_over_many_tiles(gdn, rows, dtype, d, page):  # noqa: F811
    """More tiles a CTA than stages in flight, so that copies wait for stages to come free."""
    new, lens, two = ROWS[rows]
    assert blocks_of(new, 8, 2)[1] == two and tiles_a_cta(new, lens, 8, 2) > 6
    check(gdn, new, lens, 8, 2, d, page, dtype, packed=False)
