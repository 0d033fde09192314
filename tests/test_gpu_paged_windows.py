"""gdn_paged_attention: windows as wide as their type, which leave out no key, over rows that have
more tokens than keys (positions from below zero) and rows that have not."""
import pytest

from test_gpu_paged_attention import check, gdn  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 200, 2**30])
@pytest.mark.parametrize("new,lens,Hq", [([9], [4], 1), ([9], [4], 8), ([260], [101], 2), ([300, 5], [300, 700], 4)])
def test_widest_windows(gdn, dtype, window, new, lens, Hq):  # noqa: F811
    check(gdn, new, lens, Hq, 1, 64, 16, dtype, window=window)
