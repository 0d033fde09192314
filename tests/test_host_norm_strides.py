"""The stride of a gate that is not there is not looked at.  Each call is refused for the
overlap of its output, the last of the checks, so nothing is launched."""
import pytest

ALIAS = 3
A, GiB = 1 << 32, 1 << 30


@pytest.fixture(scope="module")
def L():
    from gated_deltanet_recurrence_02_gb300 import build, gdn
    build.build()
    return gdn.lib()


@pytest.mark.parametrize("stride", [0, -1, -(1 << 62), (1 << 63) - 1])
def test_stride_without_a_gate(L, stride):
    # x, z, weight, out, N, H, d, strides, eps, gate, dtypes, stream
    assert L.gdn_gated_norm(A, None, None, A + 64, 4, 2, 64, 128, stride, 128, 1e-6, 0, 2, 0, None) == ALIAS
    # y, residual, gate, weights, residual_out, out, N, D, strides, scale, eps, flags, dtypes, stream
    assert L.gdn_residual_norm(A, A + GiB, None, None, None, A + 2 * GiB, A + 64, 4, 128, 128, stride, 1.0, 1e-6, 0,
                               2, 0, 0, None) == ALIAS


INVALID = 1


@pytest.mark.parametrize("n,stride", [(3, (1 << 63) - 1), (5, 1 << 62), (1 << 30, 1 << 40)])
def test_rows_past_the_address_space(L, n, stride):
    """Spans whose bytes do not fit a size: refused, wherever the product or the sum wraps."""
    def gated(xs=128, zs=128, os=128):
        return L.gdn_gated_norm(A, A + GiB, None, A + 2 * GiB, n, 1, 128, xs, zs, os, 1e-6, 1, 2, 0, None)
    assert gated(xs=stride) == gated(zs=stride) == gated(os=stride) == INVALID
    assert L.gdn_residual_norm(A, None, None, None, None, A + GiB, A + 2 * GiB, n, 128, stride, 128, 1.0, 1e-6, 0,
                               2, 2, 0, None) == INVALID
