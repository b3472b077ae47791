"""Sizes and strides at the ends of their types, on the host (no GPU needed)."""
import pytest

from test_abi_grouped import UNSUPPORTED, P, m  # noqa: F401
from test_abi_tokens import COMBINE, GRAD, CombineArgs, CombineGradArgs, call


@pytest.mark.parametrize("sizes", [
    (1000, 513, 64, 128, 9), (1000, 65536, 64, 128, 9), (1000, 4, 12, 128, 9), (1 << 26, 4, 64, 128, 9),
    (1000, 4, 1 << 18, 1 << 13, 9), (1000, 4, 1 << 30, 1 << 16, 9), ((1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 8, 65536, 9),
])
def test_product_workspace_of_unsupported_sizes(m, sizes):  # noqa: F811
    # sizes that the product itself refuses
    assert m.load().moe_grouped_int8_workspace_size(*sizes) == 0


def test_product_workspace_at_the_ends(m):  # noqa: F811
    size, most = m.load().moe_grouped_int8_workspace_size, (1 << 26) - 1
    assert size(most, 512, 8, 65536, most) == most * 65536 + most * 4
    assert size(most, 1, (1 << 27) - 8, 16, 1) == 256 + 4


WRAPS = [(1 << 62) + 64, (1 << 61) + 64, (1 << 63) - 64]  # elements whose bytes pass 2^63


@pytest.mark.parametrize("stride", WRAPS)
@pytest.mark.parametrize("rows_type", [0, 1])
def test_strides_whose_bytes_wrap(m, stride, rows_type):  # noqa: F811
    # each beside a pointer that is refused behind it, so that no call goes on
    kw = dict(rows_type=rows_type, rows_stride=stride, y=None)
    assert call(m, "moe_combine", CombineArgs, COMBINE, kw) == UNSUPPORTED
    kw = dict(rows_type=rows_type, rows_stride=stride, drows=P + 8)
    assert call(m, "moe_combine_grad", CombineGradArgs, GRAD, kw) == UNSUPPORTED
    kw = dict(dy_type=rows_type, dy_stride=stride, drows=P + 8)
    assert call(m, "moe_combine_grad", CombineGradArgs, GRAD, kw) == UNSUPPORTED
