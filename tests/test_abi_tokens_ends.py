"""Sizes and strides at the ends of their types, on the host (no GPU needed)."""
import pytest

from test_abi_grouped import m  # noqa: F401


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
