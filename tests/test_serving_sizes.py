"""Sizes of the serving operators that do not fit 32 bits are refused before they
reach the library, which would see their low 32 bits."""
import pytest

from adaptive_top_sparse_quest_b200 import TwError, build, prefix_workspace_bytes


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


@pytest.mark.parametrize("sizes", [(2 ** 32 + 1, 8, 2, 16), (4, 2 ** 32 + 8, 2, 16),
                                   (4, 8, 2 ** 32 + 2, 16), (4, 8, 2, 2 ** 32)])
def test_prefix_workspace_past_32_bits(sizes):
    with pytest.raises(ValueError):
        prefix_workspace_bytes(*sizes)


@pytest.mark.parametrize("sizes", [(-1, 8, 2, 16), (4, 8, 3, 16), (4, 8, 2, -16), (4, 8, 2, 24)])
def test_prefix_workspace_refusals(sizes):
    with pytest.raises(TwError):
        prefix_workspace_bytes(*sizes)
    assert prefix_workspace_bytes(4, 8, 2, 32) > prefix_workspace_bytes(4, 8, 2, 0) > 0
