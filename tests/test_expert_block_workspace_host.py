"""Sizes of the workspaces of the operators of expert blocks (no GPU needed): the first 256
bytes of each are the header that every call leaves to the error word and the counters."""
import pytest

from tests.util import build_lib

HEADER = 256


@pytest.fixture(scope="module")
def M():
    try:
        build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    import bit_quantized_expert_moe_gb300 as M
    return M


@pytest.mark.parametrize("T,R,D", [(1000, 9000, 2048), (1024, 8192, 2048), (1, 600, 32768), (64, 1500, 12304)])
def test_rows_to_codes_have_the_header_beside_codes_and_scales(M, T, R, D):
    assert M.quantize_rows_workspace_size(T, R, D) >= HEADER + T * D + 4 * T


def test_rows_to_codes_without_a_workspace_need_no_header(M):
    assert M.quantize_rows_workspace_size(8, 64, 768) == 0
