"""Rows whose numbers the kernels' 32-bit steps would carry past the largest integer
are refused on the host (no GPU needed; nothing is launched with the pointers)."""
import pytest

from tests.util import build_lib

UNSUPPORTED = 3
BF16 = 0
P = 0x100000  # 16-byte aligned, never dereferenced
BIG = 1 << 62
MOST = 2 ** 31 - 2 ** 24 - 1


@pytest.fixture(scope="module")
def lib():
    try:
        build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    import bit_quantized_expert_moe_gb300 as M
    return M.lib()


@pytest.mark.parametrize("rows", [MOST + 1, 2 ** 31 - 1])
def test_rows_beyond_the_limit_are_refused(lib, rows):
    for fn in (lib.moe_grouped_mm, lib.moe_grouped_mm_dx, lib.moe_grouped_mm_dw):
        assert fn(BF16, P, P, P, rows, 2, 8, 8, P, P, BIG, None) == UNSUPPORTED
    assert lib.moe_swiglu(BF16, P, P, P, rows, 8, P, None) == UNSUPPORTED
    assert lib.moe_swiglu_backward(BF16, P, P, P, P, rows, 8, P, P, None) == UNSUPPORTED
    norm = (BF16, BF16, rows, 8, 1, 1.0, 1e-6, P, P, P)
    assert lib.moe_block_norm(*norm, P, P, P, P, None) == UNSUPPORTED
    assert lib.moe_block_norm_backward(*norm, P, P, P, P, P, P, P, P, P, P, BIG, None) == UNSUPPORTED


def test_steps_stay_within_32_bits_up_to_the_limit():
    """The largest numbers that the kernels' row loops form on 152 SMs."""
    sms, top = 152, 2 ** 31
    for threads in (32, 64, 128, 256, 512):  # of a row group of the norms
        groups = min(1024 // threads, 15)
        assert MOST + 5 * sms * groups < top                 # forward: four steps of loads ahead
        rows = -(-MOST // (sms * groups))                    # backward: consecutive rows of a group
        assert (sms * groups - 1) * rows + rows < top
    assert MOST + 5 * sms * 8 < top                          # gated activation, backward
    assert MOST + 256 < top                                  # rows of a tile rounded up
