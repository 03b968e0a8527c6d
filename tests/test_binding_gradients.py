"""An operand that requires gradients draws a warning that names what gives the gradients of
that operator, or says that nothing does.  The calls are refused after it (host tensors; no
GPU needed)."""
import re
import warnings

import pytest

from tests.util import build_lib

torch = pytest.importorskip("torch")

BF16, F32, I32, I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
# operands, which of them requires gradients, and what the warning names
CALLS = {
    "grouped_mm": ((((4, 16), BF16), ((2, 24, 16), BF16), ((3,), I32)), 1, ["grouped_mm_dx", "grouped_mm_dw"]),
    "grouped_mm_dx": ((((4, 24), BF16), ((2, 24, 16), BF16), ((3,), I32)), 0, []),
    "grouped_mm_dw": ((((4, 24), BF16), ((4, 16), BF16), ((3,), I32)), 0, []),
    "swiglu": ((((4, 32), BF16),), 0, ["swiglu_backward"]),
    "swiglu_backward": ((((4, 16), BF16), ((4, 32), BF16)), 1, []),
    "block_norm": ((((4, 16), BF16),), 0, ["block_norm_backward"]),
    "block_norm_backward": ((((4, 16), BF16), ((4, 16), BF16)), 0, []),
    "layer_norm": ((((4, 16), BF16), ((4, 16), BF16)), 1, ["layer_norm_backward"]),
    "layer_norm_backward": ((((4, 16), BF16), ((4, 16), BF16)), 0, []),
    "quantize_rows": ((((4, 16), BF16),), 0, []),
    "grouped_mm_i8": ((((4, 16), I8), ((4,), F32), ((2, 8, 16), I8), ((2, 8), F32), ((3,), I32)), 3, []),
    "expert_layer": ((((4, 64), BF16), ((4, 8), F32), ((8, 128, 64), BF16), ((8, 64, 64), BF16), 2), 2, []),
}


@pytest.fixture(scope="module")
def M():
    try:
        build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    import bit_quantized_expert_moe_gb300 as M
    return M


def test_every_operator_is_here(M):
    from bit_quantized_expert_moe_gb300 import expert16
    assert set(CALLS) == set(expert16.NAMES)


@pytest.mark.parametrize("fn", CALLS)
def test_the_warning_names_the_gradients_of_that_operator(M, fn):
    operands, which, names = CALLS[fn]
    args = [a if isinstance(a, int) else torch.zeros(a[0], dtype=a[1]) for a in operands]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError, match="device tensor"):
            getattr(M, fn)(*args)
    args[which].requires_grad_()
    with pytest.warns(UserWarning, match="record no graph") as said, pytest.raises(ValueError, match="device tensor"):
        getattr(M, fn)(*args)
    text = str(said[0].message)
    named = set(re.findall(r"[a-z_0-9]+", text)) & set(CALLS)
    assert named == {fn, *names}, text
    assert ("nothing that gives" in text) == (not names)
