"""The compiled entry points run on the device of their operands and refuse
operands of several devices before any launch.  Tensors of two devices are stood in
for by fake ones, which have shapes, types and devices but no memory (no GPU
needed)."""
import warnings

import pytest

from tests.util import build_lib

torch = pytest.importorskip("torch")
fake_tensor = pytest.importorskip("torch._subclasses.fake_tensor")

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
CALLS = {
    "grouped_mm": {"x": ((4, 16), BF16), "w": ((2, 24, 16), BF16), "offsets": ((3,), I32), "y": ((4, 24), BF16), "ws": ((4096,), U8)},
    "grouped_mm_dx": {"dy": ((4, 24), BF16), "w": ((2, 24, 16), BF16), "offsets": ((3,), I32), "dx": ((4, 16), BF16),
                      "ws": ((4096,), U8)},
    "grouped_mm_dw": {"dy": ((4, 24), BF16), "x": ((4, 16), BF16), "offsets": ((3,), I32), "dw": ((2, 24, 16), BF16),
                      "ws": ((4096,), U8)},
    "swiglu": {"gu": ((4, 32), BF16), "row_w": ((4,), F32), "row_map": ((4,), I32), "h": ((4, 16), BF16)},
    "swiglu_backward": {"dh": ((4, 16), BF16), "gu": ((4, 32), BF16), "row_w": ((4,), F32), "row_map": ((4,), I32),
                        "dgu": ((4, 32), BF16), "drow_w": ((4,), F32)},
    "block_norm": {"x": ((4, 16), BF16), "y": ((4, 16), BF16), "gamma_post": ((16,), BF16), "gate": ((2, 16), BF16),
                   "gamma_pre": ((16,), BF16), "x_out": ((4, 16), BF16), "h": ((4, 16), BF16)},
    "block_norm_backward": {"x_out": ((4, 16), BF16), "y": ((4, 16), BF16), "dx_out": ((4, 16), BF16), "dh": ((4, 16), BF16),
                            "gamma_post": ((16,), BF16), "gate": ((2, 16), BF16), "gamma_pre": ((16,), BF16),
                            "ws": ((65536,), U8)},
}


@pytest.fixture(scope="module")
def M():
    try:
        build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    import bit_quantized_expert_moe_gb300 as M
    return M


@pytest.mark.parametrize("fn,other", [(fn, name) for fn, args in CALLS.items() for name in args])
def test_operands_of_two_devices_are_refused(M, fn, other):
    with fake_tensor.FakeTensorMode():
        args = {n: torch.empty(s, dtype=t, device="cuda:1" if n == other else "cuda:0") for n, (s, t) in CALLS[fn].items()}
    with pytest.raises(ValueError, match="tensors of one device expected, not of cuda:[01] and cuda:[01]"):
        getattr(M, fn)(**args)


@pytest.mark.parametrize("fn", CALLS)
def test_one_operand_on_the_host_is_refused(M, fn):
    for host in CALLS[fn]:
        with fake_tensor.FakeTensorMode():
            args = {n: torch.empty(s, dtype=t, device="cpu" if n == host else "cuda:0") for n, (s, t) in CALLS[fn].items()}
        with pytest.raises(ValueError, match="device tensor expected"):
            getattr(M, fn)(**args)


def test_operands_that_require_gradients_are_not_passed_over_in_silence(M):
    """The operators record no graph.  The calls here are refused after the warning (host tensors)."""
    plain, grad = torch.zeros(4, 32), torch.zeros(4, 32, requires_grad=True)

    def refused(*args):
        with pytest.raises(ValueError, match="device tensor"):
            M.block_norm(*args)

    with pytest.warns(UserWarning, match="record no graph"):
        refused(grad)
    with pytest.warns(UserWarning, match="record no graph"):
        refused(plain, grad)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        refused(plain, plain)
        with torch.no_grad():
            refused(grad)
        with pytest.raises(UserWarning):  # an error where the program's filters make it one
            M.block_norm(grad)


@pytest.mark.gpu
def test_operands_that_require_gradients_are_computed_with(M):
    x, p = torch.randn(4, 32).cuda(), torch.ones(32).cuda()
    want = M.block_norm(x, gamma_pre=p)[1]
    with pytest.warns(UserWarning, match="record no graph"):
        got = M.block_norm(x, gamma_pre=p.clone().requires_grad_())[1]
    assert torch.equal(got, want) and not got.requires_grad
