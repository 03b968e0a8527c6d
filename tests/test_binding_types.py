"""The Python entry points of the int4 layer and of routing, permutation and
combine refuse tensors whose bits the kernels would read as another type, before
any launch (no GPU needed)."""
import pytest

from tests.util import build_lib

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def M():
    try:
        build_lib()
    except RuntimeError as e:  # pragma: no cover
        pytest.skip(f"cannot build: {e}")
    import bit_quantized_expert_moe_gb300 as M
    return M


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


I32, F32, F16, BF16 = torch.int32, torch.float32, torch.float16, torch.bfloat16


def layer(M):
    return M.Layer(2, 256, 256, *[zeros(1)] * 6)


CALLS = {
    "combine of fp16 rows": (lambda M: M.combine(zeros(4, 16, dtype=F16), zeros(4, dtype=I32), zeros(2, 2, dtype=F32)), "y_perm"),
    "combine of fp32 rows": (lambda M: M.combine(zeros(4, 16, dtype=F32), zeros(4, dtype=I32), zeros(2, 2, dtype=F32)), "y_perm"),
    "permute of fp32 rows": (lambda M: M.permute(zeros(2, 2, dtype=I32), 4, zeros(2, 16, dtype=F32), want_x_perm=True,
                                                 ws=zeros(4096, dtype=torch.uint8)), "x"),
    "permute of 64-bit ids": (lambda M: M.permute(zeros(2, 2, dtype=torch.int64), 4, ws=zeros(4096, dtype=torch.uint8)), "topk_ids"),
    "routing of bf16 logits": (lambda M: M.route_topk(zeros(2, 8), 2), "logits"),
    "int4 experts of fp16 rows": (lambda M: M.expert_ffn_w4a16(layer(M), zeros(4, 256, dtype=F16), zeros(3, dtype=I32),
                                                               ws=zeros(4096, dtype=torch.uint8)), "x_perm"),
}


@pytest.mark.parametrize("name", CALLS)
def test_types_that_the_kernels_do_not_read_are_refused(M, name):
    call, what = CALLS[name]
    with pytest.raises(ValueError, match=f"^{what}: torch.* expected, not torch"):
        call(M)


def test_the_layer_refuses_rows_and_logits_of_another_type(M):
    call = M.LayerCall.__new__(M.LayerCall)  # without weights on a device: refused before they are looked at
    call.L, call.T, call.k, call.ws = M.moe_w4_layer(), 2, 2, zeros(4096, dtype=torch.uint8)
    call._fn = M.lib().moe_layer_forward
    with pytest.raises(ValueError, match="^x: torch.bfloat16 expected, not torch.float16"):
        call(zeros(2, 256, dtype=F16), zeros(2, 8, dtype=F32), zeros(2, 256))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_permuted_rows_keep_their_type(M, dtype):
    """fp16 rows come out as fp16, so that the grouped products of fp16 experts
    take them: one rounding to the type, and the fp32 sums of d products (d / 8 +
    16 roundings of 2^-23 of the sum of their absolute values)."""
    g = torch.Generator().manual_seed(1)
    T, k, E, d = 37, 2, 5, 64
    x = torch.randn(T, d, generator=g).to(dtype).cuda()
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int().cuda()
    p = M.permute(ids, E, x, want_x_perm=True)
    assert p["x_perm"].dtype is dtype and torch.equal(p["x_perm"], x[(p["sorted"] // k).long()])
    w = torch.randn(E, 24, d, generator=g).to(dtype).cuda()
    y = M.grouped_mm(p["x_perm"], w, p["offsets"])
    r = 0
    for e in range(E):
        n = int(p["counts"][e])
        rows, we = p["x_perm"][r:r + n].double(), w[e].double()
        ref, terms = rows @ we.t(), rows.abs() @ we.abs().t()
        tol = 2.0 ** (-8 if dtype is BF16 else -11) * ref.abs() + (d / 8 + 16) * 2.0 ** -23 * terms + 2.0 ** -25
        assert ((y[r:r + n].double() - ref).abs() <= tol).all()
        r += n
