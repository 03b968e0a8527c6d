"""One workspace for all calls of a stream: the operators of expert blocks, the one-kernel
int4 layer and the 16-bit products, each with the result that it has in a space of its own."""
import pytest

torch = pytest.importorskip("torch")

from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


def randn(seed, dtype, *shape, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def codes(seed, *shape):
    return torch.randint(-127, 128, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int8).cuda()


@pytest.mark.parametrize("T,R,D,dtype", [(1024, 8192, 2048, BF16), (301, 9000, 2048, F16), (64, 1500, 12304, F32)])
def test_rows_to_codes_leave_the_header_as_it_is(M, T, R, D, dtype):
    x, k = randn(1, dtype, T, D), 3
    m = torch.randint(0, T * k, (R,), generator=torch.Generator().manual_seed(2), dtype=torch.int32).cuda()
    need = M.quantize_rows_workspace_size(T, R, D)
    assert need > 256
    for fill in (0, 0x5A):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got = M.quantize_rows(x, m, k, ws=ws)
        assert (ws[:256] == fill).all()
        assert all(torch.equal(a, b) for a, b in zip(got, M.quantize_rows(x, m, k)))


def test_one_workspace_for_all_calls(M):
    """Twice in turn, so that every kind of call comes behind every other one."""
    E, k, d, f, T, many = 16, 4, 512, 256, 4, 5000
    x, lg = randn(1, BF16, T, d), randn(2, F32, T, E)
    w13, w2 = randn(3, BF16, E, 2 * f, d, scale=d ** -0.5), randn(4, BF16, E, d, f, scale=f ** -0.5)
    c13, s13 = codes(5, E, 2 * f, d), randn(6, F32, E, 2 * f).abs() * 1e-3
    rows, lg_many = randn(7, BF16, many, 2 * d), randn(8, F32, many, E)
    ids, _ = M.route_topk(lg_many, k)
    perm = M.permute(ids, E)
    few = torch.arange(E + 1, dtype=torch.int32, device="cuda")  # a row an expert
    xq, xs = codes(9, perm["sorted"].numel(), d), randn(10, F32, perm["sorted"].numel()).abs()
    w16 = randn(11, BF16, E, 256, 2 * d, scale=d ** -0.5)
    gamma, beta = randn(12, BF16, 2 * d), randn(13, BF16, 2 * d)
    words = lambda *s: torch.randint(-2 ** 31, 2 ** 31, s, dtype=torch.int64).to(torch.int32).cuda()  # noqa: E731
    half = lambda v, *s: torch.full(s, v, dtype=F16, device="cuda")  # noqa: E731
    int4 = M.Layer(E=E, d_model=d, d_ff=f, w13_q=words(E, 2 * f, d // 8), w13_s=half(0.01, E, 2 * f, d // 128),
                   w13_z=half(8.0, E, 2 * f, d // 128), w2_q=words(E, d, f // 8), w2_s=half(0.01, E, d, f // 128),
                   w2_z=half(8.0, E, d, f // 128))

    def int4_layer(ws):
        out = torch.empty(T, d, dtype=BF16, device="cuda")
        M.LayerCall(int4, T, k, ws=ws)(x, lg, out)
        return out

    R = perm["sorted"].numel()
    calls = {
        "quantize_rows": (M.quantize_rows_workspace_size(many, R, 2 * d),
                          lambda ws: M.quantize_rows(rows, perm["sorted"], k, ws=ws)),
        "expert_layer": (M.expert_layer_workspace_size(T, k, E, d, f), lambda ws: [M.expert_layer(x, lg, w13, w2, k, ws=ws)]),
        "int4 layer": (M.layer_workspace_size(int4, T, k), lambda ws: [int4_layer(ws)]),
        "8-bit, many rows": (M.grouped_mm_i8_workspace_size(R, E, 2 * f, d),
                             lambda ws: [M.grouped_mm_i8(xq, xs, c13, s13, perm["offsets"], ws=ws)]),
        "8-bit, few rows": (M.grouped_mm_i8_workspace_size(E, E, 2 * f, d),
                            lambda ws: [M.grouped_mm_i8(xq[:E], xs[:E], c13, s13, few, ws=ws)]),
        "16-bit": (M.grouped_mm_workspace_size(many, E, 256, 2 * d),
                   lambda ws: [M.grouped_mm(rows, w16, few * (many // E), ws=ws)[:many // E * E]]),
        "layer norm": (M.layer_norm_backward_workspace_size(many, 2 * d),
                       lambda ws: M.layer_norm_backward(rows, rows, None, gamma, beta, ws=ws)),
    }
    want = {}
    for name, (size, call) in calls.items():
        ws = M.workspace(size)
        want[name] = [t.clone() for t in call(ws)]
        assert M.get_device_error(ws) == M.MOE_OK, name
    ws = M.workspace(max(size for size, _ in calls.values()))
    torch.cuda.synchronize()
    order = list(calls) + list(calls)[::-1] + [n for a in calls for n in (a, "expert_layer", a, "int4 layer")]
    got = [(name, calls[name][1](ws)) for name in order]  # no wait between the calls
    torch.cuda.synchronize()
    for name, outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want[name])), name
    assert M.get_device_error(ws) == M.MOE_OK
