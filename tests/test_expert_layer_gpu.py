"""The whole layer of 16-bit experts for a few tokens, on the GPU, against its formula in
64 bits.

Tolerance of an output, besides the rounding to its type (u |ref|, u = 2^-8 bf16, 2^-11
fp16, half the spacing among the subnormals), in units of 2^-24:
  - a product of L terms adds 16 of them to an fp32 accumulator at a time:
    s(L) = 2 (L / 8 + 16) of sum |a b|, as for the grouped products;
  - h = SiLU(a) u takes 1.1 |u| of the error of a (the slope of SiLU is below 1.1) and
    |SiLU(a)| of that of u, and 16 of |h| for the exponential, quotient and products;
  - h as two 16-bit numbers is off by u^2 |h| (fp16: at least 2^-25 in all);
  - weights p: 16.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
U = {BF16: 2.0 ** -8, F16: 2.0 ** -11}
SUBNORMAL = {BF16: 2.0 ** -134, F16: 2.0 ** -25}


@pytest.fixture(scope="module")
def M():
    build_lib()
    import bit_quantized_expert_moe_gb300 as M
    return M


def randn(seed, dtype, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def steps(length):
    return 2 * (length / 8 + 16)


def choose(logits, k):
    """The largest logits, equal ones by the lower expert, and their softmax in 64 bits."""
    lg = logits.double().numpy()
    ids = np.stack([np.lexsort((np.arange(lg.shape[1]), -row))[:k] for row in lg])
    top = np.take_along_axis(lg, ids, 1)
    p = np.exp(top - top[:, :1])
    return ids, p / p.sum(1, keepdims=True)


def reference(x, logits, w13, w2, k):
    """out, its tolerance and the ids."""
    T, d = x.shape
    f = w2.shape[2]
    u16 = U[x.dtype]
    ids, p = choose(logits, k)
    out = torch.zeros(T, d, dtype=torch.float64)
    tol = torch.zeros(T, d, dtype=torch.float64)
    one = 2.0 ** -24
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        xe, wd = x[t].double(), w2[e].double()
        w = w13[e].double()
        gu, big = xe @ w.T, xe.abs() @ w.abs().T
        a, u, ba, bu = gu[:, :f], gu[:, f:], big[:, :f], big[:, f:]
        s = a * torch.sigmoid(a)
        h = s * u
        dh = one * (steps(d) * (1.1 * ba * u.abs() + s.abs() * bu) + (16 + 16) * h.abs()) + u16 * u16 * h.abs()
        if x.dtype == F16:
            dh = dh + 2.0 ** -25
        pe = torch.from_numpy(p[t, j])[:, None]
        out.index_add_(0, torch.from_numpy(t), pe * (h @ wd.T))
        tol.index_add_(0, torch.from_numpy(t), pe * (dh @ wd.abs().T + one * steps(f) * (h.abs() @ wd.abs().T)))
    return out, tol + u16 * out.abs() + SUBNORMAL[x.dtype], ids


def case(seed, T, k, E, d, f, dtype):
    return (randn(seed, dtype, T, d), randn(seed + 1, torch.float32, T, E), randn(seed + 2, dtype, E, 2 * f, d, scale=d ** -0.5),
            randn(seed + 3, dtype, E, d, f, scale=f ** -0.5))


def check(got, want, tol, what=""):
    err = (got.cpu().double() - want).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), (what, (err - tol).max().item(), err.max().item())


CASES = [
    # T, k, E, d, f
    (1, 1, 1, 64, 64),
    (1, 8, 128, 2048, 768),       # one token
    (2, 2, 8, 256, 512),
    (3, 3, 5, 128, 192),
    (8, 8, 64, 512, 256),
    (5, 6, 40, 1088, 320),        # 17 blocks of 64 inputs, 5 of h
    (7, 1, 3, 64, 1088),
    (1, 4, 4, 4928, 128),         # 32 and 33 output features a CTA: tiles of two sizes
    (2, 2, 4, 192, 2112),
    (9, 2, 4, 320, 192),          # several tokens an expert: one group of 8 and two
    (16, 1, 1, 448, 128),
    (17, 8, 16, 256, 320),
    (32, 8, 8, 128, 64),          # every token at every expert
    (32, 1, 2, 576, 704),
    (27, 3, 17, 576, 320),
    (8, 32, 64, 64, 128),
    (31, 5, 200, 192, 64),
    (32, 8, 64, 1088, 320),       # more chunks than slots, one and several groups of 8
    (12, 4, 16, 1088, 1088),
    (24, 6, 30, 192, 2112),
    (14, 3, 7, 64, 192),
    (4, 6, 24, 640, 1600),        # h in three chunks an expert; up to 4 tokens, and 5
    (5, 6, 24, 640, 1600),
    (32, 8, 20, 128, 832),        # more than 16 tokens of an expert
    (32, 4, 8, 2496, 64),         # tiles of 17 output features
    (28, 6, 101, 384, 256),       # many experts of few tokens: several rounds of parts of slots
    (8, 8, 60, 256, 1600),
    (13, 5, 90, 1280, 192),
]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,k,E,d,f", CASES)
def test_expert_layer(M, T, k, E, d, f, dtype):
    x, lg, w13, w2 = case(T + E + d, T, k, E, d, f, dtype)
    want, tol, ids = reference(x, lg, w13, w2, k)
    ws = M.workspace(M.expert_layer_workspace_size(T, k, E, d, f))
    got_ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    xd, lgd, w13d, w2d = x.cuda(), lg.cuda(), w13.cuda(), w2.cuda()
    got = M.expert_layer(xd, lgd, w13d, w2d, k, ids=got_ids, ws=ws)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    check(got, want, tol)
    assert M.get_device_error(ws) == M.MOE_OK
    # a fixed order of the sums; a workspace of its own
    assert torch.equal(got, M.expert_layer(xd, lgd, w13d, w2d, k))
    assert torch.equal(got, M.expert_layer(xd, lgd, w13d, w2d, k, out=xd, ws=ws))  # in place


def test_ties_and_excluded_experts(M):
    """Equal logits go to the lower expert; experts at -inf or the lowest value are not chosen,
    or have no weight where there are no others."""
    T, k, E, d, f = 4, 3, 12, 128, 64
    x, _, w13, w2 = case(1, T, k, E, d, f, BF16)
    lg = torch.zeros(T, E)
    lg[1, :9] = float("-inf")
    lg[2, 1:] = torch.finfo(torch.float32).min
    lg[3, 2:] = float("-inf")
    lg[3, 1] = -0.0
    want, tol, ids = reference(x, lg, w13, w2, k)
    got_ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    got = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k, ids=got_ids)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    check(got, want, tol)


def test_an_expert_that_is_not_finite_spoils_its_own_tokens_alone(M):
    T, k, E, d, f = 6, 2, 8, 192, 128
    x, lg, w13, w2 = case(2, T, k, E, d, f, BF16)
    _, _, ids = reference(x, lg, w13, w2, k)
    e = int(ids[0, 0])
    clean = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k)
    w13[e, 5, 7] = float("nan")
    got = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k)
    has = torch.from_numpy((ids == e).any(1))
    assert torch.isnan(got[has]).all() and torch.equal(got[~has], clean[~has])


@pytest.mark.parametrize("T", [2, 4, 8, 20])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_down_weights_that_are_not_finite(M, T, value):
    """The tokens of other experts are as they were."""
    k, E, d, f = 2, 8, 192, 128
    x, lg, w13, w2 = case(5, T, k, E, d, f, BF16)
    lg[0, 3], lg[1, 3] = 9.0, -9.0
    _, _, ids = reference(x, lg, w13, w2, k)
    clean = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k)
    w2[3, ::5] = value
    got = M.expert_layer(x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k)
    has = torch.from_numpy((ids == 3).any(1))
    assert has[0] and not has[1]
    assert not torch.isfinite(got[has][:, ::5]).any() and torch.equal(got[~has], clean[~has])
    other = torch.arange(d) % 5 > 0
    assert torch.equal(got[:, other], clean[:, other])


def test_logits_that_are_no_numbers(M):
    """No read out of range, and other tokens are as they were."""
    T, k, E, d, f = 3, 2, 8, 128, 64
    x, lg, w13, w2 = case(3, T, k, E, d, f, BF16)
    args = w13.cuda(), w2.cuda(), k
    clean = M.expert_layer(x.cuda(), lg.cuda(), *args)
    bad = lg.clone()
    bad[1] = torch.tensor(-1, dtype=torch.int32).view(torch.float32)  # NaNs of all bits
    ws = M.workspace(M.expert_layer_workspace_size(T, k, E, d, f))
    got = M.expert_layer(x.cuda(), bad.cuda(), *args, ws=ws)
    assert torch.equal(got[[0, 2]], clean[[0, 2]])
    assert M.get_device_error(ws) == 6
    assert torch.equal(M.expert_layer(x.cuda(), lg.cuda(), *args, ws=ws), clean)


def test_no_tokens(M):
    x, lg, w13, w2 = case(4, 1, 1, 2, 64, 64, BF16)
    out = M.expert_layer(x[:0].cuda(), lg[:0].cuda(), w13.cuda(), w2.cuda(), 1)
    assert out.shape == (0, 64)


def test_calls_back_to_back_and_graphs(M):
    """One workspace for several layers, eager and as two graphs, on a stream of their own."""
    E, d, f, k = 16, 512, 192, 4
    ws = M.workspace(M.expert_layer_workspace_size(20, k, E, d, f))
    layers = [case(10 * i, 20, k, E, d, f, BF16)[2:] for i in range(3)]
    layers = [(a.cuda(), b.cuda()) for a, b in layers]
    x, lg = randn(50, BF16, 20, d).cuda(), [randn(60 + i, torch.float32, 20, E).cuda() for i in range(3)]

    def model(x, T):
        for (w13, w2), l in zip(layers, lg):
            x = M.expert_layer(x[:T], l[:T], w13, w2, k, ws=ws)
        return x

    single = {}
    for T in (1, 7, 20):
        y = x
        for (w13, w2), l in zip(layers, lg):
            y = M.expert_layer(y[:T], l[:T], w13, w2, k)
            torch.cuda.synchronize()
        single[T] = y
    for _ in range(20):
        for T in (1, 7, 20):
            assert torch.equal(model(x, T), single[T])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for T in (7, 20):
            model(x, T)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                y = model(x, T)
            graphs.append((g, y, single[T]))
        for i in range(20):
            g, y, want = graphs[i % 2]
            g.replay()
            side.synchronize()
            assert torch.equal(y, want)
    assert M.get_device_error(ws) == M.MOE_OK


def test_against_the_stages(M):
    """The layer and the chain of permute, grouped_mm, swiglu and combine: both within what
    their roundings allow of the formula."""
    T, k, E, d, f = 12, 4, 16, 512, 256
    x, lg, w13, w2 = case(5, T, k, E, d, f, BF16)
    want, tol, _ = reference(x, lg, w13, w2, k)
    xd, w13d, w2d = x.cuda(), w13.cuda(), w2.cuda()
    got = M.expert_layer(xd, lg.cuda(), w13d, w2d, k)
    check(got, want, tol)
    ids, p = M.route_topk(lg.cuda(), k)
    perm = M.permute(ids, E, xd, want_x_perm=True)
    act = M.swiglu(M.grouped_mm(perm["x_perm"], w13d, perm["offsets"]), p.view(-1), perm["sorted"])
    chain = M.combine(M.grouped_mm(act, w2d, perm["offsets"]), perm["inv"], torch.ones_like(p))
    # the chain rounds gate, up, h and y of every expert to bf16: 2^-8 each of what they add up to
    big = torch.zeros_like(want)
    ids = ids.cpu().numpy()
    for t in range(T):
        for j, e in enumerate(ids[t]):
            w = w13[e].double()
            a, u = w[:f] @ x[t].double(), w[f:] @ x[t].double()
            h = (1.1 * a.abs() * u.abs() + 2 * (a * torch.sigmoid(a) * u).abs())
            big[t] += p[t, j].item() * (w2[e].double().abs() @ h)
    assert ((chain.cpu().double() - want).abs() <= 4 * 2.0 ** -8 * big + tol).all()


def test_two_streams(M):
    """Calls on two streams with a workspace each: every launch needs all SMs, and none waits
    for one that has not started."""
    E, d, f, k, T = 16, 512, 192, 4, 9
    cases = []
    for i in range(2):
        x, lg, w13, w2 = (t.cuda() for t in case(20 * i, T, k, E, d, f, BF16))
        ws = M.workspace(M.expert_layer_workspace_size(T, k, E, d, f))
        cases.append((torch.cuda.Stream(), x, lg, w13, w2, ws, M.expert_layer(x, lg, w13, w2, k)))
    torch.cuda.synchronize()
    outs = []
    for _ in range(50):
        for s, x, lg, w13, w2, ws, want in cases:
            outs.append((M.expert_layer(x, lg, w13, w2, k, ws=ws, stream=s), want))
    torch.cuda.synchronize()
    assert all(torch.equal(got, want) for got, want in outs)
    assert all(M.get_device_error(c[5]) == M.MOE_OK for c in cases)


def test_a_barrier_wait_that_runs_out_reports_a_timeout(M):
    """The CTAs' arrival counter one short of a multiple of the grid: the first CTA passes, the
    others wait until the 2 s limit.  The call ends, reports it, and the next one is right."""
    T, k, E, d, f = 2, 2, 8, 256, 192
    x, lg, w13, w2 = case(30, T, k, E, d, f, BF16)
    want, tol, _ = reference(x, lg, w13, w2, k)
    args = x.cuda(), lg.cuda(), w13.cuda(), w2.cuda(), k
    ws = M.workspace(M.expert_layer_workspace_size(T, k, E, d, f))
    M.expert_layer(*args, ws=ws)
    assert M.get_device_error(ws) == M.MOE_OK
    n_sm = torch.cuda.get_device_properties(0).multi_processor_count
    count = ws[64:72].view(torch.int64)
    assert int(count.item()) == n_sm
    count.fill_(2 * n_sm - 1)
    M.expert_layer(*args, ws=ws)
    assert M.get_device_error(ws) == 7  # MOE_ERR_TIMEOUT
    assert int(ws[:256].count_nonzero()) == 0
    check(M.expert_layer(*args, ws=ws), want, tol)
    assert M.get_device_error(ws) == M.MOE_OK
