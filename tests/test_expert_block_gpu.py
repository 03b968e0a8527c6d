"""The example block (norms, routing, permutation, 16-bit expert products, gated
activation, combine) against the same formulas in 64 bits with automatic
differentiation, and its training steps.

Tolerance: about a dozen tensors on the way are rounded to bf16, each off by at
most 2^-9 of its values on average; independent roundings add to less than
sqrt(12) 2^-9 < 0.7 % of a result's norm, and sums of opposite signs may leave
a result a few times smaller than its terms: 3 %.
"""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from tests.util import build_lib  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def X():
    build_lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_block
    return expert_block


def reference(block, x, ids, dout, dx_out):
    """Gradients of <dout, out> + <dx_out, x'> with the experts `ids` given."""
    w = {n: t.detach().double().cpu().requires_grad_() for n, t in block.w.items()}
    x = x.double().cpu().requires_grad_()
    ids = ids.long().cpu()
    norm = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)
    h = norm(x) * w["gamma_in"]
    rw = torch.softmax((h @ w["router"].T).gather(1, ids), dim=1)
    y = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            gu = w["w13"][e] @ h[t]
            y[t] = y[t] + rw[t, j] * (w["w2"][e] @ (torch.nn.functional.silu(gu[:block.f]) * gu[block.f:]))
    x_out = x + block.alpha * w["gate"] * norm(y) * w["gamma_post"]
    out = norm(x_out) * w["gamma_out"]
    ((out * dout.double().cpu()).sum() + (x_out * dx_out.double().cpu()).sum()).backward()
    return out.detach(), x_out.detach(), x.grad, {n: t.grad for n, t in w.items()}


def near(got, ref, what):
    got = got.detach().double().cpu()
    rel = ((got - ref).norm() / ref.norm()).item()
    assert rel < 0.03, (what, rel)


@pytest.mark.parametrize("T", [1, 3, 40])
def test_block_and_its_gradients(X, T):
    block = X.ExpertBlock(d=256, f=72, E=6, k=2, alpha=0.8, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda: torch.randn(T, 256, generator=g, device="cuda").to(torch.bfloat16)
    x, dout, dx_out = rnd(), rnd(), rnd()
    s = block.forward(x)
    dx, grads = block.backward(s, dout, dx_out)
    out, x_out, rdx, rgrads = reference(block, x, s["ids"], dout, dx_out)
    near(s["out"], out, "out")
    near(s["x_out"], x_out, "x_out")
    near(dx, rdx, "dx")
    for name, r in rgrads.items():
        near(grads[name], r, name)
    import bit_quantized_expert_moe_gb300 as M
    assert M.get_device_error(block.ws) == M.MOE_OK


def test_training_lowers_the_loss(X, capsys, monkeypatch):
    monkeypatch.setattr(sys, "argv", ["expert_block.py", "--tokens", "256", "--steps", "4"])
    X.main()
    lines = capsys.readouterr().out.splitlines()
    losses = [float(line.split()[-1]) for line in lines if line.startswith("step")]
    assert len(losses) == 4 and all(b < a for a, b in zip(losses, losses[1:])), losses
    assert lines[-1].startswith("single token: (1, 1024)")
