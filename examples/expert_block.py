"""A mixture-of-experts block with 16-bit experts, forward and backward, on the
library's operators, and a few steps of training it.

    python examples/expert_block.py [--tokens 512] [--steps 5]

The block, for the residual stream x [T, d]:

    h = norm(x) gamma_in;  route h to k of E experts
    y = sum over a token's experts of weight * down_e(SiLU(gate_e h) up_e h)
    x' = x + alpha gate norm(y) gamma_post;  out = norm(x') gamma_out

The routing weight is applied between the two products (swiglu), so combine
sums with weights 1, and the gradient of combine is the permutation's gather.
The router's own product and the gradient of the softmax over the k selected
logits are plain torch.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_expert_moe_gb300 as moe  # noqa: E402


class ExpertBlock:
    """Weights, workspaces and the two passes; the gradients come as a dict with
    the names of the weights."""

    def __init__(self, d: int, f: int, E: int, k: int, alpha: float = 1.0, seed: int = 0, device="cuda"):
        self.d, self.f, self.E, self.k, self.alpha = d, f, E, k, alpha
        g = torch.Generator(device=device).manual_seed(seed)
        normal = lambda scale, *s: (torch.randn(*s, generator=g, device=device) * scale)  # noqa: E731
        bf = torch.bfloat16
        self.w = {
            "router": normal(d ** -0.5, E, d),
            "w13": normal(d ** -0.5, E, 2 * f, d).to(bf),
            "w2": normal(f ** -0.5, E, d, f).to(bf),
            "gamma_in": torch.ones(d, device=device),
            "gamma_post": torch.ones(d, device=device),
            "gate": torch.full((1, d), 0.5, device=device),
            "gamma_out": torch.ones(d, device=device),
        }
        self.ws = None

    def _workspaces(self, T: int) -> None:
        """One workspace for all calls: they follow each other on one stream."""
        R, E, d, f = T * self.k, self.E, self.d, self.f
        need = max(moe.grouped_mm_workspace_size(R, E, 2 * f, d), moe.grouped_mm_workspace_size(R, E, d, f),
                   moe.permute_workspace_size(T, self.k, E), moe.block_norm_backward_workspace_size(T, d))
        if self.ws is None or self.ws.numel() < need:
            self.ws = moe.workspace(need)

    def forward(self, x: torch.Tensor) -> dict:
        k, w = self.k, self.w
        self._workspaces(x.shape[0])
        ws = self.ws
        _, h = moe.block_norm(x, gamma_pre=w["gamma_in"])
        ids, rw = moe.route_topk(h.float() @ w["router"].t(), k)
        p = moe.permute(ids, self.E, h, want_x_perm=True, ws=ws)
        gu = moe.grouped_mm(p["x_perm"], w["w13"], p["offsets"], ws=ws)
        act = moe.swiglu(gu, rw.view(-1), p["sorted"])
        yp = moe.grouped_mm(act, w["w2"], p["offsets"], ws=ws)
        y = moe.combine(yp, p["inv"], torch.ones_like(rw))
        x_out, out = moe.block_norm(x, y, w["gamma_post"], w["gate"], w["gamma_out"], alpha=self.alpha)
        return {"x": x, "h": h, "ids": ids, "rw": rw, "perm": p, "gu": gu, "act": act, "y": y, "x_out": x_out, "out": out}

    def backward(self, s: dict, dout: torch.Tensor, dx_out: torch.Tensor | None = None):
        """(gradient of x, gradients of the weights) from those of out and of the stream x_out."""
        w, ws, k, p, g = self.w, self.ws, self.k, s["perm"], {}
        off = p["offsets"]
        dx, dy, g["gamma_post"], g["gate"], g["gamma_out"] = moe.block_norm_backward(
            s["x_out"], s["y"], dx_out, dout, w["gamma_post"], w["gate"], w["gamma_out"], self.alpha, ws=ws)
        dyp = dy[(p["sorted"] // k).long()]
        dact = moe.grouped_mm_dx(dyp, w["w2"], off, ws=ws)
        g["w2"] = moe.grouped_mm_dw(dyp, s["act"], off, ws=ws)
        dgu, drw = moe.swiglu_backward(dact, s["gu"], s["rw"].view(-1), p["sorted"])
        dxp = moe.grouped_mm_dx(dgu, w["w13"], off, ws=ws)
        g["w13"] = moe.grouped_mm_dw(dgu, p["x_perm"], off, ws=ws)
        dh = moe.combine(dxp, p["inv"], torch.ones_like(s["rw"])).float()
        # softmax over the selected logits, scattered to all experts
        drw = drw.view_as(s["rw"])
        dsel = s["rw"] * (drw - (s["rw"] * drw).sum(1, keepdim=True))
        dlogits = torch.zeros(s["x"].shape[0], self.E, device=dh.device).scatter_(1, s["ids"].long(), dsel)
        g["router"] = dlogits.t() @ s["h"].float()
        dh = (dh + dlogits @ w["router"]).to(torch.bfloat16)
        dx, _, _, _, g["gamma_in"] = moe.block_norm_backward(s["x"], None, dx, dh, gamma_pre=w["gamma_in"], ws=ws)
        return dx, g


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args()
    block = ExpertBlock(d=1024, f=512, E=32, k=4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, block.d, generator=gen, device="cuda").to(torch.bfloat16)
    target = torch.randn(a.tokens, block.d, generator=gen, device="cuda")
    for step in range(a.steps):
        s = block.forward(x)
        err = s["out"].float() - target
        loss = err.square().mean().item()
        _, grads = block.backward(s, (2 / err.numel() * err * 1024).to(torch.bfloat16))  # scaled: bf16 gradients
        for name, t in block.w.items():
            t.copy_(t.float() - 100.0 / 1024 * grads[name].float())
        print(f"step {step}: loss {loss:.4f}")
    one = block.forward(x[:1])  # a single token takes the same calls
    print("single token:", tuple(one["out"].shape), "experts", one["ids"].tolist()[0])
    if moe.get_device_error(block.ws) != moe.MOE_OK:
        raise RuntimeError("device error word set")


if __name__ == "__main__":
    main()
