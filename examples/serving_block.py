"""One block of a mixture-of-experts model as a server runs it, many requests at once:

    n      = norm of the residual stream (left by the block before)
    logits = n router_w^T                                   (a plain product)
    ids, w = sigmoid scores with a balance bias, the best groups, renormalised top-k
    f      = the experts for that routing + an ungated shared expert
    f_t   += scale B A n_t with the adapter of token t's request
    r, n   = r + gate * norm(f) and its norm, for the next block

Run it on a GB300 with ``python examples/serving_block.py``: a batch of 64 tokens, then one decode token replayed
from a CUDA graph.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fusion_backend_gb300 as fb  # noqa: E402


class ServingBlock:
    """Weights and, per number of tokens, the plan, workspaces and buffers that the server keeps."""

    H, E, TOP_K, I, IS, GROUPS, TOP_GROUPS, RANK, ADAPTERS = 2048, 128, 8, 768, 512, 8, 4, 16, 12

    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        bf = lambda *s, std=0.02: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
        self.router_w = bf(self.E, self.H)
        self.bias = torch.randn(self.E, generator=g, device="cuda") * 0.05
        self.expert_w, self.shexp_w = bf(self.E, 3, self.I, self.H), bf(3, self.IS, self.H)
        self.post_w, self.pre_w = bf(self.H, std=0.1) + 1, bf(self.H, std=0.1) + 1
        self.gate = torch.rand(self.H, generator=g, device="cuda") + 0.5
        self.lora_a = bf(self.ADAPTERS, self.RANK, self.H, std=self.H**-0.5)
        self.lora_b = bf(self.ADAPTERS, self.H, self.RANK, std=0.05)
        self.lora_scale = torch.rand(self.ADAPTERS, generator=g, device="cuda") + 0.5
        self.kept = {}

    def _keep(self, T: int):
        if T not in self.kept:
            new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
            self.kept[T] = dict(
                layer=fb.MoeFFN(fb.Shapes(T, self.H, self.E, self.TOP_K, self.I, self.IS), fb.ACT_BF16, fb.W_BF16),
                ids=new(T, self.TOP_K, dtype=torch.int32), w=new(T, self.TOP_K), out=new(T, self.H),
                ws=new(fb.moe_ffn_adapters_workspace(T, self.H, self.H, self.RANK), dtype=torch.uint8))
        return self.kept[T]

    def __call__(self, residual: torch.Tensor, normed: torch.Tensor, adapter_ids: torch.Tensor):
        """residual fp32 [T, H] and normed bf16 [T, H], both updated in place; adapter_ids int32 [T], -1: none."""
        k = self._keep(residual.shape[0])
        logits = normed.float() @ self.router_w.float().T
        fb.moe_ffn_route(logits, self.TOP_K, bias=self.bias, score=fb.SCORE_SIGMOID, groups=self.GROUPS,
                         top_groups=self.TOP_GROUPS, group_score=fb.GROUP_TOP2, ids=k["ids"], weights=k["w"])
        f = k["layer"].routed(normed, k["ids"], k["w"], self.expert_w, self.shexp_w, out=k["out"])
        fb.moe_ffn_add_adapters(f, normed, adapter_ids, self.lora_a, self.lora_b, scales=self.lora_scale,
                                workspace=k["ws"])
        return fb.moe_ffn_norm_residual(residual, f, post_norm=True, w_post=self.post_w, gate=self.gate,
                                        w_pre=self.pre_w, normed=normed)


def main() -> None:
    block = ServingBlock()
    for T in (64, 1):
        residual = torch.randn(T, block.H, device="cuda")
        _, normed = fb.moe_ffn_norm_residual(residual, w_pre=block.pre_w)
        adapters = torch.randint(-1, block.ADAPTERS, (T,), device="cuda", dtype=torch.int32)
        block(residual, normed, adapters)
        torch.cuda.synchronize()
        print(f"T={T}: residual rms {residual.square().mean().sqrt().item():.4f}, experts of token 0 "
              f"{block.kept[T]['ids'][0].tolist()}, device status {block.kept[T]['layer'].status()}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(residual, normed, adapters)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"one decode token, replayed: {start.elapsed_time(end) * 10:.1f} us a block")


if __name__ == "__main__":
    main()
