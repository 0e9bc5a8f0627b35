"""The attention half of a block as a server runs it, in front of the expert half of ``serving_block.py``:

    q k v  = n W_qkv^T                                     4-bit weights
    cache += k, v at the tokens' slots, k and q rotated by position
    o_t    = attention of q_t over its sequence's cached tokens (single tokens, or trees of drafted ones)
    a      = o W_o^T                                       4-bit weights
    r, n   = r + a and its norm, for the experts

Run it on a GB300 with ``python examples/attention_block.py``: a prompt of 40 tokens, then eight sequences' next tokens
replayed from a CUDA graph, then a tree of drafted tokens for each.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fusion_backend_gb300 as fb  # noqa: E402


def quantised(w: torch.Tensor, group: int = 32) -> torch.Tensor:
    """Rows of 4-bit codes and fp16 scales (uint8 [N, K/2 + 2 K/group]) for w [N, K]."""
    g = w.float().unflatten(1, (-1, group))
    d = (g.abs().amax(2) / 7).half()
    q = (g / d.float().clamp(min=1e-8).unsqueeze(2)).round().clamp(-8, 7).add(8).to(torch.uint8).flatten(1)
    return torch.cat((q[:, 0::2] | q[:, 1::2] << 4, d.view(torch.uint8)), 1).contiguous()


class Sequences:
    """Pages of a cache that sequences of tokens take one after the other."""

    def __init__(self, block: "AttentionBlock", count: int):
        self.page, self.free = block.PAGE, list(range(block.PAGES))[::-1]
        self.table = torch.zeros((count, block.PAGES // count), dtype=torch.int32)
        self.lens = [0] * count

    def append(self, new: list[int]):
        """Slots of `new[b]` more tokens of every sequence b, in their order, and what attention takes: the slots, the
        page table, the lengths and the rows' starts, on the GPU."""
        slots, starts = [], [0]
        for b, n in enumerate(new):
            for i in range(self.lens[b], self.lens[b] + n):
                if i % self.page == 0:
                    self.table[b, i // self.page] = self.free.pop()
                slots.append(int(self.table[b, i // self.page]) * self.page + i % self.page)
            self.lens[b] += n
            starts.append(starts[-1] + n)
        to = lambda v: torch.as_tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        return to(slots), to(self.table), to(self.lens), to(starts)


class AttentionBlock:
    H, Q_HEADS, KV_HEADS, D, PAGE, PAGES = 2048, 32, 4, 128, 16, 512

    def __init__(self, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = (self.Q_HEADS + 2 * self.KV_HEADS) * self.D
        self.qkv_w = quantised(torch.randn(rows, self.H, generator=g, device="cuda") * 0.02)
        self.out_w = quantised(torch.randn(self.H, self.Q_HEADS * self.D, generator=g, device="cuda") * 0.02)
        self.pre_w = (torch.randn(self.H, generator=g, device="cuda") * 0.1 + 1).bfloat16()
        self.inv_freq = torch.pow(1e4, -torch.arange(0, self.D, 2, device="cuda") / self.D).float()
        self.k_cache, self.v_cache = (torch.zeros(self.PAGES, self.PAGE, self.KV_HEADS, self.D, device="cuda",
                                                  dtype=torch.bfloat16) for _ in range(2))
        self.kept = {}

    def _keep(self, T: int, B: int):
        if (T, B) not in self.kept:
            new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
            heads, ws = self.Q_HEADS * self.D, fb.moe_ffn_attend_workspace(T, B, self.Q_HEADS, self.KV_HEADS, self.D)
            self.kept[T, B] = dict(qkv=new(T, self.qkv_w.shape[0]), o=new(T, heads), a=new(T, self.H, dtype=torch.float32),
                                   ws=new(ws, dtype=torch.uint8))
        return self.kept[T, B]

    def __call__(self, residual, normed, positions, slots, table, lens, starts, mask=None):
        """residual fp32 [T, H] and normed bf16 [T, H], both updated in place; the rest as `Sequences.append` gives it,
        mask int32 [T, words]: which of its sequence's new tokens a token sees (None: those up to itself)."""
        T = residual.shape[0]
        k = self._keep(T, lens.shape[0])
        fb.moe_ffn_project(normed, self.qkv_w, out=k["qkv"])
        heads = k["qkv"].view(T, -1, self.D)
        q, key, value = heads.split((self.Q_HEADS, self.KV_HEADS, self.KV_HEADS), 1)
        fb.moe_ffn_append_kv(key, value, positions, slots, self.inv_freq, self.k_cache, self.v_cache, q=q)
        fb.moe_ffn_attend(q, self.k_cache, self.v_cache, table, lens, starts, mask=mask, out=k["o"].view(T, -1, self.D),
                          workspace=k["ws"])
        fb.moe_ffn_project(k["o"], self.out_w, out=k["a"])
        return fb.moe_ffn_norm_residual(residual, k["a"], w_pre=self.pre_w, normed=normed)


def main() -> None:
    block, seqs = AttentionBlock(), None
    seqs = Sequences(block, 8)

    def step(new, positions, mask=None):
        T = sum(new)
        residual = torch.randn(T, block.H, device="cuda")
        _, normed = fb.moe_ffn_norm_residual(residual, w_pre=block.pre_w)
        args = (residual, normed, torch.tensor(positions, dtype=torch.int32, device="cuda"), *seqs.append(new), mask)
        block(*args)
        torch.cuda.synchronize()
        print(f"{T} tokens of {sum(n > 0 for n in new)} sequences: residual rms {residual.square().mean().sqrt().item():.4f}")
        return args

    step([40] * 8, list(range(40)) * 8)
    args = step([1] * 8, [40] * 8)
    # a root and two branches of two tokens, at the positions behind the last token
    sees = [0b1, 0b11, 0b101, 0b1011, 0b10101]
    step([5] * 8, [41, 42, 42, 43, 43] * 8, torch.tensor(sees * 8, dtype=torch.int32, device="cuda")[:, None])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(*args)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(100):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"eight sequences' next tokens, replayed: {start.elapsed_time(end) * 10:.1f} us a half block")


if __name__ == "__main__":
    main()
