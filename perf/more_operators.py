"""Workloads of the attention half of a block, next to the expert layer: products with 4-bit weights for few tokens, the
append of keys and values to a paged cache with the position rotation on the way, and attention over that cache for
single tokens and for trees of drafted tokens.

``own`` chooses between the plain form (elementary torch operations, 32 bits; angles of positions in 64) and the
framework's calls.  ``exact`` is the definition in 64 bits.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # product: one decode token, the query, key and value rows of one block, 32 query and 4 key heads of 128
        {"name": "project_decode", "op": "project", "T": 1, "K": 2048, "N": 5120, "group": 32, "x": "bf16", "y": "bf16",
         "bias": False, "pad": 0},
        # product: eight requests' tokens back to the hidden size, groups of 128, into an fp32 residual stream's type
        {"name": "project_out", "op": "project", "T": 8, "K": 4096, "N": 2048, "group": 128, "x": "f16", "y": "f32",
         "bias": False, "pad": 0},
        # product: a vocabulary of an odd size, four requests' logits
        {"name": "project_head", "op": "project", "T": 4, "K": 2048, "N": 100003, "group": 32, "x": "bf16", "y": "f32",
         "bias": False, "pad": 0},
        # product: drafted tokens of several requests, with a bias, inside wider rows
        {"name": "project_drafts", "op": "project", "T": 61, "K": 2048, "N": 5120, "group": 64, "x": "bf16", "y": "bf16",
         "bias": True, "pad": 8},
        # append: one new token for each of eight requests
        {"name": "append_decode", "op": "append", "T": 8, "Hq": 32, "Hkv": 4, "D": 128, "rot": 128, "inter": False,
         "x": "bf16", "cache": "bf16", "page": 16, "layout": "token", "far": 40000, "drop": 0.0},
        # append: a prompt chunk of 4096 tokens
        {"name": "append_prefill", "op": "append", "T": 4096, "Hq": 32, "Hkv": 4, "D": 128, "rot": 128, "inter": False,
         "x": "bf16", "cache": "bf16", "page": 64, "layout": "token", "far": 40000, "drop": 0.0},
        # append: a ragged padded batch far into long contexts, half of each head rotated in neighbouring pairs,
        # fp32 products, pages that hold their heads one behind the other
        {"name": "append_far", "op": "append", "T": 1531, "Hq": 14, "Hkv": 2, "D": 96, "rot": 48, "inter": True,
         "x": "f32", "cache": "f16", "page": 24, "layout": "head", "far": 1 << 20, "drop": 0.1},
        # attention: one request's next token
        {"name": "attend_one", "op": "attend", "B": 1, "n": 1, "Hq": 32, "Hkv": 4, "D": 128, "len": 2000, "spread": 1.0,
         "tree": False, "cap": 0.0, "cache": "bf16", "out": "bf16", "page": 16, "layout": "token", "rest": 0},
        # attention: the next tokens of 48 requests of very different lengths
        {"name": "attend_batch", "op": "attend", "B": 48, "n": 1, "Hq": 32, "Hkv": 4, "D": 128, "len": 12000,
         "spread": 24.0, "tree": False, "cap": 0.0, "cache": "bf16", "out": "bf16", "page": 64, "layout": "token",
         "rest": 3},
        # attention: one request's next token behind a long context
        {"name": "attend_long", "op": "attend", "B": 1, "n": 1, "Hq": 16, "Hkv": 8, "D": 64, "len": 200003, "spread": 1.0,
         "tree": False, "cap": 0.0, "cache": "f16", "out": "f16", "page": 16, "layout": "head", "rest": 0},
        # attention: a tree of 16 drafted tokens for each of 16 requests
        {"name": "attend_tree", "op": "attend", "B": 16, "n": 16, "Hq": 32, "Hkv": 4, "D": 128, "len": 8192,
         "spread": 4.0, "tree": True, "cap": 0.0, "cache": "bf16", "out": "bf16", "page": 64, "layout": "token",
         "rest": 0},
        # attention: trees of up to 61 drafted tokens, capped scores, an odd head size and pages that end inside a tile
        {"name": "attend_tree_capped", "op": "attend", "B": 5, "n": 61, "Hq": 12, "Hkv": 2, "D": 80, "len": 3001,
         "spread": 10.0, "tree": True, "cap": 30.0, "cache": "f16", "out": "f32", "page": 24, "layout": "head",
         "rest": 5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["project", "append", "attend"])
    if op == "project":
        group = rng.choice([32, 32, 64, 128])
        K = group * _log_int(rng, max(1, 128 // group), 8192 // group)
        N = _log_int(rng, 16, min(100003, 100003 * 2048 // K))
        return {"op": "project", "T": _log_int(rng, 1, 256 if N < 20000 else 16), "K": K, "N": N, "group": group,
                "x": rng.choice(["bf16", "f16"]), "y": rng.choice(["f32", "bf16", "f16"]),
                "bias": rng.random() < 0.3, "pad": rng.choice([0, 0, 8, 24])}
    D = rng.choice([64, 64, 80, 96, 128, 128, 192, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8, 16])
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128, 256])
    layout = rng.choice(["token", "head"])
    if op == "append":
        T = _log_int(rng, 1, max(1, min(8192, 4096 * 40 * 128 // ((Hq + 2 * Hkv) * D))))
        return {"op": "append", "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rng.choice([D, D, D // 2, D // 4 // 2 * 2]),
                "inter": rng.random() < 0.4, "x": rng.choice(["f32", "bf16", "f16"]),
                "cache": rng.choice(["bf16", "f16"]), "page": page, "layout": layout,
                "far": rng.choice([2048, 40000, 1 << 20]), "drop": rng.choice([0.0, 0.0, 0.1])}
    n = rng.choice([1, 1, 1, _log_int(rng, 2, 64), _log_int(rng, 2, 64)])
    B = _log_int(rng, 1, 64)
    # at most the bytes of 200,000 cached tokens of 4 heads of 128, and the products of the listed trees
    most = 200000 * 4 * 128 // (Hkv * D * B)
    if n > 1:
        most = min(most, 16 * 32 * 16 * 128 * 3200 // (Hq * n * D * B))
    return {"op": "attend", "B": B, "n": n, "Hq": Hq, "Hkv": Hkv, "D": D,
            "len": _log_int(rng, min(most, n + 1), max(n + 1, min(most, 200003))), "spread": rng.choice([1.0, 4.0, 24.0]),
            "tree": n > 1 and rng.random() < 0.7, "cap": rng.choice([0.0, 0.0, 30.0]),
            "cache": rng.choice(["bf16", "f16"]), "out": rng.choice(["cache", "cache", "f32"]), "page": page,
            "layout": layout, "rest": rng.choice([0, 0, 3])}


def _sequences(case):
    """(cached tokens, drafted tokens) of every sequence: the case's own, from its longest down to a share of it."""
    rng = random.Random(f"{case['B']} {case['len']} {case['n']}")
    out = []
    for b in range(case["B"]):
        n = case["n"] if b == 0 else rng.randint((case["n"] + 1) // 2, case["n"])
        length = case["len"] if b == 0 else int(case["len"] * math.exp(-rng.random() * math.log(case["spread"])))
        out.append((max(length, n), n))
    return out


# --------------------------------------------------------------------------------------------------------------- inputs


def _cache(pages, c, gen):
    """Keys or values [pages, page, Hkv, D], as left by earlier calls; "head": the heads of a page one behind the
    other."""
    shape = (pages, c["Hkv"], c["page"], c["D"]) if c["layout"] == "head" else (pages, c["page"], c["Hkv"], c["D"])
    t = torch.randn(shape, generator=gen, device="cuda", dtype=DTYPES[c["cache"]])
    return t.transpose(1, 2) if c["layout"] == "head" else t


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 29)
    c = dict(case)
    if c.get("out") == "cache":
        c["out"] = c["cache"]
    s = {"case": c}
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    host = random.Random(seed)
    if c["op"] == "project":
        T, K, N, g = c["T"], c["K"], c["N"], c["group"]
        s["x"] = randn(T, K + c["pad"]).to(DTYPES[c["x"]])[:, :K]
        # codes of normally distributed weights with a largest one of about 2.5 spreads a group, scales about 0.02 / 2.8
        w = torch.empty((N, K // 2 + 2 * (K // g)), dtype=torch.uint8, device="cuda")
        lo = torch.randn((N, K // 2), generator=gen, device="cuda", dtype=torch.bfloat16)
        hi = torch.randn((N, K // 2), generator=gen, device="cuda", dtype=torch.bfloat16)
        code = lambda t: t.mul_(2.8).add_(8.0).round_().clamp_(0, 15).to(torch.uint8)  # noqa: E731
        w[:, :K // 2] = code(lo) | (code(hi) << 4)
        scale = torch.rand((N, K // g), generator=gen, device="cuda").mul_(0.004).add_(0.005).to(torch.float16)
        w[:, K // 2:] = scale.view(torch.uint8)
        # rows start at multiples of 16 bytes
        row = (w.shape[1] + 15) // 16 * 16
        s["w"] = torch.nn.functional.pad(w, (0, row - w.shape[1]))
        s["bias"] = randn(N) * 0.1 if c["bias"] else None
        s["y"] = torch.empty((T, N), dtype=DTYPES[c["y"]], device="cuda")
        return s
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    if c["op"] == "append":
        T = c["T"]
        # one row of the projection holds a token's queries, keys and values
        rows = randn(T, (Hq + 2 * Hkv) * D).to(DTYPES[c["x"]])
        heads = rows.view(T, Hq + 2 * Hkv, D)
        s["q"], s["k"], s["v"] = heads[:, :Hq], heads[:, Hq:Hq + Hkv], heads[:, Hq + Hkv:]
        pages = (T + page - 1) // page + 3
        s["k_cache"], s["v_cache"] = _cache(pages, c, gen), _cache(pages, c, gen)
        # tokens of one request lie in pages of any order; some rows are padding
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(T, device="cuda")
        slots = order[at // page] * page + at % page
        if c["drop"]:
            slots = torch.where(torch.rand(T, generator=gen, device="cuda") < c["drop"], torch.full_like(slots, -1), slots)
        s["slots"] = slots.to(torch.int32)
        s["positions"] = (at + host.randint(0, max(0, c["far"] - T))).to(torch.int32)
        i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = torch.pow(1e6 if c["far"] > 100000 else 1e4, -2 * i / max(1, c["rot"])).float()
        s["q_out"] = torch.zeros((T, Hq, D), dtype=DTYPES[c["cache"]], device="cuda")
        return s
    seqs = _sequences(c)
    T = sum(n for _, n in seqs)
    need = [(length + page - 1) // page for length, _ in seqs]
    pages = sum(need) + 2
    s["q"] = randn(T + c["rest"], Hq, D).to(DTYPES[c["cache"]])
    s["k_cache"], s["v_cache"] = _cache(pages, c, gen), _cache(pages, c, gen)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    s["page_table"] = torch.zeros((c["B"], max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        s["page_table"][b, :m] = order[at:at + m]
        at += m
    s["seqs"] = seqs
    s["lens"] = torch.tensor([length for length, _ in seqs], dtype=torch.int32, device="cuda")
    s["q_start"] = torch.tensor(np.cumsum([0] + [n for _, n in seqs]), dtype=torch.int32, device="cuda")
    s["mask"] = None
    if c["tree"]:
        words = (c["n"] + 31) // 32
        bits = np.zeros((T + c["rest"], words), np.uint32)
        t = 0
        for _, n in seqs:
            # every drafted token continues one of the last few before it
            for j in range(n):
                if j:
                    bits[t + j] = bits[t + host.randint(max(0, j - 6), j - 1)]
                bits[t + j, j // 32] |= np.uint32(1 << j % 32)
            t += n
        s["mask"] = torch.from_numpy(bits.view(np.int32)).cuda()
    s["out"] = torch.zeros((T + c["rest"], Hq, D), dtype=DTYPES[c["out"]], device="cuda")
    if own:
        import fusion_backend_gb300 as fb

        s["ws"] = torch.empty(fb.moe_ffn_attend_workspace(T + c["rest"], c["B"], Hq, Hkv, D), dtype=torch.uint8,
                              device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------------------ run


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import fusion_backend_gb300 as fb

    c = s["case"]
    if c["op"] == "project":
        return fb.moe_ffn_project(s["x"], s["w"], group=c["group"], bias=s["bias"], out=s["y"])
    if c["op"] == "append":
        q = fb.moe_ffn_append_kv(s["k"], s["v"], s["positions"], s["slots"], s["inv_freq"], s["k_cache"], s["v_cache"],
                                 q=s["q"], q_out=s["q_out"], interleaved=c["inter"])
        return q, s["k_cache"], s["v_cache"]
    return fb.moe_ffn_attend(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"], s["q_start"],
                             mask=s["mask"], softcap=c["cap"], out=s["out"], workspace=s.get("ws"))


def _run_plain(s):
    return {"project": _plain_project, "append": _plain_append, "attend": _plain_attend}[s["case"]["op"]](s)


def _plain_project(s):
    c = s["case"]
    K, g = c["K"], c["group"]
    codes = s["w"][:, :K // 2]
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    d = s["w"][:, K // 2:K // 2 + 2 * (K // g)].contiguous().view(torch.float16).float()
    w = (q.unflatten(-1, (K // g, g)) * d.unsqueeze(-1)).flatten(-2)
    y = torch.matmul(s["x"].float(), w.T)
    return (y if s["bias"] is None else y + s["bias"]).to(s["y"].dtype)


def _rotate(x, cos, sin, rot, inter):
    """Rotated first `rot` elements of every head of x [T, H, D] by the angles of [T, 1, rot / 2]."""
    x = x.float()
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    rot, page = c["rot"], c["page"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()  # 64 bits: angles of far positions
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    on = s["slots"] >= 0
    q = _rotate(s["q"], cos, sin, rot, c["inter"]).to(s["q_out"].dtype)
    s["q_out"].copy_(torch.where(on[:, None, None], q, s["q_out"]))
    k = _rotate(s["k"], cos, sin, rot, c["inter"]).to(s["k_cache"].dtype)
    # the padding goes to a page of its own behind the cache, which is dropped
    spare = s["k_cache"].shape[0] * page
    at = torch.where(on, s["slots"], torch.full_like(s["slots"], spare)).long()
    for cache, new in ((s["k_cache"], k), (s["v_cache"], s["v"].to(s["v_cache"].dtype))):
        wide = torch.cat((cache, torch.zeros_like(cache[:1])))
        wide[at // page, at % page] = new
        cache.copy_(wide[:-1])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_attend(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    out = torch.zeros_like(s["out"])
    t = 0
    for b, (length, n) in enumerate(s["seqs"]):
        at = torch.arange(length, device="cuda")
        pg, off = s["page_table"][b].long()[at // page], at % page
        k, v = s["k_cache"][pg, off].float(), s["v_cache"][pg, off].float()  # [length, Hkv, D]
        q = s["q"][t:t + n].float().view(n, Hkv, Hq // Hkv, D)
        sc = torch.matmul(q.permute(1, 2, 0, 3), k.permute(1, 2, 0)[:, None]) / math.sqrt(D)  # [Hkv, G, n, length]
        if c["cap"]:
            sc = c["cap"] * torch.tanh(sc / c["cap"])
        if n > 1:
            i = torch.arange(n, device="cuda")
            if s["mask"] is None:
                seen = i[None] <= i[:, None]
            else:
                seen = (s["mask"][t:t + n][:, i // 32] >> (i % 32)) & 1 == 1
            seen = torch.cat((torch.ones((n, length - n), dtype=torch.bool, device="cuda"), seen), 1)
            sc = torch.where(seen, sc, torch.full_like(sc, -math.inf))
        p = torch.exp(sc - sc.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        o = torch.matmul(p, v.permute(1, 0, 2)[:, None])  # [Hkv, G, n, D]
        out[t:t + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, D).to(out.dtype)
        t += n
    return out


# ----------------------------------------------------------------------------------------------------------------- work


def work(case):
    c = case
    if c["op"] == "project":
        T, K, N = c["T"], c["K"], c["N"]
        return {"bytes": N * (K // 2 + 2 * (K // c["group"])) + T * K * 2 + T * N * SIZE[c["y"]] + (4 * N if c["bias"] else 0),
                "flops": 2 * T * K * N}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "append":
        on = c["T"] * (1 - c["drop"])
        return {"bytes": int(on * (Hq + 2 * Hkv) * D * (SIZE[c["x"]] + SIZE[c["cache"]])) + 8 * c["T"],
                "flops": int(on * (Hq + Hkv) * c["rot"] * 3)}
    seqs = _sequences(c)
    T = sum(n for _, n in seqs)
    out = c["cache"] if c["out"] == "cache" else c["out"]
    return {"bytes": sum(length for length, _ in seqs) * Hkv * D * 4 + T * Hq * D * (2 + SIZE[out]),
            "flops": 4 * D * Hq * sum(length * n for length, n in seqs)}


# ---------------------------------------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"project": _exact_project, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_project(s):
    c = s["case"]
    K, g = c["K"], c["group"]
    x = s["x"].double()
    y = torch.zeros((c["T"], c["N"]), dtype=torch.float64, device="cuda")
    scales = s["w"][:, K // 2:K // 2 + 2 * (K // g)].contiguous().view(torch.float16).double()
    for j in range(K // g):
        # one group of every row: even elements in the low halves of its bytes
        by = s["w"][:, j * g // 2:(j + 1) * g // 2].double()
        high = torch.floor(by / 16)
        part = x[:, j * g:(j + 1) * g:2] @ (by - 16 * high - 8).T + x[:, j * g + 1:(j + 1) * g:2] @ (high - 8).T
        y += part * scales[:, j]
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_append(s):
    c = s["case"]
    T, half, page = c["T"], c["rot"] // 2, c["page"]
    slots = s["slots"].cpu().numpy()
    f = s["inv_freq"].cpu().numpy().astype(np.longdouble)
    angle = s["positions"].cpu().numpy().astype(np.longdouble)[:, None] * f
    turn = np.exp(1j * np.asarray(np.fmod(angle, 2 * np.arccos(np.longdouble(-1))), np.float64))[:, None]

    def turned(x):
        x = x.double().cpu().numpy().copy()
        first = slice(0, 2 * half, 2) if c["inter"] else slice(0, half)
        second = slice(1, 2 * half, 2) if c["inter"] else slice(half, 2 * half)
        z = (x[..., first] + 1j * x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    q, k, v = turned(s["q"]), turned(s["k"]), s["v"].double().cpu().numpy()
    q_out = s["q_out"].double().cpu().numpy()
    kc, vc = s["k_cache"].double().cpu().numpy(), s["v_cache"].double().cpu().numpy()
    for t in range(T):
        if slots[t] >= 0:
            at = divmod(int(slots[t]), page)
            q_out[t], kc[at], vc[at] = q[t], k[t], v[t]
    return tuple(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (q_out, kc, vc))


def _exact_attend(s):
    c = s["case"]
    Hq, Hkv, D, page = c["Hq"], c["Hkv"], c["D"], c["page"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    mask = None if s["mask"] is None else s["mask"].cpu().numpy().view(np.uint32)
    start = 0
    for b, (length, n) in enumerate(s["seqs"]):
        pages = s["page_table"][b, :(length + page - 1) // page].long()
        keys = s["k_cache"].index_select(0, pages).reshape(-1, Hkv, D)[:length]
        vals = s["v_cache"].index_select(0, pages).reshape(-1, Hkv, D)[:length]
        hidden = np.zeros((n, length), bool)
        for j in range(n):
            for i in range(n):
                sees = i <= j if mask is None else bool(mask[start + j, i // 32] >> np.uint32(i % 32) & np.uint32(1))
                hidden[j, length - n + i] = not sees
        hidden = torch.from_numpy(hidden).cuda()
        for h in range(Hkv):
            kh, vh = keys[:, h].double(), vals[:, h].double()
            group = s["q"][start:start + n, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)].double()
            score = torch.einsum("jgd,id->gji", group, kh) * D**-0.5
            if c["cap"]:
                score = c["cap"] * torch.tanh(score / c["cap"])
            score = score.masked_fill(hidden[None], -math.inf)
            weight = torch.softmax(score, -1)
            out[start:start + n, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = torch.einsum("gji,id->jgd", weight, vh)
        start += n
    return out
