"""Workloads of the operators around the expert layer: routing, the experts for a given routing, the norms before and
after a block with its gate and residual scale, and the low-rank adapters of many requests.

``own`` chooses between the plain form (elementary torch operations, 32 bits, 64 where a choice between near values or
an exact integer sum needs them) and the framework's calls.  ``exact`` is the definition in 64 bits.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FLT_MAX = torch.finfo(torch.float32).max


# ---------------------------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # routing: one token of the decode layer's 128 experts, the softmax top-8 that its own router takes
        {"name": "route_decode", "op": "route", "T": 1, "E": 128, "k": 8, "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "group_score": "max", "renorm": True, "scale": 1.0, "dtype": "f32", "pad": 0, "masked": 0.0},
        # routing: a prefill chunk, sigmoid scores with a balance bias and 4 of 8 groups, logits of a bf16 product
        {"name": "route_prefill_groups", "op": "route", "T": 4096, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_score": "top2", "renorm": True, "scale": 2.5, "dtype": "bf16", "pad": 0,
         "masked": 0.0},
        # routing: a long ragged batch, rows inside a wider matrix, some experts masked out
        {"name": "route_long_ragged", "op": "route", "T": 16381, "E": 200, "k": 6, "score": "softmax", "bias": True,
         "groups": 1, "top_groups": 1, "group_score": "max", "renorm": False, "scale": 1.0, "dtype": "f32", "pad": 5,
         "masked": 0.1},
        # experts for a given routing: one token, bf16 weights, the decode layer's sizes, with its gated shared expert
        {"name": "experts_decode_bf16", "op": "experts", "T": 1, "H": 2048, "E": 128, "k": 8, "I": 768, "Is": 512,
         "wfmt": "bf16", "shared": "gated", "dropped": 0.0},
        # experts: four requests' tokens, 4-bit weights, an ungated shared expert, some choices dropped
        {"name": "experts_decode_q4", "op": "experts", "T": 4, "H": 2048, "E": 128, "k": 8, "I": 768, "Is": 512,
         "wfmt": "q4", "shared": "plain", "dropped": 0.1},
        # experts: a batch of 256 tokens on the grouped products
        {"name": "experts_batched_bf16", "op": "experts", "T": 256, "H": 2048, "E": 128, "k": 8, "I": 768, "Is": 512,
         "wfmt": "bf16", "shared": "gated", "dropped": 0.0},
        # norms: one decode token between two blocks
        {"name": "norm_decode", "op": "norm", "T": 1, "H": 2048, "y": "f32", "r": "f32", "n": "bf16", "post": True,
         "gate": "channel", "act": "linear", "alpha": 1.0, "beta": 1.0, "offset": 0.0, "pad": 0},
        # norms: a prefill chunk of the layer's fp32 output into an fp32 residual stream
        {"name": "norm_prefill_f32", "op": "norm", "T": 4096, "H": 2048, "y": "f32", "r": "f32", "n": "bf16",
         "post": True, "gate": "channel", "act": "linear", "alpha": 1.0, "beta": 1.0, "offset": 0.0, "pad": 0},
        # norms: a ragged bf16 batch of an odd width in padded rows, a sigmoid gate per element, a scaled residual
        {"name": "norm_ragged_bf16", "op": "norm", "T": 1537, "H": 2883, "y": "bf16", "r": "bf16", "n": "bf16",
         "post": True, "gate": "full", "act": "sigmoid", "alpha": 0.9, "beta": 0.5, "offset": 1.0, "pad": 13},
        # adapters: eight requests' tokens, each its own adapter of rank 16
        {"name": "adapters_decode", "op": "adapters", "T": 8, "K": 2048, "N": 2048, "R": 16, "n": 64, "w": "bf16",
         "y": "f32", "order": "mixed", "ragged": False, "none": 0.0},
        # adapters: a mixed batch of many requests, ranks from 8 to 64, a fifth of the tokens with none
        {"name": "adapters_mixed", "op": "adapters", "T": 200, "K": 2048, "N": 1536, "R": 64, "n": 48, "w": "bf16",
         "y": "bf16", "order": "mixed", "ragged": True, "none": 0.2},
        # adapters: prompts of several requests in one prefill chunk
        {"name": "adapters_prefill", "op": "adapters", "T": 8192, "K": 2048, "N": 2048, "R": 32, "n": 16, "w": "bf16",
         "y": "f32", "order": "runs", "ragged": False, "none": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "norm", "adapters"])
    if op == "route":
        E = _log_int(rng, 8, 512)
        T = _log_int(rng, 1, min(16381, 16381 * 200 // E))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8, 16) if E % g == 0])
        top_groups = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * top_groups))
        return {"op": "route", "T": T, "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.6, "groups": groups, "top_groups": top_groups,
                "group_score": rng.choice(["max", "top2"]), "renorm": rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["f32", "bf16", "f16"]),
                "pad": rng.choice([0, 0, 1, 8, 24]), "masked": rng.choice([0.0, 0.0, 0.1, 0.6])}
    if op == "experts":
        wfmt = rng.choice(["bf16", "bf16", "q4", "i8"])
        # the grouped products of more than 8 tokens round 4-bit weights to fp16, which the fp32 output would show:
        # the 4-bit and int8 weights are drawn for the decode sizes
        T = _log_int(rng, 1, 256 if wfmt == "bf16" else 8)
        E = rng.choice([8, 16, 40, 64, 128])
        H = rng.choice([256, 512, 1024, 2048])
        I = 128 * rng.randint(1, 6) if T > 8 else rng.randint(16, 768)
        Is = 128 * rng.randint(1, 4) if T > 8 else rng.randint(16, 512)
        return {"op": "experts", "T": T, "H": H, "E": E, "k": rng.randint(1, 8), "I": I, "Is": Is, "wfmt": wfmt,
                "shared": rng.choice(["gated", "plain", "none"]), "dropped": rng.choice([0.0, 0.0, 0.2, 0.7])}
    if op == "norm":
        H = _log_int(rng, 64, 8192)
        T = _log_int(rng, 1, max(1, min(16384, 4096 * 2048 // H // 2)))
        y, r = rng.choice(["f32", "bf16", "f16"]), rng.choice(["f32", "bf16"])
        return {"op": "norm", "T": T, "H": H, "y": y, "r": r, "n": rng.choice(["bf16", "f16", "f32"]),
                "post": rng.random() < 0.7, "gate": rng.choice(["none", "channel", "token", "full"]),
                "act": rng.choice(["linear", "sigmoid"]), "alpha": rng.choice([1.0, 0.9]),
                "beta": rng.choice([1.0, 0.5]), "offset": rng.choice([0.0, 1.0]), "pad": rng.choice([0, 0, 8, 3])}
    R = rng.choice([4, 8, 16, 24, 32, 64, 128])
    K = 8 * _log_int(rng, 16, 512)
    N = _log_int(rng, 96, 4096)
    T = _log_int(rng, 1, max(1, min(8192, 8192 * 2048 * 32 // (max(K, N) * max(R, 32)))))
    order = rng.choice(["mixed", "runs"])
    # tokens of many adapters in no order are a decode batch; long inputs are prompts, in runs
    if T > 512:
        order = "runs"
    return {"op": "adapters", "T": T, "K": K, "N": N, "R": R, "n": rng.choice([1, 3, 16, 64]),
            "w": rng.choice(["bf16", "f16"]), "y": rng.choice(["f32", "bf16"]), "order": order,
            "ragged": rng.random() < 0.5, "none": rng.choice([0.0, 0.3])}


# --------------------------------------------------------------------------------------------------------------- inputs


def _rows(T, W, pad, dtype, gen, scale=1.0):
    """[T, W] values inside rows of W + pad."""
    full = torch.randn((T, W + pad), generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)
    return full[:, :W]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)
    s = {"case": dict(case)}
    op = case["op"]
    rand = lambda *shape: torch.rand(shape, generator=gen, device="cuda")  # noqa: E731
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    if op == "route":
        T, E = case["T"], case["E"]
        # logits of a trained router: some experts liked more than others, a spread of about two
        full = randn(T, E + case["pad"]) * 1.5 + randn(E + case["pad"]) * 0.7
        logits = full.to(DTYPES[case["dtype"]])
        if case["masked"]:
            logits[rand(T, E + case["pad"]) < case["masked"]] = -math.inf
        s["logits"] = logits[:, :E]
        s["bias"] = randn(E) * 0.05 if case["bias"] else None
        s["ids"] = torch.empty((T, case["k"]), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((T, case["k"]), dtype=torch.float32, device="cuda")
    elif op == "experts":
        T, H, E, k, I, Is = (case[n] for n in ("T", "H", "E", "k", "I", "Is"))
        s["x"] = randn(T, H).to(torch.bfloat16)
        scores = randn(T, E) + randn(E) * 0.8
        top = torch.topk(scores, k, dim=1)
        ids = top.indices.to(torch.int32)
        if case["dropped"]:
            ids[rand(T, k) < case["dropped"]] = -1
        s["ids"], s["w"] = ids, torch.softmax(top.values, 1)
        s["expert_w"] = _weights(case["wfmt"], E * 3 * I, H, gen)
        s["shexp_w"] = None if case["shared"] == "none" else _weights(case["wfmt"], 3 * Is, H, gen)
        s["gate_w"] = (randn(H) * 0.02).to(torch.bfloat16) if case["shared"] == "gated" else None
        s["out"] = torch.empty((T, H), dtype=torch.float32, device="cuda")
        if own:
            _layer(s)
    elif op == "norm":
        T, H, pad = case["T"], case["H"], case["pad"]
        s["y"] = _rows(T, H, pad, DTYPES[case["y"]], gen, 0.3)
        s["r"] = _rows(T, H, pad, DTYPES[case["r"]], gen, 2.0)
        base = 0.0 if case["offset"] else 1.0
        s["w_post"] = randn(H) * 0.1 + base if case["post"] else None
        s["w_pre"] = (randn(H) * 0.1 + base).to(torch.bfloat16)
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
        gate = None if shape is None else randn(*shape)
        s["gate"] = gate if gate is None or case["gate"] == "channel" else gate.to(DTYPES[case["y"]])
        s["r_out"] = torch.empty((T, H), dtype=DTYPES[case["r"]], device="cuda")
        s["n_out"] = torch.empty((T, H), dtype=DTYPES[case["n"]], device="cuda")
    else:
        T, K, N, R, n = (case[m] for m in ("T", "K", "N", "R", "n"))
        dt = DTYPES[case["w"]]
        s["x"] = randn(T, K).to(dt)
        s["y"] = randn(T, N).to(DTYPES[case["y"]])
        s["a"] = (randn(n, R, K) / math.sqrt(K)).to(dt)
        s["b"] = (randn(n, N, R) * 0.1).to(dt)
        ids = torch.randint(0, n, (T,), generator=gen, device="cuda")
        if case["order"] == "runs":
            # prompts of different requests one behind the other, each the same adapter throughout
            cuts = torch.sort(torch.randint(0, T + 1, (7,), generator=gen, device="cuda")).values
            run = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
            ids = torch.randint(0, n, (8,), generator=gen, device="cuda")[run]
        if case["none"]:
            ids = torch.where(rand(T) < case["none"], torch.full_like(ids, -1), ids)
        s["ids"] = ids.to(torch.int32)
        ranks = torch.randint(max(1, R // 8), R + 1, (n,), generator=gen, device="cuda").to(torch.int32)
        s["ranks"] = ranks if case["ragged"] else None
        s["scales"] = rand(n) + 0.5
        s["out"] = torch.empty_like(s["y"])
        if own:
            import fusion_backend_gb300 as fb

            s["ws"] = torch.empty(fb.moe_ffn_adapters_workspace(T, K, N, R), dtype=torch.uint8, device="cuda")
    return s


def _weights(wfmt, rows, H, gen):
    """Stored rows of H weights with a spread of about 0.02."""
    if wfmt == "bf16":
        return torch.randn((rows, H), generator=gen, device="cuda", dtype=torch.bfloat16).mul_(0.02)
    if wfmt == "q4":
        w = torch.randint(0, 256, (rows, H // 2 + H // 16), generator=gen, device="cuda", dtype=torch.uint8)
        scale = torch.rand((rows, H // 32), generator=gen, device="cuda").mul_(0.003).add_(0.003).to(torch.float16)
        w[:, H // 2:] = scale.view(torch.uint8)
        return w
    w = torch.zeros((rows, H + 16), dtype=torch.uint8, device="cuda")
    q = torch.randn((rows, H), generator=gen, device="cuda").mul_(40).round_().clamp_(-127, 127).to(torch.int8)
    w[:, :H] = q.view(torch.uint8)
    scale = torch.rand((rows, 1), generator=gen, device="cuda").mul_(3e-4).add_(3e-4)
    w[:, H:H + 4] = scale.view(torch.uint8)
    return w


def _layer(s):
    """The plan and workspace that a server keeps for these shapes."""
    if "layer" not in s:
        import fusion_backend_gb300 as fb

        c = s["case"]
        shapes = fb.Shapes(c["T"], c["H"], c["E"], c["k"], c["I"], c["Is"])
        s["layer"] = fb.MoeFFN(shapes, fb.ACT_BF16, {"bf16": fb.W_BF16, "q4": fb.W_Q4B32, "i8": fb.W_I8}[c["wfmt"]])
    return s["layer"]


# ------------------------------------------------------------------------------------------------------------------ run


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import fusion_backend_gb300 as fb

    c = s["case"]
    if c["op"] == "route":
        return fb.moe_ffn_route(s["logits"], c["k"], bias=s["bias"],
                                score=fb.SCORE_SIGMOID if c["score"] == "sigmoid" else fb.SCORE_SOFTMAX,
                                groups=c["groups"], top_groups=c["top_groups"],
                                group_score=fb.GROUP_TOP2 if c["group_score"] == "top2" else fb.GROUP_MAX,
                                renorm=c["renorm"], scale=c["scale"], ids=s["ids"], weights=s["w"])
    if c["op"] == "experts":
        return _layer(s).routed(s["x"], s["ids"], s["w"], s["expert_w"], s["shexp_w"], s["gate_w"], out=s["out"])
    if c["op"] == "norm":
        return fb.moe_ffn_norm_residual(s["r"], s["y"], post_norm=c["post"], w_post=s["w_post"], gate=s["gate"],
                                        gate_act=fb.GATE_SIGMOID if c["act"] == "sigmoid" else fb.GATE_LINEAR,
                                        alpha=c["alpha"], beta=c["beta"], w_pre=s["w_pre"], w_offset=c["offset"],
                                        eps=1e-6, res_out=s["r_out"], normed=s["n_out"])
    return fb.moe_ffn_add_adapters(s["y"], s["x"], s["ids"], s["a"], s["b"], ranks=s["ranks"], scales=s["scales"],
                                   out=s["out"], workspace=s.get("ws"))


def _run_plain(s):
    return {"route": _plain_route, "experts": _plain_experts, "norm": _plain_norm,
            "adapters": _plain_adapters}[s["case"]["op"]](s)


def _sorted_desc(key, second):
    """Indices by key, then second (both descending), then the lower index."""
    o1 = torch.sort(second, dim=1, descending=True, stable=True).indices
    o2 = torch.sort(torch.gather(key, 1, o1), dim=1, descending=True, stable=True).indices
    return torch.gather(o1, 1, o2)


def _plain_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = s["logits"].double().clamp(max=FLT_MAX)  # 64 bits: the choice between near scores
    dead = torch.isnan(l) | (l == -math.inf)
    l = torch.where(dead, torch.full_like(l, -math.inf), l)
    if c["score"] == "softmax":
        m = l.amax(1, keepdim=True)
        z = torch.exp(l - torch.where(m == -math.inf, torch.zeros_like(m), m))
        total = z.sum(1, keepdim=True)
        sc = z / torch.where(total == 0, torch.ones_like(total), total)
    else:
        sc = 1 / (1 + torch.exp(-l))
    key = sc if s["bias"] is None else sc + s["bias"].double()
    ninf = torch.full_like(key, -math.inf)
    key = torch.where(dead, ninf, key)
    if G > 1:
        by = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values
        val = by[:, :, 0]
        if c["group_score"] == "top2" and E // G > 1:
            val = val + torch.where(by[:, :, 1] == -math.inf, torch.zeros_like(val), by[:, :, 1])
        keep = torch.sort(val, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, keep, True)
        key = torch.where(kept.repeat_interleave(E // G, 1), key, ninf)
    ids = _sorted_desc(key, l)[:, :k]
    have = torch.gather(key, 1, ids) != -math.inf
    w = torch.where(have, torch.gather(sc, 1, ids), torch.zeros((), dtype=sc.dtype, device=sc.device))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return torch.where(have, ids, torch.full_like(ids, -1)).to(torch.int32), (w * c["scale"]).float()


def _decode_rows(w, wfmt, H):
    """Stored rows as 32-bit weights."""
    if wfmt == "bf16":
        return w.float()
    if wfmt == "q4":
        codes = w[..., :H // 2]
        q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
        d = w[..., H // 2:].contiguous().view(torch.float16).float()
        return (q.unflatten(-1, (H // 32, 32)) * d.unsqueeze(-1)).flatten(-2)
    return w[..., :H].view(torch.int8).float() * w[..., H:H + 4].contiguous().view(torch.float32)


def _i8_codes(x):
    """The per-token int8 activation: scale max|x| / 127 in 32 bits, codes rounded half away from zero."""
    xs = x.abs().amax(-1, keepdim=True) / 127
    r = x / torch.where(xs == 0, torch.ones_like(xs), xs)
    q = torch.sign(r) * torch.floor(r.abs().double() + 0.5).float()
    return q.clamp(-127, 127), xs


def _ffn(x, w, wfmt, H):
    """FFN of x [..., m, H] by stored blocks w [..., 3, I, row]."""
    if wfmt == "i8":
        q, xs = _i8_codes(x)
        wq = w[..., :H].view(torch.int8)
        ws = w[..., H:H + 4].contiguous().view(torch.float32)[..., 0]
        dot = lambda i: torch.matmul(q.double(), wq[..., i, :, :].double().mT).float()  # noqa: E731  exact integers
        g = dot(0) * xs * ws[..., 0, None, :]
        u = dot(1) * xs * ws[..., 1, None, :]
        down = _decode_rows(w[..., 2, :, :], wfmt, H)
    else:
        g = torch.matmul(x, _decode_rows(w[..., 0, :, :], wfmt, H).mT)
        u = torch.matmul(x, _decode_rows(w[..., 1, :, :], wfmt, H).mT)
        down = _decode_rows(w[..., 2, :, :], wfmt, H)
    return torch.matmul(g / (1 + torch.exp(-g)) * u, down)


def _plain_experts(s):
    c = s["case"]
    T, H, E, k, I, Is, wfmt = (c[n] for n in ("T", "H", "E", "k", "I", "Is", "wfmt"))
    x = s["x"].float()
    ew = s["expert_w"].view(E, 3, I, -1)
    ok = (s["ids"] >= 0) & (s["ids"] < E)
    ids = torch.where(ok, s["ids"], torch.zeros_like(s["ids"])).long()
    w = torch.where(ok, s["w"], torch.zeros_like(s["w"]))
    out = torch.zeros((T, H), dtype=torch.float32, device="cuda")
    if T <= 8:
        for t in range(T):
            y = _ffn(x[t][None, None], ew[ids[t]], wfmt, H)
            out[t] = (w[t][:, None] * y[:, 0]).sum(0)
    else:
        dense = torch.zeros((T, E), dtype=torch.float32, device="cuda").scatter_add_(1, ids, w)
        for e in range(E):
            out += dense[:, e:e + 1] * _ffn(x, ew[e], wfmt, H)
    if s["shexp_w"] is not None:
        y = _ffn(x, s["shexp_w"].view(3, Is, -1), wfmt, H)
        if s["gate_w"] is not None:
            y = y / (1 + torch.exp(-(x * s["gate_w"].float()).sum(1, keepdim=True)))
        out = out + y
    return out


def _plain_norm(s):
    c = s["case"]
    rms = lambda v, w: v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * (c["offset"] + w.float())  # noqa: E731
    z = s["y"].float()
    if c["post"]:
        z = rms(z, s["w_post"])
    if s["gate"] is not None:
        g = s["gate"].float()
        z = z * (1 / (1 + torch.exp(-g)) if c["act"] == "sigmoid" else g)
    r = c["alpha"] * s["r"].float() + c["beta"] * z
    return r.to(s["r_out"].dtype), rms(r, s["w_pre"]).to(s["n_out"].dtype)


def _plain_adapters(s):
    c = s["case"]
    x, y = s["x"].float(), s["y"].float()
    for i in range(c["n"]):
        a, b = s["a"][i].float(), s["b"][i].float()
        on = (s["ids"] == i)[:, None]
        v = torch.matmul(x, a.mT)
        if s["ranks"] is not None:
            v = v * (torch.arange(c["R"], device="cuda") < s["ranks"][i])
        y = torch.where(on, y + s["scales"][i] * torch.matmul(v, b.mT), y)
    return y.to(s["y"].dtype)


# ----------------------------------------------------------------------------------------------------------------- work


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * size[c["dtype"]] + (4 * E if c["bias"] else 0) + 8 * T * k, "flops": 6 * T * E}
    if c["op"] == "experts":
        T, H, E, k, I = (c[n] for n in ("T", "H", "E", "k", "I"))
        Is = 0 if c["shared"] == "none" else c["Is"]
        row = {"bf16": 2 * H, "q4": H // 2 + H // 16, "i8": H + 4}[c["wfmt"]]
        slots = T * k * (1 - c["dropped"])
        distinct = E * (1 - (1 - 1 / E) ** slots) if T > 1 else slots
        return {"bytes": int((distinct * 3 * I + 3 * Is) * row + T * H * 6 + 8 * T * k),
                "flops": int(6 * H * (slots * I + T * Is))}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        gate = {"none": 0, "channel": 4 * H, "token": T * size[c["y"]], "full": T * H * size[c["y"]]}[c["gate"]]
        return {"bytes": T * H * (size[c["y"]] + 2 * size[c["r"]] + size[c["n"]]) + gate + 6 * H, "flops": 12 * T * H}
    T, K, N, R, n = (c[m] for m in ("T", "K", "N", "R", "n"))
    on = T * (1 - c["none"])
    rank = R * 0.56 if c["ragged"] else R
    used = min(n, 8, on) if c["order"] == "runs" else n * (1 - (1 - 1 / n) ** on)
    return {"bytes": int(on * K * 2 + 2 * T * N * size[c["y"]] + used * rank * (K + N) * 2),
            "flops": int(2 * on * rank * (K + N))}


# ---------------------------------------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "norm": _exact_norm,
            "adapters": _exact_adapters}[case["op"]](s)


def _exact_route(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = np.minimum(s["logits"].double().cpu().numpy(), FLT_MAX)
    l[np.isnan(l)] = -np.inf
    live = l > -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if c["score"] == "softmax":
            top = l.max(1, keepdims=True)
            z = np.where(live, np.exp(l - np.where(np.isfinite(top), top, 0.0)), 0.0)
            sc = z / np.maximum(z.sum(1, keepdims=True), 1e-300)
        else:
            sc = np.where(live, 1.0 / (1.0 + np.exp(-l)), 0.0)
    key = sc.copy() if s["bias"] is None else sc + s["bias"].double().cpu().numpy()
    key[~live] = -np.inf
    if G > 1:
        blocks = np.sort(key.reshape(T, G, E // G), axis=2)
        val = blocks[:, :, -1].copy()
        if c["group_score"] == "top2" and E // G > 1:
            second = blocks[:, :, -2]
            val += np.where(np.isfinite(second), second, 0.0)
        rank = np.argsort(-val, axis=1, kind="stable")
        out = np.ones((T, G), bool)
        np.put_along_axis(out, rank[:, :c["top_groups"]], False, axis=1)
        key[np.repeat(out, E // G, axis=1)] = -np.inf
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -l, -key), axis=1)[:, :k]
    got = np.take_along_axis(key, order, 1) > -np.inf
    w = np.where(got, np.take_along_axis(sc, order, 1), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdims=True)
        w = w / np.where(total > 0, total, 1.0)
    ids = np.where(got, order, -1).astype(np.int32)
    return torch.from_numpy(ids).cuda(), torch.from_numpy(w * c["scale"]).cuda()


def _exact_block(x, w, wfmt, H):
    """One SwiGLU block [3, I, row] on x [m, H], in 64 bits."""
    if wfmt == "bf16":
        m = w.double()
    elif wfmt == "q4":
        by = w[..., :H // 2].to(torch.int32)
        q = torch.empty((*w.shape[:-1], H), dtype=torch.float64, device=w.device)
        q[..., 0::2] = (by % 16 - 8).double()
        q[..., 1::2] = (by // 16 - 8).double()
        m = q * w[..., H // 2:].contiguous().view(torch.float16).double().repeat_interleave(32, -1)
    else:
        q, xs = _i8_codes(x.float())
        x = q.double() * xs.double()
        m = w[..., :H].view(torch.int8).double() * w[..., H:H + 4].contiguous().view(torch.float32).double()
    g, u = x @ m[0].T, x @ m[1].T
    return (g * torch.sigmoid(g) * u) @ m[2]


def _exact_experts(s):
    c = s["case"]
    E, I, Is, H, wfmt = (c[n] for n in ("E", "I", "Is", "H", "wfmt"))
    x, ids, w = s["x"].double(), s["ids"], s["w"].double()
    ew = s["expert_w"].view(E, 3, I, -1)
    out = torch.zeros((c["T"], H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            out.index_add_(0, t, w[t, j][:, None] * _exact_block(x[t], ew[e], wfmt, H))
    if s["shexp_w"] is not None:
        y = _exact_block(x, s["shexp_w"].view(3, Is, -1), wfmt, H)
        if s["gate_w"] is not None:
            y = y * torch.sigmoid(x @ s["gate_w"].double())[:, None]
        out += y
    return out


def _exact_norm(s):
    c = s["case"]
    H = c["H"]
    r, z = s["r"].double() * c["alpha"], s["y"].double()
    if c["post"]:
        z = z / torch.sqrt((z ** 2).sum(1, keepdim=True) / H + 1e-6) * (s["w_post"].double() + c["offset"])
    if s["gate"] is not None:
        g = s["gate"].double()
        z = z * (torch.sigmoid(g) if c["act"] == "sigmoid" else g)
    r = r + z * c["beta"]
    return r, r / torch.sqrt((r ** 2).sum(1, keepdim=True) / H + 1e-6) * (s["w_pre"].double() + c["offset"])


def _exact_adapters(s):
    c = s["case"]
    out = s["y"].double().clone()
    for i in torch.unique(s["ids"]).tolist():
        if i < 0:
            continue
        t = torch.nonzero(s["ids"] == i)[:, 0]
        r = c["R"] if s["ranks"] is None else int(s["ranks"][i])
        v = s["x"][t].double() @ s["a"][i, :r].double().T
        out[t] += s["scales"][i].double() * (v @ s["b"][i, :, :r].double().T)
    return out
