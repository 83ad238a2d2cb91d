"""The work of the serving operators around the quantised layers, and their plain forms.

    rms_norm            residual addition + root-mean-square norm, 16-bit and/or E4M3 output with scales
    moe_route_grouped   softmax / sigmoid router with a balancing bias, expert groups, top-k (and the padded sort)
    dense_lora_gemm     low-rank adapters of many requests beside a dense quantised projection
    moe_fp8_codes_gemm  the FP8 layer's gate/up projection on E4M3 rows with a scale each

Every plain form is written in elementary torch operations in float32, the router's scores in float64 (they are
compared with each other); `exact` gives each operator's definition in float64, without the last rounding.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
MIN_SCALE = 2.0 ** -100  # the least row scale of a quantised row (a row of zeros)
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ----------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------
def _norm(rows, n, dtype, residual, quant, out):
    return {"op": "norm", "rows": rows, "n": n, "dtype": dtype, "residual": residual, "quant": quant, "out": out}


def _route(M, E, topk, dtype, scoring, bias, groups, topk_group, group_score, renorm, scale, block):
    return {"op": "route", "M": M, "E": E, "topk": topk, "dtype": dtype, "scoring": scoring, "bias": bias,
            "groups": groups, "topk_group": topk_group, "group_score": group_score, "renorm": renorm, "scale": scale,
            "block": block}


def _lora(M, K, N, rank, adapters, seqs, dtype):
    return {"op": "lora", "M": M, "K": K, "N": N, "rank": rank, "adapters": adapters, "seqs": seqs, "dtype": dtype}


def _fp8(M, E, topk, K, N, block):
    return {"op": "fp8", "M": M, "E": E, "topk": topk, "K": K, "N": N, "block": block}


def listed():
    return [
        # one token of a decode step, into the FP8 layer: 16-bit row for the router, codes for the experts
        dict(_norm(1, 4096, "bf16", True, "row", True), name="norm token"),
        # a decode batch in front of a 16-bit layer of width 7168
        dict(_norm(64, 7168, "f16", True, "none", True), name="norm batch"),
        # an odd width (no 16-byte rows), first norm of a model, a calibrated static scale, codes only
        dict(_norm(333, 1001, "bf16", False, "static", False), name="norm odd width"),
        # a prompt batch into the FP8 layer
        dict(_norm(8192, 5120, "bf16", True, "row", True), name="norm prompts"),
        # one token, 160 experts in 8 groups of which 3 are open, sorted for the decode kernel
        dict(_route(1, 160, 6, "f32", "softmax", False, 8, 3, "max", False, 16.0, 16), name="route token"),
        # a decode batch, 16-bit logits (ties), one group, sigmoid scores with a bias
        dict(_route(61, 96, 4, "bf16", "sigmoid", True, 1, 1, "max", True, 1.0, 16), name="route batch"),
        # a prompt batch: sigmoid, bias, groups scored by their two best experts
        dict(_route(8192, 256, 8, "f32", "sigmoid", True, 8, 4, "top2", True, 2.5, 0), name="route prompts"),
        # a decode batch of requests with an adapter each
        dict(_lora(8, 4096, 4096, 16, 8, 0, "bf16"), name="adapters decode"),
        # a mixed step: a few short prompts, ragged sizes
        dict(_lora(203, 5120, 1544, 24, 6, 7, "f16"), name="adapters ragged"),
        # prompts of several requests through a wide projection
        dict(_lora(4096, 7168, 20480, 64, 8, 11, "bf16"), name="adapters prompts"),
        # gate/up of a decode batch (16-row blocks)
        dict(_fp8(16, 8, 2, 4096, 1792, 16), name="gate/up codes decode"),
        # gate/up of a prompt batch (128-row blocks)
        dict(_fp8(1024, 8, 2, 4096, 1792, 128), name="gate/up codes prompts"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "route", "lora", "fp8"))
    if op == "norm":
        n = _log(rng, 64, 8192)
        if rng.random() < 0.5:
            n = max(64, n // 8 * 8)
        rows = max(1, min(_log(rng, 1, 8192), 8192 * 5120 // n))
        quant = rng.choice(("none", "row", "static"))
        return _norm(rows, n, rng.choice(("bf16", "f16")), rng.random() < 0.7, quant,
                     quant == "none" or rng.random() < 0.5)
    if op == "route":
        groups = rng.choice((1, 1, 2, 3, 4, 8))
        size = max(2, _log(rng, 4, 256) // groups)
        open_ = rng.randint(1, groups)
        topk = rng.randint(1, min(8, open_ * size))
        M = _log(rng, 1, 8192)
        return _route(M, groups * size, topk, rng.choice(("f32", "bf16", "f16")), rng.choice(("softmax", "sigmoid")),
                      rng.random() < 0.5, groups, open_, rng.choice(("max", "top2")), rng.random() < 0.6,
                      rng.choice((1.0, 2.5, 16.0)), rng.choice((0, 16, 64)) if M <= 1024 else 0)
    if op == "lora":
        K, N = 8 * _log(rng, 32, 896), 8 * _log(rng, 32, 2560)
        rank, adapters = 8 * rng.randint(1, 8), _log(rng, 1, 32)
        most = 4096 * (7168 + 20480) * 8 * 64 // ((K + N) * rank * adapters)
        M = max(1, min(_log(rng, 1, 4096), most))
        return _lora(M, K, N, rank, adapters, 0 if M <= 64 else rng.randint(1, 24), rng.choice(("bf16", "f16")))
    E = rng.randint(2, 8)
    K, N = 128 * _log(rng, 4, 32), 16 * _log(rng, 16, 112)
    M = _log(rng, 1, 1024)
    return _fp8(M, E, rng.randint(1, min(4, E)) if M <= 512 else min(2, E), K, N, 16 if M <= 32 else rng.choice((16, 64, 128)))


# ----------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------
def _capacity(T, E, block):
    return -(-(T + min(T, E) * (block - 1)) // block) * block


def _padded_sort(ids, E, block):
    """The (token, slot) pairs sorted by expert, each expert's run padded to whole blocks: pair of every row (the
    number of pairs for a pad), expert of every block (-1 past the last), rows in use."""
    flat = ids.reshape(-1).long()
    T = flat.numel()
    cap = _capacity(T, E, block)
    dev = flat.device
    count = (flat[:, None] == torch.arange(E, device=dev)).sum(0)
    end = torch.cumsum((count + block - 1) // block * block, 0)
    start = end - (count + block - 1) // block * block
    order = torch.sort(flat, stable=True).indices
    rank = torch.arange(T, device=dev) - (torch.cumsum(count, 0) - count)[flat[order]]
    rows = torch.full((cap,), T, dtype=torch.int32, device=dev)
    rows[start[flat[order]] + rank] = order.int()
    at = torch.arange(0, cap, block, device=dev)
    blocks = (at[:, None] >= end).sum(1)
    return rows, torch.where(at < end[-1], blocks, -1).int(), end[-1:].int()


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        dt, rows, n = DTYPES[case["dtype"]], case["rows"], case["n"]
        loud = 1.0 + 20.0 * (torch.rand(n, generator=g, device="cuda") < 0.01)  # a few loud channels, as hidden states have
        s["x"] = (_normal(g, rows, n) * loud).to(dt)
        s["r"] = (_normal(g, rows, n) * loud * 3).to(dt) if case["residual"] else None
        s["w"] = (1 + 0.2 * _normal(g, n)).to(dt)
        s["static"] = 0.04
    elif case["op"] == "route":
        s["logits"] = (1.5 * _normal(g, case["M"], case["E"])).to(DTYPES[case["dtype"]])
        s["b"] = 0.05 * _normal(g, case["E"]) if case["bias"] else None
    elif case["op"] == "lora":
        dt, M, K, N, R, L = DTYPES[case["dtype"]], case["M"], case["K"], case["N"], case["rank"], case["adapters"]
        s["x"] = _normal(g, M, K).to(dt)
        s["a"] = (_normal(g, L, R, K) / math.sqrt(K)).to(dt)
        s["b"] = (_normal(g, L, N, R) * 0.5 / math.sqrt(R)).to(dt)
        s["scales"] = 0.5 + 1.5 * torch.rand(L, generator=g, device="cuda")
        s["y"] = _normal(g, M, N).to(dt)
        # one request a token, or `seqs` prompts in order; about one request in ten has no adapter
        many = case["seqs"] or M
        of = torch.randint(0, L, (many,), generator=g, device="cuda")
        of = torch.where(torch.rand(many, generator=g, device="cuda") < 0.1, -1, of)
        if case["seqs"]:
            cuts = torch.sort(torch.randint(0, M, (many - 1,), generator=g, device="cuda")).values
            of = of[(torch.arange(M, device="cuda")[:, None] >= cuts).sum(1)]
        s["ids"] = of.int()
    else:
        M, E, K, N = case["M"], case["E"], case["K"], case["N"]
        s["codes"] = (_normal(g, M, K) * 100).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
        s["row_scales"] = 0.005 + 0.01 * torch.rand(M, generator=g, device="cuda")
        # gate rows, then up rows, of every expert; one scale a row
        s["w"] = (_normal(g, E, 2 * N, K) * 64).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
        s["ws"] = (0.5 + torch.rand(E, 2 * N, generator=g, device="cuda")) / (64 * math.sqrt(K))
        s["a2"] = 0.01
        ids = torch.argsort(torch.rand(M, E, generator=g, device="cuda"), dim=1)[:, :case["topk"]]
        s["rows"], s["blocks"], s["used"] = _padded_sort(ids, E, case["block"])
        s["h"] = torch.zeros((s["rows"].numel(), N), dtype=torch.uint8, device="cuda")
        # the packed weights that a program lays out once: 16 gate rows, then their 16 up rows, in tiles of 16 rows
        # by 128 channels; a tile is two planes of 64 16-byte pieces (piece = row + 16 * (channel / 32))
        tiles = s["w"].view(E, 2, N // 16, 16, K // 128, 4, 2, 16).permute(0, 2, 1, 4, 6, 5, 3, 7)
        s["w_packed"] = tiles.reshape(-1).contiguous()
        s["ws_packed"] = s["ws"].view(E, 2, N // 16, 16).permute(0, 2, 1, 3).reshape(E, 2 * N).contiguous()
    return s


# ----------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------
def _norm_plain(s):
    t = s["x"].float()
    if s["r"] is not None:
        t = t + s["r"].float()
    y = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * s["w"].float()
    got = {}
    if s["r"] is not None:
        got["residual"] = t.to(s["x"].dtype)
    if s["out"]:
        got["out"] = y.to(s["x"].dtype)
    if s["quant"] == "row":
        scale = torch.clamp(y.abs().amax(-1) / F8_MAX, min=MIN_SCALE)
        got["scales"] = scale
        got["codes"] = (y / scale[:, None]).clamp(-F8_MAX, F8_MAX).to(F8)
    elif s["quant"] == "static":
        got["codes"] = (y / s["static"]).clamp(-F8_MAX, F8_MAX).to(F8)
    return got


def _route_plain(s):
    l, (M, E), k, G = s["logits"].double(), s["logits"].shape, s["topk"], s["groups"]
    if s["scoring"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    biased = score if s["b"] is None else score + s["b"].double()
    order = l if s["b"] is None else biased.float().double()  # without a bias the logits' own order
    if s["groups"] > 1:
        if s["group_score"] == "max":
            best = order.view(M, G, E // G).amax(-1)
        else:
            two = torch.sort(biased.float().view(M, G, E // G), dim=-1, descending=True).values
            best = two[..., 0] + two[..., 1]
        chosen = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :s["topk_group"]]
        open_ = torch.zeros((M, G), dtype=torch.bool, device=l.device).scatter_(1, chosen, True)
        order = torch.where(open_[:, :, None].expand(M, G, E // G).reshape(M, E), order, -math.inf)
    ids = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(score, 1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    got = {"weights": (w * s["scale"]).float(), "ids": ids.int()}
    if s["block"]:
        got["rows"], got["blocks"], got["used"] = _padded_sort(ids, E, s["block"])
    return got


def _lora_plain(s):
    M, (L, R, K), N = s["M"], s["a"].shape, s["N"]
    # every adapter's product, of which each token keeps its own
    t = (s["x"].float() @ s["a"].float().reshape(L * R, K).t()).view(M, L, R)
    mine = s["ids"].long()[:, None] == torch.arange(L, device="cuda")
    t = torch.where(mine[:, :, None], t * s["scales"][:, None], 0.0).reshape(M, L * R)
    s["y"].copy_(s["y"].float() + t @ s["b"].float().permute(0, 2, 1).reshape(L * R, N))
    return {"y": s["y"]}


def _fp8_plain(s):
    M, K, E, N, k = s["M"], s["K"], s["E"], s["N"], s["topk"]
    T = M * k
    x = s["codes"].view(F8).float() * s["row_scales"][:, None]
    w = s["w"].view(F8).float() * s["ws"][:, :, None]
    z = (x @ w.reshape(E * 2 * N, K).t()).view(M, E, 2, N)
    pair = s["rows"].long()
    expert = s["blocks"].long().clamp(min=0).repeat_interleave(s["block"])
    z = z[(pair // k).clamp(max=M - 1), expert]
    h = z[:, 0] / (1 + torch.exp(-z[:, 0])) * z[:, 1]
    h = torch.where((pair < T)[:, None], h / s["a2"], 0.0)
    return {"h": h.clamp(-F8_MAX, F8_MAX).to(F8)}


def run(s):
    if not own:
        return {"norm": _norm_plain, "route": _route_plain, "lora": _lora_plain, "fp8": _fp8_plain}[s["op"]](s)
    import weight_only_quantized_topk_amd as wq
    if s["op"] == "norm":
        q = s["quant"]
        r = wq.rms_norm(s["x"], s["w"], EPS, residual=s["r"], quant=None if q == "none" else q,
                        scale=s["static"] if q == "static" else None, want_out=s["out"])
        got = {}
        if r.residual is not None:
            got["residual"] = r.residual
        if r.out is not None:
            got["out"] = r.out
        if r.codes is not None:
            got["codes"] = r.codes.view(F8)
        if r.scales is not None:
            got["scales"] = r.scales
        return got
    if s["op"] == "route":
        how = {"scoring": s["scoring"], "bias": s["b"], "n_group": s["groups"], "topk_group": s["topk_group"],
               "group_score": s["group_score"], "renormalize": s["renorm"], "routed_scale": s["scale"]}
        if not s["block"]:
            w, ids = wq.moe_route_grouped(s["logits"], s["topk"], **how)
            return {"weights": w, "ids": ids}
        w, ids, rows, blocks, used = wq.moe_route_grouped_align(s["logits"], s["topk"], s["block"], **how)
        return {"weights": w, "ids": ids, "rows": rows, "blocks": blocks, "used": used}
    if s["op"] == "lora":
        return {"y": wq.dense_lora_gemm(s["x"], s["ids"], s["a"], s["b"], s["scales"], s["y"])}
    wq.moe_fp8_codes_gemm(wq.WQ_STAGE_GATE_UP, s["codes"], s["row_scales"], s["M"], s["topk"], s["E"], 2 * s["N"],
                          s["K"], s["w_packed"], s["ws_packed"], s["rows"], s["blocks"], s["used"], s["rows"].numel(),
                          s["block"], s["h"], out_scale=s["a2"])
    return {"h": s["h"].view(F8)}


# ----------------------------------------------------------------------------------------------------------------
# the least work, and the definitions
# ----------------------------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "norm":
        per = 2 + (4 if c["residual"] else 0) + (2 if c["out"] else 0) + (1 if c["quant"] != "none" else 0)
        e = c["rows"] * c["n"]
        return {"bytes": e * per + 2 * c["n"] + (4 * c["rows"] if c["quant"] == "row" else 0), "flops": 6 * e}
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        T = c["M"] * c["topk"]
        cap = _capacity(T, c["E"], c["block"]) if c["block"] else 0
        return {"bytes": c["M"] * c["E"] * size + (4 * c["E"] if c["bias"] else 0) + 8 * T
                + (4 * (cap + cap // c["block"] + 1) if cap else 0), "flops": 8 * c["M"] * c["E"]}
    if c["op"] == "lora":
        M, K, N, R = c["M"], c["K"], c["N"], c["rank"]
        used = min(c["adapters"], c["seqs"] or M)
        return {"bytes": 2 * (M * K + 2 * M * N + used * R * (K + N)) + 4 * M + 4 * used, "flops": 2 * M * R * (K + N)}
    T = c["M"] * c["topk"]
    used = min(c["E"], T)
    return {"bytes": c["M"] * (c["K"] + 4) + used * 2 * c["N"] * (c["K"] + 4) + T * c["N"], "flops": 4 * T * c["N"] * c["K"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        t = s["x"].double() if s["r"] is None else s["x"].double() + s["r"].double()
        norm = torch.linalg.vector_norm(t, dim=1, keepdim=True)
        y = t / torch.sqrt(norm * norm / case["n"] + EPS) * s["w"].double()
        top = torch.maximum(y.max(1).values, -y.min(1).values) / F8_MAX
        scale = torch.where(top > MIN_SCALE, top, MIN_SCALE) if case["quant"] == "row" else torch.full_like(top, s["static"])
        got = {"residual": t if case["residual"] else None, "out": y if case["out"] else None,
               "scales": scale if case["quant"] == "row" else None,
               "codes": torch.clip(y / scale.unsqueeze(1), -F8_MAX, F8_MAX) if case["quant"] != "none" else None}
        return {k: v for k, v in got.items() if v is not None}
    if case["op"] == "route":
        l = s["logits"].double().cpu()
        p = torch.softmax(l, 1) if case["scoring"] == "softmax" else torch.sigmoid(l)
        key = l.clone() if s["b"] is None else (p + s["b"].double().cpu()).float().double()
        G, per = case["groups"], case["E"] // case["groups"]
        if G > 1:
            if case["group_score"] == "max":
                value = torch.stack([key[:, g * per:(g + 1) * per].max(1).values for g in range(G)], 1)
            else:
                c = (p if s["b"] is None else p + s["b"].double().cpu()).float()
                value = torch.stack([torch.topk(c[:, g * per:(g + 1) * per], 2, 1).values.sum(1) for g in range(G)], 1)
            ahead = (value[:, None, :] > value[:, :, None]) | ((value[:, None, :] == value[:, :, None])
                                                              & (torch.arange(G)[None, :] < torch.arange(G)[:, None]))
            shut = ahead.sum(2) >= case["topk_group"]
            key[shut.repeat_interleave(per, 1)] = -math.inf
        ids = torch.empty((case["M"], case["topk"]), dtype=torch.int64)
        for j in range(case["topk"]):  # the first of the largest that are left
            top = key.max(1, keepdim=True).values
            ids[:, j] = (key == top).int().argmax(1)
            key.scatter_(1, ids[:, j:j + 1], -math.inf)
        w = p.gather(1, ids)
        w = w / w.sum(1, keepdim=True) if case["renorm"] else w
        return {"weights": w * case["scale"], "ids": ids.int()}
    if case["op"] == "lora":
        y = s["y"].double()
        for a in range(case["adapters"]):
            m = (s["ids"] == a).nonzero().flatten()
            if m.numel():
                y[m] += s["scales"][a].double() * ((s["x"][m].double() @ s["a"][a].double().t()) @ s["b"][a].double().t())
        return {"y": y}
    M, N, k = case["M"], case["N"], case["topk"]
    h = torch.zeros((s["rows"].numel(), N), dtype=torch.float64, device="cuda")
    for b, e in enumerate(s["blocks"].tolist()):
        at = slice(b * case["block"], (b + 1) * case["block"])
        pair = s["rows"][at].long()
        live = pair < M * k
        if e < 0 or not bool(live.any()):
            continue
        m = pair[live] // k
        x = s["codes"].view(F8)[m].double() * s["row_scales"][m].double()[:, None]
        gate, up = (x @ (s["w"][e].view(F8).double() * s["ws"][e].double()[:, None]).t()).split(N, 1)
        h[at][live] = torch.clip(gate * torch.sigmoid(gate) * up / s["a2"], -F8_MAX, F8_MAX)
    return {"h": h}
