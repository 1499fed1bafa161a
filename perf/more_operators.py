"""Workloads of the 16-bit-activation layer and the routed layer on the packed 4-bit weights.

Three operators on the group-wise packed weights W = s_W Q_W (groups of 128 along the input
channels, codes in [-7, 7]) with activations kept in fp16 or bf16:

* ``linear_a16``  Y = X W^T + (X L1) L2
* ``moe_route``   router scores of each token, its k best experts and their weights
* ``moe``         the whole routed layer: y = sum_j w_j W2_e (silu(G_e x) * (U_e x)) over a token's experts

``run`` computes a case in elementary torch operations (binary32, the router's scores in
binary64, rounded once), or, with ``own`` set, through this repository's library. ``exact``
evaluates the definitions in binary64. Shapes: the layers of ``synth.CONFIGS`` and generic sizes.
"""
import math

import torch

own = False

GROUP = 128
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one token through a small layer: nothing but launch latency
        dict(name="a16_one_token_small", op="linear_a16", b=1, m=512, n=512, r=16, dtype="fp16"),
        # one token of an interactive decode, 70B gate/up projection
        dict(name="a16_one_token_70b", op="linear_a16", b=1, m=8192, n=28672, r=128, dtype="bf16"),
        # a decode batch, 8B attention output projection
        dict(name="a16_decode", op="linear_a16", b=16, m=4096, n=4096, r=32, dtype="fp16"),
        # a ragged decode batch, 8B down projection without a low-rank pair
        dict(name="a16_decode_ragged", op="linear_a16", b=61, m=14336, n=4096, r=0, dtype="bf16"),
        # prompts of an 8B gate/up projection
        dict(name="a16_prefill", op="linear_a16", b=2048, m=4096, n=14336, r=32, dtype="fp16"),
        # a long ragged prompt, 70B gate/up projection
        dict(name="a16_prefill_70b", op="linear_a16", b=4001, m=8192, n=28672, r=128, dtype="bf16"),
        # the router of one token
        dict(name="route_one_token", op="moe_route", b=1, m=2048, experts=64, k=8, score="softmax", bias=False,
             dtype="bf16"),
        # the router of a full decode batch: many experts, sigmoid scores, a selection bias
        dict(name="route_batch", op="moe_route", b=256, m=7168, experts=256, k=8, score="sigmoid", bias=True,
             dtype="bf16"),
        # one token, many narrow experts
        dict(name="moe_one_token", op="moe", b=1, m=2048, f=768, experts=64, k=8, score="softmax", bias=False,
             dtype="bf16"),
        # one token, a few wide experts
        dict(name="moe_one_token_wide", op="moe", b=1, m=4096, f=14336, experts=8, k=2, score="softmax", bias=False,
             dtype="fp16"),
        # a ragged decode batch, sigmoid scores with a selection bias
        dict(name="moe_decode_ragged", op="moe", b=13, m=2048, f=1408, experts=60, k=4, score="sigmoid", bias=True,
             dtype="bf16"),
        # a full decode batch over all experts
        dict(name="moe_batch", op="moe", b=128, m=4096, f=1408, experts=128, k=8, score="softmax", bias=False,
             dtype="fp16"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return int(min(max(round(v / step) * step, lo), hi))


def draw(rng):
    limit = {}
    for c in listed():
        limit[c["op"]] = max(limit.get(c["op"], 0), _cost(c))
    held = max(c["experts"] * c["f"] * c["m"] for c in listed() if c["op"] == "moe")
    op = rng.choice(["linear_a16", "linear_a16", "linear_a16", "moe_route", "moe", "moe"])
    while True:
        c = dict(op=op, dtype=rng.choice(sorted(DTYPES)))
        if op == "linear_a16":
            c.update(b=_log(rng, 1, 6000), m=_log(rng, 128, 14336, 128), n=_log(rng, 16, 28672, 16),
                     r=rng.choice([0, 0, 16, 32, 48, 64, 128]))
        else:
            c.update(b=_log(rng, 1, 256), m=_log(rng, 256, 8192, 128), experts=_log(rng, 4, 300),
                     score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5)
            c["k"] = rng.randint(1, min(10, c["experts"]))
            if op == "moe":
                c["f"] = _log(rng, 128, 14336, 128)
                if c["experts"] * c["f"] * c["m"] > held:
                    continue
        if _cost(c) <= limit[op]:
            return c


def _cost(case):
    w = work(case)
    return w["bytes"] / 4e12 + w["flops"] / 1e15


def _pack(q):
    """int8 codes [n][m] -> the library's bytes: two codes a byte, then panels of 16 channels x 64 bytes."""
    n, m = q.shape
    u = q.view(torch.uint8) & 15
    rows = u[:, 0::2] | (u[:, 1::2] << 4)
    return rows.view(n // 16, 16, m // 128, 64).transpose(1, 2).contiguous().view(n, m // 2)


def _inputs(case, seed):
    """The case's tensors on the GPU, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    b, m, op = case["b"], case["m"], case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def weight(n, k):
        q = torch.clamp(torch.round(randn(n, k) * 2.2), -7, 7).to(torch.int8)
        return _pack(q)

    def scales(groups, n):
        return 0.002 + 0.008 * torch.rand(groups, n, generator=g, device=dev)

    # activations: N(0, 1) with a few outlier channels
    x = randn(b, m)
    x[:, torch.randint(0, m, (max(1, m // 200),), generator=g, device=dev)] *= 30.0
    s = {"case": case, "x": x.to(dt)}
    if op == "linear_a16":
        n, r = case["n"], case["r"]
        s["qw"], s["sw"] = weight(n, m), scales(m // GROUP, n)
        s["l1t"] = (randn(r, m) * 0.05).half() if r else None
        s["l2t"] = (randn(n, r) * 0.05).half() if r else None
        return s
    e = case["experts"]
    s["wr"] = (randn(e, m) / math.sqrt(m)).to(dt)
    s["bias"] = randn(e) * 0.1 if case["bias"] else None
    if op == "moe":
        f = case["f"]
        s["q1"] = torch.stack([weight(2 * f, m) for _ in range(e)])  # an expert's f gate rows, then its f up rows
        s["s1"] = scales(m // GROUP, e * 2 * f) * (math.sqrt(4096 / m) * 0.25)
        s["q2"] = torch.stack([weight(m, f) for _ in range(e)])
        s["s2"] = scales(f // GROUP, e * m)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# ---- one pass ----

def run(s):
    c = s["case"]
    if own:
        import w4a4_rank_gemm_amd as twq
        if c["op"] == "linear_a16":
            return twq.linear_a16(s["x"], s["qw"], s["sw"], s["l1t"], s["l2t"])
        if c["op"] == "moe_route":
            return twq.moe_route(s["x"], s["wr"], c["k"], bias=s["bias"], score=c["score"])
        return twq.moe(s["x"], s["wr"], c["k"], (s["q1"], s["s1"]), (s["q2"], s["s2"]), bias=s["bias"],
                       score=c["score"])
    return {"linear_a16": _linear_a16, "moe_route": _moe_route, "moe": _moe}[c["op"]](s)


def _dequant(qw, sw):
    """The packed weight in binary32 [n][m]; sw [m / 128][n]."""
    n, kb = qw.shape
    rows = qw.view(n // 16, kb // 64, 16, 64).transpose(1, 2).reshape(n, kb)
    lo, hi = (rows << 4).view(torch.int8) >> 4, rows.view(torch.int8) >> 4
    codes = torch.stack((lo, hi), dim=2).view(n, kb // 64, GROUP)
    return (codes.float() * sw.T[:, :, None]).view(n, 2 * kb)


def _linear_a16(s):
    x = s["x"].float()
    y = x @ _dequant(s["qw"], s["sw"]).T
    if s["l1t"] is not None:
        y += (x @ s["l1t"].float().T) @ s["l2t"].float().T
    return y.to(s["x"].dtype)


def _moe_route(s):
    c = s["case"]
    logits = s["x"].double() @ s["wr"].double().T  # in 64 bits: which expert is the k-th best hangs on it
    p = torch.softmax(logits, dim=1) if c["score"] == "softmax" else torch.sigmoid(logits)
    by = p + s["bias"].double() if s["bias"] is not None else logits
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.gather(p, 1, ids)
    return ids.to(torch.int32), (w / w.sum(dim=1, keepdim=True)).float()


def _moe(s):
    c = s["case"]
    e_, f, m = c["experts"], c["f"], c["m"]
    x = s["x"].float()
    ids, w = _moe_route(s)
    y = torch.zeros(c["b"], m, device=x.device)
    s1, s2 = s["s1"].view(-1, e_, 2 * f), s["s2"].view(-1, e_, m)
    for e in ids.unique().tolist():
        rows, slot = (ids == e).nonzero(as_tuple=True)
        gu = x[rows] @ _dequant(s["q1"][e], s1[:, e]).T
        h = gu[:, :f] / (1.0 + torch.exp(-gu[:, :f])) * gu[:, f:]
        y[rows] += w[rows, slot][:, None] * (h @ _dequant(s["q2"][e], s2[:, e]).T)
    return y.to(s["x"].dtype)


# ---- the least a pass has to move and compute ----

def work(case):
    b, m, op = case["b"], case["m"], case["op"]
    if op == "linear_a16":
        n, r = case["n"], case["r"]
        return {"bytes": 2 * b * m + n * m // 2 + 4 * n * (m // GROUP) + 2 * r * (m + n) + 2 * b * n,
                "flops": 2 * b * n * m + 2 * b * r * (m + n)}
    e, k = case["experts"], case["k"]
    route = 2 * b * m + 2 * e * m + (4 * e if case["bias"] else 0)
    if op == "moe_route":
        return {"bytes": route + 8 * b * k, "flops": 2 * b * e * m}
    f = case["f"]
    used = e * (1.0 - (1.0 - k / e) ** b)  # experts that b tokens choose, in the mean
    expert = 3 * f * m // 2 + 4 * (2 * f * (m // GROUP) + m * (f // GROUP))
    return {"bytes": int(route + used * expert + 2 * b * m), "flops": 2 * b * e * m + 6 * b * k * f * m}


# ---- the definitions in binary64 ----

def _weight64(qw, sw):
    """One packed weight [n][m] in binary64, code by code."""
    n, kb = qw.shape
    f64 = torch.float64
    part = qw.view(n // 16, kb // 64, 16, 64).permute(0, 2, 1, 3).reshape(n, kb).to(torch.int16)
    w = torch.empty(n, 2 * kb, dtype=f64, device=qw.device)
    for odd in (0, 1):
        code = (part >> (4 * odd)) & 15
        w[:, odd::2] = torch.where(code > 7, code - 16, code).to(f64)
    return w * sw.T.to(f64).repeat_interleave(GROUP, dim=1)


def _route64(case, s):
    f64 = torch.float64
    k, b = case["k"], case["b"]
    logit = torch.einsum("bm,em->be", s["x"].to(f64), s["wr"].to(f64))
    if case["score"] == "softmax":
        z = torch.exp(logit - logit.max(dim=1, keepdim=True).values)
        p = z / z.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-logit))
    left = (p + s["bias"].to(f64)) if s["bias"] is not None else logit.clone()
    ids = torch.empty(b, k, dtype=torch.int64, device=p.device)
    for j in range(k):  # the largest that is left, the first of equals
        best = left.max(dim=1, keepdim=True).values
        ids[:, j] = (left == best).to(torch.int8).argmax(dim=1)
        left[torch.arange(b, device=p.device), ids[:, j]] = -math.inf
    w = p[torch.arange(b, device=p.device)[:, None], ids]
    return ids, w / w.sum(dim=1, keepdim=True)


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    f64 = torch.float64
    x = s["x"].to(f64)
    if op == "linear_a16":
        n, m = case["n"], case["m"]
        y = torch.empty(case["b"], n, dtype=f64, device=x.device)
        step = max(16, (1 << 25) // m // 16 * 16)
        for j in range(0, n, step):  # a run of output channels at a time
            e = min(n, j + step)
            y[:, j:e] = torch.einsum("bm,nm->bn", x, _weight64(s["qw"][j:e], s["sw"][:, j:e]))
        if case["r"]:
            y += torch.einsum("br,nr->bn", torch.einsum("bm,rm->br", x, s["l1t"].to(f64)), s["l2t"].to(f64))
        return y
    ids, w = _route64(case, s)
    if op == "moe_route":
        return ids.to(torch.int32), w
    f, m, n1 = case["f"], case["m"], 2 * case["f"]
    y = torch.zeros(case["b"], m, dtype=f64, device=x.device)
    for e in range(case["experts"]):
        for j in range(case["k"]):
            on = ids[:, j] == e
            if not bool(on.any()):
                continue
            gu = torch.einsum("bm,nm->bn", x[on], _weight64(s["q1"][e], s["s1"][:, e * n1:(e + 1) * n1]))
            gate, up = gu[:, :f], gu[:, f:]
            h = gate / (1.0 + torch.exp(-gate)) * up
            y[on] += w[on, j, None] * torch.einsum("bf,mf->bm", h, _weight64(s["q2"][e], s["s2"][:, e * m:(e + 1) * m]))
    return y
