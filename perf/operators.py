"""Workloads of the adapter operators: what a training or serving step asks of them.

Four operators stand beside the fused 4-bit layer Y = s_X s_W (Q_X Q_W) + (X L1) L2:

* ``adapters``       out = y + scale_a (X A_a) B_a per token, a = the token's adapter
* ``adapters_grad``  the gradients of that product: dA_a, dB_a and dX
* ``checkpoint``     activations kept in 8 bits between forward and backward, and restored
* ``linear_dx``      the frozen layer's input gradient, dX = dY W^T, W = s_W Q_W + L1 L2

``run`` computes a case in elementary torch operations (binary32, rounded once), or, with
``own`` set, through this repository's library. ``exact`` evaluates the definitions in
binary64. Shapes: the layers of ``synth.CONFIGS`` and generic sizes.
"""
import math

import torch

own = False

GROUP = 128  # elements of one 8-bit checkpoint group
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # one request in a small model: nothing but launch latency
        dict(name="adapters_one_token", op="adapters", b=1, m=512, n=512, r=16, count=4, spread="tokens", none=0.0,
             dtype="fp16", keep_h=False),
        # a decode step of mixed requests: popular and rare adapters, some tokens without one
        dict(name="adapters_decode_mixed", op="adapters", b=61, m=4096, n=4096, r=32, count=12, spread="zipf",
             none=0.2, dtype="bf16", keep_h=False),
        # a decode step of a 70B gate/up projection, every token its own adapter
        dict(name="adapters_decode_distinct", op="adapters", b=32, m=8192, n=28672, r=64, count=32, spread="distinct",
             none=0.0, dtype="fp16", keep_h=False),
        # training forward of an 8B down projection: six jobs' tokens side by side, X A kept for the backward
        dict(name="adapters_prefill", op="adapters", b=4096, m=14336, n=4096, r=64, count=6, spread="segments",
             none=0.05, dtype="fp16", keep_h=True),
        # a short ragged batch, activations unquantized
        dict(name="grad_small", op="adapters_grad", b=197, m=512, n=528, r=16, count=3, spread="segments", none=0.1,
             dtype="fp16", saved="full"),
        # one 8B gate/up projection of a training step, activations from the 8-bit checkpoint
        dict(name="grad_checkpoint", op="adapters_grad", b=2048, m=4096, n=14336, r=32, count=8, spread="segments",
             none=0.0, dtype="fp16", saved="int8"),
        # the same layer at a long batch, higher rank, bfloat16
        dict(name="grad_long", op="adapters_grad", b=8192, m=4096, n=14336, r=64, count=16, spread="segments", none=0.0,
             dtype="bf16", saved="int8"),
        # a small layer's activations
        dict(name="checkpoint_small", op="checkpoint", b=16, m=512, dtype="fp16"),
        # the input of an 8B down projection at a long batch
        dict(name="checkpoint_long", op="checkpoint", b=8192, m=14336, dtype="bf16"),
        # a short sequence through a small layer
        dict(name="dx_small", op="linear_dx", b=16, m=512, n=512, r=16, dtype="fp16"),
        # an 8B gate/up projection
        dict(name="dx_8b", op="linear_dx", b=2048, m=4096, n=14336, r=32, dtype="bf16"),
        # a 70B gate/up projection
        dict(name="dx_70b", op="linear_dx", b=4096, m=8192, n=28672, r=128, dtype="fp16"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return int(min(max(round(v / step) * step, lo), hi))


def draw(rng):
    limit = {}
    for c in listed():
        limit[c["op"]] = max(limit.get(c["op"], 0), _cost(c))
    op = rng.choice(["adapters", "adapters", "adapters_grad", "adapters_grad", "checkpoint", "linear_dx"])
    while True:
        c = dict(op=op, b=0, m=_log(rng, 512, 14336, 128), dtype=rng.choice(sorted(DTYPES)))
        if op == "checkpoint":
            c["b"] = _log(rng, 1, 16384)
        elif op == "linear_dx":
            c.update(b=_log(rng, 1, 6000), n=_log(rng, 512, 28672, 16), r=rng.choice([0, 16, 32, 48, 64, 128]))
        else:
            c.update(b=_log(rng, 1, 8192), n=_log(rng, 512, 28672, 16), r=rng.choice([16, 32, 48, 64, 96, 128]),
                     count=_log(rng, 1, 64), spread=rng.choice(["tokens", "zipf", "distinct", "segments"]),
                     none=rng.choice([0.0, 0.1, 0.5]))
            if op == "adapters":
                c["keep_h"] = rng.random() < 0.5
            else:
                c["b"] = max(c["b"], 16)
                c["saved"] = rng.choice(["full", "int8"])
        if _cost(c) <= limit[op]:
            return c


def _cost(case):
    w = work(case)
    return w["bytes"] / 4e12 + w["flops"] / 1e15


def _index(case, seed):
    """Each token's adapter (-1: none), a CPU int32 tensor."""
    b, count = case["b"], case["count"]
    g = torch.Generator().manual_seed(seed * 7919 + 17)
    if case["spread"] == "distinct":
        idx = torch.randperm(max(b, count), generator=g)[:b] % count
    elif case["spread"] == "tokens":
        idx = torch.randint(0, count, (b,), generator=g)
    elif case["spread"] == "zipf":
        p = 1.0 / torch.arange(1, count + 1, dtype=torch.float64)
        idx = torch.multinomial(p, b, replacement=True, generator=g)
    else:  # requests of ragged lengths one after another, their adapters in no order
        cuts = torch.rand(2 * count, generator=g).sort().values
        owner = torch.randint(0, count, (2 * count + 1,), generator=g)
        idx = owner[torch.bucketize((torch.arange(b) + 0.5) / max(b, 1), cuts.double())]
    if case["none"]:
        idx = torch.where(torch.rand(b, generator=g) < case["none"], torch.full_like(idx, -1), idx)
    return idx.to(torch.int32)


def _inputs(case, seed):
    """The case's tensors on the GPU, from the seed alone."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    b, m, op = case["b"], case["m"], case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = {"case": case}
    if op != "linear_dx":  # activations: N(0, 1) with a few outlier channels
        x = randn(b, m)
        out = torch.randint(0, m, (max(1, m // 200),), generator=g, device=dev)
        x[:, out] *= 30.0
        s["x"] = x.to(dt)
    if op in ("adapters", "adapters_grad"):
        n, r, count = case["n"], case["r"], case["count"]
        s["index"] = _index(case, seed).to(dev)
        s["at"] = (randn(count, r, m) / math.sqrt(m)).to(dt)
        s["bt"] = (randn(count, n, r) * 0.05).to(dt)
        s["scale"] = 0.5 + 1.5 * torch.rand(count, generator=g, device=dev)
        if op == "adapters":
            s["y"] = randn(b, n).to(dt)
    if op in ("adapters_grad", "linear_dx"):
        n = case["n"]
        dy = randn(b, n) * 2.0 ** -8
        dy[torch.rand(b, generator=g, device=dev) < 0.05] = 0.0  # tokens the loss does not count
        s["dy"] = dy.to(dt)
    if op == "adapters_grad":
        s["dx"] = (randn(b, m) * 2.0 ** -8).to(dt)  # the frozen layer's share
        # what the forward pass kept: X A in binary32, and X whole or in 8 bits
        live = s["index"] >= 0
        h = torch.zeros(b, case["r"], device=dev)
        for a in range(case["count"]):
            rows = ((s["index"] == a) & live).nonzero()[:, 0]
            h[rows] = s["x"][rows].float() @ s["at"][a].float().T
        s["h"] = h
        if case["saved"] == "int8":
            x3 = s["x"].float().view(b, m // GROUP, GROUP)
            sc = x3.abs().amax(2) / torch.full((), 127.0, device=dev)
            q = torch.round(x3 / torch.where(sc > 0, sc, torch.ones_like(sc))[:, :, None])
            s["qc"] = q.to(torch.int8).view(b, m)
            s["sc"] = sc.T.contiguous()
            del s["x"]
    if op == "linear_dx":
        n, r = case["n"], case["r"]
        q = torch.clamp(torch.round(randn(n, m) * 2.0), -7, 7).to(torch.int8)
        u = q.view(torch.uint8) & 15
        # two codes a byte, then panels of 16 channels x 64 bytes
        rows = u[:, 0::2] | (u[:, 1::2] << 4)
        s["qw"] = rows.view(n // 16, 16, m // 128, 64).transpose(1, 2).contiguous().view(n, m // 2)
        s["sw"] = 0.002 + 0.004 * torch.rand(n, generator=g, device=dev)
        s["l1t"] = (randn(r, m) * 0.1).half() if r else None
        s["l2t"] = (randn(n, r) * 0.1).half() if r else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if "index" in s:
        # the batch's token lists, as a program has them that schedules its requests
        idx = s["index"].cpu()
        s["rows"] = [(a, (idx == a).nonzero()[:, 0].to("cuda")) for a in range(case["count"]) if (idx == a).any()]
        if own:
            import w4a4_rank_gemm_amd as twq
            s["plan"] = twq.adapter_plan(s["index"], case["count"])
    return s


# ---- one pass ----

def run(s):
    op = s["case"]["op"]
    if own:
        import w4a4_rank_gemm_amd as twq
        if op == "adapters":
            return twq.adapters(s["x"], s["at"], s["bt"], s["plan"], s["y"], s["scale"], keep_h=s["case"]["keep_h"])
        if op == "adapters_grad":
            saved = s["x"] if "x" in s else (s["qc"], s["sc"])
            return twq.adapters_grad(s["dy"], saved, s["h"], s["at"], s["bt"], s["plan"], s["scale"], dx=s["dx"])
        if op == "checkpoint":
            qc, sc = twq.checkpoint_act(s["x"])
            return twq.restore_act(qc, sc, s["x"].dtype), sc
        return twq.linear_dx(s["dy"], s["qw"], s["sw"], s["l1t"], s["l2t"])
    return {"adapters": _adapters, "adapters_grad": _adapters_grad, "checkpoint": _checkpoint,
            "linear_dx": _linear_dx}[op](s)


def _adapters(s):
    x, y = s["x"], s["y"]
    out = y.clone()
    h = torch.zeros(x.shape[0], s["at"].shape[1], device=x.device) if s["case"]["keep_h"] else None
    for a, rows in s["rows"]:
        t = x[rows].float() @ s["at"][a].float().T
        out[rows] = (y[rows].float() + s["scale"][a] * (t @ s["bt"][a].float().T)).to(y.dtype)
        if h is not None:
            h[rows] = t
    return out if h is None else (out, h)


def _adapters_grad(s):
    dy, at, bt = s["dy"], s["at"], s["bt"]
    dat, dbt, dx = torch.zeros_like(at), torch.zeros_like(bt), s["dx"].clone()
    for a, rows in s["rows"]:
        d = dy[rows].float() * s["scale"][a]
        t = d @ bt[a].float()
        if "x" in s:
            xr = s["x"][rows].float()
        else:
            xr = (s["qc"][rows].float().view(len(rows), -1, GROUP) * s["sc"].T[rows][:, :, None]).view(len(rows), -1)
        dat[a] = (t.T @ xr).to(at.dtype)
        dbt[a] = (d.T @ s["h"][rows]).to(bt.dtype)
        dx[rows] = (s["dx"][rows].float() + t @ at[a].float()).to(dx.dtype)
    return dat, dbt, dx


def _checkpoint(s):
    x = s["x"]
    b, m = x.shape
    x3 = x.float().view(b, m // GROUP, GROUP)
    sc = x3.abs().amax(2) / torch.full((), 127.0, device=x.device)  # a number would multiply by its reciprocal
    q = torch.round(x3 / torch.where(sc > 0, sc, torch.ones_like(sc))[:, :, None])
    codes, sct = q.to(torch.int8), sc.T.contiguous()
    back = codes.float() * sct.T[:, :, None]
    return back.view(b, m).to(x.dtype), sct


def _codes(qw):
    """The packed weight's codes, int8 [n][m]."""
    n, kb = qw.shape
    rows = qw.view(n // 16, kb // 64, 16, 64).transpose(1, 2).reshape(n, kb)
    lo, hi = (rows << 4).view(torch.int8) >> 4, rows.view(torch.int8) >> 4
    return torch.stack((lo, hi), dim=2).view(n, 2 * kb)


def _linear_dx(s):
    dy = s["dy"].float()
    dx = (dy * s["sw"]) @ _codes(s["qw"]).float()
    if s["l1t"] is not None:
        dx += (dy @ s["l2t"].float()) @ s["l1t"].float()
    return dx.to(s["dy"].dtype)


# ---- the least a pass has to move and compute ----

def work(case):
    b, m, op = case["b"], case["m"], case["op"]
    if op == "checkpoint":  # X in, codes out and in, scales out and in, X out
        return {"bytes": 2 * b * m + 2 * b * m + 2 * 4 * b * (m // GROUP) + 2 * b * m, "flops": 5 * b * m}
    n, r = case["n"], case["r"]
    if op == "linear_dx":
        return {"bytes": 2 * b * n + n * m // 2 + 4 * n + 2 * r * (m + n) + 2 * b * m,
                "flops": 2 * b * n * m + 2 * b * r * (m + n)}
    live = b * (1.0 - case["none"])
    used = min(case["count"], max(1, int(live)))
    weights = used * r * (m + n) * 2
    if op == "adapters":
        return {"bytes": int(weights + 4 * b + live * 2 * m + 4 * b * n + (4 * b * r if case["keep_h"] else 0)),
                "flops": int(2 * live * r * (m + n))}
    xb = 1 + 4 / GROUP if case["saved"] == "int8" else 2
    grads = case["count"] * r * (m + n) * 2
    return {"bytes": int(weights + grads + 4 * b + live * (2 * n + xb * m + 4 * r) + 4 * b * m),
            "flops": int(2 * live * r * (2 * m + 2 * n))}


# ---- the definitions in binary64 ----

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "checkpoint":
        # s = fl32(max |x| / 127) per token and group, code = nearest even of fl32(x / s)
        x = s["x"].to(f64)
        sc = torch.empty(case["m"] // GROUP, case["b"], dtype=f64, device=x.device)
        back = torch.zeros_like(x)
        for g in range(case["m"] // GROUP):
            part = x[:, g * GROUP:(g + 1) * GROUP]
            sg = (part.abs().max(dim=1).values / 127.0).float().to(f64)
            sc[g] = sg
            ok = sg > 0
            ratio = (part[ok] / sg[ok, None]).float().to(f64)
            back[ok, g * GROUP:(g + 1) * GROUP] = torch.round(ratio) * sg[ok, None]
        return back, sc
    if op == "linear_dx":
        n, m, r = case["n"], case["m"], case["r"]
        dx = torch.zeros(case["b"], m, dtype=f64, device="cuda")
        w = s["qw"].view(n // 16, m // 128, 16, 64)
        step = max(16, (1 << 24) // m // 16 * 16)
        for j in range(0, n, step):  # a run of output channels: sum over its weight rows
            e = min(n, j + step)
            part = w[j // 16:e // 16].permute(0, 2, 1, 3).reshape(e - j, m // 2).to(torch.int16)
            wd = torch.empty(e - j, m, dtype=f64, device="cuda")
            for odd in (0, 1):
                c = (part >> (4 * odd)) & 15
                wd[:, odd::2] = torch.where(c > 7, c - 16, c).to(f64)
            wd *= s["sw"][j:e, None].to(f64)
            if r:
                wd += s["l2t"][j:e].to(f64) @ s["l1t"].to(f64)
            dx += s["dy"][:, j:e].to(f64) @ wd
        return dx
    b, m, n, r = case["b"], case["m"], case["n"], case["r"]
    scale = s["scale"].to(f64)
    if op == "adapters":
        out = s["y"].to(f64)
        h = torch.zeros(b, r, dtype=f64, device="cuda")
        for a in range(case["count"]):
            on = s["index"] == a
            if bool(on.any()):
                h[on] = torch.einsum("bm,rm->br", s["x"][on].to(f64), s["at"][a].to(f64))
                out[on] += torch.einsum("br,nr->bn", h[on] * scale[a], s["bt"][a].to(f64))
        return (out, h) if case["keep_h"] else out
    dat = torch.zeros(case["count"], r, m, dtype=f64, device="cuda")
    dbt = torch.zeros(case["count"], n, r, dtype=f64, device="cuda")
    dx = s["dx"].to(f64)
    if "x" in s:
        x = s["x"].to(f64)
    else:
        x = s["qc"].to(f64) * s["sc"].to(f64).T.repeat_interleave(GROUP, dim=1)
    for a in range(case["count"]):
        on = s["index"] == a
        if bool(on.any()):
            d = s["dy"][on].to(f64)
            g = scale[a] * torch.einsum("bn,nr->br", d, s["bt"][a].to(f64))
            dat[a] = torch.einsum("br,bm->rm", g, x[on])
            dbt[a] = scale[a] * torch.einsum("bn,br->nr", d, s["h"][on].to(f64))
            dx[on] += torch.einsum("br,rm->bm", g, s["at"][a].to(f64))
    return dat, dbt, dx
