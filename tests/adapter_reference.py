"""Binary64 definitions of the adapter, checkpoint and input-gradient operators, each with
an elementwise bound on what the kernels may be off by.

Bounds: u = 2^-24 is half a step of binary32. A sum of K products in binary32, in any order,
is off by at most K u sum|products| (products of two 16-bit elements are exact there; one u
more for others, counted by taking 2 K). A value kept as two 16-bit parts is off by the
second part's rounding: fp16 2^-22 of the value and, below the normal range of the scaled
row, 2^-25 steps of a row whose largest element is at least 2^13, so 2^-38 of that; bf16
2^-18. The last rounding is eps / 2 of the result (half the smallest subnormal near 0)."""
import torch

F64 = torch.float64
U = 2.0 ** -24
SPLIT = {torch.float16: 2.0 ** -22, torch.bfloat16: 2.0 ** -18}
FLOOR = {torch.float16: 2.0 ** -38, torch.bfloat16: 0.0}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the smallest subnormal


def rounded(exact, err, dtype):
    """The bound after one rounding to dtype."""
    half = torch.finfo(dtype).eps / 2
    return err + half * (exact.abs() + err) + TINY[dtype]


def _second(h, eh, w, c, dtype):
    """c h w for h [b][r] (off by eh) and w [r][n]: value and bound before rounding."""
    r = h.shape[1]
    hc, ehc = (c * h), abs(c) * eh + U * abs(c) * h.abs()
    split = SPLIT[dtype] * hc.abs() + FLOOR[dtype] * hc.abs().amax(1, keepdim=True) + ehc
    return hc @ w, split @ w.abs() + 4 * r * U * ((hc.abs() + split) @ w.abs())


def adapters(x, at, bt, index, y, scale):
    """(out, bound), (h, bound)"""
    dtype, (b, m) = x.dtype, x.shape
    count, n, r = bt.shape
    out = torch.zeros(b, n, dtype=F64, device=x.device) if y is None else y.to(F64).clone()
    err = torch.zeros_like(out)
    h = torch.zeros(b, r, dtype=F64, device=x.device)
    eh = torch.zeros_like(h)
    for a in range(count):
        on = index == a
        if not bool(on.any()):
            continue
        c = 1.0 if scale is None else float(scale[a])
        xa, aa = x[on].to(F64), at[a].to(F64).T
        h[on], eh[on] = xa @ aa, m * U * (xa.abs() @ aa.abs())
        v, e = _second(h[on], eh[on], bt[a].to(F64).T, c, dtype)
        out[on] += v
        err[on] += e + U * out[on].abs()
    on = (index >= 0) & (index < count)
    bound = rounded(out, err, dtype)
    bound[~on] = 0.0
    return (out, bound), (h, eh)


def adapters_grad(dy, x, h, at, bt, index, scale, dx):
    """[(dat, bound), (dbt, bound), (dX, bound)]; x in binary64 (restored, if a checkpoint)."""
    dtype, b = dy.dtype, dy.shape[0]
    count, n, r = bt.shape
    m = at.shape[2]
    dat = torch.zeros(count, r, m, dtype=F64, device=dy.device)
    dbt = torch.zeros(count, n, r, dtype=F64, device=dy.device)
    ea, eb = torch.zeros_like(dat), torch.zeros_like(dbt)
    dxo = torch.zeros(b, m, dtype=F64, device=dy.device) if dx is None else dx.to(F64).clone()
    ex = torch.zeros_like(dxo)
    bf = 2.0 ** -18  # two bf16 parts, whatever the element type
    for a in range(count):
        on = index == a
        rows = int(on.sum())
        if not rows:
            continue
        c = 1.0 if scale is None else float(scale[a])
        d, ba, aa, xa, ha = dy[on].to(F64), bt[a].to(F64), at[a].to(F64), x[on].to(F64), h[on].to(F64)
        g, eg = d @ ba, n * U * (d.abs() @ ba.abs())
        v, e = _second(g, eg, aa, c, dtype)
        dxo[on] += v
        ex[on] += e + U * dxo[on].abs()
        # the factor c g s: two binary32 roundings and the split; K = the adapter's rows, three
        # products each and the joining of pieces
        gc, egc = c * g, abs(c) * (eg + (3 * U + bf) * g.abs())
        dat[a] = gc.T @ xa
        ea[a] = egc.T @ xa.abs() + 8 * rows * U * ((gc.abs() + egc).T @ xa.abs())
        hc, ehc = c * ha, abs(c) * (3 * U + bf) * ha.abs()
        dbt[a] = d.T @ hc
        eb[a] = d.abs().T @ ehc + 8 * rows * U * (d.abs().T @ (hc.abs() + ehc))
    bx = rounded(dxo, ex, dtype)
    bx[~((index >= 0) & (index < count))] = 0.0
    return [(dat, rounded(dat, ea, dtype)), (dbt, rounded(dbt, eb, dtype)), (dxo, bx)]


def linear_dx(dy, codes, sw, l1t, l2t):
    """(dX, bound); codes [n][m]"""
    dtype, n = dy.dtype, dy.shape[1]
    d, q = dy.to(F64), codes.to(F64)
    g = d * sw.to(F64)
    # fp16 of the scaled row: 2^-11 and two binary32 roundings; below its normal range 2^-25 of a
    # row whose largest element is at least 2^14
    eg = (2.0 ** -11 + 3 * U) * g.abs() + 2.0 ** -39 * g.abs().amax(1, keepdim=True)
    eg = torch.where(g == 0, torch.zeros_like(eg), eg)
    v = g @ q
    e = eg @ q.abs() + 2 * n * U * ((g.abs() + eg) @ q.abs())
    if l1t is not None:
        l1, l2 = l1t.to(F64), l2t.to(F64)
        t, et = d @ l2, 2 * n * U * (d.abs() @ l2.abs())
        # T's exponent is kept within 2^40 of G's: 2^-25 steps of 2^14 2^-40 max|G|
        top = torch.maximum(t.abs().amax(1, keepdim=True), 2.0 ** -39 * g.abs().amax(1, keepdim=True))
        et = et + (2.0 ** -22 + U) * t.abs() + 2.0 ** -38 * top
        w = t @ l1
        e = e + et @ l1.abs() + 4 * l1.shape[0] * U * ((t.abs() + et) @ l1.abs() + v.abs() + e)
        v = v + w
    return v, rounded(v, e + 2 * U * v.abs(), dtype)


def checkpoint(x):
    """(codes, scales [m/128][b]), both exact: each division rounded once to binary32 (a
    binary64 quotient of binary32 operands rounds to the same value). A group that is not
    finite: scale NaN, codes 0."""
    b, m = x.shape
    x3 = x.to(F64).view(b, m // 128, 128)
    s = (x3.abs().amax(2) / 127.0).float().to(F64)
    s = torch.where(x3.isfinite().all(2), s, torch.full_like(s, float("nan")))
    ratio = (x3 / torch.where(s > 0, s, torch.ones_like(s))[:, :, None]).float().to(F64)
    q = torch.where(s[:, :, None] > 0, torch.round(ratio).clamp(-127, 127), torch.zeros_like(ratio))
    return q.view(b, m).to(torch.int8), s.T.contiguous().float()


def same(a, b):
    """Equal element for element, NaN to NaN."""
    return a.dtype == b.dtype and torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


def check(got, want, name):
    value, bound = want
    err = (got.to(F64) - value).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                                 f"{float((err - bound).max())}, at {bad.nonzero()[0].tolist()}: "
                                 f"{float(got[tuple(bad.nonzero()[0])])} for {float(value[tuple(bad.nonzero()[0])])}")
