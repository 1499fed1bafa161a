"""Binary64 definitions of the 16-bit-activation layer, the router and the routed layer, with
elementwise bounds on what the kernels may be off by.

u = 2^-24 is half a step of binary32. Products of a 16-bit element and a code (or one of its two
16-bit parts) are exact in binary32; a sum of K of them, in any order, is off by at most K u
sum|products|. T and the experts' inner rows enter their second product as two bf16 parts
(2^-18 of the value) or two fp16 parts of a scaled row (2^-22 and 2^-38 of the row's largest)."""
import torch

from tests.adapter_reference import F64, U, rounded

BF_PARTS, F16_PARTS = 2.0 ** -18, 2.0 ** -22


def few(b, n):
    """The few-row kernels: up to 64 rows, or up to 512 blocks of 64 rows x 128 channels."""
    return b <= 64 or -(-n // 128) * -(-b // 64) <= 512


def codes_of(qw):
    """The packed weight's codes [n][m], binary64."""
    n, kb = qw.shape
    rows = qw.view(n // 16, kb // 64, 16, 64).transpose(1, 2).reshape(n, kb).to(torch.int16)
    c = torch.stack((rows & 15, rows >> 4), dim=2).view(n, 2 * kb)
    return torch.where(c > 7, c - 16, c).to(F64)


def pack(codes):
    """int8 codes [n][m] in the library's panels."""
    n, m = codes.shape
    u = codes.to(torch.int8).view(torch.uint8) & 15
    rows = u[:, 0::2] | (u[:, 1::2] << 4)
    return rows.view(n // 16, 16, m // 128, 64).transpose(1, 2).contiguous().view(n, m // 2)


def dense(qw, sw):
    """s_W Q_W [n][m]"""
    return codes_of(qw) * sw.to(F64).T.repeat_interleave(128, dim=1)


def _product(x, w, parts=1):
    """x w^T for the few-row kernels: a group's 128 (parts) products, then one multiply-add a group,
    a few more for the sums of waves and slices."""
    m = x.shape[1]
    return x @ w.T, (128 * parts + m // 128 + 40) * U * (x.abs() @ w.abs().T)


def linear_a16(x, qw, sw, l1t, l2t, tokens=None, channels=None):
    """(Y, bound) of rows of a batch of `tokens` and `channels` (all of them if not given)."""
    dtype, (b, m) = x.dtype, x.shape
    b = tokens or b
    x64, w = x.to(F64), dense(qw, sw)
    is_few = few(b, channels or qw.shape[0])
    if is_few:
        v, e = _product(x64, w)
    else:
        # sums over all of K, multiplied by a ratio (itself rounded) once a group
        v, e = x64 @ w.T, (m + 3 * (m // 128) + 40) * U * (x64.abs() @ w.abs().T)
        if dtype == torch.bfloat16:  # fp16 of a scaled row, below its normal range
            e = e + 2.0 ** -39 * x64.abs().amax(1, keepdim=True) * w.abs().sum(1)
        # groups whose scale is below 2^-90 of the channel's largest are left out
        s = sw.to(F64).abs()
        least = torch.where(s < 2.0 ** -90 * s.amax(0), s, torch.zeros_like(s)).amax(0)
        e = e + 7 * least * x64.abs().sum(1, keepdim=True)
    if l1t is not None:
        l1, l2 = l1t.to(F64), l2t.to(F64)
        t, et = x64 @ l1.T, 2 * m * U * (x64.abs() @ l1.abs().T)
        if is_few:
            et = et + BF_PARTS * (t.abs() + et)
        else:
            et = et + F16_PARTS * (t.abs() + et) + 2.0 ** -38 * t.abs().amax(1, keepdim=True)
        v = v + t @ l2.T
        e = e + et @ l2.abs().T + 8 * l2.shape[1] * U * ((t.abs() + et) @ l2.abs().T)
    return v, rounded(v, e + 4 * U * v.abs(), dtype)


def route(x, wr, k, bias=None, score="softmax", norm=True, scale=1.0):
    """(ids, weights) in binary64: the largest first, the lowest index first among equals."""
    logits = x.to(F64) @ wr.to(F64).T
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    by = logits if bias is None else p + bias.to(F64)
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if norm:
        w = w / w.sum(1, keepdim=True)
    return ids, w * scale


def experts(x, ids, weights, gate_up, down):
    """(Y, bound) of the experts' products for a given choice."""
    dtype, (b, m) = x.dtype, x.shape
    (q1, s1), (q2, s2) = gate_up, down
    n_exp, f = q1.shape[0], q1.shape[1] // 2
    s1, s2 = s1.view(-1, n_exp, 2 * f), s2.view(-1, n_exp, m)
    y = torch.zeros(b, m, dtype=F64, device=x.device)
    err = torch.zeros_like(y)
    x64 = x.to(F64)
    for i in range(b):
        for j in range(ids.shape[1]):
            a = int(ids[i, j])
            if not 0 <= a < n_exp:
                continue
            gu, egu = _product(x64[i:i + 1], dense(q1[a], s1[:, a]))
            g, up, eg, eu = gu[:, :f], gu[:, f:], egu[:, :f], egu[:, f:]
            act = g / (1 + torch.exp(-g))
            # the slope of silu is at most 1.1; exp of -g is off by (|g| + 8) 2^-23, and infinite below -88
            ea = 1.1 * eg + act.abs() * ((g.abs() + 8) * 2.0 ** -23 + 4 * U) + 1e-35
            h = act * up
            eh = ea * (up.abs() + eu) + act.abs() * eu + 2 * U * h.abs()
            eh = eh + BF_PARTS * (h.abs() + eh)
            w2 = dense(q2[a], s2[:, a])
            v, e = _product(h, w2, 2)
            e = e + eh @ w2.abs().T * 1.01
            w = float(weights[i, j])
            y[i] += w * v[0]
            err[i] += abs(w) * (e[0] + 20 * U * v[0].abs())
    return y, rounded(y, err, dtype)
