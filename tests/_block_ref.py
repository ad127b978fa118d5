"""The residual join, its gradients and the int8 product in 64 bits, with
element-wise bounds on the error of an fp32 evaluation.

A bound is ADDS * 2^-24 times the sum of the magnitudes that enter an element
(every fp32 operation errs by at most 2^-24 of its result, and a sum of n terms
by at most as many roundings as lie on one term's way), plus half a unit of the
output's type.
"""
import torch

UNIT = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
# Roundings on one element's way: a row sum takes at most 32 terms in a thread,
# 5 in a warp and 32 (64 in a cluster) across warps; an output passes two such
# sums and a dozen operations of its own.
ADDS = 2 * (32 + 5 + 64) + 24


def _norm(v, kind, eps):
    mean = v.mean(1, keepdim=True) if kind else torch.zeros_like(v[:, :1])
    rstd = 1 / torch.sqrt(((v - mean) ** 2).mean(1, keepdim=True) + eps)
    return (v - mean) * rstd, mean, rstd


def per_row(gate, rows):
    return 1.0 if gate is None else gate.repeat_interleave(rows // gate.shape[0], 0)


def forward(kind, post, eps, scale, x, y, gate, p):
    """x, y, gate and the dict p in double; r, h, stats and bounds of r and h."""
    rows, width = x.shape
    one, zero = torch.ones(width, dtype=x.dtype, device=x.device), torch.zeros(width, dtype=x.dtype, device=x.device)
    w1, b1, w2, b2 = (p.get(k) if p.get(k) is not None else d
                      for k, d in (("w_post", one), ("b_post", zero), ("w_pre", one), ("b_pre", zero)))
    mean1, rstd1 = torch.zeros_like(x[:, :1]), torch.ones_like(x[:, :1])
    if y is None:
        r, mag_r = x, x.abs()
    else:
        n, mag_n = y, y.abs()
        if post:
            hat, mean1, rstd1 = _norm(y, kind, eps)
            n = hat * w1 + b1
            mag_n = ((y.abs() + mean1.abs() + y.abs().mean(1, keepdim=True)) * rstd1 + hat.abs()) * w1.abs() + b1.abs()
        g = per_row(gate, rows)
        r = x + scale * g * n
        mag_r = x.abs() + abs(scale) * (abs(g) if gate is None else g.abs()) * mag_n
    hat2, mean2, rstd2 = _norm(r, kind, eps)
    h = hat2 * w2 + b2
    spread = (mag_r * mag_r).mean(1, keepdim=True).sqrt()       # error of the row's own statistics
    mag_h = ((mag_r + mag_r.mean(1, keepdim=True)) * rstd2 + hat2.abs() * (1 + spread * rstd2)) * w2.abs() + b2.abs()
    stats = torch.cat([mean1, rstd1, mean2, rstd2], 1)
    return r, h, stats, mag_r * ADDS * 2.0 ** -24, mag_h * ADDS * 2.0 ** -24


def within(got, want, bound, what):
    """got (any type) within bound + its rounding of want (double)."""
    unit = UNIT[got.dtype]
    limit = bound * (1 + unit) + unit * want.abs() + TINY[got.dtype]
    off = (got.double() - want).abs()
    bad = ~(off <= limit)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((off / limit)[bad].max()):.3g} times its bound")


def backward(kind, post, eps, scale, x, y, gate, p, dr, dh):
    """The formula's gradients in double, each with its bound: {name: (value, bound)}."""
    rows, width = x.shape
    one = torch.ones(width, dtype=x.dtype, device=x.device)
    r, _, stats, err_r, _ = forward(kind, post, eps, scale, x, y, gate, p)
    w1, w2 = (p.get(k) if p.get(k) is not None else one for k in ("w_post", "w_pre"))
    mean1, rstd1, mean2, rstd2 = stats.split(1, 1)
    u = 2.0 ** -24
    m = lambda v: v.mean(1, keepdim=True)                                          # noqa: E731
    zero = torch.zeros_like(x)
    dr = zero if dr is None else dr
    out = {}
    d, err_d = dr, dr.abs() * u
    hat2 = (r - mean2) * rstd2
    if dh is not None:
        # the kernel's hat2 comes from fp32 statistics and an fp32 r
        err_hat2 = (err_r + ADDS * u * (r.abs() + mean2.abs())) * rstd2 + ADDS * u * hat2.abs()
        g = dh * w2
        back = g - hat2 * m(g * hat2) - (m(g) if kind else 0)
        mag = g.abs() + m(g.abs()) + hat2.abs() * m((g * hat2).abs())
        err = ADDS * u * mag + err_hat2 * m(g * hat2).abs() + hat2.abs() * m(g.abs() * err_hat2)
        d = dr + rstd2 * back
        err_d = err_d + rstd2 * err + u * d.abs()
        out["w_pre"] = ((dh * hat2).sum(0), dh.abs() * (err_hat2 + ADDS * u * hat2.abs()))
        out["b_pre"] = (dh.sum(0), ADDS * u * dh.abs())
    else:
        out["w_pre"], out["b_pre"] = (zero.sum(0), zero), (zero.sum(0), zero)
    out["x"] = (d, err_d)
    if y is not None:
        hat1 = (y - mean1) * rstd1 if post else y
        err1 = ADDS * u * ((y.abs() + mean1.abs()) * rstd1 + hat1.abs()) if post else zero
        b1 = p.get("b_post") if p.get("b_post") is not None else 0 * one
        n = hat1 * w1 + b1 if post else y
        gr = per_row(gate, rows)
        if gate is not None:
            v = scale * d * n
            e = abs(scale) * (err_d * n.abs() + d.abs() * (err1 * w1.abs() + 4 * u * (hat1.abs() * w1.abs() + b1.abs())))
            e = e + ADDS * u * v.abs()
            fold = lambda t: t.view(gate.shape[0], rows // gate.shape[0], width).sum(1)   # noqa: E731
            v, e = fold(v), fold(e)
            if gate.shape[1] == 1:
                v, e = v.sum(1, keepdim=True), e.sum(1, keepdim=True)
            out["gate"] = (v, e)
        dn = scale * gr * d
        err_dn = abs(scale) * (abs(gr) if gate is None else gr.abs()) * err_d + 3 * u * dn.abs()
        if post:
            out["w_post"] = ((dn * hat1).sum(0), err_dn * hat1.abs() + dn.abs() * err1 + ADDS * u * (dn * hat1).abs())
            out["b_post"] = (dn.sum(0), err_dn + ADDS * u * dn.abs())
            f, err_f = dn * w1, err_dn * w1.abs() + u * (dn * w1).abs()
            dy = rstd1 * (f - hat1 * m(f * hat1) - (m(f) if kind else 0))
            mag = f.abs() + m(f.abs()) + hat1.abs() * m((f * hat1).abs())
            err = ADDS * u * mag + err_f + m(err_f) + hat1.abs() * m(err_f * hat1.abs() + f.abs() * err1) \
                + err1 * m(f * hat1).abs()
            out["y"] = (dy, rstd1 * err)
        else:
            out["y"] = (dn, err_dn)
    for k in ("w_pre", "b_pre", "w_post", "b_post"):
        if k in out:
            out[k] = (out[k][0], out[k][1].sum(0))
    return out
