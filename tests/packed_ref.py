"""64-bit references of the packed operators and the error bounds their tests use.

The bounds are first-order rounding analyses, evaluated element by element on the reference's own
values.  u = eps / 2 of the 16-bit type is the most one rounding moves a value, relatively;
float32 sums of d products are off by at most d 2^-24 of the sum of the products' magnitudes.
"""
from __future__ import annotations

import math

import torch

F32 = 2.0 ** -24


def unit(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def tiny(dtype) -> float:
    """Half the spacing of the type's subnormals: the most a rounding is off near zero."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def attention(q, k, v, lengths, causal, scale, do=None):
    """o, lse, (dq, dk, dv) of packed attention in float64 and, under the same names with "_tol",
    how far a kernel that rounds P and dS (and o for the row dot products) to the 16-bit type
    once, sums in float32 and rounds its outputs may be off."""
    dt, u = q.dtype, unit(q.dtype)
    T, hq, d = q.shape
    hkv = k.shape[1]
    z64 = dict(dtype=torch.float64, device=q.device)
    out = {"o": torch.zeros((T, hq, d), **z64), "o_tol": torch.zeros((T, hq, d), **z64),
           "lse": torch.zeros((hq, T), **z64), "lse_tol": torch.zeros((hq, T), **z64)}
    for n, h in (("dq", hq), ("dk", hkv), ("dv", hkv)):
        out[n], out[n + "_tol"] = torch.zeros((T, h, d), **z64), torch.zeros((T, h, d), **z64)
    at = 0
    for n in lengths:
        r = slice(at, at + n)
        at += n
        if n == 0:
            continue
        for h in range(hq):
            g = h // (hq // hkv)
            Q, K, V = q[r, h].double(), k[r, g].double(), v[r, g].double()
            z = Q @ K.T * scale
            if causal:
                z = z.masked_fill(torch.ones((n, n), dtype=torch.bool, device=q.device).triu(1),
                                  -math.inf)
            lse = torch.logsumexp(z, 1, keepdim=True)
            p = torch.exp(z - lse)
            o = p @ V
            # scores: d products, the scaling and the shift in float32; exp2 to 2^-21
            gam = (Q.abs() @ K.abs().T * scale).masked_fill(p == 0, 0.0).amax(1, keepdim=True)
            gam = (d + 4) * F32 * gam + 4 * F32 * lse.abs()
            rel = 2 * gam + 2.0 ** -20  # of p (numerator and row sum)
            # P below the type's normal range is off by tiny() of the row's largest (>= 1 / n ...)
            small = tiny(dt) * V.abs().sum(0, keepdim=True)
            apv = p @ V.abs()
            out["o"][r, h] = o
            out["o_tol"][r, h] = (u + n * F32 + rel) * apv + small + u * o.abs() + tiny(dt)
            out["lse"][h, r] = lse[:, 0]
            out["lse_tol"][h, r] = (rel + gam + n * F32)[:, 0] + 4 * F32 * lse[:, 0].abs()
            if do is None:
                continue
            G = do[r, h].double()
            relp = 2 * gam + 2.0 ** -20
            out["dv"][r, g] += p.T @ G
            out["dv_tol"][r, g] += (p * (u + n * F32 + relp)).T @ G.abs() + tiny(dt) * G.abs().sum(
                0, keepdim=True)
            dp = G @ V.T
            D = (G * o).sum(1, keepdim=True)
            # dP and D: d products in float32; D is taken from the rounded, stored o
            edp = (d + 2) * F32 * (G.abs() @ V.abs().T)
            eD = (G.abs() * out["o_tol"][r, h]).sum(1, keepdim=True) + (d + 2) * F32 * (
                G.abs() * o.abs()).sum(1, keepdim=True)
            ds = p * (dp - D) * scale
            eds = (u + relp + 4 * F32) * ds.abs() + p * (edp + eD) * scale
            # fp16: dS is scaled by a power of two before it is rounded, so that the largest
            # bound of |dP - D| over the head is near 2^14: its subnormals are far below
            if dt == torch.float16:
                big = 2 * G.norm(dim=1).amax() * V.norm(dim=1).amax()
                eds = eds + big * scale * 2.0 ** -37
            out["dq"][r, h] = ds @ K
            out["dq_tol"][r, h] = eds @ K.abs() + n * F32 * (ds.abs() @ K.abs())
            out["dk"][r, g] += ds.T @ Q
            out["dk_tol"][r, g] += eds.T @ Q.abs() + n * F32 * (ds.abs().T @ Q.abs())
    for n in ("dq", "dk", "dv"):
        out[n + "_tol"] = 1.01 * out[n + "_tol"] + u * out[n].abs() + tiny(dt)
    return out


def rope(x, gain, positions, inv_freq, sections, interleaved, norm, eps, dy=None):
    """y and (dx, dgain) in float64 of x [T, H, d] with positions [axes, T], and their bounds."""
    dt, u = x.dtype, unit(x.dtype)
    T, H, d = x.shape
    X = x.double()
    half = len(inv_freq)
    axis = [a for a, n in enumerate(sections) for _ in range(n)] if half else []
    ang = torch.stack([positions[axis[i]].double() * inv_freq[i] for i in range(half)], 1) \
        if half else torch.zeros((T, 0), dtype=torch.float64, device=x.device)
    lo = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
    hi = lo + 1 if interleaved else lo + half

    def turn(y, sign):
        y = y.clone()
        c, s = ang.cos()[:, None], sign * ang.sin()[:, None]
        a, b = y[..., lo].clone(), y[..., hi].clone()
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        return y

    def pairs(y):  # sum of magnitudes of a pair, at both of its channels
        y = y.abs().clone()
        m = y[..., lo] + y[..., hi]
        y[..., lo], y[..., hi] = m, m
        return y

    inv = 1.0 / torch.sqrt(X.pow(2).mean(-1, keepdim=True) + eps) if norm else 1.0
    G = gain.double() if gain is not None else torch.ones(d, dtype=torch.float64, device=x.device)
    xh = X * inv
    out = {"y": turn(xh * G, 1.0)}
    # float32: sum of squares (d), root, quotient, products, rotation; angle off by 2^-23 and
    # the reference's own position * frequency product by 2^-53 of the angle
    k = (d + 12) * F32 + 2.0 ** -22 + (float(ang.abs().max()) if half else 0.0) * 2.0 ** -51
    out["y_tol"] = k * pairs(xh * G) + u * out["y"].abs() + tiny(dt)
    if dy is None:
        return out
    g = turn(dy.double(), -1.0)
    eg = k * pairs(dy.double())
    out["dgain"] = (g * xh).sum((0, 1))
    n = T * H
    out["dgain_tol"] = ((eg + k * g.abs()) * xh.abs()).sum((0, 1)) + min(n, 4096) * F32 * (
        g * xh).abs().sum((0, 1))
    if norm:
        gx = g * G
        dot = (gx * xh).mean(-1, keepdim=True)
        out["dx"] = (gx - xh * dot) * inv
        mag = (gx * xh).abs().mean(-1, keepdim=True)
        edot = 2 * k * mag + (eg * G.abs() * xh.abs()).mean(-1, keepdim=True)
        e = eg * G.abs() + 2 * k * gx.abs() + xh.abs() * (edot + 2 * k * dot.abs())
        out["dx_tol"] = e * inv + u * out["dx"].abs() + tiny(dt)
    else:
        out["dx"] = g
        out["dx_tol"] = eg + u * g.abs() + tiny(dt)
    return out


def close(got, ref, name):
    """Fails with the worst element's ratio of error to bound."""
    err = (got.double() - ref[name]).abs()
    bad = ~(err <= ref[name + "_tol"])
    if bool(bad.any()):
        ratio = torch.where(ref[name + "_tol"] > 0, err / ref[name + "_tol"], err * math.inf)
        i = int(torch.nan_to_num(ratio, nan=math.inf).argmax())
        raise AssertionError(
            f"{name}: {int(bad.sum())} of {bad.numel()} values off, worst {float(ratio.flatten()[i])}"
            f" x its bound at {i} (got {float(got.flatten()[i])}, want "
            f"{float(ref[name].flatten()[i])})")
