"""Plain 64-bit forms of the operators around the gated delta rule (gated scan, short convolution, RMS norm)
and of their gradients, on the CPU, and how far a 32-bit computation of each may be from them.

Test infrastructure only. Every function takes the tensors the kernels take and upcasts them exactly. The
second value of a pair is an absolute bound, element by element, on the error of a computation in 32 bits
before its result is rounded to the output's type; U is half a step of fp32."""
from __future__ import annotations

import torch

U = 2.0 ** -24


def f64(t):
    return None if t is None else t.detach().cpu().double()


def sequences(B, T, cu=None):
    """[(first token, one behind the last token)] over the flattened token axis."""
    if cu is None:
        return [(b * T, (b + 1) * T) for b in range(B)]
    c = [min(max(int(v), 0), B * T) for v in cu]
    return list(zip(c[:-1], c[1:]))


# ---- gated scan ---------------------------------------------------------------------------------


def scan_fwd(x, g, s0, cu=None):
    """(h, final state), each with its bound. A step multiplies by exp(g) (off by 2 + |g| half steps) and adds
    (one more), so errors run through the same recurrence as the values: e_t = a e_{t-1} + k U |h|_t with |h|
    the recurrence on absolute values."""
    B, T, D = x.shape
    x, g = f64(x).reshape(-1, D), f64(g).reshape(-1, D)
    seqs = sequences(B, T, cu)
    h, e = torch.zeros_like(x), torch.zeros_like(x)
    fin = torch.zeros(len(seqs), D, dtype=torch.float64)
    fe = torch.zeros_like(fin)
    for n, (p, q) in enumerate(seqs):
        c = torch.zeros(D, dtype=torch.float64) if s0 is None else f64(s0)[n].clone()
        m, err = c.abs(), torch.zeros_like(c)
        for t in range(p, q):
            a = torch.exp(g[t])
            k = 4 + g[t].abs().clamp(max=100)
            m = a * m + x[t].abs()
            err = a * err + k * U * m
            c = a * c + x[t]
            h[t], e[t] = c, err
        fin[n], fe[n] = c, err
    return (h.reshape(B, T, D), e.reshape(B, T, D)), (fin, fe)


def scan_bwd(x, g, s0, d_h, d_fin, cu=None):
    """dict of (value, bound) for dx, dg, d_initial_state."""
    B, T, D = x.shape
    (h, e), _ = scan_fwd(x, g, s0, cu)
    h, e = h.reshape(-1, D), e.reshape(-1, D)
    g, d_h = f64(g).reshape(-1, D), f64(d_h).reshape(-1, D)
    seqs = sequences(B, T, cu)
    dx, dg, ex, eg = (torch.zeros_like(h) for _ in range(4))
    d0 = torch.zeros(len(seqs), D, dtype=torch.float64)
    e0 = torch.zeros_like(d0)
    for n, (p, q) in enumerate(seqs):
        mu = torch.zeros(D, dtype=torch.float64) if d_fin is None else f64(d_fin)[n].clone()
        m, err = mu.abs(), torch.zeros_like(mu)
        for t in range(q - 1, p - 1, -1):
            a = torch.exp(g[t])
            k = 4 + g[t].abs().clamp(max=100)
            lam, m = d_h[t] + mu, d_h[t].abs() + m
            dx[t], ex[t] = lam, err + U * m
            mu, m = a * lam, a * m
            err = a * err + k * U * m
            before = h[t - 1] if t > p else (torch.zeros_like(mu) if s0 is None else f64(s0)[n])
            eb = e[t - 1] if t > p else 0.0
            dg[t] = mu * before
            eg[t] = err * before.abs() + mu.abs() * eb + err * eb + U * dg[t].abs()
        d0[n], e0[n] = mu, err
    return dict(dx=(dx.reshape(B, T, D), ex.reshape(B, T, D)), dg=(dg.reshape(B, T, D), eg.reshape(B, T, D)),
                d_initial_state=(d0, e0))


# ---- short convolution --------------------------------------------------------------------------


def _inputs(x, s0, n, p, q, W):
    head = torch.zeros(W - 1, x.shape[1], dtype=torch.float64) if s0 is None else f64(s0)[n]
    return torch.cat([head, x[p:q]])


def conv_fwd(x, w, b, s0, silu, cu=None):
    """((y, bound), final state). z sums W + 1 products in any order; silu's slope is at most 1.1, and its
    own evaluation (exp, sum, quotient) is off by at most 8 + |z| half steps."""
    B, T, D = x.shape
    x, w = f64(x).reshape(-1, D), f64(w)
    W = w.shape[1]
    seqs = sequences(B, T, cu)
    y, e = torch.zeros_like(x), torch.zeros_like(x)
    fin = torch.zeros(len(seqs), W - 1, D, dtype=torch.float64)
    for n, (p, q) in enumerate(seqs):
        q = max(p, q)
        ext = _inputs(x, s0, n, p, q, W)
        L = q - p
        z = torch.zeros(L, D, dtype=torch.float64) + (0 if b is None else f64(b))
        mag = z.abs()
        for j in range(W):
            z = z + ext[j:j + L] * w[:, j]
            mag = mag + (ext[j:j + L] * w[:, j]).abs()
        ez = (W + 1) * U * mag
        if silu:
            y[p:q] = z * torch.sigmoid(z)
            e[p:q] = 1.1 * ez + (8 + z.abs().clamp(max=100)) * U * y[p:q].abs()
        else:
            y[p:q], e[p:q] = z, ez
        fin[n] = ext[L:]
    return (y.reshape(B, T, D), e.reshape(B, T, D)), fin


def conv_bwd(x, w, b, s0, d_y, d_fin, silu, cu=None):
    """dict of (value, bound) for dx, dweight, dbias, d_initial_state. A sum of n terms in any order is off by
    at most n half steps of the sum of absolute values."""
    B, T, D = x.shape
    x, w, d_y = f64(x).reshape(-1, D), f64(w), f64(d_y).reshape(-1, D)
    W = w.shape[1]
    seqs = sequences(B, T, cu)
    dx, ex = torch.zeros_like(x), torch.zeros_like(x)
    d0 = torch.zeros(len(seqs), W - 1, D, dtype=torch.float64)
    e0 = torch.zeros_like(d0)
    dw, aw, ew = torch.zeros_like(w), torch.zeros_like(w), torch.zeros_like(w)
    db, ab, eb = (torch.zeros(D, dtype=torch.float64) for _ in range(3))
    count = 0
    for n, (p, q) in enumerate(seqs):
        q = max(p, q)
        ext = _inputs(x, s0, n, p, q, W)
        L = q - p
        count += L
        z = torch.zeros(L, D, dtype=torch.float64) + (0 if b is None else f64(b))
        mag = z.abs()
        for j in range(W):
            z = z + ext[j:j + L] * w[:, j]
            mag = mag + (ext[j:j + L] * w[:, j]).abs()
        dz = d_y[p:q].clone()
        edz = torch.zeros_like(dz)
        if silu:
            s = torch.sigmoid(z)
            dz = dz * s * (1 + z * (1 - s))
            # |silu''| <= 0.5; its slope is at most 1.1 and formed of factors off by 8 + |z| half steps each
            edz = d_y[p:q].abs() * (0.5 * (W + 1) * U * mag + (20 + 2 * z.abs().clamp(max=100)) * U * (0.1 + s * (1 + z.abs() * (1 - s))))
        de, ee = torch.zeros_like(ext), torch.zeros_like(ext)
        ma = torch.zeros_like(ext)
        if d_fin is not None:
            de[L:] += f64(d_fin)[n]
            ma[L:] += f64(d_fin)[n].abs()
        for j in range(W):
            de[j:j + L] += dz * w[:, j]
            ma[j:j + L] += (dz * w[:, j]).abs()
            ee[j:j + L] += edz * w[:, j].abs()
            dw[:, j] += (dz * ext[j:j + L]).sum(0)
            aw[:, j] += (dz * ext[j:j + L]).abs().sum(0)
            ew[:, j] += (edz * ext[j:j + L].abs()).sum(0)
        ee += (W + 1) * U * ma
        db += dz.sum(0)
        ab += dz.abs().sum(0)
        eb += edz.sum(0)
        d0[n], e0[n] = de[:W - 1], ee[:W - 1]
        dx[p:q], ex[p:q] = de[W - 1:], ee[W - 1:]
    return dict(dx=(dx.reshape(B, T, D), ex.reshape(B, T, D)), dweight=(dw, ew + (count + 1) * U * aw),
                dbias=(db, eb + (count + 1) * U * ab), d_initial_state=(d0, e0))


# ---- RMS norm -----------------------------------------------------------------------------------

# The mean of squares is a sum of positive terms: rows of up to 16384 values, at most 64 a thread and then a tree
# over threads, are off by at most 64 + 10 half steps of it, and its inverse root by half of that and 4 more.
RSTD = (74 / 2 + 4) * U


def rms_fwd(x, res, w, eps):
    """(y, its bound, r in the input's type)."""
    r = x.detach().cpu()
    if res is not None:
        r = (r.float() + res.detach().cpu().float()).to(x.dtype)
    v = r.double()
    y = v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps) * f64(w)
    return y, y.abs() * (RSTD + 3 * U), r


def rms_bwd(r, w, d_y, d_res, eps):
    """dict of (value, bound) for dx, dweight."""
    r, w, dy = f64(r), f64(w), f64(d_y)
    D = r.shape[-1]
    r, dy = r.reshape(-1, D), dy.reshape(-1, D)
    rstd = 1 / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    rh, u = r * rstd, dy * w
    mean, amean = (u * rh).mean(-1, keepdim=True), (u * rh).abs().mean(-1, keepdim=True)
    dx = rstd * (u - rh * mean)
    # the mean's sum is off by 74 half steps of the absolute sum, its factors by 2 RSTD and 4 more
    e = rstd * (u.abs() * (RSTD + 4 * U) + rh.abs() * (amean * (74 * U + 3 * RSTD + 6 * U)))
    if d_res is not None:
        dr = f64(d_res).reshape(-1, D)
        dx = dx + dr
        e = e + U * dx.abs()
    n = r.shape[0]
    dw, aw = (dy * rh).sum(0), (dy * rh).abs().sum(0)
    return dict(dx=(dx.reshape(f64(d_y).shape), e.reshape(f64(d_y).shape)), dweight=(dw, aw * (RSTD + (n + 3) * U)))
