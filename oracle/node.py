"""fp64 numpy oracle of the node operators: nodes grouped by type, typed linear map, layer norm of irreps
features, each with its first- and second-order gradients written out per block.

Conventions as for the convolution: rows [dim], blocks in irreps order, [mul][2l+1] with m fastest."""

from __future__ import annotations

import numpy as np

from . import irreps as I


def blocks(s):
    """[(offset, mul, 2l+1, l, parity)]"""
    out, off = [], 0
    for b in I.parse(s):
        out.append((off, b.mul, 2 * b.l + 1, b.l, b.p))
        off += b.dim
    return out, off


# ---- grouping ----------------------------------------------------------------------------------------


def group(types, n_types):
    key = np.where((types >= 0) & (types < n_types), types, n_types)
    perm = np.argsort(key, kind="stable")
    return perm, np.array([np.count_nonzero(key < t) for t in range(n_types + 1)])


# ---- typed linear map ----------------------------------------------------------------------------------


def linear_paths(irreps_in, irreps_out):
    """([(in block, out block, weight offset)], weights of a type), output block by output block"""
    bi, bo = blocks(irreps_in)[0], blocks(irreps_out)[0]
    out, w = [], 0
    for o in bo:
        for i in bi:
            if i[3:] == o[3:]:
                out.append((i, o, w))
                w += i[1] * o[1]
    return out, w


def linear(irreps_in, irreps_out, types, x, w):
    """out[n, i3, w, m] = sum_p sum_u W[type n][p][u][w] x[n, i1, u, m]; rows of no type are zero"""
    paths, _ = linear_paths(irreps_in, irreps_out)
    out = np.zeros((len(x), blocks(irreps_out)[1]))
    for t in range(len(w)):
        r = np.flatnonzero(types == t)
        for (oi, ci, d, _, _), (oo, co, _, _, _), k in paths:
            a = x[r, oi:oi + ci * d].reshape(-1, ci, d)
            out[r, oo:oo + co * d] += np.einsum("num,uw->nwm", a, w[t, k:k + ci * co].reshape(ci, co)).reshape(-1, co * d)
    return out


def linear_backward(irreps_in, irreps_out, types, x, w, g):
    paths, _ = linear_paths(irreps_in, irreps_out)
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    for t in range(len(w)):
        r = np.flatnonzero(types == t)
        for (oi, ci, d, _, _), (oo, co, _, _, _), k in paths:
            a = x[r, oi:oi + ci * d].reshape(-1, ci, d)
            b = g[r, oo:oo + co * d].reshape(-1, co, d)
            m = w[t, k:k + ci * co].reshape(ci, co)
            dx[r, oi:oi + ci * d] += np.einsum("nwm,uw->num", b, m).reshape(-1, ci * d)
            dw[t, k:k + ci * co] = np.einsum("num,nwm->uw", a, b).ravel()
    return dx, dw


def linear_double_backward(irreps_in, irreps_out, types, x, w, g, gg_x, gg_w):
    """(d_g, d_x, d_w) of <gg_x, dx> + <gg_w, dw>"""
    d_g = linear(irreps_in, irreps_out, types, gg_x, w) + linear(irreps_in, irreps_out, types, x, gg_w)
    d_x = linear_backward(irreps_in, irreps_out, types, x, gg_w, g)[0]
    d_w = linear_backward(irreps_in, irreps_out, types, gg_x, w, g)[1]
    return d_g, d_x, d_w


# ---- layer norm ------------------------------------------------------------------------------------------


def _norm_blocks(irreps, x, eps, w, b):
    """per block: slice, shape, h, r, channel weights [mul, 1], weight slice, bias slice or None, centring"""
    bl, _ = blocks(irreps)
    iw = ib = 0
    for o, mul, d, l, p in bl:
        s = slice(o, o + mul * d)
        c = x[:, s].reshape(-1, mul, d)
        pr = (lambda t: t - t.mean((1, 2), keepdims=True)) if l == 0 else (lambda t: t)
        c = pr(c)
        r = ((c * c).mean((1, 2), keepdims=True) + eps) ** -0.5
        bs = None
        if l == 0 and p == 1:
            bs = slice(ib, ib + mul)
            ib += mul
        ws = slice(iw, iw + mul)
        iw += mul
        yield s, (mul, d), c * r, r, ws, bs, pr


def norm_sizes(irreps):
    bl, _ = blocks(irreps)
    return sum(b[1] for b in bl), sum(b[1] for b in bl if b[3] == 0 and b[4] == 1)


def norm(irreps, x, w, b, eps):
    y = np.empty_like(x)
    for s, _, h, _, ws, bs, _ in _norm_blocks(irreps, x, eps, w, b):
        v = h * w[ws][:, None]
        if bs is not None:
            v = v + b[bs][:, None]
        y[:, s] = v.reshape(len(x), s.stop - s.start)
    return y


def norm_backward(irreps, x, w, g, eps):
    nw, nb = norm_sizes(irreps)
    dx, dw, db = np.empty_like(x), np.zeros(nw), np.zeros(nb)
    mean = lambda t: t.mean((1, 2), keepdims=True)  # noqa: E731
    for s, (mul, d), h, r, ws, bs, pr in _norm_blocks(irreps, x, eps, w, None):
        gb = g[:, s].reshape(-1, mul, d)
        gh = gb * w[ws][:, None]
        dx[:, s] = pr(r * (gh - h * mean(gh * h))).reshape(len(x), s.stop - s.start)
        dw[ws] = (gb * h).sum((0, 2))
        if bs is not None:
            db[bs] = gb.sum((0, 2))
    return dx, dw, db


def norm_double_backward(irreps, x, w, g, gg_x, gg_w, gg_b, eps):
    """(d_g, d_x, d_w) of <gg_x, dx> + <gg_w, dw> + <gg_b, db>"""
    d_g, d_x, d_w = np.empty_like(x), np.empty_like(x), np.zeros(len(w))
    mean = lambda t: t.mean((1, 2), keepdims=True)  # noqa: E731
    for s, (mul, d), h, r, ws, bs, pr in _norm_blocks(irreps, x, eps, w, None):
        gb = g[:, s].reshape(-1, mul, d)
        a = pr(gg_x[:, s].reshape(-1, mul, d))
        wc, al = w[ws][:, None], gg_w[ws][:, None]
        gh, ag = gb * wc, gb * al
        a1, a2, g2, k = mean(a * gh), mean(a * h), mean(gh * h), mean(ag * h)
        t = r * (a - h * a2)
        y = wc * t + al * h
        if bs is not None:
            y = y + gg_b[bs][:, None]
        v = pr(r * ag - r * r * (gh * a2 + a * g2) - h * (r * r * (a1 - 3 * g2 * a2) + r * k))
        d_g[:, s], d_x[:, s] = y.reshape(len(x), s.stop - s.start), v.reshape(len(x), s.stop - s.start)
        d_w[ws] = (gb * t).sum((0, 2))
    return d_g, d_x, d_w
