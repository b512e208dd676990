"""Cases of the node-level operators next to the convolution: the equivariant layer norm, the typed linear map
(one weight per node type, groups of ragged sizes) and the grouping of the nodes by type.

Features are rows [dim], blocks in irreps order, each block [mul][2l+1] with m fastest; fp32 throughout.
A case is a dict: op (norm | linear | group), direction (forward | backward | double_backward), n nodes,
irreps (norm) or irreps_in / irreps_out (linear), types, padded (the share of rows that are padding of a batch
of graphs: zero features, type -1).
"""

import math

import torch

own = False

EPS = 1e-5
MULS = (1, 2, 3, 5, 7, 8, 12, 16, 17, 21, 24, 32, 33, 37, 48, 50, 64, 77, 80, 96, 100, 128)


def listed():
    mace, sweep = "64x0e+64x1o+64x2e", "32x0e+32x1o+32x2e"
    wide = "128x0e+128x1o+128x2e+128x3o"
    return [
        # one small molecule at inference: a layer's norm and its linear map, where the call's latency is all
        dict(name="norm_forward_tiny", op="norm", direction="forward", n=64, irreps="8x0e+8x1o", padded=False),
        dict(name="linear_forward_tiny", op="linear", direction="forward", n=64, irreps_in="8x0e+8x1o",
             irreps_out="8x0e+8x1o", types=4, padded=False),
        # one training step on a 4096-atom cell (the default benchmark's layer)
        dict(name="norm_backward_mace", op="norm", direction="backward", n=4096, irreps=mace, padded=False),
        dict(name="linear_backward_mace", op="linear", direction="backward", n=4096, irreps_in=mace, irreps_out=mace,
             types=10, padded=False),
        # force training (the gradient of a gradient) on a batch of graphs padded to a fixed size, odd multiplicities
        dict(name="norm_double_backward_odd", op="norm", direction="double_backward", n=20011,
             irreps="37x0e+21x1o+5x2e+3x0o", padded=True),
        dict(name="linear_double_backward_odd", op="linear", direction="double_backward", n=3001,
             irreps_in="37x0e+21x1o+5x2e", irreps_out="50x0e+19x1o+7x2e", types=7, padded=True),
        # inference on 8192 atoms, from a wide layer into a narrower one
        dict(name="linear_forward_wide", op="linear", direction="forward", n=8192, irreps_in=wide, irreps_out=sweep,
             types=5, padded=False),
        # a large batch: 262 144 nodes, 0.6 GB a feature tensor
        dict(name="norm_forward_large", op="norm", direction="forward", n=262144, irreps=mace, padded=True),
        dict(name="linear_backward_large", op="linear", direction="backward", n=262144, irreps_in=mace,
             irreps_out=mace, types=16, padded=True),
        # once per graph: the sender graph of one molecule batch, and of the capacity run's 1.2 M atoms
        dict(name="group_small", op="group", direction="forward", n=4096, types=10, padded=False),
        dict(name="group_large", op="group", direction="forward", n=1222309, types=89, padded=True),
    ]


def draw(rng):
    def irreps(most):
        """Up to four blocks l <= 3 with multiplicities of MULS and at most `most` floats a row."""
        ls = [l for l in range(4) if rng.random() < (0.95, 0.75, 0.55, 0.3)[l]] or [rng.randrange(4)]
        out, left = [], most
        for l in ls:
            m = [m for m in MULS if m * (2 * l + 1) <= left]
            if m:
                # equal multiplicities as often as unlike ones
                mul = out[0][0] if out and rng.random() < 0.5 and out[0][0] in m else rng.choice(m)
                out.append((mul, l))
                left -= mul * (2 * l + 1)
        if rng.random() < 0.2 and left >= 8 * (2 * out[-1][1] + 1):
            out.append((8, out[-1][1]))  # a second block of one degree and parity
        return out

    def text(blocks):
        return "+".join("%dx%d%s" % (m, l, "eo"[l % 2]) for m, l in blocks)

    def size(low, high):
        return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))

    op = rng.choice(("norm", "norm", "linear", "linear", "linear", "group"))
    if op == "group":
        return dict(op=op, direction="forward", n=size(1, 1222309), types=size(1, 118), padded=rng.random() < 0.5)
    direction = rng.choice(("forward", "backward", "double_backward"))
    blocks = irreps(2048)
    dim = sum(m * (2 * l + 1) for m, l in blocks)
    if op == "norm":
        n = size(1, min(262144, 50_000_000 // dim))
        return dict(op=op, direction=direction, n=n, irreps=text(blocks), padded=rng.random() < 0.5)
    outs = [(m if rng.random() < 0.5 else rng.choice(MULS), l) for m, l in blocks]
    flops = sum(a * b * (2 * l + 1) for a, l in blocks for b, k in outs if k == l)
    wide = max(dim, sum(m * (2 * l + 1) for m, l in outs))
    n = size(1, min(262144, 50_000_000 // wide, 6_000_000_000 // flops))
    return dict(op=op, direction=direction, n=n, irreps_in=text(blocks), irreps_out=text(outs), types=size(1, 32),
                padded=rng.random() < 0.5)


def blocks_of(irreps):
    """[(offset, multiplicity, l, even)] of an irreps string."""
    out, off = [], 0
    for t in irreps.split("+"):
        mul, ir = t.split("x")
        out.append((off, int(mul), int(ir[:-1]), ir[-1] == "e"))
        off += int(mul) * (2 * int(ir[:-1]) + 1)
    return out


def dim_of(irreps):
    return sum(m * (2 * l + 1) for _, m, l, _ in blocks_of(irreps))


def paths_of(irreps_in, irreps_out):
    """[(in offset, c_in, out offset, c_out, 2l+1, weight offset)]: output block by output block, every input block of
    its degree and parity; a weight block is [c_in][c_out]."""
    out, w = [], 0
    for oo, mo, lo, eo in blocks_of(irreps_out):
        for oi, mi, li, ei in blocks_of(irreps_in):
            if (li, ei) == (lo, eo):
                out.append((oi, mi, oo, mo, 2 * lo + 1, w))
                w += mi * mo
    return out, w


# ---- inputs -------------------------------------------------------------------------------------------------------


def inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n = case["n"]
    real = torch.ones(n, 1, device="cuda")
    if case["padded"]:  # about one row in eight, behind each graph of the batch
        real = (torch.rand(n, 1, generator=g, device="cuda") > 0.125).float()
    s = {}
    if case["op"] in ("linear", "group"):
        share = torch.arange(1, case["types"] + 1, device="cuda").float() ** -0.7  # a few common elements, many rare ones
        t = torch.multinomial(share, n, replacement=True, generator=g).int()
        s["types"] = torch.where(real[:, 0] > 0, t, torch.full_like(t, -1))
        s["n_types"] = case["types"]
    if case["op"] == "group":
        return s
    d_in = dim_of(case["irreps"] if case["op"] == "norm" else case["irreps_in"])
    d_out = d_in if case["op"] == "norm" else dim_of(case["irreps_out"])
    # activations: rows of unlike size, and (norm) scalars off their mean
    s["x"] = rand(n, d_in) * torch.exp(0.5 * rand(n, 1)) * real
    if case["op"] == "norm":
        for o, m, l, e in blocks_of(case["irreps"]):
            if l == 0:
                s["x"][:, o:o + m] += 0.5 * real
        s["weight"] = 1 + 0.1 * rand(sum(m for _, m, _, _ in blocks_of(case["irreps"])))
        s["bias"] = 0.1 * rand(sum(m for _, m, l, e in blocks_of(case["irreps"]) if l == 0 and e))
    else:
        paths, numel = paths_of(case["irreps_in"], case["irreps_out"])
        s["weight"] = rand(case["types"], numel)
        for oi, ci, oo, co, d, w in paths:
            s["weight"][:, w:w + ci * co] /= math.sqrt(ci)
    if case["direction"] != "forward":
        s["g"] = rand(n, d_out) * real
    if case["direction"] == "double_backward":
        s["gg_x"] = rand(n, d_in) * real
        s["gg_weight"] = 0.1 * rand(*s["weight"].shape)
        if case["op"] == "norm":
            s["gg_bias"] = 0.1 * rand(*s["bias"].shape)
    return s


def prepare(case, seed):
    s = inputs(case, seed)
    s["case"] = case
    if case["op"] == "linear":
        # rows of each type, filled up with row n: the index of a batched product over the types
        order = torch.argsort(s["types"].long(), stable=True)
        t = s["types"].long()[order]
        order, t = order[t >= 0], t[t >= 0]
        counts = torch.bincount(t, minlength=case["types"])
        first = torch.cumsum(counts, 0) - counts
        s["rows"] = torch.full((case["types"], max(1, int(counts.max()))), case["n"], dtype=torch.long, device="cuda")
        place = torch.arange(len(t), device="cuda") - first[t]
        s["rows"][t, place] = order
        s["slot"] = torch.full((case["n"],), s["rows"].numel(), dtype=torch.long, device="cuda")
        s["slot"][order] = t * s["rows"].shape[1] + place  # where a node's row is in that product (behind it: no type)
    if own:
        import equivariant_gnn_tensor_receiver_b200 as T
        if case["op"] == "norm":
            s["plan"] = T.NormPlan(case["irreps"], eps=EPS)
        elif case["op"] == "linear":
            s["plan"] = T.LinearPlan(case["irreps_in"], case["irreps_out"], n_types=case["types"])
            s["groups"] = T.NodeGroups(s["types"], case["types"])
    return s


# ---- one pass -----------------------------------------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        return run_own(s, case["op"], case["direction"])
    if case["op"] == "group":
        return plain_group(s["types"], s["n_types"])
    if case["op"] == "norm":
        bl = blocks_of(case["irreps"])
        if case["direction"] == "forward":
            return plain_norm_forward(bl, s["x"], s["weight"], s["bias"])
        if case["direction"] == "backward":
            return plain_norm_backward(bl, s["x"], s["weight"], s["g"])
        return plain_norm_double_backward(bl, s["x"], s["weight"], s["g"], s["gg_x"], s["gg_weight"], s["gg_bias"])
    paths = paths_of(case["irreps_in"], case["irreps_out"])[0]
    x, w, rows, slot = s["x"], s["weight"], s["rows"], s["slot"]
    if case["direction"] == "forward":
        return linear_rows(paths, x, w, rows, slot, dim_of(case["irreps_out"]))
    if case["direction"] == "backward":
        return linear_rows(paths, s["g"], w, rows, slot, x.shape[1], True), linear_weight(paths, x, s["g"], rows, w)
    d_g = linear_rows(paths, s["gg_x"], w, rows, slot, s["g"].shape[1])
    d_g += linear_rows(paths, x, s["gg_weight"], rows, slot, s["g"].shape[1])
    d_x = linear_rows(paths, s["g"], s["gg_weight"], rows, slot, x.shape[1], True)
    return d_g, d_x, linear_weight(paths, s["gg_x"], s["g"], rows, w)


def run_own(s, op, direction):
    import equivariant_gnn_tensor_receiver_b200 as T
    if op == "group":
        groups = T.NodeGroups(s["types"], s["n_types"])
        return groups.perm, groups.offsets
    p = s["plan"]
    if op == "norm":
        if direction == "forward":
            return T.norm_forward(p, s["x"], s["weight"], s["bias"])
        if direction == "backward":
            r = T.norm_backward(p, s["x"], s["weight"], s["g"])
            return r["dx"], r["dweight"], r["dbias"]
        r = T.norm_double_backward(p, s["x"], s["weight"], s["g"], s["gg_x"], s["gg_weight"], s["gg_bias"])
        return r["d_g"], r["d_x"], r["d_weight"]
    if direction == "forward":
        return T.linear_forward(p, s["groups"], s["x"], s["weight"])
    if direction == "backward":
        r = T.linear_backward(p, s["groups"], s["x"], s["weight"], s["g"])
        return r["dx"], r["dweight"]
    r = T.linear_double_backward(p, s["groups"], s["x"], s["weight"], s["g"], s["gg_x"], s["gg_weight"])
    return r["d_g"], r["d_x"], r["d_weight"]


# ---- plain forms: elementary torch operations in fp32 -------------------------------------------------------------


def plain_group(types, n_types):
    """Nodes in the order of their type, in ascending order inside one (type -1, padding, behind all), and where each
    type begins."""
    key = torch.where(types < 0, torch.full_like(types, n_types), types)
    key, perm = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(n_types + 1, dtype=key.dtype, device=key.device))
    return perm.int(), offsets.int()


def normalised(x, o, m, l):
    """(centred and normalised block [n, m, 2l+1], 1 / its root mean square [n, 1, 1])."""
    c = x[:, o:o + m * (2 * l + 1)].reshape(-1, m, 2 * l + 1)
    if l == 0:
        c = c - c.mean((1, 2), keepdim=True)
    r = (c.square().mean((1, 2), keepdim=True) + EPS).rsqrt()
    return c * r, r


def plain_norm_forward(bl, x, weight, bias):
    out, iw, ib = [], 0, 0
    for o, m, l, even in bl:
        y = normalised(x, o, m, l)[0] * weight[iw:iw + m, None]
        iw += m
        if l == 0 and even:
            y = y + bias[ib:ib + m, None]
            ib += m
        out.append(y.flatten(1))
    return torch.cat(out, 1)


def plain_norm_backward(bl, x, weight, g):
    dx, dw, db, iw = [], [], [torch.empty(0, device=x.device)], 0
    for o, m, l, even in bl:
        h, r = normalised(x, o, m, l)
        gb = g[:, o:o + m * (2 * l + 1)].reshape_as(h)
        gh = gb * weight[iw:iw + m, None]
        iw += m
        d = r * (gh - h * (gh * h).mean((1, 2), keepdim=True))
        if l == 0:
            d = d - d.mean((1, 2), keepdim=True)
            if even:
                db.append(gb.sum((0, 2)))
        dx.append(d.flatten(1))
        dw.append((gb * h).sum((0, 2)))
    return torch.cat(dx, 1), torch.cat(dw), torch.cat(db)


def plain_norm_double_backward(bl, x, weight, g, gg_x, gg_weight, gg_bias):
    mean = lambda t: t.mean((1, 2), keepdim=True)  # noqa: E731
    d_g, d_x, d_w, iw, ib = [], [], [], 0, 0
    for o, m, l, even in bl:
        h, r = normalised(x, o, m, l)
        gb = g[:, o:o + m * (2 * l + 1)].reshape_as(h)
        a = gg_x[:, o:o + m * (2 * l + 1)].reshape_as(h)
        w, al = weight[iw:iw + m, None], gg_weight[iw:iw + m, None]
        iw += m
        if l == 0:
            a = a - mean(a)
        gh, ag = gb * w, gb * al
        a1, a2, g2, k = mean(a * gh), mean(a * h), mean(gh * h), mean(ag * h)
        t = r * (a - h * a2)
        y = w * t + al * h
        if l == 0 and even:
            y = y + gg_bias[ib:ib + m, None]
            ib += m
        v = r * ag - r * r * (gh * a2 + a * g2) - h * (r * r * (a1 - 3 * g2 * a2) + r * k)
        if l == 0:
            v = v - mean(v)
        d_g.append(y.flatten(1))
        d_x.append(v.flatten(1))
        d_w.append((gb * t).sum((0, 2)))
    return torch.cat(d_g, 1), torch.cat(d_x, 1), torch.cat(d_w)


def linear_rows(paths, x, weight, rows, slot, dim, transposed=False):
    """Block by block, the rows of every type times its weight (or that transposed); rows of no type are zero."""
    x = torch.cat((x, x.new_zeros(1, x.shape[1])))
    out = x.new_zeros(slot.shape[0], dim)
    for oi, ci, oo, co, d, w in paths:
        b = weight[:, w:w + ci * co].view(-1, ci, co)
        if transposed:
            oi, ci, oo, co, b = oo, co, oi, ci, b.transpose(1, 2)
        a = x[:, oi:oi + ci * d].reshape(-1, ci, d).transpose(1, 2)[rows]  # [type, row, m, c_in]
        y = torch.bmm(a.flatten(1, 2), b).view(*rows.shape, d, co).transpose(2, 3)
        y = y.reshape(-1, co * d)
        out[:, oo:oo + co * d] += torch.cat((y, y.new_zeros(1, co * d)))[slot]
    return out


def linear_weight(paths, x, g, rows, weight):
    x, g = torch.cat((x, x.new_zeros(1, x.shape[1]))), torch.cat((g, g.new_zeros(1, g.shape[1])))
    out = torch.zeros_like(weight)
    for oi, ci, oo, co, d, w in paths:
        a = x[:, oi:oi + ci * d].reshape(-1, ci, d).transpose(1, 2)[rows].flatten(1, 2)
        b = g[:, oo:oo + co * d].reshape(-1, co, d).transpose(1, 2)[rows].flatten(1, 2)
        out[:, w:w + ci * co] = torch.bmm(a.transpose(1, 2), b).flatten(1)
    return out


# ---- what a pass cannot do without ----------------------------------------------------------------------------------


def work(case):
    n = case["n"]
    if case["op"] == "group":
        return {"bytes": 8 * n + 4 * (case["types"] + 1), "flops": 0}
    k = ("forward", "backward", "double_backward").index(case["direction"])
    if case["op"] == "norm":
        dim, nw = dim_of(case["irreps"]), sum(m for _, m, _, _ in blocks_of(case["irreps"]))
        # forward x -> y; backward x, g -> dx; double backward x, g, gg_x -> d_g, d_x
        return {"bytes": 4 * ((2, 3, 5)[k] * n * dim + (2, 3, 3)[k] * nw), "flops": (8, 14, 40)[k] * n * dim}
    paths, numel = paths_of(case["irreps_in"], case["irreps_out"])
    a, b, w = n * dim_of(case["irreps_in"]), n * dim_of(case["irreps_out"]), case["types"] * numel
    mults = n * sum(ci * co * d for _, ci, _, co, d, _ in paths)
    # forward x -> out; backward x, g -> dx, dw; double backward x, gg_x, g -> d_g, d_x, d_w
    return {"bytes": 4 * ((a + b + w, 2 * a + b + 2 * w, 3 * a + 2 * b + 3 * w)[k] + n),
            "flops": 2 * mults * (1, 2, 4)[k]}


# ---- the same from the definitions, in 64 bits ------------------------------------------------------------------------


def exact(case, seed):
    s = inputs(case, seed)
    if case["op"] == "group":
        return None
    f = {k: v.double().requires_grad_(k in ("x", "weight", "bias", "g"))
         for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    x, w = f["x"], f["weight"]
    if case["op"] == "norm":
        parts, iw, ib = [], 0, 0
        for o, m, l, even in blocks_of(case["irreps"]):
            c = x[:, o:o + m * (2 * l + 1)]
            if l == 0:
                c = c - c.sum(1, keepdim=True) / m
            c = c / torch.sqrt((c * c).sum(1, keepdim=True) / c.shape[1] + EPS)
            c = c * w[iw:iw + m].repeat_interleave(2 * l + 1)
            iw += m
            if l == 0 and even:
                c = c + f["bias"][ib:ib + m]
                ib += m
            parts.append(c)
        out = torch.cat(parts, 1)
    else:
        out = x.new_zeros(case["n"], dim_of(case["irreps_out"]))
        for t in range(case["types"]):
            r = torch.nonzero(s["types"] == t)[:, 0]
            if not len(r):
                continue
            y = x.new_zeros(len(r), out.shape[1])
            for oi, ci, oo, co, d, o in paths_of(case["irreps_in"], case["irreps_out"])[0]:
                p = torch.einsum("num,uw->nwm", x[r, oi:oi + ci * d].view(-1, ci, d), w[t, o:o + ci * co].view(ci, co))
                y = y + torch.nn.functional.pad(p.flatten(1), (oo, out.shape[1] - oo - co * d))
            out = out.index_add(0, r, y)
    if case["direction"] == "forward":
        return out.detach()
    # the gradients by automatic differentiation of the definition
    names = [k for k in ("x", "weight", "bias") if k in f]
    twice = case["direction"] == "double_backward"
    keep = [f[k] for k in names]
    first = torch.autograd.grad(out, keep, f["g"], create_graph=twice, materialize_grads=True)
    if not twice:
        return tuple(first)
    psi = sum((d * f["gg_" + k]).sum() for d, k in zip(first, names))
    second = torch.autograd.grad(psi, [f["g"], f["x"], f["weight"]], materialize_grads=True)
    return tuple(second)
