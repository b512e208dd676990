"""Node operators on the device against the fp64 oracle (inputs rounded to fp32 first).

Tolerances, fixed before the first run.  Row outputs (y, dx, d_g, d_x, out): 1e-5 of the tensor's largest
value, the library's bar for its fp32 path: an element collects at most some 150 roundings of 2^-24
(statistics over at most 20 terms a lane plus a tree, 20 more elementwise; sums over at most 512 channels
enter through trees or fp32 chains whose errors add at random).  Sums over rows (dweight, dbias, d_weight):
element by element, 96 * 2^-24 times the sum of the terms' magnitudes: no element's additions form a chain of
more than 64 per lane here, the terms carry up to 30 roundings of their own (3xTF32 products 2^-22 each).
TF32 mode: 5e-3 as elsewhere in the library.  The scalars of a block with a variance far under eps are
divided by sqrt(eps), which no tolerance here has to cover: the inputs avoid cancellation in the mean."""

import numpy as np
import pytest

from oracle import node as O

pytestmark = pytest.mark.gpu

TOL = 1e-5
SUM = 96 * 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module")
def T():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import equivariant_gnn_tensor_receiver_b200 as T
    T.lib()
    return T


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def f32(a):
    return a.astype(np.float32).astype(np.float64)


def dev(a, dtype=None, shift=0):
    """on the device; shift > 0: at that many floats behind a 256-byte boundary"""
    import torch
    t = torch.as_tensor(np.ascontiguousarray(a)).to(dtype or torch.float32)
    buf = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
    v = buf[shift:].view(t.shape)
    v.copy_(t)
    return v


def host(t):
    return t.detach().double().cpu().numpy()


def rows_close(got, want, tol=TOL):
    got = host(got)
    assert got.shape == want.shape
    if want.size:
        assert np.abs(got - want).max() <= tol * max(np.abs(want).max(), 1e-30)


def sums_close(got, want, mags, k=SUM):
    got = host(got)
    assert got.shape == want.shape
    assert (np.abs(got - want) <= k * mags + 1e-30).all()


# ---- grouping ----------------------------------------------------------------------------------------


@pytest.mark.parametrize("n,n_types", [(0, 3), (1, 1), (31, 2), (64, 4), (1000, 256), (8192, 10), (8193, 7),
                                       (50_001, 89), (300_000, 1), (2_500_000, 256)])
def test_group_nodes(T, n, n_types):
    import torch
    t = rng(n).integers(-2, n_types + 2, size=n)
    for dtype in (torch.int32, torch.int64):
        G = T.NodeGroups(dev(t, dtype), n_types)
        key = np.where((t >= 0) & (t < n_types), t, n_types)
        assert np.array_equal(G.perm.cpu().numpy(), np.argsort(key, kind="stable"))
        assert np.array_equal(G.offsets.cpu().numpy(), np.searchsorted(np.sort(key), np.arange(n_types + 1)))


def test_group_far_types_are_no_types(T):
    import torch
    t = np.array([0, 2 ** 32, -2 ** 31, 2 ** 31 - 1, 1, 2 ** 40 + 1])
    G = T.NodeGroups(dev(t, torch.int64), 2)
    assert G.perm.cpu().tolist() == [0, 4, 1, 2, 3, 5] and G.offsets.cpu().tolist() == [0, 1, 2]


# ---- layer norm ----------------------------------------------------------------------------------------

NORMS = [("8x0e+8x1o", 64), ("64x0e+64x1o+64x2e", 700), ("37x0e+21x1o+5x2e+3x0o", 333), ("1x0e", 5), ("1x3o", 9),
         ("3x0o+2x0e+5x3o+1x0e", 40), ("128x0e+128x1o+128x2e+128x3o", 50), ("4096x0e", 17), ("2563x0e+100x1o", 6),
         ("10240x0e", 3), ("9000x0e+7x1e", 2), ("16x0e", 1), ("128x0e", 12345), ("+".join(["4x0e"] * 12), 100),
         ("300x1o", 70), ("33x1o+33x1e", 1), ("640x0e", 129), ("2560x0e", 30), ("64x0e+64x1o+64x2e", 0)]


def norm_inputs(irreps, n, seed):
    r = rng(seed)
    dim = O.blocks(irreps)[1]
    nw, nb = O.norm_sizes(irreps)
    x = r.normal(size=(n, dim)) * np.exp(0.5 * r.normal(size=(n, 1))) + 0.3
    if n > 3:
        x[2] = 0  # a padding row
    d = dict(x=x, g=r.normal(size=(n, dim)), a=r.normal(size=(n, dim)), w=1 + 0.3 * r.normal(size=nw),
             b=r.normal(size=nb), al=r.normal(size=nw), be=r.normal(size=nb))
    if n > 3:
        d["g"][2] = d["a"][2] = 0
    return {k: f32(v) for k, v in d.items()}


def norm_check(T, irreps, n, shift=0):
    import torch
    d = norm_inputs(irreps, n, 7 + n)
    t = {k: dev(v, shift=shift) for k, v in d.items()}
    p = T.NormPlan(irreps, eps=EPS)
    eps = float(np.float32(EPS))
    rows_close(T.norm_forward(p, t["x"], t["w"], t["b"]), O.norm(irreps, d["x"], d["w"], d["b"], eps))
    one, zero = np.ones_like(d["w"]), np.zeros_like(d["b"])
    rows_close(T.norm_forward(p, t["x"]), O.norm(irreps, d["x"], one, zero, eps))
    r = T.norm_backward(p, t["x"], t["w"], t["g"])
    dx, dw, db = O.norm_backward(irreps, d["x"], d["w"], d["g"], eps)
    # magnitudes of the sums' terms: |g h| and |g|
    mags = O.norm_backward(irreps, d["x"], d["w"], d["g"], eps)
    h = O.norm(irreps, d["x"], one, zero, eps)
    mag = lambda q: np.concatenate([np.abs(q[:, o:o + m * k].reshape(-1, m, k)).sum((0, 2))  # noqa: E731
                                    for o, m, k, _, _ in O.blocks(irreps)[0]])
    rows_close(r["dx"], dx)
    # the error of h itself (up to 40 roundings of the block's largest h) multiplies |g|
    hmax = np.abs(h).max() if h.size else 0
    sums_close(r["dweight"], dw, mag(d["g"] * h) + hmax * mag(d["g"]))
    bl = O.blocks(irreps)[0]
    b0 = [np.abs(d["g"][:, o:o + m]).sum(0) for o, m, _, l, par in bl if l == 0 and par == 1]
    sums_close(r["dbias"], db, np.concatenate(b0) if b0 else np.zeros(0))
    r = T.norm_double_backward(p, t["x"], t["w"], t["g"], t["a"], t["al"], t["be"])
    d_g, d_x, d_w = O.norm_double_backward(irreps, d["x"], d["w"], d["g"], d["a"], d["al"], d["be"], eps)
    rows_close(r["d_g"], d_g)
    rows_close(r["d_x"], d_x, 2e-5 if O.blocks(irreps)[1] < 32 else TOL)
    # d_w = sum g t; t's error is relative to its own largest value
    tt = O.norm_double_backward(irreps, d["x"], one, d["g"], d["a"], 0 * one, zero, eps)[0]
    sums_close(r["d_weight"], d_w, mag(d["g"] * tt) + (np.abs(tt).max() if tt.size else 0) * mag(d["g"]))
    # cotangents None = zero, outputs left out
    r2 = T.norm_double_backward(p, t["x"], t["w"], t["g"], gg_x=t["a"], want=("d_g",))
    assert list(r2) == ["d_g"]
    rows_close(r2["d_g"], O.norm_double_backward(irreps, d["x"], d["w"], d["g"], d["a"], 0 * one, zero, eps)[0])
    r3 = T.norm_double_backward(p, t["x"], None, t["g"], gg_weight=t["al"])
    w3 = O.norm_double_backward(irreps, d["x"], one, d["g"], 0 * d["a"], d["al"], zero, eps)
    rows_close(r3["d_g"], w3[0])
    assert not r3["d_weight"].any()
    r4 = T.norm_backward(p, t["x"], None, t["g"], want=("dweight",))
    assert torch.equal(r4["dweight"], T.norm_backward(p, t["x"], t["w"], t["g"])["dweight"])


@pytest.mark.parametrize("irreps,n", NORMS)
def test_norm(T, irreps, n):
    norm_check(T, irreps, n)


@pytest.mark.parametrize("irreps,n", [("8x0e+8x1o", 70), ("64x0e+64x1o", 33), ("640x0e", 9), ("2560x0e", 5)])
def test_norm_of_tensors_off_16_bytes(T, irreps, n):
    norm_check(T, irreps, n, shift=1)


def test_norm_rows_are_independent_and_repeatable(T):
    """NaN and infinity stay in their row; repeated calls agree bit for bit; nothing else moves"""
    import torch
    irreps = "64x0e+64x1o+64x2e"
    d = norm_inputs(irreps, 300, 1)
    p = T.NormPlan(irreps)
    x, g, w = dev(d["x"]), dev(d["g"]), dev(d["w"])
    clean = T.norm_forward(p, x, w)
    bad = x.clone()
    bad[7, 3] = float("nan")
    bad[9, 100] = float("inf")
    y = T.norm_forward(p, bad, w)
    keep = [i for i in range(300) if i not in (7, 9)]
    assert torch.equal(y[keep], clean[keep]) and y[7, :64].isnan().all() and torch.equal(y[7, 64:], clean[7, 64:])
    a, b = T.norm_backward(p, x, w, g), T.norm_backward(p, x, w, g)
    assert all(torch.equal(a[k], b[k]) for k in a)


# ---- typed linear map -----------------------------------------------------------------------------------

LINEARS = [
    ("8x0e+8x1o", "8x0e+8x1o", 64, 4), ("64x0e+64x1o+64x2e", "64x0e+64x1o+64x2e", 700, 10),
    ("37x0e+21x1o+5x2e", "50x0e+19x1o+7x2e", 301, 7), ("1x0e", "1x0e", 3, 1), ("5x0e+4x0e+3x1o", "4x0e+2x1o+6x0e", 90, 3),
    ("128x0e+128x1o+128x2e+128x3o", "32x0e+32x1o+32x2e", 400, 5), ("4x1o", "4x1e", 20, 2), ("8x0e", "8x0e+4x2e", 50, 3),
    ("16x3o+12x2e", "20x3o+8x2e", 77, 256), ("64x0e", "64x0e", 3000, 2), ("260x0e+100x1o", "130x0e+260x1o", 150, 3),
    ("32x0e+16x1o", "32x0e+16x1o", 0, 3), ("64x1o", "64x1o", 1, 5), ("96x0e+64x0e", "72x0e", 333, 4),
    ("200x0e+4x0e", "64x0e", 140, 2), ("64x0e+64x1o+64x2e", "64x0e+64x1o+64x2e", 4096, 10),
    ("32x0e+32x1o", "64x0e+32x1o", 2500, 60), ("128x0e+128x1o+128x2e", "96x0e+130x1o+8x2e", 1500, 9),
    ("20x0e+20x0e+20x0e+20x0e+20x0e+300x1o", "16x0e+8x1o", 900, 31),
    # small channels with enough rows for the tensor cores, and odd ones of every kind
    ("16x0e+5x1o+1x3o", "12x0e+7x1o+3x3o", 30_000, 3), ("37x0e+21x1o+5x2e", "50x0e+19x1o+7x2e", 1101, 7),
    ("16x3o+12x2e", "20x3o+8x2e", 12_345, 256), ("1x0e", "1x0e", 700, 2), ("5x0e+4x0e+3x1o", "4x0e+2x1o+6x0e", 600, 3),
    ("260x0e+100x1o", "130x0e+260x1o", 600, 3), ("65x0e+129x1o", "63x0e+65x1o", 515, 1),
    ("4x1o", "4x1e", 700, 2), ("8x0e", "8x0e+4x2e", 5000, 3), ("64x0e+32x3o", "64x0e+100x3o", 5000, 40)]


def linear_inputs(irr, n, n_types, seed, padded=0.15):
    r = rng(seed)
    di, do, nw = O.blocks(irr[0])[1], O.blocks(irr[1])[1], O.linear_paths(*irr)[1]
    t = r.integers(0, n_types, size=n)
    if n_types > 2:
        t[t == 1] = 0  # a type without nodes
    t[r.random(n) < padded] = -1
    d = dict(x=r.normal(size=(n, di)), a=r.normal(size=(n, di)), g=r.normal(size=(n, do)),
             w=r.normal(size=(n_types, nw)), al=r.normal(size=(n_types, nw)))
    return t, {k: f32(v) for k, v in d.items()}


def linear_check(T, irr, n, n_types, gemm="fp32", shift=0, padded=0.15):
    import torch
    t, d = linear_inputs(irr, n, n_types, 11 + n, padded)
    p = T.LinearPlan(*irr, n_types=n_types, gemm=gemm)
    G = T.NodeGroups(dev(t, torch.int32), n_types)
    v = {k: dev(a, shift=shift) for k, a in d.items()}
    tol, k = (5e-3, 5e-3) if gemm == "tf32" else (TOL, SUM)
    out = T.linear_forward(p, G, v["x"], v["w"])
    rows_close(out, O.linear(*irr, t, d["x"], d["w"]), tol)
    assert not out[torch.as_tensor(t < 0)].any()
    r = T.linear_backward(p, G, v["x"], v["w"], v["g"])
    dx, dw = O.linear_backward(*irr, t, d["x"], d["w"], d["g"])
    mags = O.linear_backward(*irr, t, np.abs(d["x"]), d["w"], np.abs(d["g"]))[1]
    rows_close(r["dx"], dx, tol)
    sums_close(r["dweight"], dw, mags, k)
    again = T.linear_backward(p, G, v["x"], v["w"], v["g"], want=("dweight",))
    assert list(again) == ["dweight"] and torch.equal(again["dweight"], r["dweight"])
    r = T.linear_double_backward(p, G, v["x"], v["w"], v["g"], v["a"], v["al"])
    d_g, d_x, d_w = O.linear_double_backward(*irr, t, d["x"], d["w"], d["g"], d["a"], d["al"])
    rows_close(r["d_g"], d_g, tol)
    rows_close(r["d_x"], d_x, tol)
    sums_close(r["d_weight"], d_w, O.linear_backward(*irr, t, np.abs(d["a"]), d["w"], np.abs(d["g"]))[1], k)
    z = T.linear_double_backward(p, G, v["x"], v["w"], v["g"])
    assert not any(q.any() for q in z.values())
    one = T.linear_double_backward(p, G, v["x"], v["w"], v["g"], gg_weight=v["al"])
    rows_close(one["d_g"], O.linear(*irr, t, d["x"], d["al"]), tol)
    assert not one["d_weight"].any()
    assert T._lib.tpconv_linear_device_status(p) == 0


@pytest.mark.parametrize("i,o,n,n_types", LINEARS)
def test_linear(T, i, o, n, n_types):
    linear_check(T, (i, o), n, n_types)


@pytest.mark.parametrize("gemm", ["tf32", "simt"])
@pytest.mark.parametrize("k", [0, 1, 2, 5, 8])
def test_linear_modes(T, k, gemm):
    i, o, n, n_types = LINEARS[k]
    linear_check(T, (i, o), n, n_types, gemm=gemm)


@pytest.mark.parametrize("k", [0, 1, 8])
def test_linear_of_tensors_off_16_bytes(T, k):
    i, o, n, n_types = LINEARS[k]
    linear_check(T, (i, o), n, n_types, shift=1)


@pytest.mark.parametrize("padded", [0.0, 1.0])
def test_linear_all_or_no_rows(T, padded):
    linear_check(T, ("64x0e+32x1o", "32x0e+64x1o"), 500, 3, padded=padded)


def test_linear_many_nodes_of_one_type(T):
    """long sums: the weight gradient over 60 000 rows of one type, checked at 1e-5 of its largest value"""
    import torch
    irr = ("64x0e+32x1o",) * 2
    t, d = linear_inputs(irr, 40_000, 3, 5)
    t[:20_000] = 2
    p = T.LinearPlan(*irr, n_types=3)
    G = T.NodeGroups(dev(t, torch.int32), 3)
    v = {k: dev(a) for k, a in d.items()}
    r = T.linear_backward(p, G, v["x"], v["w"], v["g"])
    dx, dw = O.linear_backward(*irr, t, d["x"], d["w"], d["g"])
    rows_close(r["dx"], dx)
    rows_close(r["dweight"], dw)


def test_linear_nan_stays_in_its_row(T):
    import torch
    irr = ("64x0e+64x1o",) * 2
    t, d = linear_inputs(irr, 600, 3, 6)
    p = T.LinearPlan(*irr, n_types=3)
    G = T.NodeGroups(dev(t, torch.int32), 3)
    x, w = dev(d["x"]), dev(d["w"])
    clean = T.linear_forward(p, G, x, w)
    x[torch.as_tensor(t < 0)] = float("nan")  # padding rows may hold anything
    i = int(np.flatnonzero(t >= 0)[5])
    x[i, 2] = float("inf")
    y = T.linear_forward(p, G, x, w)
    keep = np.arange(600) != i
    assert torch.equal(y[torch.as_tensor(keep)], clean[torch.as_tensor(keep)])
    dw = T.linear_backward(p, G, torch.where(torch.isinf(x), torch.zeros_like(x), x), w, dev(d["g"]))["dweight"]
    assert torch.isfinite(dw).all()


# ---- streams, graphs, a run of all ------------------------------------------------------------------------


def test_refusals_on_the_device(T):
    import torch
    p = T.NormPlan("8x0e")
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        T.norm_forward(p, torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        T.norm_forward(p, torch.zeros(8, 4, device="cuda").t())
    with pytest.raises(ValueError):
        T.norm_forward(p, x.double())
    with pytest.raises(ValueError):
        T.norm_forward(p, x, torch.ones(7, device="cuda"))
    with pytest.raises(ValueError):
        T.norm_forward(p, x, torch.ones(8))
    with pytest.raises(T.TPConvError):
        T.norm_forward(p, x, out=x)
    with pytest.raises(ValueError):
        T.norm_backward(p, x, None, x, want=("dy",))
    with pytest.raises(ValueError):
        T.NodeGroups(x, 3)
    with pytest.raises(ValueError):
        T.NodeGroups(torch.zeros(4, dtype=torch.int32, device="cuda"), 257)
    q = T.LinearPlan("8x0e", "4x0e", n_types=2)
    G = T.NodeGroups(torch.zeros(4, dtype=torch.int32, device="cuda"), 2)
    w = torch.zeros(2, 32, device="cuda")
    with pytest.raises(ValueError):
        T.linear_forward(q, T.NodeGroups(torch.zeros(4, dtype=torch.int32, device="cuda"), 3), x, w)
    with pytest.raises(ValueError):
        T.linear_forward(q, G, x[:3], w)
    with pytest.raises(ValueError):
        T.linear_forward(q, G, x, w[:1])
    with pytest.raises(TypeError):
        T.linear_backward(q, G, x, w, None)


def test_streams_and_captured_graphs(T):
    """An explicit stream; then norm + linear and their gradients captured into two graphs and replayed on new
    inputs in turn, against the eager calls bit for bit."""
    import torch
    irr, n = "64x0e+64x1o+64x2e", 500
    t, d = linear_inputs((irr, irr), n, 6, 3)
    p, q = T.NormPlan(irr), T.LinearPlan(irr, irr, n_types=6)
    G = T.NodeGroups(dev(t, torch.int32), 6)
    x, g, w = dev(d["x"]), dev(d["g"]), dev(d["w"])

    def run():
        h = T.norm_forward(p, x)
        y = T.linear_forward(q, G, h, w)
        r = T.linear_backward(q, G, h, w, g)
        s = T.norm_backward(p, x, None, r["dx"])
        return [h, y, r["dweight"], s["dx"], s["dweight"]]

    eager = [v.clone() for v in run()]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = T.linear_forward(q, G, T.norm_forward(p, x, stream=st), w, stream=st)
    st.synchronize()
    assert torch.equal(other, eager[1])
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run())
        graphs.append(gr)
    for seed in (1, 2):
        x.copy_(dev(f32(rng(seed).normal(size=x.shape))))
        g.copy_(dev(f32(rng(seed + 9).normal(size=g.shape))))
        want = [v.clone() for v in run()]
        for gr, o in zip(graphs, outs):
            gr.replay()
            assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_block_of_all_differentiated_twice(T):
    """norm -> typed linear -> convolution -> typed linear on a padded graph, as a layer uses them: energies,
    forces and the gradient of a force loss, against fp64 automatic differentiation of the definitions around
    the convolution's oracle."""
    import torch
    import workloads as W
    from oracle import conv
    irr, lsh, R = "16x0e+16x1o", 2, 4
    rowptr, col, vec = W.random_graph(40, 160, 4)
    N = 40
    r = rng(8)
    types = r.integers(0, 3, size=N)
    types[[5, 17]] = -1
    torch.manual_seed(1)
    norm = T.EquivariantNorm(irr)
    up, down = T.TypedLinear(irr, irr, 3), T.TypedLinear(irr, "8x0e", 3)
    cv = T.TPConv(irr, lsh, irr, R)
    with torch.no_grad():
        norm.weight.add_(0.2 * torch.randn_like(norm.weight))
        norm.bias.add_(0.2 * torch.randn_like(norm.bias))
    groups = T.NodeGroups(dev(types, torch.int32), 3)
    x = dev(f32(r.normal(size=(N, 64)))).requires_grad_(True)
    v = dev(f32(vec)).requires_grad_(True)
    graph = T.Graph(dev(rowptr, torch.int32), dev(col, torch.int32), v)
    seed = dev(f32(r.normal(size=(N, 8))))
    cx, cvv = dev(f32(r.normal(size=(N, 64)))), dev(f32(r.normal(size=vec.shape)))
    params = [norm.weight, norm.bias, up.weight, cv.theta, down.weight]
    out = down(cv(up(norm(x), groups), graph), groups)
    dx, dv = torch.autograd.grad((out * seed).sum(), [x, v], create_graph=True)
    second = torch.autograd.grad((dx * cx).sum() + (dv * cvv).sum(), [x] + params, allow_unused=True)
    first = torch.autograd.grad((down(cv(up(norm(x), groups), graph), groups) * seed).sum(), params)

    # the definitions in fp64 on the host: the convolution is linear in x through a matrix per edge vector set,
    # taken from its oracle's backward by differences in nothing: its own first and second order adjoints
    prob = conv.Problem(irr, lsh, irr, R, "bessel", (5.0,))
    th = host(cv.theta)
    x64, w64, b64 = host(x), host(norm.weight), host(norm.bias)
    u64, d64, s64, v64 = host(up.weight), host(down.weight), host(seed), host(v)
    eps = float(np.float32(EPS))
    h = O.norm(irr, x64, w64, b64, eps)
    y = O.linear(irr, irr, types, h, u64)
    z = conv.forward(prob, rowptr, col, v64, y, th)
    o = O.linear(irr, "8x0e", types, z, d64)
    rows_close(out, o)
    gz, gd = O.linear_backward(irr, "8x0e", types, z, d64, s64)
    cb = conv.backward(prob, rowptr, col, v64, y, th, gz)
    gh, gu = O.linear_backward(irr, irr, types, h, u64, cb["dx"])
    gx, gw, gb = O.norm_backward(irr, x64, w64, gh, eps)
    rows_close(dx, gx, 2e-5)  # four operators in a row, half a bar each
    rows_close(dv, cb["dvec"], 2e-5)
    for got, want in zip(first, (gw, gb, gu, cb["dtheta"], gd)):
        rows_close(got, want, 2e-5)
    # second order, back through the four adjoints
    c64, k64 = host(cx), host(cvv)
    a_gh, a_x, a_w = O.norm_double_backward(irr, x64, w64, gh, c64, 0 * w64, 0 * b64, eps)
    a_gy, a_h, a_u = O.linear_double_backward(irr, irr, types, h, u64, cb["dx"], a_gh, 0 * u64)
    cd = conv.double_backward(prob, rowptr, col, v64, y, th, gz, a_gy, k64, None)
    # d_g of the convolution flows into gz = down^T seed: its weight only
    d_down = O.linear_double_backward(irr, "8x0e", types, z, d64, s64, cd["d_g"], 0 * d64)[2]
    # d_x of the convolution flows into y
    bh, bu = O.linear_backward(irr, irr, types, h, u64, cd["d_x"])
    bx, bw, bb = O.norm_backward(irr, x64, w64, bh + a_h, eps)
    for got, want in zip(second, (a_x + bx, a_w + bw, bb, a_u + bu, cd["d_theta"], d_down)):
        rows_close(got, want, 4e-5)  # eight adjoints in a row


def test_modules_as_a_training_program_uses_them(T):
    """frozen weights, no weights, a third derivative refused, a captured backward of the modules"""
    import torch
    irr = "8x0e+4x1o"
    x = torch.randn(30, 20, device="cuda", requires_grad=True)
    n = T.EquivariantNorm(irr, affine=False)
    (gx,) = torch.autograd.grad(n(x).square().sum(), x, create_graph=True)
    (gg,) = torch.autograd.grad(gx.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(gg.sum(), x)
    lin = T.TypedLinear(irr, irr, 2).requires_grad_(False)
    G = T.NodeGroups(torch.zeros(30, dtype=torch.int32, device="cuda"), 2)
    lin(x, G).sum().backward()  # an expanded cotangent, no weight gradient wanted
    assert lin.weight.grad is None and x.grad is not None


def test_expired_waits_are_reported_and_recovered(T):
    """With a wait limit of 1 ns the tensor-core kernels' bounded waits run out on purpose: the call returns, the
    status says so once, and the next call is right again."""
    import torch
    L = T._lib
    irr = ("64x0e+64x1o+64x2e",) * 2
    t, d = linear_inputs(irr, 3000, 4, 2)
    p = T.LinearPlan(*irr, n_types=4)
    G = T.NodeGroups(dev(t, torch.int32), 4)
    x, w, g = dev(d["x"]), dev(d["w"]), dev(d["g"])
    want = (T.linear_forward(p, G, x, w), T.linear_backward(p, G, x, w, g, want=("dweight",))["dweight"])
    assert L.tpconv_linear_device_status(p) == L.TPCONV_OK
    try:
        L.tpconv_set_wait_limit(1)
        T.linear_forward(p, G, x, w)
        a = L.tpconv_linear_device_status(p)
        T.linear_backward(p, G, x, w, g, want=("dweight",))
        b = L.tpconv_linear_device_status(p)
    finally:
        L.tpconv_set_wait_limit(0)
    assert (a, b) == (L.TPCONV_ERR_TIMEOUT, L.TPCONV_ERR_TIMEOUT)
    assert L.tpconv_linear_device_status(p) == L.TPCONV_OK
    got = (T.linear_forward(p, G, x, w), T.linear_backward(p, G, x, w, g, want=("dweight",))["dweight"])
    assert L.tpconv_linear_device_status(p) == L.TPCONV_OK
    assert all(torch.equal(u, v) for u, v in zip(got, want))


FIRST_CALL_CAPTURED = """
import torch
import equivariant_gnn_tensor_receiver_b200 as T
irr, n = "48x0e+16x1o", 1500
x = torch.randn(n, 96, device="cuda")
types = torch.randint(-1, 3, (n,), device="cuda", dtype=torch.int32)
norm, lin = T.EquivariantNorm(irr), T.TypedLinear(irr, irr, 3)
x.requires_grad_(True)
params = [x, norm.weight, norm.bias, lin.weight]

def step():
    groups = T.NodeGroups(types, 3)
    out = lin(norm(x), groups)
    first = torch.autograd.grad(out.square().sum(), params, create_graph=True)
    second = torch.autograd.grad(first[0].square().sum(), params)
    return [out, *first, *second]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):   # the first call of every kernel
    held = step()
for _ in range(2):
    with torch.no_grad():
        x.copy_(torch.randn_like(x))
        types.copy_(torch.randint(-1, 3, (n,), device="cuda", dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, step()):
        assert torch.equal(a, b)
print("captured ok")
"""


def test_first_calls_may_be_captured():
    """A fresh process whose first call of every operator is a captured one, first and second order; the replays
    on new features and new types agree bit for bit with eager calls."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_CAPTURED], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout + r.stderr


def test_two_streams_at_once(T):
    """the same plan, groups and weights from two streams at a time, each call with a workspace of its own"""
    import torch
    irr = ("64x0e+64x1o",) * 2
    t, d = linear_inputs(irr, 3000, 5, 4)
    p, q = T.LinearPlan(*irr, n_types=5), T.NormPlan(irr[0])
    G = T.NodeGroups(dev(t, torch.int32), 5)
    x, w, g, a = dev(d["x"]), dev(d["w"]), dev(d["g"]), dev(d["a"])

    def run(v, stream=None):
        r = T.linear_backward(p, G, v, w, g, stream=stream)
        s = T.norm_backward(q, v, None, g, stream=stream)
        return [r["dx"], r["dweight"], s["dx"], s["dweight"], s["dbias"]]

    want = [[u.clone() for u in run(v)] for v in (x, a)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, v in enumerate((x, a)):
            got[i].append(run(v, streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(u, v) for u, v in zip(r, want[i]))


@pytest.mark.parametrize("n", [40, 700, 5000, 40000])
def test_gradients_together_and_one_by_one(T, n):
    """The kernels of one call overlap: all gradients together, call after call with one workspace and changing
    inputs, each read at once by work behind it, equal the gradients asked for alone, bit for bit; eagerly and
    captured."""
    import torch
    irr = ("64x0e+32x1o+8x2e",) * 2
    t, d = linear_inputs(irr, n, 7, 6)
    p, q = T.LinearPlan(*irr, n_types=7), T.NormPlan(irr[0])
    G = T.NodeGroups(dev(t, torch.int32), 7)
    w = dev(d["w"])
    v = dev(f32(rng(5).normal(size=w.shape)))
    rows = [dev(d[k]) for k in ("x", "g", "a")]

    def bytes_of(plan, op):
        return max(plan.workspace_bytes(op, n), 256)

    ws = torch.empty(max(bytes_of(k, o) for k in (p, q) for o in (1, 2)), dtype=torch.uint8, device="cuda")

    def together(x, g, a):
        b = T.linear_backward(p, G, x, w, g, ws=ws)
        c = T.linear_double_backward(p, G, x, w, g, gg_x=a, gg_weight=v, ws=ws)
        e = T.norm_backward(q, x, None, g, ws=ws)
        f = T.norm_double_backward(q, x, None, g, gg_x=a, ws=ws)
        return [u.clone() for r in (b, c, e, f) for u in r.values()]

    def alone(x, g, a):
        out = []
        for k in ("dx", "dweight"):
            out.append(T.linear_backward(p, G, x, w, g, want=(k,))[k])
            torch.cuda.synchronize()
        for k in ("d_g", "d_x", "d_weight"):
            out.append(T.linear_double_backward(p, G, x, w, g, gg_x=a, gg_weight=v, want=(k,))[k])
            torch.cuda.synchronize()
        for k in ("dx", "dweight", "dbias"):
            out.append(T.norm_backward(q, x, None, g, want=(k,))[k])
            torch.cuda.synchronize()
        for k in ("d_g", "d_x", "d_weight"):
            out.append(T.norm_double_backward(q, x, None, g, gg_x=a, want=(k,))[k])
            torch.cuda.synchronize()
        return out

    turns = [(rows[i % 3], rows[(i + 1) % 3], rows[(i + 2) % 3]) for i in range(3)]
    want = [alone(*r) for r in turns]
    got = [together(*turns[i % 3]) for i in range(9)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = [together(*r) for r in turns]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for i, r in enumerate(got + held):
        assert len(r) == len(want[i % 3])
        for u, z in zip(r, want[i % 3]):
            assert torch.equal(u, z)


def test_rows_beyond_32_bits(T):
    """More than 2^31 floats in a tensor: only the last rows hold anything, and they and the weight gradients come
    out as for those rows alone (norm: bit for bit; linear: another kernel, 2 TOL of the largest value)."""
    import torch
    irr, n, k = "64x0e+64x1o+64x2e", 3800011, 300
    dim = 576
    assert n * dim > 2 ** 31
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    r = rng(8)
    few = {s: dev(f32(r.normal(size=(k, dim)))) for s in "xg"}
    t = torch.arange(n, dtype=torch.int32, device="cuda") % 4
    t[-k:] = dev(r.integers(-1, 4, k), torch.int32)
    p, q = T.LinearPlan(irr, irr, n_types=4), T.NormPlan(irr)
    w = dev(f32(r.normal(size=(4, p.weight_numel))))
    G, H = T.NodeGroups(t, 4), T.NodeGroups(t[-k:], 4)
    x, g = torch.zeros(n, dim, device="cuda"), torch.zeros(n, dim, device="cuda")
    x[-k:], g[-k:] = few["x"], few["g"]
    assert torch.equal(T.norm_forward(q, x)[-k:], T.norm_forward(q, few["x"]))
    assert torch.equal(T.norm_backward(q, x, None, g, want=("dx",))["dx"][-k:],
                       T.norm_backward(q, few["x"], None, few["g"], want=("dx",))["dx"])

    def close(a, b):
        assert (a - b).abs().max() <= 2 * TOL * b.abs().max()

    close(T.linear_forward(p, G, x, w)[-k:], T.linear_forward(p, H, few["x"], w))
    a, b = T.linear_backward(p, G, x, w, g), T.linear_backward(p, H, few["x"], w, few["g"])
    close(a["dx"][-k:], b["dx"])
    close(a["dweight"], b["dweight"])
    assert not a["dx"][:-k].any()
    torch.cuda.empty_cache()
