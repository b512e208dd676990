"""Node operators at the limits of their contract, on the device: the largest graphs, long sums, caller-owned
buffers on explicit streams.  Tolerances stand beside each test."""

import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import node as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import equivariant_gnn_tensor_receiver_b200 as T
    T.lib()
    return T


@pytest.mark.parametrize("gemm", ["fp32", "simt"])
def test_linear_of_the_most_nodes(T, gemm):
    """2^31 - 1 nodes, nearly all of one type, some of no type behind them: counts of tiles and the steps past the
    last node stay below 2^31.  Small whole numbers, so every product and sum is exact."""
    import torch
    n, few = 2 ** 31 - 1, 1000
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB")
    types = torch.ones(n, dtype=torch.int32, device="cuda")
    types[3:7] = 0
    types[-5:] = -1
    G = T.NodeGroups(types, 2)
    assert G.offsets.tolist() == [0, 4, n - 5]
    assert G.perm[:6].tolist() == [3, 4, 5, 6, 0, 1] and G.perm[-6:].tolist() == list(range(n - 6, n))
    p = T.LinearPlan("1x0e", "1x0e", n_types=2, gemm=gemm)
    w = torch.tensor([[3.0], [2.0]], device="cuda")
    x = torch.randint(1, 100, (n, 1), device="cuda", dtype=torch.int8).float()
    want = x * 2
    want[3:7] = 3 * x[3:7]
    want[-5:] = 0
    out = torch.full_like(x, -1)
    T.linear_forward(p, G, x, w, out=out)
    assert torch.equal(out, want)
    del want
    g = out.zero_()
    g[:few], g[-few:] = 1, 2
    r = T.linear_backward(p, G, x, w, g)
    some = torch.cat((x[:few], 2 * x[-few:-5]))[:, 0]
    a = x[3:7].sum()
    assert r["dweight"].tolist() == [[a.item()], [(some.sum() - a).item()]]
    dx = r["dx"]
    assert (dx[:few, 0] == torch.where(types[:few] == 0, 3.0, 2.0)).all() and (dx[-few:-5] == 4).all()
    assert not dx[-5:].any() and not dx[few:-few].any()
    assert T._lib.tpconv_linear_device_status(p) == 0
    del x, g, out, dx, r, G, types
    torch.cuda.empty_cache()


def calls_with_buffers(T):
    """name, call(ws or out, stream), elements and type of the caller's buffer"""
    import torch
    n, irr = 600, "64x0e+32x1o"
    dim = 160
    p, q = T.LinearPlan(irr, irr, n_types=3), T.NormPlan(irr)
    G = T.NodeGroups(torch.arange(n, dtype=torch.int32, device="cuda") % 3, 3)
    x, g, a = (torch.randn(n, dim, device="cuda") for _ in range(3))
    w = torch.randn(3, p.weight_numel, device="cuda")
    kb = lambda plan, op: (plan.workspace_bytes(op, n), torch.uint8)  # noqa: E731
    rows = (n * dim, torch.float32)
    return [
        ("linear_forward out", lambda b, s: T.linear_forward(p, G, x, w, out=b.view(n, dim), stream=s), rows),
        ("linear_forward ws", lambda b, s: T.linear_forward(p, G, x, w, ws=b, stream=s), (1 << 20, torch.uint8)),
        ("linear_backward ws", lambda b, s: T.linear_backward(p, G, x, w, g, ws=b, stream=s), kb(p, 1)),
        ("linear_double_backward ws", lambda b, s: T.linear_double_backward(p, G, x, w, g, a, w, ws=b, stream=s),
         kb(p, 2)),
        ("norm_forward out", lambda b, s: T.norm_forward(q, x, out=b.view(n, dim), stream=s), rows),
        ("norm_backward ws", lambda b, s: T.norm_backward(q, x, None, g, ws=b, stream=s), kb(q, 1)),
        ("norm_double_backward ws", lambda b, s: T.norm_double_backward(q, x, None, g, a, ws=b, stream=s), kb(q, 2)),
    ]


def test_buffers_of_the_caller_are_held_for_the_stream(T):
    """A caller drops ``out`` or ``ws`` right after a call on another stream that is still busy: the allocator does
    not hand the memory to the current stream before the call is done."""
    import torch
    side = torch.cuda.Stream()
    for name, call, (numel, dtype) in calls_with_buffers(T):
        new = lambda: torch.empty(numel, dtype=dtype, device="cuda")  # noqa: E731
        call(new(), side)  # (the first call loads its kernels, which waits for the device)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        b = new()
        at = b.data_ptr()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)  # some 0.1 s of work ahead of the call
        call(b, side)
        busy = not side.query()
        del b
        other = new()
        assert busy and other.data_ptr() != at, name
        side.synchronize()


def test_refused_buffers_on_a_stream(T):
    """what is wrong with ``out`` or ``ws`` is said as without a stream, and the current device and stream stay"""
    import torch
    side = torch.cuda.Stream()
    x = torch.zeros(4, 8, device="cuda")
    q = T.NormPlan("8x0e")
    here = torch.cuda.current_stream()
    for bad, error in ((3, TypeError), (torch.zeros(1 << 16, dtype=torch.uint8), ValueError)):
        with pytest.raises(error):
            T.norm_backward(q, x, None, x.clone(), ws=bad, stream=side)
    for bad, error in ((3, TypeError), (torch.zeros(4, 8), ValueError), (x[:3], ValueError)):
        with pytest.raises(error):
            T.norm_forward(q, x, out=bad, stream=side)
    assert torch.cuda.current_stream() == here and torch.cuda.current_device() == 0


@pytest.mark.parametrize("i,o,gemm", [("1024x0e", "704x0e", "fp32"), ("512x1o", "512x1o", "simt")])
def test_linear_weight_gradient_of_many_rows(T, i, o, gemm):
    """The FP32 kernel (wide plans take it in every mode) over up to 240 000 nodes of one type, 64-bit sums beside it.
    Terms of one sign, so nothing cancels.  Tolerance: chains of 256 additions, at most 938 of them added up (l = 1:
    704 of three rows a node in four pieces), each with a rounding of at most 2^-24 of the sum, spread evenly: a
    standard deviation under sqrt(256 + 938) 2^-24 / sqrt(3) = 1.2e-6 of it; 1e-5 is eight of those."""
    import torch
    n = 300_000
    torch.manual_seed(3)
    p = T.LinearPlan(i, o, n_types=3, gemm=gemm)
    types = torch.randint(-1, 2, (n,), dtype=torch.int32, device="cuda")
    types[:240_000] = 1
    G = T.NodeGroups(types, 3)
    x, g = torch.rand(n, p.dim_in, device="cuda").add_(0.5), torch.rand(n, p.dim_out, device="cuda").add_(0.5)
    w = torch.zeros(3, p.weight_numel, device="cuda")
    dw = T.linear_backward(p, G, x, w, g, want=("dweight",))["dweight"]
    q = p.paths[0]
    d = 2 * q["l"] + 1
    for t in range(3):
        want = torch.zeros(q["c_in"], q["c_out"], dtype=torch.float64, device="cuda")
        for rows in torch.nonzero(types == t)[:, 0].split(20_000):
            a, b = x[rows].double().view(-1, q["c_in"], d), g[rows].double().view(-1, q["c_out"], d)
            want += a.transpose(1, 2).reshape(-1, q["c_in"]).t() @ b.transpose(1, 2).reshape(-1, q["c_out"])
        assert ((dw[t].view_as(want).double() - want).abs() <= 1e-5 * want).all()
    assert T._lib.tpconv_linear_device_status(p) == 0


def test_linear_weight_gradient_keeps_infinities(T):
    """gemm "simt": an infinity among thousands of rows of a type, and a sum that overflows, stay infinite"""
    import torch
    n = 20_000
    torch.manual_seed(4)
    p = T.LinearPlan("3x0e", "2x0e", gemm="simt")
    G = T.NodeGroups(torch.zeros(n, dtype=torch.int32, device="cuda"), 1)
    x, g = torch.rand(n, 3, device="cuda") + 0.5, torch.rand(n, 2, device="cuda") + 0.5
    g[:, 1] *= -1
    x[5, 0] = float("inf")
    x[:, 1] = 3e38
    dw = T.linear_backward(p, G, x, torch.zeros(1, 6, device="cuda"), g)["dweight"].view(3, 2)
    inf = float("inf")
    assert dw[:2].tolist() == [[inf, -inf], [inf, -inf]] and torch.isfinite(dw[2]).all()


@pytest.mark.parametrize("irr,n,gemm", [("8x0e", 300, "simt"), ("64x0e+64x1o", 3000, "fp32")])
def test_linear_of_offsets_that_do_not_ascend(T, irr, n, gemm):
    """groups that overlap: results are undefined, but nothing behind the workspace gets into them, and no wait
    runs out"""
    import torch
    L = T._lib
    p = T.LinearPlan(irr, irr, n_types=4, gemm=gemm)
    perm = torch.arange(n, dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, n, 0, n, 0], dtype=torch.int32, device="cuda")
    x, g = (torch.randn(n, p.dim_in, device="cuda") for _ in range(2))
    w = torch.randn(4, p.weight_numel, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    need = p.workspace_bytes(T.OP_BACKWARD, n)
    ws = torch.zeros(need // 4 + (1 << 22), device="cuda")
    ws[need // 4:] = float("nan")
    st = L.lib().tpconv_linear_backward(p.handle, n, perm.data_ptr(), offsets.data_ptr(), x.data_ptr(), w.data_ptr(),
                                        g.data_ptr(), dx.data_ptr(), dw.data_ptr(), ws.data_ptr(), need,
                                        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert st == 0 and L.tpconv_linear_device_status(p) == 0
    assert torch.isfinite(dw).all() and torch.isfinite(dx).all() and ws[need // 4:].isnan().all()


def test_linear_weight_gradient_of_sixty_thousand_rows(T):
    """the tensor-core kernel over 61 000 nodes of one type (183 000 rows for l = 1), each element against 64-bit
    sums.  Terms of one sign.  Tolerance 1e-5 of the sum: 2^-22 a product (operands of 22 bits), at most 128 rows in
    the accumulator, whose additions cut off (2^-23 each, so 1.5e-5 if all went one way; a third of that is what
    chopping a growing sum of 128 terms loses on average), some ten additions of those per CTA and 148 joined."""
    import torch
    irr, n = "64x0e+32x1o", 80_000
    torch.manual_seed(5)
    p = T.LinearPlan(irr, irr, n_types=3)
    types = torch.randint(-1, 2, (n,), dtype=torch.int32, device="cuda")
    types[:61_000] = 2
    types = types[torch.randperm(n, device="cuda")]
    x, g = torch.rand(n, 160, device="cuda").add_(0.5), torch.rand(n, 160, device="cuda").add_(0.5)
    w = torch.zeros(3, p.weight_numel, device="cuda")
    dw = T.linear_backward(p, T.NodeGroups(types, 3), x, w, g, want=("dweight",))["dweight"]
    for q, o, c, d in zip(p.paths, (0, 64), (64, 32), (1, 3)):
        a, b = (v[:, o:o + c * d].double().view(n, c, d) for v in (x, g))
        for t in range(3):
            m = (types == t).double()[:, None, None]
            want = torch.einsum("num,nwm->uw", a * m, b)
            got = dw[t, q["weight_offset"]:q["weight_offset"] + c * c].view(c, c).double()
            assert ((got - want).abs() <= 1e-5 * want).all()


def test_modules_differentiated_twice_on_the_tensor_cores(T):
    """norm -> typed linear at a size that runs on the tensor cores, first and second order against the 64-bit oracle:
    two operators in a row, half a bar (1e-5 of the largest value) each, and twice that for the second order"""
    import torch
    i, o, n, n_types = "64x0e+64x1o+8x2e", "72x0e+64x1o+16x2e", 1500, 5
    r = np.random.Generator(np.random.PCG64(2))
    f32 = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    dev = lambda a: torch.as_tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    host = lambda a: a.detach().double().cpu().numpy()  # noqa: E731
    types = r.integers(-1, n_types, size=n)
    torch.manual_seed(1)
    norm, lin = T.EquivariantNorm(i), T.TypedLinear(i, o, n_types)
    with torch.no_grad():
        norm.weight.add_(0.2 * torch.randn_like(norm.weight))
        norm.bias.add_(0.2 * torch.randn_like(norm.bias))
    G = T.NodeGroups(torch.as_tensor(types, dtype=torch.int32, device="cuda"), n_types)
    di, do = lin.plan.dim_in, lin.plan.dim_out
    X, S, C = f32(r.normal(size=(n, di)) + 0.3), f32(r.normal(size=(n, do))), f32(r.normal(size=(n, di)))
    x = dev(X).requires_grad_(True)
    params = [norm.weight, norm.bias, lin.weight]
    out = lin(norm(x), G)
    first = torch.autograd.grad((out * dev(S)).sum(), [x] + params, create_graph=True)
    second = torch.autograd.grad((first[0] * dev(C)).sum(), [x] + params, allow_unused=True)
    w, b, u = host(norm.weight), host(norm.bias), host(lin.weight)
    eps = float(np.float32(1e-5))
    h = O.norm(i, X, w, b, eps)
    gh, gu = O.linear_backward(i, o, types, h, u, S)
    gx, gw, gb = O.norm_backward(i, X, w, gh, eps)
    # <C, dx> = <C, norm_backward(x, w, lin^T(S, u))>
    a_gh, a_x, a_w = O.norm_double_backward(i, X, w, gh, C, 0 * w, 0 * b, eps)
    _, a_h, a_u = O.linear_double_backward(i, o, types, h, u, S, a_gh, 0 * u)
    assert not a_h.any()
    close = lambda got, want, tol: np.abs(host(got) - want).max() <= tol * np.abs(want).max()  # noqa: E731
    assert close(out, O.linear(i, o, types, h, u), 2e-5)
    for got, want in zip(first, (gx, gw, gb, gu)):
        assert close(got, want, 2e-5)
    assert close(second[0], a_x, 4e-5) and close(second[1], a_w, 4e-5) and close(second[3], a_u, 4e-5)
    assert second[2] is None or not second[2].any()
    assert T._lib.tpconv_linear_device_status(lin.plan) == 0


def test_third_derivatives_are_refused_by_name(T):
    import torch
    irr = "8x0e+4x1o"
    x = torch.randn(30, 20, device="cuda", requires_grad=True)
    G = T.NodeGroups(torch.zeros(30, dtype=torch.int32, device="cuda"), 2)
    norm, lin = T.EquivariantNorm(irr), T.TypedLinear(irr, irr, 2)
    for f, name in ((norm, "EquivariantNorm"), (lambda v: lin(v, G), "TypedLinear")):
        (gx,) = torch.autograd.grad(f(x).pow(3).sum(), x, create_graph=True)
        (gg,) = torch.autograd.grad(gx.square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match=name + " is differentiable twice; a third derivative"):
            torch.autograd.grad(gg.sum(), x)


CAPTURED_BACKWARD = """
import torch
import equivariant_gnn_tensor_receiver_b200 as T
irr, n = "48x0e+16x1o", 1500
torch.manual_seed(0)
x = torch.randn(n, 96, device="cuda")
types = torch.randint(-1, 3, (n,), device="cuda", dtype=torch.int32)
norm, lin = T.EquivariantNorm(irr), T.TypedLinear(irr, irr, 3)
params = [norm.weight, norm.bias, lin.weight]
x.requires_grad_(True)

def step():
    for p in params:
        p.grad = None
    energy = lin(norm(x), T.NodeGroups(types, 3)).square().sum()
    (force,) = torch.autograd.grad(energy, x, create_graph=True)
    (energy + force.square().sum()).backward(inputs=params)

side = torch.cuda.Stream()
side.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(side):
    for _ in range(3):
        step()
torch.cuda.current_stream().wait_stream(side)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
held = [p.grad for p in params]
for _ in range(2):
    with torch.no_grad():
        x.copy_(torch.randn_like(x))
        types.copy_(torch.randint(-1, 3, (n,), device="cuda", dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = [g.clone() for g in held]
    step()
    assert all(torch.equal(a, p.grad) for a, p in zip(got, params))
print("captured ok")
"""


def test_a_captured_backward_of_the_modules():
    """a force-training step with .backward(), captured and replayed on new features and types, against eager steps
    bit for bit; in a process of its own, as a capture that goes wrong may end it"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CAPTURED_BACKWARD], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout + r.stderr
