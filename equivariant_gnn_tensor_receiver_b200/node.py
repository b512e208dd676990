"""Node operators next to the convolution: nodes grouped by type, the typed linear map (one weight per
node type) and the layer norm of irreps features.  As in ``api.py`` the caching allocator owns all
device memory and no arithmetic of an operator happens here; the modules are differentiable twice.

Arguments are checked against the plan (shape, dtype, device, contiguity) before anything is launched.
A call runs on the tensors' device and on ``stream`` (default: that device's current stream); outputs
and workspace are allocated for that stream.
"""

from __future__ import annotations

import contextlib

import torch

from . import _lib as L


def _need(name, t, shape, device, dtype=torch.float32):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")


def _cuda_device(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must be on a CUDA device")
    return t.device


def _wanted(want, names):
    if isinstance(want, str) or any(w not in names for w in want):
        raise ValueError(f"want: expected names of {names}, got {want!r}")
    return want


@contextlib.contextmanager
def _on(device, stream, *tensors):
    """The device current and, with an explicit stream, that stream too: what is allocated inside belongs to it
    and the inputs are not reused before its work on them is done."""
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield
            for t in tensors:
                if t is not None and t.numel():
                    t.record_stream(stream)


def _new(wanted, shape, device):
    return torch.empty(shape, dtype=torch.float32, device=device) if wanted else None


def _ws_for(ws, nbytes, device):
    """The caller's workspace, checked, or a fresh one."""
    if ws is None:
        return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
    if _cuda_device("ws", ws) != device:
        raise ValueError(f"ws: expected a tensor on {device}, got {ws.device}")
    return ws


class NodeGroups:
    """The nodes of a graph by type, computed once: ``perm`` [N] holds the node ids of type 0, 1, ...
    (ascending inside a type) and behind them those of no group (any type outside [0, n_types): padding),
    ``offsets`` [n_types + 1] where each type begins.  ``types`` is an int32 (or int64) vector on the device."""

    def __init__(self, types, n_types, stream=None):
        dev = _cuda_device("types", types)
        if types.dim() != 1 or types.dtype not in (torch.int32, torch.int64):
            raise ValueError("types: expected a vector of int32 or int64")
        n_types = int(n_types)
        if not 1 <= n_types <= L.MAX_TYPES:
            raise ValueError(f"n_types: expected 1..{L.MAX_TYPES}, got {n_types}")
        self.N, self.n_types, self.device = types.numel(), n_types, dev
        with _on(dev, stream, types):
            if types.dtype == torch.int64:  # no wrap-around of far values into a type
                types = torch.where((types >= 0) & (types < n_types), types, -1).to(torch.int32)
            t = types.contiguous()
            self.perm = torch.empty(self.N, dtype=torch.int32, device=dev)
            self.offsets = torch.empty(n_types + 1, dtype=torch.int32, device=dev)
            ws = torch.empty(L.tpconv_group_workspace_size(self.N, n_types), dtype=torch.uint8, device=dev)
            L.tpconv_group_nodes(self.N, n_types, t, self.perm, self.offsets, ws, stream)


# ---- typed linear map ---------------------------------------------------------------------------------


def _linear_args(plan, groups, **t):
    if not isinstance(groups, NodeGroups):
        raise TypeError("groups: expected NodeGroups")
    if groups.n_types != plan.n_types:
        raise ValueError(f"groups: {groups.n_types} types, the plan has {plan.n_types}")
    shapes = {"x": (groups.N, plan.dim_in), "g": (groups.N, plan.dim_out), "weight": (plan.n_types, plan.weight_numel)}
    for k, v in t.items():
        base = k[3:] if k.startswith("gg_") else ("g" if k == "out" else k)
        if v is None and not k.startswith("gg_") and k != "out":
            raise TypeError(f"{k}: expected a tensor")
        _need(k, v, shapes[base], groups.device)
    return groups.N, groups.device


def linear_forward(plan, groups, x, weight, out=None, ws=None, stream=None):
    """out[N, dim_out]: every node's features times the weight of its type; rows of no group are zero."""
    N, dev = _linear_args(plan, groups, x=x, weight=weight, out=out)
    with _on(dev, stream, x, weight, groups.perm, groups.offsets):
        if out is None:
            out = _new(True, (N, plan.dim_out), dev)
        ws = _ws_for(ws, L.tpconv_linear_workspace_size(plan, L.OP_FORWARD, N), dev)
        L.tpconv_linear_forward(plan, N, groups.perm, groups.offsets, x, weight, out, ws, stream)
    return out


def linear_backward(plan, groups, x, weight, g, want=("dx", "dweight"), ws=None, stream=None):
    """{"dx": [N, dim_in], "dweight": [n_types, weight_numel]} for the cotangent g of the output."""
    N, dev = _linear_args(plan, groups, x=x, weight=weight, g=g)
    _wanted(want, ("dx", "dweight"))
    with _on(dev, stream, x, weight, g, groups.perm, groups.offsets):
        outs = {"dx": _new("dx" in want, (N, plan.dim_in), dev),
                "dweight": _new("dweight" in want, (plan.n_types, plan.weight_numel), dev)}
        ws = _ws_for(ws, L.tpconv_linear_workspace_size(plan, L.OP_BACKWARD, N), dev)
        L.tpconv_linear_backward(plan, N, groups.perm, groups.offsets, x, weight, g, outs["dx"], outs["dweight"], ws,
                                 stream)
    return {k: v for k, v in outs.items() if v is not None}


def linear_double_backward(plan, groups, x, weight, g, gg_x=None, gg_weight=None, want=("d_g", "d_x", "d_weight"),
                           ws=None, stream=None):
    """Gradients of <gg_x, dx> + <gg_weight, dweight> by g, x and weight (a cotangent None = zero)."""
    N, dev = _linear_args(plan, groups, x=x, weight=weight, g=g, gg_x=gg_x, gg_weight=gg_weight)
    _wanted(want, ("d_g", "d_x", "d_weight"))
    with _on(dev, stream, x, weight, g, gg_x, gg_weight, groups.perm, groups.offsets):
        outs = {"d_g": _new("d_g" in want, (N, plan.dim_out), dev), "d_x": _new("d_x" in want, (N, plan.dim_in), dev),
                "d_weight": _new("d_weight" in want, (plan.n_types, plan.weight_numel), dev)}
        ws = _ws_for(ws, L.tpconv_linear_workspace_size(plan, L.OP_DOUBLE_BACKWARD, N), dev)
        L.tpconv_linear_double_backward(plan, N, groups.perm, groups.offsets, x, weight, g, gg_x, gg_weight,
                                        outs["d_g"], outs["d_x"], outs["d_weight"], ws, stream)
    return {k: v for k, v in outs.items() if v is not None}


# ---- layer norm ----------------------------------------------------------------------------------------


def _norm_args(plan, x, **t):
    dev = _cuda_device("x", x)
    if x.dim() != 2:
        raise ValueError(f"x: expected shape (N, {plan.dim}), got {tuple(x.shape)}")
    N = x.shape[0]
    rows, w, b = (N, plan.dim), (plan.weight_numel,), (plan.bias_numel,)
    shapes = {"x": rows, "g": rows, "out": rows, "weight": w, "bias": b}
    _need("x", x, rows, dev)
    for k, v in t.items():
        if v is None and k == "g":
            raise TypeError("g: expected a tensor")
        _need(k, v, shapes[k[3:] if k.startswith("gg_") else k], dev)
    return N, dev


def norm_forward(plan, x, weight=None, bias=None, out=None, stream=None):
    """The layer norm of x[N, dim]; weight None stands for ones, bias None for zeros."""
    N, dev = _norm_args(plan, x, weight=weight, bias=bias, out=out)
    with _on(dev, stream, x, weight, bias):
        if out is None:
            out = _new(True, (N, plan.dim), dev)
        L.tpconv_norm_forward(plan, N, x, weight, bias, out, stream)
    return out


def norm_backward(plan, x, weight, g, want=("dx", "dweight", "dbias"), ws=None, stream=None):
    """{"dx", "dweight", "dbias"} for the cotangent g of the output."""
    N, dev = _norm_args(plan, x, weight=weight, g=g)
    _wanted(want, ("dx", "dweight", "dbias"))
    with _on(dev, stream, x, weight, g):
        outs = {"dx": _new("dx" in want, (N, plan.dim), dev),
                "dweight": _new("dweight" in want, (plan.weight_numel,), dev),
                "dbias": _new("dbias" in want, (plan.bias_numel,), dev)}
        ws = _ws_for(ws, L.tpconv_norm_workspace_size(plan, L.OP_BACKWARD, N), dev)
        L.tpconv_norm_backward(plan, N, x, weight, g, outs["dx"], outs["dweight"], outs["dbias"], ws, stream)
    return {k: v for k, v in outs.items() if v is not None}


def norm_double_backward(plan, x, weight, g, gg_x=None, gg_weight=None, gg_bias=None,
                         want=("d_g", "d_x", "d_weight"), ws=None, stream=None):
    """Gradients of <gg_x, dx> + <gg_weight, dweight> + <gg_bias, dbias> by g, x and weight."""
    N, dev = _norm_args(plan, x, weight=weight, g=g, gg_x=gg_x, gg_weight=gg_weight, gg_bias=gg_bias)
    _wanted(want, ("d_g", "d_x", "d_weight"))
    with _on(dev, stream, x, weight, g, gg_x, gg_weight, gg_bias):
        outs = {"d_g": _new("d_g" in want, (N, plan.dim), dev), "d_x": _new("d_x" in want, (N, plan.dim), dev),
                "d_weight": _new("d_weight" in want, (plan.weight_numel,), dev)}
        ws = _ws_for(ws, L.tpconv_norm_workspace_size(plan, L.OP_DOUBLE_BACKWARD, N), dev)
        L.tpconv_norm_double_backward(plan, N, x, weight, g, gg_x, gg_weight, gg_bias, outs["d_g"], outs["d_x"],
                                      outs["d_weight"], ws, stream)
    return {k: v for k, v in outs.items() if v is not None}


# ---- torch autograd glue: as for the convolution, the backward of a backward is the library's double
# backward; a third derivative raises ----------------------------------------------------------------


def _c(t):
    return None if t is None else t.detach().contiguous()


def _names(flags, names):
    return tuple(n for f, n in zip(flags, names) if f)


class _LinearFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, plan, groups):
        ctx.plan, ctx.groups = plan, groups
        ctx.save_for_backward(x, weight)
        return linear_forward(plan, groups, _c(x), _c(weight))

    @staticmethod
    def backward(ctx, g):
        x, weight = ctx.saved_tensors
        dx, dw = _LinearBwdFn.apply(x, weight, g, ctx.plan, ctx.groups, ctx.needs_input_grad[:2])
        return dx, dw, None, None


class _LinearBwdFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, g, plan, groups, flags):
        ctx.plan, ctx.groups = plan, groups
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, g)
        r = linear_backward(plan, groups, _c(x), _c(weight), _c(g), want=_names(flags, ("dx", "dweight")))
        return r.get("dx"), r.get("dweight")

    @staticmethod
    def backward(ctx, gg_x, gg_weight):
        d_x, d_w, d_g = _LinearDblFn.apply(*ctx.saved_tensors, gg_x, gg_weight, ctx.plan, ctx.groups,
                                           ctx.needs_input_grad[:3])
        return d_x, d_w, d_g, None, None, None


class _LinearDblFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, g, gg_x, gg_weight, plan, groups, flags):
        r = linear_double_backward(plan, groups, _c(x), _c(weight), _c(g), _c(gg_x), _c(gg_weight),
                                   want=_names(flags, ("d_x", "d_weight", "d_g")))
        return r.get("d_x"), r.get("d_weight"), r.get("d_g")

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("TypedLinear is differentiable twice; a third derivative is not provided")


class TypedLinear(torch.nn.Module):
    """Linear map of irreps features with one weight per node type.

    ``forward(x, groups)`` takes x[N, dim_in] and the nodes' ``NodeGroups``; padding rows (no group) come out
    zero.  The weight is [n_types][weight_numel], normal with standard deviation 1/sqrt(fan-in of the output
    block).  ``gemm``: "fp32", "tf32" or "simt", as for ``TPConv``.  Differentiable twice in x and the weight.
    """

    def __init__(self, irreps_in, irreps_out, n_types=1, gemm="fp32", device="cuda"):
        super().__init__()
        self.plan = L.LinearPlan(irreps_in, irreps_out, n_types, gemm)
        fan = {}
        for p in self.plan.paths:
            fan[p["out_block"]] = fan.get(p["out_block"], 0) + p["c_in"]
        w = torch.empty(self.plan.n_types, self.plan.weight_numel)
        for p in self.plan.paths:
            o = p["weight_offset"]
            w[:, o:o + p["c_in"] * p["c_out"]].normal_(0, fan[p["out_block"]] ** -0.5)
        self.weight = torch.nn.Parameter(w.to(device=device, dtype=torch.float32))

    def forward(self, x, groups: NodeGroups):
        return _LinearFn.apply(x, self.weight, self.plan, groups)


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, plan):
        ctx.plan = plan
        ctx.save_for_backward(x, weight)
        return norm_forward(plan, _c(x), _c(weight), _c(bias))

    @staticmethod
    def backward(ctx, g):
        x, weight = ctx.saved_tensors
        dx, dw, db = _NormBwdFn.apply(x, weight, g, ctx.plan, ctx.needs_input_grad[:3])
        return dx, dw, db, None


class _NormBwdFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, g, plan, flags):
        ctx.plan = plan
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, weight, g)
        r = norm_backward(plan, _c(x), _c(weight), _c(g), want=_names(flags, ("dx", "dweight", "dbias")))
        return r.get("dx"), r.get("dweight"), r.get("dbias")

    @staticmethod
    def backward(ctx, gg_x, gg_weight, gg_bias):
        d_x, d_w, d_g = _NormDblFn.apply(*ctx.saved_tensors, gg_x, gg_weight, gg_bias, ctx.plan,
                                         ctx.needs_input_grad[:3])
        return d_x, d_w, d_g, None, None


class _NormDblFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, g, gg_x, gg_weight, gg_bias, plan, flags):
        r = norm_double_backward(plan, _c(x), _c(weight), _c(g), _c(gg_x), _c(gg_weight), _c(gg_bias),
                                 want=_names(flags, ("d_x", "d_weight", "d_g")))
        return r.get("d_x"), r.get("d_weight"), r.get("d_g")

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("EquivariantNorm is differentiable twice; a third derivative is not provided")


class EquivariantNorm(torch.nn.Module):
    """Layer norm of irreps features: every block of a node is divided by the root mean square of its entries
    (scalars less their mean first) and scaled per channel; 0e blocks get a bias.  On scalars alone it is the
    plain layer norm.  Differentiable twice in x, the weight and the bias."""

    def __init__(self, irreps, eps=1e-5, affine=True, device="cuda"):
        super().__init__()
        self.plan = L.NormPlan(irreps, eps)
        make = lambda t: torch.nn.Parameter(t.to(device=device)) if affine else None  # noqa: E731
        self.weight = make(torch.ones(self.plan.weight_numel))
        self.bias = make(torch.zeros(self.plan.bias_numel))

    def forward(self, x):
        return _NormFn.apply(x, self.weight, self.bias, self.plan)
