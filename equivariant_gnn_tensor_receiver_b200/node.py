"""Node operators next to the convolution: nodes grouped by type, the typed linear map (one weight per
node type) and the layer norm of irreps features.  As in ``api.py`` the caching allocator owns all
device memory and no arithmetic of an operator happens here; the modules are differentiable twice.

Arguments are checked against the plan (shape, dtype, device, contiguity) before anything is launched.
A call runs on the tensors' device and on ``stream`` (default: that device's current stream); outputs
and workspace are allocated for that stream, and what the caller brings is held for it.

The tensor-core kernels of the typed linear map bound their waits (2 s).  A call does not report one that ran
out (its outputs are then not valid): ``_lib.tpconv_linear_device_status(plan)`` does, for all linear plans of
the device since the last query.
"""

from __future__ import annotations

import torch

from . import _lib as L

_F32, _I32 = torch.float32, torch.int32


def _refuse(name, t, shape, dev, dtype):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must be on a CUDA device")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: expected a tensor on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name}: tensor must be contiguous")


def _ptr(name, t, shape, dev, optional=False):
    """Device address of a checked fp32 tensor (None stands for a null pointer where that is allowed)."""
    if t is None and optional:
        return None
    if (not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype is not _F32 or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(name, t, shape, dev, _F32)
    return t.data_ptr()


def _device_of(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name}: tensor must be on a CUDA device")
    return t.get_device()


def _wanted(want, names):
    if isinstance(want, str) or any(w not in names for w in want):
        raise ValueError(f"want: expected names of {names}, got {want!r}")
    return want


class _Here:
    """No context to enter: the device is current and the call runs on its current stream."""

    def __enter__(self):
        pass

    def __exit__(self, *_):
        pass


class _There:
    """The device current and, with an explicit stream, that stream too: what is allocated inside belongs to it,
    and what the caller brings (inputs, ``out``, ``ws``) is not reused before its work on them is done."""

    def __init__(self, dev, stream, tensors):
        self.dev, self.stream, self.tensors = torch.cuda.device(dev), stream, tensors

    def __enter__(self):
        self.dev.__enter__()
        if self.stream is not None:
            self.outer = torch.cuda.stream(self.stream)
            self.outer.__enter__()

    def __exit__(self, *e):
        if self.stream is not None:
            self.outer.__exit__(*e)
            for t in self.tensors:
                if isinstance(t, torch.Tensor) and t.is_cuda and t.numel():  # (a refused one may be anything)
                    t.record_stream(self.stream)
        self.dev.__exit__(*e)


_HERE = _Here()


def _on(dev, stream, *tensors):
    if stream is None and dev == torch.cuda.current_device():
        return _HERE
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"stream: expected a stream of cuda:{dev}, got one of cuda:{stream.device_index}")
    return _There(dev, stream, tensors)


def _raw_stream(dev, stream):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _new(x, wanted, *shape):
    """A new tensor beside x and its address, or two Nones."""
    if not wanted:
        return None, None
    t = x.new_empty(shape)
    return t, t.data_ptr()


def _workspace(ws, nbytes, x):
    """(tensor to keep, address, bytes): the caller's workspace or a fresh one."""
    if ws is None:
        if not nbytes:
            return None, None, 0
        ws = x.new_empty(nbytes, dtype=torch.uint8)
    elif _device_of("ws", ws) != x.get_device():
        raise ValueError(f"ws: expected a tensor on {x.device}, got {ws.device}")
    elif not ws.is_contiguous():
        raise ValueError("ws: tensor must be contiguous")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _run(name, *args):
    st = getattr(L.lib(), name)(*args)
    if st:
        raise L.TPConvError(name, st)


class NodeGroups:
    """The nodes of a graph by type, computed once: ``perm`` [N] holds the node ids of type 0, 1, ...
    (ascending inside a type) and behind them those of no group (any type outside [0, n_types): padding),
    ``offsets`` [n_types + 1] where each type begins.  ``types`` is an int32 (or int64) vector on the device."""

    def __init__(self, types, n_types, stream=None):
        dev = _device_of("types", types)
        if types.dim() != 1 or types.dtype not in (torch.int32, torch.int64):
            raise ValueError("types: expected a vector of int32 or int64")
        n_types = int(n_types)
        if not 1 <= n_types <= L.MAX_TYPES:
            raise ValueError(f"n_types: expected 1..{L.MAX_TYPES}, got {n_types}")
        self.N, self.n_types, self.device, self._dev = types.numel(), n_types, types.device, dev
        with _on(dev, stream, types):
            if types.dtype == torch.int64:  # no wrap-around of far values into a type
                types = torch.where((types >= 0) & (types < n_types), types, -1).to(_I32)
            t = types.contiguous()
            self.perm = t.new_empty(self.N)
            self.offsets = t.new_empty(n_types + 1)
            _ws, wp, wn = _workspace(None, L.tpconv_group_workspace_size(self.N, n_types), t)
            _run("tpconv_group_nodes", self.N, n_types, t.data_ptr(), self.perm.data_ptr(), self.offsets.data_ptr(),
                 wp, wn, _raw_stream(dev, stream))
        self._perm, self._offsets = self.perm.data_ptr(), self.offsets.data_ptr()


# ---- typed linear map ---------------------------------------------------------------------------------


def _groups(plan, groups):
    if not isinstance(groups, NodeGroups):
        raise TypeError("groups: expected NodeGroups")
    if groups.n_types != plan.n_types:
        raise ValueError(f"groups: {groups.n_types} types, the plan has {plan.n_types}")
    N = groups.N
    return N, groups._dev, (N, plan.dim_in), (N, plan.dim_out), (plan.n_types, plan.weight_numel)


def linear_forward(plan, groups, x, weight, out=None, ws=None, stream=None):
    """out[N, dim_out]: every node's features times the weight of its type; rows of no group are zero."""
    N, dev, rin, rout, w = _groups(plan, groups)
    px, pw = _ptr("x", x, rin, dev), _ptr("weight", weight, w, dev)
    with _on(dev, stream, x, weight, groups.perm, groups.offsets, out, ws):
        if out is None:
            out, po = _new(x, True, *rout)
        else:
            po = _ptr("out", out, rout, dev)
        _ws, wp, wn = _workspace(ws, plan.workspace_bytes(L.OP_FORWARD, N), x)
        _run("tpconv_linear_forward", plan.handle, N, groups._perm, groups._offsets, px, pw, po, wp, wn,
             _raw_stream(dev, stream))
    return out


def linear_backward(plan, groups, x, weight, g, want=("dx", "dweight"), ws=None, stream=None):
    """{"dx": [N, dim_in], "dweight": [n_types, weight_numel]} for the cotangent g of the output."""
    N, dev, rin, rout, w = _groups(plan, groups)
    px, pw, pg = _ptr("x", x, rin, dev), _ptr("weight", weight, w, dev), _ptr("g", g, rout, dev)
    _wanted(want, ("dx", "dweight"))
    with _on(dev, stream, x, weight, g, groups.perm, groups.offsets, ws):
        dx, pdx = _new(x, "dx" in want, *rin)
        dw, pdw = _new(x, "dweight" in want, *w)
        _ws, wp, wn = _workspace(ws, plan.workspace_bytes(L.OP_BACKWARD, N), x)
        _run("tpconv_linear_backward", plan.handle, N, groups._perm, groups._offsets, px, pw, pg, pdx, pdw, wp, wn,
             _raw_stream(dev, stream))
    return {k: v for k, v in (("dx", dx), ("dweight", dw)) if v is not None}


def linear_double_backward(plan, groups, x, weight, g, gg_x=None, gg_weight=None, want=("d_g", "d_x", "d_weight"),
                           ws=None, stream=None):
    """Gradients of <gg_x, dx> + <gg_weight, dweight> by g, x and weight (a cotangent None = zero)."""
    N, dev, rin, rout, w = _groups(plan, groups)
    px, pw, pg = _ptr("x", x, rin, dev), _ptr("weight", weight, w, dev), _ptr("g", g, rout, dev)
    pa, pal = _ptr("gg_x", gg_x, rin, dev, True), _ptr("gg_weight", gg_weight, w, dev, True)
    _wanted(want, ("d_g", "d_x", "d_weight"))
    with _on(dev, stream, x, weight, g, gg_x, gg_weight, groups.perm, groups.offsets, ws):
        d_g, pdg = _new(x, "d_g" in want, *rout)
        d_x, pdx = _new(x, "d_x" in want, *rin)
        d_w, pdw = _new(x, "d_weight" in want, *w)
        _ws, wp, wn = _workspace(ws, plan.workspace_bytes(L.OP_DOUBLE_BACKWARD, N), x)
        _run("tpconv_linear_double_backward", plan.handle, N, groups._perm, groups._offsets, px, pw, pg, pa, pal, pdg,
             pdx, pdw, wp, wn, _raw_stream(dev, stream))
    return {k: v for k, v in (("d_g", d_g), ("d_x", d_x), ("d_weight", d_w)) if v is not None}


# ---- layer norm ----------------------------------------------------------------------------------------


def _rows(plan, x):
    dev = _device_of("x", x)
    if x.dim() != 2:
        raise ValueError(f"x: expected shape (N, {plan.dim}), got {tuple(x.shape)}")
    N = x.shape[0]
    rows = (N, plan.dim)
    return N, dev, rows, _ptr("x", x, rows, dev)


def norm_forward(plan, x, weight=None, bias=None, out=None, stream=None):
    """The layer norm of x[N, dim]; weight None stands for ones, bias None for zeros."""
    N, dev, rows, px = _rows(plan, x)
    pw = _ptr("weight", weight, (plan.weight_numel,), dev, True)
    pb = _ptr("bias", bias, (plan.bias_numel,), dev, True)
    with _on(dev, stream, x, weight, bias, out):
        if out is None:
            out, po = _new(x, True, *rows)
        else:
            po = _ptr("out", out, rows, dev)
        _run("tpconv_norm_forward", plan.handle, N, px, pw, pb, po, _raw_stream(dev, stream))
    return out


def norm_backward(plan, x, weight, g, want=("dx", "dweight", "dbias"), ws=None, stream=None):
    """{"dx", "dweight", "dbias"} for the cotangent g of the output."""
    N, dev, rows, px = _rows(plan, x)
    pw, pg = _ptr("weight", weight, (plan.weight_numel,), dev, True), _ptr("g", g, rows, dev)
    _wanted(want, ("dx", "dweight", "dbias"))
    with _on(dev, stream, x, weight, g, ws):
        dx, pdx = _new(x, "dx" in want, *rows)
        dw, pdw = _new(x, "dweight" in want, plan.weight_numel)
        db, pdb = _new(x, "dbias" in want, plan.bias_numel)
        _ws, wp, wn = _workspace(ws, plan.workspace_bytes(L.OP_BACKWARD, N), x)
        _run("tpconv_norm_backward", plan.handle, N, px, pw, pg, pdx, pdw, pdb, wp, wn, _raw_stream(dev, stream))
    return {k: v for k, v in (("dx", dx), ("dweight", dw), ("dbias", db)) if v is not None}


def norm_double_backward(plan, x, weight, g, gg_x=None, gg_weight=None, gg_bias=None,
                         want=("d_g", "d_x", "d_weight"), ws=None, stream=None):
    """Gradients of <gg_x, dx> + <gg_weight, dweight> + <gg_bias, dbias> by g, x and weight."""
    N, dev, rows, px = _rows(plan, x)
    nw = (plan.weight_numel,)
    pw, pg = _ptr("weight", weight, nw, dev, True), _ptr("g", g, rows, dev)
    pa, pal = _ptr("gg_x", gg_x, rows, dev, True), _ptr("gg_weight", gg_weight, nw, dev, True)
    pbe = _ptr("gg_bias", gg_bias, (plan.bias_numel,), dev, True)
    _wanted(want, ("d_g", "d_x", "d_weight"))
    with _on(dev, stream, x, weight, g, gg_x, gg_weight, gg_bias, ws):
        d_g, pdg = _new(x, "d_g" in want, *rows)
        d_x, pdx = _new(x, "d_x" in want, *rows)
        d_w, pdw = _new(x, "d_weight" in want, plan.weight_numel)
        _ws, wp, wn = _workspace(ws, plan.workspace_bytes(L.OP_DOUBLE_BACKWARD, N), x)
        _run("tpconv_norm_double_backward", plan.handle, N, px, pw, pg, pa, pal, pbe, pdg, pdx, pdw, wp, wn,
             _raw_stream(dev, stream))
    return {k: v for k, v in (("d_g", d_g), ("d_x", d_x), ("d_weight", d_w)) if v is not None}


# ---- torch autograd glue: as for the convolution, the backward of a backward is the library's double
# backward; a third derivative raises.  A backward computes the gradients of all inputs that require one, those too
# that torch.autograd.grad was not asked for: the context does not tell them apart ---------------------------------


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
