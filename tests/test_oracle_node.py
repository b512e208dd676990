"""Pins of the node operators' oracle: its gradients against central differences of its forwards (first order)
and of its gradients (second order), the plain layer norm of torch in fp64,
equivariance under rotations, and closed cases."""

import numpy as np
import pytest

from oracle import node as O
from oracle import so3

EPS = 1e-3
IRREPS = ["5x0e", "3x0e+2x1o", "4x0e+3x0o+2x1o+1x2e+2x1e", "2x2e+2x3o", "1x0e", "3x1o+2x1o"]


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def diff(f, z, v, h=1e-6):
    """central difference of the scalar f at z along v"""
    return (f(z + h * v) - f(z - h * v)) / (2 * h)


@pytest.mark.parametrize("irreps", IRREPS)
def test_norm_gradients_match_differences(irreps):
    r = rng(1)
    nw, nb = O.norm_sizes(irreps)
    dim = O.blocks(irreps)[1]
    x, g, a = r.normal(size=(3, 6, dim))
    w, al = r.normal(size=(2, nw))
    b, be = r.normal(size=(2, nb))
    dx, dw, db = O.norm_backward(irreps, x, w, g, EPS)
    L = lambda x, w, b: (g * O.norm(irreps, x, w, b, EPS)).sum()  # noqa: E731
    vx, vw, vb = r.normal(size=x.shape), r.normal(size=nw), r.normal(size=nb)
    assert np.isclose(diff(lambda t: L(t, w, b), x, vx), (dx * vx).sum(), rtol=1e-6, atol=1e-7)
    assert np.isclose(diff(lambda t: L(x, t, b), w, vw), (dw * vw).sum(), rtol=1e-6, atol=1e-7)
    if nb:
        assert np.isclose(diff(lambda t: L(x, w, t), b, vb), (db * vb).sum(), rtol=1e-6, atol=1e-7)

    def psi(g, x, w):
        p, q, s = O.norm_backward(irreps, x, w, g, EPS)
        return (a * p).sum() + (al * q).sum() + (be * s).sum()

    d_g, d_x, d_w = O.norm_double_backward(irreps, x, w, g, a, al, be, EPS)
    vg = r.normal(size=g.shape)
    assert np.isclose(diff(lambda t: psi(t, x, w), g, vg), (d_g * vg).sum(), rtol=1e-6, atol=1e-6)
    assert np.isclose(diff(lambda t: psi(g, t, w), x, vx), (d_x * vx).sum(), rtol=1e-5, atol=1e-5)
    assert np.isclose(diff(lambda t: psi(g, x, t), w, vw), (d_w * vw).sum(), rtol=1e-6, atol=1e-6)


@pytest.mark.parametrize("c", [1, 2, 7])
def test_norm_of_scalars_is_the_plain_layer_norm(c):
    torch = pytest.importorskip("torch")
    r = rng(2)
    x, w, b = r.normal(size=(4, c)), r.normal(size=c), r.normal(size=c)
    t = torch.tensor(x, requires_grad=True)
    y = torch.nn.functional.layer_norm(t, (c,), torch.tensor(w), torch.tensor(b), EPS)
    assert np.allclose(y.detach().numpy(), O.norm(f"{c}x0e", x, w, b, EPS), atol=1e-12)
    g = r.normal(size=x.shape)
    y.backward(torch.tensor(g))
    assert np.allclose(t.grad.numpy(), O.norm_backward(f"{c}x0e", x, w, g, EPS)[0], atol=1e-10)


def test_norm_of_zero_rows_is_the_bias():
    irreps = "3x0e+2x1o"
    b = np.array([1.0, -2.0, 3.0])
    y = O.norm(irreps, np.zeros((2, 9)), np.ones(5), b, EPS)
    assert np.array_equal(y, np.tile(np.r_[b, np.zeros(6)], (2, 1)))


def rotate(irreps, x, R):
    y = np.empty_like(x)
    for o, mul, d, l, p in O.blocks(irreps)[0]:
        D = so3.wigner_D_lstsq(l, R)
        y[:, o:o + mul * d] = np.einsum("ab,nub->nua", D,
                                        x[:, o:o + mul * d].reshape(-1, mul, d)).reshape(len(x), -1)
    return y


def random_rotation(r):
    q, _ = np.linalg.qr(r.normal(size=(3, 3)))
    return q * np.sign(np.linalg.det(q))


@pytest.mark.parametrize("irreps", IRREPS)
def test_norm_and_linear_are_equivariant(irreps):
    r = rng(3)
    R = random_rotation(r)
    nw, nb = O.norm_sizes(irreps)
    x = r.normal(size=(5, O.blocks(irreps)[1]))
    w, b = r.normal(size=nw), r.normal(size=nb)
    assert np.allclose(O.norm(irreps, rotate(irreps, x, R), w, b, EPS), rotate(irreps, O.norm(irreps, x, w, b, EPS), R),
                       atol=1e-9)
    t = np.array([0, 1, 1, -1, 0])
    lw = r.normal(size=(2, O.linear_paths(irreps, irreps)[1]))
    assert np.allclose(O.linear(irreps, irreps, t, rotate(irreps, x, R), lw),
                       rotate(irreps, O.linear(irreps, irreps, t, x, lw), R), atol=1e-9)


@pytest.mark.parametrize("irr", [("3x0e+2x1o", "4x0e+1x1o"), ("2x0e+3x0e+1x2e", "2x2e+5x0e+2x0o"), ("4x1o", "4x1e")])
def test_linear_gradients_match_differences(irr):
    r = rng(4)
    di, do = O.blocks(irr[0])[1], O.blocks(irr[1])[1]
    n, T, nw = 7, 3, O.linear_paths(*irr)[1]
    t = np.array([0, 2, 2, -1, 0, 5, 2])  # type 1 empty, nodes 3 and 5 in no group
    x, a = r.normal(size=(2, n, di))
    w, al = r.normal(size=(2, T, nw))
    g = r.normal(size=(n, do))
    dx, dw = O.linear_backward(*irr, t, x, w, g)
    vx, vw, vg = r.normal(size=x.shape), r.normal(size=w.shape), r.normal(size=g.shape)
    L = lambda x, w: (g * O.linear(*irr, t, x, w)).sum()  # noqa: E731
    assert np.isclose(diff(lambda z: L(z, w), x, vx), (dx * vx).sum(), atol=1e-6)
    assert np.isclose(diff(lambda z: L(x, z), w, vw), (dw * vw).sum(), atol=1e-6)
    assert not dx[[3, 5]].any() and not dw[1].any() and not O.linear(*irr, t, x, w)[[3, 5]].any()

    def psi(g, x, w):
        p, q = O.linear_backward(*irr, t, x, w, g)
        return (a * p).sum() + (al * q).sum()

    d_g, d_x, d_w = O.linear_double_backward(*irr, t, x, w, g, a, al)
    assert np.isclose(diff(lambda z: psi(z, x, w), g, vg), (d_g * vg).sum(), atol=1e-6)
    assert np.isclose(diff(lambda z: psi(g, z, w), x, vx), (d_x * vx).sum(), atol=1e-6)
    assert np.isclose(diff(lambda z: psi(g, x, z), w, vw), (d_w * vw).sum(), atol=1e-6)


def test_grouping_by_hand():
    perm, off = O.group(np.array([2, 0, -1, 2, 7, 0, 1]), 3)
    assert perm.tolist() == [1, 5, 6, 0, 3, 2, 4] and off.tolist() == [0, 2, 3, 5]
