"""Plain fp64 forms of the dense products with epilogues, of the gated block and of their
gradients, with bounds on the error a computation in fp32 makes before its final rounding.

The bounds.  U = 2^-24 is half a step of fp32, U8 = 2^-8 half a step of bf16, both relative
to the value.  A sum of n products in fp32, in any order, is off by at most (n + 4) U times
the sum of the products' magnitudes (four for the bias, the residual and the operands'
products).  The activations are evaluated through e^x and 1/x, each within a few steps, and
e^x with x rounded, which costs |x| U more; the exponents are |z| (silu), z^2/2 (gelu) and
1.6 |z| + 0.072 |z|^3 (gelu_tanh), so 4 U (8 + z^2 + |z|^3 / 8) relative to the magnitudes of
the terms covers all three (2^-126 for what underflows).

CUT.  The e4m3 matrix instruction first adds groups of eight consecutive products, cut off
13 bits below 2^(ea + eb) of the group's leading product (ea, eb the exponents of its
factors): 256 * 256 + 4 gives 256 * 256 and 256 * 256 + 8 is exact, 240 * 240 + 1 gives
240 * 240 and + 2 is exact, while a 1 in the next group of eight is kept beside 448 * 448.
The leading product itself has 8 bits and loses nothing, so a group of products p loses less
than 7 * 2^-13 max |p|, and a row at most CUT = 7 * 2^-13 times the sum of the magnitudes.
(e2m1 products are multiples of 1/4 up to 36, 8 bits: nothing is cut.)"""
import numpy as np
from scipy.special import erfc, expit

U, U8 = 2.0 ** -24, 2.0 ** -8
CUT = 7 * 2.0 ** -13
C, A3 = np.sqrt(2 / np.pi), 0.044715


def f(z, act):
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "silu":
        return z * expit(z)
    if act == "gelu":
        return 0.5 * z * erfc(-z * np.sqrt(0.5))
    if act == "gelu_tanh":
        return z * expit(2 * C * (z + A3 * z ** 3))      # (1 + tanh(u) = 2 / (1 + e^-2u), which cancels nothing)
    return z


def df(z, act):
    """f' and the sum of its terms' magnitudes."""
    if act == "relu":
        d = (z > 0).astype(np.float64)
        return d, d
    if act == "silu":
        s = expit(z)
        return s + z * s * (1 - s), s + np.abs(z) * s * (1 - s)
    if act == "gelu":
        p, q = 0.5 * erfc(-z * np.sqrt(0.5)), z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
        return p + q, p + np.abs(q)
    if act == "gelu_tanh":
        s = expit(2 * C * (z + A3 * z ** 3))
        q = z * s * (1 - s) * 2 * C * (1 + 3 * A3 * z * z)
        return s + q, s + np.abs(q)
    return np.ones_like(z), np.ones_like(z)


def _eval(z, act):
    """Relative error of evaluating f or f' (against the sum of its terms)."""
    if act in ("none", "relu"):
        return np.zeros_like(z)
    return 4 * U * (8 + z * z + np.abs(z) ** 3 / 8)


def _f_err(z, ez, act):
    """Error of f(z) from an error ez of z (the slopes stay below 1.13) and its evaluation."""
    return 1.13 * ez + _eval(z, act) * np.abs(f(z, act)) + 2.0 ** -120


def act_forward(z, mag, K, bias=None, act="none", residual=None, cut=0.0):
    """(D, its bound, Z, its bound) from the exact sums z = A B^T and mag, a bound on the sums
    of the products' magnitudes; cut: CUT for e4m3 operands."""
    b = 0.0 if bias is None else bias[None]
    z = z + b
    ez = (K + 4) * U * (mag + np.abs(b)) + cut * mag
    d, e = f(z, act), _f_err(z, ez, act)
    if residual is not None:
        d = d + residual
        e = e + U * np.abs(d)
    return d, e, z, ez


def glu_forward(z, mag, K, act="silu"):
    """(H, bound, Z, bound) from z = X W13^T."""
    i = z.shape[1] // 2
    ez = (K + 4) * U * mag
    g, u = z[:, :i], z[:, i:]
    fe = _f_err(g, ez[:, :i], act)
    h = f(g, act) * u
    return h, fe * np.abs(u) + (np.abs(f(g, act)) + fe) * ez[:, i:] + 2 * U * np.abs(h), z, ez


def _products(dz, edz, A, B):
    """(dA, bound, dB, bound) from dz and the error of the bf16 dz that enters the products."""
    M, N = dz.shape
    a = np.abs(dz) + edz
    return (dz @ B, edz @ np.abs(B) + (N + 4) * U * (a @ np.abs(B)),
            dz.T @ A, edz.T @ np.abs(A) + (M + 4) * U * (a.T @ np.abs(A)))


def act_backward(dD, z, A, B, act="none"):
    """((dA, bound), (dB, bound), (dbias, bound)); z is the bf16 pre-activation's value."""
    d, terms = df(z, act)
    dz = dD * d
    e = np.abs(dD) * (_eval(z, act) * terms + 2 * U * np.abs(d) + 2.0 ** -120)
    dA, ea, dB, eb = _products(dz, e + U8 * (np.abs(dz) + e), A, B)
    db = dz.sum(0)
    return (dA, ea), (dB, eb), (db, e.sum(0) + (dD.shape[0] + 4) * U * (np.abs(dz) + e).sum(0))


def glu_backward(dH, z, X, W13, act="silu"):
    """((dX, bound), (dW13, bound))."""
    i = z.shape[1] // 2
    g, u = z[:, :i], z[:, i:]
    d, terms = df(g, act)
    dz = np.concatenate([dH * u * d, dH * f(g, act)], 1)
    eg = np.abs(dH * u) * (_eval(g, act) * terms + 3 * U * np.abs(d) + 2.0 ** -120)
    eu = np.abs(dH) * (_f_err(g, 0.0, act) + 2 * U * np.abs(f(g, act)))
    e = np.concatenate([eg, eu], 1)
    dX, ex, dW, ew = _products(dz, e + U8 * (np.abs(dz) + e), X, W13)
    return (dX, ex), (dW, ew)
