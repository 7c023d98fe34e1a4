"""64-bit references of the products of 8-bit integers and of gated blocks, and
the error bounds their results must keep, on CPU tensors."""
import math

import torch

from rows_reference import U32, half_step, stored

ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def quantize(X):
    """(Q int8, scale float32): the exact quotient decides, ties to even."""
    X = X.double()
    M, K = X.shape
    top = X.abs().amax(1) if K else torch.zeros(M, dtype=torch.float64)
    scale = (top / 127.0).float()
    bad = ~torch.isfinite(top)
    scale[bad] = math.nan
    s = scale.double()[:, None]
    on = (s > 0).expand(M, K)
    q = torch.zeros_like(X)
    q[on] = torch.round((X / s)[on])       # rounds halves to even
    return q.clamp(-127, 127).to(torch.int8), scale


def _ones(n, t, like):
    return torch.ones(n, dtype=torch.float64, device=like.device) if t is None else t.double()


def i8_sums(X, W, xs, ws):
    """(value, bound) of the scaled sums: the sum's rounding to fp32 and the two
    products with the scales."""
    S = X.double() @ W.double().t()
    S = S * _ones(X.shape[0], xs, X)[:, None] * _ones(W.shape[0], ws, X)[None, :]
    return S, 3.01 * U32 * S.abs()


def gemm_i8(X, W, Y, xs, ws, alpha, beta, dt):
    S, e = i8_sums(X, W, xs, ws)
    out, bound = alpha * S, abs(alpha) * (e + 1.01 * U32 * S.abs())
    if beta != 0:
        out = out + beta * Y.double()
        bound = bound + 1.01 * U32 * ((alpha * S).abs() + (beta * Y.double()).abs())
    return out, stored(bound, out, dt)


def act(name, g):
    """value, slope, and how far fp32 evaluations of them may be off.

    The exponential and erfc are within 4 units in the last place (8u), each
    product, sum and quotient adds u; where an argument t is itself rounded by r,
    exp(t) moves by r relative, and r is |t| times its relative rounding."""
    u = U32
    if name == "relu":
        on = (g > 0).double()
        return g * on, on, 0 * g, 0 * g
    if name == "silu":
        s, r = torch.sigmoid(g), torch.sigmoid(-g)
        v, d = g * s, s * (1 + g * r)
        return v, d, 14 * u * v.abs(), 30 * u * s * (1 + g.abs() * r)
    if name == "gelu":
        p = torch.special.ndtr(g)
        f = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        c = (16 + 4 * g * g) * u       # erfc's argument is rounded twice: (2 x^2 + 1) 2u
        return g * p, p + g * f, c * (g * p).abs(), 2 * c * (p + g.abs() * f)
    k = math.sqrt(8 / math.pi)
    t = k * (g + 0.044715 * g ** 3)
    s, r = torch.sigmoid(t), torch.sigmoid(-t)
    tail = g * s * r * k * (1 + 3 * 0.044715 * g * g)
    c = (20 + 6 * t.abs()) * u
    return g * s, s + tail, c * (g * s).abs(), 2 * c * (s + tail.abs())


def glu(X, W, name, dt, xs=None, ws=None):
    """{"H": (value, bound), "Z": ...}"""
    if X.dtype == torch.int8:
        Z, e = i8_sums(X, W, xs, ws)
    else:
        K = X.shape[1]
        X, W = X.double(), W.double()
        Z, e = X @ W.t(), 4 * (K + 4) * U32 * (X.abs() @ W.abs().t())
    F = W.shape[0] // 2
    g, u, eg, eu = Z[:, :F], Z[:, F:], e[:, :F], e[:, F:]
    a, _, ea, _ = act(name, g)
    ea = ea + 1.2 * eg                 # no activation's slope passes 1.13
    H = a * u
    bound = ea * (u.abs() + eu) + a.abs() * eu + 1.01 * U32 * H.abs()
    return {"H": (H, stored(bound, H, dt)), "Z": (Z, stored(e, Z, dt))}


def glu_grad(dH, X, W, Z, name, dX, dW, beta_x, beta_w, dw_dt):
    """{"dX": (value, bound), "dW": ...}; Z None: from X and W."""
    dt = X.dtype
    M, K = X.shape
    F = dH.shape[1]
    X, W, dH = X.double(), W.double(), dH.double()
    if Z is None:
        Z, e = X @ W.t(), 4 * (K + 4) * U32 * (X.abs() @ W.abs().t())
    else:
        Z, e = Z.double(), torch.zeros_like(Z, dtype=torch.float64)
    g, u, eg, eu = Z[:, :F], Z[:, F:], e[:, :F], e[:, F:]
    a, d, ea, ed = act(name, g)
    ea = ea + 1.2 * eg
    ed = ed + 1.0 * eg                 # no second derivative passes 0.8
    if name == "relu":
        ed = ed + (g.abs() <= eg) * (eg > 0)
    D = torch.cat((dH * u * d, dH * a), 1)
    eD = torch.cat((dH.abs() * (u.abs() * ed + eu * (d.abs() + ed)), dH.abs() * ea), 1)
    eD = stored(eD + 3 * U32 * D.abs(), D, dt)
    out = {}
    for n, (A, eA, B, old, beta, t) in {"dX": (D, eD, W, dX, beta_x, dt),
                                        "dW": (D.t(), eD.t(), X, dW, beta_w, dw_dt)}.items():
        v = A @ B
        bound = eA @ B.abs() + 4 * (A.shape[1] + 4) * U32 * ((A.abs() + eA) @ B.abs())
        if beta != 0:
            v = v + beta * old.double()
            bound = bound + 4 * U32 * (beta * old.double()).abs()
        out[n] = (v, stored(bound, v, t))
    return out


__all__ = ["ACTS", "act", "gemm_i8", "glu", "glu_grad", "half_step", "i8_sums", "quantize"]
