"""64-bit references of the products whose rows choose their own weights, and
the error bounds their results must keep, on CPU tensors."""
import torch

U32 = 2.0 ** -24                      # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def stored(bound, value, dtype):
    """A bound on a value before it is rounded to dtype, as one on the result."""
    eta = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -150
    return bound * (1 + half_step(dtype)) + half_step(dtype) * value.abs() + eta


def chosen(rows, L):
    """[(adapter, its rows)]"""
    return [(a, (rows == a).nonzero()[:, 0]) for a in range(L)]


def ranks_of(ranks, L, R):
    return [R] * L if ranks is None else [min(max(int(r), 0), R) for r in ranks]


def scales_of(scale, L):
    return [1.0] * L if scale is None else [float(s) for s in scale.double()]


def lora(X, W, A, B, rows, Y, scale, ranks, alpha, beta):
    """(Y, bound): the result in 64 bits and how far a call's may be off.
    Sums of K + R terms in fp32: 4*(K+R+4)*u of the sum of magnitudes."""
    M, K = X.shape
    L, R = A.shape[:2]
    dt = X.dtype
    X, W, A, B = X.double(), W.double(), A.double(), B.double()
    out, mag = X @ W.t(), X.abs() @ W.abs().t()
    rk, sc = ranks_of(ranks, L, R), scales_of(scale, L)
    for a, at in chosen(rows, L):
        if not at.numel() or not rk[a]:
            continue
        down, up = A[a, :rk[a]], B[a, :, :rk[a]]
        out[at] += sc[a] * ((X[at] @ down.t()) @ up.t())
        mag[at] += abs(sc[a]) * ((X[at].abs() @ down.abs().t()) @ up.abs().t())
    bound = 4 * (K + R + 4) * U32 * abs(alpha) * mag
    out = alpha * out
    if beta != 0:
        out = out + beta * Y.double()
        bound = bound + 4 * U32 * (beta * Y.double()).abs()
    return out, stored(bound, out, dt)


def lora_grad(dY, X, W, A, B, rows, dX, dA, dB, scale, ranks, alpha, beta_x, beta_ab):
    """{"dX": (value, bound), ...}: each sum of n fp32 terms 4*(n+4)*u, and the
    inner product's own where one sum feeds another."""
    M, K = X.shape
    N = W.shape[0]
    L, R = A.shape[:2]
    dt = X.dtype
    dY, X, W, A, B = (t.double() for t in (dY, X, W, A, B))
    ox, mx = dY @ W, dY.abs() @ W.abs()
    oa, ma = torch.zeros(L, R, K).double(), torch.zeros(L, R, K).double()
    ob, mb = torch.zeros(L, N, R).double(), torch.zeros(L, N, R).double()
    rk, sc = ranks_of(ranks, L, R), scales_of(scale, L)
    for a, at in chosen(rows, L):
        r = rk[a]
        if not at.numel() or not r:
            continue
        down, up = A[a, :r], B[a, :, :r]
        G, g = sc[a] * (dY[at] @ up), abs(sc[a]) * (dY[at].abs() @ up.abs())
        ox[at] += G @ down
        mx[at] += g @ down.abs()
        oa[a, :r] = G.t() @ X[at]
        ma[a, :r] = g.t() @ X[at].abs()
        ob[a, :, :r] = sc[a] * (dY[at].t() @ (X[at] @ down.t()))
        mb[a, :, :r] = abs(sc[a]) * (dY[at].abs().t() @ (X[at].abs() @ down.abs().t()))

    def done(out, mag, n, beta, old, dtype):
        out, bound = alpha * out, 4 * (n + 4) * U32 * abs(alpha) * mag
        if beta != 0:
            out = out + beta * old.double()
            bound = bound + 4 * U32 * (beta * old.double()).abs()
        return out, stored(bound, out, dtype)
    return {"dX": done(ox, mx, N + R, beta_x, dX, dt),
            "dA": done(oa, ma, M + N, beta_ab, dA, torch.float32),
            "dB": done(ob, mb, M + K, beta_ab, dB, torch.float32)}


def moe(X, router, W1, W2, top_k, Y, renorm, alpha, beta):
    """(Y, its bound, ids, weights, their bound).

    g and u: sums of D terms, 4*D*u of the magnitudes.  silu's slope is at most
    1.1 and its value and the product add a few units.  fp16: h is then held
    in 11 bits with its block's exponent: half a step of fp16 of its own value,
    or 2^-24 of the largest of its row.  The sum over F and the choices: 4*(F+k+4)*u.  A
    weight's exponent is a difference of 64-bit logits rounded to fp32, u of
    it, and exp and the quotient add some units."""
    M, D = X.shape
    E, _, F = W2.shape
    dt = X.dtype
    X, router, W1, W2 = (t.double() for t in (X, router, W1, W2))
    logits = X @ router.t()
    key = torch.where(logits.isnan(), torch.full_like(logits, -float("inf")), logits)
    ids = torch.empty(M, top_k, dtype=torch.int64)
    for t in range(M):
        ids[t] = torch.tensor(sorted(range(E), key=lambda e: (-float(key[t, e]), e))[:top_k])
    top = key.gather(1, ids)
    base = key.max(dim=1, keepdim=True).values
    w = (top - base).exp()
    w = w / (w.sum(1, keepdim=True) if renorm else (key - base).exp().sum(1, keepdim=True))
    dw = w * 2 * U32 * ((key - base).abs().max(dim=1, keepdim=True).values + E + 16)
    out, bound = torch.zeros(M, D).double(), torch.zeros(M, D).double()
    for t in range(M):
        for j in range(top_k):
            e = int(ids[t, j])
            h, dh = W1[e] @ X[t], 4 * (D + 4) * U32 * (W1[e].abs() @ X[t].abs())
            g, u, dg, du = h[:F], h[F:], dh[:F], dh[F:]
            s = g * torch.sigmoid(g)
            a = s * u
            da = 1.1 * dg * (u.abs() + du) + s.abs() * du + 16 * U32 * a.abs()
            if dt == torch.float16:
                da = da + half_step(dt) * (a.abs() + da) + 2.0 ** -24 * (a.abs() + da).max()
            y, m = W2[e] @ a, W2[e].abs() @ a.abs()
            out[t] += w[t, j] * y
            bound[t] += w[t, j] * (W2[e].abs() @ da + 4 * (F + top_k + 4) * U32 * m) \
                + dw[t, j] * m
    out, bound = alpha * out, abs(alpha) * bound
    if beta != 0:
        out = out + beta * Y.double()
        bound = bound + 4 * U32 * (beta * Y.double()).abs()
    return out, stored(bound, out, dt), ids, w, dw + U32 * w


def worst(got, want, bound):
    """The largest |got - want| / bound; infinite where one is finite and the
    other is not."""
    got = got.double().cpu()
    fine = torch.isfinite(want)
    if not torch.equal(fine, torch.isfinite(got)):
        return float("inf")
    if not fine.any():
        return 0.0
    return float(((got - want).abs()[fine] / bound[fine].clamp_min(1e-300)).max())
