"""Products of 8-bit integers and gated feed-forward blocks, as they are measured:

  i8        rows to 8-bit integers with a scale each, and their product with
            8-bit weights: Y = xs[m] ws[n] (Q W^T), the sum in whole numbers
  glu       a gated block: [G U] = X W^T, H = act(G) * U, in floating point or
            in 8-bit integers; with [G U] kept where a backward pass follows
  glu_grad  its gradients dX and dW, from the kept [G U] or without it

`run` computes them in their plain form (elementary torch operations in 32
bits), or with this library's calls where `own` is true.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def _i8(name, M, N, K, dtype="f16", pad=0, given=False):
    """dtype: of the activations and of Y; given: the rows come in 8 bits
    already; pad: bytes between the rows of Q and W, elements between X's."""
    return {"name": name, "op": "i8", "dtype": dtype, "M": M, "N": N, "K": K, "pad": pad,
            "given": given}


def _glu(name, M, F, K, dtype="f16", pad=0, act="silu", kept=False, i8=False, op="glu"):
    """kept: [G U] is written (glu), or given (glu_grad)."""
    return {"name": name, "op": op, "dtype": dtype, "M": M, "F": F, "K": K, "pad": pad,
            "act": act, "kept": kept, "i8": i8}


def listed():
    return [
        # one token through a small projection: all latency
        _i8("i8_token", 1, 1024, 1024),
        # a decode step of 48 requests on a large projection
        _i8("i8_decode", 48, 4096, 4096),
        # the prompts of a batch
        _i8("i8_prompt", 4096, 4096, 4096),
        # rows that another step left in 8 bits; odd lengths, unaligned rows, fp32 results
        _i8("i8_ragged_f32", 1000, 3000, 517, dtype="f32", pad=3, given=True),
        # one token through a small block
        _glu("glu_token", 1, 1024, 1024),
        # a decode step of 48 requests, weights and tokens in 8 bits
        _glu("glu_decode_i8", 48, 8192, 4096, i8=True),
        # forward pass of a training step: [G U] is kept
        _glu("glu_train", 4096, 8192, 4096, kept=True),
        # prompts in 8 bits, the tanh form of gelu
        _glu("glu_prompt_i8", 2048, 8192, 4096, i8=True, act="gelu_tanh"),
        # fp32, odd lengths, rows that do not start aligned
        _glu("glu_ragged_f32", 1000, 1500, 517, dtype="f32", pad=2, act="gelu"),
        # backward pass of a small batch that kept nothing: G and U once more
        _glu("glu_grad_small", 257, 1024, 1024, op="glu_grad"),
        # backward pass of a large batch
        _glu("glu_grad_batch", 4096, 4096, 4096, kept=True, op="glu_grad"),
        # fp32, odd lengths, unaligned rows
        _glu("glu_grad_ragged_f32", 1000, 1500, 517, dtype="f32", pad=2, act="gelu", kept=True,
             op="glu_grad"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _size(rng, lo, hi):
    """Mostly multiples of 64 (as projections have), else any number."""
    n = _log(rng, lo, hi)
    return max(lo, n // 64 * 64) if rng.random() < 0.6 else n


def draw(rng):
    most = {op: max(work(c)["flops"] for c in listed() if c["op"] == op)
            for op in ("i8", "glu", "glu_grad")}
    while True:
        op = rng.choice(("i8", "i8", "glu", "glu", "glu_grad"))
        dtype = "f32" if rng.random() < 0.25 else "f16"
        pad = rng.choice((0, 0, 0, 1, 8))
        M = _log(rng, 16 if op == "glu_grad" else 1, 4096)
        K = _size(rng, 256, 8192)
        if op == "i8":
            c = _i8("", M, _size(rng, 256, 8192), K, dtype, pad, rng.random() < 0.3)
        else:
            c = _glu("", M, _size(rng, 256, 8192), K, dtype, pad,
                     rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu")),
                     rng.random() < 0.5, op == "glu" and rng.random() < 0.4, op)
            if c["i8"]:
                c["kept"] = False
        # an fp32 product costs some eight times an fp16 one of its size
        slow = 8 if dtype == "f32" and op != "i8" and not c["i8"] else 1
        if work(c)["flops"] * slow <= most[op]:
            del c["name"]
            return c


def work(case):
    c = case
    eb = 2 if c["dtype"] == "f16" else 4
    M, K = c["M"], c["K"]
    if c["op"] == "i8":
        N = c["N"]
        return {"bytes": (1.0 if c["given"] else eb) * M * K + 1.0 * N * K + eb * M * N
                + 4.0 * (M + N), "flops": 2.0 * M * N * K}
    F = c["F"]
    if c["op"] == "glu":
        wb = 1 if c["i8"] else eb
        return {"bytes": eb * (1.0 * M * K + M * F * (3 if c["kept"] else 1)) + wb * 2.0 * F * K
                + (4.0 * (M + 2 * F) if c["i8"] else 0.0), "flops": 4.0 * M * F * K}
    return {"bytes": eb * (1.0 * M * F * (3 if c["kept"] else 1) + 2.0 * M * K + 4.0 * F * K),
            "flops": (8.0 if c["kept"] else 12.0) * M * F * K}


# ------------------------------------------------------------------ inputs

def _rows_of(gen, rows, cols, dtype, pad, std=1.0):
    """A rows x cols matrix of normal numbers, `pad` elements between its rows."""
    t = torch.randn(rows, cols + pad, generator=gen, device=gen.device)
    return t.mul_(std).to(dtype)[:, :cols]


def _room(rows, cols, dtype, pad, dev):
    return torch.empty(rows, cols + pad, dtype=dtype, device=dev)[:, :cols]


def _tokens(gen, rows, cols, dtype, pad):
    """Activations as a norm layer leaves them: rows of a like size, a few
    columns larger than the others."""
    t = _rows_of(gen, rows, cols, torch.float32, pad)
    t *= 0.5 + torch.rand(rows, 1, generator=gen, device=gen.device)
    wide = torch.rand(cols, generator=gen, device=gen.device) < 0.01
    t *= torch.where(wide, 6.0, 1.0)
    out = _room(rows, cols, dtype, pad, gen.device)
    return out.copy_(t)


def _in_8_bits(gen, rows, cols, pad):
    """Weights in 8 bits and each row's scale."""
    t = torch.randn(rows, cols, generator=gen, device=gen.device).div_(math.sqrt(cols))
    scale = t.abs().amax(1) / 127.0
    q = _room(rows, cols, torch.int8, pad, gen.device)
    q.copy_((t / scale[:, None]).round_())
    return q, scale


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, pad = DTYPES[c["dtype"]], c["pad"]
    M, K = c["M"], c["K"]
    s = {"op": c["op"]}
    i8 = c["op"] == "i8" or c["i8"]
    if i8:
        if c.get("given"):
            s["Q"], s["xs"] = _in_8_bits(gen, M, K, pad)
            s["xs"] *= math.sqrt(K)
        else:
            s["X"] = _tokens(gen, M, K, dt, pad)
            s["Q"] = _room(M, K, torch.int8, pad, dev)
            s["xs"] = torch.empty(M, dtype=torch.float32, device=dev)
    if c["op"] == "i8":
        s["W"], s["ws"] = _in_8_bits(gen, c["N"], K, pad)
        s["Y"] = _room(M, c["N"], dt, pad, dev)
        return s
    F = c["F"]
    s["act"], s["i8"] = c["act"], c["i8"]
    if i8:
        s["W"], s["ws"] = _in_8_bits(gen, 2 * F, K, pad)
    else:
        s["X"] = _rows_of(gen, M, K, dt, pad)
        # gate rows, then up rows
        s["W"] = _rows_of(gen, 2 * F, K, dt, pad, 1.0 / math.sqrt(K))
    if c["op"] == "glu":
        s["H"] = _room(M, F, dt, pad, dev)
        s["Z"] = _room(M, 2 * F, dt, pad, dev) if c["kept"] else None
        return s
    s["dH"] = _rows_of(gen, M, F, dt, pad, 0.05)
    s["Z"] = None
    if c["kept"]:
        s["Z"] = _room(M, 2 * F, dt, pad, dev)
        s["Z"].copy_(s["X"].float() @ s["W"].float().t())
    s["dX"] = _room(M, K, dt, pad, dev)
    s["dW"] = _room(2 * F, K, dt, pad, dev)
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_quantize(X):
    """A quotient may lie next to the border of two whole numbers: 64 bits."""
    top = X.float().abs().amax(1)
    # by a tensor: a division by a number is a product with its reciprocal
    scale = torch.where(top.isfinite(), top / torch.full_like(top, 127.0), math.nan)
    q = (X.double() / scale.double()[:, None]).round().nan_to_num(0.0, 0.0, 0.0)
    return q.float(), scale


def _plain_act(act, g):
    """act(g) and its derivative."""
    if act == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if act == "silu":
        s = 1.0 / (1.0 + (-g).exp())
        return g * s, s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        # the normal distribution's function, with no digits lost at its low end
        p = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * p, p + g * (-0.5 * g * g).exp() / math.sqrt(2.0 * math.pi)
    k = math.sqrt(8.0 / math.pi)
    s = 1.0 / (1.0 + (-k * (g + 0.044715 * g * g * g)).exp())
    return g * s, s + g * s * (1.0 - s) * k * (1.0 + 3 * 0.044715 * g * g)


def _plain_rows(s):
    """The rows in 8 bits as numbers, and their scales."""
    return _plain_quantize(s["X"]) if "X" in s else (s["Q"].float(), s["xs"])


def _plain_i8(s):
    Q, xs = _plain_rows(s)
    Y = (Q @ s["W"].float().t()) * xs[:, None] * s["ws"][None, :]
    return {"Y": Y.to(s["Y"].dtype), "scale": xs}


def _plain_glu(s):
    dt = s["H"].dtype
    F = s["W"].shape[0] // 2
    if s["i8"]:
        Q, xs = _plain_rows(s)
        Z = (Q @ s["W"].float().t()) * xs[:, None] * s["ws"][None, :]
    else:
        Z = s["X"].float() @ s["W"].float().t()
    H = _plain_act(s["act"], Z[:, :F])[0] * Z[:, F:]
    out = {"H": H.to(dt)}
    if s["Z"] is not None:
        out["Z"] = Z.to(dt)
    return out


def _plain_glu_grad(s):
    dt = s["X"].dtype
    F = s["dH"].shape[1]
    X, W, dH = s["X"].float(), s["W"].float(), s["dH"].float()
    Z = X @ W.t() if s["Z"] is None else s["Z"].float()
    a, slope = _plain_act(s["act"], Z[:, :F])
    dZ = torch.cat((dH * Z[:, F:] * slope, dH * a), 1)
    return {"dX": (dZ @ W).to(dt), "dW": (dZ.t() @ X).to(dt)}


def run(state):
    s = state
    if own:
        import dense_gemm_fp32_amd as dg
        if s["op"] == "glu_grad":
            dg.glu_grad(s["dH"], s["X"], s["W"], dX=s["dX"], dW=s["dW"], act=s["act"], Z=s["Z"])
            return {"dX": s["dX"], "dW": s["dW"]}
        if s["op"] == "glu" and not s["i8"]:
            dg.glu(s["X"], s["W"], s["H"], act=s["act"], Z=s["Z"])
            return {"H": s["H"]} if s["Z"] is None else {"H": s["H"], "Z": s["Z"]}
        if "X" in s:
            dg.quantize(s["X"], s["Q"], s["xs"])
        if s["op"] == "glu":
            return {"H": dg.glu(s["Q"], s["W"], s["H"], act=s["act"], x_scale=s["xs"],
                                w_scale=s["ws"])}
        dg.gemm_i8(s["Q"], s["W"], s["Y"], x_scale=s["xs"], w_scale=s["ws"])
        return {"Y": s["Y"], "scale": s["xs"]}
    return {"i8": _plain_i8, "glu": _plain_glu, "glu_grad": _plain_glu_grad}[s["op"]](s)


# ------------------------------------------------------------------ in 64 bits

def _exact_rows(s):
    if "X" not in s:
        return s["Q"].double(), s["xs"].double()
    X = s["X"].double()
    # a row's scale is a 32-bit number
    scale = (X.abs().max(dim=1).values / 127).float().double()
    q = torch.where(scale[:, None] > 0, X / scale[:, None], torch.zeros_like(X))
    low = q.floor()
    up = (q - low > 0.5) | ((q - low == 0.5) & (low.remainder(2) == 1))
    return low + up, scale


def _exact_act(act, g):
    if act == "relu":
        return g.clamp(min=0), torch.where(g > 0, 1.0, 0.0).double()
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == "gelu":
        p = torch.special.ndtr(g)
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))
    inner = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * inner


def exact(case, seed):
    s = prepare(case, seed)
    W = s["W"].double()
    if s["op"] == "i8":
        q, xs = _exact_rows(s)
        return {"Y": torch.outer(xs, s["ws"].double()) * (q @ W.t()), "scale": xs}
    F = W.shape[0] // 2
    if s["op"] == "glu":
        if s["i8"]:
            q, xs = _exact_rows(s)
            x, W = q * xs[:, None], W * s["ws"].double()[:, None]
        else:
            x = s["X"].double()
        G, U = x @ W[:F].t(), x @ W[F:].t()
        H = _exact_act(s["act"], G)[0] * U
        return {"H": H} if s["Z"] is None else {"H": H, "Z": torch.cat((G, U), 1)}
    x, dH = s["X"].double(), s["dH"].double()
    if s["Z"] is None:
        G, U = x @ W[:F].t(), x @ W[F:].t()
    else:
        G, U = s["Z"][:, :F].double(), s["Z"][:, F:].double()
    a, slope = _exact_act(s["act"], G)
    dG, dU = dH * U * slope, dH * a
    return {"dX": dG @ W[:F] + dU @ W[F:], "dW": torch.cat((dG.t() @ x, dU.t() @ x), 0)}
