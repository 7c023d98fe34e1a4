"""The products whose rows choose their own weights, as they are measured:

  lora       Y = X W^T + scale_a (X A_a^T) B_a^T, a = the adapter of the row
  lora_grad  its gradients: dX, and dA_a and dB_a of every adapter
  moe        a mixture-of-experts layer for a few tokens: router, the top_k
             experts of each token, gated experts, weighted sum

`run` computes them in their plain form (elementary torch operations in 32
bits), or with this library's calls where `own` is true.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def _lora(name, M, N, K, L, R, seg, dtype="f16", pad=0, op="lora"):
    """seg: mean rows of a request (1: one token each); pad: elements between
    the rows of X, Y and W beyond their length."""
    return {"name": name, "op": op, "dtype": dtype, "M": M, "N": N, "K": K, "L": L, "R": R,
            "seg": seg, "pad": pad}


def _moe(name, M, D, F, E, top_k, dtype="f16", pad=0):
    return {"name": name, "op": "moe", "dtype": dtype, "M": M, "D": D, "F": F, "E": E,
            "top_k": top_k, "pad": pad}


def listed():
    return [
        # one token of one request on a small projection: all latency
        _lora("lora_token", 1, 1024, 1024, 4, 8, 1),
        # a decode step: a token of each of 48 requests, any of 64 adapters, on a large projection
        _lora("lora_decode", 48, 4096, 4096, 64, 16, 1),
        # prompts of eight tenants, a few hundred tokens each, with wide adapters
        _lora("lora_prompt", 4096, 4096, 4096, 8, 64, 300),
        # fp32 with odd lengths and rows that do not start aligned
        _lora("lora_ragged_f32", 1000, 3000, 517, 5, 12, 77, dtype="f32", pad=2),
        # training step of a small batch with three adapters in it
        _lora("lora_grad_small", 257, 1024, 1024, 3, 8, 60, op="lora_grad"),
        # training step of one adapter over a long batch
        _lora("lora_grad_one", 4096, 4096, 4096, 1, 16, 4096, op="lora_grad"),
        # training step over a batch of several tenants, with wide adapters and an odd length
        _lora("lora_grad_many", 2049, 2048, 4096, 8, 64, 200, op="lora_grad"),
        # fp32 training step, odd lengths, unaligned rows
        _lora("lora_grad_ragged_f32", 1000, 3000, 517, 5, 12, 77, dtype="f32", pad=2,
              op="lora_grad"),
        # one token through a small layer: all latency
        _moe("moe_token", 1, 1024, 512, 8, 2),
        # a decode step of 16 requests over many small experts
        _moe("moe_decode", 16, 2048, 1024, 64, 6),
        # the largest: 64 tokens, every expert read
        _moe("moe_batch", 64, 4096, 2048, 32, 4),
        # fp32, odd lengths, unaligned rows
        _moe("moe_ragged_f32", 5, 1001, 499, 16, 3, dtype="f32", pad=2),
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
            for op in ("lora", "lora_grad", "moe")}
    most_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(("lora", "lora", "lora_grad", "moe", "moe"))
        dtype = "f32" if rng.random() < 0.25 else "f16"
        pad = rng.choice((0, 0, 0, 1, 8))
        if op == "moe":
            E = _log(rng, 4, 128)
            c = _moe("", _log(rng, 1, 64), _size(rng, 256, 4096), _size(rng, 128, 2048), E,
                     rng.randint(1, min(8, E)), dtype, pad)
        else:
            M = _log(rng, 1, 4096) if op == "lora" else _log(rng, 16, 4096)
            seg = 1 if op == "lora" and M <= 128 and rng.random() < 0.7 else _log(rng, 1, M)
            c = _lora("", M, _size(rng, 256, 4096), _size(rng, 256, 4096), _log(rng, 1, 64),
                      rng.choice((4, 8, 16, 16, 24, 32, 64, rng.randint(1, 64))), seg, dtype, pad,
                      op)
        w = work(c)
        # an fp32 product costs some eight times an fp16 one of its size
        if w["flops"] * (8 if dtype == "f32" else 1) <= most[op] and w["bytes"] <= most_bytes:
            del c["name"]
            return c


def work(case):
    c = case
    eb = 2 if c["dtype"] == "f16" else 4
    if c["op"] == "moe":
        M, D, F, E, k = (c[x] for x in ("M", "D", "F", "E", "top_k"))
        used = E * (1.0 - (1.0 - k / E) ** M)          # experts that some token chose
        return {"bytes": eb * (2.0 * M * D + E * D + used * 3.0 * D * F) + 8.0 * M * k,
                "flops": 2.0 * M * E * D + 6.0 * M * k * D * F}
    M, N, K, L, R = (c[x] for x in ("M", "N", "K", "L", "R"))
    requests = -(-M // c["seg"])
    used = L * (1.0 - (1.0 - 0.9 / L) ** requests) if L > 1 else 1.0
    r = R if L == 1 else 0.6 * R                       # mean rank (see _adapters)
    share = 1.0 if L == 1 else 0.9                     # rows that have an adapter
    ab = used * r * (K + N)
    if c["op"] == "lora":
        return {"bytes": eb * (M * K + N * K + M * N + ab) + 4.0 * M,
                "flops": 2.0 * M * N * K + 2.0 * share * M * r * (K + N)}
    # dY, X and W read, dX written; A and B read; dA and dB written whole (fp32)
    return {"bytes": eb * (2.0 * M * K + M * N + N * K + ab) + 4.0 * L * R * (K + N) + 4.0 * M,
            "flops": 2.0 * M * N * K + 2.0 * share * M * r * (3 * K + 2 * N)}


# ------------------------------------------------------------------ inputs

def _rows_of(gen, rows, cols, dtype, pad, std=1.0):
    """A rows x cols matrix of normal numbers, `pad` elements between its rows."""
    t = torch.randn(rows, cols + pad, generator=gen, device=gen.device)
    return t.mul_(std).to(dtype)[:, :cols]


def _adapters(gen, c):
    """The adapter of each row (request after request, -1: none), and each
    adapter's rank and scale: a quarter of them have R/4, a quarter R/2."""
    M, L, R = c["M"], c["L"], c["R"]
    if L == 1:
        rows = torch.zeros(M, dtype=torch.int32, device=gen.device)
        ranks = torch.full((1,), R, dtype=torch.int32, device=gen.device)
    else:
        n = -(-M // c["seg"])
        cuts = torch.randint(0, M, (n - 1,), generator=gen, device=gen.device) if c["seg"] > 1 \
            else torch.arange(1, M, device=gen.device)
        request = torch.zeros(M, dtype=torch.int64, device=gen.device)
        request.index_add_(0, cuts, torch.ones_like(cuts))
        request = request.cumsum(0)
        chosen = torch.randint(0, L, (n,), generator=gen, device=gen.device)
        none = torch.rand(n, generator=gen, device=gen.device) < 0.1
        rows = torch.where(none, torch.full_like(chosen, -1), chosen)[request].to(torch.int32)
        size = torch.randint(0, 4, (L,), generator=gen, device=gen.device)
        part = torch.tensor([R, R, (R + 1) // 2, (R + 3) // 4], device=gen.device)
        ranks = part[size].to(torch.int32)
    scale = 0.5 + 1.5 * torch.rand(L, generator=gen, device=gen.device)
    return rows, ranks, scale


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, pad = DTYPES[c["dtype"]], c["pad"]
    s = {"op": c["op"]}
    if c["op"] == "moe":
        M, D, F, E, k = (c[x] for x in ("M", "D", "F", "E", "top_k"))
        s["X"] = _rows_of(gen, M, D, dt, pad)
        s["router"] = _rows_of(gen, E, D, dt, 0, 1.5 / math.sqrt(D))
        # gate rows then up rows of each expert, and its down projection
        s["W1"] = torch.empty(E, 2 * F, D, dtype=dt, device=dev).normal_(0, 1.0 / math.sqrt(D),
                                                                         generator=gen)
        s["W2"] = torch.empty(E, D, F, dtype=dt, device=dev).normal_(0, 1.0 / math.sqrt(F),
                                                                     generator=gen)
        s["top_k"] = k
        s["Y"] = torch.empty(M, D, dtype=dt, device=dev)
        s["ids"] = torch.empty(M, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(M, k, dtype=torch.float32, device=dev)
        return s
    M, N, K, L, R = (c[x] for x in ("M", "N", "K", "L", "R"))
    s["X"] = _rows_of(gen, M, K, dt, pad)
    s["W"] = _rows_of(gen, N, K, dt, pad, 1.0 / math.sqrt(K))
    s["A"] = torch.empty(L, R, K, dtype=dt, device=dev).normal_(0, 1.0 / math.sqrt(K),
                                                                generator=gen)
    s["B"] = torch.empty(L, N, R, dtype=dt, device=dev).normal_(0, 0.5 / math.sqrt(R),
                                                                generator=gen)
    s["rows"], s["ranks"], s["scale"] = _adapters(gen, c)
    if c["op"] == "lora":
        s["Y"] = torch.empty(M, N + pad, dtype=dt, device=dev)[:, :N]
        return s
    s["dY"] = _rows_of(gen, M, N, dt, pad, 0.05)
    s["dX"] = torch.empty(M, K + pad, dtype=dt, device=dev)[:, :K]
    s["dA"] = torch.empty(L, R, K, dtype=torch.float32, device=dev)
    s["dB"] = torch.empty(L, N, R, dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------ the plain forms

def _mask(s):
    """M x L x R: scale_a where row m has adapter a and r is below its rank."""
    L, R, _ = s["A"].shape
    ids = torch.arange(L, device=s["A"].device)
    chosen = s["rows"][:, None] == ids[None, :]
    used = torch.arange(R, device=s["A"].device)[None, :] < s["ranks"][:, None]
    return chosen[:, :, None] * (used * s["scale"][:, None])[None, :, :]


def _plain_lora(s):
    L, R, K = s["A"].shape
    N = s["W"].shape[0]
    X = s["X"].float()
    A = s["A"].float().reshape(L * R, K)
    B = s["B"].float().permute(1, 0, 2).reshape(N, L * R)
    V = (X @ A.t()) * _mask(s).reshape(-1, L * R)
    return (X @ s["W"].float().t() + V @ B.t()).to(s["X"].dtype)


def _plain_lora_grad(s):
    L, R, K = s["A"].shape
    N = s["W"].shape[0]
    X, dY = s["X"].float(), s["dY"].float()
    A = s["A"].float().reshape(L * R, K)
    B = s["B"].float().permute(1, 0, 2).reshape(N, L * R)
    mask = _mask(s).reshape(-1, L * R)
    G = (dY @ B) * mask
    V = (X @ A.t()) * mask
    dX = (dY @ s["W"].float() + G @ A).to(s["X"].dtype)
    dA = (G.t() @ X).reshape(L, R, K)
    dB = (dY.t() @ V).reshape(N, L, R).permute(1, 0, 2).contiguous()
    return {"dX": dX, "dA": dA, "dB": dB}


def _plain_moe(s):
    M, D = s["X"].shape
    E, D2, F = s["W2"].shape
    k = s["top_k"]
    # the router's order is decided in 64 bits: two logits may lie close together
    logits = s["X"].double() @ s["router"].double().t()
    order = logits.sort(dim=1, descending=True, stable=True)
    ids = order.indices[:, :k]
    top = order.values[:, :k]
    w = (top - top[:, :1]).exp()
    w = (w / w.sum(1, keepdim=True)).float()
    X = s["X"].float()
    if M * k < E:
        # few tokens: the chosen experts' weights alone
        pick = ids.reshape(-1)
        x = X[:, None, :].expand(M, k, D).reshape(M * k, D, 1)
        h = (s["W1"][pick].float() @ x).reshape(M * k, 2 * F)
        g, u = h[:, :F], h[:, F:]
        a = g / (1.0 + (-g).exp()) * u
        y = (s["W2"][pick].float() @ a[:, :, None]).reshape(M, k, D)
        y = (y * w[:, :, None]).sum(1)
    else:
        h = (X @ s["W1"].float().reshape(E * 2 * F, D).t()).reshape(M, E, 2 * F)
        g, u = h[:, :, :F], h[:, :, F:]
        dense = torch.zeros(M, E, device=X.device).scatter_(1, ids, w)
        a = g / (1.0 + (-g).exp()) * u * dense[:, :, None]
        y = a.reshape(M, E * F) @ s["W2"].float().permute(0, 2, 1).reshape(E * F, D2)
    return {"Y": y.to(s["X"].dtype), "ids": ids.to(torch.int32), "weights": w}


def run(state):
    s = state
    if own:
        import dense_gemm_fp32_amd as dg
        if s["op"] == "lora":
            return dg.lora(s["X"], s["W"], s["A"], s["B"], s["rows"], s["Y"], scale=s["scale"],
                           ranks=s["ranks"])
        if s["op"] == "lora_grad":
            dg.lora_grad(s["dY"], s["X"], s["W"], s["A"], s["B"], s["rows"], dX=s["dX"],
                         dA=s["dA"], dB=s["dB"], scale=s["scale"], ranks=s["ranks"])
            return {"dX": s["dX"], "dA": s["dA"], "dB": s["dB"]}
        dg.moe(s["X"], s["router"], s["W1"], s["W2"], s["top_k"], s["Y"], ids=s["ids"],
               weights=s["weights"])
        return {"Y": s["Y"], "ids": s["ids"], "weights": s["weights"]}
    if s["op"] == "lora":
        return _plain_lora(s)
    if s["op"] == "lora_grad":
        return _plain_lora_grad(s)
    return _plain_moe(s)


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    X = s["X"].double()
    if s["op"] == "moe":
        return _exact_moe(s, X)
    rows, ranks, scale = s["rows"].tolist(), s["ranks"].tolist(), s["scale"].double()
    rows = torch.tensor(rows)
    W = s["W"].double()
    if s["op"] == "lora":
        Y = X @ W.t()
        for a, r in enumerate(ranks):
            at = (rows == a).nonzero()[:, 0].to(X.device)
            down = s["A"][a, :r].double()
            up = s["B"][a, :, :r].double()
            Y[at] += scale[a] * ((X[at] @ down.t()) @ up.t())
        return Y
    dY = s["dY"].double()
    dX = dY @ W
    dA, dB = torch.zeros_like(s["A"].double()), torch.zeros_like(s["B"].double())
    for a, r in enumerate(ranks):
        at = (rows == a).nonzero()[:, 0].to(X.device)
        down, up = s["A"][a, :r].double(), s["B"][a, :, :r].double()
        G = scale[a] * (dY[at] @ up)
        dX[at] += G @ down
        dA[a, :r] = G.t() @ X[at]
        dB[a, :, :r] = scale[a] * (dY[at].t() @ (X[at] @ down.t()))
    return {"dX": dX, "dA": dA, "dB": dB}


def _exact_moe(s, X):
    M, k = X.shape[0], s["top_k"]
    F = s["W2"].shape[2]
    logits = X @ s["router"].double().t()
    Y = torch.zeros_like(X)
    ids = torch.zeros(M, k, dtype=torch.int32, device=X.device)
    weights = torch.zeros(M, k, dtype=torch.float64, device=X.device)
    left = logits.clone()
    for j in range(k):
        best = left.max(dim=1, keepdim=True).values
        # the lowest index among equals
        ids[:, j] = (left == best).to(torch.int32).argmax(dim=1).to(torch.int32)
        weights[:, j] = logits.gather(1, ids[:, j:j + 1].long())[:, 0]
        left.scatter_(1, ids[:, j:j + 1].long(), -math.inf)
    weights = torch.softmax(weights, dim=1)
    for e in range(s["W1"].shape[0]):
        token, slot = (ids == e).nonzero(as_tuple=True)
        if token.numel() == 0:
            continue
        h = X[token] @ s["W1"][e].double().t()
        a = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:]
        Y[token] += weights[token, slot][:, None] * (a @ s["W2"][e].double().t())
    return {"Y": Y, "ids": ids, "weights": weights}
