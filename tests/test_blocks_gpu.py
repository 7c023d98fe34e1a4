"""Products of 8-bit integers and gated blocks on the GPU, against 64-bit
references within derived bounds."""
import ctypes
import math

import pytest
import torch

import blocks_reference as ref
from gemm_harness import note
from rows_reference import worst

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "f32": torch.float32}
GPU = "cuda:0"


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, shape, dtype, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def whole(g, shape):
    return torch.randint(-127, 128, shape, generator=g).to(torch.int8)


def scales(g, n):
    return 0.01 + torch.rand(n, generator=g) / 50


def padded(t, pad):
    """A device copy of t with `pad` elements after each row that no call may
    read or write (NaN; 99 among integers), and the view of t in it."""
    fill = float("nan") if t.is_floating_point() else 99
    big = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), fill, dtype=t.dtype)
    big[..., :t.shape[-1]] = t
    big = big.to(GPU)
    return big, big[..., :t.shape[-1]]


def pads_intact(big, cols):
    tail = big[..., cols:]
    if tail.numel() == 0:
        return True
    return bool((torch.isnan(tail) if tail.is_floating_point() else tail == 99).all())


def near(work, *tensors):
    """The tensors where their reference is computed: large ones on the GPU."""
    return [t if t is None or work < 1e9 else t.to(GPU) for t in tensors]


def unset(rows, cols, dtype, pad):
    """An output that holds nothing yet."""
    return padded(torch.full((rows, cols), 77 if dtype == torch.int8 else float("nan"),
                             dtype=dtype), pad)


# ---------------------------------------------------------------- rows to 8-bit integers

QUANT = [(1, 1, 0), (1, 4096, 0), (3, 7, 1), (5, 8, 0), (2, 15, 0), (17, 16, 3), (4, 17, 0),
         (33, 255, 1), (64, 2048, 0), (9, 2049, 0), (130, 517, 8), (3, 20000, 0), (1, 131071, 1),
         (2000, 64, 0), (300, 8192, 0), (3, 12345, 1), (40, 16384, 0)]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", QUANT, ids=lambda c: "x".join(map(str, c)))
def test_quantize(dt, case):
    import dense_gemm_fp32_amd as dg
    M, K, pad = case
    note("quantize %s %r" % (dt, case))
    g = gen(M * 7 + K)
    X = normal(g, (M, K), DT[dt]) * torch.exp2(torch.randint(-8, 6, (M, 1), generator=g)).to(DT[dt])
    want, scale = ref.quantize(X)
    x = padded(X, pad)[1]
    big, q = unset(M, K, torch.int8, pad)
    s = torch.full((M,), -1.0, device=GPU)
    out = dg.quantize(x, q, s)
    assert out[0] is q and out[1] is s
    torch.cuda.synchronize()
    assert torch.equal(s.cpu(), scale) and torch.equal(q.cpu(), want)
    assert pads_intact(big, K)


def test_quantize_most_rows():
    """As many rows as a call takes, of one element each."""
    import dense_gemm_fp32_amd as dg
    M = 1 << 24
    note("quantize %d rows" % M)
    x = ((torch.arange(M, device=GPU) % 4001 - 2000).float() / 16).half()[:, None]
    q, s = dg.quantize(x)
    assert torch.equal(q[:, 0], (torch.sign(x[:, 0]) * 127).to(torch.int8))
    top = torch.full((1,), 127.0, device=GPU)
    assert torch.equal(s, x[:, 0].float().abs() / top)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_quantize_ties_and_odd_rows(dt):
    """Quotients on and next to the border of two whole numbers; rows of zeros, of
    the type's smallest and largest values, with infinities and NaN."""
    import dense_gemm_fp32_amd as dg
    t, info = DT[dt], torch.finfo(DT[dt])
    rows = []
    for top in (127.0, 254.0, 63.5, 127.0 * 2 ** -10):       # scales 1, 2, 0.5, 2^-10
        k = torch.arange(-126, 127) + 0.5
        rows.append(torch.cat((torch.tensor([top]), k * (top / 127.0))))
    for top in (1.0, 3.7, 100.0 / 3, 6.1e-5 * 7):            # borders of scales that are no powers of 2
        top = float(torch.tensor(top, dtype=t))
        s = float((torch.tensor([top]).double() / 127).float())
        x = ((torch.arange(-126, 127) + 0.5).double() * s).to(t)
        rows.append(torch.cat((torch.tensor([top]), x.float())))
    n = 254
    rows += [torch.zeros(n), torch.full((n,), info.max), torch.full((n,), -info.max),
             torch.full((n,), info.tiny), torch.linspace(-info.max, info.max, n)]
    tiny = torch.arange(n) * (2.0 ** -24 if dt == "f16" else 2.0 ** -149)
    rows += [tiny, tiny / tiny.max() * info.tiny * 3]
    for bad in (math.inf, -math.inf, math.nan):
        r = torch.arange(n).float()
        r[n // 2] = bad
        rows.append(r)
    X = torch.stack([r.to(t) for r in rows])
    if dt == "f32":       # one step either side of each border
        step = X[:8].view(torch.int32)
        X = torch.cat((X, (step + 1).view(torch.float32), (step - 1).view(torch.float32)))
        X[-16:, 0] = X[:8, 0].repeat(2)
    want, scale = ref.quantize(X)
    q, s = dg.quantize(X.to(GPU))
    assert torch.equal(torch.isnan(s.cpu()), torch.isnan(scale))
    assert torch.equal(s.cpu().nan_to_num(), scale.nan_to_num())
    assert torch.equal(q.cpu(), want)


def test_quantize_without_columns():
    import dense_gemm_fp32_amd as dg
    q, s = dg.quantize(torch.empty(5, 0, device=GPU))
    assert q.shape == (5, 0) and s.tolist() == [0.0] * 5


# ---------------------------------------------------------------- products of 8-bit integers

I8 = [
    # M, N, K, pad, alpha, beta, scales
    (1, 1, 1, 0, 1.0, 0.0, True),
    (1, 64, 64, 0, 1.0, 0.0, True),
    (1, 1024, 1024, 0, 1.0, 0.0, True),
    (2, 5, 15, 1, 1.5, -0.5, True),
    (3, 33, 16, 0, 1.0, 0.0, False),
    (7, 130, 17, 3, -1.0, 1.0, True),
    (16, 256, 4096, 0, 1.0, 0.0, True),
    (17, 520, 63, 0, 1.0, 1.0, True),
    (33, 96, 2000, 16, 1.0, 0.0, True),
    (48, 1000, 130, 1, 1.0, 0.5, False),
    (64, 4096, 256, 0, 1.0, 0.0, True),
    (65, 257, 129, 0, 1.0, 0.0, True),
    (100, 128, 128, 0, 1.0, 0.0, True),
    (129, 384, 640, 0, 2.0, 0.25, True),
    (200, 515, 517, 3, 1.0, 0.0, True),
    (256, 2048, 1024, 0, 1.0, 0.0, True),
    (300, 260, 1536, 16, 1.0, 1.0, True),
    (513, 1032, 255, 0, 1.0, 0.0, True),
    (700, 96, 3000, 0, 1.0, 0.0, True),
    (1000, 1500, 517, 5, -0.5, 0.0, True),
    (1030, 2050, 272, 0, 1.0, 0.0, True),
    (2100, 4160, 144, 0, 1.0, 1.0, True),
    (4096, 512, 192, 32, 1.0, 0.0, False),
    (40, 4000, 131071, 0, 1.0, 0.0, True),
    (1100, 8200, 2000, 0, 1.0, 0.5, True),
    (200, 6000, 1040, 0, 1.0, -1.0, True),
    (300, 6000, 1031, 1, 1.0, 0.0, True),
    (16, 9000, 300, 4, 1.0, 0.0, True),
    (64, 8200, 512, 0, 1.0, 1.0, True),
    (90, 700, 6643, 8, 1.0, 0.0, True),
    (30, 8300, 390, 1, 1.0, 0.0, True),
    (40, 9000, 300, 1, 1.0, 1.0, True),
    (64, 8200, 270, 1, 1.0, 0.0, True),
]


# few rows: each height and width of a workgroup, in rows that start anywhere
FEW = [(33, 2070), (17, 4096), (17, 2070), (33, 4096), (33, 2749), (65, 2070), (17, 8181),
       (33, 8181), (49, 8181)]
I8 += [(M, N, 71, 1, 1.0, 0.0, True) for M, N in FEW]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", I8, ids=lambda c: "x".join(map(str, c[:4])))
def test_gemm_i8(dt, case):
    import dense_gemm_fp32_amd as dg
    M, N, K, pad, alpha, beta, scaled = case
    note("gemm_i8 %s %r" % (dt, case))
    g, t = gen(M * 31 + N), DT[dt]
    X, W = whole(g, (M, K)), whole(g, (N, K))
    top = 0.5 / math.sqrt(K)
    xs, ws = (scales(g, M) * top, scales(g, N)) if scaled else (None, None)
    if not scaled and dt == "f16":
        alpha *= 2.0 ** -12      # sums of whole numbers pass fp16's largest
    Y = normal(g, (M, N), t) if beta else torch.full((M, N), float("nan"), dtype=t)
    want, bound = (v.cpu() for v in ref.gemm_i8(*near(M * N * K, X, W, Y, xs, ws), alpha, beta, t))
    x, w = padded(X, pad)[1], padded(W, pad)[1]
    big, y = padded(Y, pad)
    up = lambda v: None if v is None else v.to(GPU)  # noqa: E731
    assert dg.gemm_i8(x, w, y, x_scale=up(xs), w_scale=up(ws), alpha=alpha, beta=beta) is y
    torch.cuda.synchronize()
    assert worst(y, want, bound) <= 1.0
    assert pads_intact(big, N)


def test_gemm_i8_sums_are_exact():
    """Sums at the edges of 32 bits: -128 and 127 in every place, and sums beyond
    2^24 that differ by one."""
    import dense_gemm_fp32_amd as dg
    K = 131071
    for M in (1, 40, 300):
        X = torch.full((M, K), 127, dtype=torch.int8)
        X[0] = -128
        W = torch.stack((torch.full((K,), -128), torch.full((K,), 127))).to(torch.int8)
        y = torch.empty(M, 2, device=GPU)
        dg.gemm_i8(X.to(GPU), W.to(GPU), y)
        S = X.double() @ W.double().t()
        assert torch.equal(y.cpu(), S.float())
    # 512 columns of 127 * 127, less what makes whole numbers of 24 bits
    M, N, K = 70, 65, 1040
    X = torch.full((M, K), 127, dtype=torch.int8)
    W = torch.full((N, K), 127, dtype=torch.int8)
    W[:, 1039] = torch.arange(N).to(torch.int8)
    X[:, 1039] = 1
    y = torch.empty(M, N, device=GPU)
    dg.gemm_i8(X.to(GPU), W.to(GPU), y)
    S = X.double() @ W.double().t()
    assert float(S.max()) < 2 ** 24 and torch.equal(y.cpu().double(), S)


# few rows in two forms, then each tile
SCALED = [(1, 200, 144), (3, 40, 1000), (20, 300, 256), (64, 8200, 270), (130, 1030, 300),
          (700, 1500, 130), (2100, 4160, 144)]


@pytest.mark.parametrize("M,N,K", SCALED)
def test_scales_are_taken_in_the_order_that_is_documented(M, N, K):
    """The sum, rounded to fp32, times the row's scale, times the column's, times alpha:
    bit for bit; a product that leaves fp32 on the way does not come back."""
    import dense_gemm_fp32_amd as dg
    g = gen(M + N)
    X, W = whole(g, (M, K)), whole(g, (N, K))
    xs, ws = scales(g, M), scales(g, N)
    xs[0], ws[:N // 2] = 2.0 ** 120, ws[:N // 2] * 2.0 ** -100
    if M > 1:
        xs[1], ws[N // 2:] = 2.0 ** -110, ws[N // 2:] * 2.0 ** 100
    S = (X.double() @ W.double().t()).float()
    Z = (S * xs[:, None]) * ws[None, :]
    assert not torch.equal(Z, (S * ws[None, :]) * xs[:, None])
    alpha = 1.37
    want = torch.tensor(alpha) * Z
    y = torch.empty(M, N, device=GPU)
    dg.gemm_i8(X.to(GPU), W.to(GPU), y, x_scale=xs.to(GPU), w_scale=ws.to(GPU), alpha=alpha)
    same = lambda a, b: torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))  # noqa: E731
    assert torch.isinf(want[0]).any() and same(y.cpu(), want)
    F = N // 2
    h = torch.empty(M, F, device=GPU)
    dg.glu(X.to(GPU), W.to(GPU), h, act="relu", x_scale=xs.to(GPU), w_scale=ws.to(GPU))
    want = torch.where(Z[:, :F] <= 0, torch.zeros(()), Z[:, :F]) * Z[:, F:]
    assert same(h.cpu(), want)


@pytest.mark.parametrize("M", [1, 20, 130, 700])
def test_gemm_i8_scales_that_are_not_finite_stay_in_their_rows(M):
    import dense_gemm_fp32_amd as dg
    g = gen(M)
    N, K = 200, 144
    X, W = whole(g, (M, K)), whole(g, (N, K))
    xs, ws = scales(g, M), scales(g, N)
    xs[M // 2], ws[3], ws[N - 1] = math.nan, math.inf, math.nan
    y = torch.empty(M, N, device=GPU)
    dg.gemm_i8(X.to(GPU), W.to(GPU), y, x_scale=xs.to(GPU), w_scale=ws.to(GPU))
    want, bound = ref.gemm_i8(X, W, None, xs, ws, 1.0, 0, torch.float32)
    ok = torch.isfinite(want)
    y = y.cpu()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert worst(y[ok], want[ok], bound[ok]) <= 1.0


def test_gemm_i8_degenerate():
    import dense_gemm_fp32_amd as dg
    y = torch.full((3, 4), 2.0, device=GPU)
    e = torch.empty(3, 0, dtype=torch.int8, device=GPU), torch.empty(4, 0, dtype=torch.int8,
                                                                     device=GPU)
    dg.gemm_i8(*e, y, beta=0.5)
    assert y.tolist() == [[1.0] * 4] * 3
    nan = torch.full((3,), math.nan, device=GPU)
    q = torch.ones(3, 8, dtype=torch.int8, device=GPU), torch.ones(4, 8, dtype=torch.int8,
                                                                   device=GPU)
    dg.gemm_i8(*q, y, x_scale=nan, alpha=0.0, beta=3.0)
    assert y.tolist() == [[3.0] * 4] * 3
    y.fill_(math.nan)
    dg.gemm_i8(*e, y)
    assert y.tolist() == [[0.0] * 4] * 3


# ---------------------------------------------------------------- gated blocks

GLU = [
    # M, F, K, pad, act, Z kept
    (1, 1, 1, 0, "silu", True),
    (1, 1024, 1024, 0, "silu", False),
    (1, 64, 64, 0, "relu", True),
    (2, 5, 7, 1, "gelu", True),
    (3, 33, 8, 0, "gelu_tanh", False),
    (8, 130, 17, 3, "silu", True),
    (16, 520, 2048, 0, "gelu", False),
    (17, 96, 1000, 8, "relu", True),
    (33, 257, 65, 0, "gelu_tanh", True),
    (48, 1000, 264, 0, "silu", False),
    (64, 2048, 256, 0, "silu", True),
    (65, 127, 129, 1, "silu", True),
    (100, 128, 128, 0, "gelu", True),
    (129, 384, 328, 0, "silu", False),
    (200, 515, 517, 3, "gelu_tanh", True),
    (257, 1024, 512, 0, "silu", True),
    (300, 260, 768, 8, "relu", False),
    (513, 1032, 136, 0, "silu", True),
    (1000, 750, 259, 5, "gelu", True),
    (1030, 2050, 72, 0, "silu", True),
    (2100, 2112, 96, 0, "gelu_tanh", False),
    (2048, 4096, 64, 0, "silu", True),
    (1100, 4100, 1000, 0, "gelu_tanh", True),
    (64, 4200, 528, 0, "relu", True),
    (150, 1800, 1030, 2, "silu", False),
    (17, 8000, 96, 8, "gelu", True),
    (700, 1100, 1040, 0, "silu", True),
    (30, 4300, 390, 1, "silu", False),
    (40, 8300, 200, 1, "gelu", True),
    (64, 8200, 270, 1, "relu", False),
    (1500, 1024, 1104, 0, "silu", True),
    (1100, 4100, 2600, 0, "silu", False),
]


GLU += [(M, F, 71, 1, "silu", True) for M, F in FEW]
GLU += [(33, 4082, 70, 1, "silu", True), (17, 8216, 70, 1, "gelu", True)]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", GLU, ids=lambda c: "x".join(map(str, c)))
def test_glu(dt, case):
    import dense_gemm_fp32_amd as dg
    M, F, K, pad, name, kept = case
    note("glu %s %r" % (dt, case))
    g, t = gen(M * 31 + F), DT[dt]
    X, W = normal(g, (M, K), t), normal(g, (2 * F, K), t, 1.5 / math.sqrt(K))
    want = {k: [v.cpu() for v in e] for k, e in ref.glu(*near(M * F * K, X, W), name, t).items()}
    x, w = padded(X, pad)[1], padded(W, pad)[1]
    bigh, h = unset(M, F, t, pad)
    bigz, z = unset(M, 2 * F, t, pad)
    assert dg.glu(x, w, h, act=name, Z=z if kept else None) is h
    torch.cuda.synchronize()
    assert worst(h, *want["H"]) <= 1.0
    assert pads_intact(bigh, F) and pads_intact(bigz, 2 * F)
    if kept:
        assert worst(z, *want["Z"]) <= 1.0
    else:
        assert pads_intact(bigz, 0)


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", GLU, ids=lambda c: "x".join(map(str, c)))
def test_glu_i8(dt, case):
    import dense_gemm_fp32_amd as dg
    M, F, K, pad, name, scaled = case
    note("glu_i8 %s %r" % (dt, case))
    g, t = gen(M * 37 + F), DT[dt]
    X, W = whole(g, (M, K)), whole(g, (2 * F, K))
    xs, ws = scales(g, M), scales(g, 2 * F) / math.sqrt(K)
    up = (lambda v: v.to(GPU)) if scaled else (lambda v: None)
    if not scaled:          # sums of a few units: scales of 1 would leave fp16's range
        X, W = (torch.randint(-1, 2, m.shape, generator=g).to(torch.int8) for m in (X, W))
        xs = ws = None
    X_, W_, xs_, ws_ = near(M * F * K, X, W, xs, ws)
    want = {k: [v.cpu() for v in e] for k, e in ref.glu(X_, W_, name, t, xs_, ws_).items()}
    x, w = padded(X, pad)[1], padded(W, pad)[1]
    bigh, h = unset(M, F, t, pad)
    dg.glu(x, w, h, act=name, x_scale=up(xs), w_scale=up(ws))
    torch.cuda.synchronize()
    assert worst(h, *want["H"]) <= 1.0
    assert pads_intact(bigh, F)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_activations_over_their_range(dt, name):
    """Gates from -100 to 100 and at both zeros, each times an up value: K = 2
    picks them out of X."""
    import dense_gemm_fp32_amd as dg
    t = DT[dt]
    gates = torch.cat((torch.linspace(-100, 100, 1601), torch.tensor([0.0, -0.0]),
                       torch.logspace(-6, 1, 100), -torch.logspace(-6, 1, 100)))
    X = torch.stack((gates, torch.full_like(gates, 1.5)), 1).to(t)
    W = torch.tensor([[1.0, 0.0], [0.0, 1.0]], dtype=t)
    want = ref.glu(X, W, name, t)["H"]
    h = torch.empty(len(gates), 1, dtype=t, device=GPU)
    dg.glu(X.to(GPU), W.to(GPU), h, act=name)
    # where act(g) leaves the normal numbers, to their smallest
    assert worst(h, want[0], want[1] + 150 * torch.finfo(torch.float32).tiny) <= 1.0


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_activations_at_the_end_of_the_normal_numbers(name):
    """Gates whose exponential is one of the smallest normal numbers, or below them,
    where it may count as 0: the activation and its derivative are then within 2^-117,
    above that as good as anywhere.  An up value and a gradient of 2^20 bring them into
    range."""
    import dense_gemm_fp32_amd as dg
    g = torch.linspace(-105.0, -80.0, 2001) if name == "silu" else \
        torch.linspace(-14.6, -12.0, 1001) if name == "gelu" else torch.linspace(-10.9, -9.5, 1001)
    n, up = len(g), 2.0 ** 20
    G = g.double()
    v, d, ev, ed = ref.act(name, G)
    if name == "gelu":     # (the reference's distribution function ends near g = -8)
        p, f = 0.5 * torch.erfc(-G / math.sqrt(2)), torch.exp(-G * G / 2) / math.sqrt(2 * math.pi)
        c = (16 + 4 * G * G) * ref.U32
        v, d, ev, ed = G * p, p + G * f, c * (G * p).abs(), 2 * c * (p + G.abs() * f)
    # |t| of exp(-|t|); gelu: -g^2 / 2, whose two ends meet the same exponential
    t = {"silu": G.abs(), "gelu": G * G / 2,
         "gelu_tanh": math.sqrt(8 / math.pi) * (G + 0.044715 * G ** 3).abs()}[name]
    low = torch.where(t > 125 * math.log(2), 2.0 ** -117, 0.0).double()
    assert 100 < int((low == 0).sum()) < n - 100
    ev, ed = ev + low, ed + low
    W = torch.tensor([[1.0, 0.0], [0.0, up]], device=GPU)
    h = torch.empty(n, 1, device=GPU)
    dg.glu(torch.stack((g, torch.ones(n)), 1).to(GPU), W, h, act=name)
    assert worst(h[:, 0], v * up, ev * up + ref.U32 * (v * up).abs()) <= 1.0
    # dX = [dG, dU], dG = 2^20 * 1 * act'(g), dU = 2^20 * act(g)
    dX = torch.empty(n, 2, device=GPU)
    dg.glu_grad(torch.full((n, 1), up, device=GPU), torch.zeros(n, 2, device=GPU),
                torch.eye(2, device=GPU), dX=dX, act=name,
                Z=torch.stack((g, torch.ones(n)), 1).to(GPU))
    assert worst(dX[:, 0], d * up, ed * up + 2 * ref.U32 * (d * up).abs()) <= 1.0
    assert worst(dX[:, 1], v * up, ev * up + 2 * ref.U32 * (v * up).abs()) <= 1.0


@pytest.mark.parametrize("name", ref.ACTS)
def test_activations_of_gates_whose_square_leaves_fp32(name):
    """Gates up to 1e30: the activation is the gate or 0, its derivative 1 or 0."""
    import dense_gemm_fp32_amd as dg
    gates = torch.tensor([1e10, 1e18, 1e20, 1e30, -1e10, -1e18, -1e20, -1e30])
    n, on = len(gates), (gates > 0).float()
    Z = torch.stack((gates, torch.full((n,), 2.0)), 1)
    X, dH = gates[:, None], torch.full((n, 1), 3.0)
    h, dX = (torch.empty(n, 1, device=GPU) for _ in range(2))
    dg.glu(X.to(GPU), torch.tensor([[1.0], [1e-30]], device=GPU), h, act=name)
    up = gates * torch.tensor(1e-30)
    assert torch.allclose(h[:, 0].cpu(), gates * on * up, rtol=2 ** -20, atol=1e-30)
    dg.glu_grad(dH.to(GPU), X.to(GPU), torch.tensor([[1.0], [0.0]], device=GPU), dX=dX, act=name,
                Z=Z.to(GPU))
    # dX = dG * 1 + dU * 0, dG = 3 * 2 * act'(g)
    assert torch.equal(dX[:, 0].cpu() + 0.0, 6.0 * on)


@pytest.mark.parametrize("M", [3, 70, 300])
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_glu_infinities_stay_in_their_rows(dt, M):
    import dense_gemm_fp32_amd as dg
    g, t = gen(M), DT[dt]
    F, K = 200, 136
    X, W = normal(g, (M, K), t), normal(g, (2 * F, K), t, 0.1)
    clean = ref.glu(X, W, "silu", t)
    X[M // 2, K - 1] = math.inf
    X[0, 0] = math.nan
    W[7, 3] = math.nan
    W[F + 11, K - 1] = -math.inf
    h = torch.empty(M, F, dtype=t, device=GPU)
    z = torch.empty(M, 2 * F, dtype=t, device=GPU)
    dg.glu(X.to(GPU), W.to(GPU), h, Z=z)
    rows = [i for i in range(M) if i not in (0, M // 2)]
    cols = [i for i in range(F) if i not in (7, 11)]
    pick = lambda v: v[rows][:, cols]  # noqa: E731
    assert worst(pick(h.cpu()), *(pick(v) for v in clean["H"])) <= 1.0
    Z = X.double() @ W.double().t()
    assert torch.equal(torch.isnan(z.cpu()), torch.isnan(Z))
    assert torch.equal(torch.isinf(z.cpu()), torch.isinf(Z))


def test_glu_without_columns():
    import dense_gemm_fp32_amd as dg
    for t in (torch.float16, torch.float32):
        h, z = torch.ones(3, 4, dtype=t, device=GPU), torch.ones(3, 8, dtype=t, device=GPU)
        dg.glu(torch.empty(3, 0, dtype=t, device=GPU), torch.empty(8, 0, dtype=t, device=GPU), h,
               Z=z)
        assert not h.any() and not z.any()
        q = torch.empty(3, 0, dtype=torch.int8, device=GPU)
        h.fill_(1)
        dg.glu(q, torch.empty(8, 0, dtype=torch.int8, device=GPU), h)
        assert not h.any()


# ---------------------------------------------------------------- their gradients

GRAD = [
    # M, F, K, pad, act, Z given, beta_x, beta_w, dW in fp32
    (1, 1, 1, 0, "silu", True, 0.0, 0.0, False),
    (1, 64, 64, 0, "silu", False, 0.0, 0.0, True),
    (3, 5, 7, 1, "gelu", True, 1.0, -0.5, False),
    (17, 130, 96, 8, "gelu_tanh", False, 0.0, 1.0, True),
    (33, 256, 512, 0, "relu", True, 0.0, 0.0, False),
    (64, 96, 200, 0, "silu", False, 0.5, 0.0, False),
    (65, 127, 129, 3, "gelu", False, 0.0, 0.0, True),
    (129, 300, 264, 0, "silu", True, 0.0, 1.0, True),
    (257, 512, 384, 0, "silu", False, 0.0, 0.0, False),
    (300, 515, 131, 5, "gelu_tanh", True, 1.0, 1.0, False),
    (512, 640, 256, 0, "relu", False, 0.0, 0.0, True),
    (1000, 375, 259, 1, "gelu", True, 0.0, 0.0, False),
    (1030, 1024, 136, 0, "silu", False, 0.0, 0.0, False),
    (19, 700, 2100, 0, "gelu_tanh", True, 0.0, 1.0, False),
    (40, 2100, 1000, 4, "silu", False, 1.0, 0.0, True),
    (900, 1000, 520, 0, "silu", True, 0.5, 0.0, False),
    (2000, 100, 1500, 2, "gelu", True, 0.0, 0.0, True),
    (130, 1500, 1001, 1, "silu", False, 0.0, -1.0, False),
    (1024, 1536, 1024, 0, "silu", True, 0.0, 1.0, True),
    (1100, 1500, 1024, 0, "gelu", False, 1.0, 0.0, False),
    (257, 2048, 520, 0, "relu", False, 0.0, 0.0, False),
    (2048, 1024, 2048, 0, "silu", True, 0.0, 0.0, False),
]


def grad_inputs(case, dt):
    M, F, K, pad, name, kept, beta_x, beta_w, dw32 = case
    g, t = gen(M * 31 + F), DT[dt]
    X, W = normal(g, (M, K), t), normal(g, (2 * F, K), t, 1.0 / math.sqrt(K))
    dH = normal(g, (M, F), t, 0.05)
    Z = (X.double() @ W.double().t()).to(t) if kept else None
    tw = torch.float32 if dw32 else t
    return X, W, dH, Z, normal(g, (M, K), t), normal(g, (2 * F, K), tw), tw


GRAD += [(M, F, 71, 1, "silu", False, 0.0, 0.0, False) for M, F in FEW]
GRAD += [(2048, 1024, 2048, 0, "silu", True, 0.0, 0.0, True),
         (2048, 2048, 200, 0, "gelu_tanh", False, 0.0, 0.0, False),
         (1200, 2048, 264, 0, "silu", False, 0.0, 0.0, False),
         (17, 4082, 72, 0, "silu", False, 0.0, 0.0, False),
         # rows that start anywhere, sums over whole steps; rows of one to four
         (128, 160, 101, 1, "silu", False, 1.0, 1.0, False),
         (320, 256, 37, 3, "gelu", True, 0.0, 1.0, False),
         (64, 32, 130, 1, "relu", True, 0.0, 0.0, True),
         (70, 80, 1, 0, "silu", False, 0.0, 0.0, False),
         (70, 80, 2, 0, "silu", True, 1.0, 0.0, False),
         (70, 80, 3, 2, "gelu", False, 0.0, 0.0, False),
         (70, 80, 4, 1, "silu", False, 0.0, 1.0, False),
         (33, 4082, 72, 0, "gelu", False, 0.0, 0.0, False),
         (49, 4082, 72, 0, "silu", False, 1.0, 0.0, False)]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", GRAD, ids=lambda c: "x".join(map(str, c)))
def test_glu_grad(dt, case):
    import dense_gemm_fp32_amd as dg
    M, F, K, pad, name, kept, beta_x, beta_w, dw32 = case
    note("glu_grad %s %r" % (dt, case))
    X, W, dH, Z, oldx, oldw, tw = grad_inputs(case, dt)
    old = near(M * F * K, oldx, oldw)
    want = ref.glu_grad(*near(M * F * K, dH, X, W, Z), name, *old, beta_x, beta_w, tw)
    want = {k: [v.cpu() for v in e] for k, e in want.items()}
    x, w, d = (padded(v, pad)[1] for v in (X, W, dH))
    z = padded(Z, pad)[1] if kept else None
    bigx, dx = padded(oldx, pad) if beta_x else unset(M, K, DT[dt], pad)
    bigw, dw = padded(oldw, pad) if beta_w else unset(2 * F, K, tw, pad)
    out = dg.glu_grad(d, x, w, dX=dx, dW=dw, act=name, Z=z, beta_x=beta_x, beta_w=beta_w)
    torch.cuda.synchronize()
    assert out[0] is dx and out[1] is dw
    assert worst(dx, *want["dX"]) <= 1.0 and worst(dw, *want["dW"]) <= 1.0
    assert pads_intact(bigx, K) and pads_intact(bigw, K)
    # one of the two alone: the same bits
    one = torch.full_like(dx, 1.0).copy_(oldx.to(GPU))
    dg.glu_grad(d, x, w, dX=one, act=name, Z=z, beta_x=beta_x)
    assert torch.equal(one, dx)
    one = torch.full_like(dw, 1.0).copy_(oldw.to(GPU))
    dg.glu_grad(d, x, w, dW=one, act=name, Z=z, beta_w=beta_w)
    assert torch.equal(one, dw)


@pytest.mark.parametrize("dt,M,F,K", [("f32", 1536, 1664, 2048), ("f16", 2048, 2304, 2176),
                                      ("f16", 2050, 2304, 2183), ("f32", 1536, 1664, 2051),
                                      ("f16", 2048, 3712, 4096)])
def test_glu_grad_large(dt, M, F, K):
    """Sizes at which the products run one after the other, and beside them those
    whose rows do not start at 16 bytes; the reference in 64 bits on the GPU."""
    import dense_gemm_fp32_amd as dg
    note("glu_grad large %s %d %d %d" % (dt, M, F, K))
    g, t = torch.Generator(device=GPU), DT[dt]
    g.manual_seed(M)
    draw = lambda s, q: (torch.randn(*s, generator=g, device=GPU) * q).to(t)  # noqa: E731
    X, W, dH = draw((M, K), 1.0), draw((2 * F, K), K ** -0.5), draw((M, F), 0.05)
    oldx, oldw = draw((M, K), 0.1), draw((2 * F, K), 0.1)
    want = ref.glu_grad(dH, X, W, None, "silu", oldx, oldw, 1.0, 1.0, t)
    dX, dW = oldx.clone(), oldw.clone()
    dg.glu_grad(dH, X, W, dX=dX, dW=dW, beta_x=1.0, beta_w=1.0)
    for got, (value, bound) in ((dX, want["dX"]), (dW, want["dW"])):
        assert worst(got, value.cpu(), bound.cpu()) <= 1.0


class KernelNode(ctypes.Structure):
    """hipKernelNodeParams"""
    _fields_ = [("block", ctypes.c_uint * 3), ("extra", ctypes.c_void_p), ("func", ctypes.c_void_p),
                ("grid", ctypes.c_uint * 3), ("params", ctypes.c_void_p),
                ("shared", ctypes.c_uint)]


def kernels_of(call):
    """Names of the kernels that call() launches, from a graph of them that is never
    replayed."""
    from dense_gemm_fp32_amd import binding
    lib = binding._lib
    lib.hipKernelNameRefByPtr.restype = ctypes.c_char_p
    lib.hipKernelNameRefByPtr.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    raw, n = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t()
    assert lib.hipGraphGetNodes(raw, None, ctypes.byref(n)) == 0
    nodes = (ctypes.c_void_p * max(n.value, 1))()
    assert lib.hipGraphGetNodes(raw, nodes, ctypes.byref(n)) == 0
    names = []
    for node in nodes[:n.value]:
        p = KernelNode()
        assert lib.hipGraphKernelNodeGetParams(ctypes.c_void_p(node), ctypes.byref(p)) == 0
        names.append(lib.hipKernelNameRefByPtr(p.func, None).decode())
    return names


def on_gpu(g, shape, dtype, std, ld=None):
    """Normal numbers on the GPU, in rows `ld` elements apart with NaN between them."""
    big = torch.full((shape[0], ld or shape[1]), math.nan, dtype=dtype, device=GPU)
    view = big[:, :shape[1]]
    view.copy_(torch.randn(*shape, generator=g, device=GPU) * std)
    return big, view


IN_TURN = [
    # dtype, M, F, K, distance of rows (None: K), act, Z given, beta_x, beta_w, dW in fp32
    ("f16", 2048, 3712, 4096, None, "gelu", True, 0.0, 0.0, False),
    ("f16", 2048, 3712, 4096, None, "silu", True, 0.0, 1.0, True),
    ("f16", 1100, 6800, 4100, 4104, "silu", False, 0.5, 0.0, True),
    ("f16", 2050, 3701, 4003, 4016, "gelu_tanh", True, -1.0, 0.5, False),
    ("f16", 17, (1 << 21) + 8, 16, None, "silu", True, 0.0, 0.0, False),
    ("f32", 1536, 1664, 2048, None, "gelu", True, 0.0, 0.0, False),
    ("f32", 1537, 1665, 2051, 2052, "silu", False, 0.0, 1.0, False),
    # (whether C is read decides how the first product is split)
    ("f32", 2760, 5504, 3344, None, "relu", True, 1.0, 0.0, False),
    ("f32", 2760, 5504, 3344, None, "silu", True, 0.0, 0.0, False),
]


def in_turn(case):
    """(call(dX, dW, stream, workspace), [old dX, old dW], reference's arguments)"""
    import dense_gemm_fp32_amd as dg
    dt, M, F, K, ld, name, kept, beta_x, beta_w, dw32 = case
    g, t = torch.Generator(device=GPU), DT[dt]
    g.manual_seed(M + F)
    X, W = on_gpu(g, (M, K), t, 1.0, ld)[1], on_gpu(g, (2 * F, K), t, K ** -0.5, ld)[1]
    dH = on_gpu(g, (M, F), t, 0.05)[1]
    Z = on_gpu(g, (M, 2 * F), t, 1.0)[1] if kept else None
    tw = torch.float32 if dw32 else t
    old = [on_gpu(g, (M, K), t, 0.1 if beta_x else math.nan, ld),
           on_gpu(g, (2 * F, K), tw, 0.1 if beta_w else math.nan, ld)]

    def call(dX, dW, stream=None, workspace=None):
        dg.glu_grad(dH, X, W, dX=dX, dW=dW, act=name, Z=Z, beta_x=beta_x, beta_w=beta_w,
                    stream=stream, workspace=workspace)
    return call, old, (dH, X, W, Z, name, old[0][1], old[1][1], beta_x, beta_w, tw)


@pytest.mark.parametrize("case", IN_TURN, ids=lambda c: "x".join(map(str, c)))
def test_glu_grad_products_in_turn(case):
    """Gradients whose products run one after the other: with and without Z, in either
    type of dW, over outputs that are not read, columns that end inside 16 bytes, one
    output alone; the reference in 64 bits on the GPU."""
    dt, M, F, K, ld = case[:5]
    note("glu_grad in turn %r" % (case,))
    call, old, args = in_turn(case)
    want = ref.glu_grad(*args)
    bigs, outs = zip(*((b, b[:, :K]) for b in (o[0].clone() for o in old)))
    call(*outs)
    torch.cuda.synchronize()
    for out, big, n in zip(outs, bigs, ("dX", "dW")):
        assert worst(out, *(v.cpu() for v in want[n])) <= 1.0, n
        assert pads_intact(big, K)
    for i in (0, 1):
        one = old[i][1].clone()
        call(*((one, None) if i == 0 else (None, one)))
        assert torch.equal(one, outs[i])
    names = kernels_of(lambda: call(*outs))
    assert not any("proj_products" in k for k in names), names


@pytest.mark.parametrize("dt,M,F,K,ld", [("f16", 257, 1024, 1024, None), ("f16", 1024, 6000, 5200, None),
                                         ("f16", 2048, 2304, 2176, None), ("f16", 1100, 40, 61, None),
                                         ("f16", 17, 4082, 72, 73), ("f32", 1000, 1500, 517, None),
                                         ("f32", 1300, 1800, 2051, None)])
def test_glu_grad_products_in_one_launch(dt, M, F, K, ld):
    """Which sizes take the one launch of both products: fewer rows than 1025 or less
    work in fp16, less work in fp32, rows that do not start at 16 bytes."""
    import dense_gemm_fp32_amd as dg
    g, t = torch.Generator(device=GPU), DT[dt]
    g.manual_seed(M)
    X, W, dH = (on_gpu(g, s, t, 0.1, ld if s[1] == K else None)[1]
                for s in ((M, K), (2 * F, K), (M, F)))
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    names = kernels_of(lambda: dg.glu_grad(dH, X, W, dX=dX, dW=dW))
    assert sum("proj_products" in k for k in names) == 1, names


@pytest.mark.parametrize("case", [IN_TURN[1], IN_TURN[2], IN_TURN[3], IN_TURN[6], IN_TURN[7]],
                         ids=lambda c: "x".join(map(str, c)))
def test_glu_grad_products_in_turn_as_they_are_called(case, monkeypatch):
    """The same bits again, on another stream, in a workspace of exactly the bytes named
    (nothing beyond it is written, a smaller one is refused) and in captured graphs, two
    of them alive, each with a workspace of its own."""
    import dense_gemm_fp32_amd as dg
    from dense_gemm_fp32_amd import binding
    note("glu_grad in turn, calls %r" % (case,))
    call, old, args = in_turn(case)
    plain, needs = binding._call_rows, []

    def watch(fn, dev, stream, workspace, need, rest):
        needs.append(need)
        return plain(fn, dev, stream, workspace, need, rest)
    monkeypatch.setattr(binding, "_call_rows", watch)
    fresh = lambda: [o[1].clone() for o in old]  # noqa: E731
    want = fresh()
    call(*want)
    need = needs[0]
    side = torch.cuda.Stream()
    room = torch.full((need + 4096,), 170, dtype=torch.uint8, device=GPU)
    for how in (dict(), dict(stream=side), dict(workspace=room[:need])):
        outs = fresh()
        torch.cuda.synchronize()
        call(*outs, **how)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), how
    assert bool((room[need:] == 170).all())
    with pytest.raises(dg.GemmError, match="too small"):
        call(*fresh(), workspace=room[:need - 256])
    graphs, X = [], args[1]
    outs = fresh()
    for _ in range(2):
        space = torch.empty(need, dtype=torch.uint8, device=GPU)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(*outs, workspace=space)
        graphs.append((graph, space))
    for k in range(4):
        X.mul_(-0.75)
        want = fresh()
        call(*want)
        for o, v in zip(outs, fresh()):
            o.copy_(v)
        torch.cuda.synchronize()
        graphs[k % 2][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k


@pytest.mark.parametrize("M", [17, 33, 49])
def test_glu_grad_widest(M):
    """A width at which the rows of [dG dU] pass 8 MiB, in rows of X and W that
    start anywhere."""
    import dense_gemm_fp32_amd as dg
    F, K, t = (1 << 21) + 5, 17, torch.float16
    note("glu_grad widest %d" % M)
    g = torch.Generator(device=GPU)
    g.manual_seed(M)
    draw = lambda s, q: (torch.randn(*s, generator=g, device=GPU) * q).to(t)  # noqa: E731
    X, W, dH = draw((M, K), 1.0), draw((2 * F, K), K ** -0.5), draw((M, F), 0.05)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    dg.glu_grad(dH, X, W, dX=dX, dW=dW, act="silu")
    want = ref.glu_grad(dH, X, W, None, "silu", None, None, 0.0, 0.0, t)
    assert worst(dX, *(v.cpu() for v in want["dX"])) <= 1.0
    assert worst(dW, *(v.cpu() for v in want["dW"])) <= 1.0


@pytest.mark.parametrize("name", ref.ACTS)
def test_glu_grad_against_differences(name):
    """sum(dH * H(X, W)) moved along a direction of X and one of W, both sides in
    the library's fp32: differences of step h leave h^2 and u/h."""
    import dense_gemm_fp32_amd as dg
    g = gen(5)
    M, F, K = 40, 72, 96
    X, W, dH = (normal(g, s, torch.float32, q).to(GPU) for s, q in
                (((M, K), 1.0), ((2 * F, K), 0.1), ((M, F), 1.0)))
    vx, vw = normal(g, (M, K), torch.float32).to(GPU), normal(g, (2 * F, K), torch.float32).to(GPU)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    dg.glu_grad(dH, X, W, dX=dX, dW=dW, act=name)

    def loss(x, w):
        h = torch.empty(M, F, device=GPU)
        dg.glu(x, w, h, act=name)
        return float((h.double() * dH.double()).sum())
    h = 2.0 ** -9
    for slope, f in ((float((dX.double() * vx.double()).sum()), lambda s: loss(X + s * vx, W)),
                     (float((dW.double() * vw.double()).sum()),
                      lambda s: loss(X, W + s * 0.1 * vw) * 10)):
        diff = (f(h) - f(-h)) / (2 * h)
        # M F terms of order 1, third derivatives of order K^1.5 / 1000 (relu: kinks
        # within h of a gate, a share h of them): both well under 1% of the norm
        size = math.sqrt(M * F * K)
        assert abs(diff - slope) <= 0.02 * size


@pytest.mark.parametrize("kept", [True, False])
@pytest.mark.parametrize("M,F", [(1, 1), (40, 3), (700, 600)])
def test_halves_of_the_gate_s_gradients(M, F, kept):
    """dG and dU of halves are rounded once, ties to even, with subnormal numbers kept
    and an overflow infinite: seen through weights of 2^10 and an fp32 dW.  Every sum is
    of multiples of 2^-24 (2^-34 in dW), fewer than 2^24 of them: exact in any order."""
    import dense_gemm_fp32_amd as dg
    g, t = gen(M), torch.float16
    dH = (torch.randint(-40, 41, (M, F), generator=g) * 2.0 ** -24).to(t)
    up = 0.125 * (1 + torch.arange(M) % 7).to(t)[:, None]
    # G = 1, U = up: X = [2^-10, up, 0 ..], gate rows [2^10, 0 ..], up rows [0, 1, 0 ..]
    X, W = torch.zeros(M, 8, dtype=t), torch.zeros(2 * F, 8, dtype=t)
    X[:, 0], X[:, 1:2], W[:F, 0], W[F:, 1] = 2.0 ** -10, up, 2.0 ** 10, 1.0
    Z = torch.cat((torch.ones(M, F), up.expand(M, F)), 1).to(t) if kept else None
    D = torch.cat((dH.double() * up.double(), dH.double()), 1)
    assert M == 1 or float((D.half().double() - D).abs().max()) == 2.0 ** -25
    D = D.half().double()                      # torch's rounding: to even, subnormals kept
    dX, dW = torch.empty(M, 8, dtype=t, device=GPU), torch.empty(2 * F, 8, device=GPU)
    args = [v.to(GPU) for v in (dH, X, W)]
    z = None if Z is None else Z.to(GPU)
    dg.glu_grad(*args, dX=dX, dW=dW, act="relu", Z=z)
    assert torch.equal(dX.cpu(), (D @ W.double()).half())
    assert torch.equal(dW.cpu(), (D.t() @ X.double()).float())
    args[0][M - 1, F - 1], args[1][M - 1, 1] = 60000.0, 2.0
    if z is not None:
        z[M - 1, F:] = 2.0
    dg.glu_grad(*args, dX=dX, dW=dW, act="relu", Z=z)
    dX = dX.cpu()
    assert torch.isinf(dX[M - 1, 0]) and torch.isfinite(dX[:M - 1]).all()


def test_glu_grad_degenerate():
    import dense_gemm_fp32_amd as dg
    t = torch.float16
    e = lambda *s: torch.empty(*s, dtype=t, device=GPU)  # noqa: E731
    dw = torch.ones(8, 6, dtype=t, device=GPU)
    dg.glu_grad(e(0, 4), e(0, 6), e(8, 6), dX=e(0, 6), dW=dw, beta_w=2.0)
    assert bool((dw == 2).all())
    dw32 = torch.full((8, 6), math.nan, device=GPU)
    dg.glu_grad(e(0, 4), e(0, 6), e(8, 6), dW=dw32)
    assert not dw32.any()
    dx = torch.ones(3, 6, dtype=t, device=GPU)
    dg.glu_grad(e(3, 0), e(3, 6), e(0, 6), dX=dx, dW=e(0, 6), beta_x=3.0)
    assert bool((dx == 3).all())


# ---------------------------------------------------------------- together, and how they are called

def block_i8(dg, X, W1, s1, W2, s2, Q, xs, H, Q2, hs, Y, stream=None):
    """A feed-forward block in 8-bit integers, as a model calls it."""
    dg.quantize(X, Q, xs, stream=stream)
    dg.glu(Q, W1, H, x_scale=xs, w_scale=s1, stream=stream)
    dg.quantize(H, Q2, hs, stream=stream)
    return dg.gemm_i8(Q2, W2, Y, x_scale=hs, w_scale=s2, beta=1.0, stream=stream)


def block_inputs(M, D, F, seed):
    g = gen(seed)
    X = normal(g, (M, D), torch.float16)
    W1, s1 = ref.quantize(normal(g, (2 * F, D), torch.float32, D ** -0.5))
    W2, s2 = ref.quantize(normal(g, (D, F), torch.float32, F ** -0.5))
    return X, W1, s1, W2, s2


def block_buffers(M, D, F):
    e = lambda *s, dtype=torch.float16: torch.empty(*s, dtype=dtype, device=GPU)  # noqa: E731
    return (e(M, D, dtype=torch.int8), e(M, dtype=torch.float32), e(M, F),
            e(M, F, dtype=torch.int8), e(M, dtype=torch.float32))


@pytest.mark.parametrize("M,D,F", [(1, 512, 256), (40, 512, 768), (300, 320, 640)])
def test_block_in_8_bits(M, D, F):
    """Each step against the 64-bit reference of what the step before left."""
    import dense_gemm_fp32_amd as dg
    X, W1, s1, W2, s2 = block_inputs(M, D, F, M)
    Q, xs, H, Q2, hs = bufs = block_buffers(M, D, F)
    Y = X.to(GPU)
    block_i8(dg, Y.clone(), W1.to(GPU), s1.to(GPU), W2.to(GPU), s2.to(GPU), *bufs, Y)
    torch.cuda.synchronize()
    q, s = ref.quantize(X)
    assert torch.equal(Q.cpu(), q) and torch.equal(xs.cpu(), s)
    assert worst(H, *ref.glu(q, W1, "silu", torch.float16, s, s1)["H"]) <= 1.0
    q, s = ref.quantize(H.cpu())
    assert torch.equal(Q2.cpu(), q) and torch.equal(hs.cpu(), s)
    assert worst(Y, *ref.gemm_i8(q, W2, X, s, s2, 1.0, 1.0, torch.float16)) <= 1.0


@pytest.mark.parametrize("kept", [False, True])
def test_training_step_of_a_block(kept):
    """Y = glu(X) W2^T and back, every step with the library: each gradient
    against the reference of what the step before left."""
    import dense_gemm_fp32_amd as dg
    g, t = gen(9), torch.float16
    M, D, F = 200, 256, 384
    X, W1 = normal(g, (M, D), t), normal(g, (2 * F, D), t, D ** -0.5)
    W2, dY = normal(g, (D, F), t, F ** -0.5), normal(g, (M, D), t, 0.05)
    x, w1, w2, dy = (v.to(GPU) for v in (X, W1, W2, dY))
    H, dH = (torch.empty(M, F, dtype=t, device=GPU) for _ in range(2))
    Z = torch.empty(M, 2 * F, dtype=t, device=GPU) if kept else None
    Y = x.clone()
    dg.glu(x, w1, H, Z=Z)
    dg.gemm(H, w2.t(), Y, beta=1.0)
    dg.gemm(dy, w2, dH)
    dX, dW1 = dy.clone(), torch.zeros(2 * F, D, device=GPU)
    for _ in range(2):       # two batches into one fp32 gradient
        dg.glu_grad(dH, x, w1, dX=dX if _ == 0 else None, dW=dW1, Z=Z, beta_x=1.0, beta_w=1.0)
    torch.cuda.synchronize()
    want = ref.glu_grad(dH.cpu(), X, W1, None if Z is None else Z.cpu(), "silu", dY, None, 1.0, 0,
                        torch.float32)
    assert worst(dX, *want["dX"]) <= 1.0
    value, bound = want["dW"]
    assert worst(dW1, 2 * value, 2 * bound + 2 ** -22 * value.abs()) <= 1.0


CALLS = ["quantize", "gemm_i8", "gemm_i8 many", "gemm_i8 odd", "glu", "glu many", "glu odd",
         "glu f32", "glu_i8", "glu_i8 many", "glu_grad", "glu_grad odd", "glu_grad f32"]


def call_of(name):
    """(call(stream, workspace), outputs, inputs that a caller may fill anew)"""
    import dense_gemm_fp32_amd as dg
    g = gen(len(name))
    M, F, K = {"many": (700, 528, 320), "odd": (130, 131, 259)}.get(name.split()[-1],
                                                                   (40, 192, 256))
    t = torch.float32 if "f32" in name else torch.float16
    X, W = normal(g, (M, K), t).to(GPU), normal(g, (2 * F, K), t, K ** -0.5).to(GPU)
    q, w = whole(g, (M, K)).to(GPU), whole(g, (2 * F, K)).to(GPU)
    xs, ws = scales(g, M).to(GPU), (scales(g, 2 * F) / math.sqrt(K)).to(GPU)
    if name == "quantize":
        out = torch.empty(M, K, dtype=torch.int8, device=GPU), torch.empty(M, device=GPU)
        return (lambda s, v: dg.quantize(X, *out, stream=s)), out, [X]
    if name.startswith("gemm_i8"):
        out = torch.empty(M, 2 * F, dtype=t, device=GPU)
        return (lambda s, v: dg.gemm_i8(q, w, out, x_scale=xs, w_scale=ws, workspace=v,
                                        stream=s)), (out,), [xs]
    if name.startswith("glu_grad"):
        dH = normal(g, (M, F), t, 0.05).to(GPU)
        out = torch.empty_like(X), torch.empty_like(W)
        return (lambda s, v: dg.glu_grad(dH, X, W, *out, workspace=v, stream=s)), out, [X, dH]
    out = torch.empty(M, F, dtype=t, device=GPU)
    if name.startswith("glu_i8"):
        return (lambda s, v: dg.glu(q, w, out, x_scale=xs, w_scale=ws, workspace=v,
                                    stream=s)), (out,), [xs]
    return (lambda s, v: dg.glu(X, W, out, workspace=v, stream=s)), (out,), [X]


def clear(outs):
    for o in outs:
        o.fill_(77 if o.dtype == torch.int8 else math.nan)


@pytest.mark.parametrize("name", CALLS)
def test_calls_repeat_bit_for_bit_on_any_stream(name):
    call, outs, _ = call_of(name)
    call(None, None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    room = torch.empty(64 << 20, dtype=torch.uint8, device=GPU)
    for how in ("again", "stream", "raw", "current", "workspace"):
        clear(outs)
        torch.cuda.synchronize()
        if how == "again":
            call(None, None)
        elif how == "stream":
            call(side, None)
        elif how == "raw":
            call(side.cuda_stream, None)
        elif how == "current":
            with torch.cuda.stream(side):
                call(None, None)
        else:
            room.fill_(255)      # nothing in it needs an initial value
            call(None, room)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), how


@pytest.mark.parametrize("name", CALLS)
def test_calls_in_a_graph(name):
    """Captured and replayed with new inputs, eager calls and synchronisations
    between the replays; two graphs alive, each with a workspace of its own."""
    call, outs, inputs = call_of(name)
    call(None, None)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        room = torch.empty(64 << 20, dtype=torch.uint8, device=GPU)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(None, room)
        graphs.append((graph, room))
    for k in range(4):
        for t in inputs:
            t.mul_(-0.75)
        call(None, None)
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        clear(outs)
        torch.cuda.synchronize()
        graphs[k % 2][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k


@pytest.mark.parametrize("name", CALLS)
def test_workspaces_of_the_size_named(name, monkeypatch):
    """A workspace of the bytes that the *_workspace function names is enough and
    nothing beyond it is written; one that is smaller is refused."""
    from dense_gemm_fp32_amd import binding
    import dense_gemm_fp32_amd as dg
    if name == "quantize":
        return
    call, outs, _ = call_of(name)
    seen = []
    plain = binding._call_rows

    def watch(fn, dev, stream, workspace, need, args):
        seen.append(need)
        return plain(fn, dev, stream, workspace, need, args)
    monkeypatch.setattr(binding, "_call_rows", watch)
    call(None, None)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    need = seen[0]
    room = torch.full((need + 4096,), 170, dtype=torch.uint8, device=GPU)
    clear(outs)
    call(None, room[:need] if need else None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert bool((room[need:] == 170).all())
    if need:
        with pytest.raises(dg.GemmError, match="too small"):
            call(None, room[:need - 256])
        with pytest.raises(dg.GemmError, match="aligned"):
            call(None, room[1:])


@pytest.mark.parametrize("name", ["gemm_i8 odd", "glu odd", "glu_grad", "glu many"])
def test_calls_at_once_on_two_streams(name):
    """Two calls under way at the same time, each with outputs of its own."""
    first, second = call_of(name), call_of(name)
    first[0](None, None)
    torch.cuda.synchronize()
    want = [o.clone() for o in first[1]]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    clear(first[1])
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (call, outs, _) in zip(streams, (first, second)):
            call(s, None)
    torch.cuda.synchronize()
    for _, outs, _ in (first, second):
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_rows_beyond_32_bits():
    """Rows more than 2^31 elements from the first."""
    import dense_gemm_fp32_amd as dg
    g = gen(1)
    far = (1 << 30) + 64          # three rows of it
    K, N = 96, 80
    X, W = whole(g, (3, K)), whole(g, (2 * N, K))
    big = torch.zeros(2 * far + K, dtype=torch.int8, device=GPU)
    x = big.as_strided((3, K), (far, 1))
    x.copy_(X)
    y = torch.empty(3, 2 * N, device=GPU)
    dg.gemm_i8(x, W.to(GPU), y)
    assert torch.equal(y.cpu().double(), X.double() @ W.double().t())
    w = big.as_strided((3, K), (far, 1))
    dg.gemm_i8(W.to(GPU), w, torch.empty(2 * N, 3, device=GPU))
    out = torch.empty(2 * N, 3, device=GPU)
    dg.gemm_i8(W.to(GPU), w, out)
    assert torch.equal(out.cpu().double(), (W.double() @ X.double().t()))
    del big, x, w
    t = torch.float16
    far = (1 << 30) + 8
    big = torch.zeros(2 * far + 4 * N, dtype=t, device=GPU)
    Xh, Wh = normal(g, (3, K), t), normal(g, (2 * N, K), t, 0.1)
    want = ref.glu(Xh, Wh, "gelu", t)
    h = big.as_strided((3, N), (far, 1))
    z = torch.empty(3, 2 * N, dtype=t, device=GPU)
    dg.glu(Xh.to(GPU), Wh.to(GPU), h, act="gelu", Z=z)
    assert worst(h.cpu(), *want["H"]) <= 1.0
    z2 = big.as_strided((3, 2 * N), (far, 1))
    dg.glu(Xh.to(GPU), Wh.to(GPU), torch.empty(3, N, dtype=t, device=GPU), act="gelu", Z=z2)
    assert torch.equal(z2, z)
    dH = normal(g, (3, N), t, 0.05).to(GPU)
    near, apart = torch.empty(3, K, dtype=t, device=GPU), big.as_strided((3, K), (far, 1))
    dg.glu_grad(dH, Xh.to(GPU), Wh.to(GPU), dX=near, act="gelu", Z=z)
    z2.copy_(z)
    dg.glu_grad(dH, Xh.to(GPU), Wh.to(GPU), dX=torch.empty_like(near), act="gelu", Z=z2)
    dg.glu_grad(dH, Xh.to(GPU), Wh.to(GPU), dX=apart, act="gelu", Z=z)
    assert torch.equal(apart, near)


def test_gradients_of_rows_beyond_32_bits():
    """dH, the kept [G U], X and both outputs in rows more than 2^31 elements from the
    first: the bits of the same rows close together."""
    import dense_gemm_fp32_amd as dg
    g, t = gen(4), torch.float16
    far, F, K = (1 << 30) + 8, 80, 96
    X, W = normal(g, (3, K), t).to(GPU), normal(g, (2 * F, K), t, 0.1).to(GPU)
    dH, Z = normal(g, (3, F), t, 0.05).to(GPU), normal(g, (3, 2 * F), t).to(GPU)
    near = torch.empty(3, K, dtype=t, device=GPU), torch.empty(2 * F, K, dtype=t, device=GPU)
    dg.glu_grad(dH, X, W, *near, act="gelu", Z=Z)
    want = ref.glu_grad(dH.cpu(), X.cpu(), W.cpu(), Z.cpu(), "gelu", None, None, 0, 0, t)
    assert worst(near[0], *want["dX"]) <= 1.0 and worst(near[1], *want["dW"]) <= 1.0
    big = torch.zeros(2 * far + 1024, dtype=t, device=GPU)
    apart = lambda cols, at: big[at:].as_strided((3, cols), (far, 1))  # noqa: E731
    z, d = apart(2 * F, 0).copy_(Z), apart(F, 256).copy_(dH)
    for h, kept in ((dH, z), (d, Z), (d, z)):
        out = torch.full_like(near[0], math.nan), torch.full_like(near[1], math.nan)
        dg.glu_grad(h, X, W, *out, act="gelu", Z=kept)
        assert all(torch.equal(a, b) for a, b in zip(out, near))
    # rows of X are copied, so the sums' order may be another one
    x, dx = apart(K, 512).copy_(X), apart(K, 768)
    dw = torch.full_like(near[1], math.nan)
    dg.glu_grad(d, x, W, dX=dx, dW=dw, act="gelu", Z=z)
    assert worst(dx, *want["dX"]) <= 1.0 and worst(dw, *want["dW"]) <= 1.0


MOST = 1 << 24


@pytest.mark.parametrize("what", ["rows", "columns of few rows", "columns of many rows"])
def test_products_of_the_most_rows_and_columns(what):
    """As many rows, or rows of W, as a call takes, 4096 of them over and over: whole
    numbers, so that the results are those of the 4096 bit for bit."""
    import dense_gemm_fp32_amd as dg
    P, K = 4096, 16
    note("products of the most %s" % what)
    g = gen(len(what))
    M, N = (MOST, 6) if what == "rows" else (3 if "few" in what else 70, MOST)
    X, W = whole(g, (min(M, P), K)), whole(g, (min(N, P), K))
    xs, ws = 2.0 ** -(torch.arange(len(X)) % 5), 2.0 ** -(torch.arange(len(W)) % 7)
    S = (X.double() @ W.double().t()) * xs.double()[:, None] * ws.double()[None, :]
    over = lambda t, n: t.to(GPU).repeat(n // len(t), *(1,) * (t.dim() - 1))  # noqa: E731
    x, w, a, b = over(X, M), over(W, N), over(xs, M), over(ws, N)
    y = torch.full((M, N), math.nan, device=GPU)
    dg.gemm_i8(x, w, y, x_scale=a, w_scale=b)
    want = S.float().to(GPU)
    assert bool((y.view(M // len(X), len(X), N // len(W), len(W)) == want[:, None]).all())


@pytest.mark.parametrize("what", ["rows", "columns of few rows", "columns of many rows"])
def test_blocks_of_the_most_rows_and_columns(what):
    """The same of gated blocks and their gradients: relu of whole numbers."""
    import dense_gemm_fp32_amd as dg
    P, K, t = 4096, 8, torch.float16
    note("blocks of the most %s" % what)
    g = gen(len(what))
    M, F = (MOST, 2) if what == "rows" else (3 if "few" in what else 70, MOST // 2)
    small = lambda *s: torch.randint(-2, 3, s, generator=g).to(t)  # noqa: E731
    X, G, U = small(min(M, P), K), small(min(F, P), K), small(min(F, P), K)
    dH = torch.zeros(min(M, P), min(F, P))
    dH[::16, ::max(1, F // 32768)] = 1.0  # few: sums stay below 2^24
    over = lambda v, n: v.to(GPU).repeat(n // len(v), 1)  # noqa: E731
    x, w = over(X, M), torch.cat((over(G, F), over(U, F)))
    d = dH.to(t).to(GPU).repeat(M // len(dH), F // dH.shape[1])
    g1, u1 = X.float() @ G.float().t(), X.float() @ U.float().t()
    H = (g1.clamp(min=0) * u1).to(GPU)
    h = torch.full((M, F), math.nan, dtype=t, device=GPU)
    dg.glu(x, w, h, act="relu")
    periods = (M // len(X), len(X), F // len(G), len(G))
    assert bool((h.view(periods).float() == H.half().float()[:, None]).all())
    del h
    dX = torch.full((M, K), math.nan, dtype=t, device=GPU)
    dW = torch.full((2 * F, K), math.nan, device=GPU)
    dg.glu_grad(d, x, w, dX=dX, dW=dW, act="relu")
    dG, dU = dH * u1 * (g1 > 0), dH * g1.clamp(min=0)
    once = (dG.double() @ G.double() + dU.double() @ U.double()) * periods[2]
    assert float(once.abs().max()) < 2 ** 24
    assert bool((dX.view(-1, len(X), K) == once.float().half().to(GPU)).all())
    for part, D in ((dW[:F], dG), (dW[F:], dU)):
        sums = (D.double().t() @ X.double()) * periods[0]
        assert float(sums.abs().max()) < 2 ** 24
        assert bool((part.view(-1, len(G), K) == sums.float().to(GPU)).all())


@pytest.mark.parametrize("N", [6016, 6600])
def test_many_rows_far_apart(N):
    """200 rows, 2^24 bytes from one to the next: operands are copied for the tiles
    (the more columns) or streamed, outputs are written where they lie.  Another way
    sums in another order, so halves are held to the reference."""
    import dense_gemm_fp32_amd as dg
    g = gen(2)
    M, K, far, t = 200, 144, (1 << 24) + 16, torch.float16
    X, W = whole(g, (M, K)), whole(g, (N, K))
    big = torch.zeros(M * far, dtype=torch.int8, device=GPU)
    x = big.as_strided((M, K), (far, 1))
    x.copy_(X)
    near, w = torch.empty(M, N, device=GPU), W.to(GPU)
    dg.gemm_i8(X.to(GPU), w, near)
    assert torch.equal(near.cpu().double(), X.double() @ W.double().t())
    out = torch.empty(M, N, device=GPU)
    dg.gemm_i8(x, w, out)
    assert torch.equal(out, near)
    wide = big.view(torch.float32).as_strided((M, N), (far // 4, 1))
    dg.gemm_i8(X.to(GPU), w, wide)
    assert torch.equal(wide, near)
    F = N // 2
    X, W, dH = normal(g, (M, K), t), normal(g, (N, K), t, 0.1), normal(g, (M, F), t, 0.05)
    xh, wh, d = X.to(GPU), W.to(GPU), dH.to(GPU)
    half = big.view(t)
    xf, zf = half.as_strided((M, K), (far // 2, 1)), half[K:].as_strided((M, N), (far // 2, 1))
    want = ref.glu(X, W, "silu", t)
    h, z = torch.empty(M, F, dtype=t, device=GPU), torch.empty(M, N, dtype=t, device=GPU)
    dg.glu(xh, wh, h, Z=zf)
    assert worst(h, *want["H"]) <= 1.0 and worst(zf, *want["Z"]) <= 1.0
    xf.copy_(xh)
    dg.glu(xf, wh, h, Z=z)
    assert worst(h, *want["H"]) <= 1.0 and worst(z, *want["Z"]) <= 1.0
    want = ref.glu_grad(dH, X, W, z.cpu(), "silu", None, None, 0, 0, t)
    a = [torch.empty(M, K, dtype=t, device=GPU), torch.empty(N, K, dtype=t, device=GPU)]
    for rows, kept in ((xh, z), (xf, z), (xh, zf.copy_(z))):
        dg.glu_grad(d, rows, wh, *a, Z=kept)
        assert worst(a[0], *want["dX"]) <= 1.0 and worst(a[1], *want["dW"]) <= 1.0


def test_wrappers_refuse_on_the_gpu():
    import dense_gemm_fp32_amd as dg
    h = torch.zeros(4, 8, dtype=torch.float16, device=GPU)
    q = torch.zeros(4, 8, dtype=torch.int8, device=GPU)
    w, wq = torch.zeros(6, 8, dtype=torch.float16, device=GPU), torch.zeros(6, 8, dtype=torch.int8,
                                                                            device=GPU)
    out = torch.zeros(4, 3, dtype=torch.float16, device=GPU)
    for match, call in (
            ("Z goes", lambda: dg.glu(q, wq, out, Z=torch.zeros(4, 6, dtype=torch.float16,
                                                                device=GPU))),
            ("x_scale", lambda: dg.glu(h, w, out, x_scale=torch.ones(4, device=GPU))),
            ("W must be", lambda: dg.glu(h, wq, out)), ("W must be", lambda: dg.glu(q, w, out)),
            ("W must be 6 x 8", lambda: dg.glu(h, w[:5], out)),
            ("H must be", lambda: dg.glu(h[:3], w, out)),
            ("rows", lambda: dg.glu(h, w.t().contiguous().t(), out)),
            ("x_scale must be 4", lambda: dg.gemm_i8(q, wq, torch.zeros(4, 6, device=GPU),
                                                     x_scale=torch.ones(3, device=GPU))),
            ("w_scale must be 6", lambda: dg.gemm_i8(q, wq, torch.zeros(4, 6, device=GPU),
                                                     w_scale=torch.ones(6, device=GPU).half())),
            ("act must be", lambda: dg.glu(h, w, out, act="tanh")),
            ("dW must be", lambda: dg.glu_grad(out, h, w, dW=w.double())),
            ("Q must be", lambda: dg.quantize(h, torch.zeros(4, 7, dtype=torch.int8, device=GPU))),
            ("scale must be", lambda: dg.quantize(h, q, torch.zeros(5, device=GPU)))):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(dg.GemmError, match="131071"):
        dg.gemm_i8(torch.zeros(1, 131072, dtype=torch.int8, device=GPU),
                   torch.zeros(1, 131072, dtype=torch.int8, device=GPU),
                   torch.zeros(1, 1, device=GPU))
