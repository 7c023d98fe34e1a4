"""Products of 8-bit integers and gated blocks: argument checks, workspace sizes
and the references, without a GPU."""
import math

import pytest
import torch

import blocks_reference as ref

P = 1 << 20      # a device address that is never read: the checks come first


def entry(name, args):
    import dense_gemm_fp32_amd as dg
    return getattr(dg, name)(*args.values())


QUANT = dict(M=4, K=8, X=P, ldx=8, Q=P, ldq=8, scale=P, stream=None)
QUANT_BAD = [
    (-601, dict(M=-1)), (-601, dict(M=(1 << 24) + 1)), (-602, dict(K=-1)), (-604, dict(ldx=7)),
    (-606, dict(ldq=7)), (-604, dict(K=0, ldx=0)), (-603, dict(X=None)), (-605, dict(Q=None)),
    (-607, dict(scale=None)), (0, dict(M=0, X=None, Q=None, scale=None)),
]
I8 = dict(M=4, N=6, K=8, alpha=1.0, X=P, ldx=8, x_scale=None, W=P, ldw=8, w_scale=None, beta=0.0,
          Y=P, ldy=6, workspace=P, workspace_bytes=1 << 30, stream=None)
I8_BAD = [
    (-701, dict(M=-1)), (-701, dict(M=(1 << 24) + 1)), (-702, dict(N=-1)),
    (-702, dict(N=(1 << 24) + 1)), (-703, dict(K=-1)), (-703, dict(K=131072, ldx=131072)),
    (-706, dict(ldx=7)), (-709, dict(ldw=7)), (-713, dict(ldy=5)), (-705, dict(X=None)),
    (-708, dict(W=None)), (-712, dict(Y=None)), (-712, dict(K=0, X=None, W=None, Y=None)),
    (0, dict(M=0, X=None, Y=None)), (0, dict(N=0, W=None, Y=None)),
    (0, dict(K=0, beta=1.0, X=None, Y=None)), (0, dict(alpha=0.0, beta=1.0, W=None, Y=None)),
]
GLU = dict(M=4, F=6, K=8, act=0, X=P, ldx=8, W=P, ldw=8, H=P, ldh=6, Z=None, ldz=0, workspace=P,
           workspace_bytes=1 << 30, stream=None)
GLU_BAD = [
    (-801, dict(M=-1)), (-801, dict(M=(1 << 24) + 1)), (-802, dict(F=-1)),
    (-802, dict(F=(1 << 23) + 1)), (-803, dict(K=-1)), (-803, dict(K=(1 << 24) + 1)),
    (-804, dict(act=-1)), (-804, dict(act=4)), (-806, dict(ldx=7)), (-808, dict(ldw=7)),
    (-810, dict(ldh=5)), (-812, dict(Z=P, ldz=11)), (-805, dict(X=None)), (-807, dict(W=None)),
    (-809, dict(H=None)), (0, dict(M=0, X=None, H=None)), (0, dict(F=0, W=None, H=None)),
]
GLU_I8 = dict(M=4, F=6, K=8, act=0, X=P, ldx=8, x_scale=None, W=P, ldw=8, w_scale=None, H=P, ldh=6,
              workspace=P, workspace_bytes=1 << 30, stream=None)
GLU_I8_BAD = [
    (-901, dict(M=-1)), (-902, dict(F=(1 << 23) + 1)), (-903, dict(K=131072, ldx=131072)),
    (-904, dict(act=4)), (-906, dict(ldx=7)), (-909, dict(ldw=7)), (-912, dict(ldh=5)),
    (-905, dict(X=None)), (-908, dict(W=None)), (-911, dict(H=None)), (0, dict(M=0, X=None)),
]
GRAD = dict(M=4, F=6, K=8, act=0, dH=P, lddh=6, X=P, ldx=8, W=P, ldw=8, Z=None, ldz=0, beta_x=0.0,
            dX=P, lddx=8, beta_w=0.0, dW=P, lddw=8, workspace=P, workspace_bytes=0, stream=None)
GRAD_BAD = [
    (-1001, dict(M=-1)), (-1002, dict(F=(1 << 23) + 1)), (-1003, dict(K=-1)),
    (-1004, dict(act=7)), (-1006, dict(lddh=5)), (-1008, dict(ldx=7)), (-1010, dict(ldw=7)),
    (-1012, dict(Z=P, ldz=11)), (-1015, dict(lddx=7)), (-1018, dict(lddw=7)),
    (-1005, dict(dH=None)), (-1007, dict(X=None)), (-1009, dict(W=None)),
    (-1019, dict(workspace=P + 1)), (-1020, dict()),
    # with Z, X is read for dW only and W for dX only; what is not wanted is not looked at
    (-1020, dict(Z=P, ldz=12, dW=None, X=None, ldx=0, lddw=0)),
    (-1020, dict(Z=P, ldz=12, dX=None, W=None, ldw=0, lddx=0)),
    (-1007, dict(dW=None, X=None)), (-1009, dict(dX=None, W=None)),
    (0, dict(dX=None, dW=None, dH=None, X=None, W=None)), (0, dict(K=0, dH=None)),
    (0, dict(M=0, beta_w=1.0, dH=None)), (0, dict(F=0, beta_x=1.0, dH=None)),
]
ENTRIES = [("gemm_quant_i8", ("f16", "f32"), QUANT, QUANT_BAD, 600),
           ("gemm_i8", ("f16", "f32"), I8, I8_BAD, 700),
           ("gemm_glu", ("f16", "f32"), GLU, GLU_BAD, 800),
           ("gemm_glu_i8", ("f16", "f32"), GLU_I8, GLU_I8_BAD, 900),
           ("gemm_glu_grad", ("f16", "f16f32", "f32"), GRAD, GRAD_BAD, 1000)]
CHECKS = [(n, t, a, b, c) for n, ts, a, bad, b in ENTRIES for t in ts for c in bad]


@pytest.mark.parametrize("name,dt,args,base,case", CHECKS,
                         ids=lambda v: str(v) if not isinstance(v, tuple) else
                         "%d-%s" % (v[0], "-".join(v[1])))
def test_argument_checks(name, dt, args, base, case):
    import dense_gemm_fp32_amd as dg
    want, change = case
    assert entry("%s_%s" % (name, dt), dict(args, **change)) == want
    if want:
        assert dg.gemm_status_string(want).startswith("%s: invalid argument %d:"
                                                      % (name, -base - want))


def test_workspace_sizes():
    import dense_gemm_fp32_amd as dg
    for fn, dtypes, good in ((dg.gemm_glu_workspace, (0, 1, 2), (300, 520, 264)),
                             (dg.gemm_glu_grad_workspace, (0, 1), (300, 520, 264))):
        for dtype in dtypes:
            for aligned in (0, 1):
                n = fn(dtype, *good, aligned)
                assert n % 256 == 0 and n <= fn(dtype, *good, 0)
                for i in range(3):
                    assert fn(dtype, *(good[:i] + (0,) + good[i + 1:]), aligned) == 0
        assert fn(3, *good, 0) == 0 and fn(-1, *good, 0) == 0
    for aligned in (0, 1):
        assert dg.gemm_i8_workspace(300, 520, 264, aligned) % 256 == 0
        assert dg.gemm_i8_workspace(300, 520, 131072, aligned) == 0
        assert dg.gemm_i8_workspace((1 << 24) + 1, 520, 264, aligned) == 0
        # beyond 32 bits: [dG dU] alone
        assert dg.gemm_glu_grad_workspace(1, 1 << 22, 1 << 10, 64, aligned) >= 1 << 34
        assert dg.gemm_glu_workspace(2, 16, 16, 131072, aligned) == 0


def whole_rows(n, dt):
    """n elements filled up to whole 16 bytes."""
    v = 4 if dt == "f32" else 8
    return (n + v - 1) // v * v


def grad_call(dt, M, F, K, ws, odd=0, **change):
    """A call whose arguments are valid, for rows of X and W that start at 16 bytes, or
    (odd) do not."""
    ldk = whole_rows(K, dt) + odd
    return entry("gemm_glu_grad_" + dt, dict(
        GRAD, M=M, F=F, K=K, lddh=F, ldx=ldk, ldw=ldk, ldz=2 * F, lddx=K, lddw=K,
        workspace_bytes=ws, **change))


# The addresses are no memory: without a GPU a call whose arguments pass ends with the
# runtime's error, on a GPU it would run.
@pytest.mark.skipif(torch.cuda.is_available(), reason="would run on the GPU")
@pytest.mark.parametrize("dt", ["f32", "f16", "f16f32"])
def test_gradients_take_the_workspace_named_whatever_is_asked(dt):
    """Betas, the outputs' rows, which outputs are wanted and whether Z is kept change
    how the products of the backward pass are split, but never ask for more than
    gemm_glu_grad_workspace says."""
    import random
    import dense_gemm_fp32_amd as dg
    rng = random.Random(7)
    sizes = [(2760, 5504, 3344), (5376, 5632, 2560), (4608, 6912, 4096), (7040, 8160, 3824),
             (2464, 6176, 3152), (2992, 5392, 5808)]
    sizes += [tuple(rng.randrange(16, 8192) // 16 * 16 + rng.choice((0, 0, 0, 5))
                    for _ in range(3)) for _ in range(400)]
    changes = [dict(beta_x=bx, beta_w=bw, Z=z) for bx in (0.0, 1.0) for bw in (0.0, 1.0)
               for z in (None, P)]
    changes += [dict(beta_x=0.5, dW=None), dict(beta_w=-1.0, dX=None), dict(beta_x=math.nan),
                dict(dX=P + 4, dW=P + 4, beta_x=1.0, beta_w=1.0)]
    for s in sizes:
        for odd in (0, 1):
            need = dg.gemm_glu_grad_workspace(0 if dt == "f32" else 1, *s, 0 if odd else 1)
            for c in changes:
                assert grad_call(dt, *s, need, odd, **c) > 0, (s, odd, c)
            assert grad_call(dt, *s, 0, odd) == -1020


def test_wrappers_refuse():
    import dense_gemm_fp32_amd as dg
    h, q = torch.zeros(2, 4), torch.zeros(2, 4, dtype=torch.int8)
    with pytest.raises(ValueError, match="GPU"):
        dg.quantize(h)
    with pytest.raises(ValueError, match="GPU"):
        dg.gemm_i8(q, q, torch.zeros(2, 2))
    with pytest.raises(ValueError, match="GPU"):
        dg.glu(h, torch.zeros(6, 4), torch.zeros(2, 3))
    with pytest.raises(ValueError, match="GPU"):
        dg.glu_grad(torch.zeros(2, 3), h, torch.zeros(6, 4), dX=torch.zeros(2, 4))
    with pytest.raises(ValueError, match="dtype"):
        dg.quantize(h.double())
    with pytest.raises(ValueError, match="dtype"):
        dg.glu(q, q, torch.zeros(2, 1, dtype=torch.int8))
    from dense_gemm_fp32_amd import binding
    with pytest.raises(ValueError, match="silu, gelu"):
        binding._act("tanh")
    assert list(binding.ACTIVATIONS) == list(ref.ACTS)


def test_calls_without_workspace_run_on_the_tensors_gpu(monkeypatch):
    from dense_gemm_fp32_amd import binding
    now, calls = [0], []

    class Change:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.before, now[0] = now[0], self.dev

        def __exit__(self, *_):
            now[0] = self.before
    monkeypatch.setattr(binding, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Change)

    def fn(*args):
        calls.append((now[0],) + args)
        return 0
    for dev in (0, 1):
        binding._call(fn, dev, 5, (7,))
        assert calls[-1] == (dev, 7, 5) and now[0] == 0
    with pytest.raises(binding.GemmError):
        binding._call(lambda *a: -601, 0, 5, (7,))


def test_reference_quantize_by_hand():
    X = torch.tensor([[127.0, -0.5, 1.5, 2.5, -126.6], [0.0] * 5, [1.0, math.inf, 0, 0, 0],
                      [math.nan, 1.0, 0, 0, 0]])
    q, s = ref.quantize(X)
    assert q.tolist() == [[127, 0, 2, 2, -127], [0] * 5, [0] * 5, [0] * 5]
    assert s[0] == 1.0 and s[1] == 0.0 and math.isnan(s[2]) and math.isnan(s[3])


def test_reference_activations():
    """Values by hand, slopes by differences."""
    g = torch.tensor([0.0, 1.0, -2.0, 30.0, -30.0], dtype=torch.float64)
    e = math.exp
    assert torch.allclose(ref.act("silu", g)[0], torch.tensor(
        [0.0, 1 / (1 + e(-1)), -2 / (1 + e(2)), 30.0, -30 * e(-30)], dtype=torch.float64))
    assert abs(float(ref.act("gelu", g)[0][1]) - 0.8413447460685429) < 1e-15
    assert abs(float(ref.act("gelu_tanh", g)[0][1]) - 0.8411919906082768) < 1e-12
    assert ref.act("relu", g)[0].tolist() == [0.0, 1.0, 0.0, 30.0, 0.0]
    x = torch.linspace(-6, 6, 241, dtype=torch.float64) + 0.0013
    h = 1e-5
    for n in ref.ACTS:
        v, d, ev, ed = ref.act(n, x)
        slope = (ref.act(n, x + h)[0] - ref.act(n, x - h)[0]) / (2 * h)
        assert float((slope - d).abs().max()) < 1e-8
        assert float(d.abs().max()) < 1.2
        second = (ref.act(n, x + h)[1] - ref.act(n, x - h)[1]) / (2 * h)
        assert n == "relu" or float(second.abs().max()) < 1.0


@pytest.mark.parametrize("name", ref.ACTS)
def test_reference_gradient_is_the_forward_s(name):
    g = torch.Generator().manual_seed(3)
    X, W, dH = (torch.randn(*s, generator=g).double().requires_grad_()
                for s in ((9, 4), (10, 4), (9, 5)))
    Z = X @ W.t()
    a = {"silu": torch.nn.functional.silu, "relu": torch.relu,
         "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[name](Z[:, :5])
    H = a * Z[:, 5:]
    (H * dH.detach()).sum().backward()
    x, w, d = X.detach(), W.detach(), dH.detach()
    # in 64 bits the reference rounds nothing of its own
    assert torch.allclose(ref.glu(x, w, name, torch.float32)["H"][0], H.detach(), rtol=1e-12,
                          atol=1e-12)
    for z in (None, Z.detach()):
        got = ref.glu_grad(d, x, w, z, name, None, None, 0, 0, torch.float32)
        assert torch.allclose(got["dX"][0], X.grad, rtol=1e-12, atol=1e-12)
        assert torch.allclose(got["dW"][0], W.grad, rtol=1e-12, atol=1e-12)


def test_reference_gemm_i8_by_hand():
    X = torch.tensor([[1, -2], [127, 127]], dtype=torch.int8)
    W = torch.tensor([[3, 4], [-127, 127]], dtype=torch.int8)
    Y = torch.ones(2, 2)
    out, _ = ref.gemm_i8(X, W, Y, torch.tensor([0.5, 2.0]), torch.tensor([1.0, 0.25]), 2.0, 3.0,
                         torch.float32)
    # sums [-5, -381; 889, 0], times scales, times 2, plus 3
    assert out.tolist() == [[-2.0, -92.25], [3559.0, 3.0]]
