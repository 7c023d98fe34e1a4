"""Argument checks, refusals and workspace sizes of the products whose rows
choose their own weights, without a GPU, and their references against
hand-worked values."""
import pytest
import torch

import rows_reference as ref

P = 0x10000           # a non-null, aligned address; never dereferenced here

LORA = dict(M=4, N=6, K=8, alpha=1.0, X=P, ldx=8, W=P, ldw=8, beta=0.0, Y=P, ldy=6, L=3, R=2, A=P,
            lda=8, stride_a=16, B=P, ldb=2, stride_b=12, scale=None, ranks=None, rows=P,
            workspace=P, workspace_bytes=0, stream=None)

LORA_BAD = [
    (-301, dict(M=-1)), (-302, dict(N=-1)), (-303, dict(K=-1)), (-306, dict(ldx=7)),
    (-308, dict(ldw=7)), (-311, dict(ldy=5)), (-312, dict(L=-1)), (-312, dict(L=65536)),
    (-313, dict(R=-1)), (-313, dict(R=257, ldb=257)), (-315, dict(lda=7)),
    (-316, dict(stride_a=-1)), (-318, dict(ldb=1)), (-319, dict(stride_b=-1)),
    (-305, dict(X=None)), (-307, dict(W=None)), (-310, dict(Y=None)), (-314, dict(A=None)),
    (-317, dict(B=None)), (-322, dict(rows=None)), (-323, dict(workspace=P + 16)),
    (-324, dict(workspace_bytes=0)), (-301, dict(M=-1, N=-1, X=None)),
    (-310, dict(K=0, ldx=1, ldw=1, beta=0.5, Y=None)),
    # nothing to do: no memory is looked at
    (0, dict(M=0, X=None, W=None, Y=None, A=None, B=None, rows=None)),
    (0, dict(N=0, ldy=1, X=None, W=None, Y=None, A=None, B=None, rows=None)),
    (0, dict(alpha=0.0, beta=1.0, X=None, W=None, Y=None, A=None, B=None, rows=None)),
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", LORA_BAD, ids=lambda c: "%d-%s" % (c[0], "-".join(c[1])))
def test_lora_argument_checks(dt, case):
    import dense_gemm_fp32_amd as dg
    want, change = case
    assert getattr(dg, "gemm_lora_" + dt)(*dict(LORA, **change).values()) == want
    if want:
        assert dg.gemm_status_string(want).startswith("gemm_lora: invalid argument %d:"
                                                      % (-300 - want))


GRAD = dict(M=4, N=6, K=8, alpha=1.0, dY=P, lddy=6, X=P, ldx=8, W=P, ldw=8, L=3, R=2, A=P, lda=8,
            stride_a=16, B=P, ldb=2, stride_b=12, scale=None, ranks=None, rows=P, beta_x=0.0, dX=P,
            lddx=8, beta_ab=0.0, dA=P, ldda=8, stride_da=16, dB=P, lddb=2, stride_db=12,
            workspace=P, workspace_bytes=0, stream=None)

GRAD_BAD = [
    (-401, dict(M=-1)), (-402, dict(N=-1)), (-403, dict(K=-1)), (-406, dict(lddy=5)),
    (-408, dict(ldx=7)), (-410, dict(ldw=7)), (-411, dict(L=65536)), (-412, dict(R=300, ldb=300)),
    (-414, dict(lda=7)), (-415, dict(stride_a=-1)), (-417, dict(ldb=1)), (-418, dict(stride_b=-1)),
    (-424, dict(lddx=7)), (-427, dict(ldda=7)), (-428, dict(stride_da=15)), (-430, dict(lddb=1)),
    (-431, dict(stride_db=11)), (-405, dict(dY=None)), (-407, dict(X=None)), (-409, dict(W=None)),
    (-413, dict(A=None)), (-416, dict(B=None)), (-421, dict(rows=None)),
    (-432, dict(workspace=P + 128)), (-433, dict()),
    (0, dict(dX=None, dA=None, dB=None, dY=None, X=None, W=None)),
    # not wanted, so not looked at
    (-433, dict(dX=None, W=None, ldw=0, lddx=0)), (-433, dict(dA=None, dB=None, X=None)),
    (0, dict(M=0, beta_ab=1.0)), (0, dict(alpha=0.0, beta_x=1.0, beta_ab=1.0, dY=None)),
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", GRAD_BAD, ids=lambda c: "%d-%s" % (c[0], "-".join(c[1])))
def test_lora_grad_argument_checks(dt, case):
    import dense_gemm_fp32_amd as dg
    want, change = case
    assert getattr(dg, "gemm_lora_grad_" + dt)(*dict(GRAD, **change).values()) == want
    if want:
        assert dg.gemm_status_string(want).startswith("gemm_lora_grad: invalid argument %d:"
                                                      % (-400 - want))


MOE = dict(M=4, D=8, F=6, E=5, top_k=2, renorm=1, alpha=1.0, X=P, ldx=8, Wr=P, ldr=8, W1=P, ld1=8,
           stride1=96, W2=P, ld2=6, stride2=48, beta=0.0, Y=P, ldy=8, ids=None, weights=None,
           workspace=P, workspace_bytes=0, stream=None)

MOE_BAD = [
    (-501, dict(M=-1)), (-501, dict(M=257)), (-502, dict(D=0)), (-503, dict(F=0)),
    (-504, dict(E=0)), (-504, dict(E=1025)), (-505, dict(top_k=0)), (-505, dict(top_k=6)),
    (-505, dict(E=100, top_k=65)), (-506, dict(renorm=2)), (-509, dict(ldx=7)),
    (-511, dict(ldr=7)), (-513, dict(ld1=7)), (-514, dict(stride1=-1)), (-516, dict(ld2=5)),
    (-517, dict(stride2=-1)), (-520, dict(ldy=7)), (-508, dict(X=None)), (-510, dict(Wr=None)),
    (-512, dict(W1=None)), (-515, dict(W2=None)), (-519, dict(Y=None)),
    (-523, dict(workspace=P + 1)), (-524, dict()),
    (0, dict(M=0, X=None, Y=None)), (0, dict(alpha=0.0, beta=1.0, X=None, Y=None)),
]


@pytest.mark.parametrize("dt", ["f16", "f32"])
@pytest.mark.parametrize("case", MOE_BAD, ids=lambda c: "%d-%s" % (c[0], "-".join(c[1])))
def test_moe_argument_checks(dt, case):
    import dense_gemm_fp32_amd as dg
    want, change = case
    assert getattr(dg, "gemm_moe_" + dt)(*dict(MOE, **change).values()) == want
    if want:
        assert dg.gemm_status_string(want).startswith("gemm_moe: invalid argument %d:"
                                                      % (-500 - want))


def test_workspace_sizes():
    import dense_gemm_fp32_amd as dg
    for fn, good in ((dg.gemm_lora_workspace, (33, 40, 50, 3, 8)),
                     (dg.gemm_lora_grad_workspace, (33, 40, 50, 3, 8)),
                     (dg.gemm_moe_workspace, (33, 40, 50, 8, 2))):
        for dtype in (0, 1):
            n = fn(dtype, *good)
            assert n > 0 and n % 256 == 0
            for i in range(5):
                assert fn(dtype, *(good[:i] + (0,) + good[i + 1:])) == 0
        assert fn(2, *good) == 0
    # sizes beyond 32 bits
    most = 1 << 24
    assert dg.gemm_lora_grad_workspace(0, most, 64, 64, 1, 256) > 1 << 33
    for i in range(3):
        for fn in (dg.gemm_lora_workspace, dg.gemm_lora_grad_workspace):
            sizes = [16, 16, 16, 2, 8]
            sizes[i] = most + 1
            assert fn(1, *sizes) == 0
    assert dg.gemm_moe_workspace(1, 2, most + 1, 16, 4, 2) == 0
    assert dg.gemm_moe_workspace(1, 2, 16, most + 1, 4, 2) == 0


def test_gradients_workspace_goes_with_the_rows():
    """Adapters without rows in the batch take nothing but their place in the list of
    first rows: 4 bytes each."""
    import dense_gemm_fp32_amd as dg
    for dtype in (0, 1):
        for M, N, K, R in ((256, 4096, 4096, 16), (5000, 700, 333, 64), (1, 64, 64, 8)):
            few, many = (dg.gemm_lora_grad_workspace(dtype, M, N, K, L, R) for L in (64, 60000))
            assert 0 < many - few <= 4 * (60000 - 64) + 256
    # 256 rows: two sets of partial sums a chunk of 64 rows, beside the products' own
    assert dg.gemm_lora_grad_workspace(1, 256, 4096, 4096, 1000, 16) < 64 << 20


def test_sizes_beyond_the_limit():
    """Refused as argument 1, 2 or 3, whatever the others are."""
    import dense_gemm_fp32_amd as dg
    big = (1 << 24) + 1
    for dt in ("f16", "f32"):
        for i, n in enumerate("MNK"):
            for base, args, name in ((-300, LORA, "gemm_lora_"), (-400, GRAD, "gemm_lora_grad_")):
                got = getattr(dg, name + dt)(*dict(args, **{n: big}).values())
                assert got == base - 1 - i
        for i, n in ((2, "D"), (3, "F")):
            assert getattr(dg, "gemm_moe_" + dt)(*dict(MOE, **{n: big}).values()) == -500 - i


def test_calls_run_on_the_tensors_gpu(monkeypatch):
    """Where another GPU than the tensors' is current, a call changes to theirs
    and back, since a default stream means the current one's."""
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

    def entry(*args):
        calls.append((now[0],) + args)
        return 0
    for dev in (0, 1):
        binding._call_rows(entry, dev, 5, None, 0, (7,))
        assert calls[-1] == (dev, 7, None, 0, 5) and now[0] == 0


def test_wrappers_refuse_cpu_tensors():
    import dense_gemm_fp32_amd as dg
    X, W, A, B = torch.zeros(2, 4), torch.zeros(3, 4), torch.zeros(1, 2, 4), torch.zeros(1, 3, 2)
    rows = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        dg.lora(X, W, A, B, rows, torch.zeros(2, 3))
    with pytest.raises(ValueError, match="GPU"):
        dg.lora_grad(torch.zeros(2, 3), X, W, A, B, rows, dX=torch.zeros(2, 4))
    with pytest.raises(ValueError, match="GPU"):
        dg.moe(X, torch.zeros(3, 4), torch.zeros(3, 4, 4), torch.zeros(3, 4, 2), 1,
               torch.zeros(2, 4))
    with pytest.raises(ValueError, match="dtype"):
        dg.lora(X.double(), W.double(), A.double(), B.double(), rows, torch.zeros(2, 3).double())


def test_wrappers_refuse_sizes_beyond_32_bits():
    """Sizes and distances of rows that an int does not hold are refused, not cut to
    its 32 bits (which a multiple of 2^32 more would pass)."""
    from dense_gemm_fp32_amd import binding
    f16, big = torch.float16, 1 << 32

    def far(shape, strides):
        return torch.empty_strided(shape, strides, dtype=f16, device="meta")
    dev = far((1, 1), (1, 1)).get_device()
    for t in (far((4, 8), (big + 8, 1)), far((big + 4, 8), (8, 1)), far((1, big + 8), (big + 8, 1))):
        with pytest.raises(ValueError, match="32 bits"):
            binding._rows("X", t, *t.shape, f16, dev)
    for t in (far((3, 4, 8), (64, big + 8, 1)), far((3, big + 4, 8), (64, 8, 1)),
              far((big + 3, 4, 8), (32, 8, 1)), far((3, 1, big + 8), (64, 8, 1))):
        with pytest.raises(ValueError, match="32 bits"):
            binding._stack("A", t, *t.shape, f16, dev)
    t = far((4, 8), ((1 << 31) - 1, 1))
    assert binding._rows("X", t, 4, 8, f16, dev) == (1 << 31) - 1
    t = far((3, 4, 8), (big, 8, 1))
    assert binding._stack("A", t, 3, 4, 8, f16, dev) == (8, big)


def test_reference_lora_by_hand():
    X = torch.tensor([[1.0, 2.0], [3.0, -1.0], [1.0, 1.0]])
    W = torch.tensor([[1.0, 0.0], [0.0, 1.0]])
    A = torch.tensor([[[1.0, 1.0]], [[2.0, 0.0]]])
    B = torch.tensor([[[1.0], [10.0]], [[-1.0], [0.5]]])
    rows = torch.tensor([0, 1, -1], dtype=torch.int32)
    Y = torch.ones(3, 2)
    out, _ = ref.lora(X, W, A, B, rows, Y, torch.tensor([2.0, 1.0]), None, 1.0, 3.0)
    # row 0: x + 2*3*[1, 10] + 3; row 1: x + 6*[-1, 0.5] + 3; row 2: x + 3
    assert out.tolist() == [[10.0, 65.0], [0.0, 5.0], [4.0, 4.0]]
    out, _ = ref.lora(X, W, A, B, rows, Y, None, torch.tensor([0, 9]), 1.0, 0)
    assert out.tolist() == [[1.0, 2.0], [-3.0, 2.0], [1.0, 1.0]]


def test_reference_gradient_is_the_forward_s():
    g = torch.Generator().manual_seed(3)
    X, W, A, B, dY = (torch.randn(*s, generator=g).double().requires_grad_()
                      for s in ((9, 4), (5, 4), (3, 2, 4), (3, 5, 2), (9, 5)))
    rows = torch.tensor([0, 2, 2, -1, 1, 0, 5, 1, 2], dtype=torch.int32)
    scale = torch.tensor([0.5, 2.0, -1.0])
    out = X @ W.t()
    mask = (rows[:, None] == torch.arange(3)[None, :]).double()
    out = out + torch.einsum("ik,ark,anr,ia->in", X, A, B, mask * scale.double())
    (out * dY.detach()).sum().backward()
    d = [t.detach() for t in (dY, X, W, A, B)]
    want = ref.lora_grad(*d, rows, None, None, None, scale, None, 1.0, 0, 0)
    for n, t in (("dX", X), ("dA", A), ("dB", B)):
        assert torch.allclose(want[n][0], t.grad, rtol=1e-12, atol=1e-12)
    assert torch.allclose(ref.lora(*d[1:], rows, None, scale, None, 1.0, 0)[0], out.detach(),
                          rtol=1e-12, atol=1e-12)


def test_reference_moe_by_hand():
    X = torch.tensor([[1.0, 2.0]])
    router = torch.tensor([[1.0, 0.0], [0.0, 1.0], [0.0, 1.0]])
    W1 = torch.zeros(3, 2, 2)
    W1[:, 0, 0], W1[:, 1, 1] = 1.0, torch.tensor([1.0, 2.0, 3.0])   # g = 1, u = 2, 4, 6
    W2 = torch.ones(3, 2, 1)
    out, _, ids, w, _ = ref.moe(X, router, W1, W2, 2, None, True, 1.0, 0)
    assert ids.tolist() == [[1, 2]] and w.tolist() == [[0.5, 0.5]]
    silu = 1.0 / (1.0 + 2.718281828459045 ** -1)
    assert abs(float(out[0, 0]) - silu * 5.0) < 1e-12
    _, _, _, w, _ = ref.moe(X, router, W1, W2, 2, None, False, 1.0, 0)
    e = 2.718281828459045
    assert abs(float(w[0, 0]) - e / (2 * e + 1)) < 1e-12
