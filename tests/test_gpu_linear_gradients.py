"""GPU tests of klein_op_linear_backward where its fp32 gradients carry remainders: values that are not finite, and the
activations' derivatives in their tails."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_linear import kb, pitched, randn  # noqa: E402,F401


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(64, 128, 72), (700, 2056, 520), (2100, 2312, 2056), (5000, 264, 136), (80, 5000, 100)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_infinite_operands_stay_infinite(kb, m, n, k, act):
    """One infinity in w, then in x: fp32 gradients are infinite where their sums are, of the sign of dz, and have their
    old bits elsewhere (with an fp32 dout they are sums of two products, one of dz in bf16 and one of what that left).
    Two infinities against the same sign of dz are one, against both signs a NaN."""
    x, w = pitched(randn(0, m, k).bfloat16()), pitched(randn(1, n, k).bfloat16())
    z = randn(2, m, n).abs().bfloat16() + 1  # act' > 0
    dout = randn(3, m, n)
    dout[dout == 0] = 1
    dout[:, 3] = dout[:, 3].bfloat16().float()  # some remainders are 0 with act none
    dout[5] = dout[5].bfloat16().float()
    ws = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")

    def grads():
        dx, dw = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
        kb.klein_op_linear_backward(dout, x, w, ws, dx=dx, dw=dw, preact=z, act=act)
        assert kb.klein_sync()[0] == 0
        return dx, dw

    dx0, dw0 = grads()
    assert torch.isfinite(dx0).all() and torch.isfinite(dw0).all()
    for rows in ((3,), (n - 1,), (3, n // 2)):  # w's rows; n - 1 lies in the last part of a cut contraction
        kept = w[list(rows), 7].clone()
        w[list(rows), 7] = math.inf
        dx, dw = grads()
        want = dx0.clone()
        want[:, 7] = sum(dout[:, j] * math.inf for j in rows)
        assert torch.equal(dx.nan_to_num(1e38), want.nan_to_num(1e38)) and torch.equal(dx.isnan(), want.isnan()), rows
        assert torch.equal(dw, dw0)
        w[list(rows), 7] = kept
    for rows in ((5,), (m - 1,), (5, m // 2)):
        kept = x[list(rows), 9].clone()
        x[list(rows), 9] = -math.inf
        dx, dw = grads()
        want = dw0.clone()
        want[:, 9] = sum(dout[i] * -math.inf for i in rows)
        assert torch.equal(dw.nan_to_num(1e38), want.nan_to_num(1e38)) and torch.equal(dw.isnan(), want.isnan()), rows
        assert torch.equal(dx, dx0)
        x[list(rows), 9] = kept


@pytest.mark.gpu
def test_nan_operands_stay_nan(kb):
    m, n, k = 700, 2056, 520
    x, w, dout = randn(0, m, k).bfloat16(), randn(1, n, k).bfloat16(), randn(3, m, n)
    w[n - 2, 4] = math.nan
    x[m - 2, 6] = math.nan
    ws = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    dx, dw = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
    kb.klein_op_linear_backward(dout, x, w, ws, dx=dx, dw=dw)
    assert kb.klein_sync()[0] == 0
    for got, col in ((dx, 4), (dw, 6)):
        assert torch.isnan(got[:, col]).all()
        got[:, col] = 0
        assert torch.isfinite(got).all()


def derivative(z, act):
    """(act'(z), the size of the terms it is the sum of, the exponent's argument) in float64."""
    if act == "silu":
        u, du = z, torch.ones_like(z)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        u, du = c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z ** 2)
    s, t = torch.sigmoid(u), z * du * torch.sigmoid(u) * torch.sigmoid(-u)
    return s + t, s.abs() + t.abs(), u.abs()


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_derivative_tails(kb, act):
    """act' to a relative error, as long as fp32 holds it: dz = dbias of a single row with dout = 1. The exponential's
    argument carries eight roundings of 2^-24 of its size (z^3 and its constants; the product with log2 e), each of which
    moves the exponential by that much relative, and sixteen more of the result cover the division and the sums."""
    end = 87.0 if act == "silu" else 9.9  # e^-87 is above fp32's least normal number
    z = torch.cat([torch.linspace(-end, end, 4000, device="cuda"),
                   torch.tensor([0.0, -40.0, -40.5, -60.0, 39.0, 41.0, 60.0], device="cuda").clamp(-end, end)]).bfloat16()
    big = torch.tensor([120.0, 300.0, 1e15, 3e38, math.inf], device="cuda").bfloat16()
    z = torch.cat([z, big, -big, torch.tensor([math.nan], device="cuda").bfloat16()])
    n = z.numel()
    x, w = torch.ones(1, 8, device="cuda", dtype=torch.bfloat16), torch.ones(n, 8, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(kb.klein_linear_backward_workspace_size(1, n, 8), dtype=torch.uint8, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        dout, db = torch.ones(1, n, device="cuda", dtype=dtype), torch.empty(n, device="cuda")
        kb.klein_op_linear_backward(dout, x, w, ws, dbias=db, preact=z[None], act=act)
        assert kb.klein_sync()[0] == 0
        inside = n - 11
        ref, size, arg = derivative(z[:inside].double(), act)
        tol = 2.0 ** -24 * (8 * arg + 16) * size
        err = (db[:inside].double() - ref).abs()
        assert (err <= tol).all(), (z[:inside][err > tol][:5], db[:inside][err > tol][:5])
        assert (db[inside:inside + 5] == 1).all()
        assert (db[inside + 5:inside + 10] == 0).all()
        assert torch.isnan(db[-1])
        # an infinite dout keeps the derivative's sign where that is not 0
        dout.fill_(math.inf)
        kb.klein_op_linear_backward(dout, x, w, ws, dbias=db, preact=z[None], act=act)
        assert kb.klein_sync()[0] == 0
        safe = ref.abs() > 1e-3 * size
        assert torch.equal(db[:inside][safe], (ref[safe] * math.inf).float())


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_operands_that_are_not_needed(kb, act):
    """dx takes w alone, dw takes x alone, dbias neither."""
    m, n, k = 700, 264, 520
    x, w, dout = randn(0, m, k).bfloat16(), randn(1, n, k).bfloat16(), randn(2, m, n).bfloat16()
    z = randn(3, m, n).bfloat16() if act != "none" else None
    ws = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    bf = dict(dtype=torch.bfloat16, device="cuda")

    def call(xx, ww, wsp, **want):
        kb.klein_op_linear_backward(dout, xx, ww, wsp, preact=z, act=act, **want)
        assert kb.klein_sync()[0] == 0
        return want

    both = call(x, w, ws, dx=torch.zeros(m, k, **bf), dw=torch.zeros(n, k, **bf), dbias=torch.zeros(n, device="cuda"))
    dx = call(None, w, ws, dx=torch.zeros(m, k, **bf))["dx"]
    dw = call(x, None, ws, dw=torch.zeros(n, k, **bf))["dw"]
    one = torch.empty(kb.klein_linear_backward_workspace_size(m, n, 1), dtype=torch.uint8, device="cuda")
    db = call(None, None, one, dbias=torch.zeros(n, device="cuda"))["dbias"]
    db2 = call(None, w, ws, dx=torch.zeros(m, k, **bf), dbias=torch.zeros(n, device="cuda"))["dbias"]
    assert torch.equal(dx, both["dx"]) and torch.equal(dw, both["dw"])
    assert torch.equal(db, both["dbias"]) and torch.equal(db2, both["dbias"])
    before = kb.klein_launch_count()
    for xx, ww, want in ((x, None, "dx"), (None, w, "dw"), (None, None, "dx"), (None, None, "dw")):
        with pytest.raises(kb.KleinError):
            call(xx, ww, ws, **{want: torch.zeros((m, k) if want == "dx" else (n, k), **bf)})
    for bad in (x[:-1], x.float(), x[:, ::2], x[0], x.cpu()):  # what is given is looked at, needed or not
        with pytest.raises(kb.KleinError):
            call(bad, w, ws, dx=torch.zeros(m, k, **bf))
    with pytest.raises(kb.KleinError):
        call(x, w[:, :-8], ws, dw=torch.zeros(n, k, **bf))
    assert kb.klein_launch_count() == before
