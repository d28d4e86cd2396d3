"""GPU tests of klein_op_linear and klein_op_linear_backward against the formulas in float64.

Tolerances. Both sides read the same bf16 operands, whose products are exact in fp32. The kernels
sum them in chunks of at most 512 by the tensor core, which truncates, then in fp32 rounded to
nearest: for normal operands the error of a sum of k products of size s is far below
1e-6 s sqrt(k) + 2^-24 |sum| times a small factor; SUM = 1e-5 of s sqrt(k) covers the worst of
the elements. On top of it come half a step of the output type (bf16 2^-8 relative, fp32 2^-24),
a few fp32 roundings of the epilogue (1e-5 relative with the fast exponential: its argument's
rounding grows with |z|, at most 2^-24 * 90 = 5e-6), and in the backward pass half a bf16 step of every
dz for a bf16 gradient (2^-8 |dz|, which the sums add up as at most 2^-8 times the product of the magnitudes),
2^-16 for an fp32 one, which takes the rounding's remainder along (itself rounded: 2^-8 of 2^-8).
"""
import math

import pytest

torch = pytest.importorskip("torch")

SUM = 1e-5
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def kb():
    from conftest import ensure_built
    ensure_built()
    import latent_flow_matching_joint_b200 as kb
    return kb


def pitched(t, extra=0):
    """A bf16 matrix in rows of a pitch that is a multiple of 8, NaN between its columns and the pitch."""
    m, k = t.shape
    whole = torch.full((m, (k + 7) // 8 * 8 + 8 * extra), float("nan"), dtype=torch.bfloat16, device="cuda")
    whole[:, :k] = t
    return whole[:, :k]


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def act_grad64(z, act):
    z = z.detach().clone().requires_grad_(True)
    return torch.autograd.grad(act64(z, act).sum(), z)[0]


def check_forward(kb, m, n, k, act="none", bias=False, residual=None, out=torch.bfloat16, save=False, alpha=1.0,
                  pad=0, in_place=False, seed=0):
    x = pitched(randn(seed, m, k).bfloat16(), pad)
    w = pitched((randn(seed + 1, n, k) / math.sqrt(k)).bfloat16(), pad)
    b = randn(seed + 2, n) if bias else None
    r = None if residual is None else randn(seed + 3, m, n + pad).to(residual)[:, :n]
    whole = torch.full((m, n + pad), 7.0, dtype=out, device="cuda")
    y = whole[:, :n]
    if in_place:
        y.copy_(r)
    z = torch.full((m, n + pad), 5.0, dtype=torch.bfloat16, device="cuda") if save else None
    ws = torch.empty(kb.klein_linear_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    kb.klein_op_linear(x, w, y, ws, bias=b, residual=y if in_place else r, act=act, alpha=alpha,
                       preact=None if z is None else z[:, :n])
    assert kb.klein_sync()[0] == 0
    zr = x.double() @ w.double().T
    size = 1.0  # rms of one product times sqrt(k): unit rows of x against rows of w of norm about 1
    if bias:
        zr = zr + b.double()
    ref = alpha * act64(zr, act)
    if r is not None:
        ref = ref + r.double()
    slope = 1.13  # |act'| <= 1.13 for gelu, 1.1 for silu
    tol = abs(alpha) * (slope * SUM * size + 1e-5 * zr.abs()) + HALF[out] * ref.abs() + 1e-7
    assert ((y.double() - ref).abs() <= tol).all(), ((y.double() - ref).abs() - tol).max()
    assert (whole[:, n:] == 7.0).all()
    if save:
        assert ((z[:, :n].double() - zr).abs() <= SUM * size + 1e-5 * zr.abs() + HALF[torch.bfloat16] * zr.abs()).all()
        assert (z[:, n:] == 5.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 256, 256), (1, 17, 2500), (2, 1000, 77), (3, 9, 4096), (4, 2049, 320),
                                   (5, 128, 64), (5, 1, 9), (16, 16, 16), (80, 24, 1000), (127, 129, 65), (128, 128, 4096),
                                   (129, 255, 513), (300, 100, 5000), (512, 1280, 2560), (1961, 37, 130),
                                   (1961, 2049, 200), (2560, 5120, 1088), (4608, 16, 2560), (4608, 9216, 16),
                                   (16, 16, 12289), (17, 3000, 5000), (33, 40, 12300), (97, 2000, 515), (640, 544, 64),
                                   (700, 300, 5000), (1000, 515, 1027), (300, 1104, 2048), (5000, 24, 4104),
                                   (257, 257, 5003)])
def test_linear_shapes(kb, m, n, k):
    check_forward(kb, m, n, k)
    check_forward(kb, m, n, k, act="gelu", bias=True, residual=torch.float32, out=torch.float32, save=True, alpha=0.5,
                  pad=3, seed=10)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("residual", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(3, 200), (200, 200), (1500, 2056)])  # the last on the large product's kernel
def test_linear_epilogues(kb, act, residual, out, m, k):
    check_forward(kb, m, 136, k, act=act, bias=True, residual=residual, out=out, save=True, alpha=2.0)
    check_forward(kb, m, 131, k, act=act, residual=residual, out=out, alpha=-1.0, pad=1)
    if residual is out:
        check_forward(kb, m, 136, k, act=act, residual=residual, out=out, in_place=True)


@pytest.mark.gpu
@pytest.mark.parametrize("k", [8, 16, 64, 65, 192, 193, 256])
@pytest.mark.parametrize("m,n", [(5000, 5000), (700, 9000), (20000, 264), (9000, 1032)])
def test_linear_short_k_with_residual(kb, m, n, k):
    """An adapter's second half over many tiles, onto the frozen layer's output."""
    for in_place in (False, True):
        check_forward(kb, m, n, k, residual=torch.bfloat16, alpha=2.0, in_place=in_place)
    check_forward(kb, m, n, k, act="silu", bias=True, residual=torch.bfloat16, save=True)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(2, 100, 3000), (64, 100, 12288), (300, 700, 9216), (2000, 3000, 4096)])
def test_linear_long_sums_keep_fp32(kb, m, n, k):
    """fp32 output of long sums: the norm of the error is that of fp32 sums, not of a truncating accumulator
    (1.1e-9 k = 1e-5 at k = 9216)."""
    x, w = randn(1, m, k).bfloat16(), randn(2, n, k).bfloat16()
    y = torch.empty(m, n, device="cuda")
    ws = torch.empty(kb.klein_linear_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    kb.klein_op_linear(x, w, y, ws)
    ref = x.double() @ w.double().T
    assert ((y.double() - ref).norm() / ref.norm()).item() <= 2e-6


@pytest.mark.gpu
def test_linear_activation_tails(kb):
    """Pre-activations from -1e30 to 1e30, infinities and NaN."""
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 12.0, -12.0, 88.0, -88.0, 100.0, -100.0, 1e15, -1e15, 1e30, -1e30,
                      float("inf"), float("nan")], device="cuda").bfloat16()
    for m in (1, 8):  # both kernels
        x = torch.zeros(m, 8, device="cuda", dtype=torch.bfloat16)
        x[:, 0] = 1
        w = torch.zeros(16, 8, device="cuda", dtype=torch.bfloat16)
        w[:, 0] = z
        for act in ("silu", "gelu"):
            y = torch.empty(m, 16, device="cuda")
            pre = torch.empty(m, 16, device="cuda", dtype=torch.bfloat16)
            kb.klein_op_linear(x, w, y, act=act, preact=pre)
            ref = act64(z.double(), act)
            assert torch.isnan(y[:, 15]).all() and torch.isnan(pre[:, 15]).all()
            assert (y[:, 14] == math.inf).all()
            assert ((y[:, :14].double() - ref[:14]).abs() <= 1e-5 * ref[:14].abs() + 1e-12).all()
            dx, dw = torch.empty(m, 8, device="cuda"), torch.empty(16, 8, device="cuda")
            dbias = torch.empty(16, device="cuda")
            ws = torch.empty(kb.klein_linear_backward_workspace_size(m, 16, 8), dtype=torch.uint8, device="cuda")
            dout = torch.ones(m, 16, device="cuda", dtype=torch.bfloat16)
            kb.klein_op_linear_backward(dout, x, w, ws, dw=dw, dbias=dbias, preact=pre, act=act)
            slope = m * act_grad64(z[:14].double().clamp(-60, 60), act)
            assert ((dbias[:14].double() - slope).abs() <= 1e-5 * m).all()
            assert ((dw[:14, 0].double() - slope).abs() <= m * (2.0 ** -16 * 1.13 + 1e-5)).all()


def check_backward(kb, m, n, k, act="none", dout_type=torch.bfloat16, dx_type=torch.bfloat16, dw_type=torch.bfloat16,
                   alpha=1.0, pad=0, want=("dx", "dw", "dbias"), seed=0):
    x = pitched(randn(seed, m, k).bfloat16(), pad)
    w = pitched(randn(seed + 1, n, k).bfloat16())
    dout = randn(seed + 2, m, n + pad).to(dout_type)[:, :n]
    z = randn(seed + 3, m, n + pad).mul(2).bfloat16()[:, :n] if act != "none" else None
    out = {"dx": torch.full((m, k + pad), 7.0, dtype=dx_type, device="cuda"),
           "dw": torch.full((n, k + pad), 7.0, dtype=dw_type, device="cuda"),
           "dbias": torch.full((n,), 7.0, device="cuda")}
    ws = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    given = {name: (t if name == "dbias" else t[:, :k]) if name in want else None for name, t in out.items()}
    kb.klein_op_linear_backward(dout, x, w, ws, preact=z, act=act, alpha=alpha, **given)
    assert kb.klein_sync()[0] == 0
    dz = alpha * dout.double()
    if z is not None:
        dz = dz * act_grad64(z.double(), act)
    exact_dz = act == "none" and dout_type == torch.bfloat16 and math.log2(abs(alpha)).is_integer()
    for name, a, b, length in (("dx", dz, w.double(), n), ("dw", dz.T, x.double(), m)):
        if name not in want:
            assert (out[name] == 7.0).all()
            continue
        ref, mag = a @ b, a.abs() @ b.abs()
        fp32 = out[name].dtype == torch.float32
        half = 0.0 if exact_dz else 1e-5 + (2.0 ** -16 if fp32 else 2.0 ** -8)
        tol = half * mag + SUM * dz.abs().max() * 4 * math.sqrt(length) + HALF[out[name].dtype] * ref.abs() * 1.01
        err = (out[name][:, :k].double() - ref).abs()
        assert (err <= tol).all(), (name, (err - tol).max())
        # the roundings of dz are independent: in norm they add up like sqrt, not like the bound above
        assert (err.norm() / ref.norm()).item() <= (8e-6 if fp32 else 5e-3)
        assert (out[name][:, k:] == 7.0).all()
    if "dbias" in want:
        ref, mag = dz.sum(0), dz.abs().sum(0)
        assert ((out["dbias"].double() - ref).abs() <= 1e-5 * mag).all()
    else:
        assert (out["dbias"] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 100, 64), (2, 17, 9), (16, 16, 16), (80, 24, 1000), (127, 129, 65),
                                   (128, 4096, 128), (129, 255, 513), (300, 5000, 100), (512, 1280, 2560),
                                   (1961, 37, 130), (1961, 2049, 200), (4608, 16, 2560), (4608, 2560, 16),
                                   (2560, 1088, 5120)])
def test_linear_backward_shapes(kb, m, n, k):
    check_backward(kb, m, n, k)
    check_backward(kb, m, n, k, act="gelu", dout_type=torch.float32, dx_type=torch.float32, dw_type=torch.float32,
                   alpha=0.5, pad=3, seed=10)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dout_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("want", [("dx",), ("dw",), ("dbias",), ("dx", "dw"), ("dw", "dbias")])
def test_linear_backward_parts(kb, act, dout_type, want):
    check_backward(kb, 150, 72, 136, act=act, dout_type=dout_type, dw_type=torch.float32, alpha=3.0, want=want)


@pytest.mark.gpu
def test_linear_gradients_match_differences(kb):
    """Directional derivative of L = sum(dout * y) along random directions of x, w and bias, y from the kernel
    itself in fp32, against the kernel's gradients."""
    m, n, k = 40, 24, 64
    x, w = randn(1, m, k).bfloat16(), (randn(2, n, k) / 8).bfloat16()
    b, dout = randn(3, n), randn(4, m, n).bfloat16()
    pre = torch.empty(m, n, device="cuda", dtype=torch.bfloat16)
    y = torch.empty(m, n, device="cuda")

    def loss(xx, ww, bb):
        kb.klein_op_linear(xx, ww, y, bias=bb, act="silu", alpha=2.0, preact=pre)
        return (dout.double() * y.double()).sum().item()

    loss(x, w, b)
    dx, dw, db = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    ws = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    kb.klein_op_linear_backward(dout, x, w, ws, dx=dx, dw=dw, dbias=db, preact=pre, act="silu", alpha=2.0)
    for which, value, grad in (("x", x, dx), ("w", w, dw), ("b", b, db)):
        step = randn(9, *value.shape) * 0.05 * value.float().abs().mean()
        hi, lo = (value.float() + step).to(value.dtype), (value.float() - step).to(value.dtype)
        args = {"x": x, "w": w, "b": b}
        up = loss(*{**args, which: hi}.values())
        down = loss(*{**args, which: lo}.values())
        expected = (grad.double() * (hi.double() - lo.double())).sum().item()
        # second-order terms cancel; third-order ones and dz's bf16 rounding remain
        assert abs(up - down - expected) <= 1e-2 * (grad.double() * (hi.double() - lo.double())).norm().item() + 2e-3


@pytest.mark.gpu
def test_linear_same_bits_every_time(kb):
    m, n, k = 200, 300, 9000  # split over k
    x, w, dout = randn(1, m, k).bfloat16(), randn(2, n, k).bfloat16(), randn(3, m, n).bfloat16()
    assert kb.klein_linear_workspace_size(m, n, k) > 0
    first = None
    for fill in (0, 255):
        ws = torch.full((kb.klein_linear_workspace_size(m, n, k),), fill, dtype=torch.uint8, device="cuda")
        wb = torch.full((kb.klein_linear_backward_workspace_size(m, n, k),), fill, dtype=torch.uint8, device="cuda")
        y, dx, dw = torch.empty(m, n, device="cuda"), torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
        db = torch.empty(n, device="cuda")
        kb.klein_op_linear(x, w, y, ws)
        kb.klein_op_linear_backward(dout, x, w, wb, dx=dx, dw=dw, dbias=db)
        if first is None:
            first = (y, dx, dw, db)
        else:
            assert all(torch.equal(a, b) for a, b in zip(first, (y, dx, dw, db)))


@pytest.mark.gpu
def test_linear_on_a_stream_and_in_a_graph(kb):
    m, n, k = 200, 300, 12288
    x, w, r = randn(1, m, k).bfloat16(), randn(2, n, k).bfloat16(), randn(3, m, n)
    ws = torch.empty(kb.klein_linear_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    want = torch.empty(m, n, device="cuda")
    kb.klein_op_linear(x, w, want, ws, residual=r)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = torch.zeros(m, n, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        kb.klein_op_linear(x, w, got, ws, residual=r)
    s.synchronize()
    assert torch.equal(got, want)
    got.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kb.klein_op_linear(x, w, got, ws, residual=r)
    for _ in range(2):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    x.mul_(2)  # the graph reads the operands anew
    graph.replay()
    kb.klein_op_linear(x, w, want, ws, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.gpu
def test_offsets_that_pass_32_bits(kb):
    """Rows of a pitch of 2^23 elements: the last ones stand 2^31 elements and more behind the first."""
    m, n, k, pitch = 300, 264, 200, 1 << 23

    def far(t):
        flat = torch.empty((m - 1) * pitch + t.shape[1], dtype=t.dtype, device="cuda")
        view = flat.as_strided(t.shape, (pitch, 1))
        view.copy_(t)
        return view

    w = (randn(1, n, k) / math.sqrt(k)).bfloat16()
    ws = torch.empty(kb.klein_linear_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    wsb = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    # One far tensor at a time: x, the residual and output in place, the saved sums, then dout and dx.
    x, r = randn(0, m, k).bfloat16(), randn(2, m, n).bfloat16()
    for which in ("x", "out", "z"):
        y = far(r) if which == "out" else r.clone()
        z = torch.zeros(m, n, dtype=torch.bfloat16, device="cuda")
        z = far(z) if which == "z" else z
        kb.klein_op_linear(far(x) if which == "x" else x, w, y, ws, residual=y, act="silu", preact=z)
        assert kb.klein_sync()[0] == 0
        zr = x.double() @ w.double().T
        ref = act64(zr, "silu") + r.double()
        tol = 1.13 * SUM + 1e-5 * zr.abs() + HALF[torch.bfloat16] * ref.abs() + 1e-7
        assert ((y.double() - ref).abs() <= tol).all(), which
        assert ((z.double() - zr).abs() <= SUM + (1e-5 + HALF[torch.bfloat16]) * zr.abs()).all(), which
        del y, z
    dout = randn(3, m, n).bfloat16()
    for which in ("dout", "dx"):
        dx = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
        dx = far(dx) if which == "dx" else dx
        dw = torch.zeros(n, k, dtype=torch.float32, device="cuda")
        kb.klein_op_linear_backward(far(dout) if which == "dout" else dout, x, w, wsb, dx=dx, dw=dw)
        assert kb.klein_sync()[0] == 0
        dxr, dwr = dout.double() @ w.double(), dout.double().T @ x.double()
        dxs, dws = dout.double().abs() @ w.double().abs(), dout.double().abs().T @ x.double().abs()
        assert ((dx.double() - dxr).abs() <= HALF[torch.bfloat16] * dxr.abs() + SUM * dxs).all(), which
        assert ((dw.double() - dwr).abs() <= HALF[torch.float32] * dwr.abs() + SUM * dws).all(), which
        del dx


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(64, 128, 72), (700, 2056, 520)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_infinite_gradients_stay_infinite(kb, m, n, k, act):
    """One infinity in dout: fp32 gradients have it, with its sign, where the sums do, and nothing else changes."""
    x, w = randn(0, m, k).bfloat16(), randn(1, n, k).bfloat16()
    x[x == 0], w[w == 0] = 1, 1
    z = randn(2, m, n).abs().bfloat16() + 1  # act' > 0
    dout = randn(3, m, n)
    ws = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")

    def grads():
        dx, dw, db = (torch.zeros(s, device="cuda") for s in ((m, k), (n, k), (n,)))
        kb.klein_op_linear_backward(dout, x, w, ws, dx=dx, dw=dw, dbias=db, preact=z, act=act)
        assert kb.klein_sync()[0] == 0
        return dx, dw, db

    before = grads()
    i, j = m - 3, n // 2 + 1
    dout[i, j] = -math.inf
    dx, dw, db = grads()
    assert torch.equal(dx[i], -math.inf * w[j].float())
    assert torch.equal(dw[j], -math.inf * x[i].float())
    assert db[j] == -math.inf
    for got, old, row in ((dx, before[0], i), (dw, before[1], j), (db, before[2], j)):
        got[row] = old[row]
        assert torch.equal(got, old)
