"""GPU tests of the large product's kernel in klein_op_linear: its own epilogue on whole tiles (rows by TMA, a column to
a lane where TMA cannot take them) and the second launch that finishes cut tiles, at sizes that the few-row kernel does
not take. The workspace size says which: 0 where every tile stays whole.

Tolerances as in test_gpu_linear: sums SUM, half a step of the output, 1e-5 of z for the epilogue's fp32."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_linear import HALF, SUM, act64, act_grad64, kb, randn  # noqa: E402,F401

BF, F32 = torch.bfloat16, torch.float32


def few_rows(m, n, k):
    """The sizes that klein_op_linear gives to the few-row kernel."""
    blocks = (m + 31) // 32
    return m <= 16 or (blocks * ((n + 15) // 16) <= 640 and blocks * n * k <= 12 << 20)


def workspace(kb, m, n, k, cut):
    assert not few_rows(m, n, k)
    size = kb.klein_linear_workspace_size(m, n, k)
    assert (size > 0) == cut
    return torch.empty(size, dtype=torch.uint8, device="cuda")


def matrix(m, n, dtype, extra=0, offset=0, fill=7.0):
    """([m, n] view, the whole buffer): pitch n + extra, its first element `offset` into an aligned buffer."""
    flat = torch.full((offset + m * (n + extra),), fill, dtype=dtype, device="cuda")
    return flat.as_strided((m, n), (n + extra, 1), offset), flat


def untouched(view, flat, fill=7.0):
    """Nothing outside the view was written."""
    view.fill_(fill)
    return bool((flat == fill).all())


class Product:
    """x, w, bias, two residuals and the sums in float64, made once for many epilogues."""

    def __init__(self, m, n, k, seed=0):
        self.m, self.n, self.k = m, n, k
        pitch = (k + 7) // 8 * 8
        self.x, self.w = (torch.zeros(r, pitch, dtype=BF, device="cuda")[:, :k] for r in (m, n))
        self.x.copy_(randn(seed, m, k))
        self.w.copy_(randn(seed + 1, n, k) / math.sqrt(k))
        self.bias = randn(seed + 2, n)
        self.res = randn(seed + 3, m, n)
        self.acc = self.x.double() @ self.w.double().T

    def check(self, kb, ws, act="none", bias=False, residual=None, out=BF, save=False, alpha=1.0, in_place=False,
              layout=(0, 0), res_layout=None, z_layout=None):
        y, y_flat = matrix(self.m, self.n, out, *layout)
        r = None
        if residual is not None:
            r = y if in_place else matrix(self.m, self.n, residual, *(res_layout or layout))[0]
            r.copy_(self.res)
        z, z_flat = matrix(self.m, self.n, BF, *(z_layout or layout)) if save else (None, None)
        want_r = None if r is None else r.double()
        kb.klein_op_linear(self.x, self.w, y, ws, bias=self.bias if bias else None, residual=r, act=act, alpha=alpha,
                           preact=z)
        assert kb.klein_sync()[0] == 0
        zr = self.acc + self.bias.double() if bias else self.acc
        ref = alpha * act64(zr, act)
        if want_r is not None:
            ref = ref + want_r
        tol = abs(alpha) * (1.13 * SUM + 1e-5 * zr.abs()) + HALF[out] * ref.abs() + 1e-7
        what = (act, bias, residual, out, save, in_place, layout, res_layout, z_layout)
        err = (y.double() - ref).abs()
        assert (err <= tol).all(), (what, (err - tol).max().item())
        assert untouched(y, y_flat), what
        if save:
            assert ((z.double() - zr).abs() <= SUM + (1e-5 + HALF[BF]) * zr.abs()).all(), what
            assert untouched(z, z_flat), what


def every_epilogue(kb, p, ws, **layouts):
    for act in ("none", "silu", "gelu"):
        for residual in (None, BF, F32):
            for out in (BF, F32):
                for full in (False, True):
                    p.check(kb, ws, act, full, residual, out, full, 2.0, **layouts)
                if residual is out:
                    p.check(kb, ws, act, True, residual, out, True, -0.5, in_place=True, **layouts)


@pytest.mark.gpu
@pytest.mark.parametrize("m", [4999, 5120])  # 135 rows in the last tile; all of it
@pytest.mark.parametrize("n", [1032, 1072, 1112, 1144, 1192, 1272, 1280])  # 8 to 256 columns in the last tile
def test_whole_tiles(kb, m, n):
    p = Product(m, n, 192)
    every_epilogue(kb, p, workspace(kb, m, n, 192, False))


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k", [(1500, 1024, 2056), (1499, 136, 2056), (2100, 2312, 2056), (300, 1100, 5003)])
def test_cut_tiles(kb, m, n, k):
    """Every tile cut (the first two and the last), or those of the last wave."""
    p = Product(m, n, k)
    every_epilogue(kb, p, workspace(kb, m, n, k, True))


@pytest.mark.gpu
@pytest.mark.parametrize("n,layouts", [
    (1033, dict()),                                                       # an odd pitch
    (1044, dict()),                                                       # fp32 rows by TMA, bf16 ones not
    (1040, dict(layout=(8, 1))),                                          # no address on 16 bytes
    (1040, dict(layout=(8, 8), res_layout=(1, 0))),                       # the residual's pitch alone
    (1040, dict(layout=(8, 0), z_layout=(8, 1))),                         # the saved sums' address alone
])
def test_rows_that_tma_cannot_take(kb, n, layouts):
    for m, k, cut in ((4999, 192, False), (1500, 2056, True)):
        p = Product(m, n if not cut else n - 1024 + 264, k)
        ws = workspace(kb, m, p.n, k, cut)
        for residual in (None, BF, F32):
            for out in (BF, F32):
                for act in ("none", "gelu"):
                    p.check(kb, ws, act, True, residual, out, True, 2.0, **layouts)
                    p.check(kb, ws, act, False, residual, out, False, 2.0, **layouts)


@pytest.mark.gpu
@pytest.mark.parametrize("m,k,cut", [(5000, 64, False), (1500, 2056, True)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_tails(kb, m, k, cut, act):
    """Pre-activations from -1e30 to 1e30, infinities and NaN, in every 16th column."""
    n = 1024
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 12.0, -12.0, 88.0, -88.0, 100.0, -100.0, 1e15, -1e15, 1e30, -1e30,
                      math.inf, math.nan], device="cuda").bfloat16().repeat(n // 16)
    x, w = torch.zeros(m, k, device="cuda", dtype=BF), torch.zeros(n, k, device="cuda", dtype=BF)
    x[:, 0] = 1
    w[:, 0] = z
    ws = workspace(kb, m, n, k, cut)
    ref = act64(z.double(), act)
    finite, inf, nan = z.isfinite(), z == math.inf, z.isnan()
    for out in (BF, F32):
        y, pre = torch.empty(m, n, device="cuda", dtype=out), torch.empty(m, n, device="cuda", dtype=BF)
        kb.klein_op_linear(x, w, y, ws, act=act, preact=pre)
        assert kb.klein_sync()[0] == 0
        assert torch.isnan(y[:, nan]).all() and torch.isnan(pre[:, nan]).all()
        assert (y[:, inf] == math.inf).all() and (pre[:, inf] == math.inf).all()
        assert ((y[:, finite].double() - ref[finite]).abs() <= (1e-5 + HALF[out]) * ref[finite].abs() + 1e-12).all()
        assert (pre[:, finite] == z[finite]).all()
    wb = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    dout = torch.ones(m, n, device="cuda", dtype=BF)
    dw, dbias = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    kb.klein_op_linear_backward(dout, x, w, wb, dw=dw, dbias=dbias, preact=pre, act=act)
    assert kb.klein_sync()[0] == 0
    slope = m * act_grad64(z[finite].double().clamp(-60, 60), act)
    assert ((dbias[finite].double() - slope).abs() <= 1e-5 * m).all()
    assert ((dw[finite, 0].double() - slope).abs() <= m * (2.0 ** -16 * 1.13 + 1e-5)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("k,cut", [(192, False), (5000, True)])
@pytest.mark.parametrize("pitch", [1 << 23, (1 << 23) + 1])  # rows by TMA; a column to a lane
def test_offsets_that_pass_32_bits(kb, k, cut, pitch):
    """Rows of 2^23 elements and more: the last ones stand 2^31 elements behind the first. One far tensor at a time."""
    m, n = 300, 1032

    def far(t):
        flat = torch.empty((m - 1) * pitch + t.shape[1], dtype=t.dtype, device="cuda")
        view = flat.as_strided(t.shape, (pitch, 1))
        view.copy_(t)
        return view

    x, w = randn(0, m, k).bfloat16(), (randn(1, n, k) / math.sqrt(k)).bfloat16()
    r = randn(2, m, n)
    ws = workspace(kb, m, n, k, cut)
    zr = x.double() @ w.double().T
    for which, dtype in (("x", BF), ("out", BF), ("out", F32), ("residual", F32), ("z", BF)):
        if which == "x" and pitch % 8:
            continue
        res = r.to(dtype)
        y = far(torch.zeros(m, n, dtype=dtype, device="cuda")) if which == "out" else torch.empty(m, n, dtype=dtype, device="cuda")
        z = torch.zeros(m, n, dtype=BF, device="cuda")
        z = far(z) if which == "z" else z
        kb.klein_op_linear(far(x) if which == "x" else x, w, y, ws, residual=far(res) if which == "residual" else res,
                           act="silu", preact=z)
        assert kb.klein_sync()[0] == 0
        ref = act64(zr, "silu") + res.double()
        tol = 1.13 * SUM + 1e-5 * zr.abs() + HALF[dtype] * ref.abs() + 1e-7
        assert ((y.double() - ref).abs() <= tol).all(), which
        assert ((z.double() - zr).abs() <= SUM + (1e-5 + HALF[BF]) * zr.abs()).all(), which
        del y, z


@pytest.mark.gpu
def test_adapter_over_the_largest_image(kb):
    """A rank-16 adapter over 512 text and 256 x 256 image tokens, in place on the frozen layer's output: at this
    length its first half wants a workspace, and without one is refused."""
    m, k, r, n = 512 + 256 * 256, 2560, 16, 640
    x, a = randn(0, m, k).bfloat16(), (randn(1, r, k) / math.sqrt(k)).bfloat16()
    b, y0 = (randn(2, n, r) / 4).bfloat16(), randn(3, m, n).bfloat16()
    h, y = torch.empty(m, r, dtype=BF, device="cuda"), y0.clone()
    sizes = [kb.klein_linear_workspace_size(m, r, k), kb.klein_linear_workspace_size(m, n, r)]
    assert sizes[0] > 0
    with pytest.raises(kb.KleinError, match="workspace"):
        kb.klein_op_linear(x, a, h)
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    kb.klein_op_linear(x, a, h, ws)
    kb.klein_op_linear(h, b, y, ws, residual=y, alpha=2.0)
    assert kb.klein_sync()[0] == 0
    ref = x.double() @ a.double().T
    assert ((h.double() - ref).abs() <= SUM + (1e-5 + HALF[BF]) * ref.abs()).all()
    z = h.double() @ b.double().T
    ref = y0.double() + 2 * z
    assert ((y.double() - ref).abs() <= 2 * (SUM + 1e-5 * z.abs()) + HALF[BF] * ref.abs() + 1e-7).all()
