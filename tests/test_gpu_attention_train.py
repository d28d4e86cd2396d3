"""GPU tests of klein_op_attention_forward and klein_op_attention_backward against the formulas in float64.

Tolerances, per element, from the roundings the operators document (a bf16 rounding moves a value by at most
H = 2^-8 of it):
  out   H |out| for the output, H sum_j p_ij |v_j| for the probabilities
  lse   fp32 arithmetic: 128 products per score, the fast exponential and logarithm (1e-5 of the scores' size)
  dv    H |dv| + H sum_i p_ij |do_i|
  dS    H |dS| for its rounding; P times the error of D = sum_d do o, whose o carries H |o| (over up to 16 keys
        D is summed from the inputs and has only fp32's error)
  dq, dk   H of the result + scale times (error of dS) times |k| or |q|
FP32 = 3e-5 of the products' magnitudes covers fp32 sums, the recomputed scores and exponentials.
"""
import math

import pytest

torch = pytest.importorskip("torch")

H = 2.0 ** -8
FP32 = 3e-5
D = 128


@pytest.fixture(scope="module")
def kb():
    from conftest import ensure_built
    ensure_built()
    import latent_flow_matching_joint_b200 as kb
    return kb


def randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


def layout(t, kind):
    """The values of t [b, h, n, 128] in another memory layout."""
    if kind == "bnhd":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if kind == "padded":  # rows of 136 elements in planes of n + 3 rows
        b, h, n, d = t.shape
        whole = torch.full((b, h, n + 3, 136), 3.0, dtype=t.dtype, device=t.device)
        whole[:, :, :n, :d] = t
        return whole[:, :, :n, :d]
    return t.contiguous()


def mask(batch, n, n_txt, lens):
    row = torch.arange(n, device="cuda")[None]
    if lens is None:
        return torch.ones(batch, n, dtype=torch.bool, device="cuda")
    return (row < torch.tensor(lens, device="cuda").clamp(0, n_txt)[:, None]) | (row >= n_txt)


class Reference:
    """The formulas in float64 with padding rows taken out, and the error bounds."""

    def __init__(self, q, k, v, dout, use, scale, few_keys=False):
        group = q.shape[1] // k.shape[1]
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        row = use[:, None, :, None]
        q, do = (torch.where(row, t.double(), zero) for t in (q, dout))
        k, v = (torch.where(row, t.double(), zero).repeat_interleave(group, 1) for t in (k, v))
        pair = use[:, None, :, None] & use[:, None, None, :]
        s = torch.where(pair, scale * (q @ k.transpose(2, 3)), torch.full_like(zero, -math.inf))
        self.lse = torch.logsumexp(s, -1)
        p = torch.where(pair, torch.exp(s - self.lse[..., None]), zero)
        size = torch.where(pair, scale * (q.abs() @ k.abs().transpose(2, 3)), zero).amax((-2, -1), keepdim=True)
        self.out = p @ v
        self.out_tol = H * self.out.abs() + (H + FP32 * (1 + size)) * (p @ v.abs())
        self.lse_tol = 1e-6 * (2 + size.squeeze(-1) + torch.nan_to_num(self.lse.abs(), posinf=0.0))
        delta = (do * self.out).sum(-1, keepdim=True)
        dp = do @ v.transpose(2, 3)
        ds = p * (dp - delta)
        mag = p * (do.abs() @ v.abs().transpose(2, 3) + (do * self.out).abs().sum(-1, keepdim=True))
        ds_err = H * ds.abs() + FP32 * (1 + size) * mag
        if not few_keys:
            ds_err = ds_err + p * H * (do * self.out).abs().sum(-1, keepdim=True)

        def shared(t):
            return t.reshape(t.shape[0], -1, group, t.shape[2], D).sum(2)

        self.dv = shared(p.transpose(2, 3) @ do)
        self.dv_tol = H * self.dv.abs() + (H + FP32 * (1 + size[:, :1].amax(1, keepdim=True))) * shared(p.transpose(2, 3) @ do.abs())
        self.dq = scale * (ds @ k)
        self.dq_tol = H * self.dq.abs() + scale * (ds_err @ k.abs())
        self.dk = shared(scale * (ds.transpose(2, 3) @ q))
        self.dk_tol = H * self.dk.abs() + shared(scale * (ds_err.transpose(2, 3) @ q.abs()))


def within(name, got, ref, tol):
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), name
    assert (err <= 1.02 * tol + 1e-9).all(), (name, (err - tol).max().item(), err.max().item())


def run(kb, q, k, v, dout, n_txt=0, lens=None, scale=None, kinds=("bhnd",) * 5):
    b, h, n, _ = q.shape
    q, k, v, dout = (layout(t, kind) for t, kind in zip((q, k, v, dout), kinds))
    txt_len = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, dq = (layout(torch.full_like(q, 7.0), kinds[4]) for _ in range(2))
    dk, dv = (layout(torch.full_like(k, 7.0), kinds[4]) for _ in range(2))
    lse = torch.full((b, h, n), 7.0, device="cuda")
    ws = torch.full((kb.klein_attention_backward_workspace_size(b, h, n, n_txt),), 255, dtype=torch.uint8, device="cuda")
    kb.klein_op_attention_forward(q, k, v, out, lse, n_txt=n_txt, txt_len=txt_len, scale=scale)
    assert kb.klein_sync()[0] == 0
    kb.klein_op_attention_backward(q, k, v, out, lse, dout, dq, dk, dv, ws, n_txt=n_txt, txt_len=txt_len, scale=scale)
    assert kb.klein_sync()[0] == 0
    return out, lse, dq, dk, dv


def check(kb, batch, heads, kv_heads, n, n_txt=0, lens=None, scale=D ** -0.5, kinds=("bhnd",) * 5, seed=0, junk=None,
          gain=1.0):
    q = (gain * randn(seed, batch, heads, n, D)).bfloat16()
    k = (gain * randn(seed + 1, batch, kv_heads, n, D)).bfloat16()
    v, dout = randn(seed + 2, batch, kv_heads, n, D).bfloat16(), randn(seed + 3, batch, heads, n, D).bfloat16()
    use = mask(batch, n, n_txt, lens)
    if junk is not None:
        for t in (q, k, v, dout):
            t.masked_fill_(~use[:, None, :, None], junk)
    out, lse, dq, dk, dv = run(kb, q, k, v, dout, n_txt, lens, None if scale == D ** -0.5 else scale, kinds)
    ref = Reference(q, k, v, dout, use, scale)
    row = use[:, None, :].expand(batch, heads, n)
    assert (lse[~row] == -math.inf).all()
    assert torch.isfinite(lse[row]).all()
    assert ((lse.double() - ref.lse).abs()[row] <= ref.lse_tol.expand_as(row)[row]).all()
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(name, got, getattr(ref, name), getattr(ref, name + "_tol"))
        assert (got[(~use)[:, None, :].expand(got.shape[:3])] == 0).all(), name
        if kinds[4] == "padded":  # nothing between the rows is written
            whole = torch.as_strided(got, (*got.shape[:2], n + 3, 136), got.stride())
            assert (whole[:, :, n:] == 3.0).all() and (whole[:, :, :, D:] == 3.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 384, 700])
def test_lengths(kb, n):
    check(kb, 1, 2, 2, n)
    check(kb, 2, 6, 2, n, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (24, 24), (24, 8), (8, 1), (6, 3)])
def test_heads(kb, heads, kv_heads):
    check(kb, 2, heads, kv_heads, 200, seed=1)


@pytest.mark.gpu
@pytest.mark.parametrize("n,n_txt,lens", [
    (80, 80, [77, 23]),          # text only
    (80, 80, [0, 80]),           # an item with nothing in it
    (1, 1, [0, 1]),
    (300, 80, [1, 79]),
    (300, 160, [0, 160]),        # no text; all of it
    (300, 160, [128, 129]),      # a slot's end
    (300, 299, [255, 256]),
    (513, 300, [40, 300]),
    (520, 512, [130, 500]),
    (400, 80, [-5, 1000]),       # clamped to [0, n_txt]
    (129, 128, [127, 128]),
])
@pytest.mark.parametrize("junk", [None, float("nan"), float("inf"), -3.3e38])
def test_padding(kb, n, n_txt, lens, junk):
    check(kb, 2, 4, 2, n, n_txt, lens, seed=2, junk=junk)


@pytest.mark.gpu
@pytest.mark.parametrize("kinds", [("bnhd",) * 5, ("bhnd", "bnhd", "padded", "bhnd", "padded"),
                                   ("padded",) * 5, ("bnhd", "padded", "bhnd", "padded", "bnhd")])
def test_layouts(kb, kinds):
    check(kb, 2, 6, 3, 150, kinds=kinds, seed=3)
    check(kb, 2, 6, 3, 310, 100, [33, 100], kinds=kinds, seed=4, junk=float("nan"))
    check(kb, 1, 1, 1, 1, kinds=kinds, seed=4)


@pytest.mark.gpu
def test_packed_projection(kb):
    """q, k, v (and their gradients) inside one [batch, rows, heads + 2 kv heads, 128] tensor."""
    b, n, h, g = 2, 200, 6, 2
    whole = randn(1, b, n, h + 2 * g, D).bfloat16()
    grads = torch.full_like(whole, 7.0)
    parts = [t.transpose(1, 2) for t in whole.split([h, g, g], dim=2)]
    dparts = [t.transpose(1, 2) for t in grads.split([h, g, g], dim=2)]
    dout = randn(2, b, h, n, D).bfloat16()
    out, lse = torch.empty_like(dout), torch.empty(b, h, n, device="cuda")
    ws = torch.empty(kb.klein_attention_backward_workspace_size(b, h, n), dtype=torch.uint8, device="cuda")
    kb.klein_op_attention_forward(*parts, out, lse)
    kb.klein_op_attention_backward(*parts, out, lse, dout, *dparts, ws)
    ref = Reference(*parts, dout, mask(b, n, 0, None), D ** -0.5)
    within("out", out, ref.out, ref.out_tol)
    for name, got in zip(("dq", "dk", "dv"), dparts):
        within(name, got, getattr(ref, name), getattr(ref, name + "_tol"))


@pytest.mark.gpu
@pytest.mark.parametrize("scale,gain", [(0.01, 1.0), (1.0, 1.0), (D ** -0.5, 4.0)])
def test_scales(kb, scale, gain):
    """From nearly uniform probabilities to one key taking almost everything."""
    check(kb, 1, 3, 1, 270, scale=scale, gain=gain, seed=6)


@pytest.mark.gpu
def test_scores_that_climb(kb):
    """The running maximum moves in every key tile, for some rows of a warp and not for others."""
    n = 600
    q = torch.linspace(0, 1.5, n, device="cuda")[None, None, :, None] * (1 + 0.1 * randn(1, 1, 2, n, D))
    k = (torch.arange(n, device="cuda") / 64.0)[None, None, :, None] * (1 + 0.1 * randn(2, 1, 2, n, D))
    v, dout = randn(3, 1, 2, n, D).bfloat16(), randn(4, 1, 2, n, D).bfloat16()
    q, k = q.bfloat16(), k.bfloat16()
    out, lse, dq, dk, dv = run(kb, q, k, v, dout)
    ref = Reference(q, k, v, dout, mask(1, n, 0, None), D ** -0.5)
    for name, got in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(name, got, getattr(ref, name), getattr(ref, name + "_tol"))
    assert ((lse.double() - ref.lse).abs() <= ref.lse_tol).all()


@pytest.mark.gpu
def test_long_sequence(kb):
    check(kb, 1, 2, 1, 4608, 512, [313], seed=7, junk=float("nan"))


@pytest.mark.gpu
def test_forward_agrees_with_the_denoisers_attention(kb):
    """24 heads without padding: the same function as klein_op_attention, to bf16 roundings of both."""
    n, rp = 300, 384
    q, k, v = (randn(i, 1, 24, n, D).bfloat16() for i in range(3))
    qp, kp = (torch.zeros(1, 24, rp, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    vt = torch.zeros(1, 24, D, rp, dtype=torch.bfloat16, device="cuda")
    qp[:, :, :n], kp[:, :, :n], vt[:, :, :, :n] = q, k, v.transpose(2, 3)
    want = torch.empty(1, n, 24 * D, dtype=torch.bfloat16, device="cuda")
    kb.klein_op_attention(qp, kp, vt, n, want)
    got = torch.empty(1, n, 24, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 24, n, device="cuda")
    kb.klein_op_attention_forward(q, k, v, got.transpose(1, 2), lse)
    ref = Reference(q, k, v, q, mask(1, n, 0, None), D ** -0.5)
    diff = (got.double() - want.reshape(got.shape).double()).abs()
    assert (diff <= 2.04 * ref.out_tol.transpose(1, 2) + 1e-9).all()


@pytest.mark.gpu
def test_gradients_match_differences(kb):
    """Directional derivatives of L = sum(dout * out), by central differences of the formula in float64."""
    b, h, g, n, n_txt, lens = 1, 4, 2, 150, 60, [37]
    q, k, v = (randn(i, b, heads, n, D).bfloat16() for i, heads in ((1, h), (2, g), (3, g)))
    dout = randn(4, b, h, n, D).bfloat16()
    use = mask(b, n, n_txt, lens)
    _, _, *grads = run(kb, q, k, v, dout, n_txt, lens)

    def loss(q, k, v):
        s = (q @ k.repeat_interleave(h // g, 1).transpose(2, 3)) * D ** -0.5
        s = s.masked_fill(~use[:, None, None, :], -math.inf)
        o = torch.softmax(s, -1) @ v.repeat_interleave(h // g, 1)
        return (o * dout.double() * use[:, None, :, None]).sum().item()

    values = [t.double() for t in (q, k, v)]
    for i, grad in enumerate(grads):
        for seed in (11, 12):
            way = randn(seed, *grad.shape).double()
            step = 1e-4
            hi, lo = list(values), list(values)
            hi[i], lo[i] = values[i] + step * way, values[i] - step * way
            slope = (loss(*hi) - loss(*lo)) / (2 * step)
            terms = grad.double() * way
            # each gradient element is off by a few independent roundings of 2^-8; six of them, added up in norm
            assert abs(terms.sum().item() - slope) <= 6 * H * terms.norm().item() + 1e-6


@pytest.mark.gpu
def test_same_bits_every_time(kb):
    q, k, v, dout = (randn(i, 2, heads, 500, D).bfloat16() for i, heads in ((1, 6), (2, 2), (3, 2), (4, 6)))
    first = run(kb, q, k, v, dout, 100, [40, 100])
    again = run(kb, q, k, v, dout, 100, [40, 100])
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.gpu
def test_stream_and_graph(kb):
    """On another stream and in a replayed graph, the lengths read when the graph runs."""
    b, h, n, n_txt = 2, 2, 300, 128
    q, k, v, dout = (randn(i, b, h, n, D).bfloat16() for i in range(4))
    lens = torch.tensor([50, 128], dtype=torch.int32, device="cuda")
    out, dq, dk, dv = (torch.empty_like(q) for _ in range(4))
    lse = torch.empty(b, h, n, device="cuda")
    ws = torch.empty(kb.klein_attention_backward_workspace_size(b, h, n, n_txt), dtype=torch.uint8, device="cuda")

    def both():
        kb.klein_op_attention_forward(q, k, v, out, lse, n_txt=n_txt, txt_len=lens)
        kb.klein_op_attention_backward(q, k, v, out, lse, dout, dq, dk, dv, ws, n_txt=n_txt, txt_len=lens)

    want = run(kb, q, k, v, dout, n_txt, [50, 128])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((out, lse, dq, dk, dv), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for new in ([50, 128], [3, 0]):
        lens.copy_(torch.tensor(new))
        for t in (out, dq, dk, dv, lse):
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        want = run(kb, q, k, v, dout, n_txt, new)
        assert all(torch.equal(x, y) for x, y in zip((out, lse, dq, dk, dv), want))


@pytest.mark.gpu
def test_offsets_that_pass_32_bits(kb):
    """The second batch row stands 2^31 elements and more behind the first, in each tensor in turn."""
    b, heads, kv_heads, n, n_txt, lens, scale = 2, 2, 1, 200, 130, [5, 130], D ** -0.5
    gap = (1 << 31) + 4096

    def far(t):
        size = t[0].numel()
        flat = torch.empty(gap + size, dtype=t.dtype, device="cuda")
        view = flat.as_strided(t.shape, (gap,) + t[0].contiguous().stride())
        view.copy_(t)
        return view

    q, dout = (randn(s, b, heads, n, D).bfloat16() for s in (1, 2))
    k, v = (randn(s, b, kv_heads, n, D).bfloat16() for s in (3, 4))
    ref = Reference(q, k, v, dout, mask(b, n, n_txt, lens), scale)
    txt_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.empty(kb.klein_attention_backward_workspace_size(b, heads, n, n_txt), dtype=torch.uint8, device="cuda")
    for which in ("q", "k", "v", "out", "dout", "dq", "dk", "dv"):
        t = {"q": q, "k": k, "v": v, "dout": dout, "out": torch.zeros_like(q), "dq": torch.zeros_like(q),
             "dk": torch.zeros_like(k), "dv": torch.zeros_like(k)}
        t[which] = far(t[which])
        lse = torch.zeros(b, heads, n, device="cuda")
        kb.klein_op_attention_forward(t["q"], t["k"], t["v"], t["out"], lse, n_txt=n_txt, txt_len=txt_len)
        kb.klein_op_attention_backward(t["q"], t["k"], t["v"], t["out"], lse, t["dout"], t["dq"], t["dk"], t["dv"], ws,
                                       n_txt=n_txt, txt_len=txt_len)
        assert kb.klein_sync()[0] == 0
        for name in ("out", "dq", "dk", "dv"):
            within(f"{name}, {which} far", t[name], getattr(ref, name), getattr(ref, name + "_tol"))
        del t


@pytest.mark.gpu
@pytest.mark.parametrize("heads,kv_heads,n,n_txt,lens", [
    (2, 2, 1, 0, None), (2, 1, 2, 0, None), (24, 24, 3, 0, None), (4, 2, 8, 0, None), (3, 1, 9, 0, None), (2, 2, 16, 0, None),
    (2, 1, 2, 1, [0, 1]), (4, 2, 302, 300, [0, 14]), (4, 4, 200, 200, [1, 16]), (2, 2, 140, 129, [0, 5])])
def test_few_keys(kb, heads, kv_heads, n, n_txt, lens):
    """Over up to 16 keys the output's rounding is not in dq and dk; padding rows hold NaN."""
    b, scale = 2, D ** -0.5
    q, dout = (randn(s, b, heads, n, D).bfloat16() for s in (1, 2))
    k, v = (randn(s, b, kv_heads, n, D).bfloat16() for s in (3, 4))
    use = mask(b, n, n_txt, lens)
    for t in (q, dout, k, v):
        t.masked_fill_(~use[:, None, :, None], float("nan"))
    ref = Reference(q, k, v, dout, use, scale, few_keys=True)
    out, lse, dq, dk, dv = run(kb, q, k, v, dout, n_txt, lens)
    rows = use[:, None, :, None]
    for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
        within(name, got, getattr(ref, name), torch.nan_to_num(getattr(ref, name + "_tol"), nan=0.0))
        assert (got.masked_select(~rows) == 0).all(), name


@pytest.mark.gpu
@pytest.mark.parametrize("after", [15, 16, 17])
def test_few_keys_border(kb, after):
    """Items of few keys and of many in one batch, around as many rows after the text as count as few."""
    b, heads, kv_heads, n_txt, scale = 4, 4, 2, 300, D ** -0.5
    n, lens = n_txt + after, [0, 1, 2, 300]
    q, dout = (randn(s, b, heads, n, D).bfloat16() for s in (1, 2))
    k, v = (randn(s, b, kv_heads, n, D).bfloat16() for s in (3, 4))
    use = mask(b, n, n_txt, lens)
    for t in (q, dout, k, v):
        t.masked_fill_(~use[:, None, :, None], float("nan"))
    few, many = (Reference(q, k, v, dout, use, scale, few_keys=f) for f in (True, False))
    _, _, dq, dk, dv = run(kb, q, k, v, dout, n_txt, lens)
    for i in range(b):
        ref = few if lens[i] + after <= 16 else many
        for name, got in (("dq", dq), ("dk", dk), ("dv", dv)):
            within(name, got[i], getattr(ref, name)[i], torch.nan_to_num(getattr(ref, name + "_tol")[i], nan=0.0))
            assert (got[i].masked_select(~use[i, None, :, None]) == 0).all(), name
