"""The training operators together, as an adapter on the attention part of a block uses them, against autograd in
float64; their binding's refusals; and calls at the edges of their ranges."""
import math

import pytest

torch = pytest.importorskip("torch")

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


class AdapterStep:
    """y = x + Wo attention(Wqkv x + 2 B (A x)) + bo, fp32 residual stream x; gradients of A, B, Wo, bo and x from
    dy. Every buffer is allocated once, as a training program keeps them."""

    def __init__(self, kb, batch, n_txt, n_img, heads, kv_heads, rank, seed=0):
        self.kb, self.b, self.n, self.n_txt = kb, batch, n_txt + n_img, n_txt
        self.h, self.g, self.r = heads, kv_heads, rank
        c, e = heads * D, (heads + 2 * kv_heads) * D
        m = batch * self.n
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.x32 = randn(seed, m, c)
        self.x = self.x32.bfloat16()
        self.wqkv = (randn(seed + 1, e, c) / math.sqrt(c)).bfloat16()
        self.a = (randn(seed + 2, rank, c) / math.sqrt(c)).bfloat16()
        self.bm = (randn(seed + 3, e, rank) / math.sqrt(rank) / 2).bfloat16()
        self.wo = (randn(seed + 4, c, c) / math.sqrt(c)).bfloat16()
        self.bo = randn(seed + 5, c)
        self.dy = randn(seed + 6, m, c).bfloat16()
        self.lens = torch.tensor([n_txt - 3 * i - 1 for i in range(batch)], dtype=torch.int32, device="cuda")
        row = torch.arange(self.n, device="cuda")
        self.use = (row[None] < self.lens[:, None]) | (row[None] >= n_txt)
        self.qkv, self.dqkv = torch.empty(m, e, **bf), torch.empty(m, e, **bf)
        self.hid, self.dhid = torch.empty(m, rank, **bf), torch.empty(m, rank, **bf)
        self.o, self.do = torch.empty(m, c, **bf), torch.empty(m, c, **bf)
        self.lse = torch.empty(batch, heads, self.n, device="cuda")
        self.y = torch.empty(m, c, device="cuda")
        self.da, self.db = torch.empty(rank, c, device="cuda"), torch.empty(e, rank, device="cuda")
        self.dwo, self.dbo = torch.empty(c, c, device="cuda"), torch.empty(c, device="cuda")
        self.dx_parts = [torch.empty(m, c, device="cuda") for _ in range(2)]
        sizes = [kb.klein_linear_workspace_size(m, p, q) for p, q in ((e, c), (rank, c), (e, rank), (c, c))]
        sizes += [kb.klein_linear_backward_workspace_size(m, p, q) for p, q in ((e, c), (rank, c), (e, rank), (c, c))]
        sizes.append(kb.klein_attention_backward_workspace_size(batch, heads, self.n, n_txt))
        self.ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")

    def heads_of(self, t):
        """q, k, v views of a packed projection, [batch, heads, rows, 128]."""
        t = t.view(self.b, self.n, self.h + 2 * self.g, D)
        return [p.transpose(1, 2) for p in t.split([self.h, self.g, self.g], dim=2)]

    def one(self, t):
        return t.view(self.b, self.n, self.h, D).transpose(1, 2)

    def run(self):
        kb, ws = self.kb, self.ws
        kb.klein_op_linear(self.x, self.wqkv, self.qkv, ws)
        kb.klein_op_linear(self.x, self.a, self.hid, ws)
        kb.klein_op_linear(self.hid, self.bm, self.qkv, ws, residual=self.qkv, alpha=2.0)  # in place
        pad = dict(n_txt=self.n_txt, txt_len=self.lens)
        kb.klein_op_attention_forward(*self.heads_of(self.qkv), self.one(self.o), self.lse, **pad)
        kb.klein_op_linear(self.o, self.wo, self.y, ws, bias=self.bo, residual=self.x32)
        kb.klein_op_linear_backward(self.dy, self.o, self.wo, ws, dx=self.do, dw=self.dwo, dbias=self.dbo)
        kb.klein_op_attention_backward(*self.heads_of(self.qkv), self.one(self.o), self.lse, self.one(self.do),
                                       *self.heads_of(self.dqkv), ws, **pad)
        kb.klein_op_linear_backward(self.dqkv, self.hid, self.bm, ws, dx=self.dhid, dw=self.db, alpha=2.0)
        kb.klein_op_linear_backward(self.dhid, self.x, self.a, ws, dx=self.dx_parts[0], dw=self.da)
        kb.klein_op_linear_backward(self.dqkv, self.x, self.wqkv, ws, dx=self.dx_parts[1])
        return [self.y, self.da, self.db, self.dwo, self.dbo, *self.dx_parts]

    def reference(self):
        x, a, bm, wo, bo = (t.double().requires_grad_(True) for t in (self.x, self.a, self.bm, self.wo, self.bo))
        qkv = x @ self.wqkv.double().T + 2.0 * (x @ a.T) @ bm.T
        q, k, v = self.heads_of(qkv)
        k, v = (t.repeat_interleave(self.h // self.g, 1) for t in (k, v))
        s = q @ k.transpose(2, 3) * D ** -0.5
        s = s.masked_fill(~self.use[:, None, None, :], -math.inf)
        o = (torch.softmax(s, -1) @ v) * self.use[:, None, :, None]
        y = self.x32.double() + o.transpose(1, 2).reshape(x.shape) @ wo.T + bo
        grads = torch.autograd.grad((y * self.dy.double()).sum(), (a, bm, wo, bo, x))
        return [y.detach(), *grads]


def relative(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


@pytest.mark.gpu
@pytest.mark.parametrize("batch,n_txt,n_img,heads,kv_heads,rank", [(1, 80, 100, 2, 2, 16), (2, 160, 221, 4, 2, 8),
                                                                   (3, 7, 1, 2, 1, 8)])
def test_adapter_step(kb, batch, n_txt, n_img, heads, kv_heads, rank):
    """Each stored bf16 tensor between x and a gradient (qkv, A x, P, o, do, dS, dqkv, d(A x)) adds a relative error
    of at most half a step, 2^-8, in norm; eight of them, 3.2e-2. y carries three (qkv, P, o) on its attention part,
    which is smaller than the residual it is added to."""
    step = AdapterStep(kb, batch, n_txt, n_img, heads, kv_heads, rank)
    y, da, db, dwo, dbo, dx0, dx1 = step.run()
    assert kb.klein_sync()[0] == 0
    ry, ra, rb, rwo, rbo, rx = step.reference()
    assert relative(y, ry) <= 3 * 2.0 ** -8
    for name, got, ref in (("a", da, ra), ("b", db, rb), ("wo", dwo, rwo), ("x", dx0 + dx1, rx)):
        assert relative(got, ref) <= 8 * 2.0 ** -8, name
    assert relative(dbo, rbo) <= 1e-6


@pytest.mark.gpu
def test_adapter_step_captured(kb):
    """The whole step as one graph, replayed on new inputs, gives the eager step's bits."""
    step = AdapterStep(kb, 2, 80, 150, 4, 2, 16)
    step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step.run()
    for seed in (50, 60):
        other = AdapterStep(kb, 2, 80, 150, 4, 2, 16, seed=seed)
        for name in ("x32", "x", "wqkv", "a", "bm", "wo", "bo", "dy"):
            getattr(step, name).copy_(getattr(other, name))
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        want = other.run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


FIRST_CALL = """
import torch
import latent_flow_matching_joint_b200 as kb
def bf(*shape): return torch.randn(*shape, device="cuda").bfloat16()
q, do, x, w = bf(1, 2, 200, 128), bf(1, 2, 200, 128), bf(1200, 1024), bf(1024, 1024)
outs = [torch.zeros(1, 2, 200, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
lse, y = torch.zeros(1, 2, 200, device="cuda"), torch.zeros(1200, 1024, device="cuda")
dx, dw = torch.zeros(1200, 1024, device="cuda"), torch.zeros(1024, 1024, device="cuda")
wa = torch.empty(kb.klein_attention_backward_workspace_size(1, 2, 200), dtype=torch.uint8, device="cuda")
wl = torch.empty(max(kb.klein_linear_workspace_size(1200, 1024, 1024),
                     kb.klein_linear_backward_workspace_size(1200, 1024, 1024)), dtype=torch.uint8, device="cuda")
def step():
    kb.klein_op_attention_forward(q, k, v, outs[0], lse)
    kb.klein_op_attention_backward(q, k, v, outs[0], lse, do, *outs[1:], wa)
    kb.klein_op_linear(x, w, y, wl)
    kb.klein_op_linear_backward(y, x, w, wl, dx=dx, dw=dw)
k, v = q.clone(), do.clone()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (*outs, lse, y, dx, dw)]
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) and a.abs().sum() > 0 for a, b in zip(got, (*outs, lse, y, dx, dw)))
print("first call captured")
"""


@pytest.mark.gpu
def test_first_calls_of_a_process_captured(kb):
    """Nothing that a call sets up at its first use stands in the way of a stream capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, env={**os.environ, "PYTHONPATH": root},
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "first call captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_two_steps_at_once(kb):
    """Two steps on two streams, each with its own workspace."""
    steps = [AdapterStep(kb, 2, 80, 1500, 8, 2, 16, seed=s) for s in (0, 100)]
    want = [[t.clone() for t in s.run()] for s in steps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for step, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                step.run()
    torch.cuda.synchronize()
    for step, w in zip(steps, want):
        got = [step.y, step.da, step.db, step.dwo, step.dbo, *step.dx_parts]
        assert all(torch.equal(a, b) for a, b in zip(got, w))


@pytest.mark.gpu
def test_binding_refusals(kb):
    def bf(*shape):
        return torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")

    def f32(*shape):
        return torch.zeros(*shape, device="cuda")

    x, w, y = bf(8, 64), bf(16, 64), bf(8, 16)
    ws = torch.empty(kb.klein_linear_backward_workspace_size(8, 16, 64), dtype=torch.uint8, device="cuda")
    bad = [lambda: kb.klein_op_linear(x.float(), w, y), lambda: kb.klein_op_linear(x, w.half(), y),
           lambda: kb.klein_op_linear(x, w, y.half()), lambda: kb.klein_op_linear(x, w, bf(16, 8)),
           lambda: kb.klein_op_linear(x, bf(16, 72), y), lambda: kb.klein_op_linear(x, w, bf(16, 8).T),
           lambda: kb.klein_op_linear(bf(64, 8).T, w, y), lambda: kb.klein_op_linear(x, w, y, bias=bf(16)),
           lambda: kb.klein_op_linear(x, w, y, bias=f32(15)), lambda: kb.klein_op_linear(x, w, y, bias=f32(32)[::2]),
           lambda: kb.klein_op_linear(x, w, y, residual=f32(8, 15)), lambda: kb.klein_op_linear(x, w, y, preact=f32(8, 16)),
           lambda: kb.klein_op_linear(x, w, y, residual=torch.zeros(8, 16)),
           lambda: kb.klein_op_linear(bf(8, 65)[:, 1:], w, y), lambda: kb.klein_op_linear(bf(9, 60)[:8, :60], bf(16, 60), y),
           lambda: kb.klein_op_linear_backward(y, x, w, ws), lambda: kb.klein_op_linear_backward(y, x, w, None, dx=x),
           lambda: kb.klein_op_linear_backward(y, x, w, ws[:100], dx=bf(8, 64)),
           lambda: kb.klein_op_linear_backward(y, x, w, ws[::2], dx=bf(8, 64)),
           lambda: kb.klein_op_linear_backward(y, x, w, ws, dx=bf(8, 64), act="silu"),
           lambda: kb.klein_op_linear_backward(y, x, w, ws, dw=bf(64, 16)),
           lambda: kb.klein_op_linear_backward(y, x, w, ws, dbias=bf(16))]
    q, k, lse = bf(2, 4, 10, D), bf(2, 2, 10, D), f32(2, 4, 10)
    wa = torch.empty(kb.klein_attention_backward_workspace_size(2, 4, 10), dtype=torch.uint8, device="cuda")
    fwd, bwd = kb.klein_op_attention_forward, kb.klein_op_attention_backward
    i32 = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad += [lambda: fwd(q.float(), k, k, bf(2, 4, 10, D), lse), lambda: fwd(q, k, bf(2, 2, 9, D), bf(2, 4, 10, D), lse),
            lambda: fwd(bf(2, 4, 10, 64), bf(2, 2, 10, 64), bf(2, 2, 10, 64), bf(2, 4, 10, 64), lse),
            lambda: fwd(q, bf(2, 3, 10, D), bf(2, 3, 10, D), bf(2, 4, 10, D), lse),
            lambda: fwd(q, k, k, bf(2, 4, 10, D), lse.double()), lambda: fwd(q, k, k, bf(2, 4, 10, D), f32(2, 10, 4)),
            lambda: fwd(q, k, k, bf(2, 4, 10, D), f32(2, 10, 4).transpose(1, 2)),
            lambda: fwd(q, k, k, bf(2, 4, D, 10).transpose(2, 3), lse), lambda: fwd(q, k, k, bf(2, 1, 10, D).expand(2, 4, 10, D), lse),
            lambda: fwd(q, bf(2, 1, 10, D).expand(2, 2, 10, D), k, bf(2, 4, 10, D), lse),
            lambda: fwd(q, k, k, bf(2, 4, 10, D), lse, n_txt=5, txt_len=i32.long()),
            lambda: fwd(q, k, k, bf(2, 4, 10, D), lse, n_txt=5, txt_len=i32[:1]),
            lambda: fwd(q, k, k, bf(2, 4, 10, D), lse, n_txt=5, txt_len=i32.cpu()),
            lambda: fwd(q, k, k, bf(2, 4, 10, D), lse, n_txt=11, txt_len=i32),
            lambda: fwd(q, k, k, bf(2, 4, 10, D), lse, scale=0.0), lambda: fwd(q[0], k[0], k[0], q[0], lse),
            lambda: bwd(q, k, k, q, lse, q, bf(2, 4, 10, D), bf(2, 2, 10, D), bf(2, 2, 10, D), wa[:16]),
            lambda: bwd(q, k, k, q, lse, q, bf(2, 4, 10, D), bf(2, 4, 10, D), bf(2, 2, 10, D), wa),
            lambda: bwd(q, k, k, q, lse, q.float(), bf(2, 4, 10, D), bf(2, 2, 10, D), bf(2, 2, 10, D), wa)]
    before = kb.klein_launch_count()
    for i, call in enumerate(bad):
        with pytest.raises(kb.KleinError):
            call()
            raise AssertionError(f"call {i} was taken")
    assert kb.klein_launch_count() == before
    assert kb.klein_sync()[0] == 0


@pytest.mark.gpu
def test_attention_offsets_past_32_bits(kb):
    """Rows 2^25 bytes apart: offsets of 10 GB in one tensor of rows [q | k | v | out | dout | dq | dk | dv]."""
    n, stride = 300, 1 << 24
    whole = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
    q, k, v, out, dout, dq, dk, dv = (torch.as_strided(whole, (1, 1, n, D), (stride * n, stride, stride, 1), i * D)
                                      for i in range(8))
    for i, t in enumerate((q, k, v, dout)):
        t.copy_(randn(i, 1, 1, n, D))
    lse = torch.empty(1, 1, n, device="cuda")
    ws = torch.empty(kb.klein_attention_backward_workspace_size(1, 1, n), dtype=torch.uint8, device="cuda")
    kb.klein_op_attention_forward(q, k, v, out, lse)
    kb.klein_op_attention_backward(q, k, v, out, lse, dout, dq, dk, dv, ws)
    near = [t.contiguous() for t in (q, k, v)]
    want = [torch.empty(1, 1, n, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    lse2 = torch.empty_like(lse)
    kb.klein_op_attention_forward(*near, want[0], lse2)
    kb.klein_op_attention_backward(*near, want[0], lse2, dout.contiguous(), *want[1:], ws)
    assert torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip((out, dq, dk, dv), want))
    del whole


@pytest.mark.gpu
def test_linear_offsets_past_32_bits(kb):
    """An output of 2.3e9 elements."""
    m, n, k = 70000, 33000, 64
    x, w = randn(1, m, k).bfloat16(), (randn(2, n, k) / 8).bfloat16()
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    kb.klein_op_linear(x, w, y, torch.empty(kb.klein_linear_workspace_size(m, n, k), dtype=torch.uint8, device="cuda"))
    rows = torch.tensor([0, 1, 255, 256, 40000, 65535, 65536, 69887, 69888, 69998, 69999], device="cuda")
    ref = x[rows].double() @ w.double().T
    assert ((y[rows].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 1e-5).all()
    # its gradient: sums over 33000 columns and 70000 rows
    dx, dw = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
    db = torch.empty(n, device="cuda")
    ws = torch.empty(kb.klein_linear_backward_workspace_size(m, n, k), dtype=torch.uint8, device="cuda")
    kb.klein_op_linear_backward(y, x, w, ws, dx=dx, dw=dw, dbias=db)
    ref = y[rows].double() @ w.double()
    assert ((dx[rows].double() - ref).norm() / ref.norm()).item() <= 2e-6
    cols = torch.tensor([0, 16383, 16384, 32767, 32768, 32999], device="cuda")
    part = y[:, cols].double()
    assert ((dw[cols].double() - part.T @ x.double()).norm() / (part.T @ x.double()).norm()).item() <= 2e-6
    assert ((db[cols].double() - part.sum(0)).abs() <= 1e-5 * part.abs().sum(0)).all()
