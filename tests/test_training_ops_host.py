"""CPU tests of the training operators' argument checks: every refusal happens before any device work, with a
negative status and a message. Addresses are made up and never read."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

A = 1 << 20  # an aligned address


@pytest.fixture(scope="module")
def kb():
    from conftest import ensure_built
    ensure_built()
    import latent_flow_matching_joint_b200 as kb
    return kb


def linear(kb, **change):
    a = dict(m=8, n=16, k=64, x=A, x_ld=64, w=A, w_ld=64, bias=None, residual=None, residual_ld=0, residual_f32=0, act=0,
             alpha=1.0, out=A, out_ld=16, out_f32=0, preact=None, preact_ld=0)
    ws, ws_bytes = change.pop("ws", None), change.pop("ws_bytes", 0)
    a.update(change)
    return kb.STATUS[kb.lib.klein_op_linear(kb.KleinLinearArgs(*a.values()), ws, ws_bytes, None)]


@pytest.mark.parametrize("change,status", [
    (dict(x=None), "KLEIN_ERR_INVALID_ARG"), (dict(w=None), "KLEIN_ERR_INVALID_ARG"),
    (dict(out=None), "KLEIN_ERR_INVALID_ARG"), (dict(act=3), "KLEIN_ERR_INVALID_ARG"),
    (dict(act=-1), "KLEIN_ERR_INVALID_ARG"),
    (dict(m=0), "KLEIN_ERR_SHAPE"), (dict(n=0), "KLEIN_ERR_SHAPE"), (dict(k=0), "KLEIN_ERR_SHAPE"),
    (dict(m=-3), "KLEIN_ERR_SHAPE"), (dict(k=1 << 29, x_ld=1 << 29, w_ld=1 << 29), "KLEIN_ERR_SHAPE"),
    (dict(x_ld=56), "KLEIN_ERR_SHAPE"), (dict(w_ld=56), "KLEIN_ERR_SHAPE"), (dict(out_ld=15), "KLEIN_ERR_SHAPE"),
    (dict(x_ld=65), "KLEIN_ERR_ALIGN"), (dict(w_ld=68), "KLEIN_ERR_ALIGN"), (dict(x=A + 8), "KLEIN_ERR_ALIGN"),
    (dict(out=A + 1), "KLEIN_ERR_ALIGN"), (dict(out=A + 2, out_f32=1), "KLEIN_ERR_ALIGN"),
    (dict(bias=A + 2), "KLEIN_ERR_ALIGN"), (dict(residual=A + 64, residual_ld=8), "KLEIN_ERR_SHAPE"),
    (dict(residual=A + 2, residual_ld=16, residual_f32=1), "KLEIN_ERR_ALIGN"),
    (dict(preact=A + 64, preact_ld=15), "KLEIN_ERR_SHAPE"),
    (dict(residual=A, residual_ld=24), "KLEIN_ERR_INVALID_ARG"),                   # out itself, another pitch
    (dict(residual=A, residual_ld=16, residual_f32=1), "KLEIN_ERR_INVALID_ARG"),   # ... another type
    (dict(m=1000, n=300, out_ld=304, k=9216, x_ld=9216, w_ld=9216), "KLEIN_ERR_WORKSPACE"),
    (dict(m=1000, n=300, out_ld=304, k=9216, x_ld=9216, w_ld=9216, ws=A, ws_bytes=64), "KLEIN_ERR_WORKSPACE"),
    (dict(m=1000, n=300, out_ld=304, k=9216, x_ld=9216, w_ld=9216, ws=None, ws_bytes=1 << 40), "KLEIN_ERR_WORKSPACE"),
    (dict(m=1000, n=300, out_ld=304, k=9216, x_ld=9216, w_ld=9216, ws=A + 8, ws_bytes=1 << 40), "KLEIN_ERR_ALIGN"),
])
def test_linear_refusals(kb, change, status):
    assert linear(kb, **change) == status
    assert kb.lib.klein_last_error()


def backward(kb, **change):
    a = dict(m=8, n=16, k=64, dout=A, dout_ld=16, dout_f32=0, x=A, x_ld=64, w=A, w_ld=64, preact=None, preact_ld=0, act=0,
             alpha=1.0, dx=A, dx_ld=64, dx_f32=0, dw=A, dw_ld=64, dw_f32=0, dbias=A)
    ws, ws_bytes = change.pop("ws", A), change.pop("ws_bytes", 1 << 40)
    a.update(change)
    return kb.STATUS[kb.lib.klein_op_linear_backward(kb.KleinLinearGradArgs(*a.values()), ws, ws_bytes, None)]


@pytest.mark.parametrize("change,status", [
    (dict(dout=None), "KLEIN_ERR_INVALID_ARG"), (dict(dx=None, dw=None, dbias=None), "KLEIN_ERR_INVALID_ARG"),
    (dict(x=None), "KLEIN_ERR_INVALID_ARG"), (dict(w=None), "KLEIN_ERR_INVALID_ARG"),
    (dict(act=1), "KLEIN_ERR_INVALID_ARG"), (dict(act=7), "KLEIN_ERR_INVALID_ARG"),
    (dict(act=1, preact=A, preact_ld=8), "KLEIN_ERR_SHAPE"), (dict(act=1, preact=A + 1, preact_ld=16), "KLEIN_ERR_ALIGN"),
    (dict(m=0), "KLEIN_ERR_SHAPE"), (dict(dout_ld=8), "KLEIN_ERR_SHAPE"), (dict(dx_ld=63), "KLEIN_ERR_SHAPE"),
    (dict(dw_ld=63), "KLEIN_ERR_SHAPE"), (dict(x_ld=60), "KLEIN_ERR_ALIGN"), (dict(w=A + 2), "KLEIN_ERR_ALIGN"),
    (dict(dx=A + 2, dx_f32=1), "KLEIN_ERR_ALIGN"), (dict(dw=A + 1), "KLEIN_ERR_ALIGN"), (dict(dbias=A + 2), "KLEIN_ERR_ALIGN"),
    (dict(ws=None), "KLEIN_ERR_WORKSPACE"), (dict(ws_bytes=100), "KLEIN_ERR_WORKSPACE"), (dict(ws=A + 4), "KLEIN_ERR_ALIGN"),
])
def test_linear_backward_refusals(kb, change, status):
    assert backward(kb, **change) == status
    assert kb.lib.klein_last_error()


def attention(kb, shape=None, which="forward", ws=A, ws_bytes=1 << 40, lse=A, **views):
    s = dict(batch=2, heads=4, kv_heads=2, rows=100, n_txt=0, txt_len=None, scale=0.1)
    s.update(shape or {})

    def view(name, heads):
        v = dict(data=A, batch_stride=heads * s["rows"] * 128, head_stride=s["rows"] * 128, row_stride=128)
        change = views.get(name, {})
        if change is None:
            return None
        v.update(change)
        return ctypes.byref(kb.KleinHeads(*v.values()))

    shp = ctypes.byref(kb.KleinAttentionShape(*s.values()))
    q, out, dout, dq = (view(x, s["heads"]) for x in ("q", "out", "dout", "dq"))
    k, v, dk, dv = (view(x, s["kv_heads"]) for x in ("k", "v", "dk", "dv"))
    if which == "forward":
        rc = kb.lib.klein_op_attention_forward(shp, q, k, v, out, lse, None)
    else:
        rc = kb.lib.klein_op_attention_backward(shp, q, k, v, out, lse, dout, dq, dk, dv, ws, ws_bytes, None)
    return kb.STATUS[rc]


SHAPES = [
    (dict(batch=0), "KLEIN_ERR_SHAPE"), (dict(heads=0), "KLEIN_ERR_SHAPE"), (dict(kv_heads=0), "KLEIN_ERR_SHAPE"),
    (dict(rows=0), "KLEIN_ERR_SHAPE"), (dict(heads=5), "KLEIN_ERR_SHAPE"), (dict(n_txt=-1), "KLEIN_ERR_SHAPE"),
    (dict(n_txt=101), "KLEIN_ERR_SHAPE"), (dict(scale=0.0), "KLEIN_ERR_INVALID_ARG"),
    (dict(scale=-1.0), "KLEIN_ERR_INVALID_ARG"), (dict(scale=float("nan")), "KLEIN_ERR_INVALID_ARG"),
    (dict(scale=float("inf")), "KLEIN_ERR_INVALID_ARG"), (dict(txt_len=A + 2), "KLEIN_ERR_ALIGN"),
    (dict(batch=70000), "KLEIN_ERR_SHAPE"), (dict(heads=1 << 20, kv_heads=1 << 20), "KLEIN_ERR_SHAPE"),
]


@pytest.mark.parametrize("which", ["forward", "backward"])
@pytest.mark.parametrize("shape,status", SHAPES)
def test_attention_shape_refusals(kb, which, shape, status):
    assert attention(kb, shape, which) == status
    assert kb.lib.klein_last_error()


@pytest.mark.parametrize("which,name,change,status", [
    (which, name, change, status)
    for which, names in (("forward", "q k v out"), ("backward", "q k v out dout dq dk dv"))
    for name in names.split()
    for change, status in ((None, "KLEIN_ERR_INVALID_ARG"), (dict(data=None), "KLEIN_ERR_INVALID_ARG"),
                           (dict(data=A + 8), "KLEIN_ERR_ALIGN"), (dict(row_stride=132), "KLEIN_ERR_ALIGN"),
                           (dict(row_stride=0), "KLEIN_ERR_SHAPE"), (dict(head_stride=0), "KLEIN_ERR_SHAPE"),
                           (dict(batch_stride=-128), "KLEIN_ERR_SHAPE"), (dict(row_stride=64), "KLEIN_ERR_SHAPE"))])
def test_attention_view_refusals(kb, which, name, change, status):
    assert attention(kb, None, which, **{name: change}) == status


@pytest.mark.parametrize("change", [dict(batch_stride=128), dict(head_stride=99 * 128), dict(row_stride=136),
                                    dict(batch_stride=4 * 100 * 128 - 128)])
def test_attention_refuses_overlapping_outputs(kb, change):
    """No element of an output may have two indices; inputs may overlap themselves."""
    assert attention(kb, None, "forward", out=change) == "KLEIN_ERR_SHAPE"
    assert attention(kb, None, "backward", dq=change) == "KLEIN_ERR_SHAPE"


def test_attention_other_refusals(kb):
    assert attention(kb, None, "forward", lse=None) == "KLEIN_ERR_INVALID_ARG"
    assert attention(kb, None, "forward", lse=A + 2) == "KLEIN_ERR_ALIGN"
    assert attention(kb, None, "backward", lse=None) == "KLEIN_ERR_INVALID_ARG"
    assert attention(kb, None, "backward", ws=None) == "KLEIN_ERR_WORKSPACE"
    assert attention(kb, None, "backward", ws=A + 8) == "KLEIN_ERR_ALIGN"
    need = kb.klein_attention_backward_workspace_size(2, 4, 100, 0)
    assert attention(kb, None, "backward", ws_bytes=need - 1) == "KLEIN_ERR_WORKSPACE"
    need = kb.klein_attention_backward_workspace_size(2, 4, 100, 30)
    assert attention(kb, dict(n_txt=30, txt_len=A), "backward", ws_bytes=need - 1) == "KLEIN_ERR_WORKSPACE"


def test_outputs_at_an_inputs_address_are_refused(kb):
    """Every address apart from the pair in question."""
    def apart(names, same):
        at = {name: A * (i + 2) for i, name in enumerate(names)}
        at[same[0]] = at[same[1]]
        return at

    for same in (("out", "x"), ("out", "w"), ("out", "bias"), ("preact", "out"), ("preact", "residual"), ("preact", "x")):
        at = apart(("x", "w", "out", "bias", "preact", "residual"), same)
        assert linear(kb, residual_ld=16, preact_ld=16, **at) == "KLEIN_ERR_INVALID_ARG", same
    for same in (("dx", "x"), ("dx", "dout"), ("dw", "w"), ("dw", "dx"), ("dbias", "dw"), ("ws", "dout"), ("dx", "preact"),
                 ("dbias", "ws")):
        at = apart(("dout", "x", "w", "preact", "dx", "dw", "dbias", "ws"), same)
        assert backward(kb, preact_ld=16, act=1, **at) == "KLEIN_ERR_INVALID_ARG", same

    def views(names, same):
        return {name: dict(data=at) for name, at in apart(names, same).items()}

    for same in (("out", "q"), ("out", "k"), ("out", "v")):
        assert attention(kb, None, "forward", lse=A * 50, **views(("q", "k", "v", "out"), same)) == "KLEIN_ERR_INVALID_ARG"
    names = ("q", "k", "v", "out", "dout", "dq", "dk", "dv")
    for same in (("dq", "q"), ("dq", "dout"), ("dk", "k"), ("dv", "v"), ("dv", "dk"), ("dk", "dq"), ("dq", "out")):
        assert attention(kb, None, "backward", lse=A * 50, ws=A * 60, **views(names, same)) == "KLEIN_ERR_INVALID_ARG", same
    assert attention(kb, None, "backward", lse=A * 50, ws=A * 50, **views(names, ("q", "k"))) == "KLEIN_ERR_INVALID_ARG"


def test_workspace_sizes(kb):
    size = kb.klein_attention_backward_workspace_size
    # two floats per row of every slot of 128 rows; the text and the rows after it have their own slots
    assert size(2, 4, 100, 0) == 2 * 4 * 1 * 256 * 4
    assert size(2, 4, 100, 30) == 2 * 4 * 2 * 256 * 4
    assert size(1, 24, 66048, 512) == 24 * 516 * 256 * 4
    assert size(0, 4, 100, 0) == size(1, 1, 10, 11) == size(1, 1, 10, -1) == 0
    assert kb.klein_linear_workspace_size(0, 1, 1) == 0
    assert kb.klein_linear_workspace_size(1, 27648, 2560) == 0
    assert kb.klein_linear_workspace_size(4096, 4096, 64) == 0
    assert kb.klein_linear_workspace_size(1000, 300, 9216) > 0
    assert kb.klein_linear_backward_workspace_size(0, 1, 1) == 0
    # at least dz with its remainders
    assert kb.klein_linear_backward_workspace_size(100, 50, 70) >= 100 * 64 * 4


def test_binding_refuses_cpu_tensors(kb):
    x, w, y = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 4)
    with pytest.raises(kb.KleinError, match="CUDA"):
        kb.klein_op_linear(x, w, y)
    with pytest.raises(kb.KleinError, match="CUDA"):
        kb.klein_op_linear_backward(y, x, w, y, dw=w)
    q = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(kb.KleinError, match="CUDA"):
        kb.klein_op_attention_forward(q, q, q, q, torch.zeros(1, 1, 4))
    with pytest.raises(kb.KleinError):
        kb.klein_op_linear(x[0], w, y)
    with pytest.raises(kb.KleinError, match="activation"):
        kb.klein_op_linear(x, w, y, act="tanh")


def test_binding_takes_calls_without_the_operand_not_needed(kb):
    """They come as far as the check of the device; what is given has its shape looked at."""
    x, w, y = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16), torch.zeros(4, 6)
    for args, want in (((y, None, w, y), dict(dx=x)), ((y, x, None, y), dict(dw=w)), ((y, None, None, y), dict(dbias=y[0]))):
        with pytest.raises(kb.KleinError, match="CUDA"):
            kb.klein_op_linear_backward(*args, **want)
    for bad in (y[0], y[None]):
        with pytest.raises(kb.KleinError, match="matrix"):
            kb.klein_op_linear_backward(bad, None, w, y, dx=x)
        with pytest.raises(kb.KleinError, match="matrix"):
            kb.klein_op_linear_backward(y, None, bad, y, dx=x)
        with pytest.raises(kb.KleinError, match="matrix"):
            kb.klein_op_linear(x, bad, y)
