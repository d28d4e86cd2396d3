"""Measured cases of the training operators: attention with its row statistics, attention's
backward pass, the linear layer with a fused epilogue, and the linear layer's backward pass.

Each case is one call on synthetic tensors of the shapes that adapter training and fine-tuning of
the joint block meet: 24 heads of 128, 512 text tokens and 64 x 64 image tokens, the block's
widths, the text and timestep projections, adapters of rank 16.

`own = False` computes the operators in plain torch operations in 32 bits; `own = True` makes the
library's calls. `exact` computes them in 64 bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

HEAD_DIM = 128


def listed():
    return [
        # Text stream of a stage-1 block: two prompts padded to one multiple of 80 tokens.
        {"name": "attention_text_80", "op": "attention", "batch": 2, "heads": 24, "kv_heads": 24, "n_txt": 80,
         "n_img": 0, "txt_len": "77,23", "layout": "bnhd"},
        # The joint block at 512 text tokens + a 1024 x 1024 image, the text not padded.
        {"name": "attention_joint_4608", "op": "attention", "batch": 1, "heads": 24, "kv_heads": 24, "n_txt": 512,
         "n_img": 4096, "txt_len": "", "layout": "bnhd"},
        # A training batch of three with prompts of different lengths, an odd image grid (37 x 53), grouped heads.
        {"name": "attention_ragged_2121", "op": "attention", "batch": 3, "heads": 24, "kv_heads": 8, "n_txt": 160,
         "n_img": 1961, "txt_len": "160,41,129", "layout": "bhnd"},
        {"name": "attention_backward_text_80", "op": "attention_backward", "batch": 2, "heads": 24, "kv_heads": 24,
         "n_txt": 80, "n_img": 0, "txt_len": "77,23", "layout": "bnhd"},
        {"name": "attention_backward_joint_4608", "op": "attention_backward", "batch": 1, "heads": 24,
         "kv_heads": 24, "n_txt": 512, "n_img": 4096, "txt_len": "", "layout": "bnhd"},
        {"name": "attention_backward_ragged_2121", "op": "attention_backward", "batch": 3, "heads": 24,
         "kv_heads": 8, "n_txt": 160, "n_img": 1961, "txt_len": "160,41,129", "layout": "bhnd"},
        # First layer of the timestep embedder, one token.
        {"name": "linear_embed_1", "op": "linear", "m": 1, "n": 3072, "k": 256, "act": "silu", "alpha": 1.0,
         "bias": True, "residual": "none", "out": "bf16", "save": False},
        # Second half of a rank-16 adapter over the joint sequence, added to the frozen layer's output.
        {"name": "linear_adapter_up_4608", "op": "linear", "m": 4608, "n": 9216, "k": 16, "act": "none",
         "alpha": 2.0, "bias": False, "residual": "bf16", "out": "bf16", "save": False},
        # Text projection of two 512-token prompts from the stacked encoder layers.
        {"name": "linear_text_in_1024", "op": "linear", "m": 1024, "n": 3072, "k": 20480, "act": "none",
         "alpha": 1.0, "bias": True, "residual": "none", "out": "bf16", "save": False},
        # MLP down-projection onto the fp32 residual stream, odd row count.
        {"name": "linear_mlp_down_1961", "op": "linear", "m": 1961, "n": 3072, "k": 9216, "act": "gelu",
         "alpha": 1.0, "bias": True, "residual": "f32", "out": "f32", "save": True},
        # Gradients of a rank-16 adapter's first half over the joint sequence.
        {"name": "linear_backward_adapter_down_4608", "op": "linear_backward", "m": 4608, "n": 16, "k": 3072,
         "act": "none", "alpha": 1.0, "bias": False, "dx": "bf16", "dw": "f32"},
        # Gradients of a biased MLP layer with GELU over the joint sequence.
        {"name": "linear_backward_mlp_4608", "op": "linear_backward", "m": 4608, "n": 9216, "k": 3072,
         "act": "gelu", "alpha": 1.0, "bias": True, "dx": "bf16", "dw": "bf16"},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention_backward", "linear", "linear_backward"])
    if op.startswith("attention"):
        kv_heads = rng.choice([1, 2, 3, 4, 6, 8, 12, 24])
        heads = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 6, 8) if g * kv_heads <= 24])
        n_txt = rng.choice([0, rng.randint(1, 512), 80 * rng.randint(1, 6)])
        n_img = _log_uniform(rng, 1, 4096) if n_txt == 0 or rng.random() < 0.8 else 0
        rows = n_txt + n_img
        batch = rng.randint(1, max(1, min(4, 24 * 4608 * 4608 // (heads * rows * rows))))
        padded = n_txt > 0 and rng.random() < 0.6
        lens = ",".join(str(rng.randint(1, n_txt)) for _ in range(batch)) if padded else ""
        return {"op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads, "n_txt": n_txt, "n_img": n_img,
                "txt_len": lens, "layout": rng.choice(["bnhd", "bhnd"])}
    m = _log_uniform(rng, 1, 4608)
    n = _log_uniform(rng, 1, 9216)
    most = (1024 * 3072 * 20480) // (m * n) if op == "linear" else (4608 * 9216 * 3072) // (m * n)
    k = _log_uniform(rng, 8, max(8, min(20480, most)))
    case = {"op": op, "m": m, "n": n, "k": k, "act": rng.choice(["none", "silu", "gelu"]),
            "alpha": rng.choice([1.0, 0.5, 2.0]), "bias": rng.random() < 0.5}
    if op == "linear":
        case["residual"] = rng.choice(["none", "bf16", "f32"])
        case["out"] = rng.choice(["bf16", "f32"])
        case["save"] = rng.random() < 0.5
    else:
        case["dx"] = rng.choice(["bf16", "f32"])
        case["dw"] = rng.choice(["bf16", "f32"])
    return case


# ------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _heads(g, case, heads, unit_rms):
    """bf16 [batch][heads][rows][128] values in the case's memory layout; q and k leave the
    block's QK-RMSNorm with unit RMS per head."""
    b, n = case["batch"], case["n_txt"] + case["n_img"]
    t = _randn(g, b, heads, n, HEAD_DIM) if case["layout"] == "bhnd" else _randn(g, b, n, heads, HEAD_DIM)
    if unit_rms:
        t = t / t.square().mean(-1, keepdim=True).sqrt()
    t = t.to(torch.bfloat16)
    return t if case["layout"] == "bhnd" else t.transpose(1, 2)


def _pitched(t):
    """A bf16 matrix whose rows start on 16-byte boundaries."""
    m, k = t.shape
    whole = torch.zeros(m, (k + 7) // 8 * 8, device="cuda", dtype=torch.bfloat16)
    whole[:, :k] = t
    return whole[:, :k]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"].startswith("attention"):
        b, n, h = case["batch"], case["n_txt"] + case["n_img"], case["heads"]
        lens = [int(x) for x in case["txt_len"].split(",")] if case["txt_len"] else None
        s["n_txt"] = case["n_txt"]
        s["txt_len"] = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["q"] = _heads(g, case, h, True)
        s["k"] = _heads(g, case, case["kv_heads"], True)
        s["v"] = _heads(g, case, case["kv_heads"], False)
        if case["op"] == "attention":
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(b, h, n, device="cuda")
        else:
            s["dout"] = _heads(g, case, h, False)
            s["out"], s["lse"] = _plain_attention(s)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in "qkv")
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["x"] = _pitched(_randn(g, m, k).to(torch.bfloat16))
    s["w"] = _pitched((_randn(g, n, k) / math.sqrt(k)).to(torch.bfloat16))
    bias = _randn(g, n) * 0.1 if case["bias"] else None
    if case["op"] == "linear":
        s["bias"] = bias
        s["residual"] = None if case["residual"] == "none" else _randn(g, m, n).to(_TYPES[case["residual"]])
        s["out"] = torch.empty(m, n, device="cuda", dtype=_TYPES[case["out"]])
        s["preact"] = torch.empty(m, n, device="cuda", dtype=torch.bfloat16) if case["save"] else None
        return s
    z = s["x"].float() @ s["w"].float().T
    s["preact"] = None if case["act"] == "none" else (z if bias is None else z + bias).to(torch.bfloat16)
    s["dout"] = _randn(g, m, n).to(torch.bfloat16)
    s["dx"] = torch.empty(m, k, device="cuda", dtype=_TYPES[case["dx"]])
    s["dw"] = torch.empty(n, k, device="cuda", dtype=_TYPES[case["dw"]])
    s["dbias"] = torch.empty(n, device="cuda") if case["bias"] else None
    return s


# ------------------------------------------------------------------ plain forms (32 bits)

def _valid_rows(s):
    """[batch][1][rows]: text rows below the item's length, and every image row."""
    b, n = s["q"].shape[0], s["q"].shape[2]
    row = torch.arange(n, device="cuda")[None, None, :]
    if s["txt_len"] is None:
        return torch.ones(b, 1, n, dtype=torch.bool, device="cuda")
    return (row < s["txt_len"][:, None, None]) | (row >= s["n_txt"])


def _shared(t, heads):
    """fp32 copy of a key or value tensor, each head repeated for the query heads that share it."""
    return t.float().repeat_interleave(heads // t.shape[1], dim=1)


def _plain_probabilities(s, valid):
    h = s["q"].shape[1]
    scores = (s["q"].float() @ _shared(s["k"], h).transpose(2, 3)) * (1.0 / math.sqrt(HEAD_DIM))
    scores = torch.where(valid[:, :, None, :], scores, torch.full_like(scores, -math.inf))
    m = scores.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(scores - m)
    p = torch.where(valid[:, :, :, None], p, torch.zeros_like(p))
    return p, m, p.sum(-1, keepdim=True)


def _plain_attention(s):
    valid = _valid_rows(s)
    p, m, total = _plain_probabilities(s, valid)
    out = (p @ _shared(s["v"], s["q"].shape[1])) / torch.where(total == 0, torch.ones_like(total), total)
    lse = torch.where(total == 0, torch.full_like(total, -math.inf), m + torch.log(total)).squeeze(-1)
    return torch.empty_like(s["q"]).copy_(out), lse


def _plain_attention_backward(s):
    valid = _valid_rows(s)
    h, hkv = s["q"].shape[1], s["k"].shape[1]
    p, _, total = _plain_probabilities(s, valid)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    dout = torch.where(valid[:, :, :, None], s["dout"].float(), torch.zeros_like(p[:, :, :, :1]))
    dv = p.transpose(2, 3) @ dout
    dp = dout @ _shared(s["v"], h).transpose(2, 3)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * (1.0 / math.sqrt(HEAD_DIM))
    dq = ds @ _shared(s["k"], h)
    dk = ds.transpose(2, 3) @ s["q"].float()
    dk, dv = (t.reshape(t.shape[0], hkv, h // hkv, t.shape[2], HEAD_DIM).sum(2) for t in (dk, dv))
    return tuple(torch.empty_like(s[x]).copy_(t) for x, t in (("q", dq), ("k", dk), ("v", dv)))


def _plain_act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _plain_act_grad(z, act):
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-z))
        return sig * (1.0 + z * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _plain_linear(s):
    case = s["case"]
    z = s["x"].float() @ s["w"].float().T
    if s["bias"] is not None:
        z = z + s["bias"]
    y = case["alpha"] * _plain_act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    y = y.to(s["out"].dtype)
    return (y, z.to(torch.bfloat16)) if case["save"] else (y,)


def _plain_linear_backward(s):
    case = s["case"]
    dz = case["alpha"] * s["dout"].float()
    if case["act"] != "none":
        dz = dz * _plain_act_grad(s["preact"].float(), case["act"])
    dx = (dz @ s["w"].float()).to(s["dx"].dtype)
    dw = (dz.T @ s["x"].float()).to(s["dw"].dtype)
    return (dx, dw, dz.sum(0)) if case["bias"] else (dx, dw)


# ------------------------------------------------------------------ one pass

def _run_own(s):
    import latent_flow_matching_joint_b200 as kb
    case = s["case"]
    op = case["op"]
    if op == "attention":
        kb.klein_op_attention_forward(s["q"], s["k"], s["v"], s["out"], s["lse"], n_txt=s["n_txt"],
                                      txt_len=s["txt_len"])
        return s["out"], s["lse"]
    if "ws" not in s:  # a program keeps its workspace between calls
        if op == "attention_backward":
            size = kb.klein_attention_backward_workspace_size(case["batch"], case["heads"],
                                                              case["n_txt"] + case["n_img"], case["n_txt"])
        elif op == "linear":
            size = kb.klein_linear_workspace_size(case["m"], case["n"], case["k"])
        else:
            size = kb.klein_linear_backward_workspace_size(case["m"], case["n"], case["k"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    if op == "attention_backward":
        kb.klein_op_attention_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"],
                                       s["dv"], s["ws"], n_txt=s["n_txt"], txt_len=s["txt_len"])
        return s["dq"], s["dk"], s["dv"]
    if op == "linear":
        kb.klein_op_linear(s["x"], s["w"], s["out"], s["ws"], bias=s["bias"], residual=s["residual"],
                           act=case["act"], alpha=case["alpha"], preact=s["preact"])
        return (s["out"], s["preact"]) if case["save"] else (s["out"],)
    kb.klein_op_linear_backward(s["dout"], s["x"], s["w"], s["ws"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"],
                                preact=s["preact"], act=case["act"], alpha=case["alpha"])
    return (s["dx"], s["dw"], s["dbias"]) if case["bias"] else (s["dx"], s["dw"])


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "attention":
        return _plain_attention(state)
    if op == "attention_backward":
        return _plain_attention_backward(state)
    if op == "linear":
        return _plain_linear(state)
    return _plain_linear_backward(state)


def work(case):
    if case["op"].startswith("attention"):
        b, n, h, hkv = case["batch"], case["n_txt"] + case["n_img"], case["heads"], case["kv_heads"]
        lens = [int(x) for x in case["txt_len"].split(",")] if case["txt_len"] else [case["n_txt"]] * b
        valid = [x + case["n_img"] for x in lens]
        q_bytes, kv_bytes = 2 * HEAD_DIM * h, 2 * HEAD_DIM * hkv
        pairs = h * sum(v * v for v in valid)
        if case["op"] == "attention":  # q, k, v of the rows in use; out and lse of every row
            return {"bytes": sum(valid) * (q_bytes + 2 * kv_bytes) + b * n * (q_bytes + 4 * h),
                    "flops": 4 * HEAD_DIM * pairs}
        # q, k, v, out, dout, lse of the rows in use; dq, dk, dv of every row
        return {"bytes": sum(valid) * (3 * q_bytes + 2 * kv_bytes + 4 * h) + b * n * (q_bytes + 2 * kv_bytes),
                "flops": 10 * HEAD_DIM * pairs}
    m, n, k = case["m"], case["n"], case["k"]
    size = {"none": 0, "bf16": 2, "f32": 4}
    if case["op"] == "linear":
        per = size[case["residual"]] + size[case["out"]] + (2 if case["save"] else 0)
        return {"bytes": 2 * (m * k + n * k) + m * n * per + (4 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    per = 2 + (0 if case["act"] == "none" else 2)
    return {"bytes": 2 * (m * k + n * k) + m * n * per + m * k * size[case["dx"]] + n * k * size[case["dw"]]
            + (4 * n if case["bias"] else 0), "flops": 4 * m * n * k}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _rows_in_use(s, b):
    n = s["q"].shape[2]
    if s["txt_len"] is None:
        return np.arange(n)
    length = int(s["txt_len"][b])
    return np.concatenate([np.arange(length), np.arange(s["n_txt"], n)])


def _exact_attention(s, backward):
    """Every batch item and head alone, over the rows in use only."""
    q, k, v = s["q"], s["k"], s["v"]
    batch, heads, n, d = q.shape
    group = heads // k.shape[1]
    f64 = dict(dtype=torch.float64, device="cuda")
    out = torch.zeros(batch, heads, n, d, **f64)
    lse = torch.full((batch, heads, n), -math.inf, **f64)
    dq, dk, dv = torch.zeros(q.shape, **f64), torch.zeros(k.shape, **f64), torch.zeros(v.shape, **f64)
    for b in range(batch):
        rows = torch.from_numpy(_rows_in_use(s, b)).to("cuda")
        if rows.numel() == 0:
            continue
        for h in range(heads):
            kh = h // group
            qq, kk, vv = q[b, h, rows].double(), k[b, kh, rows].double(), v[b, kh, rows].double()
            t = torch.einsum("id,jd->ij", qq, kk) / math.sqrt(d)
            norm = torch.logsumexp(t, dim=1)
            prob = torch.exp(t - norm[:, None])
            o = torch.einsum("ij,jd->id", prob, vv)
            out[b, h, rows], lse[b, h, rows] = o, norm
            if backward:
                # L = sum(dO * O): dO/dt_ij = p_ij (v_j - o_i)
                do = s["dout"][b, h, rows].double()
                grad_t = prob * (torch.einsum("id,jd->ij", do, vv) - (do * o).sum(1)[:, None]) / math.sqrt(d)
                dq[b, h, rows] = torch.einsum("ij,jd->id", grad_t, kk)
                dk[b, kh, rows] += torch.einsum("ij,id->jd", grad_t, qq)
                dv[b, kh, rows] += torch.einsum("ij,id->jd", prob, do)
    return (dq, dk, dv) if backward else (out, lse)


def _exact_act(z, act):
    """(value, derivative)"""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "silu":
        sig = torch.sigmoid(z)
        return z * sig, sig + z * sig * torch.sigmoid(-z)
    # 0.5 z (1 + tanh u) = z sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
    u2 = 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    du2 = 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z ** 2)
    sig = torch.sigmoid(u2)
    return z * sig, sig + z * du2 * sig * torch.sigmoid(-u2)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("attention"):
        return _exact_attention(s, case["op"] == "attention_backward")
    x, w = s["x"].double(), s["w"].double()
    if case["op"] == "linear":
        z = torch.einsum("mk,nk->mn", x, w)
        z = z if s["bias"] is None else z + s["bias"].double()[None, :]
        y = case["alpha"] * _exact_act(z, case["act"])[0]
        y = y if s["residual"] is None else s["residual"].double() + y
        return (y, z) if case["save"] else (y,)
    dz = s["dout"].double() * case["alpha"]
    if case["act"] != "none":
        dz = dz * _exact_act(s["preact"].double(), case["act"])[1]
    grads = (torch.einsum("mn,nk->mk", dz, w), torch.einsum("mn,mk->nk", dz, x))
    return (*grads, torch.einsum("mn->n", dz)) if case["bias"] else grads
