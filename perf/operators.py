"""The layer-norm, attention-backward and Newton-Schulz operators: what is measured, on which sizes.

Every case names its operator ("op") and its sizes.  `run` computes a pass either in its plain form (elementary torch
operations in 32 bits) or, where `own` is true, with the library's entry points.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
NS_EPS = 1e-7
NS_STEPS = 5
NS_COEF = (3.4445, -4.7750, 2.0315)


def listed():
    return [
        # one 13x13 feature map's positions normalised over 512 channels: a call whose latency counts
        dict(name="ln_fwd 169x512 f32", op="ln_fwd", rows=169, cols=512, type="f32", param="f32", pad=0),
        # a training batch of tokens in bf16
        dict(name="ln_fwd 65536x2048 bf16", op="ln_fwd", rows=65536, cols=2048, type="bf16", param="bf16", pad=0),
        # the same small call in the backward direction, with the shortcut's delta added
        dict(name="ln_bwd 169x512 f32", op="ln_bwd", rows=169, cols=512, type="f32", param="f32", pad=0, residual=True),
        # 16 maps of 52x52 positions, 255 channels (a detection head): rows of an odd length
        dict(name="ln_bwd 43264x255 f32", op="ln_bwd", rows=43264, cols=255, type="f32", param="f32", pad=0, residual=False),
        # a training batch of wide tokens, bf16 activations with fp32 parameters
        dict(name="ln_bwd 32768x4096 bf16", op="ln_bwd", rows=32768, cols=4096, type="bf16", param="f32", pad=0, residual=True),
        # self-attention over two 13x13 maps
        dict(name="attn 2x169 h8 d64", op="attn", batch=2, len_q=169, len_k=169, heads_q=8, heads_kv=8, dim=64, type="bf16",
             causal=False, layout="qkv"),
        # self-attention over a batch of 26x26 maps, f16
        dict(name="attn 32x676 h8 d64 f16", op="attn", batch=32, len_q=676, len_k=676, heads_q=8, heads_kv=8, dim=64, type="f16",
             causal=False, layout="bshd"),
        # documents of ragged lengths packed into one row of tokens, causal, shared key/value heads
        dict(name="attn packed 8192 h16/4 d128", op="attn_packed", total=8192, docs=9, heads_q=16, heads_kv=4, dim=128, type="bf16",
             causal=True),
        # one long sequence
        dict(name="attn 1x8192 h32/8 d128", op="attn", batch=1, len_q=8192, len_k=8192, heads_q=32, heads_kv=8, dim=128, type="bf16",
             causal=True, layout="bshd"),
        # the weight gradient of a 5x5 convolution, 20 -> 50 channels
        dict(name="ortho 50x500 f32", op="ortho", batch=1, rows=50, cols=500, type="f32", out="bf16"),
        # the weight gradient of a 3x3 convolution, 256 -> 512 channels
        dict(name="ortho 512x2304 f32", op="ortho", batch=1, rows=512, cols=2304, type="f32", out="bf16"),
        # two projection matrices of a wide layer, taller than wide
        dict(name="ortho 2x8192x2048 bf16", op="ortho", batch=2, rows=8192, cols=2048, type="bf16", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ln_bwd", "attn", "attn", "attn_packed", "ortho", "ortho"])
    if op in ("ln_fwd", "ln_bwd"):
        cols = _log(rng, 17, 12000)
        rows = _log(rng, 1, max(2, min(200000, 100_000_000 // cols)))
        if rng.random() < 0.5:
            cols = (cols + 15) // 16 * 16
        t = rng.choice(["f32", "bf16", "f16"])
        c = dict(op=op, rows=rows, cols=cols, type=t, param=rng.choice([t, "f32"]), pad=rng.choice([0, 0, 8, 3]))
        if op == "ln_bwd":
            c["residual"] = rng.random() < 0.5
        return c
    if op == "attn":
        dim = rng.choice([64, 128, 128, 40, 72, 96])
        group = rng.choice([1, 1, 2, 4, 8])
        hkv = rng.choice([1, 2, 4, 8])
        causal = rng.random() < 0.5
        len_k = _log(rng, 8, 8192)  # with a single key every probability is 1 and dq, dk are rounding noise around 0
        len_q = len_k if rng.random() < 0.6 else _log(rng, 1, 8192)
        most = 8192 * 8192 * 32 // 2
        batch = max(1, min(_log(rng, 1, 64), most // max(1, len_q * len_k * hkv * group)))
        hkv = max(1, min(hkv, most // max(1, len_q * len_k * group)))
        return dict(op=op, batch=batch, len_q=len_q, len_k=len_k, heads_q=hkv * group, heads_kv=hkv, dim=dim,
                    type=rng.choice(["bf16", "bf16", "f16"]), causal=causal,
                    layout="qkv" if group == 1 and len_q == len_k and rng.random() < 0.5 else rng.choice(["bshd", "bhsd"]))
    if op == "attn_packed":
        hkv = rng.choice([1, 2, 4])
        group = rng.choice([1, 2, 4])
        total = _log(rng, 64, 8192)
        return dict(op=op, total=total, docs=rng.randint(1, min(24, max(1, total // 8))), heads_q=hkv * group, heads_kv=hkv,
                    dim=rng.choice([64, 128, 80]), type=rng.choice(["bf16", "bf16", "f16"]), causal=rng.random() < 0.7)
    rows, cols = _log(rng, 24, 4096), _log(rng, 24, 8192)
    if rng.random() < 0.5:
        rows, cols = (rows + 7) // 8 * 8, (cols + 7) // 8 * 8
    m, n = min(rows, cols), max(rows, cols)
    batch = max(1, min(_log(rng, 1, 16), 2 * 2048 * 2048 * 8192 // (m * m * n)))
    return dict(op=op, batch=batch, rows=rows, cols=cols, type=rng.choice(["f32", "bf16"]), out="bf16")


# ---- sizes ----

def _doc_ends(total, docs):
    """The ends of `docs` documents in `total` tokens: lengths that grow by a fixed rule, the second document empty where
    there are more than two (it lost all its tokens to a filter)."""
    share = [0 if (i == 1 and docs > 2) else 1 + (i * i * 7 + 3 * i) % 23 for i in range(docs)]
    run, ends = 0, []
    for s in share:
        run += s
        ends.append(total * run // sum(share))
    return [0] + ends


def _pairs(len_q, len_k, causal):
    """Allowed (query, key) pairs; causal: query i sees the keys j <= i + len_k - len_q."""
    if not causal:
        return len_q * len_k
    first = max(0, len_q - len_k)  # the first query that sees a key
    n_rows = len_q - first
    low = first + len_k - len_q + 1
    return n_rows * (low + len_k) // 2


def work(case):
    c = case
    if c["op"] in ("ln_fwd", "ln_bwd"):
        e, p = (4 if c[k] == "f32" else 2 for k in ("type", "param"))
        n, d = c["rows"] * c["cols"], c["cols"]
        if c["op"] == "ln_fwd":
            return {"bytes": 2 * n * e + 2 * d * p + 8 * c["rows"], "flops": 8 * n}
        return {"bytes": (4 if c["residual"] else 3) * n * e + d * (p + 8) + 8 * c["rows"], "flops": 14 * n}
    if c["op"] == "attn":
        tq, tk = c["batch"] * c["len_q"], c["batch"] * c["len_k"]
        pairs = c["batch"] * _pairs(c["len_q"], c["len_k"], c["causal"])
    elif c["op"] == "attn_packed":
        tq = tk = c["total"]
        ends = _doc_ends(c["total"], c["docs"])
        pairs = sum(_pairs(b - a, b - a, c["causal"]) for a, b in zip(ends, ends[1:]))
    else:
        m, n = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        e = 4 if c["type"] == "f32" else 2
        # X X^T and the square of its result are symmetric: half of each is enough
        return {"bytes": c["batch"] * m * n * (e + 2), "flops": c["batch"] * NS_STEPS * (3 * m * m * n + m * m * m)}
    byt = c["dim"] * 2 * (4 * c["heads_q"] * tq + 4 * c["heads_kv"] * tk) + 4 * c["heads_q"] * tq
    return {"bytes": byt, "flops": 10 * pairs * c["dim"] * c["heads_q"]}


# ---- inputs ----

def _randn(g, shape, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale + shift


def _rows_view(x, pad, dtype):
    """x [rows][cols] in a buffer whose rows are `pad` elements longer: a slice of a wider tensor."""
    if not pad:
        return x.to(dtype).contiguous()
    wide = torch.empty((x.shape[0], x.shape[1] + pad), device="cuda", dtype=dtype)
    wide[:, : x.shape[1]] = x
    return wide[:, : x.shape[1]]


def _mask(case, device="cuda"):
    """Allowed pairs, broadcast over heads: [len_q][len_k], or None where all are."""
    if case["op"] == "attn_packed":
        ends = torch.tensor(_doc_ends(case["total"], case["docs"]), device=device)
        at = torch.arange(case["total"], device=device)
        doc = torch.searchsorted(ends, at, right=True)
        ok = doc[:, None] == doc[None, :]
        return ok & (at[:, None] >= at[None, :]) if case["causal"] else ok
    if not case["causal"]:
        return None
    i = torch.arange(case["len_q"], device=device)[:, None]
    j = torch.arange(case["len_k"], device=device)[None, :]
    return j <= i + case["len_k"] - case["len_q"]


def _attn_forward(q, k, v, scale, ok):
    """o and the rows' log-sum-exp, [batch][len][heads][dim] in and out, one (batch, head) at a time."""
    o = torch.zeros(q.shape, device="cuda", dtype=q.dtype)
    lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), device="cuda", dtype=torch.float32)
    group = q.shape[2] // k.shape[2]
    for b in range(q.shape[0]):
        for h in range(k.shape[2]):
            qh = q[b, :, h * group:(h + 1) * group].float().transpose(0, 1)
            s = torch.matmul(qh, k[b, :, h].float().t()) * scale
            if ok is not None:
                s = s.masked_fill(~ok, -math.inf)
            m = torch.logsumexp(s, -1)
            lse[b, h * group:(h + 1) * group] = m
            p = torch.exp(s - torch.where(m == -math.inf, 0.0, m)[..., None])
            o[b, :, h * group:(h + 1) * group] = torch.matmul(p, v[b, :, h].float()).transpose(0, 1).to(q.dtype)
    return o, lse


def _place(x, layout, dtype):
    """x [batch][len][heads][dim] as that view of a buffer in the given order."""
    if layout == "bhsd":
        return x.to(dtype).transpose(1, 2).contiguous().transpose(1, 2)
    return x.to(dtype).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] in ("ln_fwd", "ln_bwd"):
        t, p = TYPES[c["type"]], TYPES[c["param"]]
        rows, cols = c["rows"], c["cols"]
        # channels of unlike scale around a shifted mean, as a residual stream has
        x = _randn(g, (rows, cols)) * (0.5 + torch.rand(cols, generator=g, device="cuda")) + 0.3
        s["x"] = _rows_view(x, c["pad"], t)
        s["gamma"] = (0.5 + torch.rand(cols, generator=g, device="cuda")).to(p)
        s["beta"] = _randn(g, (cols,), 0.1).to(p)
        xf = s["x"].float()
        if c["op"] == "ln_bwd":
            s["dy"] = _rows_view(_randn(g, (rows, cols), 0.1), c["pad"], t)
            s["residual"] = _rows_view(_randn(g, (rows, cols), 0.1), c["pad"], t) if c["residual"] else None
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt(xf.var(1, unbiased=False) + EPS)
        if own:
            import activation_backward_gb300 as cba
            code = {"f32": cba.CBA_F32, "f16": cba.CBA_F16, "bf16": cba.CBA_BF16}
            ld = cols + c["pad"]
            s["desc"] = cba.make_layernorm_desc(rows, cols, type=code[c["type"]], param_type=code[c["param"]], eps=EPS,
                                                ld_x=ld, ld_dy=ld, ld_residual=ld)
            s["out"] = torch.empty((rows, cols), device="cuda", dtype=t)
            if c["op"] == "ln_fwd":
                s["mean"], s["rstd"] = (torch.empty(rows, device="cuda") for _ in range(2))
            else:
                s["dgamma"], s["dbeta"] = (torch.empty(cols, device="cuda") for _ in range(2))
                s["ws"] = torch.empty(cba.cba_layernorm_workspace_bytes(s["desc"]), device="cuda", dtype=torch.uint8)
        return s
    if c["op"] == "ortho":
        rows, cols, r = c["rows"], c["cols"], max(1, min(c["rows"], c["cols"]) // 16)
        # a momentum of gradients: noise, and a part of low rank that stands out of it
        low = torch.matmul(_randn(g, (c["batch"], rows, r)), _randn(g, (c["batch"], r, cols)))
        s["G"] = (1e-3 * (_randn(g, (c["batch"], rows, cols)) + low / math.sqrt(r))).to(TYPES[c["type"]]).contiguous()
        if own:
            import activation_backward_gb300 as cba
            code = {"f32": cba.CBA_F32, "f16": cba.CBA_F16, "bf16": cba.CBA_BF16}
            s["desc"] = cba.make_orthogonalize_desc(c["batch"], rows, cols, in_type=code[c["type"]], out_type=code[c["out"]],
                                                    steps=NS_STEPS, coefficients=NS_COEF, eps=NS_EPS)
            s["out"] = torch.empty((c["batch"], rows, cols), device="cuda", dtype=TYPES[c["out"]])
            s["ws"] = torch.empty(cba.cba_orthogonalize_workspace_bytes(s["desc"]), device="cuda", dtype=torch.uint8)
        return s
    t, hq, hk, d = TYPES[c["type"]], c["heads_q"], c["heads_kv"], c["dim"]
    packed = c["op"] == "attn_packed"
    batch, len_q, len_k = (1, c["total"], c["total"]) if packed else (c["batch"], c["len_q"], c["len_k"])
    layout = "bshd" if packed else c["layout"]
    if layout == "qkv":
        # one projection's output: the three side by side in each token
        qkv = _randn(g, (batch, len_q, 3, hq, d)).to(t)
        q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    else:
        q = _place(_randn(g, (batch, len_q, hq, d)), layout, t)
        k, v = (_place(_randn(g, (batch, len_k, hk, d)), layout, t) for _ in range(2))
    s["scale"] = 1.0 / math.sqrt(d)
    s["ok"] = _mask(c)
    o, s["lse"] = _attn_forward(q, k, v, s["scale"], s["ok"])
    o = _place(o, layout, t)
    do = _place(_randn(g, (batch, len_q, hq, d), 0.02), layout, t)
    s.update(q=q, k=k, v=v, o=o, do=do)
    if own:
        import activation_backward_gb300 as cba
        s["ok"] = None
        outs = [torch.empty(x.shape, device="cuda", dtype=t) for x in (q, k, v)]
        seqs = {}
        s["cu"] = None
        if packed:
            ends = _doc_ends(c["total"], c["docs"])
            s["cu"] = torch.tensor(ends, device="cuda", dtype=torch.int32)
            most = max(b - a for a, b in zip(ends, ends[1:]))
            seqs = dict(sequences=c["docs"], max_q=most, max_k=most)
            for name in ("q", "k", "v", "o", "do"):
                s[name] = s[name][0]
            outs = [x[0] for x in outs]
            s["lse"] = s["lse"][0]
        s["dq"], s["dk"], s["dv"] = outs
        s["desc"] = cba.make_attention_desc(s["q"], s["k"], s["v"], s["o"], s["do"], *outs, causal=c["causal"], scale=s["scale"], **seqs)
        s["ws"] = torch.empty(cba.cba_attention_workspace_bytes(s["desc"]), device="cuda", dtype=torch.uint8)
    return s


# ---- one pass ----

def _run_own(s):
    import activation_backward_gb300 as cba
    c = s["case"]
    if c["op"] == "ln_fwd":
        cba.cba_layernorm_forward(s["desc"], s["x"], s["gamma"], s["beta"], s["out"], s["mean"], s["rstd"])
        return {"y": s["out"], "mean": s["mean"], "rstd": s["rstd"]}
    if c["op"] == "ln_bwd":
        cba.cba_layernorm_backward(s["desc"], s["x"], s["dy"], s["gamma"], s["mean"], s["rstd"], s["residual"], s["out"], s["dgamma"],
                                   s["dbeta"], s["ws"])
        return {"dx": s["out"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if c["op"] == "ortho":
        cba.cba_orthogonalize(s["desc"], s["G"], s["out"], s["ws"])
        return {"O": s["out"]}
    cba.cba_attention_backward(s["desc"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["cu"], s["cu"], s["dq"], s["dk"], s["dv"],
                               s["ws"])
    outs = {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}
    return {n: x[None] for n, x in outs.items()} if c["op"] == "attn_packed" else outs


def _ns_step(x):
    a, b, c = NS_COEF
    p = torch.matmul(x, x.transpose(1, 2))
    return a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)


def _grouped(x, heads_kv):
    """[batch][len][heads][dim] as fp32 [batch][heads_kv][heads of a group][len][dim]."""
    b, n, h, d = x.shape
    return x.float().reshape(b, n, heads_kv, h // heads_kv, d).permute(0, 2, 3, 1, 4)


def _ungrouped(x, dtype):
    b, hk, gr, n, d = x.shape
    return x.permute(0, 3, 1, 2, 4).reshape(b, n, hk * gr, d).to(dtype)


def run(state):
    s = state
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + EPS)
        y = xc * rstd[:, None] * s["gamma"].float() + s["beta"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if c["op"] == "ln_bwd":
        h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        dy = s["dy"].float()
        gr = dy * s["gamma"].float()
        dx = s["rstd"][:, None] * (gr - gr.mean(1, keepdim=True) - h * (gr * h).mean(1, keepdim=True))
        if s["residual"] is not None:
            dx = dx + s["residual"].float()
        return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * h).sum(0), "dbeta": dy.sum(0)}
    if c["op"] == "ortho":
        x = s["G"].float()
        if c["rows"] > c["cols"]:
            x = x.transpose(1, 2)
        x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + NS_EPS)
        x = _ns_step(_ns_step(_ns_step(_ns_step(_ns_step(x)))))
        if c["rows"] > c["cols"]:
            x = x.transpose(1, 2)
        return {"O": x.to(TYPES[c["out"]])}
    hk, t = c["heads_kv"], s["q"].dtype
    q, o, do = (_grouped(s[n], hk) for n in ("q", "o", "do"))
    k, v = (_grouped(s[n], hk) for n in ("k", "v"))
    lse = s["lse"].reshape(s["lse"].shape[0], hk, -1, s["lse"].shape[2], 1)
    p = torch.exp(torch.matmul(q, k.transpose(3, 4)) * s["scale"] - lse)
    if s["ok"] is not None:
        p = torch.where(s["ok"], p, 0.0)
    dv = torch.matmul(p.transpose(3, 4), do).sum(2, keepdim=True)
    ds = p * (torch.matmul(do, v.transpose(3, 4)) - (do * o).sum(-1, keepdim=True))
    dq = torch.matmul(ds, k) * s["scale"]
    dk = torch.matmul(ds.transpose(3, 4), q).sum(2, keepdim=True) * s["scale"]
    return {"dq": _ungrouped(dq, t), "dk": _ungrouped(dk, t), "dv": _ungrouped(dv, t)}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "ln_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + EPS).pow(-0.5)
        y = torch.addcmul(s["beta"].double(), (x - mean[:, None]) * rstd[:, None], s["gamma"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if c["op"] == "ln_bwd":
        x, dy, gamma = s["x"].double(), s["dy"].double(), s["gamma"].double()
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
        h = (x - mean).mul_(rstd)
        n = x.shape[1]
        m1 = torch.mv(dy, gamma)[:, None] / n
        m2 = torch.einsum("rc,rc,c->r", dy, h, gamma)[:, None] / n
        dx = (dy * gamma - m1 - h * m2) * rstd
        if s["residual"] is not None:
            dx += s["residual"].double()
        return {"dx": dx, "dgamma": torch.einsum("rc,rc->c", dy, h), "dbeta": dy.sum(0)}
    if c["op"] == "ortho":
        a, b, cc = NS_COEF
        outs = []
        for G in s["G"].double():
            X = G / (G.norm() + NS_EPS)
            left = X.shape[0] <= X.shape[1]
            for _ in range(NS_STEPS):
                # the same polynomial from either side: (a I + b S + c S^2) X with S = X X^T, or X (...) with S = X^T X
                S = X @ X.T if left else X.T @ X
                poly = a * torch.eye(S.shape[0], device="cuda", dtype=S.dtype) + b * S + cc * (S @ S)
                X = poly @ X if left else X @ poly
            outs.append(X)
        return {"O": torch.stack(outs)}
    q, k, v, o, do = (s[n].double() for n in ("q", "k", "v", "o", "do"))
    lse = s["lse"].reshape(q.shape[0], q.shape[2], -1).double()
    ok, scale = _mask(c), s["scale"]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    group = q.shape[2] // k.shape[2]
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            j = h // group
            logit = scale * (q[b, :, h] @ k[b, :, j].T)
            if ok is not None:
                logit = logit.masked_fill(~ok, -math.inf)
            # exp(-inf - -inf) of a row without keys is taken as 0
            P = torch.nan_to_num(torch.exp(logit - lse[b, h][:, None]), nan=0.0)
            dv[b, :, j] += P.T @ do[b, :, h]
            dS = P * (do[b, :, h] @ v[b, :, j].T - torch.einsum("id,id->i", do[b, :, h], o[b, :, h])[:, None]) * scale
            dq[b, :, h] = dS @ k[b, :, j]
            dk[b, :, j] += dS.T @ q[b, :, h]
    return {"dq": dq, "dk": dk, "dv": dv}
