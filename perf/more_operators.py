"""The attention-forward, query/key norm with rotation and dropout operators: what is measured, on which sizes.

Every case names its operator ("op") and its sizes.  `run` computes a pass either in its plain form (elementary torch
operations in 32 bits, whole numbers in 64) or, where `own` is true, with the library's entry points.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
BASE = 10000.0


def listed():
    return [
        # self-attention over two 13x13 maps: a call whose latency counts
        dict(name="attn_fwd 2x169 h8 d64", op="attn", batch=2, len_q=169, len_k=169, heads_q=8, heads_kv=8, dim=64, type="bf16",
             causal=False, layout="qkv"),
        # single tokens of eight sequences over a long context, four query heads to a key/value head
        dict(name="attn_fwd 8x1 over 8192 h32/8 d128", op="attn", batch=8, len_q=1, len_k=8192, heads_q=32, heads_kv=8, dim=128,
             type="bf16", causal=True, layout="bhsd"),
        # self-attention over a batch of 26x26 maps, f16
        dict(name="attn_fwd 32x676 h8 d64 f16", op="attn", batch=32, len_q=676, len_k=676, heads_q=8, heads_kv=8, dim=64, type="f16",
             causal=False, layout="bshd"),
        # documents of ragged lengths packed into one row of tokens, causal, shared key/value heads
        dict(name="attn_fwd packed 8192 h16/4 d128", op="attn_packed", total=8192, docs=9, heads_q=16, heads_kv=4, dim=128,
             type="bf16", causal=True),
        # one long prompt
        dict(name="attn_fwd 1x8192 h32/8 d128", op="attn", batch=1, len_q=8192, len_k=8192, heads_q=32, heads_kv=8, dim=128,
             type="bf16", causal=True, layout="bshd"),
        # queries and keys of two 13x13 maps, slices of one projection's output
        dict(name="qk_fwd 2x169 h8/8 d64 bf16", op="qk_fwd", batch=2, len=169, heads_q=8, heads_k=8, dim=64, rot=64, type="bf16",
             param="bf16", interleaved=False, layout="qkv", first=0),
        # a training batch's queries and keys, heads shared by four, far positions
        dict(name="qk_fwd 4x8192 h32/8 d128 bf16", op="qk_fwd", batch=4, len=8192, heads_q=32, heads_k=8, dim=128, rot=128,
             type="bf16", param="f32", interleaved=False, layout="qkv", first=100000),
        # the small call in the backward direction
        dict(name="qk_bwd 2x169 h8/8 d64 bf16", op="qk_bwd", batch=2, len=169, heads_q=8, heads_k=8, dim=64, rot=64, type="bf16",
             param="bf16", interleaved=False, layout="qkv", first=0),
        # the training batch's gradients
        dict(name="qk_bwd 4x8192 h32/8 d128 bf16", op="qk_bwd", batch=4, len=8192, heads_q=32, heads_k=8, dim=128, rot=128,
             type="bf16", param="f32", interleaved=False, layout="qkv", first=100000),
        # dropout of the block's output over two 13x13 maps, the shortcut added
        dict(name="dropout 338x512 f32", op="dropout", rows=338, cols=512, type="f32", p=0.1, residual=True, pad=0),
        # the gradient of dropout over 16 maps of 52x52 positions, 255 channels: rows of an odd length
        dict(name="dropout 43264x255 f32", op="dropout", rows=43264, cols=255, type="f32", p=0.1, residual=False, pad=0),
        # a training batch of tokens in bf16, the shortcut added
        dict(name="dropout 65536x2048 bf16", op="dropout", rows=65536, cols=2048, type="bf16", p=0.1, residual=True, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn_packed", "qk_fwd", "qk_bwd", "dropout"])
    if op == "attn":
        dim = rng.choice([64, 128, 128, 40, 72, 96])
        group = rng.choice([1, 1, 2, 4, 8, 3])
        hkv = rng.choice([1, 2, 4, 8])
        causal = rng.random() < 0.5
        len_k = _log(rng, 1, 16384)
        how = rng.random()  # prompts, single tokens, and anything between
        len_q = len_k if how < 0.5 else 1 if how < 0.7 else _log(rng, 1, 8192)
        most = 8192 * 8192 * 25 // 2
        hkv = max(1, min(hkv, most // max(1, len_q * len_k * group)))
        if len_q * len_k * hkv * group > most:
            group = 1
            len_q = max(1, min(len_q, most // len_k))
        # keys, values and queries are read whole however few the pairs: 2^19 keys and 2^20 queries at most
        batch = max(1, min(_log(rng, 1, 64), most // (len_q * len_k * hkv * group), (1 << 19) // (len_k * hkv),
                           (1 << 20) // (len_q * hkv * group)))
        return dict(op=op, batch=batch, len_q=len_q, len_k=len_k, heads_q=hkv * group, heads_kv=hkv, dim=dim,
                    type=rng.choice(["bf16", "bf16", "f16"]), causal=causal,
                    layout="qkv" if group == 1 and len_q == len_k and rng.random() < 0.5 else rng.choice(["bshd", "bhsd"]))
    if op == "attn_packed":
        hkv = rng.choice([1, 2, 4])
        group = rng.choice([1, 2, 4])
        total = _log(rng, 64, 8192)
        return dict(op=op, total=total, docs=rng.randint(1, min(24, max(1, total // 8))), heads_q=hkv * group, heads_kv=hkv,
                    dim=rng.choice([64, 128, 80]), type=rng.choice(["bf16", "bf16", "f16"]), causal=rng.random() < 0.7)
    if op in ("qk_fwd", "qk_bwd"):
        dim = rng.choice([64, 128, 128, 40, 96, 256])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4])
        t = rng.choice(["bf16", "bf16", "f16", "f32"])
        n = _log(rng, 1, max(2, min(32768, (80_000_000 if t == "f32" else 160_000_000) // ((hq + hk) * dim))))
        batch = rng.choice([b for b in (1, 1, 2, 3, 4) if b <= n])
        return dict(op=op, batch=batch, len=n // batch, heads_q=hq, heads_k=hk, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    type=t, param=rng.choice([t, "f32"]), interleaved=rng.random() < 0.3,
                    layout=rng.choice(["qkv", "bshd", "bhsd"]), first=rng.choice([0, 0, 1000, 200000]))
    cols = _log(rng, 17, 12000)
    rows = _log(rng, 1, max(2, min(200000, 65_000_000 // cols)))
    if rng.random() < 0.5:
        cols = (cols + 15) // 16 * 16
    return dict(op=op, rows=rows, cols=cols, type=rng.choice(["f32", "bf16", "f16"]), p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                residual=rng.random() < 0.6, pad=rng.choice([0, 0, 8, 3]))


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
    e = 4 if c["type"] == "f32" else 2
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        # ten rounds of two products for four elements, then a scale and a sum
        return {"bytes": (3 if c["residual"] else 2) * n * e, "flops": 7 * n}
    if c["op"] in ("qk_fwd", "qk_bwd"):
        n = c["batch"] * c["len"] * (c["heads_q"] + c["heads_k"]) * c["dim"]
        table = 4 * c["len"] * c["rot"] + 4 * c["batch"] * c["len"]
        p = 2 * c["dim"] * (4 if c["param"] == "f32" else 2)
        if c["op"] == "qk_fwd":
            return {"bytes": 2 * n * e + table + p, "flops": 7 * n}
        return {"bytes": 3 * n * e + table + p + 8 * c["dim"], "flops": 13 * n}
    if c["op"] == "attn":
        tq, tk = c["batch"] * c["len_q"], c["batch"] * c["len_k"]
        pairs = c["batch"] * _pairs(c["len_q"], c["len_k"], c["causal"])
    else:
        tq = tk = c["total"]
        ends = _doc_ends(c["total"], c["docs"])
        pairs = sum(_pairs(b - a, b - a, c["causal"]) for a, b in zip(ends, ends[1:]))
    byt = c["dim"] * 2 * (2 * c["heads_q"] * tq + 2 * c["heads_kv"] * tk) + 4 * c["heads_q"] * tq
    return {"bytes": byt, "flops": 4 * pairs * c["dim"] * c["heads_q"]}


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


def _place(x, layout, dtype):
    """x [batch][len][heads][dim] as that view of a buffer in the given order."""
    if layout == "bhsd":
        return x.to(dtype).transpose(1, 2).contiguous().transpose(1, 2)
    return x.to(dtype).contiguous()


def _empty(shape, layout, dtype):
    if layout == "bhsd":
        return torch.empty((shape[0], shape[2], shape[1], shape[3]), device="cuda", dtype=dtype).transpose(1, 2)
    return torch.empty(shape, device="cuda", dtype=dtype)


def _prepare_qk(c, g, s):
    t, p, d, hq, hk = TYPES[c["type"]], TYPES[c["param"]], c["dim"], c["heads_q"], c["heads_k"]
    shape = (c["batch"], c["len"])
    if c["layout"] == "qkv":
        # one projection's output: queries, keys and values side by side in each token
        qkv = (_randn(g, (*shape, hq + 2 * hk, d)) * (0.5 + torch.rand(d, generator=g, device="cuda"))).to(t)
        s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    else:
        s["q"], s["k"] = (_place(_randn(g, (*shape, h, d)), c["layout"], t) for h in (hq, hk))
    s["gamma_q"], s["gamma_k"] = ((0.5 + torch.rand(d, generator=g, device="cuda")).to(p) for _ in range(2))
    # a row for every position up to the last; the sequences go on where earlier tokens ended
    at = torch.arange(c["first"] + c["len"], device="cuda", dtype=torch.float64)
    freq = BASE ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
    angle = at[:, None] * freq
    s["table"] = torch.stack([torch.cos(angle), torch.sin(angle)], -1).float()
    s["pos"] = (c["first"] + torch.arange(c["len"], device="cuda", dtype=torch.int32)).expand(*shape).contiguous()
    if c["op"] == "qk_bwd":
        lay = "bhsd" if c["layout"] == "bhsd" else "bshd"
        s["dyq"], s["dyk"] = (_place(_randn(g, (*shape, h, d), 0.05), lay, t) for h in (hq, hk))
    if own:
        import activation_backward_gb300 as cba
        lay = "bhsd" if c["layout"] == "bhsd" else "bshd"
        s["outq"], s["outk"] = (_empty((*shape, h, d), lay, t) for h in (hq, hk))
        kw = dict(rot_dim=c["rot"], interleaved=c["interleaved"], positions=s["table"].shape[0], eps=EPS,
                  param_type=cba.dtype_code(p))
        if c["op"] == "qk_fwd":
            s["desc"] = cba.make_qk_norm_rope_desc(s["q"], s["k"], yq=s["outq"], yk=s["outk"], **kw)
        else:
            s["desc"] = cba.make_qk_norm_rope_desc(s["q"], s["k"], dyq=s["dyq"], dyk=s["dyk"], dq=s["outq"], dk=s["outk"], **kw)
            s["dgamma_q"], s["dgamma_k"] = (torch.empty(d, device="cuda", dtype=torch.float32) for _ in range(2))
            s["ws"] = torch.empty(cba.cba_qk_norm_rope_workspace_bytes(s["desc"]), device="cuda", dtype=torch.uint8)
    return s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "dropout":
        t = TYPES[c["type"]]
        s["x"] = _rows_view(_randn(g, (c["rows"], c["cols"])), c["pad"], t)
        s["residual"] = _rows_view(_randn(g, (c["rows"], c["cols"])), c["pad"], t) if c["residual"] else None
        # the step's random numbers are these two and the element's index
        s["seed"] = (int(seed) * 0x9E3779B97F4A7C15 + 12345) & ((1 << 64) - 1)
        s["offset"] = (int(seed) * 7919 & 0xFFFF) << 30
        if own:
            import activation_backward_gb300 as cba
            ld = c["cols"] + c["pad"]
            s["desc"] = cba.make_dropout_desc(c["rows"], c["cols"], type=cba.dtype_code(t), p=c["p"], seed=s["seed"],
                                              offset=s["offset"], ld_x=ld, ld_residual=ld)
            s["y"] = torch.empty((c["rows"], c["cols"]), device="cuda", dtype=t)
        return s
    if c["op"] in ("qk_fwd", "qk_bwd"):
        return _prepare_qk(c, g, s)
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
    s.update(q=q, k=k, v=v, scale=1.0 / math.sqrt(d))
    if not own:
        s["ok"] = _mask(c)
        return s
    import activation_backward_gb300 as cba
    s["o"] = _empty(q.shape, "bshd" if layout == "qkv" else layout, t)
    s["lse"] = torch.empty((batch, hq, len_q), device="cuda", dtype=torch.float32)
    seqs, s["cu"] = {}, None
    if packed:
        ends = _doc_ends(c["total"], c["docs"])
        s["cu"] = torch.tensor(ends, device="cuda", dtype=torch.int32)
        most = max(b - a for a, b in zip(ends, ends[1:]))
        seqs = dict(sequences=c["docs"], max_q=most, max_k=most)
        for name in ("q", "k", "v", "o", "lse"):
            s[name] = s[name][0]
    s["desc"] = cba.make_attention_desc(s["q"], s["k"], s["v"], s["o"], causal=c["causal"], scale=s["scale"], **seqs)
    s["ws"] = torch.empty(cba.cba_attention_forward_workspace_bytes(s["desc"]), device="cuda", dtype=torch.uint8)
    return s


# ---- one pass ----

def _run_own(s):
    import activation_backward_gb300 as cba
    c = s["case"]
    if c["op"] == "dropout":
        cba.cba_dropout(s["desc"], s["x"], s["residual"], None, s["y"])
        return {"y": s["y"]}
    if c["op"] == "qk_fwd":
        cba.cba_qk_norm_rope_forward(s["desc"], s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["table"], s["pos"], s["outq"], s["outk"])
        return {"q": s["outq"], "k": s["outk"]}
    if c["op"] == "qk_bwd":
        cba.cba_qk_norm_rope_backward(s["desc"], s["q"], s["k"], s["gamma_q"], s["gamma_k"], s["table"], s["pos"], s["dyq"], s["dyk"],
                                      s["outq"], s["outk"], s["dgamma_q"], s["dgamma_k"], s["ws"])
        return {"dq": s["outq"], "dk": s["outk"], "dgamma_q": s["dgamma_q"], "dgamma_k": s["dgamma_k"]}
    cba.cba_attention_forward(s["desc"], s["q"], s["k"], s["v"], s["cu"], s["cu"], s["o"], s["lse"], s["ws"])
    return {"o": s["o"][None], "lse": s["lse"][None]} if c["op"] == "attn_packed" else {"o": s["o"], "lse": s["lse"]}


LOW = 0xFFFFFFFF


def _philox(seed, counter):
    """Four words of 32 bits for each counter (int64 tensors): Philox4x32 of 10 rounds (Salmon, Moraes, Dror and Shaw,
    2011) with the seed as its key and the counter in its low half."""
    x0, x1 = counter & LOW, (counter >> 32) & LOW
    x2 = x3 = torch.zeros_like(counter)
    k0, k1 = seed & LOW, seed >> 32
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57  # products past 2^63 wrap: their bits stay
        x0, x1, x2, x3 = ((b >> 32) & LOW) ^ x1 ^ k0, b & LOW, ((a >> 32) & LOW) ^ x3 ^ k1, a & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return torch.stack([x0, x1, x2, x3], -1)


def _rotate(x, cos, sin, rot, interleaved):
    """The first `rot` elements of x [batch][len][heads][dim] turned by the angles [batch][len][1][rot / 2]."""
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _grouped(x, heads_kv):
    """[batch][len][heads][dim] as fp32 [batch][heads_kv][heads of a group][len][dim]."""
    b, n, h, d = x.shape
    return x.float().reshape(b, n, heads_kv, h // heads_kv, d).permute(0, 2, 3, 1, 4)


def run(state):
    s = state
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        p = float(torch.tensor(c["p"], dtype=torch.float32))
        words = _philox(s["seed"], s["offset"] + torch.arange((n + 3) // 4, device="cuda", dtype=torch.int64))
        keep = (words >= round(p * 2.0 ** 32)).reshape(-1)[:n].view(c["rows"], c["cols"])
        y = torch.where(keep, s["x"].float() * (1.0 / (1.0 - p)), 0.0)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(s["x"].dtype)}
    if c["op"] in ("qk_fwd", "qk_bwd"):
        cs = s["table"][s["pos"].long()][:, :, None]
        cos, sin = cs[..., 0], cs[..., 1]
        out = {}
        for name in ("q", "k"):
            x, gamma = s[name].float(), s["gamma_" + name].float()
            r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
            n = x * r
            if c["op"] == "qk_fwd":
                out[name] = _rotate(n * gamma, cos, sin, c["rot"], c["interleaved"]).to(s[name].dtype)
                continue
            dh = _rotate(s["dy" + name].float(), cos, -sin, c["rot"], c["interleaved"])
            gr = dh * gamma
            out["d" + name] = (r * (gr - n * (gr * n).mean(-1, keepdim=True))).to(s[name].dtype)
            out["dgamma_" + name] = (dh * n).sum((0, 1, 2))
        return {n: out[n] for n in (("q", "k") if c["op"] == "qk_fwd" else ("dq", "dk", "dgamma_q", "dgamma_k"))}
    hk = c["heads_kv"]
    q, k, v = (_grouped(s[n], hk) for n in ("q", "k", "v"))
    x = torch.matmul(q, k.transpose(3, 4)) * s["scale"]
    if s["ok"] is not None:
        x = torch.where(s["ok"], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    b, _, gr, n, d = o.shape
    lse = (m + torch.log(total)).reshape(b, hk * gr, n)
    return {"o": o.permute(0, 3, 1, 2, 4).reshape(b, n, hk * gr, d).to(s["q"].dtype), "lse": lse}


# ---- the definitions in 64 bits ----

def _exact_keep(seed, first, n):
    """Which of n elements are kept with their words at least the bound, in slices; the same generator from its
    published definition, the halves of its products kept apart."""
    m0, m1, w0, w1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85

    def mul(m, x):
        lo = (m & 0xFFFF) * x                 # below 2^48
        hi = (m >> 16) * x + (lo >> 16)       # below 2^49
        return hi >> 16, ((hi & 0xFFFF) << 16) | (lo & 0xFFFF)

    for at in range(0, n, 1 << 24):
        c = first + torch.arange(at // 4, (min(n, at + (1 << 24)) + 3) // 4, device="cuda", dtype=torch.int64)
        ctr = [c % (1 << 32), torch.div(c, 1 << 32, rounding_mode="floor"), c * 0, c * 0]
        for i in range(10):
            key0, key1 = ((seed % (1 << 32)) + i * w0) % (1 << 32), ((seed >> 32) + i * w1) % (1 << 32)
            h0, l0 = mul(m0, ctr[0])
            h1, l1 = mul(m1, ctr[2])
            ctr = [h1 ^ ctr[1] ^ key0, l1, h0 ^ ctr[3] ^ key1, l0]
        yield at, torch.stack(ctr, 1).view(-1)[:min(n, at + (1 << 24)) - at]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        p = float(torch.tensor(c["p"], dtype=torch.float32).double())
        y = s["x"].double().reshape(-1) / (1.0 - p)
        for at, words in _exact_keep(s["seed"], s["offset"], n):
            y[at:at + words.numel()][words.double() * 2.0 ** -32 < p] = 0.0
        y = y.view(c["rows"], c["cols"])
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    if c["op"] in ("qk_fwd", "qk_bwd"):
        out, rot = {}, c["rot"]
        turn = torch.view_as_complex(s["table"].double())[s["pos"].long()][:, :, None]
        # the two indices of each pair
        i = torch.arange(rot // 2, device="cuda")
        first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rot // 2)

        def rotated(x, w):
            z = torch.complex(x[..., first], x[..., second]) * w
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y

        for name in ("q", "k"):
            x, gamma = s[name].double(), s["gamma_" + name].double()
            rms = (x.square().sum(-1, keepdim=True) / c["dim"] + EPS).sqrt()
            if c["op"] == "qk_fwd":
                out[name] = rotated(x / rms * gamma, turn)
                continue
            dh = rotated(s["dy" + name].double(), turn.conj())
            out["dgamma_" + name] = torch.einsum("bthd,bthd->d", dh, x / rms)
            g = dh * gamma
            out["d" + name] = g / rms - x * (torch.einsum("bthd,bthd->bth", g, x)[..., None] / (c["dim"] * rms ** 3))
        return {n: out[n] for n in (("q", "k") if c["op"] == "qk_fwd" else ("dq", "dk", "dgamma_q", "dgamma_k"))}
    ok, scale = _mask(c), s["scale"]
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    if q.dim() == 3:
        q, k, v = q[None], k[None], v[None]
    o = torch.zeros_like(q)
    lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), device="cuda", dtype=torch.float64)
    group = q.shape[2] // k.shape[2]
    for b in range(q.shape[0]):
        for h in range(q.shape[2]):
            logit = scale * (q[b, :, h] @ k[b, :, h // group].T)
            if ok is not None:
                logit = logit.masked_fill(~ok, -math.inf)
            lse[b, h] = torch.logsumexp(logit, -1)
            # exp(-inf - -inf) of a row without keys is taken as 0
            o[b, :, h] = torch.nan_to_num(torch.exp(logit - lse[b, h][:, None]), nan=0.0) @ v[b, :, h // group]
    return {"o": o, "lse": lse}
