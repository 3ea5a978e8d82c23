"""Measured cases of the attention-side operators: rotary positions, norms of
queries and keys with the rotation in the same pass, and attention with capped
scores, a distance bias, document and prefix masks (forward, backward, and the
single-token form over a cache).

``own`` false: plain torch operations in 32 bits, rounded once at the end.
``own`` true: the calls of megatron_tensor_sharded_b200.  Layouts are the
framework's: queries [p][T][(h/p)*D], keys and values [p][T][(h_kv/p)*D].
"""

import math
import random

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# --------------------------------------------------------------------- cases
def _rope(name, T, h, hkv, p, D=128, r=128, layout="half", scaling="none", factor=1.0, far=0,
          dtype="bf16", op="rope"):
    return {"name": name, "op": op, "T": T, "h": h, "hkv": hkv, "p": p, "D": D, "r": r,
            "layout": layout, "scaling": scaling, "factor": factor, "far": far, "dtype": dtype}


def _attn(name, T, h, hkv, p, cap=0.0, slopes=False, docs=0, tail=0, prefix=False, causal=True,
          op="attn"):
    return {"name": name, "op": op, "T": T, "h": h, "hkv": hkv, "p": p, "cap": cap,
            "slopes": slopes, "docs": docs, "tail": tail, "prefix": prefix, "causal": causal}


def _decode(name, B, length, h, hkv, p, cap=0.0, slopes=False):
    return {"name": name, "op": "decode", "B": B, "length": length, "h": h, "hkv": hkv, "p": p,
            "cap": cap, "slopes": slopes}


def listed():
    return [
        # one decode step of 16 sequences at far positions of a lengthened context
        _rope("rope_step", 16, 64, 8, 8, scaling="bands", factor=8.0, far=120000),
        # a 4096-token prompt, grouped K/V heads, the second half of a chunked long prompt
        _rope("rope_prompt", 4096, 64, 8, 8, scaling="ramp", factor=4.0, far=28000),
        # one decode step with normed queries and keys
        _rope("norm_rope_step", 16, 64, 8, 8, far=3000, op="norm_rope"),
        # a training or prompt pass of 4096 tokens, as many K/V heads as query heads
        _rope("norm_rope_prompt", 4096, 32, 32, 4, op="norm_rope"),
        # the same step's backward on the grouped layout
        _rope("norm_rope_grad", 4096, 64, 8, 8, op="norm_rope_bwd"),
        # a short prompt whose first part is seen by everyone (prefix), capped scores
        _attn("attn_prefix_short", 130, 4, 2, 2, cap=30.0, docs=1, prefix=True),
        # capped scores over a 4096-token prompt
        _attn("attn_cap", 4096, 64, 8, 8, cap=50.0),
        # packed documents of uneven length with the distance bias, padding at the end
        _attn("attn_docs_bias", 4001, 32, 32, 4, slopes=True, docs=9, tail=37),
        # training: gradients of the capped attention
        _attn("attn_cap_grad", 4096, 32, 32, 4, cap=50.0, op="attn_bwd"),
        # training on packed documents, grouped heads
        _attn("attn_docs_grad", 1999, 64, 8, 8, slopes=True, docs=5, tail=19, op="attn_bwd"),
        # serving: one token each of 16 sequences, cache lengths uneven up to 8192
        _decode("decode_batch", 16, 8192, 64, 8, 8, cap=50.0),
        # serving: one token of one long sequence
        _decode("decode_long", 1, 32768, 64, 8, 8, slopes=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_HEADS = [(4, 2, 2), (12, 12, 2), (32, 32, 4), (64, 8, 8), (16, 16, 1), (24, 8, 4), (8, 1, 1)]


def draw(rng):
    op = rng.choice(["rope", "norm_rope", "norm_rope_bwd", "attn", "attn", "attn_bwd", "attn_bwd",
                     "decode", "decode"])
    h, hkv, p = rng.choice(_HEADS)
    if op == "decode":
        B = _log(rng, 1, 32)
        c = _decode("", B, _log(rng, 1, min(32768, 131072 // B)), h, hkv, p,
                    cap=rng.choice([0.0, rng.uniform(12, 60)]), slopes=rng.random() < 0.4)
    elif op.startswith("attn"):
        T = _log(rng, 1, 4096 if h <= 32 or op == "attn" else 2048)
        docs = rng.choice([0, 0, _log(rng, 1, 40)])
        causal = rng.random() < 0.8
        c = _attn("", T, h, hkv, p, cap=rng.choice([0.0, rng.uniform(12, 60)]),
                  slopes=rng.random() < 0.4, docs=docs,
                  tail=rng.randrange(0, max(1, T // 8)) if docs else 0,
                  prefix=bool(docs and causal and rng.random() < 0.5), causal=causal, op=op)
        while work(c)["flops"] > 3.4e11:      # no dearer than the largest listed one
            c["T"] = c["T"] * 4 // 5
            c["tail"] = min(c["tail"], c["T"] // 8)
    else:
        D = rng.choice([128, 128, 64, 96, 80])
        r = rng.choice([D, D, D // 2, 2 * rng.randrange(1, D // 2 + 1)])
        scaling = rng.choice(["none", "linear", "base", "bands", "ramp"])
        c = _rope("", _log(rng, 1, 4096), h, hkv, p, D=D, r=r,
                  layout=rng.choice(["half", "interleaved"]), scaling=scaling,
                  factor=1.0 if scaling == "none" else rng.uniform(2, 16),
                  far=rng.choice([0, _log(rng, 1, 1000000)]),
                  dtype=rng.choice(["bf16", "bf16", "f32"]), op=op)
    del c["name"]
    return c


# -------------------------------------------------------------------- inputs
BASE, ORIGINAL, LOW, HIGH = 500000.0, 8192, {"bands": 1.0, "ramp": 1.0}, {"bands": 4.0, "ramp": 32.0}
EPS = 1e-6


def _frequencies(c):
    """Angle per position of each pair, after the long-context scaling (host)."""
    r, f = c["r"], c["factor"]
    base = BASE * f ** (r / (r - 2)) if c["scaling"] == "base" and r > 2 else BASE
    w = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if c["scaling"] == "linear":
        return [x / f for x in w]
    if c["scaling"] == "bands":
        lo, hi, out = LOW["bands"], HIGH["bands"], []
        for x in w:
            turns = ORIGINAL * x / (2 * math.pi)
            s = min(1.0, max(0.0, (turns - lo) / (hi - lo)))
            out.append(x * s + x / f * (1 - s))
        return out
    if c["scaling"] == "ramp":
        at = lambda turns: r * math.log(ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(BASE))  # noqa: E731
        lo = max(math.floor(at(HIGH["ramp"])), 0)
        hi = min(math.ceil(at(LOW["ramp"])), r - 1)
        hi = hi if hi > lo else lo + 0.001
        g = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(r // 2)]
        return [x * (1 - a) + x / f * a for x, a in zip(w, g)]
    return w


def _amplitude(c):
    return 0.1 * math.log(c["factor"]) + 1 if c["scaling"] == "ramp" else 1.0


def _doc_offsets(c):
    """Where the packed documents begin and end: uneven, some of them empty."""
    n, end = c["docs"], c["T"] - c["tail"]
    rng = random.Random("%d %d %d" % (c["T"], n, c["tail"]))
    cuts = sorted(rng.randrange(0, end + 1) for _ in range(n - 1))
    if n > 4:
        cuts[1] = cuts[2]
        cuts.sort()
    return [0] + cuts + [end]


def _prefixes(c):
    rng = random.Random("p %d %d" % (c["T"], c["docs"]))
    off = _doc_offsets(c)
    return [rng.randrange(0, max(1, (b - a) // 2 + 1)) for a, b in zip(off, off[1:])]


def _lengths(c):
    """Keys already in each sequence's cache."""
    rng = random.Random("%d %d" % (c["B"], c["length"]))
    n = [rng.randrange(c["length"] // 2, c["length"]) for _ in range(c["B"])]
    n[0] = c["length"] - 1
    return n


def _normal(g, *shape, dtype=BF16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    p, h, hkv = c["p"], c["h"], c["hkv"]
    s = {"case": dict(c)}
    if c["op"] in ("rope", "norm_rope", "norm_rope_bwd"):
        T, D, dt = c["T"], c["D"], BF16 if c["dtype"] == "bf16" else F32
        s["Q"], s["K"] = _normal(g, p, T, h // p * D, dtype=dt), _normal(g, p, T, hkv // p * D, dtype=dt)
        if c["far"]:
            start = torch.randint(0, c["far"], (T,), generator=g, device="cuda")
        else:
            start = torch.zeros(T, dtype=torch.int64, device="cuda")
        s["pos"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        s["freq"] = torch.tensor(_frequencies(c), dtype=torch.float64, device="cuda")
        s["Qo"], s["Ko"] = torch.empty_like(s["Q"]), torch.empty_like(s["K"])
        if c["op"] != "rope":
            s["wq"] = 1 + 0.1 * _normal(g, D, dtype=F32)
            s["wk"] = 1 + 0.1 * _normal(g, D, dtype=F32)
        if c["op"] == "norm_rope_bwd":
            s["dQo"], s["dKo"] = _normal(g, *s["Q"].shape, dtype=dt), _normal(g, *s["K"].shape, dtype=dt)
            s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
        return s
    s["slopes"] = (torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device="cuda")
                   if c["slopes"] else None)
    if c["op"] == "decode":
        B, L = c["B"], c["length"]
        s["Q"] = _normal(g, p, B, h // p * 128)
        s["Kn"], s["Vn"] = _normal(g, p, B, hkv // p * 128), _normal(g, p, B, hkv // p * 128)
        s["Kc"], s["Vc"] = _normal(g, p, B, L, hkv // p * 128), _normal(g, p, B, L, hkv // p * 128)
        s["len"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
        s["O"] = torch.zeros_like(s["Q"])
        return s
    T = c["T"]
    s["Q"] = _normal(g, p, T, h // p * 128)
    s["K"], s["V"] = _normal(g, p, T, hkv // p * 128), _normal(g, p, T, hkv // p * 128)
    s["off"] = torch.tensor(_doc_offsets(c), dtype=torch.int32, device="cuda") if c["docs"] else None
    s["pre"] = torch.tensor(_prefixes(c), dtype=torch.int32, device="cuda") if c["prefix"] else None
    # the rows behind the last document keep what the caller had there
    s["O"], s["LSE"] = torch.zeros_like(s["Q"]), torch.zeros(p, h // p, T, device="cuda")
    if c["op"] == "attn_bwd":
        s["dO"] = _normal(g, *s["Q"].shape)
        r = _plain_attn(s)
        s["O"], s["LSE"] = r["O"], r["LSE"]
        s["dQ"], s["dK"], s["dV"] = (torch.zeros_like(s[x]) for x in "QKV")
    return s


# ---------------------------------------------------------------- plain form
def _pairs(x, r, layout):
    if layout == "half":
        return x[..., :r // 2], x[..., r // 2:r]
    return x[..., 0:r:2], x[..., 1:r:2]


def _join(a, b, rest, layout):
    if layout == "half":
        return torch.cat((a, b, rest), -1)
    return torch.cat((torch.stack((a, b), -1).flatten(-2), rest), -1)


def _turn(x, s, inverse=False):
    """Rotates the last dimension of x [p, T, heads, D] (32 bits)."""
    c = s["case"]
    f = s["pos"].double()[:, None] * s["freq"]                     # [T, r/2]
    cos = (_amplitude(c) * torch.cos(f)).float()[:, None, :]
    sin = (_amplitude(c) * torch.sin(f)).float()[:, None, :]
    if inverse:
        sin = -sin
    a, b = _pairs(x, c["r"], c["layout"])
    return _join(a * cos - b * sin, b * cos + a * sin, x[..., c["r"]:], c["layout"])


def _split(x, D):
    return x.float().view(x.shape[0], x.shape[1], -1, D)


def _plain_rope(s):
    D = s["case"]["D"]
    return {n: _turn(_split(s[n], D), s).to(s[n].dtype).view_as(s[n]) for n in ("Q", "K")}


def _plain_norm_rope(s):
    D = s["case"]["D"]

    def one(x, w):
        v = _split(x, D)
        v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w
        return _turn(v, s).to(x.dtype).view_as(x)

    return {"Q": one(s["Q"], s["wq"]), "K": one(s["K"], s["wk"])}


def _plain_norm_rope_bwd(s):
    D = s["case"]["D"]

    def one(x, w, dy):
        v, g = _split(x, D), _turn(_split(dy, D), s, inverse=True)
        rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
        xhat = v * rstd
        dw = (g * xhat).double().sum((0, 1, 2)).float()
        g = g * w
        return (rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))).to(x.dtype).view_as(x), dw

    dq, dwq = one(s["Q"], s["wq"], s["dQo"])
    dk, dwk = one(s["K"], s["wk"], s["dKo"])
    return {"dQ": dq, "dK": dk, "dwq": dwq, "dwk": dwk}


def _grouped(c):
    return c["p"], c["hkv"] // c["p"], c["h"] // c["hkv"]


def _rows(x, hk, g):
    """[p, T, hk*g*128] -> [p, hk, g, T, 128] in 32 bits."""
    return x.float().view(x.shape[0], x.shape[1], hk, g, 128).permute(0, 2, 3, 1, 4)


def _back(x, like):
    """[p, hk, g, T, 128] -> the layout and type of `like`."""
    return x.permute(0, 3, 1, 2, 4).reshape(like.shape).to(like.dtype)


def _visible(s):
    """[T, T]: whether query row i sees key row j."""
    c = s["case"]
    T = c["T"]
    i = torch.arange(T, device="cuda")
    vis = i[None, :] <= i[:, None] if c["causal"] else torch.ones(T, T, dtype=torch.bool, device="cuda")
    if s["off"] is not None:
        doc = (i[:, None] >= s["off"][None, 1:]).sum(1)           # = number of docs: behind the last
        inside = i < s["off"][-1]
        if s["pre"] is not None:
            d = doc.clamp(max=c["docs"] - 1)
            vis = vis | (i < s["off"][d] + s["pre"][d])[None, :]
        vis = vis & (doc[:, None] == doc[None, :]) & inside[:, None] & inside[None, :]
    return vis


def _scores(s, q, k):
    """Masked scores [p, hk, g, T, T] and the tanh (or None)."""
    c = s["case"]
    p, hk, g = _grouped(c)
    z = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(128))
    t = None
    if c["cap"]:
        t = torch.tanh(z / c["cap"])
        z = c["cap"] * t
    if c["slopes"]:
        i = torch.arange(c["T"], device="cuda", dtype=F32)
        z = z - s["slopes"].view(p, hk, g, 1, 1) * (i[:, None] - i[None, :]).abs()
    return torch.where(_visible(s), z, -math.inf), t


def _plain_attn(s):
    c = s["case"]
    p, hk, g = _grouped(c)
    q, k, v = _rows(s["Q"], hk, g), _rows(s["K"], hk, 1), _rows(s["V"], hk, 1)
    z, _ = _scores(s, q, k)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(z - m)
    l = e.sum(-1, keepdim=True)
    some = l > 0
    o = torch.where(some, torch.matmul(e, v) / l, 0.0)
    lse = torch.where(some, m + torch.log(l), 0.0)
    return {"O": _back(o, s["Q"]), "LSE": lse.reshape(p, hk * g, c["T"])}


def _plain_attn_bwd(s):
    c = s["case"]
    p, hk, g = _grouped(c)
    q, k, v = _rows(s["Q"], hk, g), _rows(s["K"], hk, 1), _rows(s["V"], hk, 1)
    do = _rows(s["dO"], hk, g)
    z, t = _scores(s, q, k)
    P = torch.exp(z - s["LSE"].view(p, hk, g, c["T"], 1))
    dv = torch.matmul(P.transpose(-1, -2), do).sum(2, keepdim=True)
    dP = torch.matmul(do, v.transpose(-1, -2))
    dz = P * (dP - (P * dP).sum(-1, keepdim=True))
    if t is not None:
        dz = dz * (1 - t * t)
    dz = dz * (1 / math.sqrt(128))
    dq = torch.matmul(dz, k)
    dk = torch.matmul(dz.transpose(-1, -2), q).sum(2, keepdim=True)
    return {"dQ": _back(dq, s["Q"]), "dK": _back(dk, s["K"]), "dV": _back(dv, s["V"])}


def _plain_decode(s):
    c = s["case"]
    p, hk, g = _grouped(c)
    B, L = c["B"], c["length"]
    b, n = torch.arange(B, device="cuda"), s["len"].long()
    s["Kc"][:, b, n] = s["Kn"]
    s["Vc"][:, b, n] = s["Vn"]
    q = s["Q"].float().view(p, B, hk, g, 128)
    k = s["Kc"].float().view(p, B, L, hk, 128).permute(0, 1, 3, 4, 2)
    v = s["Vc"].float().view(p, B, L, hk, 128).transpose(2, 3)
    z = torch.matmul(q, k) * (1 / math.sqrt(128))
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    j = torch.arange(L, device="cuda")
    if c["slopes"]:
        z = z - s["slopes"].view(p, 1, hk, g, 1) * (n.view(1, B, 1, 1, 1) - j).abs().float()
    z = torch.where(j <= n.view(1, B, 1, 1, 1), z, -math.inf)
    e = torch.exp(z - z.amax(-1, keepdim=True))
    o = torch.matmul(e, v) / e.sum(-1, keepdim=True)
    return {"O": o.reshape(p, B, -1).to(BF16), "K": s["Kc"], "V": s["Vc"]}


# ------------------------------------------------------------ the framework's
def _plan(tp, s):
    """The rotation's plan, which a program makes once when it starts."""
    if "plan" not in s:
        c = s["case"]
        sc = c["scaling"]
        s["plan"] = tp.rope_plan(rotary_dim=c["r"], layout=c["layout"], base=BASE, scaling=sc,
                                 factor=c["factor"], original_len=ORIGINAL,
                                 low=LOW.get(sc, 1.0), high=HIGH.get(sc, 4.0))
    return s["plan"]


def _space(s, n):
    """The workspace, which a program keeps."""
    if "ws" not in s:
        s["ws"] = torch.empty(max(256, n), dtype=torch.uint8, device="cuda")
    return s["ws"], n


def _run_own(s):
    import megatron_tensor_sharded_b200 as tp

    c = s["case"]
    op, p, h, hkv = c["op"], c["p"], c["h"], c["hkv"]
    if op in ("rope", "norm_rope", "norm_rope_bwd"):
        T, D, dt = c["T"], c["D"], tp.DTYPE[c["dtype"]]
        plan = _plan(tp, s)
        if op == "rope":
            tp.tp_rope(s["Q"], s["K"], s["pos"], s["Qo"], s["Ko"], T, p, h, hkv, D, plan, dt)
            return {"Q": s["Qo"], "K": s["Ko"]}
        if op == "norm_rope":
            tp.tp_qk_norm_rope(s["Q"], s["K"], s["wq"], s["wk"], s["pos"], s["Qo"], s["Ko"], T, p, h,
                               hkv, D, plan, EPS, dt)
            return {"Q": s["Qo"], "K": s["Ko"]}
        ws, n = _space(s, tp.tp_qk_norm_rope_backward_workspace_size(T, p, h, hkv, D))
        tp.tp_qk_norm_rope_backward(s["Q"], s["K"], s["wq"], s["wk"], s["pos"], s["dQo"], s["dKo"],
                                    s["Qo"], s["Ko"], s["dwq"], s["dwk"], ws, n, T, p, h, hkv, D,
                                    plan, EPS, dt)
        return {"dQ": s["Qo"], "dK": s["Ko"], "dwq": s["dwq"], "dwk": s["dwk"]}
    if op == "decode":
        B, L = c["B"], c["length"]
        score = tp.score_params(softcap=c["cap"], slopes=s["slopes"])
        ws, n = _space(s, tp.tp_attention_decode_workspace_size(B, L, p, h, hkv, 128))
        tp.tp_attention_decode(s["Q"], s["Kn"], s["Vn"], s["Kc"], s["Vc"], s["len"], s["O"], None,
                               ws, n, B, L, p, h, hkv, 128, score)
        return {"O": s["O"], "K": s["Kc"], "V": s["Vc"]}
    T, mask = c["T"], None
    if s["off"] is not None:
        n = tp.tp_attention_mask_size(T)
        mask = s.setdefault("mask", torch.empty(n, dtype=torch.uint8, device="cuda"))
        tp.tp_attention_mask(s["off"], c["docs"], s["pre"], c["causal"], mask, n, T)
    score = tp.score_params(softcap=c["cap"], slopes=s["slopes"], mask=mask, causal=c["causal"])
    if op == "attn":
        tp.tp_attention_scored(s["Q"], s["K"], s["V"], s["O"], s["LSE"], T, p, h, hkv, 128, score)
        return {"O": s["O"], "LSE": s["LSE"]}
    ws, n = _space(s, tp.tp_attention_scored_backward_workspace_size(T, p, h, hkv, 128))
    tp.tp_attention_scored_backward(s["Q"], s["K"], s["V"], s["O"], s["LSE"], s["dO"], s["dQ"],
                                    s["dK"], s["dV"], ws, n, T, p, h, hkv, 128, score)
    return {"dQ": s["dQ"], "dK": s["dK"], "dV": s["dV"]}


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _plain_rope, "norm_rope": _plain_norm_rope, "norm_rope_bwd": _plain_norm_rope_bwd,
            "attn": _plain_attn, "attn_bwd": _plain_attn_bwd,
            "decode": _plain_decode}[state["case"]["op"]](state)


# ---------------------------------------------------------------------- work
def _visible_pairs(c):
    T = c["T"]
    off = _doc_offsets(c) if c["docs"] else [0, T]
    pre = _prefixes(c) if c["prefix"] else [0] * (len(off) - 1)
    n = 0
    for a, b, q in zip(off, off[1:], pre):
        m, q = b - a, min(q, b - a)
        n += m * (m + 1) // 2 + q * (q - 1) // 2 if c["causal"] else m * m
    return n


def work(case):
    c = case
    op, h, hkv = c["op"], c["h"], c["hkv"]
    if op in ("rope", "norm_rope", "norm_rope_bwd"):
        n = c["T"] * (h + hkv) * c["D"]
        size = 2 if c["dtype"] == "bf16" else 4
        passes, flops = {"rope": (2, 3), "norm_rope": (2, 7), "norm_rope_bwd": (3, 14)}[op]
        return {"bytes": passes * size * n + 4 * c["T"], "flops": flops * n}
    if op == "decode":
        keys = sum(_lengths(c)) + c["B"]
        return {"bytes": 2 * 2 * 128 * hkv * keys + 2 * 2 * 128 * c["B"] * (h + hkv),
                "flops": 4 * 128 * h * keys}
    pairs, rows = _visible_pairs(c) * h, c["T"] - c["tail"]
    if op == "attn":
        return {"bytes": 2 * 128 * rows * 2 * (h + hkv) + 4 * rows * h, "flops": 4 * 128 * pairs}
    return {"bytes": 2 * 128 * rows * 4 * (h + hkv) + 4 * rows * h, "flops": 10 * 128 * pairs}


# --------------------------------------------------------- from the definition
def _exact_rope(c, s):
    dev = s["Q"].device
    r, D, T = c["r"], c["D"], c["T"]
    i = torch.arange(r // 2, dtype=torch.float64, device=dev)
    base = torch.tensor(BASE, dtype=torch.float64, device=dev)
    if c["scaling"] == "base" and r > 2:
        base = base * c["factor"] ** (r / (r - 2))
    w = base ** (-2 * i / r)
    if c["scaling"] == "linear":
        w = w / c["factor"]
    elif c["scaling"] == "bands":
        wave = 2 * math.pi / w
        mix = (ORIGINAL / wave - LOW["bands"]) / (HIGH["bands"] - LOW["bands"])
        mid = (1 - mix) * w / c["factor"] + mix * w
        w = torch.where(wave < ORIGINAL / HIGH["bands"], w,
                        torch.where(wave > ORIGINAL / LOW["bands"], w / c["factor"], mid))
    elif c["scaling"] == "ramp":
        def dim(turns):
            return r * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(BASE))
        lo, hi = max(math.floor(dim(HIGH["ramp"])), 0), min(math.ceil(dim(LOW["ramp"])), r - 1)
        keep = 1 - ((i - lo) / (max(hi - lo, 0.001) if hi != lo else 0.001)).clamp(0, 1)
        w = w / c["factor"] * (1 - keep) + w * keep
    a = 1.0 + 0.1 * math.log(c["factor"]) if c["scaling"] == "ramp" else 1.0
    turn = torch.polar(torch.full((T, r // 2), a, dtype=torch.float64, device=dev),
                       s["pos"].double().outer(w))[None, :, None]

    def rotate(x, back=False):
        """x [p, T, heads, D] as complex pairs times the unit circle's points."""
        head, rest = x[..., :r], x[..., r:]
        if c["layout"] == "half":
            z = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous())
        else:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous())
        z = z * (turn.conj() if back else turn)
        if c["layout"] == "half":
            y = torch.cat((z.real, z.imag), -1)
        else:
            y = torch.view_as_real(z).reshape(head.shape)
        return torch.cat((y, rest), -1)

    heads = lambda x: x.double().reshape(x.shape[0], T, -1, D)  # noqa: E731
    out = {}
    for n, w_, d, gn in (("Q", "wq", "dQo", "dwq"), ("K", "wk", "dKo", "dwk")):
        x = heads(s[n])
        if c["op"] == "rope":
            out[n] = rotate(x).reshape(s[n].shape)
            continue
        inv = (x.square().sum(-1, keepdim=True) / D + EPS) ** -0.5
        wt = s[w_].double()
        if c["op"] == "norm_rope":
            out[n] = rotate(x * inv * wt).reshape(s[n].shape)
            continue
        gy = rotate(heads(s[d]), back=True)
        out[gn] = torch.einsum("pthd,pthd->d", gy, x * inv)
        gx = gy * wt
        dot = (gx * x).sum(-1, keepdim=True)
        out["d" + n] = (gx * inv - x * inv ** 3 * dot / D).reshape(s[n].shape)
    return out


def _exact_attn(c, s):
    """Head by head: softmax over the keys that a query sees, and its derivative."""
    T, p, dev = c["T"], c["p"], s["Q"].device
    hq, hk = c["h"] // p, c["hkv"] // p
    row = torch.arange(T, device=dev)
    if c["docs"]:
        first = torch.full((T,), -1, device=dev)
        last, free = torch.full((T,), -2, device=dev), torch.zeros(T, dtype=torch.int64, device=dev)
        off, pre = _doc_offsets(c), _prefixes(c) if c["prefix"] else [0] * c["docs"]
        for a, b, q in zip(off, off[1:], pre):
            first[a:b], last[a:b], free[a:b] = a, b - 1, min(a + q, b) - 1
    else:
        first, last, free = torch.zeros_like(row), torch.full_like(row, T - 1), torch.full_like(row, -1)
    upto = torch.maximum(row, free) if c["causal"] else last
    upto = torch.where(last < 0, last, torch.minimum(upto, last))
    seen = (row[None, :] >= first[:, None]) & (row[None, :] <= upto[:, None])
    live = (last >= 0).double()[:, None]
    far = (row[:, None] - row[None, :]).abs().double()
    grad = c["op"] == "attn_bwd"
    out = ({"dQ": torch.zeros(s["Q"].shape, dtype=torch.float64, device=dev),
            "dK": torch.zeros(s["K"].shape, dtype=torch.float64, device=dev),
            "dV": torch.zeros(s["V"].shape, dtype=torch.float64, device=dev)} if grad else
           {"O": torch.zeros(s["Q"].shape, dtype=torch.float64, device=dev),
            "LSE": torch.zeros(s["LSE"].shape, dtype=torch.float64, device=dev)})
    for i in range(p):
        for j in range(hq):
            qs = slice(j * 128, j * 128 + 128)
            ks = slice(j * hk // hq * 128, j * hk // hq * 128 + 128)
            q, k, v = s["Q"][i, :, qs].double(), s["K"][i, :, ks].double(), s["V"][i, :, ks].double()
            z = q @ k.T / 128 ** 0.5
            u = torch.tanh(z / c["cap"]) if c["cap"] else None
            z = c["cap"] * u if c["cap"] else z
            if c["slopes"]:
                z = z - s["slopes"][i * hq + j].double() * far
            z = z.masked_fill(~seen, -math.inf)
            lse = torch.logsumexp(z, -1, keepdim=True)
            P = torch.where(seen, torch.exp(z - torch.where(live > 0, lse, 0.0)), 0.0)
            if not grad:
                out["O"][i, :, qs] = P @ v
                out["LSE"][i, j] = torch.where(live > 0, lse, 0.0)[:, 0]
                continue
            do = s["dO"][i, :, qs].double()
            o = P @ v
            dz = P * (do @ v.T - (do * o).sum(-1, keepdim=True)) / 128 ** 0.5
            if u is not None:
                dz = dz - dz * u * u
            out["dQ"][i, :, qs] = dz @ k
            out["dK"][i, :, ks] += dz.T @ q
            out["dV"][i, :, ks] += P.T @ do
    return out


def _exact_decode(c, s):
    p, B = c["p"], c["B"]
    hq, hk = c["h"] // p, c["hkv"] // p
    out = torch.zeros(s["Q"].shape, dtype=torch.float64, device=s["Q"].device)
    for b, n in enumerate(_lengths(c)):
        k = torch.cat((s["Kc"][:, b, :n], s["Kn"][:, b:b + 1]), 1).double().view(p, n + 1, hk, 128)
        v = torch.cat((s["Vc"][:, b, :n], s["Vn"][:, b:b + 1]), 1).double().view(p, n + 1, hk, 128)
        q = s["Q"][:, b].double().view(p, hk, hq // hk, 128)
        z = torch.einsum("phgd,pnhd->phgn", q, k) / 128 ** 0.5
        if c["cap"]:
            z = c["cap"] * torch.tanh(z / c["cap"])
        if c["slopes"]:
            back = torch.arange(n, -1, -1, device=z.device, dtype=torch.float64)
            z = z - s["slopes"].double().view(p, hk, hq // hk, 1) * back
        out[:, b] = torch.einsum("phgn,pnhd->phgd", torch.softmax(z, -1), v).reshape(p, -1)
    return {"O": out, "K": None, "V": None}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    return (_exact_attn if case["op"].startswith("attn") else _exact_rope)(case, s)
