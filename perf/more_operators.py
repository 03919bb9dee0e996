"""Cases of a training step's operators: the norms around a block's residual sum, the router's balance
loss and the global gradient norm.

`own` False: the operators in elementary torch operations, 32 bits throughout, each output rounded once.
`own` True: the library's calls. `exact` gives the same results from the definitions in 64 bits.

A case is a dict of plain values; "op" names the operator and direction:
  rn         h, z, statistics                   h = a x + c gate * post(u), z = pre(h): forward
  rn_bwd     dx, du, weights' gradients         its backward pass, with the reduced gradients
  bal        loss, counts, lse                  balance and z loss of a router, per-expert counts
  bal_train  the same and dlogits               and the gradient of the logits, that of the gates in it
  norm       norm, scale                        global norm of a list of gradients, factor that clips it
  clip       norm, scale, gradients             the same, and the gradients clipped in place
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS, RES, BRANCH = 1e-5, 0.875, 0.5       # of the norms; factors of the residual stream and of the branch
BAL, Z = 0.01, 0.001                      # weights of the two losses
MAX_NORM, NORM_EPS = 1.0, 1e-6
ALIGN = 128                               # values: start of each gradient in its flat buffer


def listed():
    return [
        # around a block in a decode step of a few requests
        {"name": "norms decode", "op": "rn", "rows": 5, "d": 4096, "x": "bf16", "w": "bf16", "post": "rms", "pre": "rms",
         "gate": 5},
        # the same for a long prompt
        {"name": "norms prompt", "op": "rn", "rows": 16384, "d": 4096, "x": "bf16", "w": "bf16", "post": "rms",
         "pre": "rms", "gate": 16384},
        # backward pass of a training micro-batch, 32-bit weights beside 16-bit activations
        {"name": "norms train", "op": "rn_bwd", "rows": 16384, "d": 2048, "x": "bf16", "w": "f32", "post": "layer",
         "pre": "layer", "gate": 16384},
        # backward pass with a gate for each sample (a modulated block), odd width and ragged groups
        {"name": "norms train groups odd", "op": "rn_bwd", "rows": 3001, "d": 1411, "x": "f16", "w": "f16", "post": "rms",
         "pre": "rms", "gate": 250},
        # a router's load and losses, watched on one batch of a layer of eight experts
        {"name": "balance watch", "op": "bal", "T": 4096, "E": 8, "topk": 2, "seqs": 1, "mask": False, "drop": False},
        # a small ragged batch of packed sequences, with padding and dropped pairs
        {"name": "balance small ragged", "op": "bal_train", "T": 509, "E": 64, "topk": 6, "seqs": 3, "mask": True,
         "drop": True},
        # a training micro-batch through a fine-grained layer
        {"name": "balance train", "op": "bal_train", "T": 16384, "E": 64, "topk": 6, "seqs": 1, "mask": False,
         "drop": False},
        # many packed sequences through the widest router
        {"name": "balance sequences", "op": "bal_train", "T": 131072, "E": 256, "topk": 8, "seqs": 67, "mask": True,
         "drop": False},
        # the small tensors of a model (norms, biases, a router)
        {"name": "gradient norm small", "op": "norm", "count": 67, "most": 20011, "wide": 0.5},
        # the three matrices of eight experts
        {"name": "gradient norm", "op": "norm", "count": 24, "most": 11534336, "wide": 0.0},
        # the same gradients clipped in place
        {"name": "gradient clip", "op": "clip", "count": 24, "most": 11534336, "wide": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rn", "rn", "rn_bwd", "rn_bwd", "rn_bwd", "bal", "bal_train", "bal_train", "norm", "clip"])
    if op in ("rn", "rn_bwd"):
        d = 8 * _log(rng, 16, 1024) if rng.random() < 0.6 else _log(rng, 128, 8192)
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        rows = _log(rng, 1, min(32768, 1.6e7 / d))
        return {"op": op, "rows": rows, "d": d, "x": x, "w": rng.choice([x, "f32"]),
                "post": rng.choice(["none", "rms", "layer"]), "pre": rng.choice(["none", "rms", "layer"]),
                "gate": rng.choice([0, rows, _log(rng, 1, rows)])}
    if op in ("bal", "bal_train"):
        E = rng.choice([8, 16, 64, 128, 256, _log(rng, 4, 256)])
        T = _log(rng, 1, min(131072, 3.3e7 / E))
        return {"op": op, "T": T, "E": E, "topk": rng.randint(1, min(E, 8)), "seqs": rng.choice([1, 1, _log(rng, 1, 300)]),
                "mask": rng.random() < 0.5, "drop": rng.random() < 0.3}
    count = _log(rng, 1, 500)
    return {"op": op, "count": count, "most": _log(rng, 100, 7e7 / (1 + 0.52 * (count - 1))), "wide": rng.choice([0.0, 0.3, 1.0])}


# ---- inputs -------------------------------------------------------------------------------------

def _sizes(c):
    """Values of a list's tensors: the largest, and odd fractions of it."""
    return [c["most"] if i == 0 else max(1, c["most"] * ((i * 37) % 64 + 1) // 64 - i % 3) for i in range(c["count"])]


def _places(c):
    """(32 bits?, start, values) of each gradient in the flat buffer of its type, and the two lengths."""
    at, out = [0, 0], []
    for i, n in enumerate(_sizes(c)):
        k = int((i * 0.618) % 1.0 < c["wide"])
        out.append((k, at[k], n))
        at[k] += -(-n // ALIGN) * ALIGN
    return out, at


def prepare(case, seed):
    c, gen, f32 = case, torch.Generator(device="cuda").manual_seed(seed), torch.float32

    def normal(shape, dtype=f32, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    s = {"case": c}
    if c["op"] in ("rn", "rn_bwd"):
        r, d, xt, wt = c["rows"], c["d"], DT[c["x"]], DT[c["w"]]
        s["u"] = normal((r, d), xt, 0.7, 0.05)                     # what the block put out
        s["post_w"] = normal((d,), wt, 0.1, 1.0) if c["post"] != "none" else None
        s["post_b"] = normal((d,), wt, 0.1) if c["post"] == "layer" else None
        s["pre_w"] = normal((d,), wt, 0.1, 1.0) if c["pre"] != "none" else None
        s["pre_b"] = normal((d,), wt, 0.1) if c["pre"] == "layer" else None
        s["gate"] = normal((-(-r // c["gate"]), d), wt, 0.3, 0.8) if c["gate"] else None
        x = normal((r, d), xt, 1.5, 0.25)                          # a residual stream that is off centre
        if c["op"] == "rn":
            s["x"] = x
        else:                                                      # what the forward pass kept
            s["h"] = x
            s["post_stats"], s["pre_stats"] = (_stats(t.float(), c[k]) if c[k] != "none" else None
                                               for t, k in ((s["u"], "post"), (s["h"], "pre")))
            s["dz"] = normal((r, d), xt, 0.1) if c["pre"] != "none" else None
            s["dh"] = normal((r, d), xt, 0.1)
        if own:  # what a program keeps: the outputs' buffers and the workspace
            import tile_level_copy_gb300 as tlc
            kind = {"none": tlc.MOE_NORM_NONE, "rms": tlc.MOE_NORM_RMS, "layer": tlc.MOE_NORM_LAYER}
            s["cfg"] = tlc.ResidualNormConfig(rows=r, d=d, dtype=xt, wdtype=wt, post=kind[c["post"]], pre=kind[c["pre"]],
                                              gate_rows=c["gate"], eps=EPS, residual_scale=RES, branch_scale=BRANCH)
            s["out"] = [torch.empty_like(s["u"]) for _ in range(2)]
            if c["op"] == "rn":
                s["kept"] = [torch.empty(r, 2, device="cuda") if c[k] != "none" else None for k in ("post", "pre")]
            else:
                s["ws"] = tlc.ResidualNormWorkspace(s["cfg"])
                s["grads"] = [None if s[n] is None else torch.empty_like(s[n])
                              for n in ("post_w", "post_b", "gate", "pre_w", "pre_b")]
    elif c["op"] in ("bal", "bal_train"):
        T, E, k, S = c["T"], c["E"], c["topk"], c["seqs"]
        lean = -2.4 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=f32)) / math.log(E + 1)  # a load that leans
        s["logits"] = normal((T, E)) + lean
        top, idx = torch.topk(s["logits"], k, dim=1)
        if c["drop"]:                                              # pairs beyond an expert's capacity
            idx = torch.where(torch.rand((T, k), generator=gen, device="cuda") < 0.03, -1, idx)
        s["idx"], s["gates"] = idx.to(torch.int32), torch.softmax(top, 1)
        s["mask"] = (torch.rand(T, generator=gen, device="cuda") > 0.05).to(torch.uint8) if c["mask"] else None
        s["offsets"] = None
        if S > 1:                                                  # ragged sequences, padding behind the last
            cut = torch.rand(S, generator=gen, device="cuda").sort().values
            s["offsets"] = torch.cat([torch.zeros(1, device="cuda"), (cut * T).floor()]).to(torch.int32)
        if c["op"] == "bal_train":
            s["dgates"], s["dloss"] = normal((T, k), std=1e-3), torch.full((1,), 0.5, device="cuda")
        if own:
            import tile_level_copy_gb300 as tlc
            s["cfg"] = tlc.BalanceConfig(T=T, E=E, topk=k, seqs=S, balance=BAL, z=Z)
            s["ws"], s["saved"] = tlc.BalanceWorkspace(s["cfg"]), None
            s["out"] = [torch.empty(3, device="cuda"), torch.empty(S, E, dtype=torch.int32, device="cuda"),
                        torch.empty(T, device="cuda")]
            if c["op"] == "bal_train":
                s["saved"], s["dlogits"] = tlc.balance_saved(s["cfg"]), torch.empty_like(s["logits"])
    else:
        places, (n16, n32) = _places(c)
        pad = [torch.zeros(n, dtype=torch.bool, device="cuda") for n in (n16, n32)]
        for k, o, n in places:
            pad[k][o:o + n] = True
        s["flat"] = []
        for p, t in zip(pad, (torch.bfloat16, f32)):               # gradients of layers of unlike sizes
            far = torch.exp(normal(((p.numel() + ALIGN - 1) // ALIGN, 1)))
            g = normal((far.numel(), ALIGN), std=1e-3).mul_(far).reshape(-1)[:p.numel()]
            s["flat"].append(torch.where(p, g, 0).to(t))
        if own:
            import tile_level_copy_gb300 as tlc
            s["cfg"] = tlc.GradNormConfig(max_norm=MAX_NORM, eps=NORM_EPS)
            s["list"] = tlc.GradList([s["flat"][k][o:o + n] for k, o, n in places])
            s["ws"], s["out"] = tlc.GradNormWorkspace(), torch.empty(2, device="cuda")
    return s


# ---- one pass -----------------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if op in ("rn", "rn_bwd"):
        return _own_rn(s) if own else _plain_rn(s) if op == "rn" else _plain_rn_bwd(s)
    if op in ("bal", "bal_train"):
        return _own_bal(s) if own else _plain_bal(s)
    return _own_norm(s) if own else _plain_norm(s)


WEIGHTS = ("post_w", "post_b", "gate", "pre_w", "pre_b")


def _own_rn(s):
    import tile_level_copy_gb300 as tlc
    c, out = s["case"], s["out"]
    if c["op"] == "rn":
        z = None if c["pre"] == "none" else out[1]
        tlc.residual_norm_forward(s["cfg"], s["x"], s["u"], s["post_w"], s["post_b"], s["gate"], s["pre_w"], s["pre_b"],
                                  out[0], z, *s["kept"])
        return {"h": out[0], "z": z, "post_stats": s["kept"][0], "pre_stats": s["kept"][1]}
    tlc.residual_norm_backward(s["cfg"], s["dz"], s["dh"], s["u"], s["h"], s["post_w"], s["post_b"], s["gate"], s["pre_w"],
                               s["post_stats"], s["pre_stats"], *out, *s["grads"], s["ws"])
    return {"dx": out[0], "du": out[1], **dict(zip(WEIGHTS, s["grads"]))}


def _stats(x, kind):
    """Mean (0 without centring) and 1 / sqrt(mean square + eps) of each row."""
    mean = x.mean(1) if kind == "layer" else torch.zeros_like(x[:, 0])
    y = x - mean[:, None]
    return torch.stack([mean, 1 / torch.sqrt((y * y).mean(1) + EPS)], 1)


def _num(t):
    return None if t is None else t.float()


def _rows_of(gate, rows, per):
    """The gate of every row: consecutive rows share one."""
    return 1.0 if gate is None else gate if len(gate) == 1 else gate[torch.arange(rows, device=gate.device) // per]


def _plain_rn(s):
    c, xt = s["case"], s["x"].dtype
    x, u, w, b, gate, pw, pb = (_num(s[n]) for n in ("x", "u", "post_w", "post_b", "gate", "pre_w", "pre_b"))
    v, post, pre, z = u, None, None, None
    if w is not None:
        post = _stats(u, c["post"])
        v = (u - post[:, :1]) * post[:, 1:] * w
        v = v if b is None else v + b
    h = (RES * x + BRANCH * (_rows_of(gate, c["rows"], c["gate"]) * v)).to(xt)
    if pw is not None:                                             # the norm of h as the next block's pass finds it
        y = h.float()
        pre = _stats(y, c["pre"])
        z = (y - pre[:, :1]) * pre[:, 1:] * pw
        z = (z if pb is None else z + pb).to(xt)
    return {"h": h, "z": z, "post_stats": post, "pre_stats": pre}


def _plain_rn_bwd(s):
    c, xt = s["case"], s["u"].dtype
    u, h, dz, dh, w, b, gate, pw = (_num(s[n]) for n in ("u", "h", "dz", "dh", "post_w", "post_b", "gate", "pre_w"))
    out = dict.fromkeys(WEIGHTS)

    def back(dy, x, stats, w, kind):
        """Gradient at a norm's input; at its weight and bias, row by row."""
        n = (x - stats[:, :1]) * stats[:, 1:]
        g = dy * w
        d = g - n * (g * n).mean(1, keepdim=True)
        return (d - g.mean(1, keepdim=True) if kind == "layer" else d) * stats[:, 1:], dy * n, n

    if pw is not None:
        d, dw, _ = back(dz, h, s["pre_stats"], pw, c["pre"])
        dh = dh + d
        out["pre_w"], out["pre_b"] = dw.sum(0), dz.sum(0) if c["pre"] == "layer" else None
    e = BRANCH * dh
    dv = e * _rows_of(gate, c["rows"], c["gate"])
    v = u
    du = dv
    if w is not None:
        du, dw, n = back(dv, u, s["post_stats"], w, c["post"])
        v = n * w if b is None else n * w + b
        out["post_w"], out["post_b"] = dw.sum(0), None if b is None else dv.sum(0)
    if gate is not None:
        ev, per = e * v, c["gate"]
        if len(gate) > 1:                                          # rows of a group, the last one filled up
            ev = torch.nn.functional.pad(ev, (0, 0, 0, len(gate) * per - len(ev)))
        out["gate"] = ev.view(len(gate), -1, ev.shape[1]).sum(1)
    wt = DT[c["w"]]
    return {"dx": (RES * dh).to(xt), "du": du.to(xt), **{n: None if t is None else t.to(wt) for n, t in out.items()}}


def _own_bal(s):
    import tile_level_copy_gb300 as tlc
    loss, counts, lse = s["out"]
    tlc.balance_forward(s["cfg"], s["logits"], s["idx"], loss, counts, lse, s["ws"], offsets=s["offsets"], mask=s["mask"],
                        saved=s["saved"])
    if "dgates" not in s:
        return {"loss": loss, "counts": counts, "lse": lse}
    tlc.balance_backward(s["cfg"], s["logits"], s["idx"], s["saved"], s["dlogits"], offsets=s["offsets"],
                         mask=s["mask"], gates=s["gates"], dgates=s["dgates"], dloss=s["dloss"])
    return {"loss": loss, "counts": counts, "lse": lse, "dlogits": s["dlogits"]}


def _sequences(s):
    """Each token's sequence (the count of sequences for padding) and whether it counts."""
    c, T = s["case"], s["case"]["T"]
    at = torch.arange(T, device="cuda")
    seq = torch.zeros_like(at)
    if s["offsets"] is not None:
        seq = torch.searchsorted(s["offsets"].long(), at, right=True) - 1
    ok = seq < c["seqs"]
    return seq, ok if s["mask"] is None else ok & (s["mask"] != 0)


def _plain_bal(s):
    c, l = s["case"], s["logits"]
    E, k, S = c["E"], c["topk"], c["seqs"]
    seq, ok = _sequences(s)
    top = l.amax(1, keepdim=True)
    q = torch.exp(l - top)
    total = q.sum(1, keepdim=True)
    lse, p = (torch.log(total) + top)[:, 0], q / total
    idx = s["idx"].long()
    here = ok[:, None] & (idx >= 0) & (idx < E)
    flat = torch.where(here, seq[:, None] * E + idx, S * E)
    counts = torch.zeros(S * E + 1, dtype=torch.int64, device=l.device).index_add_(0, flat.reshape(-1), torch.ones_like(flat).reshape(-1))
    counts = counts[:-1].view(S, E)
    home = torch.where(ok, seq, S)
    n = torch.zeros(S + 1, device=l.device).index_add_(0, home, torch.ones_like(lse))[:-1]
    ps = torch.where(ok[:, None], p, 0).sum(0, keepdim=True) if S == 1 else \
        torch.zeros(S + 1, E, device=l.device).index_add_(0, home, p)[:-1]
    some = n.clamp(min=1)
    full, tokens = (n > 0).sum().clamp(min=1), n.sum().clamp(min=1)
    bal = ((counts * ps).sum(1) * E / (k * some * some)).sum() / full
    z = torch.where(ok, lse * lse, 0).sum() / tokens
    out = {"loss": torch.stack([BAL * bal + Z * z, bal, z]), "counts": counts.to(torch.int32), "lse": lse}
    if "dgates" not in s:
        return out
    slope = torch.cat([counts * (E / (k * some * some * full))[:, None], torch.zeros(1, E, device=l.device)])[home]
    dl = p * (BAL * (slope - (p * slope).sum(1, keepdim=True)) + (2 * Z / tokens) * lse[:, None]) * s["dloss"]
    g, dg = s["gates"], s["dgates"]
    own_part = g * (dg - (g * dg).sum(1, keepdim=True))
    dl = dl.scatter_add(1, torch.where(here, idx, 0), torch.where(here, own_part, 0))
    return {**out, "dlogits": torch.where(ok[:, None], dl, 0)}


def _own_norm(s):
    import tile_level_copy_gb300 as tlc
    tlc.grad_norm(s["cfg"], s["list"], s["out"], s["ws"])
    if s["case"]["op"] == "norm":
        return {"norm": s["out"]}
    tlc.grad_clip(s["list"], s["out"][1:])
    return {"norm": s["out"], "g16": s["flat"][0], "g32": s["flat"][1]}


def _plain_norm(s):
    a, b = s["flat"]
    norm = torch.sqrt(a.float().square().sum() + b.square().sum())
    scale = (MAX_NORM / (norm + NORM_EPS)).clamp(max=1.0)
    out = {"norm": torch.stack([norm, scale])}
    if s["case"]["op"] == "norm":
        return out
    a.copy_(a.float() * scale)
    b.mul_(scale)
    return {**out, "g16": a, "g32": b}


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    c = case
    if c["op"] in ("rn", "rn_bwd"):
        n, e, w, back = c["rows"] * c["d"], SIZE[c["x"]], SIZE[c["w"]], c["op"] == "rn_bwd"
        vectors = sum({"none": 0, "rms": 1, "layer": 2}[c[k]] for k in ("post", "pre"))
        vectors += -(-c["rows"] // c["gate"]) if c["gate"] else 0
        stats = 8 * c["rows"] * sum(c[k] != "none" for k in ("post", "pre"))
        post, pre = c["post"] != "none", c["pre"] != "none"
        if not back:
            return {"bytes": (3 + pre) * n * e + vectors * c["d"] * w + stats, "flops": n * (3 + 7 * post + 7 * pre)}
        rows = 3 + 2 * pre + (post or bool(c["gate"]))             # dh, dx, du; dz and h; u
        return {"bytes": rows * n * e + 2 * vectors * c["d"] * w + stats, "flops": n * (3 + 14 * post + 14 * pre)}
    if c["op"] in ("bal", "bal_train"):
        T, n, k = c["T"], c["T"] * c["E"], c["topk"]
        small = 4 * T * k + (T if c["mask"] else 0) + 4 * T + 4 * c["seqs"] * c["E"]
        if c["op"] == "bal":
            return {"bytes": 4 * n + small, "flops": 6 * n}
        return {"bytes": 8 * n + small + 8 * T * k, "flops": 12 * n}
    places, _ = _places(c)
    size = sum(n * (4 if k else 2) for k, _, n in places)
    return {"bytes": size * (2 if c["op"] == "clip" else 1), "flops": (3 if c["op"] == "clip" else 2) * sum(n for _, _, n in places)}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s, c, D = prepare(case, seed), case, torch.float64
    if c["op"] in ("norm", "clip"):
        n = torch.hypot(*(torch.linalg.vector_norm(t.to(D)) for t in s["flat"]))
        f = torch.minimum(torch.ones_like(n), MAX_NORM / (n + NORM_EPS))
        out = {"norm": torch.stack([n, f])}
        return out if c["op"] == "norm" else {**out, "g16": s["flat"][0].to(D) * f, "g32": s["flat"][1].to(D) * f}
    if c["op"] in ("bal", "bal_train"):
        return _exact_bal(s, c)
    return _exact_rn(s, c) if c["op"] == "rn" else _exact_rn_bwd(s, c)


def _norm64(x, kind, w, b):
    """A norm and its statistics by their definition; kind "none" gives x."""
    if kind == "none":
        return x, None
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True) if kind == "layer" else \
        (torch.einsum("rd,rd->r", x, x)[:, None] / x.shape[1], torch.zeros_like(x[:, :1]))
    rstd = torch.rsqrt(var + EPS)
    y = (x - mean) * rstd * w.to(x.dtype)
    return y if b is None else y + b.to(x.dtype), torch.cat([mean, rstd], 1)


def _exact_rn(s, c):
    D, xt = torch.float64, s["x"].dtype
    v, post = _norm64(s["u"].to(D), c["post"], s["post_w"], s["post_b"])
    if c["gate"]:
        v = v * s["gate"].to(D).repeat_interleave(c["gate"], 0)[:c["rows"]]
    h = torch.add(RES * s["x"].to(D), v, alpha=BRANCH)
    z, pre = _norm64(h.to(xt).to(D), c["pre"], s["pre_w"], s["pre_b"])
    return {"h": h, "z": None if c["pre"] == "none" else z, "post_stats": post, "pre_stats": pre}


def _exact_rn_bwd(s, c):
    """By the chain rule through mean and rstd as the forward pass kept them: with c = x - mean,
    d mean = sum(dx) / d and d rstd = -rstd^3 sum(c dx) / d."""
    D, d, rows = torch.float64, c["d"], c["rows"]
    to = lambda n: None if s[n] is None else s[n].to(D)  # noqa: E731

    def through(dy, x, stats, w, kind):
        st = stats.to(D)
        mean, rstd = st[:, :1], st[:, 1:]
        y = x - mean
        q = torch.einsum("rd,rd,d->r", dy, y, w)[:, None]
        dx = rstd * dy * w - rstd.pow(3) * y * q / d
        if kind == "layer":
            dx = dx - rstd * (dy @ w)[:, None] / d
        return dx, torch.einsum("rd,rd->d", dy, y * rstd), y * rstd

    out = dict.fromkeys(WEIGHTS)
    dh = to("dh")
    if c["pre"] != "none":
        dx, out["pre_w"], _ = through(to("dz"), to("h"), s["pre_stats"], to("pre_w"), c["pre"])
        dh = dh + dx
        out["pre_b"] = torch.einsum("rd->d", to("dz")) if c["pre"] == "layer" else None
    group = torch.div(torch.arange(rows, device="cuda"), max(c["gate"], 1), rounding_mode="floor")
    dv = BRANCH * dh
    if c["gate"]:
        dv = dv * to("gate")[group]
    v, du = to("u"), dv
    if c["post"] != "none":
        du, out["post_w"], n = through(dv, v, s["post_stats"], to("post_w"), c["post"])
        v = n * to("post_w")
        if c["post"] == "layer":
            v = v + to("post_b")
            out["post_b"] = torch.einsum("rd->d", dv)
    if c["gate"]:
        out["gate"] = torch.zeros_like(s["gate"], dtype=D).index_add_(0, group, BRANCH * dh * v)
    return {"dx": RES * dh, "du": du, **out}


def _exact_bal(s, c):
    """Sums over the sequences by prefix sums; the gradient through log-probabilities."""
    D, T, E, k, S = torch.float64, c["T"], c["E"], c["topk"], c["seqs"]
    l = s["logits"].to(D)
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    ends = torch.tensor([0, T], device="cuda") if s["offsets"] is None else s["offsets"].long()
    live = torch.zeros(T, dtype=D, device="cuda")
    live[ends[0]:ends[-1]] = 1
    if s["mask"] is not None:
        live = live * (s["mask"] > 0)

    def per_sequence(v):
        run = torch.cat([torch.zeros(1, v.shape[1], dtype=D, device="cuda"), (v * live[:, None]).cumsum(0)])
        return run[ends[1:]] - run[ends[:-1]]

    hot = torch.zeros(T, E + 1, dtype=D, device="cuda")
    idx = torch.where((s["idx"] >= 0) & (s["idx"] < E), s["idx"], E).long()
    hot.scatter_add_(1, idx, torch.ones_like(idx, dtype=D))
    counts, ps, n = per_sequence(hot[:, :E]).round(), per_sequence(p), per_sequence(torch.ones(T, 1, dtype=D, device="cuda"))
    used = torch.count_nonzero(n).clamp(min=1)
    share = torch.where(n > 0, counts * E / (k * n), 0)
    bal = (share * torch.where(n > 0, ps / n, 0)).sum() / used
    tokens = live.sum().clamp(min=1)
    z = torch.dot(lse * lse, live) / tokens
    out = {"loss": torch.stack([BAL * bal + Z * z, bal, z]), "counts": counts.to(torch.int32), "lse": lse}
    if c["op"] == "bal":
        return out
    home = (torch.searchsorted(ends, torch.arange(T, device="cuda"), right=True) - 1).clamp(max=S - 1)
    dp = (BAL * torch.where(n > 0, share / n, 0) / used)[home]     # at the probabilities
    dlog = dp * p                                                  # at their logarithms, less lse's share
    dlse = 2 * Z * lse / tokens - dlog.sum(1)
    dl = (dlog + p * dlse[:, None]) * s["dloss"].to(D)
    g, dg = s["gates"].to(D), s["dgates"].to(D)
    dg = g * dg - g * torch.einsum("tk,tk->t", g, dg)[:, None]
    wide = torch.zeros_like(hot).scatter_add_(1, idx, dg)
    return {**out, "dlogits": (dl + wide[:, :E]) * live[:, None]}
