"""Cases of the block operators: the gated feed-forward block, layer norm and the AdamW step.

`own` False: the operators in elementary torch operations, 32 bits throughout, rounded once at the
end. `own` True: the library's calls. `exact` gives the same results from the definitions in 64 bits.

A case is a dict of plain values; "op" names the operator and direction:
  ffn        y                                  one forward pass (serving)
  ffn_train  y, dx, dW1, dW3, dW2               forward and backward pass (a training step's share)
  ln         y, mean, rstd                      layer norm, forward
  ln_bwd     dx, dw, db                         layer norm, backward, with the reduced gradients
  adamw      p, copy, m, v                      one step over all tensors, states in 32 or 8 bits
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BLOCK = 128  # values of a tensor that share a scale in the 8-bit state form
M32 = 0xFFFFFFFF


def listed():
    return [
        # one token through a fine-grained shared expert: a decode step of a single request
        {"name": "ffn one token", "op": "ffn", "T": 1, "d": 2048, "ffn": 1408},
        # a decode step of a ragged batch of requests through a large dense block
        {"name": "ffn decode batch", "op": "ffn", "T": 37, "d": 4096, "ffn": 14336},
        # a prompt through the large dense block
        {"name": "ffn prompt", "op": "ffn", "T": 4096, "d": 4096, "ffn": 14336},
        # forward and backward pass of a training micro-batch
        {"name": "ffn train", "op": "ffn_train", "T": 8192, "d": 2048, "ffn": 5632},
        # the same with odd token count and widths that no tile divides
        {"name": "ffn train ragged", "op": "ffn_train", "T": 1003, "d": 1000, "ffn": 2744},
        # the norm in front of a decode step
        {"name": "ln decode", "op": "ln", "rows": 5, "d": 4096, "x": "bf16", "w": "bf16"},
        # the norm in front of a long prompt
        {"name": "ln prompt", "op": "ln", "rows": 16384, "d": 4096, "x": "bf16", "w": "bf16"},
        # its backward pass in training, 32-bit weights beside 16-bit activations
        {"name": "ln train", "op": "ln_bwd", "rows": 16384, "d": 2048, "x": "bf16", "w": "f32"},
        # backward pass in 32 bits at an odd width
        {"name": "ln train f32 odd", "op": "ln_bwd", "rows": 1003, "d": 4099, "x": "f32", "w": "f32"},
        # the small tensors of a model (norms, biases, a router): many launches' worth of little work
        {"name": "adamw small tensors", "op": "adamw", "bits": 32, "count": 67, "most": 20011, "grad": "f32",
         "copy": False, "scaled": False, "step": 3},
        # the three matrices of eight experts, 16-bit gradients, 32-bit parameters with their 16-bit copy
        {"name": "adamw 32 bits", "op": "adamw", "bits": 32, "count": 24, "most": 11534336, "grad": "bf16",
         "copy": True, "scaled": True, "step": 1000},
        # the same with states in 8 bits
        {"name": "adamw 8 bits", "op": "adamw", "bits": 8, "count": 24, "most": 11534336, "grad": "bf16",
         "copy": True, "scaled": True, "step": 1000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_train", "ffn_train", "ln", "ln_bwd", "adamw", "adamw"])
    if op in ("ffn", "ffn_train"):
        d = 8 * _log(rng, 16, 512)        # widths 128 .. 4096 and 256 .. 14336, multiples of 8
        f = 8 * _log(rng, 32, 1792)
        most = 1.4e12 / (6 if op == "ffn" else 18) / d / f
        return {"op": op, "T": _log(rng, 1, max(2, min(8192, most))), "d": d, "ffn": f}
    if op in ("ln", "ln_bwd"):
        d = _log(rng, 128, 8192)
        x = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "rows": _log(rng, 1, min(32768, 3.3e7 / d)), "d": d, "x": x, "w": rng.choice([x, "f32"])}
    count = _log(rng, 1, 200)
    return {"op": op, "bits": rng.choice([8, 32]), "count": count, "most": _log(rng, 100, 1.2e8 / count),
            "grad": rng.choice(["f32", "bf16"]), "copy": rng.random() < 0.5, "scaled": rng.random() < 0.5,
            "step": _log(rng, 1, 100000)}


# ---- inputs -------------------------------------------------------------------------------------

LR, B1, B2, EPS, WD, RNG = 3e-4, 0.9, 0.999, 1e-8, 0.1, 20240229


def _sizes(c):
    """Element counts of an AdamW case's tensors: the largest, and odd fractions of it."""
    return [c["most"] if i == 0 else max(1, c["most"] * ((i * 37) % 64 + 1) // 64 - i % 3) for i in range(c["count"])]


def _offsets(c):
    """Start of each tensor in the flat buffers (multiples of the block), and their length."""
    at, off = 0, []
    for n in _sizes(c):
        off.append(at)
        at += -(-n // BLOCK) * BLOCK
    return off, at


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, dtype, std=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).add_(mean).to(dtype)

    s, bf = {"case": c}, torch.bfloat16
    if c["op"] in ("ffn", "ffn_train"):
        T, d, f = c["T"], c["d"], c["ffn"]
        s["x"] = normal((T, d), bf)                      # normalised activations
        s["W1"], s["W3"] = normal((f, d), bf, d ** -0.5), normal((f, d), bf, d ** -0.5)
        s["W2"] = normal((d, f), bf, f ** -0.5)
        if c["op"] == "ffn_train":
            s["dy"] = normal((T, d), bf, 0.01)
        if own:  # what a program keeps beside its weights: the outputs' buffers and the workspace
            import tile_level_copy_gb300 as tlc
            s["cfg"] = tlc.FFNConfig(T=T, d=d, ffn=f)
            s["ws"] = tlc.FFNWorkspace(s["cfg"])
            s["y"] = torch.empty_like(s["x"])
            if c["op"] == "ffn_train":
                s["saved"] = tlc.ffn_saved(s["cfg"])
                s["grads"] = [torch.empty_like(s[n]) for n in ("x", "W1", "W3", "W2")]
    elif c["op"] in ("ln", "ln_bwd"):
        r, d, xt, wt = c["rows"], c["d"], DT[c["x"]], DT[c["w"]]
        s["x"] = normal((r, d), xt, 1.5, 0.25)           # a residual stream that is off centre
        s["w"], s["b"] = normal((d,), wt, 0.1, 1.0), normal((d,), wt, 0.1)
        if c["op"] == "ln_bwd":
            s["dy"] = normal((r, d), xt, 0.1)
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + 1e-5)
        if own:
            import tile_level_copy_gb300 as tlc
            s["cfg"] = tlc.LayerNormConfig(rows=r, d=d, dtype=xt, wdtype=wt, eps=1e-5)
            s["out"] = torch.empty_like(s["x"])
            if c["op"] == "ln":
                s["stats"] = [torch.empty(r, device="cuda") for _ in range(2)]
            else:
                s["ws"] = tlc.LayerNormWorkspace(s["cfg"])
                s["wgrads"] = [torch.empty_like(s["w"]) for _ in range(2)]
    else:
        off, n = _offsets(c)
        pad = torch.zeros(n, device="cuda")              # 1 where a tensor has a value, 0 in between
        for o, k in zip(off, _sizes(c)):
            pad[o:o + k] = 1
        s["p"] = normal((n,), torch.float32, 0.02) * pad
        s["g"] = (normal((n,), torch.float32, 1e-3) * torch.exp(normal((n,), torch.float32, 1.0)) * pad).to(DT[c["grad"]])
        s["scale"] = torch.full((1,), 0.37, device="cuda") if c["scaled"] else None
        s["copy"] = torch.zeros(n, dtype=bf, device="cuda") if c["copy"] else None
        m = normal((n,), torch.float32, 3e-4) * pad
        v = (normal((n,), torch.float32, 1e-3) * torch.exp(normal((n,), torch.float32, 1.0)) * pad).square()
        if c["bits"] == 32:
            s["m"], s["v"] = m, v
        else:                                            # a state as an earlier step left it
            s["m"], s["ms"] = _encode(m, 7, 2.0 ** -120, torch.zeros_like(m, dtype=torch.int32))
            s["v"], s["vs"] = _encode(v, 15, 2.0 ** -112, torch.zeros_like(m, dtype=torch.int32))
        if own:
            import tile_level_copy_gb300 as tlc
            s["cfg"] = tlc.AdamWConfig(lr=LR, beta1=B1, beta2=B2, eps=EPS, weight_decay=WD, bits=c["bits"], seed=RNG)
            cut = [slice(o, o + k) for o, k in zip(off, _sizes(c))]
            blocks = [slice(o // BLOCK, (o + k + BLOCK - 1) // BLOCK) for o, k in zip(off, _sizes(c))]
            view = lambda t, at: None if t is None else [t[a] for a in at]  # noqa: E731
            eight = c["bits"] == 8
            s["list"] = tlc.AdamWList(s["cfg"], view(s["p"], cut), view(s["g"], cut), view(s["m"], cut), view(s["v"], cut),
                                      m_scale=view(s["ms"], blocks) if eight else None,
                                      v_scale=view(s["vs"], blocks) if eight else None, copy=view(s["copy"], cut))
            if eight:
                s["mv"] = [torch.zeros(n, device="cuda") for _ in range(2)]
                s["values"] = tlc.AdamWValues(s["list"], view(s["mv"][0], cut), view(s["mv"][1], cut))
    return s


# ---- one pass -----------------------------------------------------------------------------------

def run(state):
    s, op = state, state["case"]["op"]
    if op in ("ffn", "ffn_train"):
        return _own_ffn(s) if own else _plain_ffn(s)
    if op in ("ln", "ln_bwd"):
        return _own_ln(s) if own else _plain_ln(s)
    return _own_adamw(s) if own else _plain_adamw(s)


def _own_ffn(s):
    import tile_level_copy_gb300 as tlc
    saved = s.get("saved")
    tlc.ffn_forward(s["cfg"], s["x"], s["W1"], s["W3"], s["W2"], s["y"], s["ws"], saved=saved)
    if saved is None:
        return {"y": s["y"]}
    dx, d1, d3, d2 = s["grads"]
    tlc.ffn_backward(s["cfg"], s["x"], s["W1"], s["W3"], s["W2"], s["dy"], saved, dx, d1, d3, d2, s["ws"])
    return {"y": s["y"], "dx": dx, "dW1": d1, "dW3": d3, "dW2": d2}


def _plain_ffn(s):
    x, w1, w3, w2 = (s[n].float() for n in ("x", "W1", "W3", "W2"))
    g, u = x @ w1.T, x @ w3.T
    sg = 1 / (1 + torch.exp(-g))
    h = g * sg * u
    y = h @ w2.T
    bf = torch.bfloat16
    if "dy" not in s:
        return {"y": y.to(bf)}
    dy = s["dy"].float()
    dh = dy @ w2
    dg, du = dh * u * sg * (1 + g * (1 - sg)), dh * g * sg
    return {"y": y.to(bf), "dx": (dg @ w1 + du @ w3).to(bf), "dW1": (dg.T @ x).to(bf), "dW3": (du.T @ x).to(bf),
            "dW2": (dy.T @ h).to(bf)}


def _own_ln(s):
    import tile_level_copy_gb300 as tlc
    if "stats" in s:
        tlc.layernorm_forward(s["cfg"], s["x"], s["w"], s["b"], s["out"], *s["stats"])
        return {"y": s["out"], "mean": s["stats"][0], "rstd": s["stats"][1]}
    dw, db = s["wgrads"]
    tlc.layernorm_backward(s["cfg"], s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["out"], dw, db, s["ws"])
    return {"dx": s["out"], "dw": dw, "db": db}


def _plain_ln(s):
    x, w = s["x"].float(), s["w"].float()
    if "dy" not in s:
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1 / torch.sqrt((c * c).mean(1) + 1e-5)
        return {"y": (c * rstd[:, None] * w + s["b"].float()).to(s["x"].dtype), "mean": mean, "rstd": rstd}
    dy = s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gy = dy * w
    dx = s["rstd"][:, None] * (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True))
    wt = s["w"].dtype
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0).to(wt), "db": dy.sum(0).to(wt)}


def _own_adamw(s):
    import tile_level_copy_gb300 as tlc
    tlc.adamw_step(s["cfg"], s["list"], s["case"]["step"], grad_scale=s["scale"])
    out = {"p": s["p"], "copy": s["copy"], "m": s["m"], "v": s["v"]}
    if s["case"]["bits"] == 8:
        tlc.adamw_read_state(s["cfg"], s["list"], s["values"])
        out["m"], out["v"] = s["mv"]
    return out


def _plain_adamw(s):
    c, p, t = s["case"], s["p"], s["case"]["step"]
    g = s["g"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    eight = c["bits"] == 8
    m0 = _decode(s["m"], s["ms"], 2.0 ** 120) if eight else s["m"]
    v0 = _decode(s["v"], s["vs"], 2.0 ** 112) if eight else s["v"]
    m = m0 * B1 + g * (1 - B1)
    v = v0 * B2 + (g * g) * (1 - B2)
    root = torch.sqrt(v) * (1 / math.sqrt(1 - B2 ** t)) + EPS
    p.copy_(p * (1 - LR * WD) - (LR / (1 - B1 ** t)) * m / root)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    out = {"p": p, "copy": s["copy"]}
    if eight:
        r = _noise(p.numel(), t, p.device)
        _put(s, "m", *_encode(m, 7, 2.0 ** -120, ((r & 0xFFFF) << 4) + 8))
        _put(s, "v", *_encode(v, 15, 2.0 ** -112, ((r >> 16) << 4) + 8))
        return {**out, "m": _decode(s["m"], s["ms"], 2.0 ** 120), "v": _decode(s["v"], s["vs"], 2.0 ** 112)}
    s["m"].copy_(m)
    s["v"].copy_(v)
    return {**out, "m": s["m"], "v": s["v"]}


def _put(s, name, codes, scales):
    s[name].copy_(codes)
    s[name + "s"].copy_(scales)


def _mix(x, k):
    """32 bits in, 32 bits out (as int64): multiply-xorshift rounds with a second key between them."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & M32
    x = ((x ^ (x >> 15)) + k) & M32
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _noise(n, step, device):
    """The step's 32 random bits for each value: a hash of the seed, the step and the value's index."""
    k0 = _mix((RNG & M32) ^ (step & M32), RNG >> 32)
    k1 = _mix(k0 ^ 0x9E3779B9, (step >> 32) & M32)
    return _mix(torch.arange(n, dtype=torch.int64, device=device) ^ k0, k1).to(torch.int64)


def _encode(x, top, down, r):
    """Codes and scale bytes of a state: each block of 128 is scaled by a power of two so that its
    largest value lies in [2^top, 2^(top + 1)), and each value keeps its leading bits (3 of mantissa),
    rounded up where the bits cut off and the 20 random bits r carry."""
    b = x.view(-1, BLOCK)
    most = b.abs().amax(1)
    e = (most.view(torch.int32) >> 23) - 127
    k = (e - top).clamp(-126, 126)
    t = (b * ((127 - k) << 23).view(torch.float32)[:, None]) * down
    bits = t.reshape(-1).view(torch.int32)
    code = ((bits & 0x7FFFFFFF) + r) >> 20
    code = torch.where(bits < 0, code | 0x80, code).to(torch.uint8)
    fine = torch.isfinite(most)
    code = torch.where(fine[:, None], code.view(-1, BLOCK), 0).reshape(-1)
    return code, torch.where(fine, k + 127, 255).to(torch.uint8)


def _decode(code, scale, up):
    """The values that codes and scale bytes stand for."""
    c = code.to(torch.int32)
    signed = up == 2.0 ** 120
    x = (((c & 0x7F) if signed else c) << 20).view(torch.float32) * up
    if signed:
        x = torch.where(c >= 0x80, -x, x)
    f = torch.where(scale == 255, torch.nan, (scale.to(torch.int32) << 23).view(torch.float32))
    return (x.view(-1, BLOCK) * f[:, None]).reshape(-1)


# ---- what a pass cannot do without --------------------------------------------------------------

def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] in ("ffn", "ffn_train"):
        T, d, f = c["T"], c["d"], c["ffn"]
        if c["op"] == "ffn":
            return {"bytes": 2 * (2 * T * d + 3 * d * f), "flops": 6 * T * d * f}
        return {"bytes": 2 * (4 * T * d + 6 * d * f), "flops": 18 * T * d * f}
    if c["op"] in ("ln", "ln_bwd"):
        n, e, w = c["rows"] * c["d"], size[c["x"]], size[c["w"]]
        if c["op"] == "ln":
            return {"bytes": 2 * n * e + 2 * c["d"] * w + 8 * c["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * c["d"] * w + 8 * c["rows"], "flops": 14 * n}
    n = sum(_sizes(c))
    states = 16 if c["bits"] == 32 else 4 + 8  # read and written; 8 bits: and their values returned
    return {"bytes": n * (8 + size[c["grad"]] + (2 if c["copy"] else 0) + states), "flops": 16 * n}


# ---- the definitions in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s, c = prepare(case, seed), case
    D = torch.float64
    if c["op"] in ("ffn", "ffn_train"):
        return _exact_ffn(s, c["op"] == "ffn_train")
    if c["op"] == "ln":
        x = s["x"].to(D)
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = torch.rsqrt(var + 1e-5)
        return {"y": torch.addcmul(s["b"].to(D), (x - mean[:, None]) * rstd[:, None], s["w"].to(D)), "mean": mean, "rstd": rstd}
    if c["op"] == "ln_bwd":
        # the derivative of y = w (x - mean) rstd + b, with d mean = sum(dx) / d and
        # d rstd = -rstd^3 sum((x - mean) dx) / d; mean and rstd as the forward pass kept them
        x, dy, w = s["x"].to(D), s["dy"].to(D), s["w"].to(D)
        mean, rstd, d = s["mean"].to(D)[:, None], s["rstd"].to(D)[:, None], x.shape[1]
        z = x - mean
        a = torch.matmul(dy, w)[:, None]
        q = torch.einsum("rd,rd,d->r", dy, z, w)[:, None]
        return {"dx": rstd * (dy * w) - rstd * a / d - rstd ** 3 * z * q / d, "dw": torch.einsum("rd,rd->d", dy, z * rstd),
                "db": torch.einsum("rd,r->d", dy, torch.ones_like(rstd[:, 0]))}
    return _exact_adamw(s, c)


def _exact_ffn(s, train):
    D, f = torch.float64, s["W1"].shape[0]
    x = s["x"].to(D)
    y, dx = torch.zeros_like(x), torch.zeros_like(x)
    d1, d3, d2 = [], [], []
    for at in range(0, f, 2048):  # the hidden columns in parts: each adds to y and dx
        w1, w3, w2 = s["W1"][at:at + 2048].to(D), s["W3"][at:at + 2048].to(D), s["W2"][:, at:at + 2048].to(D)
        g, u = torch.matmul(x, w1.T), torch.matmul(x, w3.T)
        sg = torch.sigmoid(g)
        y += torch.matmul(g * sg * u, w2.T)
        if train:
            dy = s["dy"].to(D)
            dh = torch.matmul(dy, w2)
            dg, du = dh * u * (sg + g * sg * (1 - sg)), dh * (g * sg)
            dx += torch.matmul(dg, w1) + torch.matmul(du, w3)
            d1.append(torch.matmul(dg.T, x))
            d3.append(torch.matmul(du.T, x))
            d2.append(torch.matmul(dy.T, g * sg * u))
    if not train:
        return {"y": y}
    return {"y": y, "dx": dx, "dW1": torch.cat(d1), "dW3": torch.cat(d3), "dW2": torch.cat(d2, 1)}


def _exact_adamw(s, c):
    """One step in 64 bits. The 8-bit form's rounding is part of its definition: up with probability
    equal to the part cut off, as the step's random bits decide; here by division and floor."""
    D, t = torch.float64, c["step"]
    g = s["g"].to(D)
    if s["scale"] is not None:
        g = g * s["scale"].to(D)
    table = lambda up, bias, sign: torch.tensor(  # noqa: E731
        [(-1.0 if sign and k >= 128 else 1.0) * ((k & 7) / 8 + ((k & up) >> 3 > 0)) * 2.0 ** (max((k & up) >> 3, 1) - bias)
         for k in range(256)], dtype=D, device="cuda")
    if c["bits"] == 8:
        wide = lambda sc: (torch.pow(2.0, sc.to(D) - 127) * (sc > 0)).repeat_interleave(BLOCK)  # noqa: E731
        m0 = table(0x78, 7, True)[s["m"].long()] * wide(s["ms"])
        v0 = table(0xF8, 15, False)[s["v"].long()] * wide(s["vs"])
    else:
        m0, v0 = s["m"].to(D), s["v"].to(D)
    m = torch.lerp(g, m0, B1)
    v = torch.lerp(g.square(), v0, B2)
    step = (m / (1 - B1 ** t)) / (torch.sqrt(v / (1 - B2 ** t)) + EPS)
    p = s["p"].to(D) - LR * (WD * s["p"].to(D) + step)
    out = {"p": p, "copy": p if c["copy"] else None, "m": m, "v": v}
    if c["bits"] == 8:
        r = _noise(p.numel(), t, p.device)
        out["m"] = _nearby(m, 7, 6, r & 0xFFFF)
        out["v"] = _nearby(v, 15, 14, r >> 16)
    return out


def _nearby(x, top, lowest, r):
    """x rounded to 4 significant bits in blocks whose largest value is in [2^top, 2^(top+1)) after
    scaling; below 2^-lowest the steps are even. r in [0, 2^16): up where the part cut off plus
    (r + 1/2) / 2^16 reaches 1."""
    b = x.view(-1, BLOCK)
    most = b.abs().amax(1)
    k = (torch.floor(torch.log2(most.clamp_min(1e-300))) - top).clamp(-126, 126)[:, None]
    y = b.abs() * torch.pow(2.0, -k)
    e = torch.floor(torch.log2(y.clamp_min(2.0 ** -lowest))).clamp_min(-lowest)
    unit = torch.pow(2.0, e - 3)
    n = torch.floor(y / unit + (r.view(-1, BLOCK).to(torch.float64) + 0.5) / 65536)
    return (torch.sign(b) * n * unit * torch.pow(2.0, k)).reshape(-1)
