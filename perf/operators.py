"""Cases of the row operators: the norms around a transformer block, 8-bit checkpoints, the gated activation.

Each case is one call of one operator on tensors of real size: ``listed`` gives
the fixed ones, ``draw`` more of the same ranges.  ``run`` computes a case
either in plain torch operations (``own`` false) or through the library's
calls (``own`` true); ``exact`` computes it in 64 bits.

An operator's name in a case ("op"):
  norm_fwd   h' = alpha*h + gate*post(u), n = pre(h')
  norm_bwd   its gradients, from the kept tensors or from 8-bit checkpoints
  gated_fwd  z = phi(a)*b
  gated_bwd  its gradients (and z again), from the kept tensors or from checkpoints
  store      a tensor into 8 bits with a scale for every 128 columns of a row
  load       values from 8 bits, optionally scaled and shifted by column
"""
import math

import torch

own = False

GROUP = 128
QMAX = {"e4m3": 448.0, "int8": 127.0}
QTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


def _norm(name, op, rows, cols, dtype, post, pre, gate, q8, bias=False, alpha=1.0):
    """post, pre: "none", "rms" or "layer"; gate: -1 none, 0 one for all rows, else rows a gate row covers."""
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "post": post, "pre": pre,
            "gate": gate, "q8": q8, "bias": bias, "alpha": alpha}


def _gated(name, op, rows, cols, dtype, act, q8, again=False):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "act": act, "q8": q8, "again": again}


def listed():
    return [
        # serving: eight sequences of one new token each, nothing is kept
        _norm("norm_fwd_decode", "norm_fwd", 8, 4096, "bf16", "rms", "rms", -1, "none"),
        # training: 16 k tokens, both norms, a learned gate per column, xhat kept in 8 bits
        _norm("norm_fwd_train", "norm_fwd", 16384, 4096, "bf16", "rms", "rms", 0, "e4m3"),
        # a conditioned block (a gate row for each sequence) of odd width, layer norms, everything kept
        _norm("norm_fwd_odd", "norm_fwd", 3001, 1021, "f16", "layer", "layer", 750, "none", True, 0.7),
        # the backward of norm_fwd_train, from its checkpoints
        _norm("norm_bwd_train", "norm_bwd", 16384, 4096, "bf16", "rms", "rms", 0, "e4m3"),
        # a wide conditioned block, layer norms with shifts, two sequences
        _norm("norm_bwd_wide", "norm_bwd", 2048, 8192, "bf16", "layer", "layer", 1024, "e4m3", True, 0.7),
        # the backward of an odd width, from kept 32-bit tensors
        _norm("norm_bwd_odd", "norm_bwd", 3001, 1021, "f32", "layer", "layer", 750, "none", True, 0.7),
        # serving: four tokens through the gated activation of a feed-forward block
        _gated("gated_fwd_decode", "gated_fwd", 4, 11008, "f16", "gelu_tanh", "none"),
        # training: the gated activation of 8 k tokens, its inputs kept in 8 bits
        _gated("gated_fwd_train", "gated_fwd", 8192, 14336, "bf16", "silu", "int8"),
        # its backward, with z computed again for the gradient of the weights behind it
        _gated("gated_bwd_train", "gated_bwd", 8192, 14336, "bf16", "silu", "int8", True),
        # a short ragged batch of odd width
        _gated("gated_bwd_odd", "gated_bwd", 777, 2731, "f16", "gelu", "e4m3"),
        # any activation into 8 bits
        {"name": "store", "op": "store", "rows": 16384, "cols": 5120, "dtype": "bf16", "q8": "e4m3"},
        # the block's input again from the kept xhat, for the gradient of its first weights
        {"name": "load", "op": "load", "rows": 16384, "cols": 4096, "dtype": "bf16", "q8": "e4m3", "bias": False},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "gated_fwd", "gated_bwd", "store", "load"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    cols = _log(rng, 64, 14336 if op.startswith("gated") else 8192)
    shape = rng.random()
    if shape < 0.6:
        cols = max(64, cols // 64 * 64)  # widths that models have
    elif shape < 0.8:
        cols = max(8, cols // 8 * 8)
    rows = _log(rng, 1, max(2, min(16384, (2 << 24) // cols if dtype == "f32" else (4 << 24) // cols)))
    c = {"op": op, "rows": rows, "cols": cols, "dtype": dtype}
    if op.startswith("norm"):
        kind = rng.choice(["rms", "layer"])
        post = rng.choice([kind, kind, "none"])
        gate = rng.choice([-1, 0, max(1, rows // 3)])
        q8 = rng.choice(["none", "e4m3"])
        c |= {"post": post, "pre": kind, "gate": gate, "q8": q8, "bias": kind == "layer", "alpha": rng.choice([1.0, 0.7])}
    elif op.startswith("gated"):
        c |= {"act": rng.choice(["silu", "gelu", "gelu_tanh"]), "q8": rng.choice(["none", "e4m3", "int8"]),
              "again": op == "gated_bwd" and rng.random() < 0.5}
    elif op == "store":
        c |= {"q8": rng.choice(["e4m3", "int8"])}
    else:
        c |= {"q8": rng.choice(["e4m3", "int8"]), "bias": rng.random() < 0.5}
    return c


# ------------------------------------------------------------------ inputs

def _groups(cols):
    return -(-cols // GROUP)


def _values(gen, rows, cols, dtype, size=1.0, offset=0.0):
    """Activations as blocks give them: columns of unequal size, a few much larger, a few rows of padding (zeros)."""
    column = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda")) * size
    column[torch.randint(0, cols, (max(1, cols // 512),), generator=gen, device="cuda")] *= 20.0
    x = torch.randn(rows, cols, generator=gen, device="cuda") * column
    if offset:
        x += offset * torch.randn(rows, 1, generator=gen, device="cuda")
    if rows > 64:
        x[torch.randint(0, rows, (rows // 64,), generator=gen, device="cuda")] = 0.0
    return x.to(dtype)


def _weights(gen, *shape, mean=1.0):
    return mean + 0.2 * torch.randn(*shape, generator=gen, device="cuda")


def _quantise(x, form):
    """Codes and scales of a float32 [rows, cols]: amax of every 128 columns onto the format's largest value."""
    rows, cols = x.shape
    groups = _groups(cols)
    padded = torch.nn.functional.pad(x, (0, groups * GROUP - cols)).view(rows, groups, GROUP)
    amax = padded.abs().amax(-1)
    top = torch.full_like(amax, QMAX[form])
    by = torch.where(amax > 0, torch.div(top, amax), torch.zeros_like(amax))
    scaled = (padded * by[..., None]).view(rows, groups * GROUP)[:, :cols]
    codes = scaled.to(torch.float8_e4m3fn) if form == "e4m3" else scaled.round().to(torch.int8)
    return codes.contiguous(), amax / QMAX[form]


def _dequantise(codes, scale):
    cols = codes.shape[1]
    return codes.float() * scale.repeat_interleave(GROUP, 1)[:, :cols]


def _normalise(x, kind, eps):
    """(xhat, mean, rstd) of the rows of a float32 tensor."""
    if kind == "none":
        return x, None, None
    mean = x.mean(-1) if kind == "layer" else None
    centred = x - mean[:, None] if kind == "layer" else x
    rstd = torch.rsqrt(centred.square().mean(-1) + eps)
    return centred * rstd[:, None], mean, rstd


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rows, cols, dtype, op = case["rows"], case["cols"], DTYPE[case["dtype"]], case["op"]
    new = lambda *shape, dtype=dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    codes = lambda: new(rows, cols, dtype=QTYPE[case["q8"]])  # noqa: E731
    scales = lambda: new(rows, _groups(cols), dtype=torch.float32)  # noqa: E731
    s = {"case": dict(case)}
    if op.startswith("norm"):
        post, pre, gated, kept = case["post"], case["pre"], case["gate"] >= 0, case["q8"] == "none"
        s["u"] = _values(gen, rows, cols, dtype)
        s["h"] = _values(gen, rows, cols, dtype, 2.0, 0.5)
        s["gate"] = None
        if gated:
            n_gates = 1 if case["gate"] == 0 else -(-rows // case["gate"])
            s["gate"] = _weights(gen, n_gates, cols, mean=0.5)
        s["gamma_post"] = _weights(gen, cols) if post != "none" else None
        s["beta_post"] = _weights(gen, cols, mean=0.0) if post != "none" and case["bias"] else None
        s["gamma_pre"] = _weights(gen, cols)
        s["beta_pre"] = _weights(gen, cols, mean=0.0) if case["bias"] else None
        row = lambda on: new(rows, dtype=torch.float32) if on else None  # noqa: E731
        if op == "norm_fwd":
            s["h_out"], s["n"] = new(rows, cols), new(rows, cols)
            s["mean_post"], s["rstd_post"] = row(post == "layer" and kept), row(post != "none")
            s["mean_pre"], s["rstd_pre"] = row(pre == "layer" and kept), row(True)
            if not kept:
                s["q_post"], s["scale_post"], s["q_pre"], s["scale_pre"] = codes(), scales(), codes(), scales()
            return s
        # what the forward leaves for the backward, and the gradients that reach it
        uhat, s["mean_post"], s["rstd_post"] = _normalise(s["u"].float(), post, EPS)
        hout = _residual(s, uhat)
        xhat, s["mean_pre"], s["rstd_pre"] = _normalise(hout, pre, EPS)
        if kept:
            s["h_out"] = hout.to(dtype)
        else:
            (s["q_post"], s["scale_post"]), (s["q_pre"], s["scale_pre"]) = _quantise(uhat, case["q8"]), _quantise(xhat, case["q8"])
            del s["u"], s["mean_post"], s["mean_pre"]
        del s["h"]
        s["dh_out"], s["dn"] = _values(gen, rows, cols, dtype, 0.05), _values(gen, rows, cols, dtype, 0.05)
        s["dh"], s["du"] = new(rows, cols), new(rows, cols)
        like = lambda w: None if w is None else torch.empty_like(w)  # noqa: E731
        for k in ("gamma_post", "beta_post", "gate", "gamma_pre", "beta_pre"):
            s["d" + k] = like(s[k])
        s["workspace"] = None
        return s
    if op.startswith("gated"):
        kept = case["q8"] == "none"
        packed = _values(gen, rows, 2 * cols, dtype, 1.0, 0.3)  # one product gives both halves
        s["a"], s["b"] = packed[:, :cols], packed[:, cols:]
        if op == "gated_fwd":
            s["z"] = new(rows, cols)
            if not kept:
                s["qa"], s["scale_a"], s["qb"], s["scale_b"] = codes(), scales(), codes(), scales()
            return s
        if not kept:
            (s["qa"], s["scale_a"]), (s["qb"], s["scale_b"]) = (_quantise(s[k].float(), case["q8"]) for k in "ab")
            del s["a"], s["b"]
        s["dz"] = _values(gen, rows, cols, dtype, 0.05)
        s["packed"] = new(rows, 2 * cols)  # the gradient of that product's result
        s["da"], s["db"] = s["packed"][:, :cols], s["packed"][:, cols:]
        s["z"] = new(rows, cols) if case["again"] else None
        return s
    x = _values(gen, rows, cols, dtype, 1.0, 0.3)
    if op == "store":
        s["x"], s["q"], s["scale"] = x, codes(), scales()
        return s
    s["q"], s["scale"] = _quantise(x.float(), case["q8"])
    s["gamma"] = _weights(gen, cols)
    s["beta"] = _weights(gen, cols, mean=0.0) if case["bias"] else None
    s["y"] = new(rows, cols)
    return s


# ---------------------------------------------------------- the plain forms

def _gate_rows(s):
    """The gate of every row: [rows, cols], [1, cols] or the number 1."""
    if s["gate"] is None:
        return 1.0
    per = s["case"]["gate"]
    return s["gate"] if per == 0 else s["gate"].repeat_interleave(per, 0)[: s["case"]["rows"]]


def _residual(s, uhat):
    p = uhat
    if s["gamma_post"] is not None:
        p = uhat * s["gamma_post"]
    if s["beta_post"] is not None:
        p = p + s["beta_post"]
    return s["case"]["alpha"] * s["h"].float() + _gate_rows(s) * p


def _plain_norm_fwd(s):
    c, dtype = s["case"], s["u"].dtype
    uhat, mean_post, rstd_post = _normalise(s["u"].float(), c["post"], EPS)
    hout = _residual(s, uhat)
    xhat, mean_pre, rstd_pre = _normalise(hout, c["pre"], EPS)
    n = xhat * s["gamma_pre"]
    if s["beta_pre"] is not None:
        n = n + s["beta_pre"]
    out = {"h_out": hout.to(dtype), "n": n.to(dtype), "rstd_post": rstd_post, "rstd_pre": rstd_pre}
    if c["q8"] == "none":
        return out | {"mean_post": mean_post, "mean_pre": mean_pre}
    out["q_post"], out["scale_post"] = _quantise(uhat, c["q8"])
    out["q_pre"], out["scale_pre"] = _quantise(xhat, c["q8"])
    return out


def _back_through(g, xhat, rstd, kind):
    """The gradient of a norm's input from the gradient of xhat."""
    if kind == "none":
        return g
    d = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(-1, keepdim=True)
    return d * rstd[:, None]


def _plain_norm_bwd(s):
    c, dtype = s["case"], s["dn"].dtype
    if c["q8"] == "none":
        uhat, xhat = s["u"].float(), s["h_out"].float()
        if s["mean_post"] is not None:
            uhat = uhat - s["mean_post"][:, None]
        if s["rstd_post"] is not None:
            uhat = uhat * s["rstd_post"][:, None]
        if s["mean_pre"] is not None:
            xhat = xhat - s["mean_pre"][:, None]
        xhat = xhat * s["rstd_pre"][:, None]
    else:
        uhat, xhat = _dequantise(s["q_post"], s["scale_post"]), _dequantise(s["q_pre"], s["scale_pre"])
    dn = s["dn"].float()
    t = s["dh_out"].float() + _back_through(dn * s["gamma_pre"], xhat, s["rstd_pre"], c["pre"])
    p = uhat if s["gamma_post"] is None else uhat * s["gamma_post"]
    if s["beta_post"] is not None:
        p = p + s["beta_post"]
    dp = t * _gate_rows(s)
    e = dp if s["gamma_post"] is None else dp * s["gamma_post"]
    out = {"dh": (c["alpha"] * t).to(dtype), "du": _back_through(e, uhat, s["rstd_post"], c["post"]).to(dtype)}
    out["dgamma_pre"] = (dn * xhat).sum(0)
    if s["beta_pre"] is not None:
        out["dbeta_pre"] = dn.sum(0)
    if s["gamma_post"] is not None:
        out["dgamma_post"] = (dp * uhat).sum(0)
    if s["beta_post"] is not None:
        out["dbeta_post"] = dp.sum(0)
    if s["gate"] is not None:
        per = c["gate"] or c["rows"]
        each = t * p
        whole = c["rows"] // per * per
        parts = [each[:whole].view(-1, per, c["cols"]).sum(1)]
        if whole < c["rows"]:
            parts.append(each[whole:].sum(0, keepdim=True))
        out["dgate"] = torch.cat(parts)
    return out


def _phi(a, act):
    """(phi(a), phi'(a)) in the type of a."""
    if act == "silu":
        sig = 1.0 / (1.0 + torch.exp(-a))
        return a * sig, sig * (1.0 + a * (1.0 - sig))
    if act == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
        return a * cdf, cdf + a * torch.exp(-0.5 * a * a) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    th = torch.tanh(k * (a + 0.044715 * a * a * a))
    return 0.5 * a * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * a * (1.0 - th * th) * k * (1.0 + 3 * 0.044715 * a * a)


def _plain_gated_fwd(s):
    c = s["case"]
    a, b = s["a"].float(), s["b"].float()
    out = {"z": (_phi(a, c["act"])[0] * b).to(s["z"].dtype)}
    if c["q8"] != "none":
        out["qa"], out["scale_a"] = _quantise(a, c["q8"])
        out["qb"], out["scale_b"] = _quantise(b, c["q8"])
    return out


def _plain_gated_bwd(s):
    c, dtype = s["case"], s["dz"].dtype
    if c["q8"] == "none":
        a, b = s["a"].float(), s["b"].float()
    else:
        a, b = _dequantise(s["qa"], s["scale_a"]), _dequantise(s["qb"], s["scale_b"])
    phi, slope = _phi(a, c["act"])
    dz = s["dz"].float()
    out = {"da": (dz * b * slope).to(dtype), "db": (dz * phi).to(dtype)}
    if c["again"]:
        out["z"] = (phi * b).to(dtype)
    return out


def _plain_load(s):
    y = _dequantise(s["q"], s["scale"]) * s["gamma"]
    return {"y": (y if s["beta"] is None else y + s["beta"]).to(s["y"].dtype)}


def _plain_store(s):
    q, scale = _quantise(s["x"].float(), s["case"]["q8"])
    return {"q": q, "scale": scale}


# ------------------------------------------------------- the library's calls

def _own_norm(s):
    import place_batchnorm_activation_b200 as iabn
    c = s["case"]
    kind = {"none": iabn.IABN_NORM_NONE, "rms": iabn.IABN_NORM_RMS, "layer": iabn.IABN_NORM_LAYER}
    how = {"post": kind[c["post"]], "pre": kind[c["pre"]], "residual_scale": c["alpha"], "rows_per_gate": max(0, c["gate"]),
           "gamma_post": s["gamma_post"], "beta_post": s["beta_post"], "gate": s["gate"], "gamma_pre": s["gamma_pre"]}
    if c["op"] == "norm_fwd":
        how |= {"beta_pre": s["beta_pre"], "eps_post": EPS, "eps_pre": EPS}
        out = {k: s[k] for k in ("h_out", "n", "rstd_post", "rstd_pre")}
        if c["q8"] == "none":
            iabn.block_norm_forward(s["u"], s["h"], s["h_out"], s["n"], mean_post=s["mean_post"], rstd_post=s["rstd_post"],
                                    mean_pre=s["mean_pre"], rstd_pre=s["rstd_pre"], **how)
            return out | {"mean_post": s["mean_post"], "mean_pre": s["mean_pre"]}
        iabn.block_norm_forward_checkpoint8(s["u"], s["h"], s["h_out"], s["n"], q_post=s["q_post"], scale_post=s["scale_post"],
                                            rstd_post=s["rstd_post"], q_pre=s["q_pre"], scale_pre=s["scale_pre"],
                                            rstd_pre=s["rstd_pre"], **how)
        return out | {k: s[k] for k in ("q_post", "scale_post", "q_pre", "scale_pre")}
    if s["workspace"] is None:
        s["workspace"] = iabn.new_block_norm_workspace(c["rows"], c["cols"], max(0, c["gate"]), device=s["dn"].device)
    grads = {k: s[k] for k in ("dgamma_post", "dbeta_post", "dgate", "dgamma_pre", "dbeta_pre")}
    if c["q8"] == "none":
        iabn.block_norm_backward(s["u"], s["h_out"], s["dh_out"], s["dn"], s["dh"], s["du"], s["workspace"],
                                 mean_post=s["mean_post"], rstd_post=s["rstd_post"], mean_pre=s["mean_pre"],
                                 rstd_pre=s["rstd_pre"], **how, **grads)
    else:
        iabn.block_norm_backward_checkpoint8(s["q_post"], s["q_pre"], s["dh_out"], s["dn"], s["dh"], s["du"], s["workspace"],
                                             scale_post=s["scale_post"], rstd_post=s["rstd_post"], scale_pre=s["scale_pre"],
                                             rstd_pre=s["rstd_pre"], **how, **grads)
    return {"dh": s["dh"], "du": s["du"]} | {k: v for k, v in grads.items() if v is not None}


def _own_gated(s):
    import place_batchnorm_activation_b200 as iabn
    c = s["case"]
    act = {"silu": iabn.IABN_GLU_SILU, "gelu": iabn.IABN_GLU_GELU, "gelu_tanh": iabn.IABN_GLU_GELU_TANH}[c["act"]]
    if c["op"] == "gated_fwd":
        if c["q8"] == "none":
            iabn.gated_forward(s["a"], s["b"], s["z"], act=act)
            return {"z": s["z"]}
        iabn.gated_forward_checkpoint8(s["a"], s["b"], s["z"], s["qa"], s["scale_a"], s["qb"], s["scale_b"], act=act)
        return {k: s[k] for k in ("z", "qa", "scale_a", "qb", "scale_b")}
    if c["q8"] == "none":
        iabn.gated_backward(s["a"], s["b"], s["dz"], s["da"], s["db"], z=s["z"], act=act)
    else:
        iabn.gated_backward_checkpoint8(s["qa"], s["scale_a"], s["qb"], s["scale_b"], s["dz"], s["da"], s["db"], z=s["z"], act=act)
    return {"da": s["da"], "db": s["db"]} | ({"z": s["z"]} if c["again"] else {})


def _own_checkpoint(s):
    import place_batchnorm_activation_b200 as iabn
    if s["case"]["op"] == "store":
        iabn.checkpoint8_store(s["x"], s["q"], s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    iabn.checkpoint8_load(s["q"], s["scale"], s["y"], gamma=s["gamma"], beta=s["beta"])
    return {"y": s["y"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return _own_norm(state) if op.startswith("norm") else _own_gated(state) if op.startswith("gated") else _own_checkpoint(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "gated_fwd": _plain_gated_fwd,
            "gated_bwd": _plain_gated_bwd, "store": _plain_store, "load": _plain_load}[op](state)


# --------------------------------------------------------------------- work

def work(case):
    rows, cols, op = case["rows"], case["cols"], case["op"]
    e, s = rows * cols, DTYPE[case["dtype"]].itemsize
    kept = case["q8"] == "none"
    code = e + 4 * rows * _groups(cols)  # codes and scales of one tensor
    if op.startswith("norm"):
        post = case["post"] != "none"
        stats = 4 * rows * (1 + post)
        if kept:
            stats += 4 * rows * ((case["pre"] == "layer") + (case["post"] == "layer"))
        gates = 0 if case["gate"] < 0 else 4 * cols * (1 if case["gate"] == 0 else -(-rows // case["gate"]))
        params = 4 * cols * (1 + post) * (1 + case["bias"])
        if op == "norm_fwd":
            return {"bytes": 4 * e * s + (0 if kept else 2 * code) + stats + params + gates, "flops": 16 * e}
        wants_u = post or case["gate"] >= 0
        saved = (e * s if kept else code) * (1 + wants_u)
        return {"bytes": 4 * e * s + saved + stats + 2 * (params + gates), "flops": 32 * e}
    if op == "gated_fwd":
        return {"bytes": 3 * e * s + (0 if kept else 2 * code), "flops": 12 * e}
    if op == "gated_bwd":
        return {"bytes": (3 + case["again"]) * e * s + (2 * e * s if kept else 2 * code), "flops": 20 * e}
    params = 0 if op == "store" else 4 * cols * (1 + case["bias"])
    return {"bytes": e * s + code + params, "flops": 3 * e}


# ------------------------------------------------------------------ 64 bits

def _exact_scale(v, form):
    cols = v.shape[1]
    return torch.stack([v[:, k:k + GROUP].abs().amax(1) for k in range(0, cols, GROUP)], 1) / QMAX[form]


def _exact_codes(v, form):
    """(the codes before their rounding, the scales); whole codes have no value between."""
    scale = _exact_scale(v, form)
    if form == "int8":
        return None, scale
    wide = torch.cat([scale[:, k:k + 1].expand(-1, min(GROUP, v.shape[1] - k * GROUP)) for k in range(scale.shape[1])], 1)
    return torch.where(wide > 0, v / wide.clamp_min(1e-300), 0.0), scale


def _exact_values(codes, scale):
    v = codes.double()
    for k in range(scale.shape[1]):
        v[:, k * GROUP:(k + 1) * GROUP] *= scale[:, k:k + 1].double()
    return v


def _exact_stats(x, kind):
    if kind == "none":
        return None, None
    mean = x.sum(1) / x.shape[1] if kind == "layer" else None
    second = torch.einsum("rd,rd->r", x, x) / x.shape[1]
    if kind == "layer":
        y = x - mean[:, None]
        second = torch.einsum("rd,rd->r", y, y) / x.shape[1]
    return mean, (second + EPS) ** -0.5


def _exact_hat(x, mean, rstd):
    y = x.clone() if mean is None else x - mean[:, None].double()
    return y if rstd is None else y * rstd[:, None].double()


def _exact_norm(s):
    c = s["case"]
    rows, cols = c["rows"], c["cols"]
    one = torch.ones(cols, dtype=torch.float64, device="cuda")
    gamma = one if s["gamma_post"] is None else s["gamma_post"].double()
    beta = 0 * one if s["beta_post"] is None else s["beta_post"].double()
    gate = one[None] if s["gate"] is None else s["gate"].double()
    which = torch.arange(rows, device="cuda") // c["gate"] if c["gate"] > 0 else torch.zeros(rows, dtype=torch.int64, device="cuda")
    if c["op"] == "norm_fwd":
        u = s["u"].double()
        mean_post, rstd_post = _exact_stats(u, c["post"])
        uhat = _exact_hat(u, mean_post, rstd_post)
        hout = torch.addcmul(gate[which] * (gamma * uhat + beta), s["h"].double(), torch.full_like(one, c["alpha"]))
        mean_pre, rstd_pre = _exact_stats(hout, c["pre"])
        xhat = _exact_hat(hout, mean_pre, rstd_pre)
        n = xhat * s["gamma_pre"].double() + (0.0 if s["beta_pre"] is None else s["beta_pre"].double())
        out = {"h_out": hout, "n": n, "rstd_post": rstd_post, "rstd_pre": rstd_pre}
        if c["q8"] == "none":
            return out | {"mean_post": mean_post, "mean_pre": mean_pre}
        out["q_post"], out["scale_post"] = _exact_codes(uhat, c["q8"])
        out["q_pre"], out["scale_pre"] = _exact_codes(xhat, c["q8"])
        return out
    if c["q8"] == "none":
        uhat = _exact_hat(s["u"].double(), s["mean_post"], s["rstd_post"])
        xhat = _exact_hat(s["h_out"].double(), s["mean_pre"], s["rstd_pre"])
    else:
        uhat, xhat = _exact_values(s["q_post"], s["scale_post"]), _exact_values(s["q_pre"], s["scale_pre"])
    dn = s["dn"].double()
    g = dn * s["gamma_pre"].double()
    slope = torch.einsum("rd,rd->r", g, xhat) / cols
    level = g.sum(1) / cols if c["pre"] == "layer" else 0 * slope
    t = s["dh_out"].double() + s["rstd_pre"].double()[:, None] * (g - level[:, None] - slope[:, None] * xhat)
    du = t * gate[which] * gamma
    if c["post"] != "none":
        slope = torch.einsum("rd,rd->r", du, uhat) / cols
        level = du.sum(1) / cols if c["post"] == "layer" else 0 * slope
        du = s["rstd_post"].double()[:, None] * (du - level[:, None] - slope[:, None] * uhat)
    out = {"dh": c["alpha"] * t, "du": du, "dgamma_pre": torch.einsum("rd,rd->d", dn, xhat)}
    with_u = torch.zeros_like(gate).index_add_(0, which, t * uhat)
    alone = torch.zeros_like(gate).index_add_(0, which, t)
    if s["beta_pre"] is not None:
        out["dbeta_pre"] = dn.sum(0)
    if s["gamma_post"] is not None:
        out["dgamma_post"] = (gate * with_u).sum(0)
    if s["beta_post"] is not None:
        out["dbeta_post"] = (gate * alone).sum(0)
    if s["gate"] is not None:
        out["dgate"] = gamma * with_u + beta * alone
    return out


def _exact_gated(s):
    c = s["case"]
    if c["op"] == "gated_fwd" or c["q8"] == "none":
        a, b = s["a"].double(), s["b"].double()
    else:
        a, b = _exact_values(s["qa"], s["scale_a"]), _exact_values(s["qb"], s["scale_b"])
    # phi(a) = a*w(a): phi' = w + a*w'
    if c["act"] == "silu":
        w = torch.sigmoid(a)
        dw = w * torch.sigmoid(-a)
    elif c["act"] == "gelu":
        w = 0.5 * torch.erfc(-a / math.sqrt(2.0))
        dw = torch.exp(-a.square() / 2) / math.sqrt(2 * math.pi)
    else:
        k = 2 * math.sqrt(2.0 / math.pi)
        w = torch.sigmoid(k * (a + 0.044715 * a ** 3))  # (1 + tanh x)/2 = sigmoid(2x)
        dw = w * (1 - w) * k * (1 + 0.134145 * a.square())
    if c["op"] == "gated_fwd":
        out = {"z": a * w * b}
        if c["q8"] != "none":
            out["qa"], out["scale_a"] = _exact_codes(a, c["q8"])
            out["qb"], out["scale_b"] = _exact_codes(b, c["q8"])
        return out
    dz = s["dz"].double()
    out = {"da": dz * b * (w + a * dw), "db": dz * a * w}
    return out | {"z": a * w * b} if c["again"] else out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("norm"):
        return _exact_norm(s)
    if case["op"].startswith("gated"):
        return _exact_gated(s)
    if case["op"] == "store":
        q, scale = _exact_codes(s["x"].double(), case["q8"])
        return {"q": q, "scale": scale}
    y = _exact_values(s["q"], s["scale"]) * s["gamma"].double()
    return {"y": y if s["beta"] is None else y + s["beta"].double()}
