"""Plain 64-bit forms of the row operators (iabn_block.h) on CPU tensors, each
with a bound of the error that the 32-bit arithmetic of a kernel may have.

Bounds.  U = 2^-24 is half a step of fp32, relative.  A sum of terms w_i that
passes through a chain of at most L fp32 additions is off by at most
L U sum |w_i| (first order).  In a row's sums a lane adds at most 32 elements
before trees of at most 5 + 5 levels; K = 64 covers these, the division by the
width, eps and the root.  A column's sum over R rows passes through at most R
additions whatever their order.  Then, to first order:
  mean      K U mean|v|                        (+ the mean of v's own error)
  rstd      K U rstd                           (+ rstd^2 rms of v's own error)
  vhat      K U (|vhat| + rstd mean|v|)        (+ rstd (e + mean e) + |vhat| rstd rms(e))
and products, sums and differences add 4 U of the size of their terms.  A
rounding to the storage type t adds eps(t)/2 of the value and, in fp16, at most
half its smallest step.
"""
import math

import torch

U = 2.0 ** -24
K = 64.0
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -149}
GROUP = 128
QMAX = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
NONE, RMS, LAYER = 0, 1, 2


def stored(want, err, dtype):
    """The bound after a rounding to `dtype`."""
    half = torch.finfo(dtype).eps / 2
    return err + half * (want.abs() + err) + TINY[dtype]


def check(got, want, bound, what):
    got = got.detach().cpu().double().reshape(want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    ok = ~torch.isnan(want)
    off = (got - want).abs()[ok] / bound.expand(want.shape)[ok]
    off = torch.where(got[ok] == want[ok], torch.zeros_like(off), off)
    if off.numel() and not float(off.max()) <= 1.0:
        k = int(off.argmax())
        raise AssertionError(f"{what}: {int((off > 1).sum())} of {off.numel()} out of tolerance, worst "
                             f"{float(off.max()):.3g} x: got {float(got[ok][k])!r} want {float(want[ok][k])!r}")


def groups(cols):
    return -(-cols // GROUP)


def quantise(x, form):
    """The stated rounding of a float32 tensor, in fp32 arithmetic: codes and scales."""
    rows, cols = x.shape
    g = groups(cols)
    p = torch.nn.functional.pad(x, (0, g * GROUP - cols)).reshape(rows, g, GROUP)
    amax = p.abs().amax(-1)
    by = torch.full_like(amax, QMAX[form]) / amax
    flat = amax < 2.0 ** -110
    by = torch.where(flat, torch.zeros_like(by), by)
    scale = torch.where(flat, torch.zeros_like(amax), amax * torch.tensor(1.0 / QMAX[form]))
    bad = ~torch.isfinite(p).all(-1)
    scale = torch.where(bad, torch.full_like(scale, math.nan), scale)
    by = torch.where(bad, torch.zeros_like(by), by)
    v = (p * by[..., None]).reshape(rows, g * GROUP)[:, :cols]
    codes = v.to(form) if form == torch.float8_e4m3fn else torch.nan_to_num(v).round().to(torch.int8)
    return codes.contiguous(), scale


def wide(scale, cols):
    return scale.double().repeat_interleave(GROUP, 1)[:, :cols]


def values(codes, scale):
    """What codes stand for, and the error of the kernel's fp32 product."""
    v = codes.cpu().to(torch.float32).double() * wide(scale.cpu(), codes.shape[1])
    return v, U * v.abs()


def code_bound(want, err, scale, form):
    """How far the value of a code may be from `want` (known to within err)."""
    s = wide(scale.cpu(), want.shape[1])
    if form == torch.int8:
        return err + s * (0.5 + 1e-4)
    return err + torch.maximum((want.abs() + err) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-4)


def norm(v, e, kind, eps):
    """(vhat, its error, mean, its error, rstd, its error) of the rows of v, known to within e."""
    if kind == NONE:
        return v, e, None, None, None, None
    absmean = v.abs().mean(-1, keepdim=True)
    mean, merr = torch.zeros_like(absmean), torch.zeros_like(absmean)
    if kind == LAYER:
        mean, merr = v.mean(-1, keepdim=True), K * U * absmean + e.mean(-1, keepdim=True)
    c = v - mean
    rstd = ((c * c).mean(-1, keepdim=True) + eps) ** -0.5
    # vhat's own error goes through both the numerator and rstd
    d = e + merr
    rms = (d * d).mean(-1, keepdim=True).sqrt()
    rerr = rstd * (K * U + rstd * rms)
    vhat = c * rstd
    err = rstd * d + vhat.abs() * rerr / rstd + 4 * U * vhat.abs()
    return vhat, err, mean[:, 0], merr[:, 0], rstd[:, 0], rerr[:, 0]


def _col(p, like):
    return like if p is None else p.cpu().double()


def gate_rows(gate, rows_per_gate, rows, cols):
    if gate is None:
        return torch.ones(1, cols, dtype=torch.float64)
    g = gate.cpu().double().reshape(-1, cols)
    return g[torch.arange(rows) // rows_per_gate] if rows_per_gate else g


def forward(u, h, o):
    """{name: (value, bound before storage)} of the block norm's forward; `o` holds the parameters."""
    rows, cols = h.shape
    one, zero = torch.ones(cols, dtype=torch.float64), torch.zeros(cols, dtype=torch.float64)
    h = h.cpu().double()
    out = {}
    if u is None:
        hout, e = h, torch.zeros_like(h)
    else:
        u = u.cpu().double()
        uhat, eu, mean, merr, rstd, rerr = norm(u, torch.zeros_like(u), o["post"], o["eps_post"])
        out["uhat"] = (uhat, eu)
        if rstd is not None:
            out["rstd_post"], out["mean_post"] = (rstd, rerr), (mean, merr)
        ga, be = _col(o["gamma_post"], one), _col(o["beta_post"], zero)
        gate = gate_rows(o["gate"], o["rows_per_gate"], rows, cols)
        p = ga * uhat + be
        hout = o["residual_scale"] * h + gate * p
        e = gate.abs() * (ga.abs() * eu + 4 * U * ((ga * uhat).abs() + be.abs())) \
            + 4 * U * ((o["residual_scale"] * h).abs() + (gate * p).abs())
    out["h_out"] = (hout, e)
    if o["pre"] != NONE:
        xhat, ex, mean, merr, rstd, rerr = norm(hout, e, o["pre"], o["eps_pre"])
        out["xhat"], out["rstd_pre"], out["mean_pre"] = (xhat, ex), (rstd, rerr), (mean, merr)
        ga, be = _col(o["gamma_pre"], one), _col(o["beta_pre"], zero)
        out["n"] = (ga * xhat + be, ga.abs() * ex + 4 * U * ((ga * xhat).abs() + be.abs()))
    return out


def kept_hat(v, mean, rstd):
    """(v - mean)*rstd of a kept tensor with the forward's own statistics, and its error."""
    v = v.cpu().double()
    m = torch.zeros(v.shape[0], 1, dtype=torch.float64) if mean is None else mean.cpu().double()[:, None]
    r = torch.ones(v.shape[0], 1, dtype=torch.float64) if rstd is None else rstd.cpu().double()[:, None]
    return (v - m) * r, 3 * U * (v.abs() + m.abs()) * r


def backward(uhat, eu, xhat, ex, dh_out, dn, o):
    """{name: (value, bound before storage)} of the block norm's backward from the normalised values
    (known to within eu, ex), with o["rstd_post"], o["rstd_pre"] as the call gets them."""
    like = dh_out if dh_out is not None else dn
    rows, cols = like.shape
    one, zero = torch.ones(cols, dtype=torch.float64), torch.zeros(cols, dtype=torch.float64)
    mean = lambda v: v.mean(-1, keepdim=True)  # noqa: E731
    t = torch.zeros(rows, cols, dtype=torch.float64) if dh_out is None else dh_out.cpu().double()
    et = torch.zeros_like(t)
    out = {}

    def through(g, eg, v, ev, kind, rstd):
        """rstd*(g - [mean g] - v mean(g v)) and its error."""
        if kind == NONE:
            return g, eg
        level = mean(g) if kind == LAYER else torch.zeros(rows, 1, dtype=torch.float64)
        elevel = (mean(eg) + K * U * mean(g.abs())) if kind == LAYER else 0.0
        slope = mean(g * v)
        eslope = mean(eg * v.abs() + g.abs() * ev) + K * U * mean((g * v).abs())
        r = rstd.cpu().double()[:, None]
        err = eg + elevel + v.abs() * eslope + slope.abs() * ev \
            + 4 * U * (g.abs() + level.abs() + (v * slope).abs())
        return r * (g - level - v * slope), r * err

    if o["pre"] != NONE:
        n = dn.cpu().double()
        g = n * _col(o["gamma_pre"], one)
        d, ed = through(g, U * g.abs(), xhat, ex, o["pre"], o["rstd_pre"])
        t, et = t + d, ed + 4 * U * (t.abs() + d.abs())
        out["dgamma_pre"] = ((n * xhat).sum(0), (rows * U * (n * xhat).abs() + n.abs() * ex).sum(0))
        out["dbeta_pre"] = (n.sum(0), rows * U * n.abs().sum(0))
    out["dh"] = (o["residual_scale"] * t, abs(o["residual_scale"]) * (et + 2 * U * t.abs()))
    ga, be = _col(o["gamma_post"], one), _col(o["beta_post"], zero)
    gate = gate_rows(o["gate"], o["rows_per_gate"], rows, cols)
    e = t * gate * ga
    if uhat is None:
        uhat, eu = torch.zeros_like(t), torch.zeros_like(t)
    out["du"] = through(e, (gate * ga).abs() * et + 4 * U * e.abs(), uhat, eu, o["post"], o["rstd_post"])
    which = torch.arange(rows) // o["rows_per_gate"] if o["rows_per_gate"] else torch.zeros(rows, dtype=torch.int64)
    n_gates = 1 if not o["rows_per_gate"] else -(-rows // o["rows_per_gate"])
    by_gate = lambda v: torch.zeros(n_gates, cols, dtype=torch.float64).index_add_(0, which, v)  # noqa: E731
    A, B = by_gate(t * uhat), by_gate(t)
    L = (rows + 8) * U
    eA = by_gate(et * uhat.abs() + t.abs() * eu + L * (t * uhat).abs())
    eB = by_gate(et + L * t.abs())
    sA, sB = by_gate((t * uhat).abs()), by_gate(t.abs())
    G = gate_rows(o["gate"], 0, rows, cols) if o["gate"] is not None else gate.expand(n_gates, cols)
    out["dgate"] = (ga * A + be * B, ga.abs() * (eA + 4 * U * sA) + be.abs() * (eB + 4 * U * sB))
    out["dgamma_post"] = ((G * A).sum(0), (G.abs() * (eA + L * sA)).sum(0))
    out["dbeta_post"] = ((G * B).sum(0), (G.abs() * (eB + L * sB)).sum(0))
    return out


def phi(a, act):
    """(w, a w') with phi = a w, in 64 bits; act 0 silu, 1 gelu, 2 gelu by tanh."""
    if act == 0:
        w = torch.sigmoid(a)
        return w, a * w * torch.sigmoid(-a)
    if act == 1:
        return 0.5 * torch.erfc(-a * math.sqrt(0.5)), a * torch.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    y = k * (a + 0.044715 * a ** 3)
    w = torch.sigmoid(y)
    return w, a * w * torch.sigmoid(-y) * k * (1 + 3 * 0.044715 * a * a)


def phi_error(a, act, dtype):
    """Error of w and of a w' in a kernel.  The exponent of e^x is off by a few
    U |x| (|x| up to 88 counts), the fast exponential and division of the
    16-bit types by a few more; erfc by a few ulp of itself plus its argument's
    rounding (U x^2 relative)."""
    w, aw = phi(a, act)
    x = a.abs() if act == 0 else a * a if act == 1 else (1.6 * (a.abs() + 0.045 * a.abs() ** 3))
    rel = U * (32 + 8 * x.clamp(max=100.0))
    # e^x below the smallest normal number of fp32 may be flushed
    return rel * w + 2.0 ** -120, rel * (aw.abs() + a.abs() * w) + 2.0 ** -120


def gated(a, b, act, dtype, ea=0.0, eb=0.0, dz=None):
    """{name: (value, bound before storage)}; a, b in 64 bits, known to within ea, eb."""
    w, aw = phi(a, act)
    ew, eaw = phi_error(a, act, dtype)
    # |phi'| <= 1.13, |phi''| <= 1 of all three
    p, ep = a * w, a.abs() * ew + 1.2 * ea + 2 * U * (a * w).abs()
    out = {"z": (p * b, ep * b.abs() + p.abs() * eb + 4 * U * (p * b).abs())}
    if dz is None:
        return out
    s, es = w + aw, ew + eaw + 1.0 * ea + 4 * U * (w + aw.abs())
    out["da"] = (dz * b * s, (dz * b).abs() * es + (dz * s).abs() * eb + 4 * U * (dz * b * s).abs())
    out["db"] = (dz * p, dz.abs() * ep + 4 * U * (dz * p).abs())
    return out
