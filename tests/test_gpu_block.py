"""The row operators (iabn_block.h) on the GPU against their 64-bit forms
(block_ref, which derives the bounds), over types, widths, norms, gates and
checkpoint formats; then what a program does with them: in place, on other
streams, captured, strided, empty, very large, and all together.

Every output sits between guard bands, so a write outside it fails the test."""
import math

import pytest

import block_ref as ref
from gpu_util import Guarded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import place_batchnorm_activation_b200 as iabn  # noqa: E402

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4M3, INT8 = torch.float8_e4m3fn, torch.int8
NONE, RMS, LAYER = 0, 1, 2
EPS = {"eps_post": 1e-5, "eps_pre": 1e-4}


class Buffers:
    """Guarded outputs by name."""

    def __init__(self):
        self.g = {}

    def new(self, name, shape, dtype, fill=None):
        numel = math.prod(shape)
        b = Guarded(numel, torch.uint8 if dtype == E4M3 else dtype, "cuda")
        if dtype in (F32, BF16, F16):
            b.t.fill_(float("nan"))       # an element that is not written shows
        if fill is not None:
            b.t.copy_(fill.reshape(-1))
        self.g[name] = b
        t = b.t.view(E4M3) if dtype == E4M3 else b.t
        return t.view(shape)

    def intact(self):
        torch.cuda.synchronize()
        bad = [k for k, v in self.g.items() if not v.intact()]
        assert not bad, f"written outside {bad}"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def values(rows, cols, dtype, seed, size=1.0, level=0.0):
    g = gen(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(0.5 * torch.randn(cols, generator=g)) * size
    x[:, seed % cols] *= 30.0               # an outlying column
    x += level * torch.randn(rows, 1, generator=g)
    return x.to(dtype).cuda()


def params(rows, cols, post, pre, gated, per, bias, seed):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    n_gates = 1 if per == 0 else -(-rows // per)
    on = lambda k, v: v if k else None  # noqa: E731
    return dict(post=post, pre=pre, rows_per_gate=per, residual_scale=0.7,
                gamma_post=on(post, 1 + 0.3 * r(cols)), beta_post=on(post and bias, r(cols)),
                gate=on(gated, 0.5 + 0.5 * r(n_gates, cols)), gamma_pre=on(pre, 1 + 0.3 * r(cols)),
                beta_pre=on(pre and bias, r(cols)))


def run_forward(u, h, o, form=None, buf=None, **kw):
    """The forward's outputs by name (None where the case has none)."""
    rows, cols = h.shape
    buf = buf or Buffers()
    out = {"h_out": buf.new("h_out", (rows, cols), h.dtype) if u is not None else None,
           "n": buf.new("n", (rows, cols), h.dtype) if o["pre"] else None}
    row = lambda k, on: buf.new(k, (rows,), F32) if on else None  # noqa: E731
    out["rstd_post"], out["rstd_pre"] = row("rstd_post", o["post"]), row("rstd_pre", o["pre"])
    if form is None:
        out["mean_post"] = row("mean_post", o["post"] == LAYER)
        out["mean_pre"] = row("mean_pre", o["pre"] == LAYER)
        call = iabn.block_norm_forward
    else:
        g = ref.groups(cols)
        for k, on in (("post", u is not None), ("pre", o["pre"])):
            out["q_" + k] = buf.new("q_" + k, (rows, cols), form) if on else None
            out["scale_" + k] = buf.new("scale_" + k, (rows, g), F32) if on else None
        call = iabn.block_norm_forward_checkpoint8
    stats = {k: v for k, v in out.items() if k not in ("h_out", "n")}
    call(u, h, out["h_out"], out["n"], **{**EPS, **o}, **stats, **kw)
    buf.intact()
    return out


def check_forward(u, h, o, form, got, what):
    want = ref.forward(u, h, {**EPS, **o})
    for k in ("h_out", "n"):
        if got[k] is not None:
            v, e = want[k]
            ref.check(got[k], v, ref.stored(v, e, h.dtype), f"{what} {k}")
    for k in ("rstd_post", "rstd_pre", "mean_post", "mean_pre"):
        if got.get(k) is not None:
            v, e = want[k]
            ref.check(got[k], v, ref.stored(v, e, F32), f"{what} {k}")
    if form is None:
        return
    for k, hat in (("post", "uhat"), ("pre", "xhat")):
        q, s = got["q_" + k], got["scale_" + k]
        if q is None:
            continue
        v, e = want[hat]
        read, _ = ref.values(q, s)
        ref.check(read, v, ref.code_bound(v, e, s, form) + 1e-30, f"{what} code {k}")
        # the largest of a group takes the format's largest code
        top = torch.nn.functional.pad(q.cpu().float().abs(), (0, -q.shape[1] % 128)).view(q.shape[0], -1, 128).amax(-1)
        assert ((top == ref.QMAX[form]) | (s.cpu() == 0)).all(), f"{what} {k}: codes do not fill their range"


def run_backward(src_u, src_x, dh_out, dn, o, stats, buf=None, want=None, **kw):
    """src_*: the kept tensor or (codes, scales).  want: names of the parameter gradients."""
    like = dh_out if dh_out is not None else dn
    rows, cols = like.shape
    buf = buf or Buffers()
    out = {"dh": buf.new("dh", (rows, cols), like.dtype), "du": buf.new("du", (rows, cols), like.dtype)}
    for k in ("gamma_post", "beta_post", "gate", "gamma_pre", "beta_pre"):
        if o[k] is not None and (want is None or "d" + k in want):
            out["d" + k] = buf.new("d" + k, tuple(o[k].shape), F32)
    ws = buf.new("ws", (iabn.block_norm_workspace_size(rows, cols, o["rows_per_gate"]),), torch.uint8)
    ws.fill_(0xff)                         # whatever it held before (NaN) is not read
    a = {k: o[k] for k in ("post", "pre", "rows_per_gate", "residual_scale", "gamma_post", "gate", "gamma_pre",
                           "beta_post")}
    grads = {k: v for k, v in out.items() if k not in ("dh", "du")}
    if isinstance(src_u, tuple) or isinstance(src_x, tuple):
        (qu, su), (qx, sx) = src_u or (None, None), src_x or (None, None)
        stats = {k: v for k, v in stats.items() if k.startswith("rstd")}
        iabn.block_norm_backward_checkpoint8(qu, qx, dh_out, dn, out["dh"], out["du"], ws, scale_post=su,
                                             scale_pre=sx, **stats, **a, **grads, **kw)
    else:
        iabn.block_norm_backward(src_u, src_x, dh_out, dn, out["dh"], out["du"], ws, **stats, **a, **grads, **kw)
    buf.intact()
    return out


def backward_want(src_u, src_x, dh_out, dn, o, stats):
    hat = lambda s, m, r: (None, None) if s is None else ref.values(*s) if isinstance(s, tuple) \
        else ref.kept_hat(s, stats.get(m), stats.get(r))  # noqa: E731
    uhat, eu = hat(src_u, "mean_post", "rstd_post")
    xhat, ex = hat(src_x, "mean_pre", "rstd_pre")
    return ref.backward(uhat, eu, xhat, ex, dh_out, dn, {**o, **stats})


def check_backward(got, want, dtype, what):
    for k, t in got.items():
        v, e = want[k]
        ref.check(t, v, ref.stored(v, e, dtype if k in ("dh", "du") else F32) + 1e-37, f"{what} {k}")


WIDTHS = [1, 2, 7, 8, 64, 127, 128, 129, 200, 256, 257, 512, 1000, 1021, 1024, 2056, 4096, 4104, 5120, 8192,
          8193, 12000, 16384, 20001, 32768]


def off_boundary(t):
    """The same values one element behind a 16-byte boundary."""
    if t is None:
        return None
    flat = torch.empty(t.numel() + 16, dtype=t.dtype, device=t.device)
    out = flat[1:1 + t.numel()].view(t.shape)
    out.copy_(t)
    return out


def one(rows, cols, dtype, post, pre, gated, per, bias, form, seed=0, place=lambda t: t):
    """Forward, then the backward from what it kept, both against 64 bits."""
    what = f"{rows}x{cols} {dtype} post {post} pre {pre} gate {gated}/{per} {form}"
    o = params(rows, cols, post, pre, gated, per, bias, seed + 3)
    u = place(values(rows, cols, dtype, seed, 1.0, 0.3))
    h = place(values(rows, cols, dtype, seed + 1, 2.0, 0.5))
    got = run_forward(u, h, o, form)
    check_forward(u, h, o, form, got, what)
    dh_out = place(values(rows, cols, dtype, seed + 5, 0.1))
    dn = place(values(rows, cols, dtype, seed + 6, 0.1)) if pre else None
    stats = {k: got.get(k) for k in ("mean_post", "rstd_post", "mean_pre", "rstd_pre") if got.get(k) is not None}
    if form is None:
        src_u, src_x = u, got["h_out"] if pre else None
    else:
        src_u = (got["q_post"], got["scale_post"])
        src_x = (got["q_pre"], got["scale_pre"]) if pre else None
    o["beta_pre"] = o["beta_pre"] if pre else None
    back = run_backward(src_u, src_x, dh_out, dn, o, {"rstd_post": None, "rstd_pre": None} | stats)
    check_backward(back, backward_want(src_u, src_x, dh_out, dn, o, {"rstd_post": None, "rstd_pre": None} | stats),
                   dtype, what)


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind,form,dtype", [(RMS, E4M3, BF16), (LAYER, None, F16), (LAYER, INT8, F32), (RMS, None, F32),
                                             (LAYER, None, F32), (LAYER, E4M3, BF16)])
def test_block_norm_widths(cols, kind, form, dtype):
    rows = 5 if cols > 8192 else 19
    one(rows, cols, dtype, kind, kind, True, 4, kind == LAYER, form, seed=cols)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("post", [NONE, RMS, LAYER])
@pytest.mark.parametrize("pre", [NONE, RMS, LAYER])
@pytest.mark.parametrize("gated,per,bias,form", [(False, 0, False, None), (True, 0, True, INT8), (True, 7, True, E4M3),
                                                 (True, 1, False, None)])
def test_block_norm_forms(dtype, post, pre, gated, per, bias, form):
    one(23, 264, dtype, post, pre, gated, per, bias, form, seed=post + 3 * pre)


@pytest.mark.parametrize("rows", [1, 2, 7, 147, 149, 296, 297, 1201])
@pytest.mark.parametrize("cols,per", [(72, 0), (72, 5), (73, 4), (520, 300), (1032, 2), (1021, 100), (4096, 64)])
def test_block_norm_rows(rows, cols, per):
    one(rows, cols, BF16, RMS, RMS, True, per, False, E4M3, seed=rows)


@pytest.mark.parametrize("dtype,form", [(BF16, E4M3), (F16, None), (F32, INT8), (F32, None)])
@pytest.mark.parametrize("cols", [1, 9, 256, 1000, 4096, 4099, 9000, 32768])
def test_block_norm_off_16_byte_boundaries(cols, dtype, form):
    one(7, cols, dtype, LAYER, LAYER, True, 3, True, form, seed=cols, place=off_boundary)
    one(7, cols, dtype, RMS, RMS, False, 0, False, form, seed=cols, place=off_boundary)


@pytest.mark.parametrize("cols", [40, 41, 1024, 9000, 9001])
@pytest.mark.parametrize("post,pre", [(RMS, LAYER), (NONE, NONE), (NONE, RMS)])
def test_block_norm_gate_of_more_rows_than_there_are(cols, post, pre):
    """One gate row that covers more rows than the call has; widths that share
    rows in clusters, with and without a norm to wait for."""
    one(6, cols, BF16, post, pre, True, 1 << 40, True, INT8, seed=cols)
    one(6, cols, F32, post, pre, True, 7, True, None, seed=cols)


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, give what they
    give one after the other."""
    rows, cols = 900, 2056
    o = params(rows, cols, RMS, LAYER, True, 300, True, 1)
    sets = []
    for k in range(2):
        u, h = values(rows, cols, BF16, 10 * k), values(rows, cols, BF16, 10 * k + 1)
        f = run_forward(u, h, o, E4M3)
        g = [values(rows, cols, BF16, 10 * k + 2), values(rows, cols, BF16, 10 * k + 3)]
        src = ((f["q_post"], f["scale_post"]), (f["q_pre"], f["scale_pre"]))
        stats = {"rstd_post": f["rstd_post"], "rstd_pre": f["rstd_pre"]}
        sets.append((src, g, stats, run_backward(*src, *g, o, stats), torch.cuda.Stream()))
    keys = ("post", "pre", "rows_per_gate", "residual_scale", "gamma_post", "beta_post", "gate", "gamma_pre")
    outs = []
    for _, g, _, want, _ in sets:
        t = {k: torch.empty_like(v) for k, v in want.items()}
        outs.append((t, iabn.new_block_norm_workspace(rows, cols, 300, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for (src, g, stats, want, stream), (t, ws) in zip(sets, outs):
            (qu, su), (qx, sx) = src
            grads = {k: v for k, v in t.items() if k not in ("dh", "du")}
            iabn.block_norm_backward_checkpoint8(qu, qx, g[0], g[1], t["dh"], t["du"], ws, scale_post=su, scale_pre=sx,
                                                 **stats, **grads, **{k: o[k] for k in keys}, stream=stream)
    torch.cuda.synchronize()
    for (_, _, _, want, _), (t, _) in zip(sets, outs):
        for k in want:
            assert torch.equal(want[k], t[k]), k


@pytest.mark.parametrize("form", [None, E4M3])
def test_block_norm_without_u_and_partial_gradients(form):
    """The norm of h alone; gradients that are not wanted are left out."""
    rows, cols = 33, 320
    o = params(rows, cols, NONE, LAYER if form is None else RMS, False, 0, True, 1) | {"residual_scale": 1.0}
    h = values(rows, cols, BF16, 2, 2.0, 1.0)
    got = run_forward(None, h, o, form)
    check_forward(None, h, o, form, got, "alone")
    dn = values(rows, cols, BF16, 3, 0.1)
    stats = {"rstd_post": None} | {k: got[k] for k in ("mean_pre", "rstd_pre") if got.get(k) is not None}
    src = h if form is None else (got["q_pre"], got["scale_pre"])
    for dh_out in (None, values(rows, cols, BF16, 4, 0.1)):
        for wanted in ((), ("dgamma_pre",), ("dgamma_pre", "dbeta_pre")):
            back = run_backward(None, src, dh_out, dn, o, stats, want=wanted)
            want = backward_want(None, src, dh_out, dn, o, stats)
            check_backward(back, want, BF16, f"alone {wanted}")
    # du not wanted, and no pre-norm: dh alone
    dh = torch.empty_like(h)
    ws = iabn.new_block_norm_workspace(rows, cols, device="cuda")
    iabn.block_norm_backward(None, None, dn, None, dh, None, ws, post=NONE, pre=NONE, residual_scale=0.5)
    assert torch.equal(dh, (dn.float() * 0.5).to(BF16))


def test_block_norm_gradient_against_differences():
    """<du, v> + <dh, w> of the kernels against the central difference of the
    64-bit forward along (v, w).  The difference quotient of step s is off by
    s^2/6 of a third derivative (about 1e-10 here) and the kernels by their
    bound, summed over the elements."""
    rows, cols = 11, 200
    o = params(rows, cols, LAYER, LAYER, True, 4, True, 8)
    u, h = values(rows, cols, F32, 1), values(rows, cols, F32, 2, 2.0)
    got = run_forward(u, h, o)
    dh_out, dn = values(rows, cols, F32, 3, 0.1), values(rows, cols, F32, 4, 0.1)
    stats = {k: got[k] for k in ("mean_post", "rstd_post", "mean_pre", "rstd_pre")}
    back = run_backward(u, got["h_out"], dh_out, dn, o, stats)
    bound = backward_want(u, got["h_out"], dh_out, dn, o, stats)
    v, w = torch.randn(rows, cols, generator=gen(5)).double(), torch.randn(rows, cols, generator=gen(6)).double()

    def loss(s):
        f = ref.forward(u.cpu().double() + s * v, h.cpu().double() + s * w, {**EPS, **o})
        return float((f["h_out"][0] * dh_out.cpu().double()).sum() + (f["n"][0] * dn.cpu().double()).sum())

    slope = (loss(1e-5) - loss(-1e-5)) / 2e-5
    along = float((back["du"].cpu().double() * v).sum() + (back["dh"].cpu().double() * w).sum())
    # h_out and the statistics are the forward's rounded ones: 2^-24 of them, seen through n's slope
    allowed = float((bound["du"][1] * v.abs()).sum() + (bound["dh"][1] * w.abs()).sum())
    assert abs(along - slope) <= 4 * allowed + 1e-6 * abs(slope)


# ------------------------------------------------------------ 8-bit checkpoints

@pytest.mark.parametrize("form", [E4M3, INT8])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols,ld", [(1, 1, 1), (3, 7, 7), (5, 128, 128), (4, 129, 131), (9, 256, 512), (7, 300, 300),
                                          (6, 1024, 1032), (3, 5120, 5120), (2, 10001, 10001)])
def test_checkpoint8_is_the_stated_rounding(form, dtype, rows, cols, ld):
    """Codes and scales are those of the stated fp32 arithmetic, bit for bit; so is
    the value read back, but for the storage type's rounding."""
    big = (torch.randn(rows, ld, generator=gen(cols)) * torch.exp(2 * torch.randn(rows, ld, generator=gen(1)))).to(dtype)
    if rows > 2:
        big[1] = 0
        big[2, 0] = 1e-30 if dtype != F16 else 6e-8
    x = big.cuda()[:, :cols]
    buf = Buffers()
    q, s = buf.new("q", (rows, cols), form), buf.new("s", (rows, ref.groups(cols)), F32)
    iabn.checkpoint8_store(x, q, s)
    buf.intact()
    want_q, want_s = ref.quantise(x.cpu().float(), form)
    assert torch.equal(q.cpu().float(), want_q.float())
    assert torch.equal(s.cpu(), want_s)
    y = buf.new("y", (rows, ld), dtype, torch.full((rows, ld), 7.0))
    iabn.checkpoint8_load(q, s, y[:, :cols])
    buf.intact()
    wide = (want_q.float() * want_s.repeat_interleave(128, 1)[:, :cols]).to(dtype)
    assert torch.equal(y[:, :cols].cpu(), wide)
    assert (y[:, cols:] == 7.0).all()
    ga, be = torch.randn(cols, generator=gen(2)).cuda(), torch.randn(cols, generator=gen(3)).cuda()
    v, e = ref.values(q, s)
    for g, b in ((ga, None), (None, be), (ga, be)):
        iabn.checkpoint8_load(q, s, y[:, :cols], gamma=g, beta=b)
        gd = torch.ones(cols) if g is None else g.cpu()
        bd = torch.zeros(cols) if b is None else b.cpu()
        w = gd.double() * v + bd.double()
        ref.check(y[:, :cols], w, ref.stored(w, gd.double().abs() * e + 2 * ref.U * (w.abs() + bd.double().abs()), dtype),
                  "load")


@pytest.mark.parametrize("form", [E4M3, INT8])
def test_checkpoint8_special_values(form):
    x = torch.randn(8, 300, generator=gen(1))
    x[1, 5], x[2, 130], x[3, 299] = math.nan, math.inf, -math.inf
    x[4] = torch.finfo(F32).max
    x[5, :128] = 7.6e-34
    x[6, :128] = 7.8e-34
    x[7] = torch.finfo(F32).tiny / 8
    q, s = torch.empty(8, 300, dtype=form, device="cuda"), torch.empty(8, 3, device="cuda")
    iabn.checkpoint8_store(x.cuda(), q, s)
    y = torch.empty(8, 300, device="cuda")
    iabn.checkpoint8_load(q, s, y)
    y = y.cpu()
    bad = torch.zeros(8, 300, dtype=torch.bool)
    bad[1, :128] = bad[2, 128:256] = bad[3, 256:] = True
    assert torch.equal(torch.isnan(y), bad)
    assert (y[5, :128] == 0).all() and (y[7] == 0).all()
    assert (y[6, :128] > 7e-34).all()
    ok = ~bad
    ok[5, :128] = ok[7] = False
    bound = ref.code_bound(x.double(), torch.zeros(8, 300).double(), s, form)
    assert ((y.double() - x.double()).abs()[ok] <= (bound + 1e-40)[ok]).all()


# ------------------------------------------------------------ gated activation

def gated_inputs(rows, cols, dtype, packed, seed=0):
    x = torch.randn(rows, 2 * cols, generator=gen(seed)) * torch.exp(0.7 * torch.randn(2 * cols, generator=gen(seed + 1)))
    x[0, : min(cols, 6)] = torch.tensor([0.0, -0.0, 20.0, -20.0, 9.0, -9.0])[: min(cols, 6)]
    x = x.to(dtype).cuda()
    if packed:
        return x[:, :cols], x[:, cols:]
    return x[:, :cols].contiguous(), x[:, cols:].contiguous()


@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("rows,cols,packed", [(1, 1, False), (3, 7, True), (2, 128, True), (5, 264, False), (4, 1000, True),
                                              (3, 2731, True), (2, 11008, True), (700, 136, True)])
def test_gated_activation(act, dtype, rows, cols, packed):
    a, b = gated_inputs(rows, cols, dtype, packed, seed=cols)
    dz = values(rows, cols, dtype, 9, 0.1)
    A, B, Z = a.cpu().double(), b.cpu().double(), dz.cpu().double()
    for form in (None, E4M3, INT8):
        buf = Buffers()
        z = buf.new("z", (rows, cols), dtype)
        grads = buf.new("grads", (rows, 2 * cols), dtype)
        da, db = grads[:, :cols], grads[:, cols:]
        again = buf.new("again", (rows, cols), dtype)
        want = ref.gated(A, B, act, dtype, dz=Z)
        if form is None:
            iabn.gated_forward(a, b, z, act=act)
            iabn.gated_backward(a, b, dz, da, db, z=again, act=act)
            back = want
        else:
            g = ref.groups(cols)
            qa, sa = buf.new("qa", (rows, cols), form), buf.new("sa", (rows, g), F32)
            qb, sb = buf.new("qb", (rows, cols), form), buf.new("sb", (rows, g), F32)
            iabn.gated_forward_checkpoint8(a, b, z, qa, sa, qb, sb, act=act)
            for x, q, s in ((a, qa, sa), (b, qb, sb)):
                wq, ws = ref.quantise(x.cpu().float(), form)
                assert torch.equal(q.cpu().float(), wq.float()) and torch.equal(s.cpu(), ws)
            iabn.gated_backward_checkpoint8(qa, sa, qb, sb, dz, da, db, z=again, act=act)
            va, ea = ref.values(qa, sa)
            vb, eb = ref.values(qb, sb)
            back = ref.gated(va, vb, act, dtype, ea, eb, dz=Z)
        buf.intact()
        for k, got, w in (("z", z, want), ("z", again, back), ("da", da, back), ("db", db, back)):
            v, e = w[k]
            ref.check(got, v, ref.stored(v, e, dtype) + 1e-36, f"{act} {form} {k}")
        # without z the gradients are the same bits
        other = torch.empty_like(grads)
        if form is None:
            iabn.gated_backward(a, b, dz, other[:, :cols], other[:, cols:], act=act)
        else:
            iabn.gated_backward_checkpoint8(qa, sa, qb, sb, dz, other[:, :cols], other[:, cols:], act=act)
        assert torch.equal(other.view(torch.uint8), grads.view(torch.uint8))


@pytest.mark.parametrize("act", [0, 1, 2])
def test_gated_activation_far_values(act):
    """Where phi is 0 or a, its slope 0 or 1, up to the largest numbers."""
    a = torch.tensor([[40.0, 200.0, 1e4, 1e15, 1e30, 3e38, -40.0, -200.0, -1e4, -1e15, -1e30, -3e38]]).cuda()
    one = torch.ones_like(a)
    z, da, db = torch.empty_like(a), torch.empty_like(a), torch.empty_like(a)
    iabn.gated_backward(a, one, one, da, db, z=z, act=act)
    up = a > 0
    assert torch.equal(z[up], a[up]) and torch.equal(db[up], a[up]) and torch.equal(da[up], one[up])
    assert (z[~up].abs() < 1e-15).all() and (db[~up].abs() < 1e-15).all() and (da[~up].abs() < 1e-14).all()


# ------------------------------------------------------------ how they are used

def test_in_place():
    rows, cols = 37, 520
    o = params(rows, cols, LAYER, LAYER, True, 0, True, 1)
    u, h = values(rows, cols, BF16, 2), values(rows, cols, BF16, 3, 2.0)
    want = run_forward(u, h, o)
    for swap in (False, True):
        u2, h2 = u.clone(), h.clone()
        ho, n = (u2, h2) if swap else (h2, u2)
        iabn.block_norm_forward(u2, h2, ho, n, **{**EPS, **o})
        assert torch.equal(ho, want["h_out"]) and torch.equal(n, want["n"])
    dh_out, dn = values(rows, cols, BF16, 4, 0.1), values(rows, cols, BF16, 5, 0.1)
    stats = {k: want[k] for k in ("mean_post", "rstd_post", "mean_pre", "rstd_pre")}
    back = run_backward(u, want["h_out"], dh_out, dn, o, stats)
    ws = iabn.new_block_norm_workspace(rows, cols, device="cuda")
    keys = ("post", "pre", "rows_per_gate", "residual_scale", "gamma_post", "gate", "gamma_pre")
    for a, b in ((0, 1), (1, 0), (2, 3), (3, 2), (0, 2), (3, 1)):
        t = [dh_out.clone(), dn.clone(), u.clone(), want["h_out"].clone()]
        iabn.block_norm_backward(t[2], t[3], t[0], t[1], t[a], t[b], ws, **stats, **{k: o[k] for k in keys})
        assert torch.equal(t[a], back["dh"]) and torch.equal(t[b], back["du"]), (a, b)
    p = values(rows, 2 * cols, BF16, 6)
    a, b = p[:, :cols], p[:, cols:]
    dz = values(rows, cols, BF16, 7)
    want, z = torch.empty_like(p), torch.empty_like(dz)
    iabn.gated_backward(a, b, dz, want[:, :cols], want[:, cols:], z=z)
    iabn.gated_backward(a, b, dz, a, b, z=dz)
    assert torch.equal(p, want) and torch.equal(dz, z)


@pytest.mark.parametrize("cols", [72, 73, 264, 2048, 2049, 8192])
def test_a_bad_row_stays_in_its_row(cols):
    """NaN and infinities in one row change no bit of the others."""
    rows = 21
    o = params(rows, cols, LAYER, LAYER, True, 0, True, 1)
    u, h = values(rows, cols, F32, 2), values(rows, cols, F32, 3)
    clean = run_forward(u, h, o, INT8)
    bad_u, bad_h = u.clone(), h.clone()
    bad_u[3, cols - 1], bad_u[9, 0], bad_h[14, cols // 2] = math.nan, math.inf, -math.inf
    got = run_forward(bad_u, bad_h, o, INT8)
    rest = [r for r in range(rows) if r not in (3, 9, 14)]
    for k, t in got.items():
        assert torch.equal(t[rest], clean[k][rest]), k
        if k in ("n",):
            assert torch.isnan(t[[3, 9, 14]]).all(), k
    assert torch.isnan(got["scale_post"][[3, 9]]).all() and torch.isnan(got["scale_pre"][[3, 9, 14]]).all()


def test_zero_rows_and_constant_rows():
    o = params(4, 256, LAYER, RMS, False, 0, False, 1)
    u = torch.zeros(4, 256, device="cuda", dtype=BF16)
    u[1] = 1000.0
    u[2] = torch.randn(256, generator=gen(1)).to(BF16).cuda() + 10000
    u[3, 7] = 1e-3
    h = torch.zeros(4, 256, device="cuda", dtype=BF16)
    for form in (None, E4M3, INT8):
        got = run_forward(u, h, o, form)
        check_forward(u, h, o, form, got, "constant rows")
        assert (got["n"][:2] == 0).all()


def test_no_rows():
    e = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    x, cols = e(0, 64), 64
    q, s = e(0, 64, dtype=INT8), e(0, 1, dtype=F32)
    iabn.block_norm_forward(x, x, x, x)
    iabn.block_norm_forward_checkpoint8(x, x, x, x, q_post=q, scale_post=s, q_pre=q, scale_pre=s)
    iabn.gated_forward(x, x, x)
    iabn.gated_forward_checkpoint8(x, x, x, q, s, q, s)
    iabn.gated_backward_checkpoint8(q, s, q, s, x, x, x)
    iabn.checkpoint8_store(x, q, s)
    iabn.checkpoint8_load(q, s, x)
    before = iabn.iabn_kernel_launches()
    g = {k: torch.full((cols,), math.nan, device="cuda") for k in ("dgamma_post", "dbeta_post", "dgate", "dgamma_pre",
                                                                   "dbeta_pre")}
    gate = torch.ones(cols, device="cuda")
    iabn.block_norm_backward(x, x, x, x, x, x, iabn.new_block_norm_workspace(0, cols, device="cuda"), gate=gate, **g)
    assert all((v == 0).all() for v in g.values())
    assert iabn.iabn_kernel_launches() == before + 1


def test_repeats_give_the_same_bits_and_other_streams_work():
    rows, cols = 777, 1032
    o = params(rows, cols, RMS, RMS, True, 100, False, 1)
    u, h = values(rows, cols, BF16, 2), values(rows, cols, BF16, 3)
    dh_out, dn = values(rows, cols, BF16, 4), values(rows, cols, BF16, 5)
    f = run_forward(u, h, o, E4M3)
    src = ((f["q_post"], f["scale_post"]), (f["q_pre"], f["scale_pre"]))
    stats = {"rstd_post": f["rstd_post"], "rstd_pre": f["rstd_pre"]}
    b = run_backward(*src, dh_out, dn, o, stats)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for how in ("again", "argument", "current"):
        if how == "current":
            with torch.cuda.stream(side):
                f2, b2 = run_forward(u, h, o, E4M3), run_backward(*src, dh_out, dn, o, stats)
        else:
            kw = {"stream": side} if how == "argument" else {}
            torch.cuda.synchronize()
            f2, b2 = run_forward(u, h, o, E4M3, **kw), run_backward(*src, dh_out, dn, o, stats, **kw)
        for x, y in ((f, f2), (b, b2)):
            for k in x:
                assert x[k] is None or torch.equal(x[k].view(torch.uint8), y[k].view(torch.uint8)), (how, k)


def test_captured_and_replayed_with_a_shared_workspace():
    """Two captured graphs that share a workspace, replayed one after the other
    on new inputs, give what eager calls give."""
    rows, cols, per = 130, 640, 50
    o = params(rows, cols, RMS, LAYER, True, per, True, 1)
    keys = ("post", "pre", "rows_per_gate", "residual_scale", "gamma_post", "beta_post", "gate", "gamma_pre")
    ws = iabn.new_block_norm_workspace(rows, cols, per, device="cuda")
    sets = []
    for k in range(2):
        t = {n: torch.empty(rows, cols, dtype=BF16, device="cuda") for n in ("u", "h", "h_out", "n", "dh_out", "dn", "dh", "du")}
        t |= {n: torch.empty(rows, cols, dtype=E4M3, device="cuda") for n in ("q_post", "q_pre")}
        t |= {n: torch.empty(rows, 5, device="cuda") for n in ("scale_post", "scale_pre")}
        t |= {n: torch.empty(rows, device="cuda") for n in ("rstd_post", "rstd_pre")}
        t |= {"dgamma_post": torch.empty(cols, device="cuda"), "dgate": torch.empty_like(o["gate"])}
        sets.append(t)

    def call(t):
        iabn.block_norm_forward_checkpoint8(
            t["u"], t["h"], t["h_out"], t["n"], **{k: t[k] for k in ("q_post", "scale_post", "q_pre", "scale_pre", "rstd_post",
                                                                     "rstd_pre")}, **{**EPS, **o})
        iabn.block_norm_backward_checkpoint8(
            t["q_post"], t["q_pre"], t["dh_out"], t["dn"], t["dh"], t["du"], ws,
            **{k: t[k] for k in ("scale_post", "scale_pre", "rstd_post", "rstd_pre", "dgamma_post", "dgate")},
            **{k: o[k] for k in keys})
        iabn.checkpoint8_load(t["q_pre"], t["scale_pre"], t["n"], gamma=o["gamma_pre"], beta=o["beta_pre"])

    def fill(t, seed):
        for i, n in enumerate(("u", "h", "dh_out", "dn")):
            t[n].copy_(values(rows, cols, BF16, seed + i))

    graphs = []
    for k, t in enumerate(sets):
        fill(t, 10 * k)
        call(t)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(t)
        graphs.append(g)
    for k, t in enumerate(sets):
        fill(t, 100 + 10 * k)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    got = [{n: v.clone() for n, v in t.items()} for t in sets]
    for t, w in zip(sets, got):
        call(t)
        torch.cuda.synchronize()
        for n in t:
            assert torch.equal(t[n].view(torch.uint8), w[n].view(torch.uint8)), n


def test_offsets_past_32_bits():
    """Tensors of more than 2^31 elements: the last rows are what a call on
    them alone gives."""
    cols = 32768
    rows = (1 << 31) // cols + 70
    u = torch.empty(rows, cols, dtype=BF16, device="cuda")
    u.view(-1)[: 1 << 20].normal_()
    h = torch.zeros_like(u)
    last = slice(rows - 66, rows)
    u[last].normal_()
    h[last].normal_()
    o = dict(post=RMS, pre=RMS)
    q, s = torch.empty(rows, cols, dtype=INT8, device="cuda"), torch.empty(rows, cols // 128, device="cuda")
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    r, r2 = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    ho, n = torch.empty_like(u), torch.empty_like(u)

    def call(k):
        iabn.block_norm_forward_checkpoint8(u[k], h[k], ho[k], n[k], q_post=q[k], scale_post=s[k], q_pre=q2[k],
                                            scale_pre=s2[k], rstd_post=r[k], rstd_pre=r2[k], **o)
        return [t[last].clone() for t in (ho, n, q, s, q2, s2, r, r2)]

    whole, part = call(slice(None)), call(last)
    assert all(torch.equal(a, b) for a, b in zip(whole, part))

    def back(k):
        ws = iabn.new_block_norm_workspace(u[k].shape[0], cols, device="cuda")
        iabn.block_norm_backward_checkpoint8(q[k], q2[k], u[k], h[k], ho[k], n[k], ws, scale_post=s[k], scale_pre=s2[k],
                                             rstd_post=r[k], rstd_pre=r2[k], **o)
        return [t[last].clone() for t in (ho, n)]

    # (rows that were never set hold zeros or noise in h: the rest of the rows only matter to themselves)
    whole, part = back(slice(None)), back(last)
    assert all(torch.equal(a, b) for a, b in zip(whole, part))

    def gate(k):
        iabn.gated_forward_checkpoint8(u[k], h[k], ho[k], q[k], s[k], q2[k], s2[k])
        first = [t[last].clone() for t in (ho, q, s, q2, s2)]
        iabn.gated_backward_checkpoint8(q[k], s[k], q2[k], s2[k], ho[k], n[k], h[k])
        return first + [n[last].clone(), h[last].clone()]

    keep = h[last].clone()
    whole = gate(slice(None))
    h[last] = keep
    part = gate(last)
    assert all(torch.equal(a, b) for a, b in zip(whole, part))


def test_binding_refuses_wrong_tensors():
    rows, cols = 4, 256
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    f = torch.zeros(cols, device="cuda")
    y = [torch.empty_like(x) for _ in range(4)]
    q, s = torch.zeros(rows, cols, dtype=INT8, device="cuda"), torch.zeros(rows, 2, device="cuda")
    bad = iabn.IabnError
    for call in (lambda: iabn.block_norm_forward(x.float(), x, y[0], y[1]),
                 lambda: iabn.block_norm_forward(x[:2], x, y[0], y[1]),
                 lambda: iabn.block_norm_forward(x.view(2 * rows, cols // 2), x, y[0], y[1]),
                 lambda: iabn.block_norm_forward(x, x, y[0], y[1], gamma_pre=f[:255]),
                 lambda: iabn.block_norm_forward(x, x, y[0], y[1], gamma_pre=f.to(BF16)),
                 lambda: iabn.block_norm_forward(x, x, y[0], y[1], gamma_pre=f.cpu()),
                 lambda: iabn.block_norm_forward(x, x, y[0], y[1], gate=f, rows_per_gate=2),
                 lambda: iabn.block_norm_forward(x, x, y[0], y[1], gate=f, rows_per_gate=-1),
                 lambda: iabn.block_norm_forward(x, x, y[0], y[1], rstd_pre=f),
                 lambda: iabn.block_norm_forward(x, x.int(), y[0], y[1]),
                 lambda: iabn.block_norm_forward(x.t().contiguous().t(), x, y[0], y[1]),
                 lambda: iabn.block_norm_forward_checkpoint8(x, x, y[0], y[1], q_post=q),
                 lambda: iabn.block_norm_forward_checkpoint8(x, x, y[0], y[1], q_post=q, scale_post=s[:, :1].contiguous()),
                 lambda: iabn.block_norm_forward_checkpoint8(x, x, y[0], y[1], q_post=q, scale_post=s, q_pre=q.view(E4M3),
                                                             scale_pre=s),
                 lambda: iabn.block_norm_forward_checkpoint8(x, x, y[0], y[1], q_post=q.view(torch.uint8), scale_post=s),
                 lambda: iabn.block_norm_backward(x, x, x, x, y[0], y[1], torch.empty(16, dtype=torch.uint8, device="cuda"),
                                                  rstd_post=f[:rows], rstd_pre=f[:rows]),
                 lambda: iabn.block_norm_backward(x, x, x, x, y[0], y[1], torch.empty(1 << 24, dtype=torch.uint8),
                                                  rstd_post=f[:rows], rstd_pre=f[:rows]),
                 lambda: iabn.gated_forward(x, x[:, :128], y[0]),
                 lambda: iabn.gated_forward(x[:, :128], y[1].view(-1)[:rows * 128].view(rows, 128), y[0][:, :128].contiguous()),
                 lambda: iabn.gated_forward(x, x, y[0].float()),
                 lambda: iabn.gated_backward_checkpoint8(q, s, q.view(E4M3), s, x, y[0], y[1]),
                 lambda: iabn.checkpoint8_store(x, None, None),
                 lambda: iabn.checkpoint8_store(x, q[:2], s[:2]),
                 lambda: iabn.checkpoint8_load(q, s, y[0], gamma=f[:8])):
        with pytest.raises(bad):
            call()


@pytest.mark.parametrize("form", [None, INT8, E4M3])
def test_a_feed_forward_block_and_its_gradients(form):
    """A pre-norm, two products with the gated activation between, the block
    norm behind them, and the whole way back, as a training step runs them.

    Each stage of the 64-bit chain takes the values that the codes of the run
    stand for, so that only fp32 rounding is left: a stage is off by about K U
    = 4e-6 of its terms' size, seven stages and products of 96 to 160 terms
    with cancellation lose less than a factor of 25 of that."""
    torch.backends.cuda.matmul.allow_tf32 = False
    rows, cols, inner, per = 60, 96, 160, 25
    g = gen(11)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    h0, w1, w2 = r(rows, cols), r(2 * inner, cols) / 10, r(cols, inner) / 12
    g0, g1, g2, b2, gate = 1 + 0.2 * r(cols), 1 + 0.2 * r(cols), 1 + 0.2 * r(cols), r(cols), r(3, cols)
    dh_out, dn = r(rows, cols), r(rows, cols)
    new = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    n0, r0, packed = new(rows, cols), new(rows), new(rows, 2 * inner)
    z, h1, n1, r1, r2 = new(rows, inner), new(rows, cols), new(rows, cols), new(rows), new(rows)
    how = dict(post=RMS, pre=RMS, rows_per_gate=per, gamma_post=g1, gate=gate, gamma_pre=g2)
    k = {}
    if form is not None:
        for name, c in (("q0", cols), ("qa", inner), ("qb", inner), ("q1", cols), ("q2", cols)):
            k[name], k["s" + name] = new(rows, c, dtype=form), new(rows, ref.groups(c))
    # forward
    if form is None:
        iabn.block_norm_forward(None, h0, None, n0, post=NONE, gamma_pre=g0, rstd_pre=r0)
    else:
        iabn.block_norm_forward_checkpoint8(None, h0, None, n0, post=NONE, gamma_pre=g0, rstd_pre=r0, q_pre=k["q0"],
                                            scale_pre=k["sq0"])
    torch.matmul(n0, w1.t(), out=packed)
    a, b = packed[:, :inner], packed[:, inner:]
    if form is None:
        iabn.gated_forward(a, b, z)
    else:
        iabn.gated_forward_checkpoint8(a, b, z, k["qa"], k["sqa"], k["qb"], k["sqb"])
    u = z @ w2.t()
    if form is None:
        iabn.block_norm_forward(u, h0, h1, n1, beta_pre=b2, rstd_post=r1, rstd_pre=r2, **how)
    else:
        iabn.block_norm_forward_checkpoint8(u, h0, h1, n1, beta_pre=b2, rstd_post=r1, rstd_pre=r2, q_post=k["q1"],
                                            scale_post=k["sq1"], q_pre=k["q2"], scale_pre=k["sq2"], **how)
    # backward
    ws = iabn.new_block_norm_workspace(rows, cols, per, device="cuda")
    dg0, dg1, dg2, db2, dgate = new(cols), new(cols), new(cols), new(cols), new(3, cols)
    du, dh, dpacked, dh0 = new(rows, cols), new(rows, cols), new(rows, 2 * inner), new(rows, cols)
    grads = dict(dgamma_post=dg1, dgate=dgate, dgamma_pre=dg2, dbeta_pre=db2, rstd_post=r1, rstd_pre=r2)
    if form is None:
        iabn.block_norm_backward(u, h1, dh_out, dn, dh, du, ws, **how, **grads)
        iabn.gated_backward(a, b, du @ w2, dpacked[:, :inner], dpacked[:, inner:])
        z2, n02 = z, n0
    else:
        iabn.block_norm_backward_checkpoint8(k["q1"], k["q2"], dh_out, dn, dh, du, ws, scale_post=k["sq1"],
                                             scale_pre=k["sq2"], **how, **grads)
        z2, n02 = new(rows, inner), new(rows, cols)
        iabn.gated_backward_checkpoint8(k["qa"], k["sqa"], k["qb"], k["sqb"], du @ w2, dpacked[:, :inner],
                                        dpacked[:, inner:], z=z2)
        iabn.checkpoint8_load(k["q0"], k["sq0"], n02, gamma=g0)
    dw2, dw1 = du.t() @ z2, dpacked.t() @ n02
    dn0 = dpacked @ w1
    if form is None:
        iabn.block_norm_backward(None, h0, dh, dn0, dh0, None, ws, post=NONE, gamma_pre=g0, rstd_pre=r0, dgamma_pre=dg0)
    else:
        iabn.block_norm_backward_checkpoint8(None, k["q0"], dh, dn0, dh0, None, ws, post=NONE, gamma_pre=g0,
                                             scale_pre=k["sq0"], rstd_pre=r0, dgamma_pre=dg0)
    torch.cuda.synchronize()

    # the same in 64 bits
    D = lambda t: t.cpu().double()  # noqa: E731
    rms = lambda v: v * ((v * v).mean(-1, keepdim=True) + 1e-6) ** -0.5  # noqa: E731
    which = torch.arange(rows) // per
    H0, W1, W2 = D(h0), D(w1), D(w2)
    X0 = rms(H0)
    P = X0 * D(g0) @ W1.t()
    A, B = P[:, :inner], P[:, inner:]
    Z = A * torch.sigmoid(A) * B
    Uh = rms(Z @ W2.t())
    H1 = H0 + D(gate)[which] * Uh * D(g1)
    X1 = rms(H1)
    rho = [D(v)[:, None] for v in (r0, r1, r2)]

    def near(got, want, what):
        off = float((D(got) - want).norm() / want.norm())
        assert off < 1e-4, f"{what}: {off:.3g}"

    near(h1, H1, "h1")
    near(n1, X1 * D(g2) + D(b2), "n1")
    if form is not None:
        for name, v in (("q0", X0), ("qa", A), ("qb", B), ("q1", Uh), ("q2", X1)):
            got = ref.values(k[name], k["s" + name])[0]
            bound = ref.code_bound(v, 1e-4 * v.abs().amax(), k["s" + name], form)
            assert ((got - v).abs() <= bound).all(), name
        X0, A, B, Uh, X1 = (ref.values(k[n], k["s" + n])[0] for n in ("q0", "qa", "qb", "q1", "q2"))
        Z = A * torch.sigmoid(A) * B
    back = lambda gr, x, p: p * (gr - x * (gr * x).mean(-1, keepdim=True))  # noqa: E731
    DN = D(dn)
    T = D(dh_out) + back(DN * D(g2), X1, rho[2])
    G = D(gate)[which]
    DU = back(T * G * D(g1), Uh, rho[1])
    DZ = DU @ W2
    S = torch.sigmoid(A)
    DP = torch.cat([DZ * B * (S + A * S * (1 - S)), DZ * A * S], 1)
    DN0 = DP @ W1
    near(dg2, (DN * X1).sum(0), "dgamma_pre")
    near(db2, DN.sum(0), "dbeta_pre")
    near(dg1, (T * G * Uh).sum(0), "dgamma_post")
    near(dgate, torch.zeros(3, cols, dtype=torch.float64).index_add_(0, which, T * Uh * D(g1)), "dgate")
    near(du, DU, "du")
    near(dw2, DU.t() @ Z, "dw2")
    near(dpacked, DP, "dpacked")
    near(dw1, DP.t() @ (X0 * D(g0)), "dw1")
    near(dg0, (DN0 * X0).sum(0), "dgamma_0")
    near(dh0, T + back(DN0 * D(g0), X0, rho[0]), "dh0")


@pytest.mark.parametrize("dtype,value", [(BF16, 1e20), (F32, 1e20), (F32, 1e22), (F16, 6e4)])
@pytest.mark.parametrize("cols", [256, 512, 600, 1024, 1536, 2056, 3000, 4096, 5120, 8192, 8200, 9001, 20001, 32768])
def test_constant_rows_of_large_values(cols, dtype, value):
    """A layer norm of rows whose every value is the same: the variance is 0 (but
    for what the mean's rounding leaves of the value), whatever part of the
    row's warps has columns, and nothing is NaN.

    A row's sum is exact, as count * value takes fewer than 24 bits of a value of
    8 bits (bf16; the fp32 values are rounded to bf16).  Its product with 1/cols is
    off by at most 2^-23 of the mean, so where cols is a power of two nothing is
    lost; elsewhere the deviation d <= 2^-22 |mean| from the mean gives a variance
    of at most d^2."""
    u = torch.full((3, cols), value, dtype=dtype, device="cuda").to(BF16).to(dtype)
    u[1] = -u[1]
    u[2] = torch.randn(cols, generator=gen(1)).to(dtype).cuda()
    h = torch.zeros_like(u)
    for form in (None, E4M3):
        o = params(3, cols, LAYER, LAYER, False, 0, False, 1) | {"gamma_post": None, "gamma_pre": None}
        got = run_forward(u, h, o, form)
        assert not any(torch.isnan(t.float()).any() for t in got.values() if t is not None)
        if form is None:
            mean = u[:2, 0].float()
            assert ((got["mean_post"][:2] - mean).abs() <= 2.0 ** -22 * mean.abs()).all()
            least = 1.0 / (EPS["eps_post"] + (2.0 ** -22 * mean.double()) ** 2).sqrt()
            assert (got["rstd_post"][:2].double() >= least * (1 - 1e-5)).all()
            assert (got["rstd_post"][:2].double() <= EPS["eps_post"] ** -0.5 * (1 + 1e-5)).all()
        if cols & (cols - 1) == 0:
            assert (got["h_out"][:2] == 0).all() and (got["n"][:2] == 0).all()
    # the ordinary row beside them
    w = u[2:].double()
    want = (w - w.mean()) * ((w - w.mean()).square().mean() + EPS["eps_post"]) ** -0.5
    step = torch.finfo(dtype).eps
    assert ((got["h_out"][2:].double() - want).abs() <= (step + 1e-5) * (1 + want.abs())).all()


def test_binding_refuses_missing_tensors_and_scalars():
    x = torch.zeros(4, 256, dtype=BF16, device="cuda")
    y = [torch.empty_like(x) for _ in range(4)]
    f, tiny, scalar = torch.zeros(4, device="cuda"), torch.zeros(1, 1, device="cuda"), torch.zeros((), device="cuda")
    for call in (lambda: iabn.block_norm_backward(x, x, x, x, y[0], y[1], None, rstd_post=f, rstd_pre=f),
                 lambda: iabn.gated_forward(x, None, y[0]), lambda: iabn.gated_forward(None, x, y[0]),
                 lambda: iabn.gated_backward(x, x, x, None, y[0]), lambda: iabn.gated_backward(x, x, x, y[0], None),
                 lambda: iabn.gated_backward(None, None, x, y[0], y[1]),
                 lambda: iabn.block_norm_forward(scalar, tiny, torch.empty_like(tiny), torch.empty_like(tiny))):
        with pytest.raises(iabn.IabnError):
            call()


@pytest.mark.parametrize("dtype,form", [(BF16, None), (F16, E4M3), (F32, None)])
@pytest.mark.parametrize("cols,rows", [(1, 300), (7, 700), (73, 400), (1021, 333), (2049, 150), (4104, 60), (9001, 20),
                                       (10240, 20), (20001, 7), (32768, 5)])
def test_in_place_at_any_width(cols, rows, dtype, form):
    """Outputs over inputs where a warp's copies take in words of its
    neighbours' rows, and where a cluster shares a row."""
    per = rows // 2
    o = params(rows, cols, LAYER, LAYER, True, per, True, 1)
    u, h = values(rows, cols, dtype, 2), values(rows, cols, dtype, 3, 2.0)
    want = run_forward(u, h, o, form)
    call = iabn.block_norm_forward if form is None else iabn.block_norm_forward_checkpoint8
    kept = {k: torch.empty_like(v) for k, v in want.items() if k not in ("h_out", "n")}
    for swap in (False, True):
        u2, h2 = u.clone(), h.clone()
        ho, n = (u2, h2) if swap else (h2, u2)
        call(u2, h2, ho, n, **{**EPS, **o}, **kept)
        assert torch.equal(ho, want["h_out"]) and torch.equal(n, want["n"]), swap
        for k, v in kept.items():
            assert torch.equal(v.view(torch.uint8), want[k].view(torch.uint8)), k
    dh_out, dn = values(rows, cols, dtype, 4, 0.1), values(rows, cols, dtype, 5, 0.1)
    o["beta_pre"] = None
    ws = iabn.new_block_norm_workspace(rows, cols, per, device="cuda")
    a = {k: o[k] for k in ("post", "pre", "rows_per_gate", "residual_scale", "gamma_post", "beta_post", "gate", "gamma_pre")}
    if form is None:
        stats = {k: want[k] for k in ("mean_post", "rstd_post", "mean_pre", "rstd_pre")}
        src, pairs = (u, want["h_out"]), ((0, 1), (1, 0), (2, 3), (3, 2), (0, 2), (3, 1))
        back = run_backward(*src, dh_out, dn, o, stats)
    else:
        stats = {k: want[k] for k in ("rstd_post", "rstd_pre")}
        src, pairs = ((want["q_post"], want["scale_post"]), (want["q_pre"], want["scale_pre"])), ((0, 1), (1, 0))
        back = run_backward(*src, dh_out, dn, o, stats)
    grads = {k: torch.empty_like(v) for k, v in back.items() if k not in ("dh", "du")}
    for i, j in pairs:
        t = [dh_out.clone(), dn.clone()] + ([s.clone() for s in src] if form is None else [])
        if form is None:
            iabn.block_norm_backward(t[2], t[3], t[0], t[1], t[i], t[j], ws, **stats, **a, **grads)
        else:
            iabn.block_norm_backward_checkpoint8(src[0][0], src[1][0], t[0], t[1], t[i], t[j], ws, scale_post=src[0][1],
                                                 scale_pre=src[1][1], **stats, **a, **grads)
        for k, v in (grads | {"dh": t[i], "du": t[j]}).items():
            assert torch.equal(v.view(torch.uint8), back[k].view(torch.uint8)), (k, i, j)
    # the gated activation over its own inputs, packed and apart
    p, dz = values(rows, 2 * cols, dtype, 6), values(rows, cols, dtype, 7)
    want, z = torch.empty_like(p), torch.empty_like(dz)
    iabn.gated_backward(p[:, :cols], p[:, cols:], dz, want[:, :cols], want[:, cols:], z=z)
    for over in (0, 1):
        a, b = p[:, :cols].contiguous(), p[:, cols:].contiguous()
        iabn.gated_forward(a, b, (a, b)[over])
        assert torch.equal((a, b)[over], z), over
    iabn.gated_backward(p[:, :cols], p[:, cols:], dz, p[:, :cols], p[:, cols:], z=dz)
    assert torch.equal(p, want) and torch.equal(dz, z)


@pytest.mark.parametrize("form,dtype", [(None, F32), (INT8, BF16), (E4M3, F32)])
@pytest.mark.parametrize("cols", [72, 73, 264, 1021, 2048, 2049, 8192, 9001, 12000])
def test_a_bad_row_stays_in_its_row_backward(cols, form, dtype):
    """NaN and infinities in a row's gradients, statistics or scales change no
    bit of the other rows' gradients, nor of the gates that other rows have;
    the sums over rows that a bad element enters are NaN or infinite there."""
    rows, per = 24, 6
    o = params(rows, cols, LAYER, LAYER, True, per, True, 1)
    u, h = values(rows, cols, dtype, 2), values(rows, cols, dtype, 3)
    f = run_forward(u, h, o, form)
    o["beta_pre"] = torch.zeros(cols, device="cuda")
    dh_out, dn = values(rows, cols, dtype, 4, 0.1), values(rows, cols, dtype, 5, 0.1)
    names = ("mean_post", "rstd_post", "mean_pre", "rstd_pre") if form is None else ("rstd_post", "rstd_pre")
    stats = {k: f[k] for k in names}
    src = (u, f["h_out"]) if form is None else ((f["q_post"], f["scale_post"]), (f["q_pre"], f["scale_pre"]))
    clean = run_backward(*src, dh_out, dn, o, stats)
    bad_dn, bad_dh = dn.clone(), dh_out.clone()
    bad_dn[1, cols // 2], bad_dn[4, cols - 1] = math.nan, math.inf
    bad_dh[2, 0] = -math.inf
    bad_stats = {k: v.clone() for k, v in stats.items()}
    bad_stats["rstd_pre"][12] = math.nan
    if form is None:
        bad_src = (u.clone(), f["h_out"])
        bad_src[0][13, cols // 3] = math.inf
    else:
        bad_src = ((f["q_post"], f["scale_post"].clone()), src[1])
        bad_src[0][1][13, -1] = math.nan
    got = run_backward(*bad_src, bad_dh, bad_dn, o, bad_stats)
    bad = (1, 2, 4, 12, 13)
    rest = [r for r in range(rows) if r not in bad]
    for k in ("dh", "du"):
        assert torch.equal(got[k][rest], clean[k][rest]), k
        assert not torch.isfinite(got["du"][list(bad)].float()).all(-1).any(), k
    assert torch.isnan(got["dh"][[1, 12]]).all()
    # an infinite g makes both means infinite: g - inf - x (+-inf) is infinite or NaN in every column
    assert not torch.isfinite(got["dh"][4]).any()
    # gate rows 1 and 3 (rows 6-11 and 18-23) have no bad row
    assert torch.equal(got["dgate"][[1, 3]], clean["dgate"][[1, 3]])
    assert not torch.isfinite(got["dgate"][0]).any()
    assert torch.isnan(got["dbeta_pre"][cols // 2]) and not torch.isfinite(got["dbeta_pre"][cols - 1])
    if cols > 8:
        c = [k for k in range(cols) if k not in (cols // 2, cols - 1)]
        assert torch.equal(got["dbeta_pre"][c], clean["dbeta_pre"][c])


def test_two_to_the_31_rows():
    """The most rows that a call may have: the last rows, the gate rows that end
    with them and their sums."""
    rows, per = (1 << 31) - 1, 1 << 30
    dh_out = torch.zeros(rows, 1, dtype=BF16, device="cuda")
    u = torch.ones(rows, 1, dtype=BF16, device="cuda")
    spots = [0, 1, 8, per - 1, per, per + 9, rows - 10, rows - 2, rows - 1]
    for i, r in enumerate(spots):
        dh_out[r], u[r] = i + 1.0, 2.0
    gate, dgate = torch.tensor([[0.5], [4.0]], device="cuda"), torch.empty(2, 1, device="cuda")
    ws = iabn.new_block_norm_workspace(rows, 1, per, device="cuda")
    # both in place: dh over dh_out, du over u
    iabn.block_norm_backward(u, None, dh_out, None, dh_out, u, ws, gate=gate, dgate=dgate, post=NONE, pre=NONE,
                             rows_per_gate=per, residual_scale=2.0)
    for i, r in enumerate(spots):
        assert dh_out[r].item() == 2.0 * (i + 1) and u[r].item() == (0.5 if r < per else 4.0) * (i + 1), r
    assert int(torch.count_nonzero(dh_out)) == len(spots) == int(torch.count_nonzero(u))
    # t u over the gate's rows: 2 (1 + .. + 4) and 2 (5 + .. + 9)
    assert dgate.view(-1).tolist() == [20.0, 70.0]
    # and forward: n = h/|h| of single columns
    h, n, r = u, dh_out, torch.empty(rows, device="cuda")
    iabn.block_norm_forward(None, h, None, n, rstd_pre=r, post=NONE, pre=RMS, eps_pre=0.25)
    for i, k in enumerate(spots):
        v = (0.5 if k < per else 4.0) * (i + 1)
        assert abs(n[k].item() - v / math.sqrt(v * v + 0.25)) < 2.0 ** -8 and abs(r[k].item() * math.sqrt(v * v + 0.25) - 1) < 1e-5
    assert int(torch.count_nonzero(n)) == len(spots) and r[7].item() == 2.0


def test_the_same_bits_at_a_training_size():
    """16384 x 4096 with RMS norms and e4m3 codes: again and again the same bits,
    whatever runs between; and the codes are the stated rounding of the values
    that the kernel's own statistics give (those of another summation order may
    fall on the other side of a tie)."""
    rows, cols = 16384, 4096
    r = lambda s: torch.randn(rows, cols, generator=torch.Generator("cuda").manual_seed(s), device="cuda")  # noqa: E731
    u, h, other = r(1).to(BF16), (2 * r(2)).to(BF16), r(3).to(BF16)
    gamma, gate = torch.rand(cols, device="cuda") + 0.5, torch.rand(1, cols, device="cuda")
    new = lambda dtype: torch.empty(rows, cols, dtype=dtype, device="cuda")  # noqa: E731
    f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731

    def outputs():
        return dict(h_out=new(BF16), n=new(BF16), q_post=new(E4M3), q_pre=new(E4M3), scale_post=f32(rows, 32),
                    scale_pre=f32(rows, 32), rstd_post=f32(rows), rstd_pre=f32(rows))

    def call(x, out, **kw):
        k = {n: v for n, v in out.items() if n not in ("h_out", "n")}
        iabn.block_norm_forward_checkpoint8(x, h, out["h_out"], out["n"], gamma_post=gamma, gate=gate, **k, **kw)

    first, again, noise, side = outputs(), outputs(), outputs(), torch.cuda.Stream()
    call(u, first)
    torch.cuda.synchronize()
    for turn in range(6):
        for v in again.values():
            v.view(torch.uint8).fill_(0xff)
        call(other, noise, **({"stream": side} if turn % 2 else {}))
        call(u, again)
        torch.cuda.synchronize()
        for k in first:
            assert torch.equal(first[k].view(torch.uint8), again[k].view(torch.uint8)), (turn, k)
    some = slice(None, None, 257)
    uhat = u[some].float() * first["rstd_post"][some, None]
    q, _ = ref.quantise(uhat.cpu(), E4M3)
    assert torch.equal(q.float(), first["q_post"][some].cpu().float())
    # (a residual scale of 1: the sum is rounded once whether or not it is fused)
    hout = h[some].float() + uhat * (gamma * gate[0])
    q, _ = ref.quantise((hout * first["rstd_pre"][some, None]).cpu(), E4M3)
    assert torch.equal(q.float(), first["q_pre"][some].cpu().float())


FIRST_CALL_IN_A_CAPTURE = """
import torch, place_batchnorm_activation_b200 as iabn
rows, cols = {rows}, {cols}
new = lambda *s: torch.randn(*s, device="cuda")
u, h, dh_out, dn = (new(rows, cols).bfloat16() for _ in range(4))
beta, gate = new(cols), new(2, cols)
out = {{k: torch.empty_like(u) for k in ("h_out", "n", "dh", "du", "z", "da", "db")}}
stats = {{k: torch.empty(rows, device="cuda") for k in ("mean_post", "rstd_post", "mean_pre", "rstd_pre")}}
grads = {{"dgamma_post": torch.empty(cols, device="cuda"), "dgate": torch.empty(2, cols, device="cuda")}}
per, ws = -(-rows // 2), iabn.new_block_norm_workspace(rows, cols, -(-rows // 2), device="cuda")
q, s = torch.empty_like(u, dtype=torch.int8), torch.empty(rows, -(-cols // 128), device="cuda")
def call():
    how = dict(post=2, pre=2, rows_per_gate=per, beta_post=beta, gate=gate)
    iabn.block_norm_forward(u, h, out["h_out"], out["n"], **stats, **how)
    iabn.block_norm_backward(u, out["h_out"], dh_out, dn, out["dh"], out["du"], ws, **stats, **grads, **how)
    iabn.gated_backward(u, h, dn, out["da"], out["db"], z=out["z"])
    iabn.checkpoint8_store(out["n"], q, s)
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in [*out.values(), *stats.values(), *grads.values(), q, s]]
call()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
           for a, b in zip(got, [*out.values(), *stats.values(), *grads.values(), q, s]))
print("same")
"""


@pytest.mark.parametrize("rows,cols", [(70, 4096), (40, 1021), (9, 9000)])
def test_a_first_call_inside_a_capture(rows, cols):
    """A program's first calls of the operators may be the ones it captures."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE.format(rows=rows, cols=cols)], cwd=root, timeout=120,
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_more_gate_rows_than_the_column_pass_has_blocks():
    """A gate row a token, 9001 of them, and the sums over them."""
    one(9001, 40, BF16, RMS, LAYER, True, 1, True, E4M3, seed=3)
    one(9001, 9, F32, LAYER, RMS, True, 2, True, None, seed=4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cols", [40, 1024, 4096, 9000])
def test_outputs_off_16_byte_boundaries(cols, dtype):
    """Inputs on 16-byte boundaries, one output or many of them not."""
    rows = 11
    o = params(rows, cols, RMS, LAYER, True, 4, True, 1)
    u, h = values(rows, cols, dtype, 2), values(rows, cols, dtype, 3, 2.0)
    dh_out, dn = values(rows, cols, dtype, 4, 0.1), values(rows, cols, dtype, 5, 0.1)

    class Off(Buffers):
        def __init__(self, which):
            super().__init__()
            self.which = which

        def new(self, name, shape, dt, fill=None):
            if name not in self.which:
                return super().new(name, shape, dt, fill)
            n = math.prod(shape)
            flat = super().new(name, (n + 1,), dt)
            return flat[1:].view(shape)

    for form in (None, INT8):
        for which in (("n",), ("h_out", "n", "q_post", "q_pre", "dh", "du", "dgamma_post", "dgate")):
            got = run_forward(u, h, o, form, Off(which))
            check_forward(u, h, o, form, got, f"off {which}")
            stats = {k: got[k] for k in ("mean_pre", "rstd_post", "rstd_pre") if got.get(k) is not None}
            src = (u, got["h_out"]) if form is None else ((got["q_post"], got["scale_post"]), (got["q_pre"], got["scale_pre"]))
            back = run_backward(*src, dh_out, dn, o | {"beta_pre": None}, stats, Off(which))
            check_backward(back, backward_want(*src, dh_out, dn, o, stats), dtype, f"off {which}")


@pytest.mark.parametrize("dtype,form", [(BF16, None), (BF16, INT8), (F32, E4M3)])
@pytest.mark.parametrize("cols", [264, 1021, 4096, 9000])
def test_outputs_that_are_not_wanted(cols, dtype, form):
    """Each optional output left out by itself: the others are the same bits.
    (Layer norms, whose kernels do not depend on which sums are asked for.)"""
    rows, per = 10, 4
    o = params(rows, cols, LAYER, LAYER, True, per, True, 1)
    u, h = values(rows, cols, dtype, 2), values(rows, cols, dtype, 3, 2.0)
    full = run_forward(u, h, o, form)
    names = [k for k in full if k not in ("h_out", "n")]
    pairs = [(k,) for k in names if "_p" in k and k[:2] not in ("q_", "sc")]
    pairs += [("q_post", "scale_post"), ("q_pre", "scale_pre")] if form is not None else []
    call = iabn.block_norm_forward if form is None else iabn.block_norm_forward_checkpoint8
    for left in [("h_out",), *pairs, tuple(n for n in names if form is None or n.startswith("rstd"))]:
        out = {k: None if k in left else torch.empty_like(v) for k, v in full.items()}
        call(u, h, out["h_out"], out["n"], **{**EPS, **o}, **{k: v for k, v in out.items() if k not in ("h_out", "n")})
        for k, v in out.items():
            assert v is None or torch.equal(v.view(torch.uint8), full[k].view(torch.uint8)), (left, k)
    dh_out, dn = values(rows, cols, dtype, 4, 0.1), values(rows, cols, dtype, 5, 0.1)
    o["beta_pre"] = torch.zeros(cols, device="cuda")
    stats = {k: full[k] for k in (("mean_post", "rstd_post", "mean_pre", "rstd_pre") if form is None else ("rstd_post", "rstd_pre"))}
    src = (u, full["h_out"]) if form is None else ((full["q_post"], full["scale_post"]), (full["q_pre"], full["scale_pre"]))
    grads = ("dgamma_post", "dbeta_post", "dgate", "dgamma_pre", "dbeta_pre")
    whole = run_backward(*src, dh_out, dn, o, stats)
    check_backward(whole, backward_want(*src, dh_out, dn, o, stats), dtype, "whole")
    for left in (*((g,) for g in grads), grads[:3], grads[3:], grads):
        back = run_backward(*src, dh_out, dn, o, stats, want=[g for g in grads if g not in left])
        assert set(whole) - set(back) == set(left)
        for k, v in back.items():
            assert torch.equal(v.view(torch.uint8), whole[k].view(torch.uint8)), (left, k)
    # du not wanted
    ws = iabn.new_block_norm_workspace(rows, cols, per, device="cuda")
    a = {k: o[k] for k in ("post", "pre", "rows_per_gate", "residual_scale", "gamma_post", "beta_post", "gate", "gamma_pre")}
    out = {k: torch.empty_like(v) for k, v in whole.items() if k != "du"}
    g = {k: v for k, v in out.items() if k != "dh"}
    if form is None:
        iabn.block_norm_backward(*src, dh_out, dn, out["dh"], None, ws, **stats, **a, **g)
    else:
        iabn.block_norm_backward_checkpoint8(src[0][0], src[1][0], dh_out, dn, out["dh"], None, ws, scale_post=src[0][1],
                                             scale_pre=src[1][1], **stats, **a, **g)
    for k, v in out.items():
        assert torch.equal(v.view(torch.uint8), whole[k].view(torch.uint8)), k
    # no gradient through the residual stream: as one of zeros
    zero = run_backward(*src, torch.zeros_like(dh_out), dn, o, stats)
    none = run_backward(*src, None, dn, o, stats)
    for k, v in none.items():
        assert torch.equal(v, zero[k]), k
