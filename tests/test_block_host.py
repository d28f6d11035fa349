"""The row operators (iabn_block.h) without a GPU: the header and the library
agree, bad arguments are refused on the host, and the 64-bit forms that the
GPU tests compare with have the gradients that they state.

The refusals of the C entry points take fake device addresses; every case
carries a defect that the host checks catch first, and they are skipped where
a GPU is present, so a fake address never reaches a kernel."""
import os
import re
import shutil
import subprocess

import pytest
import torch

import block_ref as ref
import place_batchnorm_activation_b200 as iabn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "iabn_block.h")
no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake device addresses are only passed without a GPU")
FAKE = 1 << 32
MB = 1 << 24
OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE, CUDA = 0, 1, 2, 3, 4, 5


def test_header_binding_and_library_agree():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(iabn_[a-z0-9_]+)\s*\(", text))) == sorted(iabn.BLOCK_EXPORTS)
    for name in iabn.BLOCK_EXPORTS:
        assert hasattr(iabn.lib(), name)


@pytest.mark.parametrize("compiler,flags", [("gcc", ["-std=c11"]), ("g++", ["-x", "c++", "-std=c++17"])])
def test_header_compiles_as_c_and_structs_match(tmp_path, compiler, flags):
    if shutil.which(compiler) is None:
        pytest.skip(f"{compiler} not available")
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "iabn_block.h"\n'
                   'int main(void) { printf("%zu %zu %d", sizeof(iabn_block_desc), sizeof(iabn_gated_desc),'
                   ' IABN_Q8_GROUP); return 0; }\n')
    exe = tmp_path / "sizes"
    subprocess.run([compiler, *flags, "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                    os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    import ctypes
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(iabn.IabnBlockDesc), ctypes.sizeof(iabn.IabnGatedDesc), 128]


# ------------------------------------------------- refusals of the C calls

def desc(rows=16, cols=64, per=0, dtype=1, post=1, pre=1, form=0, alpha=1.0, e1=1e-6, e2=1e-6):
    return iabn.IabnBlockDesc(rows, cols, per, dtype, post, pre, form, alpha, e1, e2)


def at(k):
    return FAKE + k * MB


def fwd(d=None, **kw):
    a = dict(u=at(0), h=at(1), h_out=at(2), n=at(3), gamma_post=None, beta_post=None, gate=None,
             gamma_pre=None, beta_pre=None, mean_post=None, rstd_post=None, mean_pre=None, rstd_pre=None)
    a.update(kw)
    return iabn.lib().iabn_block_norm_forward(desc() if d is None else d, *a.values(), None)


def fwd8(d=None, **kw):
    a = dict(u=at(0), h=at(1), h_out=at(2), n=at(3), gamma_post=None, beta_post=None, gate=None,
             gamma_pre=None, beta_pre=None, rstd_post=None, rstd_pre=None, q_post=at(4), scale_post=at(5),
             q_pre=at(6), scale_pre=at(7))
    a.update(kw)
    return iabn.lib().iabn_block_norm_forward_checkpoint8(desc() if d is None else d, *a.values(), None)


def bwd(d=None, ws=at(20), ws_bytes=MB, eight=False, **kw):
    if eight:
        a = dict(q_post=at(0), scale_post=at(1), q_pre=at(2), scale_pre=at(3))
    else:
        a = dict(u=at(0), h_out=at(2))
    a |= dict(dh_out=at(4), dn=at(5), dh=at(6), du=at(7), gamma_post=None, beta_post=None, gate=None,
              gamma_pre=None)
    if not eight:
        a |= dict(mean_post=None)
    a |= dict(rstd_post=at(8))
    if not eight:
        a |= dict(mean_pre=None)
    a |= dict(rstd_pre=at(9), dgamma_post=None, dbeta_post=None, dgate=None, dgamma_pre=None, dbeta_pre=None)
    assert set(kw) <= set(a)
    a.update(kw)
    f = iabn.lib().iabn_block_norm_backward_checkpoint8 if eight else iabn.lib().iabn_block_norm_backward
    return f(desc() if d is None else d, *a.values(), ws, ws_bytes, None)


@no_gpu_only
@pytest.mark.parametrize("call", [fwd, fwd8, bwd, lambda d=None: bwd(d, eight=True)])
def test_block_descriptor_refusals(call):
    assert call() == CUDA     # valid: reaches the runtime, which has no device here
    nan, inf = float("nan"), float("inf")
    for bad, want in ((desc(rows=-1), INVALID), (desc(cols=0), INVALID), (desc(dtype=3), INVALID),
                      (desc(dtype=-1), INVALID), (desc(post=3), INVALID), (desc(pre=-1), INVALID),
                      (desc(per=-1), INVALID), (desc(alpha=nan), INVALID), (desc(alpha=inf), INVALID),
                      (desc(e1=-1.0), INVALID), (desc(e2=nan), INVALID), (desc(e1=inf), INVALID),
                      (desc(cols=32769), UNSUPPORTED), (desc(rows=1 << 31), UNSUPPORTED),
                      (desc(rows=1 << 41), UNSUPPORTED)):
        assert call(bad) == want


@no_gpu_only
def test_block_forward_refusals():
    lib = iabn.lib()
    assert lib.iabn_block_norm_forward(None, *[at(0)] * 13, None) == INVALID
    for kw in (dict(h=None), dict(h_out=None, n=None), dict(n=None)):
        assert fwd(**kw) == INVALID
    # n is there exactly with a pre-norm; nothing of an absent norm is given
    assert fwd(desc(pre=0)) == INVALID
    assert fwd(desc(pre=0), n=None) == CUDA
    for k in ("gamma_pre", "beta_pre", "rstd_pre", "mean_pre"):
        assert fwd(desc(pre=0), n=None, **{k: at(9)}) == INVALID
    for k in ("gamma_post", "beta_post", "rstd_post", "mean_post"):
        assert fwd(desc(post=0), **{k: at(9)}) == INVALID
    assert fwd(mean_post=at(9)) == INVALID and fwd(mean_pre=at(9)) == INVALID   # RMS has no mean
    assert fwd(desc(post=2), mean_post=at(9)) == CUDA
    # without u: the norm of h alone
    assert fwd(desc(post=0), u=None, h_out=None) == CUDA
    assert fwd(u=None, h_out=None) == INVALID
    assert fwd(desc(post=0), u=None) == INVALID
    assert fwd(desc(post=0), u=None, h_out=None, gate=at(9)) == INVALID
    assert fwd(desc(post=0, alpha=0.5), u=None, h_out=None) == INVALID
    # alignment: that of the element
    for k in ("u", "h", "h_out", "n"):
        assert fwd(**{k: at(10) + 1}) == MISALIGNED
        assert fwd(**{k: at(10) + 2}) == CUDA
    for k in ("gamma_post", "beta_post", "gate", "gamma_pre", "beta_pre", "rstd_post", "rstd_pre"):
        assert fwd(**{k: at(10) + 2}) == MISALIGNED
    # overlaps: an output may be an input, not a part of one, and not another output
    for k in ("h_out", "n"):
        for src in (at(0), at(1)):
            assert fwd(**{k: src}) == CUDA
            assert fwd(**{k: src + 64}) == INVALID
    assert fwd(h_out=at(2), n=at(2)) == INVALID
    assert fwd(n=at(2) + 16 * 64 * 2 - 2) == INVALID
    assert fwd(n=at(2) + 16 * 64 * 2) == CUDA
    # no rows: nothing is looked at
    assert fwd(desc(rows=0), u=None, h=None, h_out=None, n=None) == OK


@no_gpu_only
def test_block_forward_checkpoint8_refusals():
    assert fwd8(desc(form=2)) == INVALID and fwd8(desc(form=-1)) == INVALID
    for k in ("q_post", "scale_post", "q_pre", "scale_pre"):
        assert fwd8(**{k: None}) == INVALID
    assert fwd8(q_post=None, scale_post=None) == CUDA
    assert fwd8(desc(pre=0), n=None) == INVALID      # xhat's checkpoint without a pre-norm
    assert fwd8(desc(pre=0), n=None, q_pre=None, scale_pre=None) == CUDA
    assert fwd8(desc(post=0), u=None, h_out=None) == INVALID
    assert fwd8(scale_pre=at(7) + 2) == MISALIGNED
    assert fwd8(q_pre=at(6) + 1) == CUDA             # bytes have no alignment
    for bad in (at(0), at(1), at(2), at(3), at(4) + 64):
        assert fwd8(q_pre=bad) == INVALID


@no_gpu_only
@pytest.mark.parametrize("eight", [False, True])
def test_block_backward_refusals(eight):
    b = lambda d=None, **kw: bwd(d, eight=eight, **kw)  # noqa: E731
    x = "q_pre" if eight else "h_out"
    u = "q_post" if eight else "u"
    assert b(dh=None) == INVALID
    assert b(dn=None) == INVALID and b(desc(pre=0)) == INVALID
    assert b(desc(pre=0), dn=None) == CUDA
    assert b(desc(pre=0), dn=None, dh_out=None) == INVALID
    assert b(dh_out=None) == CUDA and b(du=None) == CUDA
    assert b(**{x: None}) == INVALID and b(**{u: None}) == INVALID
    assert b(rstd_post=None) == INVALID and b(rstd_pre=None) == INVALID
    assert b(desc(post=0), **{u: None}) == CUDA                       # not needed without its norm ..
    assert b(desc(post=0), gate=at(10), dgate=at(11), **{u: None}) == INVALID   # .. unless the gate learns
    assert b(dgate=at(11)) == INVALID
    for k in ("gamma_post", "beta_post", "dgamma_post", "dbeta_post"):
        assert b(desc(post=0), **{k: at(10)}) == INVALID
    for k in ("gamma_pre", "dgamma_pre", "dbeta_pre"):
        assert b(desc(pre=0), dn=None, **{k: at(10)}) == INVALID
    if eight:
        assert b(scale_post=None) == INVALID and b(scale_pre=None) == INVALID
        assert b(desc(form=2)) == INVALID
        assert b(dh=at(0)) == INVALID                # never over codes
    else:
        assert b(desc(post=2)) == INVALID and b(desc(pre=2)) == INVALID    # a layer norm's mean
        assert b(desc(post=2), mean_post=at(10)) == CUDA
        assert b(dh=at(0)) == CUDA and b(du=at(2)) == CUDA
        assert b(u=at(10) + 1) == MISALIGNED
    for k in ("dh_out", "dn", "dh", "du"):
        assert b(**{k: at(12) + 1}) == MISALIGNED
    for k in ("rstd_pre", "dgamma_pre", "gamma_pre"):
        assert b(**{k: at(12) + 2}) == MISALIGNED
    assert b(dh=at(4)) == CUDA and b(du=at(5)) == CUDA and b(du=at(4)) == CUDA
    assert b(dh=at(4) + 2) == INVALID and b(du=at(6)) == INVALID
    need = iabn.block_norm_workspace_size(16, 64)
    assert need > 0 and need % 256 == 0
    assert b(ws=None) == WORKSPACE and b(ws=at(20) + 8) == WORKSPACE
    assert b(ws_bytes=need - 1) == WORKSPACE and b(ws_bytes=need) == CUDA


def test_block_workspace_size():
    size = iabn.block_norm_workspace_size
    assert size(0, 64) > 0
    for bad in ((-1, 64), (4, 0), (4, 32769), (1 << 31, 64)):
        assert size(*bad) == 0
    assert size(16, 64, -1) == 0
    assert size(1000, 64, 1) > size(1000, 64, 100) > size(1000, 64)
    # the largest sizes stay in range
    assert size((1 << 31) - 1, 32768, 1) > (1 << 31) * 32768 * 8


def gated_desc(rows=16, cols=64, ld=128, ldg=128, dtype=1, act=0, form=0):
    return iabn.IabnGatedDesc(rows, cols, ld, ldg, dtype, act, form)


HALF = 64 * 2    # bytes of one half of a packed row


def gf(d=None, eight=False, **kw):
    a = dict(a=at(0), b=at(0) + HALF, z=at(1))
    if eight:
        a |= dict(qa=at(2), sa=at(3), qb=at(4), sb=at(5))
    assert set(kw) <= set(a)
    a.update(kw)
    f = iabn.lib().iabn_gated_forward_checkpoint8 if eight else iabn.lib().iabn_gated_forward
    return f(gated_desc() if d is None else d, *a.values(), None)


def gb(d=None, eight=False, **kw):
    a = dict(qa=at(2), sa=at(3), qb=at(4), sb=at(5)) if eight else dict(a=at(0), b=at(0) + HALF)
    a |= dict(dz=at(6), da=at(7), db=at(7) + HALF, z=None)
    assert set(kw) <= set(a)
    a.update(kw)
    f = iabn.lib().iabn_gated_backward_checkpoint8 if eight else iabn.lib().iabn_gated_backward
    return f(gated_desc() if d is None else d, *a.values(), None)


@no_gpu_only
@pytest.mark.parametrize("call", [gf, gb])
@pytest.mark.parametrize("eight", [False, True])
def test_gated_refusals(call, eight):
    c = lambda d=None, **kw: call(d, eight=eight, **kw)  # noqa: E731
    assert c() == CUDA
    for bad in (gated_desc(rows=-1), gated_desc(cols=0), gated_desc(dtype=3), gated_desc(act=3),
                gated_desc(act=-1)):
        assert c(bad) == INVALID
    assert c(gated_desc(cols=1 << 31, ld=1 << 31, ldg=1 << 31)) == UNSUPPORTED
    assert c(gated_desc(rows=1 << 40, ld=1 << 30, ldg=1 << 30)) == UNSUPPORTED
    assert c(gated_desc(rows=0)) == OK
    if eight:
        assert c(gated_desc(form=2)) == INVALID
        for k in ("qa", "sa", "qb", "sb"):
            assert c(**{k: None}) == INVALID
        assert c(sa=at(3) + 2) == MISALIGNED
    reads_ab = call is gf or not eight
    assert c(gated_desc(ld=63)) == (INVALID if reads_ab else CUDA)
    assert c(gated_desc(ldg=63)) == (INVALID if call is gb else CUDA)
    for k in ("a", "b") if reads_ab else ():
        assert c(**{k: None}) == INVALID and c(**{k: at(10) + 1}) == MISALIGNED
    assert c(z=at(10) + 1) == MISALIGNED


@no_gpu_only
def test_gated_overlaps():
    assert gf(z=at(0)) == INVALID                                  # z's rows lie closer than a's
    assert gf(gated_desc(ld=64), b=at(9), z=at(0)) == CUDA         # the same tensor
    assert gf(gated_desc(ld=64), b=at(9), z=at(9)) == CUDA
    assert gf(gated_desc(ld=64), b=at(9), z=at(9) + 2) == INVALID
    assert gf(b=at(0)) == CUDA                                     # a*phi(a): inputs may overlap
    assert gf(eight=True, qa=at(4)) == INVALID and gf(eight=True, qa=at(0)) == INVALID
    assert gb(da=at(0), db=at(0) + HALF) == CUDA                   # over the kept a and b
    assert gb(da=at(0) + HALF, db=at(0)) == CUDA
    assert gb(da=at(7), db=at(7) + HALF - 2) == INVALID and gb(db=at(7) + HALF + 2) == INVALID
    assert gb(da=at(7), db=at(7)) == INVALID
    assert gb(da=at(6)) == INVALID
    assert gb(gated_desc(ldg=64), da=at(6), db=at(9)) == CUDA      # over dz
    assert gb(z=at(6)) == CUDA and gb(z=at(7)) == INVALID
    assert gb(eight=True, z=at(2)) == INVALID and gb(eight=True, da=at(4)) == INVALID
    assert gb(gated_desc(rows=1), db=at(7) + HALF) == CUDA and gb(gated_desc(rows=1), db=at(7) + HALF - 2) == INVALID


@no_gpu_only
def test_checkpoint8_refusals():
    lib = iabn.lib()

    def st(rows=16, cols=64, ld=64, dtype=1, form=0, x=at(0), q=at(1), s=at(2)):
        return lib.iabn_checkpoint8_store(rows, cols, ld, dtype, form, x, q, s, None)

    def ld(rows=16, cols=64, ld=64, dtype=1, form=0, x=at(0), q=at(1), s=at(2), g=None, b=None):
        return lib.iabn_checkpoint8_load(rows, cols, ld, dtype, form, q, s, g, b, x, None)

    for f in (st, ld):
        assert f() == CUDA and f(rows=0, x=None, q=None, s=None) == OK
        for kw in (dict(rows=-1), dict(cols=0), dict(ld=63), dict(dtype=5), dict(form=2), dict(x=None),
                   dict(q=None), dict(s=None), dict(q=at(0) + 100)):
            assert f(**kw) == INVALID
        assert f(x=at(0) + 1) == MISALIGNED and f(s=at(2) + 1) == MISALIGNED
        assert f(rows=1 << 41) == UNSUPPORTED and f(cols=1 << 31, ld=1 << 31) == UNSUPPORTED
    assert ld(g=at(3) + 2) == MISALIGNED


# --------------------------------------------------- refusals of the binding

def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1)
    for call in (lambda: iabn.block_norm_forward(x, x, x, x),
                 lambda: iabn.block_norm_forward_checkpoint8(x, x, x, x),
                 lambda: iabn.block_norm_backward(x, x, x, x, x, x, x),
                 lambda: iabn.block_norm_backward_checkpoint8(q, q, x, x, x, x, x),
                 lambda: iabn.gated_forward(x, x, x), lambda: iabn.gated_backward(x, x, x, x, x),
                 lambda: iabn.gated_forward_checkpoint8(x, x, x, q, s, q, s),
                 lambda: iabn.gated_backward_checkpoint8(q, s, q, s, x, x, x),
                 lambda: iabn.checkpoint8_store(x, q, s), lambda: iabn.checkpoint8_load(q, s, x)):
        with pytest.raises(iabn.IabnError, match="not on a CUDA device"):
            call()


def test_binding_refuses_a_missing_tensor():
    x = torch.zeros(4, 64)
    for call in (lambda: iabn.block_norm_forward(x, None, x, x), lambda: iabn.block_norm_forward_checkpoint8(x, None, x, x),
                 lambda: iabn.block_norm_backward(x, x, x, x, None, x, x),
                 lambda: iabn.block_norm_backward_checkpoint8(x, x, x, x, None, x, x),
                 lambda: iabn.gated_forward(x, x, None), lambda: iabn.gated_backward(x, x, None, x, x),
                 lambda: iabn.gated_forward_checkpoint8(x, x, None, x, x, x, x),
                 lambda: iabn.gated_backward_checkpoint8(x, x, x, x, None, x, x),
                 lambda: iabn.checkpoint8_store(None, x, x), lambda: iabn.checkpoint8_load(x, x, None)):
        with pytest.raises(iabn.IabnError, match="is needed"):
            call()


def test_binding_refuses_more_rows_a_gate_than_64_bits_hold():
    """A descriptor would cut 2^64 + 3 to 3, and more gate rows would be read than there are."""
    from place_batchnorm_activation_b200.block import _Call
    c = object.__new__(_Call)
    c.rows, c.cols = 16, 64
    for per in (-1, 1 << 63, (1 << 64) + 3):
        with pytest.raises(iabn.IabnError, match="rows_per_gate"):
            c.gate(torch.zeros(1, 64), "gate", per)


def test_binding_rows_of():
    from place_batchnorm_activation_b200.block import _rows_of
    p = torch.zeros(6, 5, 20)
    assert _rows_of(p, "p") == (30, 20, 20)
    assert _rows_of(p[..., 10:], "p") == (30, 10, 20)
    assert _rows_of(p[:, 0, :10], "p") == (6, 10, 100)
    assert _rows_of(p[0, 0], "p") == (1, 20, 20)
    assert _rows_of(p[:1, :1, 3:], "p") == (1, 17, 17)
    assert _rows_of(p[:, :1, 3:], "p") == (6, 17, 100)
    for bad in (p.transpose(1, 2), p[..., ::2], p[:, :3], torch.zeros(())):
        with pytest.raises(iabn.IabnError):
            _rows_of(bad, "p")


# ------------------------------------------------------ the 64-bit reference

def options(post, pre, cols, rows, per, gated, seed=0, biased=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    on = lambda k, v: v if k else None  # noqa: E731
    n_gates = 1 if per == 0 else -(-rows // per)
    return dict(post=post, pre=pre, eps_post=1e-5, eps_pre=1e-4, residual_scale=0.7, rows_per_gate=per,
                gamma_post=on(post, 1 + 0.3 * r(cols)), beta_post=on(post and biased, r(cols)),
                gate=on(gated, r(n_gates, cols)), gamma_pre=on(pre, 1 + 0.3 * r(cols)),
                beta_pre=on(pre and biased, r(cols)))


@pytest.mark.parametrize("post", [0, 1, 2])
@pytest.mark.parametrize("pre", [0, 1, 2])
@pytest.mark.parametrize("gated,per", [(False, 0), (True, 0), (True, 3)])
def test_reference_gradients_are_those_of_the_reference_forward(post, pre, gated, per):
    """The stated gradients against automatic differentiation of the stated
    forward and against its central differences, in 64 bits."""
    rows, cols = 7, 12
    o = options(post, pre, cols, rows, per, gated, seed=post * 9 + pre * 3 + per)
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    leaves = {"u": r(rows, cols), "h": r(rows, cols)} | {k: v for k, v in o.items() if torch.is_tensor(v)}
    dh_out, dn = r(rows, cols), r(rows, cols)

    def loss(v):
        f = ref.forward(v["u"], v["h"], {**o, **v})
        return (f["h_out"][0] * dh_out).sum() + ((f["n"][0] * dn).sum() if pre else 0.0)

    for v in leaves.values():
        v.requires_grad_(True)
    auto = dict(zip(leaves, torch.autograd.grad(loss(leaves), list(leaves.values()))))
    leaves = {k: v.detach() for k, v in leaves.items()}
    f = ref.forward(leaves["u"], leaves["h"], {**o, **leaves})
    zero = torch.zeros(rows, cols, dtype=torch.float64)
    b = ref.backward(f["uhat"][0], zero, f["xhat"][0] if pre else None, zero, dh_out, dn if pre else None,
                     {**o, **leaves, "rstd_post": f["rstd_post"][0] if post else None,
                      "rstd_pre": f["rstd_pre"][0] if pre else None})
    for k, want in auto.items():
        got = b["d" + k][0].reshape(want.shape)
        assert torch.allclose(got, want, rtol=1e-9, atol=1e-9), k
        step = r(*leaves[k].shape)
        up, down = ({**leaves, k: leaves[k] + s * step} for s in (1e-5, -1e-5))
        slope = (loss(up) - loss(down)) / 2e-5
        assert abs(float(slope) - float((want * step).sum())) < 1e-5 * (1 + abs(float(slope)))


@pytest.mark.parametrize("act,torch_form", [
    (0, torch.nn.functional.silu), (1, torch.nn.functional.gelu),
    (2, lambda a: torch.nn.functional.gelu(a, approximate="tanh"))])
def test_reference_gated_activation(act, torch_form):
    a = torch.linspace(-12, 12, 401, dtype=torch.float64, requires_grad=True)
    b = torch.randn(401, dtype=torch.float64, requires_grad=True)
    dz = torch.randn(401, dtype=torch.float64)
    z = torch_form(a) * b
    da, db = torch.autograd.grad(z, (a, b), dz)
    got = ref.gated(a.detach(), b.detach(), act, torch.float32, dz=dz)
    for k, want in (("z", z.detach()), ("da", da), ("db", db)):
        assert torch.allclose(got[k][0], want, rtol=1e-9, atol=1e-12), k


@pytest.mark.parametrize("form", [torch.float8_e4m3fn, torch.int8])
def test_reference_quantiser(form):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(9, 300, generator=g) * torch.logspace(-30, 30, 9)[:, None]
    x[2], x[3, 128:256], x[4, 5], x[5, 299] = 0.0, 1e-34, float("nan"), float("-inf")
    codes, scale = ref.quantise(x, form)
    v, _ = ref.values(codes, scale)
    assert (v[2] == 0).all() and (v[3, 128:256] == 0).all() and (scale[2] == 0).all()
    assert torch.isnan(v[4, :128]).all() and torch.isnan(v[5, 256:]).all()
    ok = ~torch.isnan(v)
    ok[3, 128:256] = False
    bound = ref.code_bound(x.double(), torch.zeros_like(v), scale, form)
    assert ((v - x.double()).abs()[ok] <= bound[ok]).all()
    assert not torch.isnan(v[4, 128:]).any() and not torch.isnan(v[5, :256]).any()


@pytest.mark.parametrize("form", [torch.float8_e4m3fn, torch.int8])
def test_stated_errors_of_the_checkpoints(form):
    """What the header says of a value's error, with the roundings to fp32: five
    of 2^-24 each of a value that is at most 127 scales (int8), a half-step being
    scale/2, or of 17/16 of a value whose half-step is 2^-4 of it, or of 2^-6
    scales whose half-step is 2^-10 (e4m3): at most 5 * 254 * 2^-24 < 2^-13 of the
    half-step.  The scale is amax * fl(1/Q): the float of amax / Q or the next one."""
    top = ref.QMAX[form]
    g = torch.Generator().manual_seed(7)
    x = torch.randn(64, 512, generator=g) * torch.exp(2 * torch.randn(64, 512, generator=g))
    amax = x.view(64, 4, 128).abs().amax(-1)
    # values on the ties between two codes, where the error is a half-step
    ties = torch.arange(0, 127, dtype=torch.float32) + 0.5
    x[:32, :127] = ties * (amax[:32, :1] / 127.0)
    amax = x.view(64, 4, 128).abs().amax(-1)
    codes, scale = ref.quantise(x, form)
    inverse = torch.tensor(1.0 / top)
    assert torch.equal(scale, amax * inverse)
    ulp = (scale.view(torch.int32) - (amax / top).view(torch.int32)).abs()
    assert int(ulp.max()) == 1        # they do differ, and by no more
    value = (codes.float() * scale.repeat_interleave(128, 1)).double()
    wide = scale.double().repeat_interleave(128, 1)
    half = wide / 2 if form == torch.int8 else torch.maximum(x.double().abs() * 2.0 ** -4, wide * 2.0 ** -10)
    assert ((value - x.double()).abs() <= half * (1 + 2.0 ** -13)).all()
