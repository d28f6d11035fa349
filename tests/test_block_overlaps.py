"""Overlaps of the row operators' tensors (iabn_block.h): an output in the
storage type may be an input in it, as a whole; every other overlap of an
output (codes, scales, statistics, parameter gradients and the workspace
included) with an input or another output is refused.

Without a GPU, on fake addresses: a call whose tensors lie apart gets as far
as the runtime, which has no device."""
import itertools

import pytest

import test_block_host as host
from test_block_host import CUDA, HALF, INVALID, MB, at, desc, gated_desc, no_gpu_only

ROWS, COLS, PER = 16, 64, 4
F = 4                                   # bytes of a float


def meet(call, outputs, inputs, in_place=()):
    """Every pair that may not meet is refused, at either end of either tensor.
    outputs, inputs: {argument: (address, bytes)} as in the call's defaults."""
    assert call() == CUDA
    for (a, (pa, na)), (b, (pb, nb)) in itertools.chain(itertools.permutations(outputs.items(), 2),
                                                        itertools.product(outputs.items(), inputs.items())):
        if (a, b) not in in_place:
            assert call(**{a: pb}) == INVALID, (a, b)
        last = pb + nb - 4 if a != "ws" else pb + (nb - 1) // 16 * 16
        assert call(**{a: last}) == INVALID, (a, b, "at its end")
        first = pb - (na - 1) // 16 * 16 if na > 16 else pb
        if (a, b) not in in_place or first != pb:
            assert call(**{a: first}) == INVALID, (a, b, "at its start")
        assert call(**{a: pb + (nb + 15) // 16 * 16}) == CUDA, (a, b, "behind it")


@no_gpu_only
@pytest.mark.parametrize("eight", [False, True])
def test_forward(eight):
    e = ROWS * COLS
    params = dict(gamma_post=at(10), beta_post=at(11), gate=at(12), gamma_pre=at(13), beta_pre=at(14))
    stats = dict(rstd_post=at(15), rstd_pre=at(16)) | ({} if eight else dict(mean_post=at(17), mean_pre=at(18)))
    d = desc(per=PER, post=2, pre=2)
    call = lambda **kw: (host.fwd8 if eight else host.fwd)(d, **{**params, **stats, **kw})  # noqa: E731
    outputs = dict(h_out=(at(2), 2 * e), n=(at(3), 2 * e)) | {k: (p, F * ROWS) for k, p in stats.items()}
    if eight:
        outputs |= dict(q_post=(at(4), e), scale_post=(at(5), F * ROWS), q_pre=(at(6), e), scale_pre=(at(7), F * ROWS))
    inputs = dict(u=(at(0), 2 * e), h=(at(1), 2 * e))
    inputs |= {k: (p, F * COLS * (ROWS // PER if k == "gate" else 1)) for k, p in params.items()}
    meet(call, outputs, inputs, {(o, i) for o in ("h_out", "n") for i in ("u", "h")})


@no_gpu_only
@pytest.mark.parametrize("eight", [False, True])
def test_backward(eight):
    e = ROWS * COLS
    params = dict(gamma_post=at(10), beta_post=at(11), gate=at(12), gamma_pre=at(13))
    grads = dict(dgamma_post=at(14), dbeta_post=at(15), dgate=at(16), dgamma_pre=at(17), dbeta_pre=at(18))
    stats = {} if eight else dict(mean_post=at(21), mean_pre=at(22))
    d = desc(per=PER, post=2, pre=2)
    call = lambda **kw: host.bwd(d, eight=eight, **{**params, **grads, **stats, **kw})  # noqa: E731
    size = host.iabn.block_norm_workspace_size(ROWS, COLS, PER)
    wide = lambda k, p: (p, F * COLS * (ROWS // PER if k.endswith("gate") else 1))  # noqa: E731
    outputs = dict(dh=(at(6), 2 * e), du=(at(7), 2 * e), ws=(at(20), size)) | {k: wide(k, p) for k, p in grads.items()}
    inputs = dict(dh_out=(at(4), 2 * e), dn=(at(5), 2 * e), rstd_post=(at(8), F * ROWS), rstd_pre=(at(9), F * ROWS))
    inputs |= {k: wide(k, p) for k, p in params.items()} | {k: (p, F * ROWS) for k, p in stats.items()}
    kept = ("dh_out", "dn")
    if eight:
        inputs |= dict(q_post=(at(0), e), scale_post=(at(1), F * ROWS), q_pre=(at(2), e), scale_pre=(at(3), F * ROWS))
    else:
        inputs |= dict(u=(at(0), 2 * e), h_out=(at(2), 2 * e))
        kept += ("u", "h_out")
    meet(call, outputs, inputs, {(o, i) for o in ("dh", "du") for i in kept})
    # what is not read may lie anywhere
    alone = desc(post=0, pre=2)
    assert host.bwd(alone, eight=eight, **stats, **{("q_post" if eight else "u"): at(6)}) == CUDA
    # the workspace may be larger than it has to be, and hold outputs behind what it has to be
    assert call(ws=at(20), ws_bytes=MB, dgamma_pre=at(20) + size) == CUDA
    assert call(ws=at(20), ws_bytes=MB, dgamma_pre=at(20) + size - F) == INVALID


@no_gpu_only
def test_float_outputs_are_not_in_place():
    """fp32 storage, sizes that coincide: still not an output in the storage type."""
    one = desc(rows=1, dtype=0)
    assert host.bwd(one, dgamma_pre=at(5)) == INVALID
    assert host.fwd(desc(cols=1, dtype=0), rstd_pre=at(0)) == INVALID


@no_gpu_only
def test_gated_forward():
    e, scale = ROWS * COLS, F * ROWS
    call = lambda **kw: host.gf(gated_desc(ld=COLS), eight=True, **{**dict(a=at(0), b=at(9)), **kw})  # noqa: E731
    meet(call, dict(z=(at(1), 2 * e), qa=(at(2), e), sa=(at(3), scale), qb=(at(4), e), sb=(at(5), scale)),
         dict(a=(at(0), 2 * e), b=(at(9), 2 * e)), {("z", "a"), ("z", "b")})


@no_gpu_only
def test_gated_backward():
    e, scale = ROWS * COLS, F * ROWS
    call = lambda **kw: host.gb(gated_desc(ldg=COLS), eight=True, **{**dict(da=at(7), db=at(8), z=at(9)), **kw})  # noqa: E731
    meet(call, dict(da=(at(7), 2 * e), db=(at(8), 2 * e), z=(at(9), 2 * e)),
         dict(dz=(at(6), 2 * e), qa=(at(2), e), sa=(at(3), scale), qb=(at(4), e), sb=(at(5), scale)),
         {(o, "dz") for o in ("da", "db", "z")})
    assert host.gb(da=at(0), db=at(0) + HALF) == CUDA


@no_gpu_only
def test_checkpoint8():
    lib, e = host.iabn.lib(), ROWS * COLS

    def store(x=at(0), q=at(1), s=at(2)):
        return lib.iabn_checkpoint8_store(ROWS, COLS, COLS, 1, 0, x, q, s, None)

    def load(y=at(0), q=at(1), s=at(2), g=at(3), b=at(4)):
        return lib.iabn_checkpoint8_load(ROWS, COLS, COLS, 1, 0, q, s, g, b, y, None)

    meet(store, dict(q=(at(1), e), s=(at(2), F * ROWS)), dict(x=(at(0), 2 * e)))
    meet(load, dict(y=(at(0), 2 * e)), dict(q=(at(1), e), s=(at(2), F * ROWS), g=(at(3), F * COLS), b=(at(4), F * COLS)))
