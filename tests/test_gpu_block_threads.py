"""The row operators (iabn_block.h) called by several host threads at once:
every call is taken, and each gives the bits of a call by itself."""
import ctypes
import os
import shutil
import subprocess

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import place_batchnorm_activation_b200 as iabn  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class ConcurrentCall(ctypes.Structure):
    _fields_ = [("desc", iabn.IabnBlockDesc)] + [(k, ctypes.c_void_p) for k in ("u", "h", "h_out", "n", "beta_pre", "stream")] \
        + [("refused", ctypes.c_long)]


@pytest.mark.parametrize("widths", [(1536, 4096), (1536, 2560, 3584, 4096), (4608, 8192)])
def test_widths_of_one_kernel_from_several_threads(tmp_path, widths):
    """Widths that one kernel serves with different amounts of shared memory."""
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    so = tmp_path / "concurrent_calls.so"
    subprocess.run(["gcc", "-std=gnu11", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-pthread", "-I",
                    os.path.join(ROOT, "include"), os.path.join(ROOT, "tests", "c", "concurrent_calls.c"), "-o", str(so)],
                   check=True)
    keep, calls = [], (ConcurrentCall * len(widths))()
    for k, cols in enumerate(widths):
        u, h, beta = (torch.randn(s, device="cuda") for s in ((3, cols), (3, cols), (cols,)))
        u, h = u.bfloat16(), h.bfloat16()
        want = [torch.empty_like(u) for _ in range(2)]
        iabn.block_norm_forward(u, h, *want, beta_pre=beta)
        got, stream = [torch.zeros_like(u) for _ in range(2)], torch.cuda.Stream()
        d = iabn.IabnBlockDesc(3, cols, 0, iabn.IABN_BF16, iabn.IABN_NORM_RMS, iabn.IABN_NORM_RMS, 0, 1.0, 1e-6, 1e-6)
        calls[k] = ConcurrentCall(d, u.data_ptr(), h.data_ptr(), got[0].data_ptr(), got[1].data_ptr(), beta.data_ptr(),
                                  stream.cuda_stream, 0)
        keep.append((u, h, beta, want, got, stream))
    torch.cuda.synchronize()
    f = ctypes.CDLL(str(so)).concurrent_forward
    f.argtypes = [ctypes.c_void_p, ctypes.POINTER(ConcurrentCall), ctypes.c_int, ctypes.c_long]
    entry = ctypes.cast(iabn.lib().iabn_block_norm_forward, ctypes.c_void_p)
    assert f(entry, calls, len(widths), 20000) == 0
    torch.cuda.synchronize()
    assert [c.refused for c in calls] == [0] * len(widths)
    for _, _, _, want, got, _ in keep:
        assert all(torch.equal(a, b) for a, b in zip(want, got))
