"""A call whose launch the CUDA runtime refuses returns SV_ERR_CUDA, and the calls behind it are as good as before.

The refusal is the runtime's own, on the host: a launch into the legacy stream while another stream of
the same context captures a graph in the global mode.  Nothing is enqueued by it; the capture ends without a graph."""

import ctypes

import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


def runtime():
    for name in ("libcudart.so.13", "libcudart.so", "/usr/local/cuda/lib64/libcudart.so"):
        try:
            return ctypes.CDLL(name)
        except OSError:
            continue
    pytest.skip("no shared CUDA runtime to capture with")


def test_calls_behind_a_refused_launch():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()
    rt = runtime()
    H, D, page = 1, 64, 16
    x = torch.randn(1, 4, H, D, device="cuda").bfloat16()
    pool = torch.zeros(2, sb.sv_kv4_page_bytes(H, D, page), dtype=torch.uint8, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    table, starts, ws = i32(0).reshape(1, 1), i32(0), torch.zeros(64, dtype=torch.uint8, device="cuda")
    out = torch.zeros(4, 40, device="cuda", dtype=torch.bfloat16)
    W, s = torch.zeros(40, 32, dtype=torch.uint8, device="cuda"), torch.zeros(40, 1, dtype=torch.bfloat16, device="cuda")
    wl = torch.zeros(sb.sv_linear_w4_workspace_size(4, 40, 64), dtype=torch.uint8, device="cuda")
    wp = torch.zeros(sb.sv_kv_pages_workspace_size(2, 1), dtype=torch.uint8, device="cuda")
    src, dst = i32(0), i32(1)

    calls = [
        lambda st: sb.sv_kv4_append(x, x, 0, 0, 0, sb.SV_BF16, pool, 2, page, table, 1, starts, None, 1, 4, H, D, ws, 4, st),
        lambda st: sb.sv_linear_w4(x, 64, W, 0, s, None, 64, None, None, 0, 0, out, 0, sb.SV_BF16, 4, 40, 64, wl, wl.numel(), st),
        lambda st: sb.sv_kv_copy_pages([pool], [pool.shape[1]], 1, 2, src, dst, 1, wp, wp.numel(), st),
    ]
    good = torch.cuda.Stream()
    for call in calls:
        call(good)  # (attributes and properties are set up outside of a capture)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    handle = ctypes.c_void_p()
    assert rt.cudaStreamCreate(ctypes.byref(handle)) == 0  # (a stream that the legacy stream waits for)
    for call in calls:
        assert rt.cudaStreamBeginCapture(handle, 0) == 0
        try:
            with pytest.raises(sb.SVError) as refused:
                call(0)
            assert refused.value.status == sb.SV_ERR_CUDA
        finally:
            graph = ctypes.c_void_p()
            rt.cudaStreamEndCapture(handle, ctypes.byref(graph))
            rt.cudaGetLastError()
        pool.zero_()
        torch.cuda.synchronize()
        for again in calls:
            again(other)
        other.synchronize()
        assert pool[0].any() and torch.equal(pool[0], pool[1])
    assert rt.cudaStreamDestroy(handle) == 0
