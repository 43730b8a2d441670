"""sv_linear's scales far from 1: their product is the factor of the sum, whichever kernel a
call's rows select, so a large one and a small one do not leave float32's range between them."""

import numpy as np
import pytest

from oracle import layer as oy
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_linear import Case, _lib, f64  # noqa: F401  (the fixture builds the library)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("big", [2.0 ** 115, 2.0 ** -115])
@pytest.mark.parametrize("M,N,K", [(2, 300, 2048), (40, 300, 64), (100, 200, 136), (200, 260, 2048), (600, 700, 264)])
def test_a_large_scale_and_a_small_one(M, N, K, big):
    c = Case(M, N, K, dtype="e4m3", out="f32", res=False)
    c.x[:, :K] = (c.x[:, :K].float() * 64).to(c.x.dtype)  # (sums up to 2^18)
    c.W[:, :K] = (c.W[:, :K].float() * 64).to(c.W.dtype)
    c.sx *= big
    c.sw /= big
    c.run()
    assert sb.sv_read_device_flags(c.ws) == 0
    ref, absp = oy.linear(f64(c.x)[:, :K], f64(c.W)[:, :K], f64(c.sx), f64(c.sw), f64(c.bias), 0, None)
    # K float32 additions cut or rounded, the two products and the stored value
    bound = (K + 8) * 2.0 ** -23 * absp + 2.0 ** -22 * (np.abs(ref) + 4)
    assert np.all(np.abs(f64(c.o) - ref) <= bound)


def test_the_same_bits_from_every_kernel():
    """A row's results do not depend on how many rows a call has, where its sum is one chain."""
    K, N = 64, 300
    c = Case(600, N, K, dtype="e4m3", out="f32", act=sb.SV_ACT_SILU)
    want = c.run().o.clone()
    for M in (1, 17, 40, 100, 129, 300):
        o = torch.empty(M, N, device="cuda")
        sb.sv_linear(c.x[:M], c.x.stride(0), c.sx[:M], c.W, c.W.stride(0), c.sw, c.code, c.bias, c.res[:M], 0,
                     sb.SV_ACT_SILU, o, 0, sb.SV_F32, M, N, K, c.ws, c.ws.numel())
        assert torch.equal(o, want[:M]), M
