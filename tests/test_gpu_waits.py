"""A bounded wait that runs out: the call ends, reports SV_FLAG_TIMEOUT and leaves NaN, never
results of an earlier call; the next call is sound.  The waits are told to give up without a
try, so that the copies and products on their way have to be waited for at the kernel's end."""

import contextlib

import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_attention import SENTINEL
from tests.test_gpu_attention import Case as Attention
from tests.test_gpu_attention import _lib  # noqa: F401  (the fixture builds the library)
from tests.test_gpu_linear import Case as Linear

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@contextlib.contextmanager
def no_patience():
    sb.lib().sv_internal_wait_tries(0)
    try:
        yield
        torch.cuda.synchronize()
    finally:
        sb.lib().sv_internal_wait_tries(-1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,page", [(1, 16), (40, 16), (3, 7)])
def test_attention(B, page, D):
    c = Attention([300 + 3 * b for b in range(B)], [b % 3 for b in range(B)], 2, prefix=200, page=page, D=D)
    c.run().check()  # parts of an earlier call lie in the workspace
    c.out.fill_(SENTINEL)
    c.lse.fill_(SENTINEL)
    with no_patience():
        c.run()
    assert sb.sv_read_device_flags(c.ws) == sb.SV_FLAG_TIMEOUT
    for b in range(B):
        k = int(c.ks[b])
        assert torch.isnan(c.out[b, :k + 1]).all() and torch.isnan(c.lse[b, :k + 1]).all()
        assert (c.out[b, k + 1:] == SENTINEL).all() and (c.lse[b, k + 1:] == SENTINEL).all()
    c.run().check()


# M, N, K, output: one CTA and a cluster per tile of few rows; clusters that share K; pairs with
# one tile, with more tiles than accumulators, and with sums in chunks
@pytest.mark.parametrize("act", [sb.SV_ACT_NONE, sb.SV_ACT_RELU, sb.SV_ACT_GELU])
@pytest.mark.parametrize("M,N,K,out", [(3, 200, 64, "bf16"), (100, 30000, 64, "f32"), (7, 300, 4096, "bf16"),
                                       (256, 500, 2048, "bf16"), (300, 1030, 128, "f32"), (2500, 5000, 264, "bf16"),
                                       (300, 300, 4096, "f32")])
def test_linear(M, N, K, out, act):
    c = Linear(M, N, K, out=out, act=act, ldo=N + 3)
    with no_patience():
        c.run()
    assert sb.sv_read_device_flags(c.ws) == sb.SV_FLAG_TIMEOUT
    assert torch.isnan(c.o[:, :N]).all() and (c.o[:, N:] == 77.0).all()
    c.ws.zero_()
    c.run()
    assert sb.sv_read_device_flags(c.ws) == 0
    assert not torch.isnan(c.o).any()
    got = c.o.clone()
    c.o.fill_(0)
    c.run()
    assert torch.equal(got[:, :N], c.o[:, :N])


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("out", ["e4m3", "bf16"])
def test_norm(out, inplace):
    """Rows that come through the ring of copies; the sum in a place of its own and over the
    residual, whose later rows are still on their way when the waits run out."""
    M, H = 700, 4104
    x, r = (torch.randn(M, H, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")

    def call():
        res = r.clone()
        s = res if inplace else torch.zeros_like(r)
        y = torch.zeros(M, H + 8, dtype=torch.uint8 if out == "e4m3" else torch.bfloat16, device="cuda")
        c = torch.zeros(M, device="cuda") if out == "e4m3" else None
        sb.sv_rmsnorm_residual(x, 0, res, 0, w, 1e-5, s, 0, sb.SV_BF16, y, H + 8,
                               sb.SV_E4M3 if out == "e4m3" else sb.SV_BF16, c, M, H)
        return (y.view(torch.float8_e4m3fn).float() if out == "e4m3" else y), c, s

    with no_patience():
        y, c, s = call()
    assert torch.isnan(y[:, :H]).all() and torch.isnan(s).all() and (y[:, H:] == 0).all()
    assert c is None or torch.isnan(c).all()
    y, c, s = call()
    assert torch.isfinite(y).all() and torch.equal(s, (x.float() + r.float()).to(torch.bfloat16))
    assert c is None or torch.isfinite(c).all()
