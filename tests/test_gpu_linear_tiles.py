"""GPU parity of sv_linear's large products: every tile shape of the pair kernel, with
several tiles per CTA pair (so that the ring, the accumulators and the column buffers are
carried from tile to tile), more than one band of eight row tiles, and ragged ends.

The shapes are those for which the rule in csrc/sv_linear.cu picks the named tile on a card
of 152 SMs; elsewhere they are products like any other.  The reference is a float64 product on
the GPU; tolerances are those of test_gpu_linear.py.
"""

import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_linear import OUT, Case, _lib  # noqa: F401  (the fixture builds the library)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


def activation(z, act):
    if act == sb.SV_ACT_RELU:
        return z.clamp(min=0)
    if act == sb.SV_ACT_SILU:
        return z / (1 + torch.exp(-z))
    if act == sb.SV_ACT_GELU:
        return 0.5 * z * torch.special.erfc(-z * 0.5 ** 0.5)
    if act == sb.SV_ACT_GELU_TANH:
        return z / (1 + torch.exp(-2 * (2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def check(c):
    assert sb.sv_read_device_flags(c.ws) == 0
    x, W = c.x[:, :c.K].double(), c.W[:, :c.K].double()
    if c.sx is not None:
        x, W = x * c.sx.double()[:, None], W * c.sw.double()[:, None]
    z, absp = x @ W.T, x.abs() @ W.abs().T
    if c.bias is not None:
        z = z + c.bias.double()
    ref = activation(z, c.act)
    if c.res is not None:
        ref = ref + c.res.double()
    bound = 1.13 * ((c.K + 8) * 2.0 ** -23 * absp) + 2.0 ** -18 * (absp + 4) * (c.act != 0)
    bound = bound + 2.0 ** -21 * (absp + 4)
    bound = bound + (OUT[c.out][2] + 2.0 ** -23) * (ref.abs() + bound)
    off = (c.o[:, :c.N].double() - ref).abs()
    wrong = ~(off <= bound)
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[:4].tolist(), float((off / bound).max()))
    assert (c.o[:, c.N:] == 77.0).all()


# M, N, K, operands, output, residual, activation: rows and columns of the tile
TILES = [
    (2061, 2058, 264, "bf16", "bf16", False, 0),     # 256 x 128
    (3109, 1922, 264, "e4m3", "f32", False, 0),      # 256 x 128
    (4099, 3087, 264, "e4m3", "bf16", True, 3),      # 512 x 128
    (4108, 3076, 48, "bf16", "f32", False, 3),       # 512 x 128
    (2052, 4260, 264, "bf16", "bf16", True, 0),      # 256 x 192
    (2060, 4233, 264, "e4m3", "f32", False, 0),      # 256 x 192
    (4382, 4245, 264, "e4m3", "bf16", True, 3),      # 512 x 192
    (4354, 4227, 48, "bf16", "f32", True, 0),        # 512 x 192
    (2053, 5394, 264, "bf16", "bf16", True, 0),      # 256 x 224
    (2066, 5377, 264, "e4m3", "f32", False, 0),      # 256 x 224
    (4366, 5392, 264, "e4m3", "bf16", False, 3),     # 512 x 224
    (4101, 5395, 48, "bf16", "f32", True, 0),        # 512 x 224
    (8192, 4096, 4096, "bf16", "bf16", False, 2),    # 512 x 224
    (512, 16384, 4096, "e4m3", "bf16", False, 3),    # 512 x 224
    (2307, 4933, 776, "bf16", "bf16", False, 0),     # 256 x 256
    (2315, 4932, 776, "bf16", "f32", False, 0),      # 256 x 256
    (8192, 4096, 1608, "bf16", "bf16", False, 4),    # 256 x 256
    (8192, 4096, 1024, "bf16", "bf16", True, 0),     # 256 x 224
    (4360, 5894, 48, "bf16", "bf16", True, 0),       # 512 x 256
    (4098, 6277, 48, "e4m3", "bf16", True, 0),       # 512 x 256
    (2600, 4700, 2120, "bf16", "f32", True, 1),      # 256 x 256, sums in chunks of k blocks
    (2305, 2100, 4200, "e4m3", "f32", False, 0),     # the same
    (2300, 1900, 2120, "bf16", "f32", False, 0),     # 256 x 128, sums in chunks of k blocks
    (2300, 1900, 4200, "e4m3", "f32", True, 2),      # the same
]


@pytest.mark.parametrize("M,N,K,dtype,out,res,act", TILES, ids=["x".join(map(str, t)) for t in TILES])
def test_tiles(M, N, K, dtype, out, res, act):
    c = Case(M, N, K, dtype=dtype, out=out, res=res, act=act)
    c.run()
    check(c)
    first = c.o.clone()
    c.o.fill_(77.0)
    c.run()
    assert torch.equal(c.o, first)


@pytest.mark.parametrize("M,N,K,dtype,out", [(4366, 5393, 264, "bf16", "bf16"), (2307, 4933, 776, "e4m3", "f32")])
def test_large_products_over_their_residual(M, N, K, dtype, out):
    """In place, in rows wider than N."""
    c = Case(M, N, K, dtype=dtype, out=out, inplace=True, ldo=N + 3, pad=1)
    c.run()
    check(c)
