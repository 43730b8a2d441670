"""sv_linear's activations alone: z is a float32 scale (of a row, or of a column) of a product
that is 1, so that it is exact, over the range where an activation is neither 0 nor z, and at
values that are not finite.

Tolerances (from the arithmetic), relative to the result, u = 2^-24:
  * a reciprocal and an exponential by the special function unit (2^-22 each), the products
    around them, and the fit of the normal tail (2^-22): 2^-20 together;
  * an exponential of an argument x that is off by r of itself is off by r |x|: SiLU x = z
    with 3 u; GELU x = z^2 / 2 with 4 u; GELU-tanh x = 2 sqrt(2/pi) (z + 0.044715 z^3) with 8 u;
  * the stored value adds half a step (bf16 2^-8, f32 2^-24).
"""

import math

import numpy as np
import pytest

from oracle import layer as oy
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_linear import OUT, _lib  # noqa: F401  (the fixture builds the library)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


def run(z, act, out, rows):
    """act(z), with `rows` rows that are all alike, or with z as the rows."""
    n = len(z)
    M, N = (rows, n) if rows else (n, 24)
    x = torch.zeros(M, 16, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(N, 16, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = W[:, 0] = 1
    o = torch.empty(M, N, dtype=OUT[out][0], device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    d = torch.from_numpy(z).cuda()
    sb.sv_linear(x, 0, None if rows else d, W, 0, d if rows else None, sb.SV_BF16, None, None, 0, act, o, 0,
                 OUT[out][1], M, N, 16, ws, 256)
    assert sb.sv_read_device_flags(ws) == 0
    o = o.double().cpu().numpy()
    got = o[0] if rows else o[:, 0]
    assert np.array_equal(o, np.broadcast_to(got if rows else got[:, None], o.shape), equal_nan=True)
    return got


def exact(z, act):
    """Without the cancellation that the oracle's 1 + erf has far below 0."""
    if act == sb.SV_ACT_GELU:
        return np.array([0.5 * v * math.erfc(-v / math.sqrt(2)) for v in z])
    if act == sb.SV_ACT_GELU_TANH:
        return z / (1 + np.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return oy.activation(z, act)


ARGUMENT = {sb.SV_ACT_NONE: lambda z: 0 * z, sb.SV_ACT_RELU: lambda z: 0 * z, sb.SV_ACT_SILU: lambda z: 3 * np.abs(z),
            sb.SV_ACT_GELU: lambda z: 2 * z * z,
            sb.SV_ACT_GELU_TANH: lambda z: 16 * math.sqrt(2 / math.pi) * np.abs(z + 0.044715 * z ** 3)}


@pytest.mark.parametrize("rows", [1, 200, 600, 0], ids=["rows", "split", "pair", "by_row"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("act", range(5))
def test_relative_error(act, out, rows):
    r = np.random.default_rng(act)
    z = np.concatenate([np.linspace(-6, 6, 3001), r.normal(size=800), r.normal(size=200) * 1e-4,
                        [0.0, -0.0, 1.0, -1.0, 20.0, 1e4, 3e38]]).astype(np.float32)
    got, ref = run(z, act, out, rows), exact(z.astype(np.float64), act)
    bound = (2.0 ** -20 * (act > 1) + ARGUMENT[act](np.minimum(np.abs(z.astype(np.float64)), 30)) * 2.0 ** -24
             + OUT[out][2] * (1 + 2.0 ** -9)) * np.abs(ref) + 2.0 ** -133
    off = np.abs(got - ref)
    assert np.all(off <= bound), (float(z[np.argmax(off / bound)]), float((off / bound).max()))


@pytest.mark.parametrize("rows", [1, 200, 600, 0], ids=["rows", "split", "pair", "by_row"])
@pytest.mark.parametrize("act", range(5))
def test_values_that_are_not_finite(act, rows):
    """The infinities and NaN become what the formula makes of them (a negative infinity
    times 0 is no number), and so do the largest values."""
    z = np.array([np.inf, -np.inf, np.nan, 3e38, -3e38, 1.0] * 4, np.float32)
    with np.errstate(all="ignore"):
        ref = oy.activation(z.astype(np.float64), act)
    got = run(z, act, "f32", rows)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    keep = ~np.isnan(ref)
    np.testing.assert_allclose(got[keep], ref[keep], rtol=1e-6)
