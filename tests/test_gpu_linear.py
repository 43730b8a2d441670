"""GPU parity of sv_linear against the float64 oracle.

Tolerances (from the arithmetic): K float32 additions of exact products, each
off by at most one step of the running sum (2^-23: the tensor cores may cut
instead of rounding), bounded by (K + 8) * 2^-23 * sum |x W| sx sw; the
activations' slope is at most 1.13 and their own float32 error at most 2^-18 of
|z| + 2^-18; the stored value adds half a step (bf16 2^-8, f32 2^-24).
"""

import numpy as np
import pytest

from oracle import layer as oy
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

IN = {"bf16": (torch.bfloat16, sb.SV_BF16, 8), "e4m3": (torch.float8_e4m3fn, sb.SV_E4M3, 16)}
OUT = {"bf16": (torch.bfloat16, sb.SV_BF16, 2.0 ** -8), "f32": (torch.float32, sb.SV_F32, 2.0 ** -24)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


def f64(t):
    return None if t is None else t.double().cpu().numpy()


class Case:
    def __init__(self, M, N, K, dtype="bf16", out="bf16", act=0, scales=True, bias=True, res=True, seed=0,
                 pad=0, pad_value=float("nan"), inplace=False, ldo=None):
        g = torch.Generator(device="cuda").manual_seed(seed * 7919 + M * 31 + N * 7 + K)
        t, self.code, unit = IN[dtype]
        self.M, self.N, self.K, self.act, self.out = M, N, K, act, out

        def rows(n, scale):
            ld = -(-K // unit) * unit + pad * unit
            buf = torch.full((n, ld), pad_value, device="cuda").to(t)
            buf[:, :K] = (torch.randn(n, K, generator=g, device="cuda") * scale).to(t)
            return buf
        self.x, self.W = rows(M, 1.0), rows(N, 1.0 if dtype == "e4m3" else 0.3)
        scales = scales and (dtype == "e4m3" or scales == "both")
        self.sx = torch.rand(M, generator=g, device="cuda") + 0.5 if scales else None
        self.sw = torch.rand(N, generator=g, device="cuda") + 0.5 if scales else None
        self.bias = torch.randn(N, generator=g, device="cuda").to(torch.bfloat16) if bias else None
        self.ldo = ldo or N
        self.o = torch.full((M, self.ldo), 77.0, dtype=OUT[out][0], device="cuda")
        self.res = None
        if res:
            self.res = torch.randn(M, N, generator=g, device="cuda").to(OUT[out][0])
            if inplace:
                self.o[:, :N] = self.res
        self.inplace = inplace and res
        self.ws = torch.zeros(sb.sv_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")

    def run(self, stream=None):
        r = self.o if self.inplace else self.res
        sb.sv_linear(self.x, self.x.stride(0), self.sx, self.W, self.W.stride(0), self.sw, self.code, self.bias,
                     r, (self.ldo if self.inplace else 0), self.act, self.o, self.ldo, OUT[self.out][1], self.M,
                     self.N, self.K, self.ws, self.ws.numel(), stream)
        return self

    def check(self):
        assert sb.sv_read_device_flags(self.ws) == 0
        x, W = f64(self.x)[:, :self.K], f64(self.W)[:, :self.K]
        ref, absp = oy.linear(x, W, f64(self.sx), f64(self.sw), f64(self.bias), self.act, f64(self.res))
        got = f64(self.o)
        half = OUT[self.out][2]
        bound = 1.13 * ((self.K + 8) * 2.0 ** -23 * absp) + 2.0 ** -18 * (absp + 4) * (self.act != 0)
        bound = bound + 2.0 ** -21 * (absp + 4) + (half + 2.0 ** -23) * (np.abs(ref) + bound)
        off = np.abs(got[:, :self.N] - ref)
        assert np.all(off <= bound), float(np.nanmax(off / bound))
        assert (got[:, self.N:] == 77.0).all()
        return got[:, :self.N]


SHAPES = [(1, 1, 1), (1, 4096, 4096), (2, 130, 64), (7, 33, 100), (15, 16, 15), (16, 1999, 1000),
          (17, 128, 129), (31, 257, 520), (33, 640, 72), (64, 129, 2056), (65, 1000, 64), (100, 96, 1),
          (128, 512, 512), (129, 256, 200), (200, 77, 333), (256, 1024, 128), (257, 300, 1032),
          (500, 129, 65), (513, 1025, 257), (1100, 2000, 192), (3, 20000, 48), (40, 5, 9000)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=["x".join(map(str, s)) for s in SHAPES])
def test_shapes(shape, dtype, out):
    Case(*shape, dtype=dtype, out=out).run().check()


@pytest.mark.parametrize("M", [1, 48, 300])
@pytest.mark.parametrize("act", range(5))
def test_activations(act, M):
    Case(M, 264, 136, act=act, out="f32", res=False).run().check()
    Case(M, 265, 136, act=act, dtype="e4m3", bias=False).run().check()


@pytest.mark.parametrize("M", [3, 40, 129, 400])
def test_optional_arguments(M):
    for scales, bias, res in [(False, False, False), (True, False, False), (False, True, False),
                              (False, False, True)]:
        Case(M, 150, 96, dtype="e4m3", scales=scales, bias=bias, res=res).run().check()
    Case(M, 150, 96, dtype="bf16", scales="both", out="f32").run().check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("M", [2, 96, 260])
def test_padded_rows(M, dtype):
    """Row strides beyond K and N: NaN between K and the stride never reaches a
    result, and columns behind N stay as they were."""
    for K, ldo in [(100, 151), (64, 152), (17, 160)]:
        Case(M, 150, K, dtype=dtype, pad=1, ldo=ldo, seed=K).run().check()


@pytest.mark.parametrize("M", [1, 50, 200, 600])
def test_residual_over_the_output(M):
    a = Case(M, 390, 128, seed=4).run()
    b = Case(M, 390, 128, seed=4, inplace=True, ldo=396).run()
    np.testing.assert_array_equal(a.check(), b.check())


@pytest.mark.parametrize("M", [1, 16, 150])
def test_unaligned_epilogue_pointers(M):
    """Bias, residual and output at an odd element: only their own alignment is needed."""
    c = Case(M, 320, 64, seed=9)
    bias = torch.zeros(321, dtype=torch.bfloat16, device="cuda")
    bias[1:] = c.bias
    res = torch.zeros(M * 320 + 1, dtype=torch.bfloat16, device="cuda")
    res[1:] = c.res.reshape(-1)
    out = torch.full((M * 320 + 1,), 77.0, dtype=torch.bfloat16, device="cuda")
    sb.sv_linear(c.x, 0, None, c.W, 0, None, c.code, bias[1:], res[1:], 0, 0, out[1:], 0, sb.SV_BF16, M, 320, 64,
                 c.ws, c.ws.numel())
    want = c.run().check()
    np.testing.assert_array_equal(f64(out[1:]).reshape(M, 320), want)
    assert out[0].item() == 77.0


@pytest.mark.parametrize("M", [4, 140])
def test_values_that_are_not_finite_stay_where_the_formula_has_them(M):
    c = Case(M, 200, 64, dtype="bf16", out="f32", res=False)
    c.x[2, 5] = float("nan")
    c.W[7, 3] = float("inf")
    got = c.run().o
    bad = ~torch.isfinite(got)
    assert bad[2].all() and bad[:, 7].all()
    bad[2] = False
    bad[:, 7] = False
    assert not bad.any()


def test_long_sums():
    """K of 16384 into 32 bits: the error stays near the float32 sums of the plain form."""
    for dtype in ("bf16", "e4m3"):
        for M in (4, 200):
            c = Case(M, 256, 16384, dtype=dtype, out="f32", bias=False, res=False, scales=False).run()
            got = c.check()
            ref, _ = oy.linear(f64(c.x), f64(c.W), None, None, None, 0, None)
            assert np.linalg.norm(got - ref) <= 5e-6 * np.linalg.norm(ref), (
                dtype, M, np.linalg.norm(got - ref) / np.linalg.norm(ref))


@pytest.mark.parametrize("M", [1, 30, 700])
def test_same_inputs_same_bits(M):
    a = Case(M, 1030, 2056, seed=2).run().o.clone()
    for _ in range(3):
        assert torch.equal(a, Case(M, 1030, 2056, seed=2).run().o)


@pytest.mark.parametrize("M", [1, 24, 300])
def test_stream_and_graph(M):
    c = Case(M, 520, 264, seed=3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c.run()
    st.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
        c.run()
    for k in (1, 2):
        c.x.copy_(torch.randn(M, c.x.shape[1], device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        c.check()


def test_two_streams_at_once():
    """Calls on two streams share nothing but the flag word."""
    a, b = Case(8, 4096, 2048, seed=1), Case(300, 4096, 2048, seed=2)
    b.ws = a.ws
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
    torch.cuda.synchronize()
    a.check()
    b.check()
