"""GPU parity of sv_linear_w4 against the float64 product of the weights that its codes stand for."""

import numpy as np
import pytest

from oracle import draft4 as o4
from oracle import layer as oy
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


def f64(t):
    return t.double().cpu().numpy()


def inputs(seed, M, N, K, group, zeros, bias, res, out):
    g = torch.Generator().manual_seed(seed)
    return {"x": torch.randn(M, K, generator=g).to(BF), "W": torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8),
            "scales": (0.01 + torch.rand(N, K // group, generator=g) * 0.05).to(BF),
            "zeros": torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None,
            "bias": torch.randn(N, generator=g).to(BF) if bias else None,
            "res": torch.randn(M, N, generator=g).to(out) if res else None}


def run(s, M, N, K, group, act, out_type, ldx=0, ldw=0, ldr=0, ldo=0, out=None, x=None, W=None, res=None, stream=None):
    cuda = lambda t: None if t is None else t.cuda()
    ws = torch.zeros(sb.sv_linear_w4_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((M, N), float("nan"), dtype=out_type, device="cuda")
    sb.sv_linear_w4(cuda(s["x"]) if x is None else x, ldx, cuda(s["W"]) if W is None else W, ldw, cuda(s["scales"]),
                    cuda(s["zeros"]), group, cuda(s["bias"]), cuda(s["res"]) if res is None else res, ldr, act, out, ldo,
                    sb.SV_F32 if out_type == torch.float32 else sb.SV_BF16, M, N, K, ws, ws.numel(), stream)
    assert sb.sv_read_device_flags(ws) == 0
    return out


def check(s, got, act, out_type, group):
    """Codes less zeros are exact; a tensor-core sum of a group is off by at most 128 cuts of 2^-23 of
    its terms' absolute sum, the groups' sums by less: 2^-15 of it over an activation of slope at most
    1.13; the rounding of the output."""
    W = o4.weights(s["W"].numpy(), f64(s["scales"]), None if s["zeros"] is None else s["zeros"].numpy(), group)
    opt = lambda t: None if t is None else f64(t)
    ref, absp = oy.linear(f64(s["x"]), W, None, None, opt(s["bias"]), act, opt(s["res"]))
    half = torch.finfo(out_type).eps / 2
    z = np.abs(absp) + (0 if s["bias"] is None else np.abs(f64(s["bias"]))[None])
    extra = 0 if s["res"] is None else 2.0 ** -24 * np.abs(f64(s["res"]))
    bound = 2.0 ** -15 * absp + 2.0 ** -20 * z + half * np.abs(ref) * (1 + 2.0 ** -8) + extra
    off = np.abs(f64(got) - ref)
    assert np.all(off <= bound), np.max(off / bound)


SHAPES = [(1, 4096, 512), (1, 16, 32), (2, 33, 96), (3, 1, 128), (8, 1999, 1024), (9, 257, 256), (16, 4096, 2048),
          (17, 100, 160), (40, 12000, 384), (64, 700, 640), (130, 64, 128), (1, 10000, 4096), (5, 9800, 192)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_linear_w4_matches_the_product(M, N, K, group):
    if K % group:
        K = -(-K // group) * group
    for i, (zeros, bias, res, act, out) in enumerate([(True, True, True, sb.SV_ACT_SILU, BF),
                                                      (False, False, False, sb.SV_ACT_NONE, torch.float32)]):
        s = inputs(M * 7 + N + K + i, M, N, K, group, zeros, bias, res, out)
        check(s, run(s, M, N, K, group, act, out), act, out, group)


@pytest.mark.parametrize("act", range(5))
@pytest.mark.parametrize("out", [BF, torch.float32])
def test_linear_w4_epilogues(act, out):
    s = inputs(act, 6, 200, 256, 64, True, True, True, out)
    check(s, run(s, 6, 200, 256, 64, act, out), act, out, 64)


@pytest.mark.parametrize("M,N", [(3, 77), (20, 9999)])
def test_linear_w4_strides(M, N):
    """Rows inside wider arrays, a residual that is the output, odd output strides."""
    K, group = 192, 64
    s = inputs(3, M, N, K, group, True, True, True, BF)
    x = torch.full((M, K + 24), float("nan"), dtype=BF, device="cuda")
    x[:, :K] = s["x"].cuda()
    W = torch.full((N, K // 2 + 32), 255, dtype=torch.uint8, device="cuda")
    W[:, :K // 2] = s["W"].cuda()
    out = torch.full((M, N + 3), 7.0, dtype=BF, device="cuda")
    out[:, :N] = s["res"].cuda()
    run(s, M, N, K, group, sb.SV_ACT_GELU, BF, ldx=K + 24, ldw=K // 2 + 32, ldr=N + 3, ldo=N + 3, out=out, x=x, W=W, res=out)
    check(s, out[:, :N], sb.SV_ACT_GELU, BF, group)
    assert torch.all(out[:, N:] == 7.0)


def test_linear_w4_rows_do_not_meet():
    """A row's output is the same in every batch of a kernel; values that are not finite stay in
    their row or column."""
    s = inputs(4, 16, 300, 512, 128, True, False, False, torch.float32)
    whole = run(s, 16, 300, 512, 128, sb.SV_ACT_NONE, torch.float32)
    s2 = dict(s, x=s["x"].clone(), scales=s["scales"].clone())
    s2["x"][5, 100], s2["x"][7, 3] = float("inf"), float("nan")
    s2["scales"][11, 2] = float("nan")
    got = run(s2, 16, 300, 512, 128, sb.SV_ACT_NONE, torch.float32)
    keep = torch.ones(16, 300, dtype=torch.bool)
    keep[[5, 7]] = False
    keep[:, 11] = False
    assert torch.equal(got.cpu()[keep], whole.cpu()[keep])
    assert not torch.isfinite(got[7]).any() and torch.isnan(got[:, 11]).all()


def test_linear_w4_large_values():
    """Scales and rows far from 1, and rows whose sums are large against their terms' signs."""
    s = inputs(5, 4, 128, 1024, 32, True, False, False, BF)
    s["x"] = (s["x"].double() * torch.tensor([1e-30, 1e30, 1.0, 1e-3]).double()[:, None]).to(BF)
    check(s, run(s, 4, 128, 1024, 32, 0, BF), 0, BF, 32)
    s = inputs(6, 4, 128, 1024, 32, False, False, False, torch.float32)
    s["x"] = (s["x"].float().abs() + 10).to(BF)
    check(s, run(s, 4, 128, 1024, 32, 0, torch.float32), 0, torch.float32, 32)


def test_linear_w4_streams_and_graphs():
    M, N, K, group = 7, 500, 256, 64
    s = inputs(7, M, N, K, group, True, True, False, BF)
    want = run(s, M, N, K, group, 1, BF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = run(s, M, N, K, group, 1, BF, stream=side)
    side.synchronize()
    assert torch.equal(other, want)
    d = {k: None if v is None else v.cuda() for k, v in s.items()}
    out = torch.empty(M, N, dtype=BF, device="cuda")
    ws = torch.zeros(sb.sv_linear_w4_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sb.sv_linear_w4(d["x"], 0, d["W"], 0, d["scales"], d["zeros"], group, d["bias"], None, 0, 1, out, 0, sb.SV_BF16, M,
                        N, K, ws, ws.numel())
    out.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("M", [9, 20, 64])
@pytest.mark.parametrize("N,K,group", [(5, 32, 32), (130, 64, 64), (1, 64, 32), (129, 128, 128), (300, 96, 32)])
def test_linear_w4_of_less_than_a_block(M, N, K, group):
    """K below a block's 128, rows below a tile's: what the copies' boxes reach outside of counts nothing."""
    s = inputs(M + N + K, M, N, K, group, True, True, False, torch.float32)
    check(s, run(s, M, N, K, group, sb.SV_ACT_NONE, torch.float32), sb.SV_ACT_NONE, torch.float32, group)


@pytest.mark.parametrize("M,N,K,group", [(64, 128, 8192, 32), (50, 200, 32768, 32), (17, 128, 16384, 32), (16, 64, 16384, 128)])
def test_linear_w4_many_blocks(M, N, K, group):
    """Every ring comes round many times, with one block of accumulators and with several."""
    s = inputs(M + N, M, N, K, group, True, False, False, torch.float32)
    first = run(s, M, N, K, group, sb.SV_ACT_NONE, torch.float32)
    check(s, first, sb.SV_ACT_NONE, torch.float32, group)
    for _ in range(20):
        assert torch.equal(run(s, M, N, K, group, sb.SV_ACT_NONE, torch.float32), first)
