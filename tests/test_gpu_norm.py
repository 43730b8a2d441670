"""GPU parity of sv_rmsnorm_residual against the float64 oracle.

Tolerances (from the arithmetic): the row's sum of squares is a float32 sum of
at most H / 32 terms per thread and ten steps of a tree, so r = rsqrt(..) is off
by at most (H / 32 + 20) * 2^-25 relative; with the products, 2^-17 up to
H = 8192 and H * 2^-30 beyond.  A bf16 result adds half a step, 2^-8.  The
stored sum is one float32 addition rounded once: equal to torch's.
"""

import numpy as np
import pytest

from oracle import layer as oy
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

DT = {"bf16": (torch.bfloat16, sb.SV_BF16), "f32": (torch.float32, sb.SV_F32)}
OUT = {"bf16": (torch.bfloat16, sb.SV_BF16), "e4m3": (torch.float8_e4m3fn, sb.SV_E4M3)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from speculative_decoding_verification_47_gb300 import build
    build.build()
    sb.lib()


def f64(t):
    return t.double().cpu().numpy()


def run(x, res, w, out, eps=1e-5, summed=True, ldo=0, stream=None):
    """x, res: row-strided views.  Returns out, scale, sum."""
    M, H = x.shape
    dt = sb.SV_BF16 if x.dtype == torch.bfloat16 else sb.SV_F32
    y = torch.zeros(M, ldo or H, dtype=torch.uint8 if out == "e4m3" else torch.bfloat16, device="cuda")
    c = torch.full((M,), -7.0, device="cuda") if out == "e4m3" else None
    s = torch.empty(M, H, dtype=x.dtype, device="cuda") if summed else None
    sb.sv_rmsnorm_residual(x, x.stride(0), res, res.stride(0) if res is not None else 0, w, eps, s, 0,
                           dt, y, ldo, OUT[out][1], c, M, H, stream)
    return (y.view(torch.float8_e4m3fn) if out == "e4m3" else y), c, s


def check(x, res, w, out, y, c, s, eps=1e-5):
    H = x.shape[1]
    rel = max(2.0 ** -17, H * 2.0 ** -30)
    es, ey = oy.rmsnorm_residual(f64(x), None if res is None else f64(res), f64(w), eps)
    if s is not None:
        want = (x.float() + (0 if res is None else res.float())).to(x.dtype)
        assert torch.equal(s, want)
    got = f64(y)[:, :H]
    if out == "bf16":
        assert np.all(np.abs(got - ey) <= (2.0 ** -8 + 2 * rel) * np.abs(ey) + 2.0 ** -133)
        return
    scale = oy.row_scale(ey)
    gc = f64(c)
    assert np.all(np.abs(gc - scale) <= rel * scale)
    # each value is a nearest e4m3 value of y / scale, up to the float32 error of that quotient
    v = ey / gc[:, None]
    grid = oy.e4m3_values()
    a = np.minimum(np.abs(v), grid[-1])
    i = np.searchsorted(grid, a)
    lo, hi = grid[np.maximum(i - 1, 0)], grid[np.minimum(i, len(grid) - 1)]
    nearest = np.minimum(np.abs(a - lo), np.abs(hi - a))
    off = np.abs(np.abs(got) - a)
    assert np.isin(np.abs(got), grid).all()
    assert np.all(off <= nearest + 4 * rel * a + 2.0 ** -140)
    assert np.all((got == 0) | (np.sign(got) == np.sign(v)))


HS = [1, 2, 7, 8, 31, 33, 512, 513, 1078, 4096, 8192, 16384, 16392, 16385, 40002]


@pytest.mark.parametrize("res", [True, False], ids=["res", "nores"])
@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", HS)
def test_rows(H, dtype, out, res):
    g = torch.Generator(device="cuda").manual_seed(H)
    M = 6
    x = torch.randn(M, H, generator=g, device="cuda").to(DT[dtype][0])
    r = (3 * torch.randn(M, H, generator=g, device="cuda")).to(DT[dtype][0]) if res else None
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    x[0] = 0  # a row of zeros (with the residual: the residual alone)
    x[1] *= 1e-3
    y, c, s = run(x, r, w, out)
    check(x, r, w, out, y, c, s)


@pytest.mark.parametrize("M", [1, 3, 2304])
def test_row_counts(M):
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, 264, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.ones(264, dtype=torch.bfloat16, device="cuda")
    y, c, s = run(x, x, w, "e4m3")
    check(x, x, w, "e4m3", y, c, s)


@pytest.mark.parametrize("M,H", [(2500, 520), (5000, 1024), (700, 4096), (2304, 4096), (400, 8192), (170, 16384),
                                 (333, 9000)])
def test_more_rows_than_fit_at_once(M, H):
    """Rows that pass through a ring of shared memory, with and without a residual, the
    sum over the residual, rows that are not finite or zero among others."""
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, H + 8, generator=g, device="cuda").to(torch.bfloat16)[:, :H]
    r = (3 * torch.randn(M, H, generator=g, device="cuda")).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    x[7] = 0
    x[M - 2] = 0
    for out in ("e4m3", "bf16"):
        for res in (r, None):
            y, c, s = run(x, res, w, out)
            check(x, res, w, out, y, c, s)
    r2 = r.clone()
    y2 = torch.zeros(M, H, dtype=torch.uint8, device="cuda")
    c2 = torch.zeros(M, device="cuda")
    sb.sv_rmsnorm_residual(x, x.stride(0), r2, 0, w, 1e-5, r2, 0, sb.SV_BF16, y2, 0, sb.SV_E4M3, c2, M, H)
    y, c, s = run(x, r, w, "e4m3")
    assert torch.equal(r2, s) and torch.equal(c2, c) and torch.equal(y2, y.view(torch.uint8))
    x[11, 5] = float("nan")
    y, c, _ = run(x, r, w, "e4m3")
    assert torch.isnan(y.float()[11]).all() and torch.isnan(c[11])
    keep = torch.arange(M, device="cuda") != 11
    assert torch.equal(y.view(torch.uint8)[keep], y2[keep]) and torch.equal(c[keep], c2[keep])


@pytest.mark.parametrize("off", [0, 1, 2, 4])
def test_strides_and_alignment(off):
    """Rows inside wider buffers, from an odd start on: values outside the rows
    are neither read (NaN) nor written."""
    g = torch.Generator(device="cuda").manual_seed(5)
    M, H, ld = 5, 200, 231 if off == 1 else 232
    buf = torch.full((M, ld), float("nan"), device="cuda").to(torch.bfloat16)
    buf[:, off:off + H] = torch.randn(M, H, generator=g, device="cuda").to(torch.bfloat16)
    x = buf[:, off:off + H]
    w = torch.randn(H, generator=g, device="cuda").to(torch.bfloat16)
    for out in ("bf16", "e4m3"):
        y, c, s = run(x, x, w, out, ldo=ld)
        check(x, x, w, out, y, c, s)
        assert (f64(y)[:, H:] == 0).all()


def test_sum_over_its_inputs():
    """The stored sum over the residual, and over x (and without a residual):
    the results of the call with a buffer of its own.  H past what a thread
    keeps, so that rows are read again after part of the sum is stored."""
    g = torch.Generator(device="cuda").manual_seed(6)
    for H in (512, 20003):
        x = torch.randn(4, H, generator=g, device="cuda").to(torch.bfloat16)
        r = torch.randn(4, H, generator=g, device="cuda").to(torch.bfloat16)
        w = torch.randn(H, generator=g, device="cuda").to(torch.bfloat16)
        y, c, s = run(x, r, w, "e4m3")
        for over in ("residual", "x"):
            x2, r2 = x.clone(), r.clone()
            t = r2 if over == "residual" else x2
            y2 = torch.zeros(4, H, dtype=torch.uint8, device="cuda")
            c2 = torch.zeros(4, device="cuda")
            sb.sv_rmsnorm_residual(x2, 0, r2, 0, w, 1e-5, t, 0, sb.SV_BF16, y2, 0, sb.SV_E4M3, c2, 4, H)
            assert torch.equal(t, s) and torch.equal(c2, c)
            assert torch.equal(y2, y.view(torch.uint8))


def test_values_that_are_not_finite_stay_in_their_row():
    H = 96
    x = torch.randn(5, H, device="cuda")
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    x[3] = 0
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    y, c, _ = run(x, None, w, "e4m3")
    y = y.float()
    assert torch.isnan(c[1:3]).all() and torch.isnan(y[1:3]).all()
    assert torch.isfinite(c[[0, 3, 4]]).all() and torch.isfinite(y[[0, 3, 4]]).all()
    assert (y[3] == 0).all() and c[3].item() == 2.0 ** -126
    check(x[[0, 4]].contiguous(), None, w, "e4m3", y[[0, 4]], c[[0, 4]], None)
    w[3] = float("nan")  # a weight that is not finite reaches every row
    y, c, _ = run(x, None, w, "e4m3")
    assert torch.isnan(c).all() and torch.isnan(y.float()).all()


def test_largest_and_smallest_rows():
    """Rows near the ends of the type's range: an eps of zero, a row whose
    normalised values are tiny because its weight is."""
    H = 64
    x = torch.full((2, H), 1e18, device="cuda")
    x[1] = 1e-18
    w = torch.full((H,), 1.0, dtype=torch.bfloat16, device="cuda")
    y, c, _ = run(x, None, w, "bf16", eps=0.0)
    check(x, None, w, "bf16", y, c, None, eps=0.0)
    w[:] = 2.0 ** -124  # y / 448 is below the smallest scale
    y, c, _ = run(x, None, w, "e4m3", eps=0.0)
    assert (c == 2.0 ** -126).all()
    assert torch.allclose(y.float(), torch.full_like(x, 4.0))


def test_stream_and_graph():
    """On a stream of its own, and captured: replays follow the inputs."""
    x = torch.randn(9, 640, device="cuda").to(torch.bfloat16)
    w = torch.ones(640, dtype=torch.bfloat16, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y, c, s = run(x, x, w, "e4m3")
    st.synchronize()
    check(x, x, w, "e4m3", y, c, s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, c, s = run(x, x, w, "e4m3")
    for k in (1, 2):
        x.copy_(torch.randn(9, 640, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        check(x, x, w, "e4m3", y, c, s)


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [513, 519, 1001, 4097, 16377, 16379])
def test_odd_rows_in_place(H, dtype, out):
    """Rows that start at every place of an aligned run of eight, with a common stride, and
    with strides that differ (16379: one element more than the runs hold).  The sum goes
    over the residual; columns behind H, which the next row's run reaches into, and the
    rows' neighbours stay as they are."""
    g = torch.Generator(device="cuda").manual_seed(H)
    M = 19
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    for pads in [(0, 0, 0), (4, 12, 20), (1, 1, 9), (1, 2, 0)]:
        t, code = DT[dtype]
        x, r = (torch.randn(M, H + p, generator=g, device="cuda").to(t) for p in pads[:2])
        x0, r0 = x.clone(), r.clone()
        ldo = H + pads[2]
        y = torch.full((M, ldo), 77, dtype=torch.uint8, device="cuda") if out == "e4m3" else torch.full(
            (M, ldo), 77.0, dtype=torch.bfloat16, device="cuda")
        kept = y.clone()
        c = torch.empty(M, device="cuda") if out == "e4m3" else None
        sb.sv_rmsnorm_residual(x, H + pads[0], r, H + pads[1], w, 1e-5, r, H + pads[1], code, y, ldo, OUT[out][1],
                               c, M, H)
        assert torch.equal(x, x0)
        assert torch.equal(r[:, H:], r0[:, H:]) and torch.equal(y[:, H:], kept[:, H:])
        got = y.view(torch.float8_e4m3fn) if out == "e4m3" else y
        check(x0[:, :H], r0[:, :H], w, out, got, c, r[:, :H])
