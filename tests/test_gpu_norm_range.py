"""sv_rmsnorm_residual over the whole range of its types: rows whose squares leave float32's
range, rows that are almost zero with an eps of zero or next to it, in every form of the
kernel and among ordinary rows.  Tolerances are those of test_gpu_norm.py (the scaling by a
power of two is exact)."""

import numpy as np
import pytest

from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_norm import DT, _lib, check, run  # noqa: F401  (the fixture builds the library)

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]

# a warp's rows, a CTA's rows, odd ones in aligned runs and one by one, rows that are read
# again, and (with enough rows) the ring of copies
SHAPES = [(9, 64), (9, 510), (9, 1024), (9, 1001), (9, 16379), (9, 40002), (2500, 1032), (700, 4104)]
SIZES = [1e30, 3e38, 1e20, 1.0, 1e-15, 1e-20, 1e-25, 1e-37, 1e-40]


def rows(M, H, dtype, g):
    x = torch.randn(M, H, generator=g, device="cuda").clamp(-1, 1)
    size = torch.tensor(SIZES, device="cuda")[torch.arange(M, device="cuda") % len(SIZES)]
    return (x * size[:, None]).to(DT[dtype][0])


@pytest.mark.parametrize("out", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,H", SHAPES)
def test_rows_of_every_size(M, H, dtype, out):
    g = torch.Generator(device="cuda").manual_seed(H)
    x = rows(M, H, dtype, g)
    r = rows(M, H, dtype, g) * 0.125
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    keep = torch.arange(M, device="cuda") % len(SIZES) != 1  # (3e38 and a residual may overflow)
    for eps in (0.0, float(np.float32(1e-37)), float(np.float32(1e-30)), 1e-5):
        y, c, s = run(x, None, w, out, eps=eps)
        check(x, None, w, out, y, c, s, eps=eps)
        y, c, s = run(x, r, w, out, eps=eps)
        check(x[keep], r[keep], w, out, y[keep], None if c is None else c[keep], s[keep], eps=eps)


@pytest.mark.parametrize("big", [2.0 ** 127, 2.0 ** 64, 2.0 ** -70, 2.0 ** -126, 2.0 ** -140])
@pytest.mark.parametrize("H", [256, 8191])
def test_one_value_among_small_ones(H, big):
    """A row's largest value alone, and beside values that vanish against it."""
    x = torch.zeros(3, H, device="cuda")
    x[0, 7] = big
    x[1] = big * 2.0 ** -9
    x[1, 0] = -big
    x[2] = big
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    for out in ("bf16", "e4m3"):
        y, c, s = run(x, None, w, out, eps=0.0)
        check(x, None, w, out, y, c, s, eps=0.0)


def test_zeros_and_values_that_are_not_finite_among_them():
    x = torch.full((6, 96), 1e30, device="cuda")
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 5] = float("nan")
    x[4] = 1e-30
    w = torch.ones(96, dtype=torch.bfloat16, device="cuda")
    y, c, _ = run(x, None, w, "e4m3", eps=0.0)
    bad = torch.tensor([False, True, True, True, False, False], device="cuda")  # 0 / 0 is no number either
    y = y.float()
    assert torch.isnan(y[bad]).all() and torch.isnan(c[bad]).all()
    assert torch.allclose(c[~bad], torch.full((3,), 1 / 448, device="cuda"), rtol=1e-6) and (y[~bad] == 448).all()
    y, _, _ = run(x, None, w, "bf16", eps=0.0)
    assert torch.isnan(y[2, 5]) and (y[2, :5] == 0).all() and torch.isnan(y[3]).all() and torch.isnan(y[1]).all()
    assert (y[~bad].float() == 1).all()
    y, c, _ = run(x[1:2], None, w, "e4m3", eps=1e-30)
    assert (y.float() == 0).all() and c.item() == 2.0 ** -126


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,H", SHAPES)
def test_sums_over_the_residual(M, H, dtype):
    """A row that is done again still has its inputs."""
    g = torch.Generator(device="cuda").manual_seed(H + 1)
    x, r = rows(M, H, dtype, g) * 0.25, rows(M, H, dtype, g) * 0.25
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    y, c, s = run(x, r, w, "e4m3", eps=0.0)
    for over in (x.clone(), r.clone()):
        first = torch.equal(over, x)
        y2, c2 = torch.zeros(M, H, dtype=torch.uint8, device="cuda"), torch.zeros(M, device="cuda")
        sb.sv_rmsnorm_residual(over if first else x, 0, r if first else over, 0, w, 0.0, over, 0, DT[dtype][1], y2, 0,
                               sb.SV_E4M3, c2, M, H)
        assert torch.equal(over, s) and torch.equal(y2, y.view(torch.uint8))
        assert torch.equal(c2.isnan(), c.isnan()) and torch.equal(c2.nan_to_num(), c.nan_to_num())  # (0 / 0)


@pytest.mark.parametrize("M,H", [(1, 512), (1, 1500), (1, 1501), (1, 20001), (2500, 1504), (700, 4104)])
def test_quotients_next_to_a_border(M, H):
    """Rows of ones (their mean square is 1): y is the weight, so each 8-bit value is that of the
    weight divided by the scale.  All bf16 values over nine powers of two below each of 128
    largest ones: the quotients that lie between two e4m3 values are among them."""
    x = torch.ones(M, H, device="cuda").to(torch.bfloat16)
    steps = np.arange(1, 256, dtype=np.float32)
    for top in range(128, 256):
        v = np.unique(np.concatenate([steps * np.float32(2.0 ** -k) for k in range(9)]))
        v = np.concatenate([[top], v[v <= top]]).astype(np.float32)
        for at in range(0, len(v), H - 1):
            w = np.zeros(H, np.float32)
            w[0] = top
            n = len(v[at:at + H - 1])
            w[1:1 + n] = v[at:at + H - 1] * np.where(np.arange(n) % 2, 1, -1)
            y, c, _ = run(x, None, torch.from_numpy(w).cuda().to(torch.bfloat16), "e4m3", eps=0.0)
            scale = np.float32(top) / np.float32(448)  # (IEEE divisions: a GPU tensor over a number is a product)
            assert (c.cpu().numpy() == scale).all()
            want = torch.from_numpy(w / scale).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            assert torch.equal(y.view(torch.uint8), want.expand(M, H))
