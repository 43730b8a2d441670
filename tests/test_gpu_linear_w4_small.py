"""sv_linear_w4 on small values of x: whole rows down to bf16's smallest, values far below the largest of
their 128, and the same rows in calls of 8 and of 9."""

import numpy as np
import pytest

from oracle import draft4 as o4
from speculative_decoding_verification_47_gb300 import binding as sb
from tests.conftest import gpu_available
from tests.test_gpu_linear_w4 import BF, _lib, check, f64, inputs, run  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("power", [-133, -130, -126, -123, -118, -113, -111, -105, -98, -96, -60, 100])
def test_rows_of_every_size(power, group):
    """Rows whose values are about 2^power, scales that bring the sums near 1: with up to 8 rows every bf16 value
    of such a row is exact."""
    s = inputs(group - power, 7, 130, 256, group, True, False, False, torch.float32)
    s["x"] = (s["x"].double() * 2.0 ** power).to(BF)
    assert s["x"].any()
    s["scales"] = (s["scales"].double() * 2.0 ** min(-power, 120)).to(BF)
    check(s, run(s, 7, 130, 256, group, sb.SV_ACT_NONE, torch.float32), sb.SV_ACT_NONE, torch.float32, group)


@pytest.mark.parametrize("far", [20, 24, 25, 26, 27, 28, 29, 30, 32, 34, 36, 38])
@pytest.mark.parametrize("largest", [1.0, 1.9921875, 2.0 ** -90, 2.0 ** 100])
def test_values_far_below_their_largest(far, largest):
    """One large value a block, of weight 0, and small ones at every place of a word: kept down to 2^-28 of the largest,
    then off by at most 2^-36 of it each."""
    M, N, K, group = 5, 96, 512, 64
    s = inputs(far, M, N, K, group, False, False, False, torch.float32)
    small = torch.rand(M, K, generator=torch.Generator().manual_seed(far)).double() + 1
    x = small * largest * 2.0 ** -far
    at = torch.arange(0, K, 128) + torch.arange(K // 128) * 29 % 128
    x[:, at] = largest
    s["x"] = x.to(BF)
    W = torch.stack([s["W"] & 15, s["W"] >> 4], -1).reshape(N, K)
    W[:, at] = 8                                            # less 8: the large values count nothing
    s["W"] = W[:, 0::2] | W[:, 1::2] << 4
    got = f64(run(s, M, N, K, group, sb.SV_ACT_NONE, torch.float32))
    w = o4.weights(s["W"].numpy(), f64(s["scales"]), None, group)
    x = f64(s["x"])
    x[:, at] = 0
    ref, absp = x @ w.T, np.abs(x) @ np.abs(w).T
    lost = 2.0 ** -36 * largest * np.abs(w).sum(1) if far > 28 else 0
    assert np.all(np.abs(got - ref) <= 2.0 ** -15 * absp + lost)


@pytest.mark.parametrize("M", [3, 12])
def test_infinite_biases_before_the_activation(M):
    """What is not finite is z: an activation may take it back to a number, as its formula does."""
    s = inputs(M, M, 40, 64, 32, False, True, False, torch.float32)
    s["bias"][3], s["bias"][7] = float("-inf"), float("inf")
    z = run(s, M, 40, 64, 32, sb.SV_ACT_NONE, torch.float32).cpu()
    relu = run(s, M, 40, 64, 32, sb.SV_ACT_RELU, torch.float32).cpu()
    assert torch.all(z[:, 3] == float("-inf")) and torch.all(z[:, 7] == float("inf"))
    assert torch.all(relu[:, 3] == 0) and torch.all(relu[:, 7] == float("inf"))
    keep = torch.ones(40, dtype=torch.bool)
    keep[[3, 7]] = False
    assert torch.isfinite(z[:, keep]).all() and torch.equal(relu[:, keep], z[:, keep].clamp(min=0))


@pytest.mark.parametrize("N,K,group", [(300, 1024, 128), (130, 416, 32)])
def test_rows_of_eight_and_of_nine(N, K, group):
    """The same rows in calls of 8 and of 9 differ by their roundings: float32 sums of at most 128 terms on either side
    (2^-15 of the terms' absolute sum, as check() has it), and x below 2^-28 of its block's largest."""
    s = inputs(1, 9, N, K, group, True, True, True, torch.float32)
    r = torch.Generator().manual_seed(2)
    s["x"] = (s["x"].double() * 2.0 ** torch.randint(-40, 1, (9, K), generator=r).double()).to(BF)
    nine = f64(run(s, 9, N, K, group, sb.SV_ACT_NONE, torch.float32))
    few = dict(s, x=s["x"][:8], res=s["res"][:8])
    eight = f64(run(few, 8, N, K, group, sb.SV_ACT_NONE, torch.float32))
    w = np.abs(o4.weights(s["W"].numpy(), f64(s["scales"]), s["zeros"].numpy(), group))
    x = np.abs(f64(s["x"])[:8])
    largest = np.pad(x, ((0, 0), (0, -K % 128))).reshape(8, -1, 128).max(2).repeat(128, 1)[:, :K]
    lost = 2.0 ** -36 * largest @ w.T
    sums = x @ w.T + np.abs(f64(s["bias"])) + np.abs(f64(s["res"])[:8])
    assert np.all(np.abs(nine[:8] - eight) <= 2 * 2.0 ** -15 * sums + lost)
